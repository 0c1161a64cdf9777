"""The int8 cache from end to end: a prompt's codes as the prolog writes them
(mla_kv_prolog_run_c8) read by the paged K/V attention as a cache of one page
per sequence, then decode steps whose codes the caller puts behind them.
Bounds of attn_ref.py and test_paged_kv_gpu.py on the codes and scales."""
import math

import pytest
import torch

from mla_attention_kv_gb300 import binding as B
from mla_attention_kv_gb300 import build as BLD
from mla_attention_kv_gb300 import inputs as I

from attn_ref import attend, check
from test_c8_gpu import make_scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    BLD.build()
    B.load()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("s", [1, 37, 64])
def test_prompt_and_decode_over_int8_codes(dtype, s):
    b, H, page, steps = 3, 8, 80, 4
    cfg = I.small_config(I.V2_LITE, num_heads=H, hidden=1024, dtype=dtype, max_pos=256)
    dt = I.torch_dtype(cfg)
    w = B.to_device({k: v for k, v in I.kv_inputs(cfg, 1, 2, 5, "prefill").items() if k not in ("hidden", "positions")})
    sc = {k: torch.tensor(v, device="cuda") for k, v in make_scales(cfg, 7).items()}
    g = torch.Generator(device="cuda").manual_seed(s)
    prolog, attn = B.MLAProlog(cfg, b * s), B.MLAAttention(cfg, b * s)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(dt)  # noqa: E731
    i32 = dict(dtype=torch.int32, device="cuda")

    def codes(n, at):
        out = prolog.alloc_c8_outputs(b, n)
        pos = (at + torch.arange(n, **i32)).repeat(b).contiguous()
        prolog.run_c8(b, n, dict(w, hidden=rand(b * n, 1024), positions=pos), sc, out)
        return out["k_nope"], out["value"], out["k_pe"]

    def attend_and_check(cache, n, L, table):
        q = rand(b * n, H, 192)
        out, lse = torch.empty(b * n, H, 128, dtype=dt, device="cuda"), torch.empty(b * n, H, device="cuda")
        attn.run_paged_kv(q[..., :128], q[..., 128:], torch.full((b,), L, **i32), table, *cache, out, lse=lse, scales=sc)
        assert attn.status() == 0 and prolog.status() == 0
        for i in range(b):
            blk = int(table[i, 0])
            k, v, e = (x[blk, :, :L].double() for x in cache)
            assert k.abs().amax() > 0
            k, v, e = k * sc["k"].double().view(H, 1, 128), v * sc["v"].double().view(H, 1, 128), e * sc["kpe"].double()
            ref, rl, tol, ltol = attend(q[i * n:i * n + n].double(), torch.cat((k, e.expand(H, L, 64)), -1), v, L - n, 1 / math.sqrt(192), dt)
            tol = tol + 2.0 ** -25 * v.abs().sum(1)[None] + 2.0 ** -23 * ref.abs()
            check(f"out[{i}]", out[i * n:i * n + n], ref, tol)
            check(f"lse[{i}]", lse[i * n:i * n + n], rl, ltol)

    # the prompt, every token's attention over the codes as they were written
    prompt = codes(s, 0)
    attend_and_check(prompt, s, s, torch.arange(b, **i32)[:, None].contiguous())
    # decode steps behind it, blocks in another order
    order = torch.tensor([2, 0, 1], **i32)
    cache = [torch.full((b, x.shape[1], page, x.shape[3]), -128, dtype=torch.int8, device="cuda") for x in prompt]
    for x, c in zip(prompt, cache):
        c[order.long(), :, :s] = x
    for step in range(steps):
        for x, c in zip(codes(1, s + step), cache):
            c[order.long(), :, s + step] = x[:, :, 0]
        attend_and_check(cache, 1, s + step + 1, order[:, None].contiguous())
    prolog.close()
    attn.close()
