"""The e4m3 linear layer behind its own row quantisation.  The linear kernel
is launched while the quantisation still runs, so what that kernel writes may
only be read behind the wait for it and by coherent loads: ld.global.nc and
__ldg are defined for memory that nothing writes during a kernel."""
import os
import re

import pytest
import torch

from mla_attention_kv_gb300 import binding as B
from mla_attention_kv_gb300 import build as BLD

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_attention_kv_gb300", "csrc")
E4 = torch.float8_e4m3fn


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


@pytest.mark.parametrize("name", ["fp8_narrow.cu", "fp8_wide.cu"])
def test_row_scales_are_read_by_coherent_loads_behind_the_wait(name):
    text = source(name)
    loads = re.findall(r"(\w+)\(\s*xs\b", text)
    assert len(loads) >= 2 and set(loads) == {"ld_behind_dep"}
    assert text.count("p.x_scale") == 1  # (xs is the only way to them)
    body = text[:text.index("p.x_scale")]
    assert "grid_dep_wait()" in body[body.rindex("else"):]  # the epilogue's own wait
    asm = re.search(r"ld_behind_dep\(const float\* p\) \{(.*?)\n\}", source("common.cuh"), re.S).group(1)
    assert "asm volatile(\"ld.global.f32" in asm


@pytest.mark.gpu
@pytest.mark.parametrize("T,K,N", [(1, 2048, 576), (16, 7168, 2112), (64, 7168, 2112), (300, 1024, 9000), (700, 1536, 4096), (2000, 1040, 5000)])
@pytest.mark.parametrize("norm", [False, True])
def test_every_call_reads_its_own_scales(T, K, N, norm):
    """Rows whose scales differ by powers of two from call to call, without a wait between the calls: each result has the bits of
    a call on codes and scales that were complete before."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    BLD.build()
    B.load()
    g = torch.Generator(device="cuda").manual_seed(T + K)
    w = torch.randn(N, K, generator=g, device="cuda").mul_(60).clamp(-448, 448).to(E4)
    ws = 0.001 * (1 + torch.rand(-(-N // 128), -(-K // 128), generator=g, device="cuda"))
    gamma = (1 + 0.1 * torch.randn(K, generator=g, device="cuda")).to(torch.bfloat16)
    h = B.MLAFp8Linear(w, ws, "bf16", T)
    base = torch.randn(T, K, generator=g, device="cuda")
    xs, want = [], []
    for i in range(8):
        up = 2.0 ** torch.randint(-6, 7, (T, 1), generator=g, device="cuda").float()
        xs.append((base.roll(i, 0) * up).to(torch.bfloat16))
        q, s = torch.empty(T, K, device="cuda").to(E4), torch.empty(-(-K // 128), T, device="cuda")
        B.mla_fp8_quant_rows(xs[i], q, s, gamma=gamma if norm else None)
        torch.cuda.synchronize()
        want.append(torch.empty(T, N, dtype=torch.bfloat16, device="cuda"))
        h.run(want[i], x_q=q, x_scale=s)
        torch.cuda.synchronize()
    got = [torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(40)]
    for i, out in enumerate(got):
        h.run(out, x=xs[i % 8], gamma=gamma if norm else None)
    torch.cuda.synchronize()
    assert h.status() == 0
    for i, out in enumerate(got):
        assert torch.equal(out, want[i % 8]), i
    h.close()
