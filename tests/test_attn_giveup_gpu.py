"""GPU tests of attention calls whose waits run out (a limit of 1 ns): they
end, write nothing outside their outputs, and leave nothing behind."""
import pytest
import torch

from mla_attention_kv_gb300 import binding as B
from mla_attention_kv_gb300 import build as BLD

from attn_ref import attend, check
from test_attn_gpu import SCALE, Paged, config, gen, rnd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    BLD.build()
    B.load()


@pytest.mark.parametrize("page", [16, 32])
def test_a_call_that_gives_up_writes_only_its_output(page):
    """A larger call of the same handle (16-row items: no waits that could run out) leaves records of rows up to 2763 for
    the pair kernel's 76 workers; then a call of 2400 rows whose workers' ranges reach over the ends of its items, with
    out and lse the first part of larger tensors."""
    H = 16
    big = Paged([1] * 700, [(37 * i) % 90 for i in range(700)], H, 16, "fp16", 9)
    small = Paged([3] * 50, [70 + i % 40 for i in range(50)], H, page, "fp16", 10)
    out = torch.full((700, H, 512), 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((700, H), 7.0, dtype=torch.float32, device="cuda")
    small.out, small.lse = out[:small.T], lse[:small.T]
    a = B.MLAAttention(config(H, "fp16"), 700, spin_budget_ns=1)
    big.run(a)
    assert a.status() == 0
    small.run(a)
    assert a.status() == 6 and a.status() == 0
    assert (out[small.T:] == 7.0).all() and (lse[small.T:] == 7.0).all()
    big.out.fill_(0)
    big.run(a)
    assert a.status() == 0
    big.check()
    b = B.MLAAttention(config(H, "fp16"), 700)
    small.run(b)
    assert b.status() == 0
    small.check()


@pytest.mark.parametrize("H,page", [(128, 16), (128, 64), (48, 32)])
@pytest.mark.parametrize("n", [1, 40])
def test_paged_limit_is_kept_and_reported(H, page, n):
    """A limit of 1 ns runs out in every call of the pair kernel (the MMA thread has to wait for the queries at least),
    the status says so once, and a handle with the usual limit is right afterwards."""
    c = Paged([n] * 8, [3000, 70, 500, 40, 41, 999, 64, 1280], H, page, "bf16", 21)
    a = B.MLAAttention(config(H, "bf16"), c.T, spin_budget_ns=1)
    for _ in range(2):
        c.run(a)
        assert a.status() == 6 and a.status() == 0
    b = B.MLAAttention(config(H, "bf16"), c.T)
    c.run(b)
    assert b.status() == 0
    c.check()


def test_prompt_limit_is_kept_and_reported():
    g = gen(1)
    x, p = rnd(g, 1, 4, 900, 128, dtype=torch.bfloat16), rnd(g, 1, 4, 900, 64, dtype=torch.bfloat16)
    q, v = rnd(g, 1, 4, 900, 128, dtype=torch.bfloat16), rnd(g, 1, 4, 900, 128, dtype=torch.bfloat16)
    guard = torch.full((1, 4, 1200, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out = guard[:, :, :900]
    a = B.MLAAttention(config(4, "bf16"), 900, spin_budget_ns=1)
    for causal in (True, False):
        a.run_prompt(q, p, x, p[:, :1], v, out, causal=causal)
        assert a.status() == 6 and a.status() == 0
    b = B.MLAAttention(config(4, "bf16"), 900)
    b.run_prompt(q, p, x, p[:, :1], v, out)
    assert b.status() == 0
    assert (guard[:, :, 900:] == 7.0).all()
    k = torch.cat((x, p[:, :1].expand(1, 4, 900, 64)), -1)[0].double()
    qq = torch.cat((q, p), -1)[0].double().transpose(0, 1)
    ref, _, tol, _ = attend(qq, k, v[0].double(), 0, SCALE, torch.bfloat16)
    check("out", out[0].transpose(0, 1), ref, tol)


def test_status_reads_one_stream_and_loses_nothing():
    """The status call waits for its own stream alone, and clears what it reads before it returns: every bad slot of a
    side stream is reported once, while the default stream is busy."""
    a = B.MLAAttention(config(2, "fp16"), 1)
    kv = torch.randn(1, 576, device="cuda").half()
    c = a.alloc_latent_caches(1, 4)
    bad = torch.tensor([4], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a.append_latent(kv[:, :512], kv[:, 512:], None, None, None, None, bad, **c, stream=side)
    assert a.status(side) == 10  # (kernels are loaded)
    torch.cuda._sleep(2_000_000_000)  # about a second
    busy = torch.cuda.Event()
    busy.record()
    for _ in range(50):
        a.append_latent(kv[:, :512], kv[:, 512:], None, None, None, None, bad, **c, stream=side)
        assert a.status(side) == 10
    assert a.status(side) == 0
    assert not busy.query()
    torch.cuda.synchronize()


def test_a_limit_of_milliseconds_is_not_run_out_by_ordinary_waits():
    """20 ms: far over any wait of a call of a few hundred microseconds, far under the default."""
    c = Paged([1] * 8, [3000, 70, 500, 40, 41, 999, 64, 1280], 128, 64, "bf16", 22)
    a = B.MLAAttention(config(128, "bf16"), c.T, spin_budget_ns=20_000_000)
    c.run(a)
    assert a.status() == 0
    c.check()


def test_appends_and_prompts_of_one_handle_overlap():
    """They use only the status word of the workspace, so calls of one handle may run on several streams at once."""
    g = gen(8)
    bf = torch.bfloat16
    a = B.MLAAttention(config(4, "bf16"), 900)
    ins = [[rnd(g, 1, h, 900, d, dtype=bf) for h, d in ((4, 128), (4, 64), (4, 128), (1, 64), (4, 128))] for _ in range(3)]
    outs = [torch.zeros_like(x[0]) for x in ins]
    want = []
    for x in ins:
        o = torch.zeros_like(x[0])
        a.run_prompt(*x, o)
        want.append(o)
    kv = rnd(g, 900, 576, dtype=bf)
    slots = torch.randperm(912, generator=g, device="cuda")[:900].to(torch.int32)
    caches = [a.alloc_latent_caches(57, 16) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, x, o, c in zip(streams, ins, outs, caches):
            a.run_prompt(*x, o, stream=s)
            a.append_latent(kv[:, :512], kv[:, 512:], None, None, None, None, slots, **c, stream=s)
    torch.cuda.synchronize()
    assert a.status() == 0
    for o, w, c in zip(outs, want, caches):
        assert torch.equal(o, w)
        assert torch.equal(c["latent_cache"].view(-1, 512)[slots.long()], kv[:, :512])
        assert torch.equal(c["kpe_cache"].view(-1, 64)[slots.long()], kv[:, 512:])
