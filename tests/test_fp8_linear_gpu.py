"""GPU tests of the e4m3 linear layer against a 64-bit evaluation.

Bound: with a = sum_b xs ws sum_k |xq wq|, the sum of a block's K products
by the tensor core (products of e4m3 values are exact; every add is off by
at most f = 2^-23 of the sum so far, whether it rounds or truncates) is off
by 128 f relative to its part of a; the product of the two scales, the
scaling and the running sum over B blocks add (B + 4) f of a; splitting the
blocks over 8 CTAs 8 f more.  The result's rounding adds u = eps / 2 of |out|,
and 2^-25 below fp16's normal range."""
import pytest
import torch

from mla_attention_kv_gb300 import binding as B
from mla_attention_kv_gb300 import build as BLD

from attn_ref import check
from test_fp8_rows_gpu import quantise

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
E4 = torch.float8_e4m3fn
F = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    BLD.build()
    B.load()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def codes(g, rows, cols, kind="random"):
    if kind == "random":  # every finite code (0x7f and 0xff are NaN)
        c = torch.randint(0, 254, (rows, cols), generator=g, device="cuda", dtype=torch.int32)
        return (c + (c > 126).int()).to(torch.uint8).view(E4)
    return torch.randn(rows, cols, generator=g, device="cuda").mul_(60).clamp(-448, 448).to(E4)


def reference(xq, xs, w, ws, dtype):
    """out and its bound; xs [blocks, T]."""
    T, K = xq.shape
    out = torch.zeros(T, w.shape[0], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    for b in range(-(-K // 128)):
        k = slice(b * 128, min(K, b * 128 + 128))
        x = xq[:, k].double() * xs[b].double()[:, None]
        y = w[:, k].double() * ws[:, b].double().repeat_interleave(128)[:w.shape[0], None]
        out += x @ y.t()
        mag += x.abs() @ y.abs().t()
    tol = (128 + -(-K // 128) + 12) * F * mag + torch.finfo(dtype).eps / 2 * 1.01 * out.abs()
    return out, tol + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def make(T, K, N, dtype, seed=1, kind="normal", pitch=0):
    g = gen(seed)
    w = codes(g, N, K, kind)
    ws = 2.0 ** torch.randint(-12, -7, (-(-N // 128), -(-K // 128)), generator=g, device="cuda").float()
    ws = ws * (1 + torch.rand(ws.shape, generator=g, device="cuda"))
    xq = codes(g, T, K + pitch, kind)[:, :K]
    xs = (0.5 + torch.rand(-(-K // 128), T, generator=g, device="cuda")) / 448
    return w, ws, xq, xs


def run_given(T, K, N, dtype, seed=1, kind="normal", pitch=0, opitch=0):
    w, ws, xq, xs = make(T, K, N, dtype, seed, kind, pitch)
    buf = torch.full((T, N + opitch), 7.0, dtype=DT[dtype], device="cuda")
    h = B.MLAFp8Linear(w, ws, dtype, T)
    h.run(buf[:, :N], x_q=xq, x_scale=xs)
    assert h.status() == 0 and h.last_launches == 1
    out, tol = reference(xq, xs, w, ws, DT[dtype])
    check("out", buf[:, :N], out, tol)
    assert (buf[:, N:] == 7.0).all()
    h.close()
    return buf[:, :N]


SIZES = [(1, 16, 8), (1, 128, 128), (1, 2048, 576), (2, 144, 136), (15, 512, 4096), (16, 7168, 2112), (17, 2112, 40), (31, 1040, 264),
         (33, 640, 1000), (64, 7168, 576), (65, 384, 520), (127, 1536, 384), (128, 2048, 2048), (3, 16384, 128)]
WIDE = [(129, 128, 8), (130, 144, 264), (255, 512, 256), (256, 256, 512), (257, 1040, 136), (517, 512, 4096), (700, 7168, 576), (1061, 2048, 2112)]


@pytest.mark.parametrize("T,K,N", SIZES)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_few_rows(T, K, N, dtype):
    run_given(T, K, N, dtype, seed=T + K, pitch=32, opitch=16)


@pytest.mark.parametrize("T,K,N", WIDE)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_many_rows(T, K, N, dtype):
    run_given(T, K, N, dtype, seed=T + K, pitch=32, opitch=16)


@pytest.mark.parametrize("T,K,N", [(8, 512, 256), (300, 512, 256)])
def test_every_code(T, K, N):
    run_given(T, K, N, "bf16", kind="random")


@pytest.mark.parametrize("T,N", [(4, 20000), (100, 40000), (2000, 5000), (4096, 3000)])
def test_more_tiles_than_sms(T, N):
    run_given(T, 256, N, "bf16", seed=N)


@pytest.mark.parametrize("T,K,N", [(1, 512, 256), (64, 2048, 576), (100, 1040, 264), (700, 1536, 1000)])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_rows_quantised_by_the_call(T, K, N, norm, dtype):
    """The same bits as quantising first; without a norm also the 64-bit reference of torch's own codes."""
    g = gen(T)
    w, ws, _, _ = make(T, K, N, dtype)
    x = torch.randn(T, K + 40, generator=g, device="cuda").to(DT[dtype])[:, 16:K + 16]
    gamma = (1 + 0.1 * torch.randn(K, generator=g, device="cuda")).to(DT[dtype]) if norm else None
    h = B.MLAFp8Linear(w, ws, dtype, T + 3)
    out = torch.full((T, N), 7.0, dtype=DT[dtype], device="cuda")
    h.run(out, x=x, gamma=gamma, eps=1e-5)
    assert h.status() == 0 and h.last_launches == 2
    q, s = torch.empty(T, K, device="cuda").to(E4), torch.empty(-(-K // 128), T, device="cuda")
    B.mla_fp8_quant_rows(x, q, s, gamma=gamma, eps=1e-5)
    again = torch.empty_like(out)
    h.run(again, x_q=q, x_scale=s)
    assert h.status() == 0 and torch.equal(out, again)
    if not norm:
        rq, rs = quantise(x.float())
        ref, tol = reference(rq.to(E4), rs.t().contiguous(), w, ws, DT[dtype])
        check("out", out, ref, tol)
    h.close()


def test_sizes_alternate_on_one_handle():
    w, ws, xq, xs = make(600, 1536, 1000, "bf16")
    h = B.MLAFp8Linear(w, ws, "bf16", 600)
    for T in (600, 1, 64, 300, 17, 600, 128, 129):
        out = torch.empty(T, 1000, dtype=torch.bfloat16, device="cuda")
        s = xs[:, :T].contiguous()
        h.run(out, x_q=xq[:T], x_scale=s)
        ref, tol = reference(xq[:T], s, w, ws, torch.bfloat16)
        check(f"out {T}", out, ref, tol)
    assert h.status() == 0
    h.close()


@pytest.mark.parametrize("T", [5, 300])
def test_captured_calls_follow_their_inputs(T):
    """Rows, weight and scales are read anew by every replay; results repeat bit for bit."""
    w, ws, _, _ = make(T, 1024, 520, "bf16")
    g = gen(4)
    x = torch.randn(T, 1024, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty(T, 520, dtype=torch.bfloat16, device="cuda")
    h = B.MLAFp8Linear(w, ws, "bf16", T)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        h.run(out, x=x)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.run(out, x=x)
    for i in range(3):
        x.copy_(torch.randn(T, 1024, generator=g, device="cuda"))
        ws.mul_(1.5)
        if i == 2:
            w.copy_(codes(g, 520, 1024, "normal"))
        graph.replay()
        first = out.clone()
        q, s = quantise(x.float())
        ref, tol = reference(q.to(E4), s.t().contiguous(), w, ws, torch.bfloat16)
        check("out", out, ref, tol)
        graph.replay()
        assert torch.equal(out, first)
    assert h.status() == 0
    h.close()


def test_two_handles_on_two_streams():
    cs = []
    for i, T in enumerate((40, 400)):
        w, ws, _, _ = make(T, 2048, 1024, "bf16", seed=i)
        x = torch.randn(T, 2048, generator=gen(9 + i), device="cuda").to(torch.bfloat16)
        cs.append((B.MLAFp8Linear(w, ws, "bf16", T), x, torch.empty(T, 1024, dtype=torch.bfloat16, device="cuda"), torch.cuda.Stream(), w, ws))
    torch.cuda.synchronize()
    for _ in range(20):
        for h, x, out, s, _, _ in cs:
            h.run(out, x=x, stream=s)
    torch.cuda.synchronize()
    for h, x, out, s, w, ws in cs:
        assert h.status() == 0
        q, sc = quantise(x.float())
        ref, tol = reference(q.to(E4), sc.t().contiguous(), w, ws, torch.bfloat16)
        check("out", out, ref, tol)
        h.close()


def test_no_rows_and_refusals():
    w, ws, xq, xs = make(4, 256, 264, "bf16")
    h = B.MLAFp8Linear(w, ws, "bf16", 4)
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(4, 264, dtype=torch.bfloat16, device="cuda")
    h.run(out[:0], x=x[:0])
    assert h.last_launches == 0
    for bad in (dict(), dict(x=x, x_q=xq, x_scale=xs), dict(x_q=xq), dict(x_q=xq, x_scale=xs, gamma=x[0]), dict(x=x.half()), dict(x=x[:, :128]),
                dict(x=x, gamma=x[0, :128]), dict(x_q=xq, x_scale=xs.t()), dict(x_q=xq, x_scale=xs[:1]), dict(x=x[:3])):
        with pytest.raises((ValueError, TypeError)):
            h.run(out, **bad)
    for o in (out[:, :256], out.half(), out.t()):
        with pytest.raises((ValueError, TypeError)):
            h.run(o, x=x)
    big = torch.zeros(5, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(B.MLAError):
        h.run(torch.zeros(5, 264, dtype=torch.bfloat16, device="cuda"), x=big)
    for a, b in ((w.float(), ws), (w, ws[:1]), (w, ws.double()), (w.cpu(), ws.cpu()), (w[0], ws)):
        with pytest.raises((ValueError, TypeError)):
            B.MLAFp8Linear(a, b, "bf16", 4)
    with pytest.raises(B.MLAError):
        B.MLAFp8Linear(w[:, :24].contiguous(), ws[:, :1].contiguous(), "bf16", 4)
    assert h.status() == 0
    h.close()
