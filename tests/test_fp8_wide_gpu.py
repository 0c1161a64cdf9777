"""GPU tests of the e4m3 linear layer's kernel for many rows (fp8_wide.cu), at
sizes that test_fp8_rule.py shows to go there: every form of a call, against
the 64-bit evaluation and bound of test_fp8_linear_gpu.py, or bit for bit."""
import pytest
import torch

from mla_attention_kv_gb300 import binding as B
from mla_attention_kv_gb300 import build as BLD

from attn_ref import check
from test_fp8_linear_gpu import DT, E4, codes, gen, make, reference, run_given
from test_fp8_rows_gpu import quantise

pytestmark = pytest.mark.gpu

# T, K, N: one K block and less, K that ends inside a block, rows and columns that end inside a tile, token tiles in several groups
GIVEN = [(128, 16, 20000), (600, 16, 4104), (1500, 128, 4096), (640, 400, 6000), (517, 512, 4104), (1000, 1040, 4096), (257, 2112, 12000),
         (300, 1024, 9000), (8400, 128, 1000), (1157, 16384, 2000)]
OWN_ROWS = [(600, 16, 4104), (300, 1024, 9000), (1000, 1040, 4096), (700, 1536, 4096)]
RANDOM = [(300, 1024, 9000), (517, 512, 4104)]
ALTERNATE = (1536, 4096, [(700, "wide"), (1, "narrow"), (64, "narrow"), (650, "wide"), (300, "narrow"), (17, "narrow"), (700, "wide"), (513, "wide"), (128, "narrow")])
REPLAY = (600, 1040, 4104)
STREAMS = [(700, 2048, 4096), (300, 1024, 9000)]
LIMIT = (700, 2048, 4096)
SIZES = {s: "wide" for s in GIVEN + OWN_ROWS + RANDOM + STREAMS + [REPLAY, LIMIT]}
SIZES.update({(T, ALTERNATE[0], ALTERNATE[1]): which for T, which in ALTERNATE[2]})


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    BLD.build()
    B.load()


@pytest.mark.parametrize("T,K,N", GIVEN)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_given_codes(T, K, N, dtype):
    run_given(T, K, N, dtype, seed=T + K, pitch=32, opitch=16)


@pytest.mark.parametrize("T,K,N", RANDOM)
def test_every_code(T, K, N):
    run_given(T, K, N, "bf16", kind="random")


@pytest.mark.parametrize("T,K,N", OWN_ROWS)
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_rows_quantised_by_the_call(T, K, N, norm, dtype):
    """The same bits as quantising first; without a norm also the 64-bit reference of torch's own codes."""
    w, ws, _, _ = make(T, K, N, dtype)
    x = torch.randn(T, K + 40, generator=gen(T), device="cuda").to(DT[dtype])[:, 16:K + 16]
    gamma = (1 + 0.1 * torch.randn(K, generator=gen(K), device="cuda")).to(DT[dtype]) if norm else None
    h = B.MLAFp8Linear(w, ws, dtype, T + 3)
    out = torch.full((T, N + 8), 7.0, dtype=DT[dtype], device="cuda")
    h.run(out[:, :N], x=x, gamma=gamma, eps=1e-5)
    assert h.status() == 0 and h.last_launches == 2 and (out[:, N:] == 7.0).all()
    q, s = torch.empty(T, K, device="cuda").to(E4), torch.empty(-(-K // 128), T, device="cuda")
    B.mla_fp8_quant_rows(x, q, s, gamma=gamma, eps=1e-5)
    again = torch.empty(T, N, dtype=DT[dtype], device="cuda")
    h.run(again, x_q=q, x_scale=s)
    assert h.status() == 0 and torch.equal(out[:, :N], again)
    if not norm:
        rq, rs = quantise(x.float())
        ref, tol = reference(rq.to(E4), rs.t().contiguous(), w, ws, DT[dtype])
        check("out", out[:, :N], ref, tol)
    h.close()


@pytest.mark.parametrize("given", [False, True])
def test_both_kernels_on_one_handle(given):
    K, N, steps = ALTERNATE
    w, ws, xq, xs = make(700, K, N, "bf16")
    x = torch.randn(700, K, generator=gen(3), device="cuda").to(torch.bfloat16)
    h = B.MLAFp8Linear(w, ws, "bf16", 700)
    outs = [torch.empty(T, N, dtype=torch.bfloat16, device="cuda") for T, _ in steps]
    scales = [xs[:, :T].contiguous() for T, _ in steps]
    torch.cuda.synchronize()
    for (T, _), out, s in zip(steps, outs, scales):
        h.run(out, **(dict(x_q=xq[:T], x_scale=s) if given else dict(x=x[700 - T:])))
    assert h.status() == 0
    for (T, _), out, s in zip(steps, outs, scales):
        if given:
            ref, tol = reference(xq[:T], s, w, ws, torch.bfloat16)
        else:
            q, sc = quantise(x[700 - T:].float())
            ref, tol = reference(q.to(E4), sc.t().contiguous(), w, ws, torch.bfloat16)
        check(f"out {T}", out, ref, tol)
    h.close()


def test_captured_calls_follow_their_inputs():
    """Rows, weight and scales are read anew by every replay; results repeat bit for bit."""
    T, K, N = REPLAY
    w, ws, _, _ = make(T, K, N, "bf16")
    g = gen(4)
    x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
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
        x.copy_(torch.randn(T, K, generator=g, device="cuda"))
        ws.mul_(1.5)
        if i == 2:
            w.copy_(codes(g, N, K, "normal"))
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
    for i, (T, K, N) in enumerate(STREAMS):
        w, ws, _, _ = make(T, K, N, "bf16", seed=i)
        x = torch.randn(T, K, generator=gen(9 + i), device="cuda").to(torch.bfloat16)
        cs.append((B.MLAFp8Linear(w, ws, "bf16", T), x, torch.empty(T, N, dtype=torch.bfloat16, device="cuda"), torch.cuda.Stream(), w, ws))
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


def test_waits_that_run_out_and_waits_that_do_not():
    """A limit of 1 ns is overrun by a first wait: the call ends, reports it once and leaves nothing behind; one of 20 ms is
    not, also behind the call's own row quantisation."""
    T, K, N = LIMIT
    w, ws, _, _ = make(T, K, N, "fp16")
    x = torch.randn(T, K, generator=gen(5), device="cuda").half()
    buf = torch.full((T + 3, N + 16), 7.0, dtype=torch.float16, device="cuda")
    a = B.MLAFp8Linear(w, ws, "fp16", T, spin_budget_ns=1)
    for _ in range(2):
        a.run(buf[:T, :N], x=x)
        assert a.status() == 6 and a.status() == 0
    assert (buf[T:] == 7.0).all() and (buf[:, N:] == 7.0).all()
    b = B.MLAFp8Linear(w, ws, "fp16", T, spin_budget_ns=20_000_000)
    for _ in range(20):
        b.run(buf[:T, :N], x=x)
    assert b.status() == 0
    q, s = quantise(x.float())
    ref, tol = reference(q.to(E4), s.t().contiguous(), w, ws, torch.float16)
    check("out", buf[:T, :N], ref, tol)
    a.close()
    b.close()
