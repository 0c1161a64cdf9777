"""GPU tests of e4m3 linear layers whose waits run out (a limit of 1 ns, which
the MMA warp's first wait always overruns): the calls end, write nothing
outside their outputs, report it once and leave nothing behind."""
import pytest
import torch

from mla_attention_kv_gb300 import binding as B
from mla_attention_kv_gb300 import build as BLD

from attn_ref import check
from test_fp8_linear_gpu import make, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    BLD.build()
    B.load()


@pytest.mark.parametrize("T,K,N", [(1, 128, 128), (5, 7168, 2112), (64, 7168, 2112), (200, 2048, 576), (600, 1536, 4096), (3000, 512, 4096)])
def test_limit_is_kept_and_reported(T, K, N):
    w, ws, xq, xs = make(T, K, N, "bf16")
    buf = torch.full((T + 3, N + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:T, :N]
    a = B.MLAFp8Linear(w, ws, "bf16", T, spin_budget_ns=1)
    for _ in range(2):
        a.run(out, x_q=xq, x_scale=xs)
        assert a.status() == 6 and a.status() == 0
    assert (buf[T:] == 7.0).all() and (buf[:, N:] == 7.0).all()
    b = B.MLAFp8Linear(w, ws, "bf16", T)
    b.run(out, x_q=xq, x_scale=xs)
    assert b.status() == 0
    ref, tol = reference(xq, xs, w, ws, torch.bfloat16)
    check("out", out, ref, tol)
    a.close()
    b.close()


def test_a_limit_of_milliseconds_is_not_run_out_by_ordinary_waits():
    """20 ms, also behind the call's own row quantisation."""
    for T in (40, 700):
        w, ws, _, _ = make(T, 2048, 1024, "fp16")
        x = torch.randn(T, 2048, device="cuda").half()
        out = torch.empty(T, 1024, dtype=torch.float16, device="cuda")
        h = B.MLAFp8Linear(w, ws, "fp16", T, spin_budget_ns=20_000_000)
        for _ in range(20):
            h.run(out, x=x)
        assert h.status() == 0
        h.close()
