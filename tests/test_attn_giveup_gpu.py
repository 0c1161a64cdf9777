"""GPU tests of attention calls whose waits run out (a limit of 1 ns): they
end, write nothing outside their outputs, and leave nothing behind."""
import pytest
import torch

from mla_attention_kv_gb300 import binding as B
from mla_attention_kv_gb300 import build as BLD

from test_attn_gpu import Paged, config

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
    assert a.status() in (0, 6) and a.status() == 0
    assert (out[small.T:] == 7.0).all() and (lse[small.T:] == 7.0).all()
    big.out.fill_(0)
    big.run(a)
    assert a.status() == 0
    big.check()
    b = B.MLAAttention(config(H, "fp16"), 700)
    small.run(b)
    assert b.status() == 0
    small.check()
