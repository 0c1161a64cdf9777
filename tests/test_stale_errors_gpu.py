"""A failed call does not make a later one fail: an error that has been
reported is taken from the CUDA runtime, which would otherwise hand it to the
next launch that asks."""
import pytest
import torch

from mla_attention_kv_gb300 import binding as B
from mla_attention_kv_gb300 import build as BLD
from mla_attention_kv_gb300 import inputs as I

from test_paged_kv_gpu import Case, config

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    BLD.build()
    B.load()


def no_linear():
    """A workspace of 35 TB."""
    w = torch.zeros(128, 16384, device="cuda").to(E4)
    with pytest.raises(B.MLAError) as e:
        B.MLAFp8Linear(w, torch.ones(1, 128, device="cuda"), "bf16", (1 << 31) - 65536)
    assert "MLA_ERR_NO_MEMORY" in str(e.value)


def no_prolog():
    """A workspace of 2 TB and more."""
    with pytest.raises(B.MLAError) as e:
        B.MLAProlog(I.R1_W8A8, 1 << 27)
    assert "MLA_ERR_NO_MEMORY" in str(e.value)


def rows():
    x = torch.randn(5, 256, device="cuda").half()
    q, s = torch.empty(5, 256, device="cuda").to(E4), torch.empty(2, 5, device="cuda")
    B.mla_fp8_quant_rows(x, q, s)


def attention():
    c = Case([1], [40], 4, 4, 16, "fp16")
    a = B.MLAAttention(config(4), 4)
    c.run(a)
    assert a.status() == 0
    c.check()
    a.close()


@pytest.mark.parametrize("call", [rows, attention])
@pytest.mark.parametrize("failure", [no_linear, no_prolog])
def test_calls_after_a_failed_create(failure, call):
    call()
    failure()
    call()
    torch.cuda.synchronize()


def test_status_after_a_failed_create():
    w = torch.zeros(128, 256, device="cuda").to(E4)
    h = B.MLAFp8Linear(w, torch.ones(1, 2, device="cuda"), "bf16", 4)
    no_linear()
    assert h.status() == 0
    h.close()
