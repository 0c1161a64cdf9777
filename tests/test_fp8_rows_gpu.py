"""GPU tests of the e4m3 row quantisation.  Without a norm every step is one
IEEE fp32 operation, so codes and scales are compared bit for bit with the
same operations in torch; with a norm, with a 64-bit evaluation."""
import pytest
import torch

from mla_attention_kv_gb300 import binding as B
from mla_attention_kv_gb300 import build as BLD

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
E4 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    BLD.build()
    B.load()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def quantise(y):
    """Codes and scales [T, blocks] of fp32 (or fp64) rows, one IEEE operation a step."""
    T, K = y.shape
    b = torch.nn.functional.pad(y, (0, -K % 128)).view(T, -1, 128)
    m = b.abs().amax(-1)
    s = (m / torch.full_like(m, 448.0)).clamp(min=2.0 ** -126)  # (a tensor: torch multiplies by a number's reciprocal)
    q = (b * (1.0 / s)[..., None]).clamp(-448, 448)
    return q.reshape(T, -1)[:, :K], s


def outputs(T, K, pitch=None):
    q = torch.full((T, pitch or K), 5.0, device="cuda").to(E4)
    return q, q[:, :K], torch.full((-(-K // 128), T), 5.0, device="cuda")


@pytest.mark.parametrize("T,K", [(1, 16), (1, 128), (3, 144), (17, 512), (64, 576), (5, 2112), (33, 7168), (300, 1040), (2, 16384)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_rows_are_exact(T, K, dtype):
    x = (torch.randn(T, K + 24, generator=gen(T + K), device="cuda") * 3).to(DT[dtype])[:, 8:K + 8]  # strided rows
    x[:, ::7] *= 20
    buf, q, s = outputs(T, K, K + 32)
    B.mla_fp8_quant_rows(x, q, s)
    ref, rs = quantise(x.float())
    assert torch.equal(s, rs.t())
    assert torch.equal(q.float(), ref.to(E4).float())
    assert (buf[:, K:].float() == 5.0).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_special_rows(dtype):
    x = torch.zeros(6, 256, dtype=DT[dtype], device="cuda")
    x[1, 3] = 1e-30 if dtype == "bf16" else 6e-8       # a subnormal or tiny value alone in its block
    x[2, 130] = -torch.finfo(DT[dtype]).max
    x[2, 131] = torch.finfo(DT[dtype]).max / 448
    x[3, :128] = torch.finfo(DT[dtype]).smallest_normal
    if dtype == "bf16":
        x[4, 5] = 9.2e-41                               # below the range of 1 / (x / 448)
    x[5, 0], x[5, 1], x[5, 200] = float("nan"), 2.0, 1.0
    _, q, s = outputs(6, 256)
    B.mla_fp8_quant_rows(x, q, s)
    f = x.float()
    f[5, 0] = 0.0
    ref, rs = quantise(f)
    assert torch.equal(s, rs.t())
    got, ref = q.float(), ref.to(E4).float()
    assert torch.isnan(got[5, 0])
    got[5, 0] = 0.0
    assert torch.equal(got, ref)
    assert (s[:, 0] == 2.0 ** -126).all() and (got[0] == 0).all()
    assert got[1, 3] != 0 or dtype == "bf16" and 1e-30 * 2.0 ** 126 < 2.0 ** -10
    assert got[2, 130] == -448 and s[1, 2] > 0


@pytest.mark.parametrize("T,K", [(1, 16), (9, 512), (64, 1536), (7, 2048), (5, 2064), (3, 7168), (2, 8192), (2, 16384), (130, 576)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_norm_rows(T, K, dtype):
    """y = x / sqrt(mean x^2 + eps) * gamma in fp32: the sum of K squares, mean, root, division and two products are
    off by at most (K + 8) 2^-24 relatively (e below), the scale by that and two roundings more; a code by half a step of
    e4m3 (2^-4 relatively, 2^-10 in the subnormal range) of a quotient that is off by 2 e + 3 * 2^-24."""
    g = gen(T * K)
    x = torch.randn(T, K, generator=g, device="cuda").to(DT[dtype])
    gamma = (1 + 0.1 * torch.randn(K, generator=g, device="cuda")).to(DT[dtype])
    _, q, s = outputs(T, K)
    B.mla_fp8_quant_rows(x, q, s, gamma=gamma, eps=1e-5)
    d = x.double()
    y = d / torch.sqrt(d.pow(2).mean(1, keepdim=True) + 1e-5) * gamma.double()
    ref, rs = quantise(y)
    e = (K + 8) * 2.0 ** -24
    assert ((s.t().double() - rs).abs() <= (e + 2.0 ** -23) * rs).all()
    tol = (2.0 ** -4 * ref.abs()).clamp(min=2.0 ** -10) + (2 * e + 3 * 2.0 ** -24) * ref.abs()
    assert ((q.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("T,K", [(1025, 512), (1500, 976), (1030, 1536), (1025, 2048), (2000, 16)])
def test_norm_many_rows(T, K):
    test_norm_rows(T, K, "bf16")


def test_many_rows_and_another_stream():
    x = torch.randn(20000, 384, generator=gen(1), device="cuda").to(torch.bfloat16)
    _, q, s = outputs(20000, 384)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    B.mla_fp8_quant_rows(x, q, s, stream=st)
    st.synchronize()
    ref, rs = quantise(x.float())
    assert torch.equal(s, rs.t()) and torch.equal(q.float(), ref.to(E4).float())


def test_more_rows_than_a_grid_has_in_its_second_dimension():
    T, K = 65535 * 16 + 21, 32
    x = torch.randn(T, K, generator=gen(2), device="cuda").to(torch.bfloat16)
    _, q, s = outputs(T, K)
    B.mla_fp8_quant_rows(x, q, s)
    ref, rs = quantise(x.float())
    assert torch.equal(s, rs.t()) and torch.equal(q.float(), ref.to(E4).float())


def test_no_rows():
    B.mla_fp8_quant_rows(torch.empty(0, 128, dtype=torch.float16, device="cuda"), torch.empty(0, 128, device="cuda").to(E4),
                         torch.empty(1, 0, device="cuda"))


def test_binding_checks():
    x = torch.zeros(2, 256, dtype=torch.float16, device="cuda")
    _, q, s = outputs(2, 256)
    for bad in (dict(q=q[:, :128]), dict(scale=s[:1]), dict(scale=s.t()), dict(q=q.float()), dict(scale=s.half()),
                dict(gamma=torch.ones(128, dtype=torch.float16, device="cuda")), dict(gamma=torch.ones(256, device="cuda")),
                dict(x=x[:, ::2]), dict(x=x[0])):
        with pytest.raises((ValueError, TypeError)):
            B.mla_fp8_quant_rows(**{**dict(x=x, q=q, scale=s), **bad})
    with pytest.raises(B.MLAError):
        B.mla_fp8_quant_rows(x[:, :24].contiguous(), torch.zeros(2, 24, device="cuda").to(E4), torch.zeros(1, 2, device="cuda"))
