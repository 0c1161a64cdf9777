"""int8 caches whose codes use little of their range (channels whose static
scale is wide for most tokens): the scores are as exact relative to the
products in them as with codes of full scale.  The bound is attn_ref.py's,
(192 + 16) 2^-23 of sum |q k| per score, whatever the codes are; the log-sum-exp
of a few keys shows the scores without a rounding to 16 bits."""
import pytest
import torch

from mla_attention_kv_gb300 import binding as B
from mla_attention_kv_gb300 import build as BLD

from test_paged_kv_gpu import Case, config, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    BLD.build()
    B.load()


class Small(Case):
    """Keys with codes in -spread .. spread, whose scales make up for them (0: one code in 24 is 1 or -1); queries of one
    sign, or of both."""

    def __init__(self, spread, one_sign, *args, **kw):
        super().__init__(*args, i8=True, **kw)
        g = gen(spread + 100)
        for s in ("k", "kpe"):
            self.scales[s] = self.scales[s] * (64.0 / max(1, spread))
        if one_sign:
            self.qn, self.qp = self.qn.abs(), self.qp.abs()
        self.keys = []
        for i, ln in enumerate(self.L):
            r = torch.arange(ln, device="cuda")
            blk, off = self.table[i].long()[r // self.k.shape[2]], r % self.k.shape[2]

            def fill(cache, width):
                most = max(1, spread)
                x = torch.randint(-most, most + 1, (ln, cache.shape[1], width), generator=g, device="cuda").to(torch.int8)
                if spread == 0:
                    x *= torch.rand(x.shape, generator=g, device="cuda") < 1 / 16
                cache[blk, :, off] = x
                return x.double()

            k = fill(self.k, 128) * self.scales["k"].double().view(self.KH, 128)
            e = fill(self.e, 64) * self.scales["kpe"].double()
            self.keys.append(torch.cat((k, e.expand(ln, self.KH, 64)), dim=-1).transpose(0, 1))


@pytest.mark.parametrize("one_sign", [False, True])
@pytest.mark.parametrize("spread", [0, 1, 3, 64])
@pytest.mark.parametrize("H,KH,n", [(4, 4, 1), (8, 2, 1), (16, 2, 1), (6, 3, 5)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_small_codes(H, KH, n, spread, one_sign, dtype):
    L = [1, 2, 5, 33, 64, 300] if n == 1 else [5, 6, 40, 300]
    c = Small(spread, one_sign, [n] * len(L), L, H, KH, 16 if H == 4 else 13, dtype, seed=H + spread)
    a = B.MLAAttention(config(H, dtype), c.T, num_kv_heads=KH)
    c.run(a)
    assert a.status() == 0
    c.check()
    a.close()
