"""GPU tests of the paged attention's 32-row items (17 to 32 query rows per
sequence) in both types: short and around tile ends, long enough to be split,
many sequences, chunks of grouped tokens, strided layouts."""
import pytest
import torch

from mla_attention_kv_gb300 import binding as B
from mla_attention_kv_gb300 import build as BLD

from test_attn_gpu import Paged, config, paged_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    BLD.build()
    B.load()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("H,n", [(17, 1), (24, 1), (32, 1), (16, 2), (10, 3), (1, 32)])
def test_lengths(H, n, dtype):
    L = [0, 1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300]
    paged_case([n] * len(L), L, H, 16, dtype, seed=H + n)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("H,n,L,page", [(32, 1, 5000, 64), (32, 1, 20011, 16), (16, 2, 9001, 7), (24, 1, 4097, 1)])
def test_long_context_is_split(H, n, L, page, dtype):
    paged_case([n], [L], H, page, dtype, seed=L)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_mixed_and_many(dtype):
    paged_case([1, 1, 1, 1], [7000, 3, 900, 2500], 32, 32, dtype, seed=3)
    paged_case([1] * 500, [(53 * i) % 131 for i in range(500)], 32, 16, dtype, seed=4)


@pytest.mark.parametrize("layout", ["plain", "combined", "heads"])
def test_ragged_and_layouts(layout):
    # (the average chunk is one token of 20 heads: 32-row items, of which the longest chunk takes five)
    paged_case([0, 1, 3, 7, 0, 0, 0, 1], [5, 1, 2, 200, 0, 64, 3, 500], 20, 16, "bf16", seed=6, lead=1, tail=1, layout=layout)


def test_large_scores():
    c = Paged([1, 1], [900, 333], 32, 16, "bf16", 12, qstd=8.0)
    a = B.MLAAttention(config(32, "bf16"), c.T)
    for i in range(2):  # keys that grow along the sequence: every tile raises the maximum
        r = torch.arange(c.L[i], device="cuda")
        c.keys[i] = (c.keys[i].float() * (0.2 + 2.0 * r / c.L[i])[:, None]).to(c.dt)
        blk = c.table[i].long()[r // 16]
        c.lat[blk, r % 16] = c.keys[i][:, :512]
        c.kc[blk, r % 16] = c.keys[i][:, 512:]
    c.run(a)
    assert a.status() == 0
    c.check()


def test_repeated_and_captured():
    c = Paged([1, 1, 1], [3000, 70, 500], 32, 16, "bf16", 21, cap=200)
    a = B.MLAAttention(config(32, "bf16"), c.T)
    c.run(a)
    torch.cuda.synchronize()
    first, flse = c.out.clone(), c.lse.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(a)
    for _ in range(2):
        c.out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, c.out) and torch.equal(flse, c.lse)
    assert a.status() == 0
    c.check()
