"""GPU tests of the paged K/V attention against a 64-bit reference, with the
bounds that attn_ref.py derives.  int8 caches: the codes times their scales
are the reference's keys and values.  Roundings beyond those there: a scale times
a query in fp32 (2^-24) and its split into two fp16 parts (2^-22 of it), 2.5 *
2^-23 of each product in a score and so within the 16 * 2^-23 that the score
bound has to spare; and the product with the value scale in fp32 (2^-24).  The
weights are rounded to fp16, the result to the I/O dtype."""
import math

import pytest
import torch

from mla_attention_kv_gb300 import binding as B
from mla_attention_kv_gb300 import build as BLD

from attn_ref import attend, check

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
SCALE = 1.0 / math.sqrt(192)
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    BLD.build()
    B.load()


def config(H, dtype="fp16"):
    return dict(kv_lora_rank=512, rope_dim=64, nope_dim=128, v_dim=128, num_heads=H, dtype=dtype, eps=1e-6, max_pos=4096)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


class Case:
    """Inputs of a call.  Unused cache rows and rows past a sequence's length hold NaN (int8: wild codes)."""

    def __init__(self, n, L, H, KH, page, dtype, seed=1, i8=False, layout="plain", lead=0, tail=0, qstd=1.0):
        g, dt = gen(seed), DT[dtype]
        self.n, self.L, self.H, self.KH, self.dt, self.i8 = n, L, H, KH, dt, i8
        self.T = lead + sum(n) + tail
        pages = [-(-x // page) for x in L]
        nb = sum(pages) + 2
        perm = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(n), max(1, max(pages))), 1 << 30, dtype=torch.int32, device="cuda")  # unread entries are wild

        def empty(heads, width):
            if layout == "token":  # [block, row, head, width] with a gap between rows
                x = torch.empty(nb, page, heads, width + 16, dtype=torch.int8 if i8 else dt, device="cuda")
                x = x.permute(0, 2, 1, 3)[..., :width]
            else:
                x = torch.empty(nb, heads, page, width, dtype=torch.int8 if i8 else dt, device="cuda")
            if i8:
                x.copy_(torch.randint(-128, 128, x.shape, generator=g, device="cuda"))
            else:
                x.fill_(NAN)
            return x

        self.k, self.v, self.e = empty(KH, 128), empty(KH, 128), empty(1, 64)
        self.scales = None
        if i8:
            u = lambda k, lo, hi: lo + (hi - lo) * torch.rand(k, generator=g, device="cuda")  # noqa: E731
            self.scales = dict(k=u(KH * 128, 0.01, 0.02), v=u(KH * 128, 0.01, 0.02), kpe=u(64, 0.02, 0.04))
        self.keys, self.vals, at = [], [], 0
        for i, (ln, pg) in enumerate(zip(L, pages)):
            blocks = perm[at:at + pg]
            at += pg
            self.table[i, :pg] = blocks
            r = torch.arange(ln, device="cuda")
            blk, off = blocks.long()[r // page], r % page

            def fill(cache, width):
                x = torch.randn(ln, cache.shape[1], width, generator=g, device="cuda")
                x = (x * 64).round().clamp(-127, 127).to(torch.int8) if i8 else x.to(dt)
                cache[blk, :, off] = x
                return x.double()

            k, v, e = fill(self.k, 128), fill(self.v, 128), fill(self.e, 64)
            if i8:
                k = k * self.scales["k"].double().view(KH, 128)
                v = v * self.scales["v"].double().view(KH, 128)
                e = e * self.scales["kpe"].double()
            self.keys.append(torch.cat((k, e.expand(ln, KH, 64)), dim=-1).transpose(0, 1))
            self.vals.append(v.transpose(0, 1))
        r = lambda *s: (torch.randn(*s, generator=g, device="cuda") * qstd).to(dt)  # noqa: E731
        if layout == "token":  # a q projection's rows, head-major
            q = r(H, self.T, 200).transpose(0, 1)
            self.qn, self.qp = q[..., :128], q[..., 136:]
        else:
            self.qn, self.qp = r(self.T, H, 128), r(self.T, H, 64)
        cu = [lead]
        for x in n:
            cu.append(cu[-1] + x)
        self.cu_list = cu
        self.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(L, dtype=torch.int32, device="cuda")
        self.out = torch.full((self.T, H, 128), 7.0, dtype=dt, device="cuda")
        self.lse = torch.full((self.T, H), 7.0, dtype=torch.float32, device="cuda")

    def run(self, a, cu=True, lse=True, stream=None):
        a.run_paged_kv(self.qn, self.qp, self.lens, self.table, self.k, self.v, self.e, self.out, cu_q=self.cu if cu else None,
                       lse=self.lse if lse else None, scales=self.scales, stream=stream)

    def check(self, scale=SCALE):
        G = self.H // self.KH
        for i, (n, L) in enumerate(zip(self.n, self.L)):
            a, b = self.cu_list[i], self.cu_list[i + 1]
            if n == 0:
                continue
            q = torch.cat((self.qn[a:b], self.qp[a:b]), dim=-1).double()
            k, v = (x.repeat_interleave(G, dim=0) for x in (self.keys[i], self.vals[i]))
            out, lse, tol, ltol = attend(q, k, v, L - n, scale, self.dt)
            if self.i8:
                # fp16 weights below the normal range, and the value scale's product
                p = v.abs().sum(1)  # [H, 128]
                tol = tol + 2.0 ** -25 * p[None] + 2.0 ** -23 * out.abs()
            check(f"out[{i}]", self.out[a:b], out, tol)
            check(f"lse[{i}]", self.lse[a:b], lse, ltol)
        for x in (self.out, self.lse):  # token rows of no sequence keep their contents
            assert (x[:self.cu_list[0]] == 7.0).all() and (x[self.cu_list[-1]:] == 7.0).all()


def run_case(*args, cu=True, kv_heads=None, **kw):
    c = Case(*args, **kw)
    a = B.MLAAttention(config(c.H, "fp16" if c.dt is torch.float16 else "bf16"), max(1, c.T), num_kv_heads=c.KH)
    c.run(a, cu=cu)
    assert a.status() == 0 and a.last_launches == (1 if c.T // len(c.n) * (c.H // c.KH) <= 2 else 2)
    c.check()
    a.close()
    return c


LENS = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 200, 777, 1500]


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("page", [1, 7, 16, 64, 2000])
def test_decode(dtype, page, i8):
    run_case([1] * len(LENS), LENS, 4, 4, page, dtype, seed=page, i8=i8, cu=False)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("H,KH", [(1, 1), (16, 16), (8, 1), (20, 5), (24, 8), (34, 2), (128, 128)])
def test_heads(H, KH, i8):
    run_case([1, 1, 1], [1, 90, 301], H, KH, 13, "bf16", seed=H, i8=i8)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("layout", ["plain", "token"])
def test_ragged_chunks(layout, i8):
    """Idle sequences, several tokens, more rows than an item has, lengths below the tokens (rows without keys)."""
    n = [0, 1, 3, 5, 2, 70, 0, 9, 33]
    L = [5, 1, 2, 0, 90, 200, 0, 9, 40]
    c = run_case(n, L, 6, 3, 16, "bf16", seed=5, i8=i8, layout=layout, lead=2, tail=3)
    assert torch.isinf(c.lse[c.cu_list[2]]).all() and (c.out[c.cu_list[2]] == 0).all()


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("H,KH", [(4, 4), (8, 4), (9, 3)])
def test_ragged_steps(H, KH, i8):
    """Few rows per head on average, single sequences with more of them than an item of the kernels for few rows has."""
    run_case([1, 0, 1, 13, 1, 1, 2, 1], [900, 7, 33, 250, 1, 4000, 65, 18], H, KH, 16, "bf16", seed=H, i8=i8)


def test_huge_queries():
    """int8: no intermediate value leaves the range of fp32 before a score does."""
    c = run_case([1, 1], [1, 1], 4, 4, 16, "bf16", seed=15, i8=True, qstd=2.0 ** 124)
    assert torch.isfinite(c.out).all() and torch.isfinite(c.lse).all()


@pytest.mark.parametrize("i8", [False, True])
def test_long_sequences_are_split(i8):
    run_case([1], [40000], 2, 2, 64, "fp16", seed=3, i8=i8)
    run_case([2, 2], [9001, 30000], 16, 4, 32, "bf16", seed=4, i8=i8, cu=False)


@pytest.mark.parametrize("i8", [False, True])
def test_many_sequences(i8):
    g = torch.Generator().manual_seed(1)
    L = torch.randint(0, 300, (700,), generator=g).tolist()
    run_case([1] * 700, L, 2, 2, 16, "fp16", seed=6, i8=i8)


@pytest.mark.parametrize("i8", [False, True])
def test_peaked_scores(i8):
    """Queries thirty times as large: single keys take all the weight, and the maxima differ widely between pieces."""
    run_case([1, 2], [5000, 311], 4, 2, 16, "bf16", seed=8, i8=i8, qstd=30.0)


def test_no_sequences_and_no_rows():
    c = Case([1], [5], 2, 2, 16, "fp16")
    a = B.MLAAttention(config(2), 4)
    a.run_paged_kv(c.qn, c.qp, c.lens[:0], c.table[:0], c.k, c.v, c.e, c.out, cu_q=c.cu[:1])
    a.run_paged_kv(c.qn[:0], c.qp[:0], c.lens, c.table, c.k, c.v, c.e, c.out[:0])
    assert a.status() == 0 and (c.out == 7.0).all()
    a.close()


@pytest.mark.parametrize("i8", [False, True])
def test_bad_blocks_and_lengths_are_reported(i8):
    c = Case([1, 1, 1], [40, 40, 40], 4, 4, 16, "fp16", i8=i8)
    a = B.MLAAttention(config(4), 4)
    good = c.table.clone()
    c.table[1, 1] = 1 << 30
    c.table[2, 2] = -1
    c.run(a)
    assert a.status() == 10 and a.status() == 0
    keep = c.out.clone()
    c.table.copy_(good)
    c.run(a)
    assert a.status() == 0
    c.check()
    assert torch.equal(c.out[0], keep[0])
    c.lens.copy_(torch.tensor([40, -5, 49], dtype=torch.int32))
    c.k[good[2, 2].long(), :, 8:] = 1  # (rows 40 .. 47 of the page come into play)
    c.v[good[2, 2].long(), :, 8:] = 1
    c.e[good[2, 2].long(), :, 8:] = 1
    c.run(a)
    assert a.status() == 11
    assert (c.out[1] == 0).all() and torch.isinf(c.lse[1]).all() and torch.equal(c.out[0], keep[0])
    assert torch.isfinite(c.out[2]).all()
    a.close()


def test_results_repeat_and_do_not_depend_on_the_batch_of_a_handle():
    c = Case([1] * 9, [700, 3, 1999, 64, 1, 300, 4096, 15, 33], 16, 16, 16, "bf16", seed=11)
    a = B.MLAAttention(config(16, "bf16"), 64)
    c.run(a)
    first = (c.out.clone(), c.lse.clone())
    big = Case([2] * 20, [900] * 20, 16, 16, 16, "bf16", seed=12)
    big.run(a)
    c.run(a)
    assert a.status() == 0 and torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])
    c.check()
    big.check()
    a.close()


@pytest.mark.parametrize("i8", [False, True])
def test_graph_replay_follows_the_lengths(i8):
    """A captured call reads lengths and tables anew at each replay; without lse too."""
    c = Case([1, 1, 1], [500, 90, 1], 8, 4, 16, "bf16", seed=13, i8=i8)
    a = B.MLAAttention(config(8, "bf16"), 4, num_kv_heads=4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run(a)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(a)
    full = c.L
    for L in (full, [17, 64, 1], [0, 1, 0], full):
        c.lens.copy_(torch.tensor(L, dtype=torch.int32))
        c.out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        keys, vals = c.keys, c.vals
        c.L, c.keys, c.vals = L, [k[:, :x] for k, x in zip(keys, L)], [v[:, :x] for v, x in zip(vals, L)]
        c.check()
        c.L, c.keys, c.vals = full, keys, vals
    keep = c.out.clone()
    c.run(a, lse=False)
    assert a.status() == 0 and torch.equal(c.out, keep)
    a.close()


def test_two_handles_on_two_streams():
    cs = [Case([1] * 5, [800, 30, 999, 5, 64], 8, 8, 16, "fp16", seed=20 + i, i8=bool(i)) for i in range(2)]
    hs = [B.MLAAttention(config(8), 8) for _ in cs]
    ss = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, a, s in zip(cs, hs, ss):
            c.run(a, stream=s)
    torch.cuda.synchronize()
    for c, a in zip(cs, hs):
        assert a.status() == 0
        c.check()
        a.close()


def test_binding_checks():
    c = Case([1], [5], 4, 2, 16, "fp16")
    a = B.MLAAttention(config(4), 4, num_kv_heads=2)
    args = dict(q_nope=c.qn, q_pe=c.qp, kv_lens=c.lens, block_table=c.table, k_cache=c.k, v_cache=c.v, kpe_cache=c.e, out=c.out)
    for bad in (dict(q_nope=c.qn[:, :2]), dict(k_cache=c.k[:, :1]), dict(v_cache=c.v[..., :64]), dict(kpe_cache=c.k), dict(out=c.out[:, :2]),
                dict(lse=c.lse[:, :1]), dict(cu_q=c.lens), dict(block_table=c.lens), dict(k_cache=c.k.to(torch.int8)),
                dict(k_cache=c.k.transpose(2, 3).contiguous().transpose(2, 3)), dict(kv_lens=c.lens.long()),
                dict(scales=dict(k=c.lse.flatten(), v=c.lse.flatten(), kpe=c.lse.flatten()))):
        with pytest.raises((ValueError, TypeError)):
            a.run_paged_kv(**{**args, **bad})
    a.run_paged_kv(**args)
    assert a.status() == 0
    a.close()
