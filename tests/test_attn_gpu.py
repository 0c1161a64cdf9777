"""GPU tests of the attention operators against 64-bit references (attn_ref.py
derives the bounds): latent cache append, paged latent attention, prompt
attention, and a run of them together with the prolog."""
import math

import pytest
import torch

from mla_attention_kv_gb300 import binding as B
from mla_attention_kv_gb300 import build as BLD
from mla_attention_kv_gb300 import inputs as I

from attn_ref import attend, check, rope

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
SCALE = 1.0 / math.sqrt(192)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    BLD.build()
    B.load()


def config(H, dtype="fp16", max_pos=4096):
    return dict(kv_lora_rank=512, rope_dim=64, nope_dim=128, v_dim=128, num_heads=H, dtype=dtype, eps=1e-6, max_pos=max_pos)


def rnd(g, *shape, dtype, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------ append
def append_case(T, H, page, dtype, seed, gamma=True, rot=True, q="strided", combined=False, max_pos=300, drop=()):
    g, dt = gen(seed), DT[dtype]
    nb = (T + page - 1) // page + 2
    kv = rnd(g, T, 640, dtype=dt)[:, 24:600]            # strided rows
    slots = torch.randperm(nb * page, generator=g, device="cuda")[:T].to(torch.int32)
    for t in drop:
        slots[t] = -1
    pos = torch.randint(0, max_pos, (T,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = max_pos - 1
    cos, sin = (x.cuda() for x in I.rope_tables(max_pos))
    gam = (1 + 0.1 * torch.randn(512, generator=g, device="cuda")).to(dt)
    if combined:
        cache = rnd(g, nb, page, 576, dtype=dt)
        lat, kc = cache[..., :512], cache[..., 512:]
    else:
        lat, kc = rnd(g, nb, page, 512, dtype=dt), rnd(g, nb, page, 64, dtype=dt)
    lat0, kc0 = lat.clone(), kc.clone()
    qpe = rnd(g, T, H, 192, dtype=dt)[..., 128:]
    qout = None
    if q == "strided":
        qout = rnd(g, H, T, 64, dtype=dt).transpose(0, 1)
    q_in = qpe.clone()
    a = B.MLAAttention(config(H, dtype, max_pos), T)
    a.append_latent(kv[:, :512], kv[:, 512:], pos if rot else None, gam if gamma else None, cos if rot else None,
                    sin if rot else None, slots, lat, kc, q_pe=qpe if q and rot else None, q_pe_out=qout)
    torch.cuda.synchronize()
    assert a.status() == 0 and a.last_launches == 1
    u = torch.finfo(dt).eps / 2
    tiny = 2.0 ** -25 if dtype == "fp16" else 0.0
    x = kv[:, :512].double()
    ref = x / torch.sqrt(x.pow(2).mean(1, keepdim=True) + 1e-6) * gam.double() if gamma else x
    c, s = cos.double()[pos.long()], sin.double()[pos.long()]
    kref = rope(kv[:, 512:].double(), c, s) if rot else kv[:, 512:].double()
    mag = rope(kv[:, 512:].double().abs(), c.abs(), -s.abs()).abs() + rope(kv[:, 512:].double().abs(), c.abs(), s.abs()).abs()
    keep = slots >= 0
    at = slots[keep].long()
    L1, K1 = lat.reshape(-1, 512), kc.reshape(-1, 64)
    # sum of 512 squares, mean, square root, two products: relative fp32 error below 300 * 2^-24 in all
    check("latent", L1[at], ref[keep], (u * 1.01 + 300 * 2.0 ** -24 if gamma else 0.0) * ref[keep].abs() + (tiny if gamma else 0.0))
    check("k_pe", K1[at], kref[keep], u * 1.01 * kref[keep].abs() + 2.0 ** -22 * mag[keep] + tiny if rot else 0 * kref[keep])
    free = torch.ones(nb * page, dtype=torch.bool, device="cuda")
    free[at] = False
    assert torch.equal(L1[free], lat0.reshape(-1, 512)[free]) and torch.equal(K1[free], kc0.reshape(-1, 64)[free])
    if q and rot:
        got = qout if qout is not None else qpe
        qd = q_in.double()
        qref = rope(qd, c[:, None], s[:, None])
        check("q_pe", got, qref, u * 1.01 * qref.abs() + 2.0 ** -22 * (qd.abs().amax() * 2) + tiny)
    a.close()


@pytest.mark.parametrize("T,H,page,dtype,drop", [(1, 1, 1, "fp16", ()), (1, 16, 16, "bf16", ()), (7, 3, 5, "bf16", (2, 6)),
                                                 (8, 128, 64, "fp16", (0,)), (33, 20, 4, "fp16", (5,)), (513, 16, 13, "bf16", (512,))])
@pytest.mark.parametrize("combined", [False, True])
def test_append(T, H, page, dtype, drop, combined):
    append_case(T, H, page, dtype, 10 + T, drop=drop, combined=combined, q="strided" if combined else "inplace")


@pytest.mark.parametrize("gamma,rot,q", [(False, True, "inplace"), (True, False, None), (False, False, None), (True, True, None)])
def test_append_options(gamma, rot, q):
    append_case(19, 4, 8, "bf16", 77, gamma=gamma, rot=rot, q=q)


def test_append_reports_bad_slots_and_positions():
    dt = torch.float16
    g = gen(5)
    kv = rnd(g, 4, 576, dtype=dt)
    cos, sin = (x.cuda() for x in I.rope_tables(8))
    gam = torch.ones(512, dtype=dt, device="cuda")
    a = B.MLAAttention(config(2, "fp16", 8), 4)
    c = a.alloc_latent_caches(2, 4)
    c["latent_cache"].fill_(3.0)
    slots = torch.tensor([0, 8, 7, -5], dtype=torch.int32, device="cuda")
    pos = torch.tensor([0, 0, 7, 0], dtype=torch.int32, device="cuda")
    a.append_latent(kv[:, :512], kv[:, 512:], pos, gam, cos, sin, slots, **c)
    assert a.status() == 10 and a.status() == 0
    assert (c["latent_cache"].view(8, 512)[1:7] == 3.0).all()
    pos = torch.tensor([0, 8, 7, 0], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    a.append_latent(kv[:, :512], kv[:, 512:], pos, gam, cos, sin, slots, **c)
    assert a.status() == 7
    pos[1] = 7  # clamped there
    d = a.alloc_latent_caches(2, 4)
    a.append_latent(kv[:, :512], kv[:, 512:], pos, gam, cos, sin, slots, **d)
    assert a.status() == 0
    assert torch.equal(c["kpe_cache"].view(8, 64)[1], d["kpe_cache"].view(8, 64)[1])


# ------------------------------------------------------------------ paged attention
class Paged:
    """Inputs of a paged call.  Unused cache rows and rows past a sequence's length hold NaN."""

    def __init__(self, n, L, H, page, dtype, seed, lead=0, tail=0, layout="plain", qstd=1.0, cap=None):
        g, dt = gen(seed), DT[dtype]
        self.n, self.L, self.H, self.page, self.dt = n, L, H, page, dt
        self.T = lead + sum(n) + tail
        pages = [(x + page - 1) // page for x in L]
        self.nb = nb = sum(pages) + 2
        cap = cap or max(1, max(pages, default=1))
        perm = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(n), cap), 1 << 30, dtype=torch.int32, device="cuda")  # unread entries are wild
        if layout == "combined":
            cache = torch.full((nb, page, 576), float("nan"), dtype=dt, device="cuda")
            self.lat, self.kc = cache[..., :512], cache[..., 512:]
        else:
            self.lat = torch.full((nb, page, 512), float("nan"), dtype=dt, device="cuda")
            self.kc = torch.full((nb, page, 64), float("nan"), dtype=dt, device="cuda")
        self.keys, at = [], 0
        for i, (ln, pg) in enumerate(zip(L, pages)):
            blocks = perm[at:at + pg]
            at += pg
            self.table[i, :pg] = blocks
            k = rnd(g, ln, 576, dtype=dt)
            r = torch.arange(ln, device="cuda")
            self.lat[blocks.long()[r // page], r % page] = k[:, :512]
            self.kc[blocks.long()[r // page], r % page] = k[:, 512:]
            self.keys.append(k)
        if layout == "heads":  # head-major queries, as a batched product leaves them
            self.ql = rnd(g, H, self.T, 512, dtype=dt, std=qstd).transpose(0, 1)
            self.qp = rnd(g, self.T, H, 192, dtype=dt, std=qstd)[..., 128:]
        else:
            self.ql = rnd(g, self.T, H, 512, dtype=dt, std=qstd)
            self.qp = rnd(g, self.T, H, 64, dtype=dt, std=qstd)
        cu = [lead]
        for x in n:
            cu.append(cu[-1] + x)
        self.cu_list = cu
        self.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(L, dtype=torch.int32, device="cuda")
        self.out = torch.full((self.T, H, 512), 7.0, dtype=dt, device="cuda")
        self.lse = torch.full((self.T, H), 7.0, dtype=torch.float32, device="cuda")

    def run(self, a, cu=True, lse=True, stream=None):
        a.run_paged(self.ql, self.qp, self.lens, self.table, self.lat, self.kc, self.out,
                    cu_q=self.cu if cu else None, lse=self.lse if lse else None, stream=stream)

    def check(self, scale=SCALE, seqs=None):
        for i, (n, L) in enumerate(zip(self.n, self.L)):
            if seqs is not None and i not in seqs:
                continue
            a, b = self.cu_list[i], self.cu_list[i + 1]
            q = torch.cat((self.ql[a:b], self.qp[a:b]), dim=-1).double()
            k = self.keys[i].double()
            out, lse, tol, ltol = attend(q, k, k[:, :512], L - n, scale, self.dt)
            check(f"out[{i}]", self.out[a:b], out, tol)
            check(f"lse[{i}]", self.lse[a:b], lse, ltol)
        # token rows of no sequence keep their contents
        assert (self.out[:self.cu_list[0]] == 7.0).all() and (self.out[self.cu_list[-1]:] == 7.0).all()
        assert (self.lse[:self.cu_list[0]] == 7.0).all() and (self.lse[self.cu_list[-1]:] == 7.0).all()


def paged_case(n, L, H, page, dtype, seed=1, **kw):
    c = Paged(n, L, H, page, dtype, seed, **kw)
    a = B.MLAAttention(config(H, dtype), max(1, c.T))
    c.run(a)
    torch.cuda.synchronize()
    assert a.status() == 0
    c.check()
    a.close()
    return c


@pytest.mark.parametrize("H,dtype", [(16, "fp16"), (16, "bf16"), (1, "fp16"), (8, "bf16"), (20, "fp16"), (64, "fp16"), (128, "bf16")])
def test_paged_decode_lengths(H, dtype):
    L = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300]
    paged_case([1] * len(L), L, H, 16, dtype, seed=H)


@pytest.mark.parametrize("page", [1, 3, 4, 8, 24, 32, 64, 100, 128])
@pytest.mark.parametrize("H", [16, 128])
def test_paged_page_sizes(page, H):
    paged_case([1, 1, 2], [257, 64, 130], H, page, "bf16", seed=page)


@pytest.mark.parametrize("H", [5, 16, 40, 128])
@pytest.mark.parametrize("layout", ["plain", "combined", "heads"])
def test_paged_ragged_chunks(H, layout):
    # chunks of no token, one, many; a chunk longer than its cache (its first rows see nothing); empty caches
    paged_case([0, 1, 3, 5, 2, 70, 0, 9], [5, 1, 2, 0, 90, 200, 0, 9], H, 16, "fp16", seed=H + 3, lead=2, tail=3, layout=layout)


@pytest.mark.parametrize("H,page", [(40, 64), (128, 32), (128, 64), (200, 96)])
@pytest.mark.parametrize("layout", ["plain", "combined", "heads"])
def test_paged_ragged_chunks_of_whole_boxes(H, page, layout):
    # as above on pages that TMA boxes fit, with sequences of several tiles and chunks of several items
    paged_case([0, 1, 3, 5, 2, 70, 0, 9], [5, 1, 2, 0, 290, 400, 0, 9], H, page, "bf16", seed=H + page, lead=2, tail=3, layout=layout)


@pytest.mark.parametrize("page", [32, 64, 16])
def test_paged_decode_lengths_around_boxes_and_tiles(page):
    L = [0, 1, 31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 255, 256, 257, 400]
    paged_case([1] * len(L), L, 128, page, "fp16", seed=page)
    paged_case([2] * len(L), L, 48, page, "bf16", seed=page + 1)


@pytest.mark.parametrize("page", [16, 64])
def test_paged_bad_block_reads_as_zeros(page):
    c = Paged([1, 1, 1], [300, 290, 77], 128, page, "bf16", 8)
    c.table[1, 1], c.keys[1][page:2 * page] = c.nb, 0
    c.table[2, 0], c.keys[2][:page] = -1, 0
    a = B.MLAAttention(config(128, "bf16"), 3)
    c.run(a)
    assert a.status() == 10 and a.status() == 0
    c.check()


@pytest.mark.parametrize("H,n,L", [(16, 1, 5000), (128, 1, 5000), (128, 2, 3001), (3, 1, 20000), (24, 3, 4097)])
def test_paged_long_context_is_split(H, n, L):
    paged_case([n], [L], H, 64, "bf16", seed=L)


def test_paged_mixed_long_and_short():
    paged_case([1, 1, 2, 1], [7000, 3, 900, 2500], 128, 32, "bf16", seed=3)
    paged_case([1, 1, 2, 1], [7000, 3, 900, 2500], 16, 32, "fp16", seed=4)


@pytest.mark.parametrize("H", [4, 128])
def test_paged_many_sequences(H):
    L = [(37 * i) % 90 for i in range(700)]
    paged_case([1] * 700, L, H, 16, "fp16", seed=9)


def test_paged_large_scores_and_running_maximum():
    """Scores of +-200 and more: weights span the whole range, the running maximum moves by large steps."""
    for H in (16, 128):
        c = Paged([1, 2], [900, 333], H, 16, "bf16", 12, qstd=8.0)
        # keys that grow along the sequence: every tile raises the maximum
        a = B.MLAAttention(config(H, "bf16"), c.T)
        for i in range(2):
            r = torch.arange(c.L[i], device="cuda")
            f = (0.2 + 2.0 * r / c.L[i])[:, None]
            c.keys[i] = (c.keys[i].float() * f).to(c.dt)
            blk = c.table[i].long()[r // 16]
            c.lat[blk, r % 16] = c.keys[i][:, :512]
            c.kc[blk, r % 16] = c.keys[i][:, 512:]
        c.run(a)
        torch.cuda.synchronize()
        c.check()


def test_paged_uniform_form_without_offsets_and_lse():
    c = Paged([2] * 5, [10, 40, 3, 2, 100], 16, 16, "fp16", 6)
    a = B.MLAAttention(config(16, "fp16"), c.T, scale=0.11)
    c.run(a, cu=False)
    torch.cuda.synchronize()
    c.check(scale=0.11)
    first = c.out.clone()
    c.out.fill_(0)
    c.lse.fill_(7.0)
    c.run(a, cu=False, lse=False)
    torch.cuda.synchronize()
    assert torch.equal(first, c.out) and (c.lse == 7.0).all()


def test_paged_reports_bad_blocks_and_lengths():
    c = Paged([1, 1], [40, 40], 16, 16, "fp16", 8)
    c.table[1, 1] = c.nb
    a = B.MLAAttention(config(16, "fp16"), 2)
    c.run(a)
    assert a.status() == 10 and a.status() == 0
    c.check(seqs=[0])
    c = Paged([1, 1], [40, 48], 16, 16, "fp16", 8, cap=3)
    c.lens[1] = 49
    c.run(a)
    assert a.status() == 11
    c.check(seqs=[0, 1])  # clamped to the table's 48
    c.lens[1] = -3
    c.run(a)
    assert a.status() == 11
    c.lens[1] = 48
    c.cu[2] = 5
    c.run(a)
    assert a.status() == 11
    c.cu[2] = 0
    c.run(a)
    assert a.status() == 11


@pytest.mark.parametrize("H", [16, 128])
def test_paged_is_repeatable_and_captured(H):
    """Same bits call after call; a captured graph replayed on new contents and lengths."""
    c = Paged([1, 2, 1], [3000, 70, 500], H, 16, "bf16", 21, cap=200)
    a = B.MLAAttention(config(H, "bf16"), c.T)
    c.run(a)
    torch.cuda.synchronize()
    first, flse = c.out.clone(), c.lse.clone()
    for _ in range(3):
        c.out.fill_(7.0)
        c.run(a)
        torch.cuda.synchronize()
        assert torch.equal(first, c.out) and torch.equal(flse, c.lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(a)
    c.ql.mul_(0.5)
    c.L = [1700, 64, 499]
    c.lens.copy_(torch.tensor(c.L, dtype=torch.int32))
    c.keys = [k[:x] for k, x in zip(c.keys, c.L)]
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        c.check()
    assert a.status() == 0


def test_paged_two_handles_on_two_streams():
    cs = [Paged([1] * 4, [900 + 100 * i for i in range(4)], 16, 16, "fp16", 30 + k) for k in range(2)]
    hs = [B.MLAAttention(config(16, "fp16"), 4) for _ in range(2)]
    ss = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, h, s in zip(cs, hs, ss):
            c.run(h, stream=s)
    torch.cuda.synchronize()
    for c in cs:
        c.check()


def test_paged_row_offsets_past_32_bits():
    """A cache of more than 2^31 elements: rows near its end are addressed right."""
    H, page, dt = 16, 64, torch.float16
    nb = (1 << 31) // (512 * page) + 40
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    lat = torch.empty(nb, page, 512, dtype=dt, device="cuda")
    kc = torch.empty(nb, page, 64, dtype=dt, device="cuda")
    g = gen(4)
    k = rnd(g, 2 * page, 576, dtype=dt)
    blocks = [nb - 1, nb - 7]
    for j, b in enumerate(blocks):
        lat[b], kc[b] = k[j * page:(j + 1) * page, :512], k[j * page:(j + 1) * page, 512:]
    for H in (16, 128):
        a = B.MLAAttention(config(H, "fp16"), 1)
        ql, qp = rnd(g, 1, H, 512, dtype=dt), rnd(g, 1, H, 64, dtype=dt)
        out = torch.empty(1, H, 512, dtype=dt, device="cuda")
        a.run_paged(ql, qp, torch.tensor([2 * page - 1], dtype=torch.int32, device="cuda"),
                    torch.tensor([blocks], dtype=torch.int32, device="cuda"), lat, kc, out)
        torch.cuda.synchronize()
        assert a.status() == 0
        kk = k[:2 * page - 1].double()
        ref, _, tol, _ = attend(torch.cat((ql, qp), -1).double(), kk, kk[:, :512], 2 * page - 2, SCALE, dt)
        check("out", out, ref, tol)


# ------------------------------------------------------------------ prompt attention
def prompt_case(lens, H, KH, dtype, seed, packed=True, causal=True, layout="heads", lead=0, tail=0, std=1.0, gaps=None):
    g, dt = gen(seed), DT[dtype]
    b = 1 if packed else len(lens)
    S = lead + sum(lens) + tail if packed else lens[0]

    def make(heads, d, s=std):
        if layout == "tokens":  # token-major memory, [b, heads, S, d] views
            return rnd(g, b, S, heads, d, dtype=dt, std=s).transpose(1, 2)
        if layout == "slices":  # slices of wider rows
            return rnd(g, b, heads, S, d + 72, dtype=dt, std=s)[..., 8:8 + d]
        return rnd(g, b, heads, S, d, dtype=dt, std=s)

    qn, qp, kn, kp, v = make(H, 128), make(H, 64), make(KH, 128), make(1, 64), make(KH, 128)
    out = torch.full((b, S, H, 128), 7.0, dtype=dt, device="cuda").transpose(1, 2) if layout == "tokens" else \
        torch.full((b, H, S, 128), 7.0, dtype=dt, device="cuda")
    lse = torch.full((b, H, S), 7.0, dtype=torch.float32, device="cuda")
    if packed:
        spans, t = [], lead
        for x in lens:
            spans.append((0, t, t + x))
            t += x
        for x in (qn, qp, kn, kp, v):  # tokens of no sequence hold NaN
            x[:, :, :lead] = float("nan")
            x[:, :, t:] = float("nan")
        cu = torch.tensor([lead] + [z for _, _, z in spans], dtype=torch.int32, device="cuda")
    else:
        spans = [(i, 0, lens[0]) for i in range(b)]
        cu = None
    a = B.MLAAttention(config(H, dtype), max(1, b * S), num_kv_heads=KH)
    a.run_prompt(qn, qp, kn, kp, v, out, cu_seqlens=cu, causal=causal, lse=lse)
    torch.cuda.synchronize()
    assert a.status() == 0
    for bi, x, z in spans:
        if x == z:
            continue
        q = torch.cat((qn[bi, :, x:z], qp[bi, :, x:z]), -1).double().transpose(0, 1)
        k = torch.cat((kn[bi, :, x:z], kp[bi, :, x:z].expand(KH, z - x, 64)), -1).double().repeat_interleave(H // KH, 0)
        vv = v[bi, :, x:z].double().repeat_interleave(H // KH, 0)
        ref, rl, tol, ltol = attend(q, k, vv, 0, SCALE, dt, causal)
        check(f"out {bi} {x}:{z}", out[bi, :, x:z].transpose(0, 1), ref, tol)
        check(f"lse {bi} {x}:{z}", lse[bi, :, x:z].transpose(0, 1), rl, ltol)
    if packed:
        for x in (out, lse[..., None]):
            assert (x[:, :, :lead] == 7.0).all() and (x[:, :, lead + sum(lens):] == 7.0).all()
    a.close()


@pytest.mark.parametrize("s", [1, 2, 31, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 640])
def test_prompt_lengths(s):
    prompt_case([s], 2, 2, "bf16", s, packed=False)
    prompt_case([s, s], 3, 3, "fp16", s + 1, packed=False, causal=False)


@pytest.mark.parametrize("layout", ["heads", "tokens", "slices"])
@pytest.mark.parametrize("H,KH", [(4, 4), (8, 2), (6, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_packed(layout, H, KH, causal):
    prompt_case([1, 0, 200, 64, 129, 3, 257], H, KH, "bf16" if causal else "fp16", 5, causal=causal, layout=layout, lead=3, tail=70)


@pytest.mark.parametrize("H", [1, 16])
def test_prompt_many_short_sequences(H):
    prompt_case([(7 * i) % 23 for i in range(300)], H, H, "fp16", 8)


def test_prompt_dense_batches_and_long():
    prompt_case([700] * 3, 16, 16, "fp16", 4, packed=False, layout="tokens")
    prompt_case([1500], 4, 4, "bf16", 5, packed=False)
    prompt_case([333] * 2, 128, 128, "bf16", 6, packed=False)


def test_prompt_large_scores():
    prompt_case([500, 77], 4, 2, "bf16", 14, std=4.0)
    prompt_case([500, 77], 4, 4, "fp16", 15, std=3.0, causal=False)


def test_prompt_reports_bad_offsets():
    dt = torch.float16
    a = B.MLAAttention(config(2, "fp16"), 100)
    x, p = torch.randn(1, 2, 100, 128, device="cuda").to(dt), torch.randn(1, 2, 100, 64, device="cuda").to(dt)
    out = torch.zeros_like(x)
    for cu in ([0, 120], [-4, 50], [0, 60, 40, 100]):
        a.run_prompt(x, p, x, p[:, :1], x, out, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert a.status() == 11, cu
    a.run_prompt(x, p, x, p[:, :1], x, out, cu_seqlens=torch.tensor([0, 100], dtype=torch.int32, device="cuda"))
    assert a.status() == 0 and torch.isfinite(out).all()


def test_prompt_captured_and_repeated():
    dt = torch.bfloat16
    g = gen(2)
    a = B.MLAAttention(config(4, "bf16"), 600)
    qn, qp, kn, kp, v = (rnd(g, 1, h, 600, d, dtype=dt) for h, d in ((4, 128), (4, 64), (4, 128), (1, 64), (4, 128)))
    out = torch.empty_like(qn)
    cu = torch.tensor([0, 100, 600], dtype=torch.int32, device="cuda")
    a.run_prompt(qn, qp, kn, kp, v, out, cu_seqlens=cu)
    torch.cuda.synchronize()
    first = out.clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        a.run_prompt(qn, qp, kn, kp, v, out, cu_seqlens=cu)
    out.zero_()
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    cu.copy_(torch.tensor([0, 0, 333], dtype=torch.int32))
    out.fill_(7.0)
    gr.replay()
    torch.cuda.synchronize()
    assert (out[:, :, 333:] == 7.0).all()
    k = torch.cat((kn, kp.expand(1, 4, 600, 64)), -1)[0, :, :333].double()
    q = torch.cat((qn, qp), -1)[0, :, :333].double().transpose(0, 1)
    ref, _, tol, _ = attend(q, k, v[0, :, :333].double(), 0, SCALE, dt)
    check("out", out[0, :, :333].transpose(0, 1), ref, tol)


@pytest.mark.parametrize("page", [16, 64])
def test_paged_waits_are_bounded(page):
    """With a wait limit of 1 ns a call may give up: it ends, reports it, and the next handle is right."""
    c = Paged([1, 2, 1], [3000, 70, 500], 128, page, "bf16", 21)
    a = B.MLAAttention(config(128, "bf16"), c.T, spin_budget_ns=1)
    for _ in range(2):
        c.run(a)
        assert a.status() in (0, 6) and a.status() == 0
    b = B.MLAAttention(config(128, "bf16"), c.T)
    c.run(b)
    assert b.status() == 0
    c.check()


def test_waits_are_bounded():
    """With a wait limit of 1 ns a call may give up: it ends, reports it, and leaves nothing behind for other handles."""
    c = Paged([1, 2, 1], [3000, 70, 500], 128, 16, "bf16", 21)
    a = B.MLAAttention(config(128, "bf16"), c.T, spin_budget_ns=1)
    c.run(a)
    assert a.status() in (0, 6) and a.status() == 0
    b = B.MLAAttention(config(128, "bf16"), c.T)
    c.run(b)
    assert b.status() == 0
    c.check()
    x, p = rnd(gen(1), 1, 4, 900, 128, dtype=torch.bfloat16), rnd(gen(2), 1, 4, 900, 64, dtype=torch.bfloat16)
    out = torch.empty_like(x)
    for budget in (1, 0):
        h = B.MLAAttention(config(4, "bf16"), 900, spin_budget_ns=budget)
        h.run_prompt(x, p, x, p[:, :1], x, out)
        assert h.status() in ((0, 6) if budget else (0,))
    k = torch.cat((x, p[:, :1].expand(1, 4, 900, 64)), -1)[0].double()
    q = torch.cat((x, p), -1)[0].double().transpose(0, 1)
    ref, _, tol, _ = attend(q, k, x[0].double(), 0, SCALE, torch.bfloat16)
    check("out", out[0].transpose(0, 1), ref, tol)


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("base", ["v2lite", "r1"])
def test_prolog_append_and_attention_together(base):
    """A prompt and then decode steps of one model: prolog -> prompt attention on the up-projected form; kv_a rows ->
    append -> paged attention on the latent form.  Both forms are the same attention: with the kv_b_proj halves
    absorbed, the last tokens' outputs agree with each other and with 64 bits."""
    cfg = I.small_config(I.CONFIGS[base], num_heads=16, hidden=1024)
    H, dt, S, new = 16, I.torch_dtype(cfg), 150, 3
    inp = I.kv_inputs(cfg, 1, S, 77, "prefill")
    d = B.to_device(inp)
    g = gen(6)
    qn, qraw = rnd(g, 1, H, S, 128, dtype=dt), rnd(g, S, H, 64, dtype=dt)
    m = B.MLAProlog(cfg, S)
    a = B.MLAAttention(cfg, S)
    # prompt form
    o = m.run(1, S, d, m.alloc_outputs(1, S))
    kv = (d["hidden"].float() @ d["W_kva"].float()).to(dt)       # kv_a rows, as a library product leaves them
    caches = a.alloc_latent_caches(16, 16)
    for c in caches.values():
        c.fill_(float("nan"))
    blocks = torch.randperm(16, generator=g, device="cuda").to(torch.int32)
    r = torch.arange(S, device="cuda")
    slots = (blocks.long()[r // 16] * 16 + r % 16).to(torch.int32)
    qpe = torch.empty_like(qraw)
    a.append_latent(kv[:, :512], kv[:, 512:], d["positions"], d["gamma_kv"], d["cos"], d["sin"], slots, **caches,
                    q_pe=qraw, q_pe_out=qpe)
    out = torch.empty(1, H, S, 128, dtype=dt, device="cuda")
    a.run_prompt(qn, qpe.transpose(0, 1)[None], o["k_nope"], o["k_pe"], o["value"], out)
    # latent form for the last `new` tokens
    W = d["W_kvb"].view(512, H, 256)
    ql = torch.einsum("htd,rhd->thr", qn[0, :, S - new:].double(), W[..., :128].double()).to(dt)
    lat = torch.empty(new, H, 512, dtype=dt, device="cuda")
    a.run_paged(ql, qpe[S - new:], torch.tensor([S], dtype=torch.int32, device="cuda"), blocks[None].contiguous(), **caches,
                out=lat)
    torch.cuda.synchronize()
    assert a.status() == 0 and m.status() == 0
    up = torch.einsum("thr,rhd->htd", lat.double(), W[..., 128:].double())
    # 64 bits from the hidden rows on
    x = d["hidden"].double() @ d["W_kva"].double()
    n = x[:, :512] / torch.sqrt(x[:, :512].pow(2).mean(1, keepdim=True) + cfg["eps"]) * d["gamma_kv"].double()
    c, s = d["cos"].double()[d["positions"].long()], d["sin"].double()[d["positions"].long()]
    kp, qp = rope(x[:, 512:], c, s), rope(qraw.double(), c[:, None], s[:, None])
    kb = torch.einsum("tr,rhd->htd", n, W.double())
    q = torch.cat((qn[0].double().transpose(0, 1), qp), -1)
    k = torch.cat((kb[..., :128], kp.expand(H, S, 64)), -1)
    ref, _, _, _ = attend(q, k, kb[..., 128:], 0, SCALE, dt)
    ref = ref.transpose(0, 1)
    norm = ref.norm()
    u = torch.finfo(dt).eps / 2
    # four roundings to dtype lie between the hidden rows and either output (kv_a rows or latents, k_nope / value or
    # absorbed queries, weights, outputs), each of relative size at most u in norm; scores of magnitude up to ~8 turn
    # a relative error of the keys and queries (two roundings each) into 8 * 4 u of the weights
    assert (out[0].double() - ref).norm() / norm <= (4 + 32) * u
    assert (up - ref[:, S - new:]).norm() / ref[:, S - new:].norm() <= (4 + 32) * u
    m.close()
    a.close()


def test_latent_rows_of_the_prolog_scattered_as_they_are():
    """mla_kv_prolog_run_latent's rows appended without norm or rotation: the same bits at their slots."""
    cfg = I.V2_LITE
    inp = I.kv_inputs(cfg, 5, 1, 91)
    d = B.to_device(inp)
    m = B.MLAProlog(cfg, 5)
    o = m.run_latent(5, 1, d, m.alloc_latent_outputs(5, 1))
    a = B.MLAAttention(cfg, 5)
    c = a.alloc_latent_caches(3, 4)
    slots = torch.tensor([11, 0, 3, -1, 7], dtype=torch.int32, device="cuda")
    a.append_latent(o["latent"], o["k_pe"].view(5, 64), None, None, None, None, slots, **c)
    torch.cuda.synchronize()
    for t, sl in enumerate(slots.tolist()):
        if sl >= 0:
            assert torch.equal(c["latent_cache"].view(-1, 512)[sl], o["latent"][t])
            assert torch.equal(c["kpe_cache"].view(-1, 64)[sl], o["k_pe"][t, 0, 0])
