"""Workloads of the operators of a serving step around the MLA KV prolog.

Four operators, in the dimensions of the DeepSeek-V2 family (rope 64, nope = value = 128):

* ``plan``: block table, slot mapping, positions and offsets of a step, made on the GPU from the requests' lengths,
  with the free pages handed out and taken back;
* ``quant``: rows to 8-bit floating point (e4m3) with a scale for each 128 columns, after an RMSNorm or not;
* ``linear``: the product of such rows with a weight in e4m3 that has a scale for each block of 128 x 128;
* ``paged_kv``: attention of each sequence's newest tokens over the paged k_nope / value / k_pe caches that the prolog
  writes, in 16 bits or as int8 codes with a scale per channel.

With ``own`` false every operator is computed by elementary torch operations in 32 bits, rounded once; with
``own`` true by the library.
"""
import math
import random

import torch

own = False

ROPE, NOPE, VDIM = 64, 128, 128
BLOCK = 128
EPS = 1e-6
E4M3_MAX = 448.0
SCALE = 1.0 / math.sqrt(NOPE + ROPE)
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one decode step of 64 sequences, pages of 64: a few hundred integers, all launch latency
        dict(name="plan_decode", op="plan", n=64, page=64, max_len=32768, kind="decode", T=64, lens=1),
        # a busy step of 256 requests: some end, some decode, some bring chunks of their prompts; small pages
        dict(name="plan_mixed", op="plan", n=256, page=16, max_len=8192, kind="mixed", T=16384, lens=2),
        # the q latent of a decode batch of R1, normalised on the way
        dict(name="quant_norm_decode_r1", op="quant", T=64, K=1536, norm=True, dtype="bf16"),
        # the hidden rows of an R1 prefill step
        dict(name="quant_hidden_r1", op="quant", T=8192, K=7168, norm=False, dtype="bf16"),
        # V2-Lite's kv_a projection of one token
        dict(name="linear_single_v2lite", op="linear", T=1, K=2048, N=576, given="x", dtype="fp16"),
        # R1's q_a and kv_a projections as one weight, a decode batch
        dict(name="linear_decode_r1", op="linear", T=64, K=7168, N=2112, given="x", dtype="bf16"),
        # R1's kv_b projection of a chunk of odd length, rows that were quantised before
        dict(name="linear_chunk_r1", op="linear", T=517, K=512, N=32768, given="q", dtype="bf16"),
        # R1's q_b projection of a prefill step
        dict(name="linear_prefill_r1", op="linear", T=8192, K=1536, N=24576, given="x", dtype="bf16"),
        # a single chat session decoding: one sequence, latency
        dict(name="paged_kv_single_v2lite", op="paged_kv", b=1, n_max=1, L_min=777, L_max=777, H=16, KH=16, dtype="fp16", cache="16",
             page=16, lens=5),
        # a decode batch of V2-Lite at every context length up to its table
        dict(name="paged_kv_decode_v2lite", op="paged_kv", b=64, n_max=1, L_min=1, L_max=4096, H=16, KH=16, dtype="fp16", cache="16",
             page=16, lens=6),
        # three-token steps (drafted tokens next to the new one) with grouped heads and an odd page size
        dict(name="paged_kv_draft_grouped", op="paged_kv", b=12, n_max=3, L_min=100, L_max=9000, H=20, KH=5, dtype="bf16", cache="16",
             page=13, lens=7),
        # a decode batch of R1 heads over the dense int8 cache that the prolog writes (one page per sequence)
        dict(name="paged_kv_c8_r1", op="paged_kv", b=16, n_max=1, L_min=1024, L_max=4096, H=128, KH=128, dtype="bf16", cache="int8",
             page=4096, lens=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "quant", "linear", "linear", "paged_kv", "paged_kv"])
    c = dict(op=op)
    if op == "plan":
        kind = rng.choice(["decode", "draft", "mixed"])
        n = _log(rng, 1, 512)
        c.update(n=n, page=rng.choice([1, 4, 13, 16, 32, 64, 128]), max_len=_log(rng, 64, 32768 if n <= 64 else 8192), kind=kind,
                 lens=rng.randrange(1 << 30))
        c["T"] = n if kind == "decode" else 4 * n if kind == "draft" else min(16384, max(8, n * _log(rng, 4, 128)))
        return c
    c["dtype"] = rng.choice(["fp16", "bf16"])
    if op == "quant":
        K = rng.choice([512, 576, 1536, 2048, 2112, 7168, 16384, 16 * _log(rng, 1, 512)])
        c.update(T=_log(rng, 1, min(16384, 8192 * 7168 // K)), K=K, norm=rng.random() < 0.5)
    elif op == "linear":
        K, N = rng.choice([(2048, 576), (512, 4096), (7168, 2112), (1536, 24576), (512, 32768), (16384, 7168), (2048, 2048),
                           (16 * _log(rng, 4, 500), 8 * _log(rng, 4, 2000))])
        most = min(8192, 8192 * 24576 * 1536 // (K * N))
        c.update(T=_log(rng, 1, most), K=K, N=N, given=rng.choice(["x", "q"]))
    else:
        KH = rng.choice([1, 2, 5, 8, 16, 16, 128])
        c.update(b=_log(rng, 1, 64), n_max=rng.choice([1, 1, 1, 2, 4, 0]), KH=KH, H=KH * rng.choice([1, 1, 1, 2, 4, 8] if KH < 128 else [1]),
                 page=rng.choice([1, 7, 16, 16, 32, 64, 64, 128, 512]), cache=rng.choice(["16", "16", "int8"]), lens=rng.randrange(1 << 30))
        if c["n_max"] == 0:
            c["n_max"] = _log(rng, 5, 32)
            c["b"] = min(c["b"], 8)
        most = max(c["n_max"], min(32768, 16 * 4096 * 128 // (c["b"] * max(KH, c["H"] * c["n_max"] // 8))))
        c["L_max"] = _log(rng, max(1, c["n_max"]), most)
        c["L_min"] = rng.choice([1, c["L_max"], max(1, c["L_max"] // 2)])
    return c


# ------------------------------------------------------------------ sizes that follow from a case
def _plan_lengths(case):
    """Host lists: cached lengths, new tokens, whether a sequence ends. Their tokens fit in T rows."""
    r = random.Random(case["lens"])
    n, top, left = case["n"], case["max_len"], case["T"]
    old, new, ended = [], [], []
    for i in range(n):
        fresh = k = e = 0
        u = r.random()
        if case["kind"] == "decode":
            k = 1
        elif case["kind"] == "draft":
            k = r.randint(1, 4)
        elif u < 0.1:
            e = 1
        elif u < 0.2:
            k = 0
        elif u < 0.7:
            k = 1
        else:
            fresh, k = r.random() < 0.5, r.randint(1, max(1, 2 * case["T"] // n))
        k = min(k, left, top)
        left -= k
        L = 0 if fresh else r.randint(0, top - k)
        old.append(L)
        new.append(k)
        ended.append(e)
    return old, new, ended


def _lengths(case):
    """New tokens and cached tokens (the new ones included) of each sequence."""
    r = random.Random(case["lens"])
    n = [r.randint((case["n_max"] + 1) // 2, case["n_max"]) if case["n_max"] > 4 else case["n_max"] for _ in range(case["b"])]
    return n, [max(k, r.randint(case["L_min"], case["L_max"])) for k in n]


def _up(a, b):
    return -(-a // b)


def work(case):
    if case["op"] == "plan":
        old, new, ended = _plan_lengths(case)
        n, page = case["n"], case["page"]
        back = sum(_up(L, page) for L, e in zip(old, ended) if e)
        out = sum(_up(L + k, page) - _up(L, page) for L, k, e in zip(old, new, ended) if not e)
        return {"bytes": 4 * (5 * n + 3) + 8 * case["T"] + 8 * (back + out), "flops": case["T"] + 4 * n}
    if case["op"] == "quant":
        T, K = case["T"], case["K"]
        return {"bytes": 3 * T * K + 4 * T * _up(K, BLOCK) + (2 * K if case["norm"] else 0), "flops": (6 if case["norm"] else 3) * T * K}
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        rows = 2 * T * K if case["given"] == "x" else T * K + 4 * T * _up(K, BLOCK)
        return {"bytes": rows + N * K + 4 * _up(N, BLOCK) * _up(K, BLOCK) + 2 * T * N, "flops": 2 * T * N * K}
    n, L = _lengths(case)
    H, KH, T = case["H"], case["KH"], sum(n)
    e = 1 if case["cache"] == "int8" else 2
    pairs = sum(k * l - k * (k - 1) // 2 for k, l in zip(n, L))
    return {"bytes": e * (KH * (NOPE + VDIM) + ROPE) * sum(L) + T * H * (2 * (NOPE + ROPE + VDIM) + 4),
            "flops": 2 * (NOPE + ROPE + VDIM) * H * pairs}


# ------------------------------------------------------------------ inputs
def _attn_config(H, dtype):
    return dict(kv_lora_rank=512, rope_dim=ROPE, nope_dim=NOPE, v_dim=VDIM, num_heads=H, dtype=dtype, eps=EPS, max_pos=32768)


def _blocks(w, rows, cols):
    """w [N, K] padded to whole blocks, as [N / rows, rows, K / cols, cols]."""
    N, K = w.shape
    w = torch.nn.functional.pad(w, (0, -K % cols, 0, -N % rows))
    return w.view(w.shape[0] // rows, rows, w.shape[1] // cols, cols)


def _quantise(x, rows):
    """e4m3 codes and scales of x (fp32) over blocks of rows x 128."""
    b = _blocks(x, rows, BLOCK)
    s = (b.abs().amax(dim=(1, 3)) / E4M3_MAX).clamp(min=2.0 ** -126)
    q = (b * (1.0 / s)[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    N, K = x.shape
    return q.view(-1, b.shape[2] * BLOCK)[:N, :K].contiguous(), s


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    i32 = dict(dtype=torch.int32, device=dev)

    def randn(*shape, std=1.0, dt=torch.float32):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * std).to(dt)

    st = dict(case=case)
    if case["op"] == "plan":
        old, new, ended = _plan_lengths(case)
        page, n = case["page"], case["n"]
        pages = [_up(x, page) for x in old]
        width = _up(case["max_len"], page)
        total = sum(pages) + sum(_up(x + k, page) - _up(x, page) for x, k in zip(old, new)) + 5
        ids = torch.randperm(total, generator=g, device=dev).to(torch.int32)
        table = torch.zeros(n, width, **i32)
        at = torch.arange(width, device=dev)[None, :] < torch.tensor(pages, device=dev)[:, None]
        table[at] = ids[: sum(pages)]
        free = torch.zeros(total, **i32)
        free[: total - sum(pages)] = ids[sum(pages):]
        st.update(new_lens=torch.tensor(new, **i32), ended=torch.tensor(ended, **i32), kv_lens=torch.tensor(old, **i32), table=table,
                  free=free, free_count=torch.tensor([total - sum(pages)], **i32), kv_out=torch.zeros(n, **i32),
                  count_out=torch.zeros(1, **i32), cu=torch.zeros(n + 1, **i32), slots=torch.zeros(case["T"], **i32),
                  positions=torch.zeros(case["T"], **i32))
        if own:
            from mla_attention_kv_gb300 import binding
            st["attn"] = binding.MLAAttention(_attn_config(16, "bf16"), case["T"])
        return st
    dt = DTYPES[case["dtype"]]
    if case["op"] == "quant":
        T, K = case["T"], case["K"]
        # activations: normal rows, some columns ten times the others
        col = 1.0 + 9.0 * (torch.rand(K, generator=g, device=dev) < 0.01).float()
        st.update(x=(randn(T, K) * col).to(dt), gamma=(1.0 + randn(K, std=0.1)).to(dt) if case["norm"] else None,
                  q=torch.empty(T, K, dtype=torch.float8_e4m3fn, device=dev),
                  scale=torch.empty(_up(K, BLOCK), T, dtype=torch.float32, device=dev))
        return st
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        w, ws = _quantise(randn(N, K, std=0.02), BLOCK)
        x = randn(T, K)
        st.update(w=w, ws=ws, out=torch.empty(T, N, dtype=dt, device=dev))
        if case["given"] == "x":
            st["x"] = x.to(dt)
        else:
            st["xq"], xs = _quantise(x, 1)
            st["xs"] = xs.t().contiguous()
        if own:
            from mla_attention_kv_gb300 import binding
            st["linear"] = binding.MLAFp8Linear(st["w"], st["ws"], case["dtype"], T)
        return st
    n, L = _lengths(case)
    H, KH, page, T = case["H"], case["KH"], case["page"], sum(n)
    pages = [_up(x, page) for x in L]
    nb = sum(pages) + (0 if page >= case["L_max"] else 3)
    table = torch.zeros(len(n), max(pages), **i32)
    at = torch.arange(max(pages), device=dev)[None, :] < torch.tensor(pages, device=dev)[:, None]
    # (a dense cache has its sequences in order)
    table[at] = (torch.arange(nb, device=dev) if page >= case["L_max"] else torch.randperm(nb, generator=g, device=dev))[: sum(pages)].to(torch.int32)
    cu = [0]
    for k in n:
        cu.append(cu[-1] + k)
    if case["cache"] == "int8":
        def codes(*shape):  # values N(0, 1) over scales of 0.01 to 0.02, clipped
            x = torch.randn(*shape, generator=g, device=dev, dtype=torch.float16)
            return x.mul_(64.0).round_().clamp_(-127, 127).to(torch.int8)

        def scales(k):
            return 0.01 + 0.01 * torch.rand(k, generator=g, device=dev)

        st.update(k=codes(nb, KH, page, NOPE), v=codes(nb, KH, page, VDIM), kpe=codes(nb, 1, page, ROPE),
                  scales=dict(k=scales(KH * NOPE), v=scales(KH * VDIM), kpe=scales(ROPE)))
    else:
        def values(*shape):
            return torch.randn(*shape, generator=g, device=dev, dtype=dt)

        st.update(k=values(nb, KH, page, NOPE), v=values(nb, KH, page, VDIM), kpe=values(nb, 1, page, ROPE), scales=None)
    st.update(q_nope=randn(T, H, NOPE, dt=dt), q_pe=randn(T, H, ROPE, dt=dt), table=table, kv_lens=torch.tensor(L, **i32),
              cu_q=torch.tensor(cu, **i32), out=torch.empty(T, H, VDIM, dtype=dt, device=dev),
              lse=torch.empty(T, H, dtype=torch.float32, device=dev))
    if own:
        from mla_attention_kv_gb300 import binding
        st["attn"] = binding.MLAAttention(_attn_config(H, case["dtype"]), T, num_kv_heads=KH)
    return st


# ------------------------------------------------------------------ the operators
def _plan_plain(st):
    page, T = st["case"]["page"], st["case"]["T"]
    table, free = st["table"], st["free"]
    dev = table.device
    old, new, ended = st["kv_lens"].long(), st["new_lens"].long(), st["ended"] != 0
    pages = (old + page - 1) // page
    back = torch.where(ended, pages, torch.zeros_like(pages))
    col = torch.arange(table.shape[1], device=dev)
    given = table[col[None, :] < back[:, None]]  # in (sequence, page) order
    count = st["free_count"].long()
    free[count + torch.arange(len(given), device=dev)] = given
    count = count + back.sum()
    old = torch.where(ended, torch.zeros_like(old), old)
    first = torch.where(ended, torch.zeros_like(pages), pages)
    need = (old + new + page - 1) // page - first
    cu = torch.zeros(len(new) + 1, dtype=torch.int64, device=dev)
    cu[1:] = new.cumsum(0)
    before = need.cumsum(0) - need
    # new pages, k-th of the step: from the top of the stack
    fresh = (col[None, :] >= first[:, None]) & (col[None, :] < (first + need)[:, None])
    k = before[:, None] + col[None, :] - first[:, None]
    table[fresh] = free[(count - 1 - k)[fresh]]
    row = torch.arange(T, device=dev)
    seq = torch.bucketize(row, cu[1:], right=True)
    real = seq < len(new)
    seq = seq.clamp(max=len(new) - 1)
    pos = torch.where(real, old[seq] + row - cu[seq], torch.zeros_like(row))
    slot = table[seq, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page
    st["slots"].copy_(torch.where(real, slot, torch.full_like(slot, -1)))
    st["positions"].copy_(pos)
    st["cu"].copy_(cu)
    st["kv_out"].copy_(old + new)
    st["count_out"].copy_(count - need.sum())
    return _plan_outputs(st)


def _plan_outputs(st):
    return [st["slots"], st["positions"], st["cu"], st["kv_out"], st["table"], st["free"], st["count_out"]]


def _quant_plain(st):
    x = st["x"].float()
    if st["gamma"] is not None:
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * st["gamma"].float()
    q, s = _quantise(x, 1)
    return [q, s.t().contiguous()]


def _linear_plain(st):
    if st["case"]["given"] == "x":
        xq, xs = _quantise(st["x"].float(), 1)
    else:
        xq, xs = st["xq"], st["xs"].t()
    K, N = st["case"]["K"], st["case"]["N"]
    x = xq.float() * xs.repeat_interleave(BLOCK, dim=1)[:, :K]
    w = st["w"].float() * st["ws"].repeat_interleave(BLOCK, dim=0)[:N].repeat_interleave(BLOCK, dim=1)[:, :K]
    return [torch.matmul(x, w.t()).to(st["out"].dtype)]


def _gather(cache, table):
    """Pages of the sequences' tables as [b, KH, L_max, d] in fp32."""
    b, pages = table.shape
    x = cache[table.long()]  # [b, pages, KH, page, d]
    return x.transpose(1, 2).reshape(b, cache.shape[1], pages * cache.shape[2], cache.shape[3]).float()


def _paged_kv_plain(st):
    case = st["case"]
    H, KH = case["H"], case["KH"]
    kv_lens, cu = st["kv_lens"].long(), st["cu_q"].long()
    T = st["q_nope"].shape[0]
    n = cu[1:] - cu[:-1]
    b, n_max = len(n), case["n_max"]
    G = H // KH
    kn, kp, v = _gather(st["k"], st["table"]), _gather(st["kpe"], st["table"]), _gather(st["v"], st["table"])
    if st["scales"] is not None:
        kn.mul_(st["scales"]["k"].view(1, KH, 1, NOPE))
        kp.mul_(st["scales"]["kpe"])
        v.mul_(st["scales"]["v"].view(1, KH, 1, VDIM))
    L_max = kn.shape[2]
    seq = torch.bucketize(torch.arange(T, device=cu.device), cu[1:], right=True)
    at = torch.arange(T, device=cu.device) - cu[seq]

    def rows(q):  # [T, H, d] -> [b, KH, n_max * G, d]
        x = torch.zeros(b, n_max, H, q.shape[-1], device=cu.device)
        x[seq, at] = q.float()
        return x.view(b, n_max, KH, G, -1).transpose(1, 2).reshape(b, KH, n_max * G, -1)

    s = torch.matmul(rows(st["q_nope"]), kn.transpose(2, 3))
    s += torch.matmul(rows(st["q_pe"]), kp.transpose(2, 3))
    s = s.mul_(SCALE).view(b, KH, n_max, G, L_max)
    last = (kv_lens - n)[:, None] + torch.arange(n_max, device=cu.device)[None, :]
    hidden = torch.arange(L_max, device=cu.device)[None, None, :] > last[:, :, None]
    s.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    v.masked_fill_((torch.arange(L_max, device=cu.device)[None, :] >= kv_lens[:, None])[:, None, :, None], 0.0)
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    s.sub_(m).exp_()
    l = s.sum(dim=-1, keepdim=True)
    s.div_(torch.where(l == 0, torch.ones_like(l), l))
    lse = (m + l.log()).view(b, KH, n_max, G).transpose(1, 2).reshape(b, n_max, H)
    out = torch.matmul(s.view(b, KH, n_max * G, L_max), v).view(b, KH, n_max, G, VDIM).transpose(1, 2).reshape(b, n_max, H, VDIM)
    return [out[seq, at].to(st["q_nope"].dtype), lse[seq, at].contiguous()]


def run(st):
    op = st["case"]["op"]
    if own:
        if op == "plan":
            st["attn"].plan_pages(st["new_lens"], st["kv_lens"], st["table"], st["free"], st["free_count"], st["case"]["page"],
                                  st["cu"], st["slots"], st["positions"], kv_lens_out=st["kv_out"], free_count_out=st["count_out"],
                                  ended=st["ended"])
            return _plan_outputs(st)
        if op == "quant":
            from mla_attention_kv_gb300 import binding
            binding.mla_fp8_quant_rows(st["x"], st["q"], st["scale"], gamma=st["gamma"], eps=EPS)
            return [st["q"], st["scale"]]
        if op == "linear":
            if st["case"]["given"] == "x":
                st["linear"].run(st["out"], x=st["x"])
            else:
                st["linear"].run(st["out"], x_q=st["xq"], x_scale=st["xs"])
            return [st["out"]]
        st["attn"].run_paged_kv(st["q_nope"], st["q_pe"], st["kv_lens"], st["table"], st["k"], st["v"], st["kpe"], st["out"],
                                cu_q=st["cu_q"], lse=st["lse"], scales=st["scales"])
        return [st["out"], st["lse"]]
    if op == "plan":
        return _plan_plain(st)
    if op == "quant":
        return _quant_plain(st)
    if op == "linear":
        return _linear_plain(st)
    return _paged_kv_plain(st)


# ------------------------------------------------------------------ 64-bit definitions
def _to_e4m3(x):
    """The nearest e4m3 value of each x (fp64, |x| <= 448), ties to even."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -9))).clamp(min=-6.0)
    step = torch.exp2(e - 3.0)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_rows(x):
    """Values of the codes and scales [T, blocks] of fp64 rows."""
    q, s = torch.zeros_like(x), []
    for k in range(0, x.shape[1], BLOCK):
        part = x[:, k:k + BLOCK]
        sk = torch.clamp(part.abs().max(dim=1).values / E4M3_MAX, min=2.0 ** -126)
        q[:, k:k + BLOCK] = _to_e4m3(part / sk[:, None])
        s.append(sk)
    return q, torch.stack(s, dim=1)


def _exact_paged(case, st):
    H, KH, page = case["H"], case["KH"], case["page"]
    G = H // KH
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    n, L = _lengths(case)
    t = 0
    for i, (k, l) in enumerate(zip(n, L)):
        rows = torch.arange(l, device="cuda")
        block, off = st["table"][i].long()[rows // page], rows % page
        pe = st["kpe"][block, 0, off].double()
        if st["scales"] is not None:
            pe = pe * st["scales"]["kpe"].double()
        gone = torch.arange(l, device="cuda")[None, :] > torch.arange(l - k, l, device="cuda")[:, None]
        for h in range(KH):
            key, val = st["k"][block, h, off].double(), st["v"][block, h, off].double()
            if st["scales"] is not None:
                key = key * st["scales"]["k"][h * NOPE:(h + 1) * NOPE].double()
                val = val * st["scales"]["v"][h * VDIM:(h + 1) * VDIM].double()
            q = st["q_nope"][t:t + k, h * G:(h + 1) * G].double()
            s = torch.einsum("ngd,ld->gnl", q, key) + torch.einsum("ngd,ld->gnl", st["q_pe"][t:t + k, h * G:(h + 1) * G].double(), pe)
            s = (s * SCALE).masked_fill(gone, -math.inf)
            z = torch.logsumexp(s, dim=-1)
            p = torch.nan_to_num(torch.exp(s - z[..., None]), nan=0.0)
            out[t:t + k, h * G:(h + 1) * G] = torch.einsum("gnl,ld->ngd", p, val)
            lse[t:t + k, h * G:(h + 1) * G] = z.t()
        t += k
    return [out, lse]


def exact(case, seed):
    global own
    if case["op"] == "plan":
        return None
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "quant":
        x = st["x"].double()
        if st["gamma"] is not None:
            x = x / torch.sqrt(x.pow(2).sum(1, keepdim=True) / case["K"] + EPS) * st["gamma"].double()
        q, s = _exact_rows(x)
        return [q, s.t().contiguous()]
    if case["op"] == "linear":
        if case["given"] == "x":
            q, s = _exact_rows(st["x"].double())
        else:
            q, s = st["xq"].double(), st["xs"].double().t()
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
        ws = st["ws"].double()
        for k in range(0, case["K"], BLOCK):
            xk = q[:, k:k + BLOCK] * s[:, k // BLOCK, None]
            wk = st["w"][:, k:k + BLOCK].double() * ws[:, k // BLOCK].repeat_interleave(BLOCK)[: case["N"], None]
            out.addmm_(xk, wk.t())
        return [out]
    return _exact_paged(case, st)
