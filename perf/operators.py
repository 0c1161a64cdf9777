"""Workloads of the attention operators that follow the MLA KV prolog.

Three operators, in the dimensions of the DeepSeek-V2 family (latent 512, rope 64, nope = value = 128):

* ``append``: RMSNorm of the compressed rows, RoPE of the key (and query) position part, scatter into the paged
  latent cache;
* ``paged``: attention of each sequence's newest tokens over its paged latent cache (decode, multi-token decode,
  chunks);
* ``prompt``: causal attention over whole prompts in the up-projected form, dense or packed.

With ``own`` false every operator is computed by elementary torch operations in 32 bits, rounded once; with
``own`` true by the library.
"""
import math
import random

import torch

own = False

RANK, ROPE, NOPE, VDIM = 512, 64, 128, 128
EPS = 1e-6
SCALE = 1.0 / math.sqrt(NOPE + ROPE)
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one decode step of a small batch, V2-Lite heads: all launch latency
        dict(name="append_decode_v2lite", op="append", T=8, H=16, dtype="fp16", page=16, max_pos=4096, lens=1),
        # one decode step of R1, batch 64
        dict(name="append_decode_r1", op="append", T=64, H=128, dtype="bf16", page=64, max_pos=32768, lens=2),
        # packed prompts of V2-Lite with an odd row count, small pages and padding rows
        dict(name="append_ragged_v2lite", op="append", T=1061, H=16, dtype="fp16", page=4, max_pos=4096, lens=3),
        # R1 prefill step of 16384 rows
        dict(name="append_prefill_r1", op="append", T=16384, H=128, dtype="bf16", page=64, max_pos=32768, lens=4),
        # a single chat session decoding: one sequence, latency
        dict(name="paged_single_v2lite", op="paged", b=1, n_max=1, L_min=777, L_max=777, H=16, dtype="fp16", page=16, lens=5),
        # a decode batch of V2-Lite at every context length up to its table
        dict(name="paged_decode_v2lite", op="paged", b=64, n_max=1, L_min=1, L_max=4096, H=16, dtype="fp16", page=16, lens=6),
        # a decode batch of R1 over long ragged contexts
        dict(name="paged_decode_r1", op="paged", b=64, n_max=1, L_min=1, L_max=32768, H=128, dtype="bf16", page=64, lens=7),
        # two-token steps (a drafted token next to the new one) of R1, few sequences with long contexts
        dict(name="paged_draft_r1", op="paged", b=4, n_max=2, L_min=20000, L_max=32768, H=128, dtype="bf16", page=64, lens=8),
        # chunked prefill: ragged chunks of up to 512 tokens behind contexts of up to 8192
        dict(name="paged_chunk_r1", op="paged", b=2, n_max=512, L_min=4096, L_max=8192, H=128, dtype="bf16", page=64, lens=9),
        # short packed prompts of odd lengths with grouped heads
        dict(name="prompt_packed_grouped", op="prompt", b=1, n=5, s_min=1, s_max=301, H=16, Hkv=4, dtype="bf16", lens=10),
        # V2-Lite prefill, 4 sequences of 4096
        dict(name="prompt_v2lite", op="prompt", b=4, n=0, s_min=4096, s_max=4096, H=16, Hkv=16, dtype="fp16", lens=11),
        # R1 prefill, one sequence of 8192
        dict(name="prompt_r1", op="prompt", b=1, n=0, s_min=8192, s_max=8192, H=128, Hkv=128, dtype="bf16", lens=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "paged", "prompt"])
    c = dict(op=op, dtype=rng.choice(["fp16", "bf16"]), lens=rng.randrange(1 << 30))
    if op == "append":
        c.update(T=_log(rng, 1, 16384), H=rng.choice([1, 8, 16, 24, 128]), page=rng.choice([1, 4, 13, 16, 32, 64, 128]),
                 max_pos=rng.choice([4096, 32768]))
    elif op == "paged":
        c.update(b=_log(rng, 1, 64), n_max=rng.choice([1, 1, 1, 2, 3, 0]), H=rng.choice([8, 16, 20, 32, 64, 128]),
                 page=rng.choice([1, 7, 16, 32, 64, 128]))
        if c["n_max"] == 0:
            c["n_max"], c["b"] = _log(rng, 4, 512), _log(rng, 1, 4)
        c["L_max"] = _log(rng, max(64, c["n_max"]), 32768 if c["n_max"] <= 3 else 8192)
        c["L_min"] = rng.choice([1, c["L_max"], max(1, c["L_max"] // 2)])
    else:
        H = rng.choice([4, 16, 24, 128])
        c.update(H=H, Hkv=H // rng.choice([1, 1, 2, 4]))
        if rng.random() < 0.5:
            n = _log(rng, 1, 12)
            c.update(b=1, n=n, s_max=_log(rng, 1, (4096 if H > 24 else 8192) // n))
            c["s_min"] = rng.choice([1, c["s_max"]])
        else:
            s = _log(rng, 1, 2048)
            c.update(b=rng.randrange(1, 5), n=0, s_min=s, s_max=s)
    return c


# ------------------------------------------------------------------ sizes that follow from a case
def _lengths(case):
    """Host-side lengths: append -> slots' holes; paged -> (new tokens, cached tokens) per sequence; prompt ->
    sequence lengths."""
    r = random.Random(case["lens"])
    if case["op"] == "paged":
        n = [r.randint((case["n_max"] + 1) // 2, case["n_max"]) if case["n_max"] > 3 else case["n_max"] for _ in range(case["b"])]
        L = [max(k, r.randint(case["L_min"], case["L_max"])) for k in n]
        return n, L
    if case["op"] == "prompt":
        if case["n"] == 0:
            return [case["s_max"]] * case["b"]
        return [r.randint(case["s_min"], case["s_max"]) for _ in range(case["n"])]
    return None


def work(case):
    e = 2
    if case["op"] == "append":
        T, H = case["T"], case["H"]
        return {"bytes": T * (2 * e * (RANK + ROPE + H * ROPE) + 8) + e * RANK + 8 * ROPE * min(T, case["max_pos"]),
                "flops": T * (4 * RANK + 3 * ROPE * (H + 1))}
    if case["op"] == "paged":
        n, L = _lengths(case)
        H, T = case["H"], sum(n)
        pairs = sum(k * l - k * (k - 1) // 2 for k, l in zip(n, L))
        return {"bytes": e * (RANK + ROPE) * sum(L) + T * H * (e * (2 * RANK + ROPE) + 4),
                "flops": 2 * (2 * RANK + ROPE) * H * pairs}
    s = _lengths(case)
    H, Hkv, T = case["H"], case["Hkv"], sum(s)
    pairs = sum(k * (k + 1) // 2 for k in s)
    return {"bytes": T * (e * (H * (NOPE + ROPE + VDIM) + Hkv * (NOPE + VDIM) + ROPE) + 4 * H),
            "flops": 2 * (NOPE + ROPE + VDIM) * H * pairs}


# ------------------------------------------------------------------ inputs
def _tables(max_pos, dev):
    j = torch.arange(ROPE, dtype=torch.float64, device=dev) % (ROPE // 2)
    ang = torch.arange(max_pos, dtype=torch.float64, device=dev)[:, None] * torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=dev), -2.0 * j / ROPE)
    return torch.cos(ang).float().contiguous(), torch.sin(ang).float().contiguous()


def _config(case):
    return dict(kv_lora_rank=RANK, rope_dim=ROPE, nope_dim=NOPE, v_dim=VDIM, num_heads=case["H"], dtype=case["dtype"], eps=EPS,
                max_pos=case.get("max_pos", 4096))


def prepare(case, seed):
    dev = "cuda"
    dt = DTYPES[case["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    i32 = dict(dtype=torch.int32, device=dev)

    def randn(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * std).to(dt)

    st = dict(case=case)
    if case["op"] == "append":
        T, H, page = case["T"], case["H"], case["page"]
        nb = (T + page - 1) // page + 2
        # the kv_a projection's rows (hidden ~ N(0,1) times weights ~ N(0, 0.02)), and a query whose last 64 of 192
        # columns per head are the position part, as a q projection leaves them
        kv = randn(T, RANK + ROPE, std=0.9)
        q = randn(T, H, NOPE + ROPE)
        slots = torch.randperm(nb * page, generator=g, device=dev)[:T].to(torch.int32)
        if T > 16:
            slots[torch.randperm(T, generator=g, device=dev)[: T // 16]] = -1  # padding rows
        cos, sin = _tables(case["max_pos"], dev)
        st.update(kv=kv, ckv=kv[:, :RANK], k_pe=kv[:, RANK:], q_pe=q[..., NOPE:],
                  positions=torch.randint(0, case["max_pos"], (T,), generator=g, **i32), slots=slots.contiguous(),
                  gamma=(1.0 + 0.1 * torch.randn(RANK, generator=g, device=dev)).to(dt), cos=cos, sin=sin,
                  latent_cache=randn(nb, page, RANK), kpe_cache=randn(nb, page, ROPE),
                  q_out=torch.empty(T, H, ROPE, dtype=dt, device=dev))
        max_tokens = T
    elif case["op"] == "paged":
        n, L = _lengths(case)
        H, page, T = case["H"], case["page"], sum(n)
        pages = [(x + page - 1) // page for x in L]
        nb = sum(pages) + 3
        perm = torch.randperm(nb, generator=g, device=dev)[: sum(pages)].to(torch.int32)
        table = torch.zeros(len(n), max(pages), **i32)
        at = torch.arange(max(pages), device=dev)[None, :] < torch.tensor(pages, device=dev)[:, None]
        table[at] = perm
        cu = [0]
        for k in n:
            cu.append(cu[-1] + k)
        # normalised latents times gamma, rotated keys; absorbed queries whose scores spread over a few units
        st.update(q_latent=randn(T, H, RANK), q_pe=randn(T, H, ROPE), latent_cache=randn(nb, page, RANK),
                  kpe_cache=randn(nb, page, ROPE), table=table, kv_lens=torch.tensor(L, **i32), cu_q=torch.tensor(cu, **i32),
                  out=torch.empty(T, H, RANK, dtype=dt, device=dev), lse=torch.empty(T, H, dtype=torch.float32, device=dev))
        max_tokens = T
    else:
        s = _lengths(case)
        H, Hkv = case["H"], case["Hkv"]
        b, S = (1, sum(s)) if case["n"] else (case["b"], s[0])
        # the prolog's head-major outputs and queries of the same kind
        st.update(q_nope=randn(b, H, S, NOPE), q_pe=randn(b, H, S, ROPE), k_nope=randn(b, Hkv, S, NOPE), k_pe=randn(b, 1, S, ROPE),
                  value=randn(b, Hkv, S, VDIM), out=torch.empty(b, H, S, VDIM, dtype=dt, device=dev),
                  lse=torch.empty(b, H, S, dtype=torch.float32, device=dev))
        cu = [0]
        for k in s:
            cu.append(cu[-1] + k)
        st["cu"] = torch.tensor(cu, **i32) if case["n"] else None
        max_tokens = b * S
    if own:
        from mla_attention_kv_gb300 import binding
        st["attn"] = binding.MLAAttention(_config(case), max_tokens, num_kv_heads=case.get("Hkv"))
    return st


# ------------------------------------------------------------------ the operators
def _rope(x, cos, sin):
    """De-interleave, then rotate halves: x [..., 64] fp32, cos / sin broadcastable."""
    x = torch.cat((x[..., 0::2], x[..., 1::2]), dim=-1)
    rot = torch.cat((-x[..., ROPE // 2:], x[..., : ROPE // 2]), dim=-1)
    return x * cos + rot * sin


def _softmax_(s):
    """In-place softmax of fp32 scores (masked entries -inf) along the last dimension, and its log-sum-exp; rows
    with no entry give zeros and -inf."""
    m = s.amax(dim=-1, keepdim=True)
    safe = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    s.sub_(safe).exp_()
    l = s.sum(dim=-1, keepdim=True)
    s.div_(torch.where(l == 0, torch.ones_like(l), l))
    return (safe + l.log()).squeeze(-1)


def _append_plain(st):
    dt = st["ckv"].dtype
    x = st["ckv"].float()
    n = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * st["gamma"].float()
    pos = st["positions"].long()
    cos, sin = st["cos"][pos], st["sin"][pos]
    k = _rope(st["k_pe"].float(), cos, sin)
    keep = st["slots"] >= 0
    at = st["slots"][keep].long()
    st["latent_cache"].view(-1, RANK)[at] = n[keep].to(dt)
    st["kpe_cache"].view(-1, ROPE)[at] = k[keep].to(dt)
    q = _rope(st["q_pe"].float(), cos[:, None], sin[:, None]).to(dt)
    return [st["latent_cache"], st["kpe_cache"], q]


def _paged_plain(st):
    case = st["case"]
    H, page = case["H"], case["page"]
    kv_lens, cu = st["kv_lens"].long(), st["cu_q"].long()
    T = st["q_latent"].shape[0]
    n = cu[1:] - cu[:-1]
    b, n_max, L_max = len(n), case["n_max"], st["table"].shape[1] * page
    # the sequences' cached rows, padded to the longest
    keys = torch.cat((st["latent_cache"][st["table"].long()].reshape(b, L_max, RANK),
                      st["kpe_cache"][st["table"].long()].reshape(b, L_max, ROPE)), dim=-1).float()
    seq = torch.bucketize(torch.arange(T, device=cu.device), cu[1:], right=True)
    at = torch.arange(T, device=cu.device) - cu[seq]
    q = torch.zeros(b, n_max, H, RANK + ROPE, device=cu.device)
    q[seq, at] = torch.cat((st["q_latent"], st["q_pe"]), dim=-1).float()
    s = torch.matmul(q.view(b, n_max * H, -1), keys.transpose(1, 2)).mul_(SCALE).view(b, n_max, H, L_max)
    last = (kv_lens - n)[:, None] + torch.arange(n_max, device=cu.device)[None, :]
    hidden = torch.arange(L_max, device=cu.device)[None, None, :] > last[:, :, None]
    s.masked_fill_(hidden[:, :, None, :], -math.inf)
    lse = _softmax_(s)
    out = torch.matmul(s.view(b, n_max * H, L_max), keys[..., :RANK]).view(b, n_max, H, RANK)
    return [out[seq, at].to(st["q_latent"].dtype), lse[seq, at].contiguous()]


def _prompt_plain(st):
    case = st["case"]
    H, Hkv, dt = case["H"], case["Hkv"], st["q_nope"].dtype
    b, S = st["q_nope"].shape[0], st["q_nope"].shape[2]
    pos = torch.arange(S, device=st["q_nope"].device)
    hidden = pos[None, :] > pos[:, None]
    if st["cu"] is not None:
        seq = torch.bucketize(pos, st["cu"][1:].long(), right=True)
        hidden = hidden | (seq[None, :] != seq[:, None])
    q = torch.cat((st["q_nope"], st["q_pe"]), dim=-1).float()
    k = torch.cat((st["k_nope"], st["k_pe"].expand(b, Hkv, S, ROPE)), dim=-1).float()
    q = q.view(b, Hkv, H // Hkv, S, NOPE + ROPE)
    s = torch.matmul(q, k.transpose(-1, -2).unsqueeze(2)).mul_(SCALE)
    s.masked_fill_(hidden, -math.inf)
    lse = _softmax_(s).view(b, H, S)
    out = torch.matmul(s, st["value"].float().unsqueeze(2)).view(b, H, S, VDIM)
    return [out.to(dt), lse]


def run(st):
    op = st["case"]["op"]
    if own:
        a = st["attn"]
        if op == "append":
            a.append_latent(st["ckv"], st["k_pe"], st["positions"], st["gamma"], st["cos"], st["sin"], st["slots"],
                            st["latent_cache"], st["kpe_cache"], q_pe=st["q_pe"], q_pe_out=st["q_out"])
            return [st["latent_cache"], st["kpe_cache"], st["q_out"]]
        if op == "paged":
            a.run_paged(st["q_latent"], st["q_pe"], st["kv_lens"], st["table"], st["latent_cache"], st["kpe_cache"], st["out"],
                        cu_q=st["cu_q"], lse=st["lse"])
            return [st["out"], st["lse"]]
        a.run_prompt(st["q_nope"], st["q_pe"], st["k_nope"], st["k_pe"], st["value"], st["out"], cu_seqlens=st["cu"], lse=st["lse"])
        return [st["out"], st["lse"]]
    if op == "append":
        return _append_plain(st)
    if op == "paged":
        return _paged_plain(st)
    return _prompt_plain(st)


# ------------------------------------------------------------------ 64-bit definitions
def _exact_append(case, st):
    T, H = case["T"], case["H"]
    lat, kpe = st["latent_cache"].double(), st["kpe_cache"].double()
    x = st["ckv"].double()
    nrm = x / torch.sqrt(x.pow(2).sum(1, keepdim=True) / RANK + EPS) * st["gamma"].double()
    c, s = st["cos"].double()[st["positions"].long()], st["sin"].double()[st["positions"].long()]

    def turn(v, c, s):  # pair (2j, 2j+1) turned by angle j, stored at j and 32 + j
        even, odd = v[..., 0::2], v[..., 1::2]
        lo = even * c[..., :32] - odd * s[..., :32]
        hi = odd * c[..., 32:] + even * s[..., 32:]
        return torch.cat((lo, hi), dim=-1)

    keep = torch.nonzero(st["slots"] >= 0).flatten()
    block, off = st["slots"][keep].long() // case["page"], st["slots"][keep].long() % case["page"]
    lat[block, off] = nrm[keep]
    kpe[block, off] = turn(st["k_pe"].double(), c, s)[keep]
    return [lat, kpe, turn(st["q_pe"].double(), c.view(T, 1, ROPE), s.view(T, 1, ROPE))]


def _exact_rows(q, k, v, first):
    """q [n, H, d], k [L, d] or [H, L, d], v alike; row i sees keys 0 .. first + i. Blocks of rows bound the memory."""
    n, H, d = q.shape
    out = torch.zeros(n, H, v.shape[-1], dtype=torch.float64, device=q.device)
    lse = torch.full((n, H), -math.inf, dtype=torch.float64, device=q.device)
    step = max(1, min(n, 1024, (1 << 28) // max(1, H * (first + n))))
    for i in range(0, n, step):
        j = min(n, i + step)
        e = first + j
        if e <= 0:
            continue
        s = torch.einsum("nhd,ld->hnl", q[i:j], k[:e]) if k.dim() == 2 else torch.bmm(q[i:j].transpose(0, 1), k[:, :e].transpose(1, 2))
        s *= SCALE
        gone = torch.arange(e, device=q.device)[None, :] > (first + torch.arange(i, j, device=q.device))[:, None]
        s = s.masked_fill(gone[None], -math.inf)
        z = torch.logsumexp(s, dim=-1)
        p = torch.exp(s - z[..., None])
        p = torch.nan_to_num(p, nan=0.0)
        o = torch.einsum("hnl,ld->nhd", p, v[:e]) if v.dim() == 2 else torch.bmm(p, v[:, :e]).transpose(0, 1)
        out[i:j], lse[i:j] = o, z.transpose(0, 1)
    return out, lse


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "append":
        return _exact_append(case, st)
    if case["op"] == "paged":
        n, L = _lengths(case)
        outs, lses, t = [], [], 0
        for i, (k, l) in enumerate(zip(n, L)):
            rows = torch.arange(l, device="cuda")
            block, off = st["table"][i].long()[rows // case["page"]], rows % case["page"]
            lat = st["latent_cache"][block, off].double()
            key = torch.cat((lat, st["kpe_cache"][block, off].double()), dim=-1)
            q = torch.cat((st["q_latent"][t:t + k], st["q_pe"][t:t + k]), dim=-1).double()
            o, z = _exact_rows(q, key, lat, l - k)
            outs.append(o)
            lses.append(z)
            t += k
        return [torch.cat(outs), torch.cat(lses)]
    H, rep = case["H"], case["H"] // case["Hkv"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    spans = [(bi, 0, s) for bi, s in enumerate(_lengths(case))] if st["cu"] is None else [
        (0, int(a), int(z)) for a, z in zip(st["cu"][:-1], st["cu"][1:])]
    for bi, a, z in spans:
        for h in range(0, H, rep):
            key = torch.cat((st["k_nope"][bi, h // rep, a:z], st["k_pe"][bi, 0, a:z]), dim=-1).double()
            q = torch.cat((st["q_nope"][bi, h:h + rep, a:z], st["q_pe"][bi, h:h + rep, a:z]), dim=-1).double().transpose(0, 1)
            o, l = _exact_rows(q, key, st["value"][bi, h // rep, a:z].double(), 0)
            out[bi, h:h + rep, a:z], lse[bi, h:h + rep, a:z] = o.transpose(0, 1), l.transpose(0, 1)
    return [out, lse]
