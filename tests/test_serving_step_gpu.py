"""A run of the serving-step operators together: prompts, decode steps, a
sequence that ends and one that takes its place.  Each step: page plan ->
e4m3 q projection -> KV prolog into the paged K/V caches, latent append with
the queries' rotation -> attention over the K/V caches -> e4m3 output
projection.  A decode step is captured once and replayed.

Each stage is compared in 64 bits on the inputs that it had (bounds of
attn_ref.py and test_fp8_linear_gpu.py); the plan with its sequential
restatement; the two caches with each other: key and value are kv_b_proj of
the cached latent, one rounding of the latent (u) and one of the product (u)
apart, with fp32 sums of 512 terms."""
import math

import pytest
import torch

from mla_attention_kv_gb300 import binding as B
from mla_attention_kv_gb300 import build as BLD
from mla_attention_kv_gb300 import inputs as I

from attn_ref import attend, check, rope
from test_fp8_linear_gpu import reference
from test_fp8_rows_gpu import quantise
from test_page_plan_gpu import plan_ref

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn
T, PAGE, BLOCKS, WIDTH = 48, 16, 24, 6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    BLD.build()
    B.load()


class Engine:
    def __init__(self, dtype):
        self.cfg = cfg = I.small_config(I.V2_LITE, num_heads=8, hidden=1024, dtype=dtype, max_pos=256)
        self.dt, self.H = I.torch_dtype(cfg), 8
        self.w = B.to_device({k: v for k, v in I.kv_inputs(cfg, 1, 2, 5, "prefill").items() if k not in ("hidden", "positions")})
        g = self.g = torch.Generator(device="cuda").manual_seed(3)

        def weight(n, k):
            q, s = [], []
            for r in range(0, n, 128):  # a scale for each block of 128 x 128
                rows = 0.03 * torch.randn(min(128, n - r), k, generator=g, device="cuda")
                b = torch.nn.functional.pad(rows, (0, -k % 128)).view(len(rows), -1, 128)
                sc = b.abs().amax((0, 2)) / 448.0
                q.append((b / sc[None, :, None]).clamp(-448, 448).to(E4).view(torch.uint8).reshape(len(rows), -1)[:, :k])
                s.append(sc)
            return torch.cat(q).contiguous().view(E4), torch.stack(s).contiguous()

        self.wq, self.sq = weight(self.H * 192, 1024)
        self.wo, self.so = weight(1024, self.H * 128)
        self.q_proj = B.MLAFp8Linear(self.wq, self.sq, dtype, T)
        self.o_proj = B.MLAFp8Linear(self.wo, self.so, dtype, T)
        self.prolog, self.attn = B.MLAProlog(cfg, T), B.MLAAttention(cfg, T)
        self.kv = self.prolog.alloc_paged_caches(BLOCKS, PAGE)
        self.lat = self.attn.alloc_latent_caches(BLOCKS, PAGE)
        for c in list(self.kv.values()) + list(self.lat.values()):
            c.fill_(float("nan"))
        i32 = dict(dtype=torch.int32, device="cuda")
        n = 3
        self.table = torch.full((n, WIDTH), -1, **i32)
        self.free = torch.randperm(BLOCKS, generator=g, device="cuda").to(torch.int32)
        self.count, self.lens = torch.tensor([BLOCKS], **i32), torch.zeros(n, **i32)
        self.new, self.ended = torch.zeros(n, **i32), torch.zeros(n, **i32)
        self.cu, self.slots, self.pos = torch.zeros(n + 1, **i32), torch.zeros(T, **i32), torch.zeros(T, **i32)
        new = lambda *s: torch.zeros(*s, dtype=self.dt, device="cuda")  # noqa: E731
        self.x, self.q, self.ctx, self.y = new(T, 1024), new(T, self.H * 192), new(T, self.H, 128), new(T, 1024)
        self.lse = torch.zeros(T, self.H, device="cuda")
        self.gamma = (1 + 0.1 * torch.randn(1024, generator=g, device="cuda")).to(self.dt)

    def step(self):
        w = self.w
        self.attn.plan_pages(self.new, self.lens, self.table, self.free, self.count, PAGE, self.cu, self.slots, self.pos, ended=self.ended)
        self.q_proj.run(self.q, x=self.x, gamma=self.gamma)
        self.prolog.run_paged(1, T, dict(w, hidden=self.x, positions=self.pos), self.slots, PAGE, self.kv)
        kv = (self.x.float() @ w["W_kva"].float()).to(self.dt)
        q = self.q.view(T, self.H, 192)
        self.qraw = q[..., 128:].clone()
        self.attn.append_latent(kv[:, :512], kv[:, 512:], self.pos, w["gamma_kv"], w["cos"], w["sin"], self.slots, **self.lat, q_pe=q[..., 128:])
        self.attn.run_paged_kv(q[..., :128], q[..., 128:], self.lens, self.table, self.kv["k_cache"], self.kv["v_cache"],
                               self.kv["kpe_cache"], self.ctx, cu_q=self.cu, lse=self.lse)
        self.o_proj.run(self.y, x=self.ctx.view(T, -1))

    def state(self):
        return [x.tolist() for x in (self.new, self.lens, self.table, self.free, self.count, self.ended)]

    def check(self, before):
        new, lens, table, free, count, ended = before
        ref, bad = plan_ref(new, lens, table, free, count[0], PAGE, T, ended)
        assert not bad
        for name, x in dict(slots=self.slots, positions=self.pos, cu=self.cu, lens=self.lens, table=self.table, free=self.free, count=self.count).items():
            assert x.tolist() == ref[name], name
        u = torch.finfo(self.dt).eps / 2
        live = ref["cu"][-1]
        # the projections, on the codes of their own row quantisation
        qc, qs = torch.empty(T, 1024, device="cuda").to(E4), torch.empty(8, T, device="cuda")
        B.mla_fp8_quant_rows(self.x, qc, qs, gamma=self.gamma)
        out, tol = reference(qc, qs, self.wq, self.sq, self.dt)
        raw = torch.cat((self.q.view(T, self.H, 192)[..., :128], self.qraw), -1).reshape(T, -1)
        check("q", raw, out, tol)
        oc, os_ = quantise(self.ctx.view(T, -1).float())
        out, tol = reference(oc.to(E4), os_.t().contiguous(), self.wo, self.so, self.dt)
        check("y", self.y[:live], out[:live], tol[:live])
        q = self.q.view(T, self.H, 192).double()
        c, s = (self.w[k].double()[self.pos.long()][:, None] for k in ("cos", "sin"))
        turned = rope(self.qraw.double(), c, s)
        check("q_pe", self.q.view(T, self.H, 192)[..., 128:], turned, u * 1.01 * turned.abs() + 2.0 ** -21 * self.qraw.double().abs().amax() + 2.0 ** -25)
        W = self.w["W_kvb"].double().view(512, self.H, 256)
        for i, (a, b, L) in enumerate(zip(ref["cu"][:-1], ref["cu"][1:], ref["lens"])):
            if L == 0:
                continue
            r = torch.arange(L, device="cuda")
            blk, off = self.table[i].long()[r // PAGE], r % PAGE
            k, v, e = (self.kv[n][blk, :, off].double().transpose(0, 1) for n in ("k_cache", "v_cache", "kpe_cache"))
            latent = self.lat["latent_cache"][blk, off].double()
            up = torch.einsum("tr,rhd->htd", latent, W)
            mag = torch.einsum("tr,rhd->htd", latent.abs(), W.abs())
            # (the kv_a product behind the latents is rounded to dtype here and shifts the norm by as much: five u in all)
            err = 5 * u * 1.01 * mag + 2.0 ** -14 * mag
            assert ((torch.cat((k, v), -1) - up).abs() <= err).all()
            if b == a:
                continue
            ctx, lse, tol, ltol = attend(q[a:b], torch.cat((k, e.expand(self.H, L, 64)), -1), v, L - (b - a), 1 / math.sqrt(192), self.dt)
            check(f"ctx[{i}]", self.ctx[a:b], ctx, tol)
            check(f"lse[{i}]", self.lse[a:b], lse, ltol)
        assert self.attn.status() == 0 and self.prolog.status() == 0 and self.q_proj.status() == 0 and self.o_proj.status() == 0

    def feed(self, new, ended=(0, 0, 0)):
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        self.ended.copy_(torch.tensor(ended, dtype=torch.int32))
        self.x.copy_(torch.randn(T, 1024, generator=self.g, device="cuda"))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_prompts_decode_and_a_new_sequence(dtype):
    e = Engine(dtype)
    for new, ended in (([31, 5, 0], (0, 0, 0)), ([1, 1, 12], (0, 0, 0)), ([1, 3, 1], (0, 0, 0)), ([1, 19, 1], (0, 1, 0)), ([1, 1, 0], (0, 0, 1)),
                       ([1, 1, 7], (0, 0, 0))):
        e.feed(new, ended)
        before = e.state()
        e.step()
        torch.cuda.synchronize()
        e.check(before)
    # a captured decode step, replayed over a page's end
    e.feed([1, 1, 1])
    keep = [x.clone() for x in (e.lens, e.table, e.free, e.count)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        e.step()
    s.synchronize()
    for x, y in zip((e.lens, e.table, e.free, e.count), keep):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        e.step()
    for _ in range(10):
        e.feed([1, 1, 1])
        before = e.state()
        graph.replay()
        torch.cuda.synchronize()
        e.check(before)
