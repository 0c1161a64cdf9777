"""Page plans of sequences that become shorter between steps (drafted tokens
that are rejected): with the pages that each sequence holds kept in an array,
no block is lost and none is in two places.  The GPU tests compare every output
with a sequential restatement of the rules; all are whole numbers."""
import random

import pytest
import torch

from mla_attention_kv_gb300 import binding as B
from mla_attention_kv_gb300 import build as BLD

from test_attn_abi import FakeHandle
from test_page_plan_gpu import handle
from test_serving_abi import PLAN, fake, packed


def plan_held(new, lens, held, table, free, count, page, T, ended):
    """The rules of mla_page_plan_held, one sequence after the other, for state that is consistent but for counts out of range."""
    n, nb, width = len(new), len(free), len(table[0])
    table, free, bad = [list(r) for r in table], list(free), set()
    up = lambda x: -(-x // page)  # noqa: E731

    def holds(i):
        h = min(max(held[i], up(lens[i])), width)
        if h != held[i]:
            bad.add(11)
        return h

    have = [holds(i) for i in range(n)]
    for i in range(n):
        if ended[i]:
            for b in table[i][:have[i]]:
                free[count] = b
                count += 1
    slots, pos, cu, out, after = [-1] * T, [0] * T, [0], [], []
    at = used = 0
    for i in range(n):
        old, h = (0, 0) if ended[i] else (lens[i], have[i])
        begin = cu[-1]
        cu.append(begin + new[i])
        ok = old + new[i] <= width * page
        if not ok:
            bad.add(11)
        need = max(0, up(old + new[i]) - h) if ok else 0
        if need and at + need > count:
            ok = False
            bad.add(12)
        if ok:
            table[i][h:h + need] = [free[count - 1 - at - m] for m in range(need)]
            if need:
                used = at + need
            for j in range(new[i]):
                p = old + j
                pos[begin + j] = p
                blk = table[i][p // page]
                if 0 <= blk < nb:
                    slots[begin + j] = blk * page + p % page
                else:
                    bad.add(10)
        at += need
        out.append(old + new[i] if ok else old)
        after.append(h + need if ok else h)
    return dict(slots=slots, positions=pos, cu=cu, lens=out, held=after, table=table, free=free, count=[count - used]), bad


class State:
    def __init__(self, n, page, width, nb, T, in_place=True):
        self.page, self.T, self.in_place = page, T, in_place
        t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.t = t
        self.lens, self.held, self.table = [0] * n, [0] * n, [[-1] * width for _ in range(n)]
        self.free, self.count = list(range(nb)), nb
        random.Random(nb).shuffle(self.free)
        self.d = dict(new=t([0] * n), ended=t([0] * n), lens=t(self.lens), held=t(self.held), table=t(self.table), free=t(self.free), count=t([nb]),
                      cu=t([0] * (n + 1)), slots=t([0] * T), positions=t([0] * T))
        self.out = {k: self.d[k].clone() for k in ("lens", "held", "count")}
        self.a = handle(T)

    def call(self):
        d, o = self.d, self.out
        more = {} if self.in_place else dict(kv_lens_out=o["lens"], free_count_out=o["count"], held_out=o["held"])
        self.a.plan_pages(d["new"], d["lens"], d["table"], d["free"], d["count"], self.page, d["cu"], d["slots"], d["positions"],
                          ended=d["ended"], held=d["held"], **more)

    def set(self, **kw):
        for k, v in kw.items():
            self.d[k].copy_(self.t(v))

    def step(self, new, ended=None, run=None):
        n = len(new)
        ended = ended or [0] * n
        self.set(new=new, ended=ended, lens=self.lens, held=self.held)
        ref, bad = plan_held(new, self.lens, self.held, self.table, self.free, self.count, self.page, self.T, ended)
        (run or self.call)()
        status = self.a.status()
        for name, want in ref.items():
            got = self.out[name] if not self.in_place and name in self.out else self.d[name]
            assert got.tolist() == want, name
        assert status == (min(bad) if bad else 0)
        if not self.in_place:
            self.set(count=ref["count"])
        self.lens, self.held, self.table, self.free, self.count = ref["lens"], ref["held"], ref["table"], ref["free"], ref["count"][0]
        return bad

    def blocks(self):
        """Every block that a sequence holds or that is free."""
        return sorted(self.free[:self.count] + [b for r, h in zip(self.table, self.held) for b in r[:h]])


@pytest.fixture
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    BLD.build()
    B.load()


@pytest.mark.gpu
@pytest.mark.parametrize("n,page", [(1, 1), (3, 4), (20, 16), (64, 3), (600, 2)])
@pytest.mark.parametrize("in_place", [True, False])
def test_rejected_drafts_lose_no_pages(lib, n, page, in_place):
    r = random.Random(n + page)
    nb = n * 12 + 3
    s = State(n, page, 12, nb, 9 * n, in_place)
    for step in range(25):
        new = [min(r.randint(0, 8), 12 * page - L) for L in s.lens]
        ended = [int(step > 3 and r.random() < 0.1) for _ in range(n)]
        assert not s.step(new, ended)
        assert s.blocks() == list(range(nb))
        # some of the tokens just planned, or all of them, are rejected, over page ends too
        s.lens = [L - r.randint(0, k) for L, k in zip(s.lens, new)]
    assert not s.step([0] * n, [1] * n)
    assert s.count == nb and s.held == [0] * n
    s.a.close()


@pytest.mark.gpu
def test_counts_out_of_range_and_too_few_pages(lib):
    s = State(3, 4, 6, 10, 40)
    assert not s.step([9, 4, 0])
    s.held = [1, 7, 0]  # fewer than nine tokens fill; more than a table row has
    assert s.step([0, 0, 1]) == {11}
    s.a.close()
    s = State(3, 4, 6, 5, 40)
    assert not s.step([9, 4, 0])
    s.lens = [1, 4, 0]
    assert s.step([11, 4, 3]) == {12}  # (the first needs none, the second the last one)
    assert s.held == [3, 2, 0] and s.blocks() == list(range(5))
    s.lens = [0, 0, 0]
    assert not s.step([4, 0, 1], [0, 1, 0])  # held pages are used again, those of the second are free
    assert s.blocks() == list(range(5))
    s.a.close()


@pytest.mark.gpu
def test_captured_steps(lib):
    """A captured plan in place; between replays the lengths are lowered on the device."""
    s = State(4, 3, 10, 44, 24)
    side = torch.cuda.Stream()
    keep = {k: v.clone() for k, v in s.d.items()}
    with torch.cuda.stream(side):
        s.call()
    side.synchronize()
    for k, v in keep.items():
        s.d[k].copy_(v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.call()
    r = random.Random(1)
    for _ in range(12):
        new = [min(5, 30 - L) for L in s.lens]
        assert not s.step(new, run=graph.replay)
        assert s.blocks() == list(range(44))
        s.lens = [L - r.randint(0, k) for L, k in zip(s.lens, new)]
    s.a.close()


@pytest.mark.gpu
def test_without_sequences_and_binding_checks(lib):
    s = State(2, 4, 3, 6, 4)
    e = s.t([])
    s.a.plan_pages(e, e, s.d["table"][:0], s.d["free"], s.d["count"], 4, s.d["cu"][:1], s.d["slots"], s.d["positions"], held=e)
    assert s.a.status() == 0 and s.d["slots"].tolist() == [-1] * 4
    args = (s.d["new"], s.d["lens"], s.d["table"], s.d["free"], s.d["count"], 4, s.d["cu"], s.d["slots"], s.d["positions"])
    for bad in (dict(held=s.d["cu"]), dict(held=s.d["held"].long()), dict(held=s.d["held"], held_out=s.d["cu"]), dict(held_out=s.d["held"])):
        with pytest.raises((ValueError, TypeError)):
            s.a.plan_pages(*args, **bad)
    s.a.close()


@pytest.mark.parametrize("held,out,over,code", [
    (0, 1, {}, 1), (1, 0, {}, 1), (0x5000004, 1, {}, 4), (1, 0x5000008, {}, 4), (1, 1, dict(lens=0), 1), (1, 1, dict(T=17), 3), (1, 1, dict(page=0), 1)])
def test_refusals(held, out, over, code):
    BLD.build()
    L = B.load()
    held, out = (fake() if x == 1 else x for x in (held, out))
    h = FakeHandle().ptr
    assert L.mla_page_plan_held(h, packed(B._PLAN_ARGS, PLAN, **over), held or None, out or None, None) == code
    assert L.mla_page_plan_held(None, packed(B._PLAN_ARGS, PLAN), fake(), fake(), None) == 1
    assert L.mla_page_plan_held(h, None, fake(), fake(), None) == 1
