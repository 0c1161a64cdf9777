"""GPU tests of the page plan against a sequential restatement of its rules on
the host: every output is a whole number and has to be equal."""
import random

import pytest
import torch

from mla_attention_kv_gb300 import binding as B
from mla_attention_kv_gb300 import build as BLD

pytestmark = pytest.mark.gpu
MAX = 0x7fffff00


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    BLD.build()
    B.load()


def handle(T):
    cfg = dict(kv_lora_rank=512, rope_dim=64, nope_dim=128, v_dim=128, num_heads=2, dtype="bf16", eps=1e-6, max_pos=64)
    return B.MLAAttention(cfg, max(1, T))


def plan_ref(new, lens, table, free, count, page, T, ended):
    """The rules of mla_page_plan, one sequence after the other.  Returns the outputs and the status bits."""
    n, nb, width = len(new), len(free), len(table[0]) if table else 0
    cap = min(width * page, MAX)
    table, free, bad = [list(r) for r in table], list(free), set()

    def clamp(x, lo, hi):
        if x < lo or x > hi:
            bad.add(11)
        return min(max(x, lo), hi)

    count = clamp(count, 0, nb)
    old = [0 if ended[i] else clamp(lens[i], 0, cap) for i in range(n)]
    for i in range(n):
        if ended[i]:
            for b in table[i][:-(-clamp(lens[i], 0, cap) // page)]:
                if count < nb:
                    free[count] = b
                    count += 1
                else:
                    bad.add(11)
    slots, pos, cu, out = [-1] * T, [0] * T, [0], []
    at = row = used = 0
    for i in range(n):
        k = clamp(new[i], 0, MAX * 2)
        begin, row = row, row + k
        cu.append(min(row, T))
        ok = row <= T and old[i] + k <= cap
        if not ok:
            bad.add(11)
        first = -(-old[i] // page)
        need = -(-(old[i] + k) // page) - first if ok else 0
        if ok and need and at + need > count:
            ok = False
            bad.add(12)
        if ok:
            for m in range(need):
                table[i][first + m] = free[count - 1 - at - m]
            if need:
                used = at + need
            for j in range(k):
                p = old[i] + j
                blk = table[i][p // page]
                pos[begin + j] = p
                if 0 <= blk < nb:
                    slots[begin + j] = blk * page + p % page
                else:
                    bad.add(10)
        at += need
        out.append(old[i] + k if ok else old[i])
    return dict(slots=slots, positions=pos, cu=cu, lens=out, table=table, free=free, count=[count - used]), bad


def run_case(new, lens, table, free, count, page, T, ended=None, in_place=False, a=None):
    ref, bad = plan_ref(new, lens, table, free, count, page, T, ended or [0] * len(new))
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    n = len(new)
    d_lens, d_count, d_table, d_free = t(lens), t([count]), t(table).reshape(n, len(table[0]) if n else 0), t(free)
    lens_out, count_out = (None, None) if in_place else (torch.full((n,), 77, dtype=torch.int32, device="cuda"), t([77]))
    cu, slots, pos = (torch.full((k,), 77, dtype=torch.int32, device="cuda") for k in (n + 1, T, T))
    h = a or handle(T)
    h.plan_pages(t(new), d_lens, d_table, d_free, d_count, page, cu, slots, pos, kv_lens_out=lens_out, free_count_out=count_out,
                 ended=None if ended is None else t(ended))
    status = h.status()
    got = dict(slots=slots, positions=pos, cu=cu, lens=d_lens if in_place else lens_out, table=d_table, free=d_free,
               count=d_count if in_place else count_out)
    for name, x in got.items():
        assert x.tolist() == ref[name], name
    assert status == (min(bad) if bad else 0)
    assert h.last_launches == 1 and h.status() == 0
    if a is None:
        h.close()
    return bad


def make(rng, n, page, width, nb, top=None):
    """Consistent state: every sequence holds its own blocks, the others are on the stack."""
    ids = list(range(nb))
    rng.shuffle(ids)
    lens, table = [], []
    for _ in range(n):
        most = min(width, len(ids) // 2) * page
        L = rng.randint(0, min(most, top or most))
        pages = -(-L // page)
        table.append([ids.pop() for _ in range(pages)] + [-9] * (width - pages))
        lens.append(L)
    return lens, table, ids + [-7] * (nb - len(ids)), len(ids)


@pytest.mark.parametrize("n,page,T", [(1, 1, 1), (1, 16, 5), (3, 13, 64), (64, 64, 64), (17, 4, 700), (512, 16, 600), (513, 1, 4097), (1300, 16, 5000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(n, page, T, in_place):
    rng = random.Random(n * 1000 + page)
    for kind in ("decode", "chunks", "idle"):
        lens, table, free, count = make(rng, n, page, 40, 45 * n + 8, top=30 * page)
        left, new = T, []
        for i in range(n):
            k = 1 if kind == "decode" else 0 if kind == "idle" else rng.randint(0, 10 * page)
            k = min(k, left, 40 * page - lens[i])
            left -= k
            new.append(k)
        assert not run_case(new, lens, table, free, count, page, T, in_place=in_place)


@pytest.mark.parametrize("n,page", [(1, 16), (5, 1), (40, 13), (700, 4)])
@pytest.mark.parametrize("in_place", [False, True])
def test_ended_sequences_give_their_pages_back(n, page, in_place):
    rng = random.Random(n)
    lens, table, free, count = make(rng, n, page, 24, 30 * n, top=20 * page)
    ended = [int(rng.random() < 0.4) for _ in range(n)]
    ended[0] = 1
    new = [0 if e and rng.random() < 0.5 else rng.randint(0, 3 * page) for e in ended]  # (some begin anew in their place)
    assert not run_case(new, lens, table, free, count, page, sum(new) + 3, ended=ended, in_place=in_place)
    # only returned pages to hand out: the newest first
    used = sum(-(-x // page) for x, e in zip(lens, ended) if not e)
    back = sum(-(-x // page) for x, e in zip(lens, ended) if e)
    run_case(new, lens, table, [-7] * (30 * n), 0, page, sum(new) + 3, ended=ended, in_place=in_place)
    assert used + back > 0
    # none ends after all
    assert not run_case(new, lens, table, free, count, page, sum(new), ended=[0] * n)


def test_no_sequences_and_no_rows():
    run_case([], [], [], [3, 1, 2], 3, 16, 4)
    a = handle(4)
    run_case([0, 0], [5, 0], [[1], [-1]], [0, 0], 1, 16, 0, a=a)
    run_case([0, 0], [5, 0], [[1], [-1]], [0, 0], 1, 16, 4, a=a)
    a.close()


def test_too_few_pages_are_reported_and_the_rows_dropped():
    # sequence 1 needs two pages where one is left; later ones that need none go on, those that need some do not
    bad = run_case([1, 20, 1, 1, 3], [16, 10, 5, 16, 0], [[4, -1, -1], [5, -1, -1], [6, -1, -1], [7, -1, -1], [-1] * 3],
                   [9, 2, 0, 0, 0, 0, 0, 0, 0, 0], 2, 16, 30)
    assert bad == {12}
    assert run_case([1], [0], [[-1]], [0, 0], 0, 16, 1) == {12}


def test_lengths_and_counts_out_of_range():
    tab = [[1, 2], [3, 4], [5, 6], [7, 0]]
    assert run_case([1, -3, 2, 1], [4, 4, 31, 40], tab, list(range(8)), 6, 16, 8) == {11}  # past the table, negative, cached too long
    assert run_case([5, 5, 5], [0, 0, 0], tab[:3], list(range(8)), 8, 16, 12) == {11}      # past row T
    assert run_case([1], [0], [[-1]], [3, 1], 9, 16, 1) == {11}                            # count past the stack
    assert run_case([1], [0], [[-1]], [3, 1], -2, 16, 1) == {11, 12}
    assert run_case([0x7fffffff, 1, 0x7fffffff], [0, 0, 5], tab[:3], list(range(8)), 8, 16, 8) == {11}
    # a stack that is full already: the returned pages are dropped
    assert run_case([0, 0], [20, 1], tab[:2], [0, 1, 2], 2, 16, 1, ended=[1, 1]) == {11}


def test_blocks_out_of_range_are_reported():
    assert run_case([2], [15], [[0, -1]], [5, -3, 99], 3, 16, 2) == {10}  # the block handed out
    assert run_case([2], [3], [[64]], [1, 0, 0], 1, 16, 2) == {10}        # the sequence's own
    assert run_case([2], [3], [[-1]], [1, 0, 0], 1, 16, 2) == {10}


def test_captured_steps_advance_the_state():
    """A captured plan, in place, replayed: sequences grow by one token a step over page ends."""
    page, n = 3, 4
    rng = random.Random(3)
    lens, table, free, count = make(rng, n, page, 20, 90, top=12)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    d = dict(new=t([1] * n), lens=t(lens), table=t(table), free=t(free), count=t([count]))
    cu, slots, pos = t([0] * (n + 1)), t([0] * 8), t([0] * 8)
    a = handle(8)

    def step():
        a.plan_pages(d["new"], d["lens"], d["table"], d["free"], d["count"], page, cu, slots, pos)

    keep = [x.clone() for x in (d["lens"], d["table"], d["free"], d["count"])]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    for x, y in zip((d["lens"], d["table"], d["free"], d["count"]), keep):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(11):
        ref, bad = plan_ref([1] * n, lens, table, free, count, page, 8, [0] * n)
        graph.replay()
        torch.cuda.synchronize()
        assert not bad and slots.tolist() == ref["slots"] and pos.tolist() == ref["positions"] and cu.tolist() == ref["cu"]
        lens, table, free, count = ref["lens"], ref["table"], ref["free"], ref["count"][0]
        assert d["lens"].tolist() == lens and d["table"].tolist() == table and d["count"].tolist() == [count]
    assert a.status() == 0
    a.close()
