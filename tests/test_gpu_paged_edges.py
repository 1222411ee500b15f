"""Edges of the paged serving step on the GPU: the page plan's shared memory by
the number of requests, in a fresh process and from several threads; bad pages
of ended requests; infinities and NaN in rows that some tokens see and others do not; selections
of heads outside their group."""
import random
import subprocess
import sys
import threading

import pytest
import torch

from tests import gpu_util as U
from tests import paged_ref as R
from tests.test_gpu_paged_step import BF, F32, Step, ints, run_plan

pytestmark = pytest.mark.gpu

# n decodes from nothing on pages of 16 rows: every request takes one page, from the top of the stack down.
FRESH = """
import torch
import routed_head_gqa_b200 as g

i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
for n in map(int, {sizes!r}.split()):
    stack, count = torch.arange(n, dtype=torch.int32, device="cuda"), i([n])
    table, slots = torch.full((n, 1), -1, dtype=torch.int32, device="cuda"), i([0] * n)
    out, left, cu, ws = i([0] * n), i([0]), i([0] * (n + 1)), torch.zeros(256, dtype=torch.uint8, device="cuda")
    g.gqe_page_plan(16, i([0] * n), i([1] * n), stack, count, table, out, left, cu, slots, ws)
    assert g.gqe_get_device_status(ws) == g.GQE_OK
    assert slots.tolist() == [16 * p for p in range(n - 1, -1, -1)] and cu.tolist() == list(range(n + 1))
    assert left.item() == 0 and out.tolist() == [1] * n
print("PLANNED")
"""


def test_plan_around_the_default_shared_memory():
    """4061 to 4096 requests, whose three prefix sums lie about the 48 KB that a kernel has without opting in, static
    shared memory included.  In a process that has planned nothing larger: the opt-in outlasts a call."""
    proc = subprocess.run([sys.executable, "-c", FRESH.format(sizes="4061 4062 4080 4095 4096")], capture_output=True, text=True, timeout=300)
    assert proc.returncode == 0 and "PLANNED" in proc.stdout, proc.stderr[-2000:]


def test_plans_of_several_sizes_from_several_threads():
    """The opt-in is the same in every call: one thread's cannot lower it between another's and its launch."""
    g = U.gqe()
    wrong = {}

    def work(n):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            stack, count, table = torch.arange(n, dtype=torch.int32, device="cuda"), ints([n]), torch.full((n, 1), -1, dtype=torch.int32, device="cuda")
            lengths, new, out, left = ints([0] * n), ints([1] * n), ints([0] * n), ints([0])
            cu, slots, ws = ints([0] * (n + 1)), ints([0] * n), torch.zeros(256, dtype=torch.uint8, device="cuda")
            stream.synchronize()
            tensors = [t.data_ptr() for t in (lengths, new, stack, count, table, out, left, cu, slots, ws)]
            codes = set()
            for i in range(20000):  # about 1 call in 100 of the larger sizes was refused
                codes.add(g._lib.gqe_page_plan(n, n, 16, n, 1, *tensors, 256, stream.cuda_stream))
                if i % 200 == 199:
                    stream.synchronize()
            if codes != {g.GQE_OK} or g.gqe_get_device_status(ws) != g.GQE_OK or slots.tolist() != [16 * p for p in range(n - 1, -1, -1)]:
                wrong[n] = codes

    threads = [threading.Thread(target=work, args=(n,)) for n in (5000, 9000, 16383, 16384)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


@pytest.mark.parametrize("page", [-1, 12, 2 ** 31 - 1])
def test_plan_reports_bad_pages_of_an_ended_request(page):
    """An ended request whose block table holds an entry outside the pool: reported in the step that pushes it, not in
    the later one of another request that takes it.  Everything else of the plan is as if the entry were a page."""
    g = U.gqe()
    lengths, new, free = [5, 3, 4], [1, -1, 1], [9, 8]
    table = [[0, 1, -1], [page, -1, -1], [3, -1, -1]]
    fp, bt, lo, fo, cu, slots, status = run_plan(g, 4, 12, 2, lengths, [1, -1, 0], free, table)
    assert status == g.GQE_ERR_INVALID_ARGUMENT
    assert lo == [6, 0, 4] and fo == 3 and fp[:3] == [9, 8, page] and bt == table and slots == [5, -1]
    # taken in the same step as well: request 2 starts its second page
    fp, bt, lo, fo, cu, slots, status = run_plan(g, 4, 12, 2, lengths, new, free, table)
    assert status == g.GQE_ERR_INVALID_ARGUMENT and lo == [6, 0, 5] and fo == 2 and slots == [5, -1]
    # a block behind the request's last row is not pushed, and so not looked at
    table[1] = [2, page, page]
    assert run_plan(g, 4, 12, 2, lengths, new, free, table)[-1] == g.GQE_OK


# ------------------------------------------------------------------ attention
def group_rows(st, b, q, tokens):
    """[T, h, d] mask of the selected heads of group q of request b's new tokens (a range)."""
    hit = torch.zeros_like(st.O, dtype=torch.bool)
    for i in tokens:
        t = st.cu[b] + i
        hit[t, st.idx[t, q].long()] = True
    return hit


def within(st, clean, sel):
    """st.O is within the tolerance of the formula on clean's inputs where sel."""
    O, mag, wob = R.attention(clean.Q, clean.K, clean.V, clean.table, clean.cu, clean.lengths, st.window, st.sinks, clean.idx, clean.gate)
    n = st.cu[-1]
    err, tol = (st.O[:n].double() - O[:n]).abs(), R.tolerance(O, mag, wob, st.dtype, max(st.lengths))[:n]
    return bool((err <= tol)[sel[:n]].all())


@pytest.mark.parametrize("kw", [dict(d=64), dict(gr=3, h=9, d=32), dict(dtype=F32, d=32, gr=3, h=9)], ids=["bf16", "bf16 3 groups", "f32 3 groups"])
def test_rows_are_taken_again_wherever_the_split_falls(kw):
    """In steps whose parts begin and end anywhere, the last new token of each chunk has values of NaN; the rows before
    it, of whole units and of split ones, are as without them.  The merge has to find the units that the tile kernel
    found."""
    for seed in range(12):
        r = random.Random(seed)
        n = r.randint(3, 160)
        new = [r.choice([1, r.randint(2, 30), r.randint(2, 150)]) for _ in range(n)]
        step = dict(new=new, ctx=[r.randint(0, 700) for _ in range(n)], k=r.choice([1, 2, 3]), ps=r.choice([4, 16, 64]), window=r.choice([0, 0, 130]),
                    sinks=3, seed=seed, **kw)
        st, clean = Step(U.gqe(), **step), Step(U.gqe(), **step)
        sees = torch.zeros_like(st.O, dtype=torch.bool)
        for b, a in enumerate(new):
            st.V.view(-1, *st.V.shape[2:])[st.rows_of(b)[-1]] = float("nan")
            for q in range(st.idx.shape[1]):
                sees |= group_rows(st, b, q, [a - 1])
        st.run()
        assert st.status() == 0
        assert torch.equal(torch.isnan(st.O), sees), step
        assert within(st, clean, ~sees), step


def test_prompt_whose_cost_needs_more_than_24_bits():
    """150000 tokens of one request, whose units see 45 million keys together: the fp32 costs that place the split are
    rounded.  At once as in parts, beside decodes."""
    kw = dict(h=2, gr=1, d=32, k=1, ps=64, seed=17)
    n, cuts = 150000, (0, 40001, 90003, 150000)
    st = Step(U.gqe(), new=[1, n, 1], ctx=[70, 0, 9], **kw)
    st.run()
    parts = torch.full_like(st.O, 7)
    for a, b in zip(cuts, cuts[1:]):
        part = Step(U.gqe(), new=[b - a], ctx=[a], **kw)
        part.K, part.V, part.bt = st.K, st.V, st.bt[1:2].contiguous()
        part.Q, part.idx, part.gate = (x[1 + a:1 + b].contiguous() for x in (st.Q, st.idx, st.gate))
        part.run()
        assert part.status() == 0
        parts[1 + a:1 + b] = part.O
    assert st.status() == 0
    # as in the test of 20000 tokens: |V| <= 6, each side rounds the weights and the result to half a step
    assert (st.O[1:1 + n].float() - parts[1:1 + n].float()).abs().max().item() <= 2 * 2 * 2.0 ** -8 * 6


SHAPES = {"bf16": dict(ps=16), "bf16 d64 ps4": dict(d=64, ps=4), "bf16 window": dict(window=150, sinks=6), "f32": dict(dtype=F32, d=64), "f32 window": dict(dtype=F32, d=32, window=70)}


@pytest.mark.parametrize("kw", SHAPES.values(), ids=SHAPES)
def test_what_rows_see_spoils_its_own_elements_only(kw):
    """A NaN in one element of a value that all rows of a request see, and an infinity in another: those elements of the
    group's selected heads are not finite, every other one is the same bit for bit.  Nothing is taken again."""
    kw = dict(new=[60, 1, 300, 1, 7], ctx=[400, 700, 900, 6000, 33], seed=21, **kw)
    st, clean = Step(U.gqe(), **kw), Step(U.gqe(), **kw)
    hit = torch.zeros_like(st.O, dtype=torch.bool)
    for b in range(5):
        row = st.rows_of(b)[kw["ctx"][b] - 3 if not st.window else st.lengths[b] - 1]
        if st.window and kw["new"][b] > 1:
            continue
        st.V.view(-1, *st.V.shape[2:])[row, 1, 3] = float("nan")
        st.V.view(-1, *st.V.shape[2:])[row, 1, 17] = float("inf")
        hit |= group_rows(st, b, 1, range(kw["new"][b]))
    hit[:, :, [i for i in range(hit.shape[2]) if i not in (3, 17)]] = False
    st.run()
    clean.run()
    assert st.status() == 0 and hit.any()
    assert torch.equal(~torch.isfinite(st.O), hit)
    assert torch.equal(st.O[~hit], clean.O[~hit])


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype,d,ctx", [(BF, 128, 900), (BF, 32, 6000), (F32, 64, 900)], ids=["bf16", "bf16 d32", "f32"])
def test_values_at_both_edges_of_a_window(dtype, d, ctx, value):
    """Rows near a value that is not finite, in cached keys that the window is leaving and in new ones: each row has it if
    it sees it.  Elements of one value are mixed: rows that see the one do not see the other."""
    kw = dict(new=[300, 5, 1], ctx=[ctx, 90, 400], window=150, sinks=4, d=d, dtype=dtype, k=3, h=10, seed=22)
    st, clean = Step(U.gqe(), **kw), Step(U.gqe(), **kw)
    hit = torch.zeros_like(st.O, dtype=torch.bool)
    planted = [(0, ctx - 100, 0, 5), (0, ctx + 37, 0, 5), (0, ctx + 210, 0, 9), (0, ctx + 211, 1, 9), (0, 3, 1, 30), (1, 92, 0, 7), (1, 2, 1, 8)]
    for b, key, q, e in planted:
        st.V.view(-1, *st.V.shape[2:])[st.rows_of(b)[key], q, e] = value
        first = st.lengths[b] - kw["new"][b]
        seen = [i for i in range(kw["new"][b]) if key <= first + i and (key > first + i - 150 or key < 4)]
        rows = group_rows(st, b, q, seen)
        rows[:, :, [x for x in range(d) if x != e]] = False
        hit |= rows
    st.run()
    assert st.status() == 0
    assert torch.equal(~torch.isfinite(st.O), hit)
    assert within(st, clean, ~hit)
    first = st.O.clone()
    st.run()
    assert torch.equal(torch.nan_to_num(first.float(), nan=77.0), torch.nan_to_num(st.O.float(), nan=77.0)), "two runs differ"


@pytest.mark.parametrize("which", ["every value of one old key", "one element", "half of the new rows", "the last new row"])
@pytest.mark.parametrize("new", [[2048], [1] * 64], ids=["prompt", "decodes"])
def test_a_request_of_nan_does_not_hold_up_the_step(new, which):
    """A step with NaN takes the time of the step without, within a factor (2 to 13 for the prompt, 1 for the decodes).
    When each row that is not finite took its whole cache again, the prompt took 570 to 790 times as long and the
    decodes 20 to 80."""
    st = Step(U.gqe(), new=new, ctx=[12000 if len(new) == 1 else 8000] * len(new), h=32, gr=8, k=2, ps=64, seed=23)

    def timed():
        st.run()
        best = 1e9
        for _ in range(3):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            st.run()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best

    clean = timed()
    rows, K, V = st.rows_of(0), st.K.view(-1, 8, 128), st.V.view(-1, 8, 128)
    if which == "one element":
        V[rows[5], :, 3] = float("nan")
    elif which == "half of the new rows":
        K[rows[-((new[0] + 1) // 2):]] = V[rows[-((new[0] + 1) // 2):]] = float("nan")
    else:
        V[rows[5 if which.startswith("every") else -1]] = float("nan")
    assert timed() <= 40 * clean
    assert st.status() == 0


HEADS = {"decodes": dict(new=[1] * 9, ctx=[400, 0, 127, 700, 63, 64, 5, 1290, 90]), "split decode": dict(new=[1], ctx=[30000], ps=64),
         "chunks": dict(new=[40, 3, 300, 1, 129], ctx=[60, 50, 10, 800, 0], pad=2), "split chunks": dict(new=[200, 256], ctx=[9000, 3000], ps=64),
         "decodes k8": dict(new=[1, 2, 1], ctx=[500, 90, 3], h=16, k=8), "d32 ps4": dict(new=[20, 1, 130], ctx=[0, 90, 200], d=32, ps=4, k=3, h=10),
         "window": dict(new=[200, 1], ctx=[700, 300], window=90, sinks=4, d=64)}


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", HEADS)
def test_bad_heads_are_skipped(name, dtype):
    """Selections outside their group, in first, last and middle tokens and slots: reported; every other selection of the
    same token and all other tokens as they are, and every slot that no good selection names is 0."""
    g = U.gqe()
    st = Step(g, seed=31, **{**HEADS[name], "dtype": dtype})
    clean = Step(g, seed=31, **{**HEADS[name], "dtype": dtype})
    T, gr, k = st.cu[-1], st.idx.shape[1], st.idx.shape[2]
    h = st.O.shape[1]
    r = random.Random(name)
    bad = [(0, 0, 0, -1), (T - 1, gr - 1, k - 1, h)]
    bad += [(r.randrange(T), r.randrange(gr), r.randrange(k), None) for _ in range(min(T // 8, 40))]
    for t, q, slot, j in bad:
        others = [x for x in (2 ** 31 - 1, -2 ** 31, (q + 1) * (h // gr), q * (h // gr) - 1) if j is None]
        st.idx[t, q, slot] = r.choice(others) if others else j
    st.run()
    assert st.status() == g.GQE_ERR_INVALID_ARGUMENT
    first = torch.arange(gr, device="cuda")[:, None] * (h // gr)
    good = (st.idx >= first) & (st.idx < first + h // gr)
    named = torch.zeros(st.O.shape[0], h, dtype=torch.bool, device="cuda")
    for slot in range(k):
        for q in range(gr):
            t = good[:T, q, slot].nonzero().flatten()
            named[t, st.idx[t, q, slot].long()] = True
    assert (st.O[:T][~named[:T]] == 0).all()
    assert (st.O[T:] == 7).all()
    assert within(st, clean, named[:, :, None].expand_as(st.O))
    # a bad selection changes nothing else, bit for bit
    clean.run()
    assert torch.equal(st.O[named], clean.O[named])


@pytest.mark.parametrize("kw", [dict(), dict(dtype=F32, d=32), dict(k=1, d=64, ps=4)], ids=["bf16", "f32", "bf16 ps4"])
@pytest.mark.parametrize("ends", [(2 ** 31 - 10, -2 ** 31), (-5, 9), (60, 20), (2 ** 31 - 1, 0)])
def test_bad_requests_beside_spoilt_rows(kw, ends):
    """Requests whose row ranges contradict each other (differences of two that wrap to a small length among them) beside
    some whose rows are taken again: skipped by that as well."""
    new, ctx = [30, 8, 8, 8, 30], [50, 100, 100, 100, 7]
    st, clean = Step(U.gqe(), new=new, ctx=ctx, seed=41, **kw), Step(U.gqe(), new=new, ctx=ctx, seed=41, **kw)
    for b in (0, 4):
        st.V.view(-1, *st.V.shape[2:])[st.rows_of(b)[-1]] = float("nan")
    st.cu_d[2], st.cu_d[3] = ends
    st.run()
    assert st.status() == st.g.GQE_ERR_INVALID_ARGUMENT
    sees = torch.zeros_like(st.O, dtype=torch.bool)
    for b in (0, 4):
        for q in range(st.idx.shape[1]):
            sees |= group_rows(st, b, q, [new[b] - 1])
    # The rows of requests 0 and 4, but for those that a range which does not contradict itself claims as well: a request
    # between two bad ones may own any rows.
    cu, T = st.cu_d.tolist(), st.cu[-1]
    kept = torch.zeros_like(sees)
    kept[:st.cu[1]] = kept[st.cu[4]:] = True
    for b in (1, 2, 3):
        if 0 <= cu[b] <= cu[b + 1] <= T and cu[b + 1] - cu[b] <= st.lengths[b]:
            kept[cu[b]:cu[b + 1]] = False
    assert kept.any() and torch.isnan(st.O[kept & sees]).all()
    assert within(st, clean, kept & ~sees)
