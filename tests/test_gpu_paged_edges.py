"""Edges of the paged serving step on the GPU: the page plan's shared memory by
the number of requests, in a fresh process and from several threads; bad pages
of ended requests; rows that are taken again, wherever the split of a step falls."""
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
