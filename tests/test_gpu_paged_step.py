"""The paged serving step on the GPU: gqe_page_plan, gqe_kv_append and
gqe_attn_chunk_paged against the plain implementations of tests/paged_ref.py
(tolerances derived there), their device-side refusals, and a run of them
together: prompts fed in chunks against the dense prefill."""
import random

import pytest
import torch

import gqe_synth
from tests import gpu_util as U
from tests import paged_ref as R

pytestmark = pytest.mark.gpu
INT = dict(dtype=torch.int32, device="cuda")


def ints(v):
    return torch.tensor(v, **INT)


# ------------------------------------------------------------------ plan
def plan_state(seed, n, ps, max_blocks, ctx_hi, spare=5):
    r = random.Random(seed)
    lengths = [r.choice([0, r.randint(0, ctx_hi), ps * r.randint(0, ctx_hi // ps)]) for _ in range(n)]
    used = sum(-(-x // ps) for x in lengths)
    num_pages = used + spare
    order = list(range(num_pages))
    r.shuffle(order)
    table, at = [], 0
    for x in lengths:
        m = -(-x // ps)
        table.append(order[at:at + m] + [-1] * (max_blocks - m))
        at += m
    return r, lengths, order[used:], table, num_pages


def run_plan(g, ps, num_pages, rows, lengths, new, free, table):
    """Returns the device results and the status."""
    n = len(lengths)
    fp = torch.full((num_pages,), -7, **INT)
    fp[:len(free)] = ints(free) if free else fp[:0]
    bt = ints(table)
    lo, fo, cu, slots = torch.full((n,), -9, **INT), ints([-9]), torch.full((n + 1,), -9, **INT), torch.full((rows,), -9, **INT)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for _ in range(2):  # a repeated call gives the same result
        g.gqe_page_plan(ps, ints(lengths), ints(new), fp, ints([len(free)]), bt, lo, fo, cu, slots, ws)
    return fp.tolist(), bt.tolist(), lo.tolist(), fo.item(), cu.tolist(), slots.tolist(), g.gqe_get_device_status(ws)


@pytest.mark.parametrize("n,ps,new_hi,pad", [(1, 1, 5, 0), (1, 65536, 3, 1), (3, 16, 40, 2), (37, 8, 1, 0), (513, 4, 9, 11),
                                             (3000, 16, 30, 100), (16384, 32, 2, 1)])
def test_plan(n, ps, new_hi, pad):
    g = U.gqe()
    ctx_hi = 3 * ps if ps > 1000 else 6 * ps + 5
    max_blocks = -(-(ctx_hi + new_hi) // ps) + 1
    r, lengths, free, table, num_pages = plan_state(n + ps, n, ps, max_blocks, ctx_hi, spare=n * (new_hi // ps + 2))
    new = [r.choice([-1, 0, 1, r.randint(0, new_hi), r.randint(0, new_hi)]) for _ in range(n)]
    rows = sum(max(a, 0) for a in new) + pad
    want_table = [list(x) for x in table]
    out, stack, cu, slots, pushed = R.plan(ps, num_pages, max_blocks, rows, lengths, new, list(free), want_table)
    fp, bt, lo, fo, cu_g, slots_g, status = run_plan(g, ps, num_pages, rows, lengths, new, free, table)
    assert status == 0
    assert lo == out and fo == len(stack) and cu_g == cu and slots_g == slots and bt == want_table
    assert fp[:len(stack)] == stack
    assert fp == (list(free) + pushed + [-7] * num_pages)[:num_pages]  # pushed on top, nothing else written


def test_plan_without_rows():
    g = U.gqe()
    fp, bt, lo, fo, cu, slots, status = run_plan(g, 4, 6, 0, [5, 3], [-1, 0], [4, 5], [[0, 1], [2, -1]])
    assert (status, lo, fo, cu, slots) == (0, [0, 3], 4, [0, 0, 0], []) and fp[:4] == [4, 5, 0, 1]


@pytest.mark.parametrize("case", ["pages", "negative", "below", "long", "rows", "stack", "huge"])
def test_plan_refused_as_a_whole(case):
    g = U.gqe()
    lengths, new, free, rows, num_pages = [5, 3, 8], [1, -1, 4], [9, 8], 7, 12
    table = [[0, 1, -1, -1], [2, -1, -1, -1], [3, 4, -1, -1]]
    if case == "pages":
        new, rows = [11, 0, 8], 19
        free = [9]
    elif case == "negative":
        lengths = [5, -3, 8]
    elif case == "below":
        new = [1, -2, 4]
    elif case == "long":
        new, rows = [1, 0, 9], 10  # 17 rows in 4 blocks of 4
    elif case == "rows":
        rows = 4
    elif case == "stack":
        num_pages = 2
    elif case == "huge":
        new = [2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1]
    fp, bt, lo, fo, cu, slots, status = run_plan(g, 4, num_pages, rows, lengths, new, free, table)
    assert status == (g.GQE_ERR_OUT_OF_PAGES if case == "pages" else g.GQE_ERR_INVALID_ARGUMENT)
    assert bt == table and lo == lengths and fo == len(free) and cu == [0, 0, 0, 0] and slots == [-1] * rows
    assert fp == free + [-7] * (num_pages - len(free))


def test_plan_reports_bad_pages():
    g = U.gqe()
    # the page on top of the stack and request 1's only page are outside the pool
    fp, bt, lo, fo, cu, slots, status = run_plan(g, 4, 12, 4, [4, 2], [2, 2], [3, 77], [[0, -1], [-5, -1]])
    assert status == g.GQE_ERR_INVALID_ARGUMENT and slots == [-1, -1, -1, -1] and lo == [6, 4]


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype,gr,d,ps,rows,sliced", [(torch.bfloat16, 8, 128, 16, 33, True), (torch.float32, 2, 32, 1, 7, False),
                                                       (torch.bfloat16, 1, 32, 64, 1, False), (torch.float32, 8, 128, 4, 500, True),
                                                       (torch.bfloat16, 3, 64, 8, 130, True), (torch.bfloat16, 5, 8, 8, 9, False)])
def test_append(dtype, gr, d, ps, rows, sliced):
    g = U.gqe()
    gen = torch.Generator(device="cuda").manual_seed(rows)
    pages = -(-rows // ps) + 3
    src = torch.randn(rows, 4 * gr, d, device="cuda", generator=gen).to(dtype)
    K_new, V_new = (src[:, gr:2 * gr], src[:, 3 * gr:]) if sliced else (src[:, :gr].contiguous(), src[:, gr:2 * gr].contiguous())
    slots = torch.randperm(pages * ps, device="cuda", generator=gen)[:rows].to(torch.int32)
    if rows > 3:
        slots[::3] = -1
    K, V = (torch.randn(pages, ps, gr, d, device="cuda", generator=gen).to(dtype) for _ in range(2))
    want_K, want_V = K.clone(), V.clone()
    keep = slots >= 0
    want_K.view(-1, gr, d)[slots[keep].long()] = K_new[keep]
    want_V.view(-1, gr, d)[slots[keep].long()] = V_new[keep]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    shape = g.make_shape(1, rows, 64, gr, gr, d, 1, dtype)
    g.gqe_kv_append(shape, K_new, V_new, slots, K, V, ws)
    assert g.gqe_get_device_status(ws) == 0
    assert torch.equal(K, want_K) and torch.equal(V, want_V)
    slots[0] = pages * ps  # past the pool: reported, the others still written
    K.zero_()
    g.gqe_kv_append(shape, K_new, V_new, slots, K, V, ws)
    assert g.gqe_get_device_status(ws) == g.GQE_ERR_INVALID_ARGUMENT
    keep[0] = False
    assert torch.equal(K.view(-1, gr, d)[slots[keep].long()], K_new[keep])


# ------------------------------------------------------------------ attention
class Step:
    """Inputs of one step: requests with `new` tokens after `ctx` cached ones, pages in random order."""

    def __init__(self, g, new, ctx, h=8, gr=2, d=128, k=2, ps=16, dtype=torch.bfloat16, window=0, sinks=0, pad=0, seed=0,
                 scale=1.0):
        self.g, self.window, self.sinks, self.dtype, self.ps = g, window, sinks, dtype, ps
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.lengths = [a + c for a, c in zip(new, ctx)]
        self.cu = [0]
        for a in new:
            self.cu.append(self.cu[-1] + a)
        T = self.cu[-1] + pad
        blocks = [-(-x // ps) for x in self.lengths]
        self.num_pages = sum(blocks) + 2
        order = torch.randperm(self.num_pages, device="cuda", generator=gen).tolist()
        self.table, at = [], 0
        for m in blocks:
            self.table.append(order[at:at + m] + [-1] * (max(blocks) + 1 - m))
            at += m
        rnd = lambda *s: (torch.randn(*s, device="cuda", generator=gen) * scale).to(dtype)  # noqa: E731
        self.K, self.V = rnd(self.num_pages, ps, gr, d), rnd(self.num_pages, ps, gr, d)
        self.Q = rnd(T, h, d)
        pick = torch.rand(T, gr, h // gr, device="cuda", generator=gen).argsort(-1)[..., :k]
        self.idx = (pick + torch.arange(gr, device="cuda")[:, None] * (h // gr)).to(torch.int32).contiguous()
        self.gate = torch.softmax(torch.randn(T, gr, k, device="cuda", generator=gen), -1)
        self.shape = g.make_shape(1, T, 64, h, gr, d, k, dtype)
        self.ws = torch.zeros(g.gqe_chunk_workspace_bytes(self.shape), dtype=torch.uint8, device="cuda")
        self.ws[256:] = 0xFF  # whatever the scratch held before
        self.O = torch.full((T, h, d), 7.0, dtype=dtype, device="cuda")
        self.bt, self.cu_d, self.len_d = ints(self.table), ints(self.cu), ints(self.lengths)

    def rows_of(self, b):
        """Flat page rows of request b's logical rows."""
        return torch.tensor([self.table[b][p // self.ps] * self.ps + p % self.ps for p in range(self.lengths[b])], device="cuda")

    def run(self, stream=None):
        self.g.gqe_attn_chunk_paged(self.shape, self.Q, self.K, self.V, self.bt, self.cu_d, self.len_d, self.window,
                                    self.sinks, self.idx, self.gate, self.O, self.ws, stream)

    def status(self):
        return self.g.gqe_get_device_status(self.ws)

    def check(self, skip=()):
        O, mag, wob = R.attention(self.Q, self.K, self.V, self.table, self.cu, self.lengths, self.window, self.sinks,
                                  self.idx, self.gate)
        tol = R.tolerance(O, mag, wob, self.dtype, max(self.lengths))
        n = self.cu[-1]
        assert (self.O[n:] == 7).all(), "rows behind the last request were written"
        for b in range(len(self.lengths)):
            rows = slice(self.cu[b], self.cu[b + 1])
            if b in skip:
                assert (self.O[rows] == 7).all(), f"request {b} was to be skipped"
                continue
            err = (self.O[rows].double() - O[rows]).abs()
            assert (err <= tol[rows]).all(), f"request {b}: worst error / tolerance {(err / tol[rows]).max().item():.3g}"


BF, F32 = torch.bfloat16, torch.float32
STEPS = {
    "one token": dict(new=[1], ctx=[0]),
    "decode": dict(new=[1] * 5, ctx=[0, 1, 127, 128, 700]),
    "decode k1 ps1": dict(new=[1] * 4, ctx=[3, 63, 64, 200], k=1, ps=1),
    "decode k8": dict(new=[1, 1], ctx=[500, 90], h=16, gr=2, k=8),
    "decode long": dict(new=[1], ctx=[30000], ps=64),
    "decode many": dict(new=[1] * 200, ctx=[(37 * i) % 301 for i in range(200)], h=4, gr=2, k=1),
    "chunk from nothing": dict(new=[1, 2, 64, 65, 200], ctx=[0] * 5),
    "chunk on a cache": dict(new=[130, 7, 1], ctx=[301, 1000, 64], pad=9),
    "chunk long": dict(new=[700], ctx=[2500], ps=256),
    "chunk k3": dict(new=[50, 43, 300], ctx=[10, 0, 77], h=12, gr=2, k=3, ps=8),
    "chunk k16": dict(new=[20, 9], ctx=[100, 5], h=32, gr=2, k=16, ps=4),
    "one group of 64": dict(new=[33], ctx=[40], h=64, gr=1, k=5, ps=2),
    "idle requests": dict(new=[0, 3, 0, 0, 70, 0], ctx=[50, 8, 0, 1, 99, 4], pad=3),
    "mixed": dict(new=[1, 90, 1, 1, 257, 1], ctx=[800, 0, 64, 1, 900, 1290], h=32, gr=8, k=2, pad=1),
    "window 1": dict(new=[1, 40], ctx=[90, 3], window=1),
    "window sinks": dict(new=[1, 1, 130], ctx=[900, 10, 400], window=100, sinks=3, ps=8),
    "window beyond": dict(new=[20, 1], ctx=[30, 60], window=1000, sinks=5),
    "window many sinks": dict(new=[70, 1, 1], ctx=[500, 333, 129], window=64, sinks=130, ps=4),
    "window ps1": dict(new=[5, 1, 200], ctx=[300, 400, 100], window=33, sinks=1, ps=1),
    "window 128": dict(new=[300, 1], ctx=[513, 640], window=128, sinks=128, ps=32, k=4, h=8),
    "window long": dict(new=[1, 64], ctx=[20000, 9000], window=4096, sinks=16, ps=64),
    "f32 decode": dict(new=[1, 1, 1], ctx=[300, 0, 64], dtype=F32),
    "f32 chunk": dict(new=[65, 3], ctx=[200, 31], dtype=F32, pad=2),
    "f32 d32": dict(new=[40, 1, 17], ctx=[0, 90, 64], dtype=F32, d=32, k=1, ps=8),
    "f32 d64 window": dict(new=[30, 1], ctx=[300, 200], dtype=F32, d=64, window=50, sinks=2, ps=2),
    "bf16 d64": dict(new=[65, 1, 300], ctx=[10, 700, 64], d=64, k=3, h=12),
    "bf16 d64 window": dict(new=[65, 1, 300], ctx=[10, 700, 64], d=64, window=70, sinks=4),
    "bf16 d32": dict(new=[33, 1], ctx=[100, 500], d=32, k=4, ps=4),
    # more requests than a block has threads: each thread of the split sums several
    "many requests": dict(new=[1] * 700 + [20] + [0, 3, 1] * 100, ctx=[(29 * i) % 97 for i in range(1001)], h=4, gr=2, k=1, pad=2),
    "many chunks": dict(new=[(i * 7) % 41 for i in range(530)], ctx=[(13 * i) % 150 for i in range(530)], h=4, gr=2, k=2, ps=32),
    # every block goes from one kind of unit to the other, in either order
    "many chunks k1 ps4": dict(new=[(i * 7) % 41 for i in range(530)], ctx=[(13 * i) % 150 for i in range(530)], h=8, gr=2, k=1, ps=4),
    "many chunks d64": dict(new=[(i * 7) % 41 for i in range(300)], ctx=[(113 * i) % 450 for i in range(300)], h=4, gr=2, k=2, d=64),
    "many chunks long": dict(new=[(i * 17) % 91 if i % 3 else 1 for i in range(300)], ctx=[(113 * i) % 450 for i in range(300)], h=16, gr=4, k=4, ps=64),
    "f32 many requests": dict(new=[1, 2, 1, 9] * 200, ctx=[(31 * i) % 90 for i in range(800)], h=4, gr=2, k=1, d=32, dtype=F32),
    # several items of both kinds for every block, some of them split
    "many items": dict(new=[1] * 300 + [70, 3, 200], ctx=[500 + (17 * i) % 300 for i in range(303)], h=16, gr=4, k=2, ps=32),
    "many items ps4": dict(new=[1] * 200 + [150, 3, 300], ctx=[300 + (17 * i) % 300 for i in range(203)], h=16, gr=4, k=2, ps=4),
    "many items f32": dict(new=[1] * 150 + [33, 5, 150], ctx=[300 + (17 * i) % 300 for i in range(153)], h=8, gr=4, k=1, d=64, dtype=F32),
    # copied pages (fewer than 16 rows), every head width, 5 .. 16 and 17 .. 128 query rows beside decodes and prompts
    **{f"rows d{d} ps{ps}": dict(new=[1, 90, 3, 1, 257, 8, 9, 64, 65], ctx=[400, 0, 64, 1, 700, 290, 130, 5, 127], d=d, ps=ps)
       for d, ps in ((128, 1), (128, 8), (64, 1), (64, 8), (32, 2), (32, 16))},
    **{f"rows window d{d} ps{ps}": dict(new=[1, 90, 3, 1, 257, 8], ctx=[400, 0, 364, 1, 700, 290], d=d, ps=ps, window=140,
                                        sinks=9, k=3, h=14) for d, ps in ((128, 2), (64, 4), (32, 1))},
    "f32 few rows": dict(new=[1, 2, 3, 4, 5, 16, 17], ctx=[200, 65, 190, 63, 0, 9, 300], k=1, dtype=F32, ps=8),
    "f32 few rows window": dict(new=[1, 2, 3, 4, 1], ctx=[200, 65, 190, 63, 700], k=1, dtype=F32, d=64, ps=1, window=40, sinks=70),
    "f32 k4": dict(new=[1, 1, 1], ctx=[129, 64, 63], h=8, gr=2, k=4, d=32, dtype=F32),
    "heads of 256": dict(new=[1, 20], ctx=[90, 200], h=256, gr=1, k=16, d=64),
    "f32 heads of 256": dict(new=[1, 20], ctx=[90, 200], h=256, gr=2, k=3, d=32, dtype=F32),
    "page of 4096": dict(new=[1, 100], ctx=[5000, 100], ps=4096),
    "peaked": dict(new=[40, 1], ctx=[400, 300], scale=4.0),
}


@pytest.mark.parametrize("name", STEPS)
def test_attention(name):
    st = Step(U.gqe(), **STEPS[name], seed=len(name))
    st.run()
    assert st.status() == 0
    st.check()
    first = st.O.clone()
    st.run()
    assert torch.equal(first, st.O), "two runs differ"


@pytest.mark.parametrize("kw", [dict(), dict(dtype=F32, d=64), dict(d=64)], ids=["bf16 d128", "f32 d64", "bf16 d64"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_unseen_rows_are_not_read(kw, value):
    """Rows past a cache's length, unused pages, and rows that the window has left hold NaN or infinities, and the
    entries of pages that the window has left are stale."""
    st = Step(U.gqe(), new=[1, 60, 1, 3], ctx=[500, 333, 17, 250], window=90, sinks=5, ps=16, seed=4, **kw)
    seen = torch.zeros(st.num_pages * st.ps, dtype=torch.bool, device="cuda")
    for b, L in enumerate(st.lengths):
        first = L - (st.cu[b + 1] - st.cu[b])
        rows = st.rows_of(b)
        at = torch.arange(L, device="cuda")
        see = (at > first - st.window) | (at < st.sinks)
        seen[rows[see]] = True
        for j in range(-(-L // st.ps)):
            if not see[j * st.ps:(j + 1) * st.ps].any():
                st.table[b][j] = 10 ** 6
    st.bt = ints(st.table)
    for x in (st.K, st.V):
        x.view(-1, *x.shape[2:])[~seen] = value
    st.run()
    assert st.status() == 0
    assert torch.isfinite(st.O.float()).all()
    st.check()


@pytest.mark.parametrize("kw", [dict(), dict(dtype=F32, d=32), dict(new=[400], ctx=[300])], ids=["bf16 d128", "f32 d32", "long"])
@pytest.mark.parametrize("which", ["K", "V", "inf V"])
def test_later_tokens_do_not_reach_earlier_rows(kw, which):
    """A NaN or infinity in one new token's key or value reaches the rows that see it and no others."""
    kw = {**dict(new=[70, 5], ctx=[100, 9]), **kw}
    st = Step(U.gqe(), seed=11, **kw)
    clean = Step(U.gqe(), seed=11, **kw)
    at = 40
    row = st.rows_of(0)[kw["ctx"][0] + at]
    x = st.K if which == "K" else st.V
    x.view(-1, *x.shape[2:])[row, 0, 3] = float("inf") if which == "inf V" else float("nan")
    st.run()
    clean.run()
    assert st.status() == 0
    hpg = 4
    hit = torch.zeros_like(st.O, dtype=torch.bool)
    for t in range(at, kw["new"][0]):
        for j in st.idx[t, 0].tolist():
            hit[t, j, slice(None) if which == "K" else 3] = True
    assert (hit[:, hpg:] == 0).all()
    bad = ~torch.isfinite(st.O.float())
    assert torch.equal(bad, hit)
    # the others as without it (a row that was taken again sums in another order)
    O, mag, wob = R.attention(clean.Q, clean.K, clean.V, clean.table, clean.cu, clean.lengths, 0, 0, clean.idx, clean.gate)
    tol = R.tolerance(O, mag, wob, st.dtype, max(st.lengths))
    n = st.cu[-1]
    ok = ~hit[:n] if which != "K" else ~hit[:n]
    assert ((st.O[:n].double() - O[:n]).abs() <= tol[:n])[ok].all()


@pytest.mark.parametrize("kw", [dict(), dict(ps=4, d=64), dict(dtype=F32, d=64)], ids=["bf16", "bf16 ps4", "f32"])
def test_one_request_of_nan(kw):
    """A request whose values are all NaN, split over many blocks, leaves the others as they are."""
    st = Step(U.gqe(), new=[1, 300, 1, 1], ctx=[90, 900, 9000, 64], gr=2, seed=12, **kw)
    for b in (1, 2):
        st.V.view(-1, *st.V.shape[2:])[st.rows_of(b)] = float("nan")
    st.run()
    assert st.status() == 0
    O, mag, wob = R.attention(st.Q, st.K, torch.nan_to_num(st.V), st.table, st.cu, st.lengths, 0, 0, st.idx, st.gate)
    tol = R.tolerance(O, mag, wob, st.dtype, max(st.lengths))
    chosen = torch.zeros(O.shape[:2], dtype=torch.bool, device="cuda")
    chosen[torch.arange(O.shape[0], device="cuda")[:, None], st.idx.flatten(1).long()] = True
    for b in (0, 3):
        rows = slice(st.cu[b], st.cu[b + 1])
        assert ((st.O[rows].double() - O[rows]).abs() <= tol[rows]).all()
    for b in (1, 2):
        rows = slice(st.cu[b], st.cu[b + 1])
        assert torch.isnan(st.O[rows][chosen[rows]]).all() and (st.O[rows][~chosen[rows]] == 0).all()


@pytest.mark.parametrize("kw", [dict(ps=64), dict(ps=8), dict(ps=64, dtype=F32)], ids=["pages", "copied pages", "f32"])
def test_cache_offsets_past_32_bits(kw):
    """Pages whose first element is behind 2^31 elements (bf16 rows of 2 KB behind 4 GB; fp32 behind 8 GB)."""
    g = U.gqe()
    st = Step(g, new=[1, 70, 1], ctx=[300, 10, 999], h=16, gr=8, k=1, seed=13, **kw)
    first = (1 << 31) // (st.ps * 8 * 128) + 1
    pages = first + st.num_pages
    big = [torch.empty(pages, *x.shape[1:], dtype=x.dtype, device="cuda") for x in (st.K, st.V)]
    # the requests' rows go in by the append
    rows = sum(st.lengths)
    flat = torch.cat([st.rows_of(b) for b in range(3)])
    slots = (flat + first * st.ps).to(torch.int32)
    src = [x.view(-1, 8, 128)[flat].contiguous() for x in (st.K, st.V)]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    g.gqe_kv_append(g.make_shape(1, rows, 64, 8, 8, 128, 1, st.dtype), *src, slots, *big, ws)
    assert g.gqe_get_device_status(ws) == 0
    small = st.K, st.V
    st.K, st.V = big
    st.bt = torch.where(st.bt >= 0, st.bt + first, st.bt)
    st.run()
    assert st.status() == 0
    st.K, st.V = small
    st.check()


def test_two_calls_at_once():
    """Two steps on two streams, each with its own workspace."""
    g = U.gqe()
    steps = [Step(g, new=[1] * 40 + [100 * i], ctx=[30 * j for j in range(41)], seed=i, window=i and 200, sinks=4) for i in (0, 1)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        for st, s in zip(steps, streams):
            st.run(s)
    torch.cuda.synchronize()
    for st in steps:
        assert st.status() == 0
        st.check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_widest_table(dtype):
    """page_size * max_blocks = 2^30, the largest allowed: the scale of the split's costs and the grid follow it."""
    st = Step(U.gqe(), new=[1, 60, 0], ctx=[900, 70000, 5], h=4, gr=1, d=32, k=2, ps=65536, dtype=dtype, seed=14)
    st.bt = torch.full((3, 1 << 14), -1, **INT)
    for b, pages in enumerate(st.table):
        st.bt[b, :len(pages)] = ints(pages)
    st.run()
    assert st.status() == 0
    st.check()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_idle_requests(dtype):
    """16384 requests of which few have work, the last among them."""
    new = [0] * 16384
    for b in (3, 700, 701, 9000, 16383):
        new[b] = 1 + b % 40
    st = Step(U.gqe(), new=new, ctx=[50 if a else 0 for a in new], h=4, gr=2, d=64, k=1, ps=8, dtype=dtype, pad=3, seed=15)
    st.run()
    assert st.status() == 0
    st.check()


@pytest.mark.parametrize("dtype,window", [(BF, 0), (BF, 300), (F32, 300)])
def test_long_prompt_at_once_and_in_parts(dtype, window):
    """20000 tokens of one request in one call, and the same in two."""
    kw = dict(h=2, gr=1, d=32, k=1, ps=64, dtype=dtype, window=window, sinks=2, seed=16)
    st = Step(U.gqe(), new=[20000], ctx=[0], **kw)
    st.run()
    whole, lengths, parts = st.O.clone(), st.lengths, torch.empty_like(st.O)
    for a, b in ((0, 7001), (7001, 20000)):
        part = Step(U.gqe(), new=[b - a], ctx=[a], **kw)
        part.K, part.V, part.bt = st.K, st.V, st.bt
        part.Q, part.idx, part.gate = (x[a:b].contiguous() for x in (st.Q, st.idx, st.gate))
        part.run()
        assert part.status() == 0
        parts[a:b] = part.O
    assert st.status() == 0 and lengths == [20000]
    # |V| <= 6 here: each side rounds weights and result to half a step, fp32 its sums over at most 20000 keys
    bound = 2 * (2 * 2.0 ** -8 * 6 if dtype == BF else 20000 * 2.0 ** -23 * 6)
    assert (whole.float() - parts.float()).abs().max().item() <= bound


def test_bad_requests_are_reported_and_skipped():
    g = U.gqe()
    for what in ("short", "long", "rows", "backwards"):
        st = Step(g, new=[3, 40, 1], ctx=[50, 60, 70], seed=2)
        if what == "short":
            st.len_d[1] = 39
        elif what == "long":
            st.len_d[1] = st.ps * st.bt.shape[1] + 1
        elif what == "rows":
            st.cu_d[3] = st.Q.shape[0] + 1
        elif what == "backwards":
            st.cu_d[1] = 50
        st.run()
        assert st.status() == g.GQE_ERR_INVALID_ARGUMENT
        if what in ("short", "long"):
            st.check(skip=(1,))
        elif what == "rows":
            st.check(skip=(2,))


def test_bad_heads_and_pages_are_reported():
    g = U.gqe()
    st = Step(g, new=[3, 40], ctx=[50, 60], seed=3)
    st.idx[5, 1, 0] = 0  # a head of group 0 in group 1
    st.run()
    assert st.status() == g.GQE_ERR_INVALID_ARGUMENT
    st = Step(g, new=[3, 40], ctx=[50, 60], seed=3)
    st.bt[1, 2] = st.num_pages  # read as page 0
    st.table[1][2] = 0
    st.run()
    assert st.status() == g.GQE_ERR_INVALID_ARGUMENT
    st.check()


def test_nothing_to_do_writes_nothing():
    st = Step(U.gqe(), new=[0, 0], ctx=[5, 9], pad=4)
    st.run()
    assert st.status() == 0
    st.check()


def test_agrees_with_the_paged_decode():
    g = U.gqe()
    st = Step(g, new=[1] * 6, ctx=[0, 5, 100, 511, 512, 1300], h=32, gr=8, k=2, seed=9)
    st.run()
    dshape = g.make_shape(6, 1, 64, 32, 8, 128, 2, BF)
    ws = torch.zeros(g.gqe_workspace_bytes(dshape, st.ps * st.bt.shape[1]), dtype=torch.uint8, device="cuda")
    O = torch.empty_like(st.O)
    g.gqe_attn_decode_paged(dshape, st.Q, st.K, st.V, st.ps, st.bt, st.len_d, st.idx, st.gate, O, ws)
    st.check()
    st.O = O
    st.check()


def test_another_stream_and_two_graphs():
    g = U.gqe()
    a, b = Step(g, new=[1, 90], ctx=[700, 64], seed=5), Step(g, new=[40] * 3, ctx=[9, 0, 300], window=33, sinks=2, seed=6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a.run(side)
    side.synchronize()
    a.check()
    graphs = []
    for st in (a, b):
        st.run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            st.run()
        graphs.append(graph)
    for st in (a, b):
        st.O.fill_(7)
        st.Q.mul_(-0.5)  # replays read the inputs as they are now
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for st in (a, b):
        assert st.status() == 0
        st.check()


# ------------------------------------------------------------------ together
def test_prompts_in_chunks_match_the_dense_prefill():
    """Three requests' prompts, fed in ragged chunks and then token by token through plan, append and attention, one
    of them replaced half way by a new request that takes its pages, give the rows of the dense prefill."""
    g = U.gqe()
    h, gr, d, k, T, dm = 32, 8, 128, 2, 150, 256
    w = gqe_synth.custom("serve", B=4, T=T, d_model=dm, h=h, g=gr, d_h=d, k=k, seed=31)
    inp = {n: U.to_dev(v) for n, v in gqe_synth.make_inputs(w).items()}
    dense = g.Buffers(g.make_shape(4, T, dm, h, gr, d, k, BF))
    dense.route(inp["x"], inp["W_r"])
    dense.prefill(inp["Q"], inp["K"], inp["V"])
    rows_max = 160
    step_shape = g.make_shape(1, rows_max, dm, h, gr, d, k, BF)
    buf = g.Buffers(step_shape)
    cache = g.PagedCache(step_shape, n_seqs=3, num_pages=32, page_size=16, max_blocks=10)
    who, at = [0, 1, 2], [0, 0, 0]  # the dense sequence in each place, its tokens so far
    r = random.Random(8)
    worst = 0.0
    for step in range(400):
        new = []
        for b in range(3):
            if b == 1 and who[b] == 1 and at[b] >= 100:
                new.append(-1)
                continue
            left = T - at[b]
            new.append(min(left, r.choice([1, 1, 0, 17, 50]) if step < 12 else 1))
        n = sum(max(a, 0) for a in new)
        src = [(who[b], at[b] + i) for b, a in enumerate(new) for i in range(max(a, 0))]
        sel = tuple(torch.tensor(x, device="cuda") for x in zip(*src)) if src else None
        packed = lambda t, n=n, sel=sel: torch.cat([t[sel], torch.full((rows_max - n, *t.shape[2:]), 3.0, dtype=t.dtype, device="cuda")]) \
            if sel is not None else torch.full((rows_max, *t.shape[2:]), 3.0, dtype=t.dtype, device="cuda")  # noqa: E731
        buf.O.fill_(7)
        buf.route(packed(inp["x"])[None], inp["W_r"])
        cache.plan(ints(new))
        cache.append(packed(inp["K"]), packed(inp["V"]))
        cache.attend(packed(inp["Q"])[None].contiguous(), buf.idx, buf.gate, buf.O)
        assert cache.status() == 0 and buf.status() == 0
        if src:
            got, want = buf.O[0, :n].float(), dense.O[sel].float()
            worst = max(worst, (got - want).abs().max().item())
        assert (buf.O[0, n:] == 7).all()
        for b, a in enumerate(new):
            if a < 0:
                who[b], at[b] = 3, 0
            else:
                at[b] += a
        assert cache.lengths.tolist() == at
        assert cache.free_count.item() == 32 - sum(-(-x // 16) for x in at)
        if min(at) == T:
            break
    assert at == [T, T, T] and who == [0, 3, 2]
    # both round weights and results to bf16 once: |difference| <= 2 * 2^-8 * (|o| + sum p |v|), with |v| <= 5 here
    assert worst <= 2 * 2.0 ** -8 * 10


def test_step_is_captured_and_replayed():
    """One decode step captured once, replayed as the caches grow past page ends."""
    g = U.gqe()
    h, gr, d, k, dm, n = 16, 8, 128, 1, 64, 5
    shape = g.make_shape(1, n, dm, h, gr, d, k, BF)
    cache = g.PagedCache(shape, n_seqs=n, num_pages=40, page_size=4, max_blocks=12, layers=2)
    gen = torch.Generator(device="cuda").manual_seed(1)
    steps = 13
    draw = lambda *s: torch.randn(*s, device="cuda", generator=gen).to(BF)  # noqa: E731
    Ks, Vs, Qs = draw(2, steps, n, gr, d), draw(2, steps, n, gr, d), draw(steps, n, h, d)
    idx = (torch.arange(gr, device="cuda")[None, :, None] * 2).expand(n, gr, 1).to(torch.int32).contiguous()
    gate = torch.ones(n, gr, 1, device="cuda")
    K, V, Q, new = [x.clone() for x in Ks[:, 0]], [x.clone() for x in Vs[:, 0]], Qs[0].clone(), ints([1] * n)
    O = [torch.zeros(n, h, d, dtype=BF, device="cuda") for _ in range(2)]

    def one():
        cache.plan(new)
        for layer in range(2):
            cache.append(K[layer], V[layer], layer)
            cache.attend(Q, idx, gate, O[layer], layer, window=6, sinks=1)

    one()  # step 0, eagerly
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    for i in range(1, steps):
        for layer in range(2):
            K[layer].copy_(Ks[layer, i])
            V[layer].copy_(Vs[layer, i])
        Q.copy_(Qs[i])
        graph.replay()
    assert cache.status() == 0
    assert cache.lengths.tolist() == [steps] * n
    # the last step against the formula
    for layer in range(2):
        table = cache.block_table.tolist()
        want, mag, wob = R.attention(Q, cache.K_pages[layer], cache.V_pages[layer], table, list(range(n + 1)), [steps] * n, 6, 1, idx, gate)
        tol = R.tolerance(want, mag, wob, BF, steps)
        assert ((O[layer].double() - want).abs() <= tol).all()
        for b in range(n):
            flat = [table[b][p // 4] * 4 + p % 4 for p in range(steps)]
            assert torch.equal(cache.K_pages[layer].view(-1, gr, d)[flat], Ks[layer, :, b])
