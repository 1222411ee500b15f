"""The operators of a serving step over a paged KV cache, as cases to be measured.

Four operators:
  plan    block tables and slot maps built on the GPU from the requests' lengths (gqe_page_plan)
  append  the step's new K/V rows written to their slots in the pages (gqe_kv_append)
  chunk   routed attention of every request's chunk of new tokens over its paged cache (gqe_attn_chunk_paged)
  window  the same with a sliding window and a few first tokens that stay visible (gqe_attn_chunk_paged)

With `own` false, `run` computes them in plain torch operations, in 32 bits, rounded once at the end; with `own` true it
makes the calls that a user of this library makes.  The requests' lengths follow from the case alone, the values (and the
order of the pages in the pool) from the seed.
"""
import math
import random

import torch

own = False

INT = torch.int32
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # A decode step of a small server: eight requests, one token each; the call's latency is what counts.
        dict(name="plan_decode", op="plan", n_seqs=8, chunks=0, new_lo=1, new_hi=1, ctx_lo=10, ctx_hi=900, ended=1, idle=0, pad=1, page_size=16),
        # A step of a large server: a thousand requests decode, forty bring a prompt's chunk, thirty have just ended.
        dict(name="plan_mixed", op="plan", n_seqs=1000, chunks=40, new_lo=17, new_hi=1500, ctx_lo=0, ctx_hi=9000, ended=30, idle=25, pad=333, page_size=16),
        # The new rows of a decode step of 40 requests, some of whose slots are padding.
        dict(name="append_decode", op="append", rows=40, skipped=3, dtype="bf16", g=8, d_h=128, page_size=16, num_pages=512, sliced=False),
        # The new rows of a prompt step, taken out of the fused q/k/v projection's output.
        dict(name="append_prompt", op="append", rows=16384, skipped=0, dtype="bf16", g=8, d_h=128, page_size=64, num_pages=1024, sliced=True),
        # A decode step of three requests with short caches, 16 query heads over 8 KV groups, one routed head each.
        dict(name="chunk_decode_few", op="chunk", n_seqs=3, chunks=0, new_lo=1, new_hi=1, ctx_lo=200, ctx_hi=1100, idle=0, pad=0, dtype="bf16", h=16, g=8, d_h=128, k=1, page_size=16, window=0, sinks=0),
        # The decode workload of the benchmark on pages: 64 requests, 1024 to 16384 cached tokens.
        dict(name="chunk_decode_many", op="chunk", n_seqs=64, chunks=0, new_lo=1, new_hi=1, ctx_lo=1023, ctx_hi=16383, idle=0, pad=0, dtype="bf16", h=32, g=8, d_h=128, k=2, page_size=64, window=0, sinks=0),
        # Two long prompts in chunks of 4096 tokens, most of each prompt cached already.
        dict(name="chunk_prompt", op="chunk", n_seqs=2, chunks=2, new_lo=4096, new_hi=4096, ctx_lo=12288, ctx_hi=28672, idle=0, pad=0, dtype="bf16", h=32, g=8, d_h=128, k=2, page_size=64, window=0, sinks=0),
        # A mixed step: decodes beside ragged chunks of prompts, two requests that wait, rows of padding at the end.
        dict(name="chunk_mixed", op="chunk", n_seqs=34, chunks=4, new_lo=100, new_hi=700, ctx_lo=30, ctx_hi=6000, idle=2, pad=37, dtype="bf16", h=32, g=8, d_h=128, k=2, page_size=16, window=0, sinks=0),
        # The small fp32 layer of the tests, ragged chunks.
        dict(name="chunk_f32", op="chunk", n_seqs=5, chunks=4, new_lo=3, new_hi=64, ctx_lo=0, ctx_hi=500, idle=0, pad=2, dtype="f32", h=8, g=2, d_h=32, k=1, page_size=8, window=0, sinks=0),
        # Streaming decode: 128 long-lived requests that see the last 1024 tokens and the first four.
        dict(name="window_decode", op="window", n_seqs=128, chunks=0, new_lo=1, new_hi=1, ctx_lo=2000, ctx_hi=32000, idle=0, pad=0, dtype="bf16", h=32, g=8, d_h=128, k=2, page_size=16, window=1024, sinks=4),
        # Prompts in chunks of 2048 tokens under a window of 2048 and 16 first tokens.
        dict(name="window_prompt", op="window", n_seqs=4, chunks=4, new_lo=2048, new_hi=2048, ctx_lo=0, ctx_hi=16384, idle=0, pad=0, dtype="bf16", h=32, g=8, d_h=128, k=2, page_size=64, window=2048, sinks=16),
        # Narrow heads, an odd window, tiny pages, ragged short chunks.
        dict(name="window_odd", op="window", n_seqs=6, chunks=4, new_lo=2, new_hi=90, ctx_lo=0, ctx_hi=400, idle=1, pad=5, dtype="bf16", h=8, g=2, d_h=64, k=3, page_size=4, window=100, sinks=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _plain_bytes(c):
    """What the plain form of an attention case holds: its score matrix and its gathered keys, in 32 bits."""
    new, ctx = _lengths(c)
    length = max(n + x for n, x in zip(new, ctx))
    j = length if not c["window"] else min(length, c["sinks"] + c["window"] + max(new) - 1)
    return 4 * c["n_seqs"] * j * c["g"] * (max(new) * c["k"] + 2 * c["d_h"])


def draw(rng):
    """One more case of the same ranges: all four operators, both types, every head width, short and long."""
    op = rng.choice(["plan", "append", "chunk", "chunk", "chunk", "window", "window"])
    if op == "plan":
        n = _log(rng, 1, 2000)
        return dict(op=op, n_seqs=n, chunks=rng.randint(0, max(1, n // 20)), new_lo=1, new_hi=_log(rng, 2, 1500), ctx_lo=0, ctx_hi=_log(rng, 10, 9000),
                    ended=rng.randint(0, n // 10), idle=rng.randint(0, n // 10), pad=rng.choice([0, 0, 1, rng.randint(2, 400)]), page_size=rng.choice([1, 8, 16, 32, 64, 256]))
    if op == "append":
        rows = _log(rng, 1, 16384)
        ps = rng.choice([1, 4, 16, 64, 256])
        return dict(op=op, rows=rows, skipped=rng.randint(0, rows // 8), dtype=rng.choice(["bf16", "bf16", "f32"]), g=rng.choice([1, 2, 4, 8]), d_h=rng.choice([32, 64, 128, 128]),
                    page_size=ps, num_pages=rows // ps + rng.randint(2, 300), sliced=rng.random() < 0.5)
    while True:
        wide = rng.random() < 0.65  # the tensor-core shape: bf16, heads of 128; else narrow heads or fp32, for which calls are smaller
        dtype, d_h = ("bf16", 128) if wide else rng.choice([("bf16", 64), ("bf16", 32), ("f32", 32), ("f32", 64), ("f32", 128)])
        h, g = rng.choice([(32, 8), (32, 8), (16, 8), (8, 2), (24, 4)])
        kind = rng.choice(["decode", "prompt", "mixed"])
        n = _log(rng, 1, 128) if kind == "decode" else rng.randint(1, 6) if kind == "prompt" else rng.randint(4, 32)
        chunks = 0 if kind == "decode" else n if kind == "prompt" else rng.randint(1, 4)
        hi = 1 if kind == "decode" else _log(rng, 2, (4096 if kind == "prompt" else 700) if wide else 200)
        ctx_hi = _log(rng, 16, 28672 if wide else 4096)
        window = 0 if op == "chunk" else _log(rng, 1, 4096)
        c = dict(op=op, n_seqs=n, chunks=chunks, new_lo=max(1, hi // 3), new_hi=hi, ctx_lo=rng.randint(0, ctx_hi // 2) if kind != "decode" else max(0, ctx_hi // 16), ctx_hi=ctx_hi,
                 idle=rng.choice([0, 0, min(1, n - 1)]) if chunks < n else 0, pad=rng.choice([0, 0, rng.randint(1, 50)]), dtype=dtype, h=h, g=g, d_h=d_h,
                 k=rng.randint(1, min(4, h // g)), page_size=rng.choice([1, 4, 16, 16, 32, 64, 256]), window=window, sinks=0 if op == "chunk" else rng.choice([0, 1, 4, 16, 64]))
        largest = work(next(x for x in listed() if x["name"] == "chunk_prompt"))["flops"]
        many = work(next(x for x in listed() if x["name"] == "chunk_decode_many"))["bytes"]
        w = work(c)
        if w["flops"] <= largest and w["bytes"] <= many and _plain_bytes(c) < 12 << 30:
            return c


def _lengths(case):
    """(new, ctx) per request, from the case alone: new tokens (-1: the request has ended) and tokens cached before them."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    n = case["n_seqs"]
    kinds = ["chunk"] * case["chunks"] + ["ended"] * case.get("ended", 0) + ["idle"] * case["idle"]
    kinds = (kinds + ["decode"] * n)[:n]
    r.shuffle(kinds)
    new, ctx = [], []
    for kind in kinds:
        new.append(r.randint(case["new_lo"], case["new_hi"]) if kind == "chunk" else {"decode": 1, "ended": -1, "idle": 0}[kind])
        ctx.append(max(r.randint(case["ctx_lo"], case["ctx_hi"]), 1 if kind in ("ended", "idle") else 0))
    return new, ctx


def _pages(rows, ps):
    return -(-rows // ps)


def _visible(length, new, window, sinks):
    """(pairs, keys): how many (new token, key) pairs a request has, and how many of its cached rows some new token sees."""
    if new <= 0:
        return 0, 0
    first = length - new
    if not window:
        return new * first + new * (new + 1) // 2, length
    pairs = 0
    for p in range(first, length):
        low = max(0, p - window + 1)
        pairs += p + 1 - low + min(sinks, low)
    low = max(0, first - window + 1)
    return pairs, length - low + min(sinks, low)


def work(case):
    op = case["op"]
    if op == "append":
        row = case["g"] * case["d_h"] * (2 if case["dtype"] == "bf16" else 4)
        return {"bytes": (case["rows"] - case["skipped"]) * 4 * row + 4 * case["rows"], "flops": 0}
    new, ctx = _lengths(case)
    if op == "plan":
        ps = case["page_size"]
        need = sum(_pages(c + n, ps) - _pages(c, ps) for n, c in zip(new, ctx) if n >= 0)
        back = sum(_pages(c, ps) for n, c in zip(new, ctx) if n < 0)
        rows = sum(max(n, 0) for n in new) + case["pad"]
        # lengths and new tokens in; prefix sums and lengths out; a page read and written for each page taken or given back; a slot per row
        return {"bytes": 16 * case["n_seqs"] + 8 * (need + back) + 4 * rows, "flops": 0}
    e = 2 if case["dtype"] == "bf16" else 4
    g, k, h, d = case["g"], case["k"], case["h"], case["d_h"]
    seen = [_visible(c + n, n, case["window"], case["sinks"]) for n, c in zip(new, ctx)]
    rows = sum(new)
    moved = sum(s[1] for s in seen) * g * d * 2 * e + rows * (g * k * d * e + h * d * e + 8 * g * k) + sum(4 * _pages(s[1], case["page_size"]) for s in seen)
    return {"bytes": moved, "flops": 4 * d * g * k * sum(s[0] for s in seen)}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    st = {"op": op, "case": case}
    ints = lambda v: torch.tensor(v, dtype=INT, device="cuda")  # noqa: E731
    perm = lambda n: torch.randperm(n, generator=gen, device="cuda").to(INT)  # noqa: E731
    normal = lambda *shape: torch.empty(shape, dtype=TYPES[case["dtype"]], device="cuda").normal_(generator=gen)  # noqa: E731
    if own:
        import routed_head_gqa_b200 as gqe
        st["gqe"] = gqe
    if op == "append":
        rows, g, d = case["rows"], case["g"], case["d_h"]
        if case["sliced"]:  # the k and v columns of a fused projection's output of 4 g query heads and g + g key and value heads
            qkv = normal(rows, 6 * g, d)
            st["K_new"], st["V_new"] = qkv[:, 4 * g:5 * g], qkv[:, 5 * g:]
        else:
            st["K_new"], st["V_new"] = normal(rows, g, d), normal(rows, g, d)
        slots = perm(case["num_pages"] * case["page_size"])[:rows].contiguous()
        slots[perm(rows)[:case["skipped"]].long()] = -1
        st["slots"] = slots
        st["K_pages"], st["V_pages"] = (normal(case["num_pages"], case["page_size"], g, d) for _ in range(2))
        if own:
            st["shape"] = gqe.make_shape(1, rows, 4 * g * d, 4 * g, g, d, 1, TYPES[case["dtype"]])
            st["workspace"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        return st
    new, ctx = _lengths(case)
    n, ps = case["n_seqs"], case["page_size"]
    if op == "plan":
        have = [_pages(c, ps) for c in ctx]
        need = [_pages(c + max(a, 0), ps) - b if a >= 0 else 0 for a, c, b in zip(new, ctx, have)]
        free = sum(need) + 10
        num_pages, blocks = sum(have) + free, max(a + b for a, b in zip(have, need)) + 1
        pages = perm(num_pages)
        st["block_table"] = _table(ints(have), pages, blocks)
        st["free_pages"] = torch.zeros(num_pages, dtype=INT, device="cuda")
        st["free_pages"][:free] = pages[sum(have):]
        st["free_count"] = ints([free])
        st["lengths"], st["new"] = ints(ctx), ints(new)
        rows = sum(max(a, 0) for a in new) + case["pad"]
        st.update(page_size=ps, lengths_out=torch.empty_like(st["lengths"]), free_count_out=torch.empty_like(st["free_count"]),
                  cu_new=torch.empty(n + 1, dtype=INT, device="cuda"), slots=torch.empty(rows, dtype=INT, device="cuda"))
        if own:
            st["workspace"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        return st
    g, k, h, d = case["g"], case["k"], case["h"], case["d_h"]
    length = [a + c for a, c in zip(new, ctx)]
    have = [_pages(x, ps) for x in length]
    num_pages = sum(have) + 3
    st["K_pages"], st["V_pages"] = normal(num_pages, ps, g, d), normal(num_pages, ps, g, d)
    st["block_table"] = _table(ints(have), perm(num_pages), max(have))
    st["lengths"] = ints(length)
    cu = [0]
    for a in new:
        cu.append(cu[-1] + a)
    st["cu_new"] = ints(cu)
    st["rows"], st["new_max"], st["len_max"] = cu[-1], max(new), max(length)
    T = cu[-1] + case["pad"]
    st["Q"] = normal(T, h, d)
    # k distinct heads of each group, and gates that sum to one over them, as the router gives them
    pick = torch.rand(T, g, h // g, generator=gen, device="cuda").argsort(-1)[..., :k]
    st["idx"] = (pick + torch.arange(g, device="cuda")[:, None] * (h // g)).to(INT).contiguous()
    st["gate"] = torch.softmax(torch.randn(T, g, k, generator=gen, device="cuda"), -1)
    st["O"] = torch.zeros(T, h, d, dtype=TYPES[case["dtype"]], device="cuda")
    if own:
        st["shape"] = gqe.make_shape(1, T, h * d, h, g, d, k, TYPES[case["dtype"]])
        st["workspace"] = torch.zeros(gqe.gqe_chunk_workspace_bytes(st["shape"]), dtype=torch.uint8, device="cuda")
    return st


def _table(have, pages, blocks):
    """Block table [n, blocks]: request b's first have[b] entries are the pages' next ones, the others -1."""
    col = torch.arange(blocks, device="cuda")
    first = torch.cumsum(have, 0) - have
    at = (first[:, None] + col).clamp(max=pages.numel() - 1)
    return torch.where(col < have[:, None], pages[at], -1).to(INT).contiguous()


# ------------------------------------------------------------------ one pass
def run(st):
    if own:
        return _run_own(st)
    return {"plan": _plan, "append": _append, "chunk": _attention, "window": _attention}[st["op"]](st)


def _run_own(st):
    gqe, op = st["gqe"], st["op"]
    if op == "plan":
        gqe.gqe_page_plan(st["page_size"], st["lengths"], st["new"], st["free_pages"], st["free_count"], st["block_table"], st["lengths_out"], st["free_count_out"], st["cu_new"],
                          st["slots"], st["workspace"])
        return {x: st[x] for x in ("free_pages", "free_count_out", "block_table", "lengths_out", "cu_new", "slots")}
    if op == "append":
        gqe.gqe_kv_append(st["shape"], st["K_new"], st["V_new"], st["slots"], st["K_pages"], st["V_pages"], st["workspace"])
        return {"K_pages": st["K_pages"], "V_pages": st["V_pages"]}
    c = st["case"]
    gqe.gqe_attn_chunk_paged(st["shape"], st["Q"], st["K_pages"], st["V_pages"], st["block_table"], st["cu_new"], st["lengths"], c["window"], c["sinks"], st["idx"], st["gate"], st["O"],
                             st["workspace"])
    return {"O": st["O"]}


def _plan(st):
    ps, length, new, table, stack = st["page_size"], st["lengths"], st["new"], st["block_table"], st["free_pages"]
    rows = st["slots"].numel()
    ended = new < 0
    add = new.clamp(min=0)
    have = (length + ps - 1) // ps
    length_out = torch.where(ended, 0, length + add)
    need = torch.where(ended, 0, (length_out + ps - 1) // ps - have)
    back = torch.where(ended, have, 0)
    col = torch.arange(table.shape[1], device="cuda")
    # the ended requests' pages go on top of the stack, in the order of requests and blocks
    given = table[col < back[:, None]]
    top = st["free_count"] + given.numel()
    stack[st["free_count"] + torch.arange(given.numel(), device="cuda")] = given
    # the new blocks take pages from the top
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None])
    taken = need.sum()
    table[fresh] = stack[top - 1 - torch.arange(int(taken), device="cuda")]
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(add, 0)])
    t = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=length.numel() - 1)
    pos = length[seq] + t - cu[seq]
    page = table[seq, (pos // ps).clamp(max=table.shape[1] - 1)]
    slots = torch.where(t < cu[-1], page * ps + pos % ps, -1)
    return {"free_pages": stack, "free_count_out": (top - taken).to(INT), "block_table": table, "lengths_out": length_out.to(INT), "cu_new": cu.to(INT), "slots": slots.to(INT)}


def _append(st):
    kept = st["slots"] >= 0
    to = st["slots"][kept].long()
    for new, pages in ((st["K_new"], st["K_pages"]), (st["V_new"], st["V_pages"])):
        pages.view(-1, *pages.shape[2:])[to] = new[kept]
    return {"K_pages": st["K_pages"], "V_pages": st["V_pages"]}


def _attention(st):
    c = st["case"]
    g, k, d, ps, window, sinks = c["g"], c["k"], c["d_h"], c["page_size"], c["window"], c["sinks"]
    n, new_max, len_max, rows = c["n_seqs"], st["new_max"], st["len_max"], st["rows"]
    cu, length = st["cu_new"].long(), st["lengths"].long()
    new = cu[1:] - cu[:-1]
    i = torch.arange(new_max, device="cuda")
    held = i < new[:, None]  # [n, new_max]: the padded layout's tokens that exist
    token = (cu[:-1, None] + i).clamp(max=max(rows - 1, 0))
    qpos = length[:, None] - new[:, None] + i
    idx = st["idx"][token].long()  # [n, new_max, g, k]
    q = st["Q"][token[..., None, None], idx].float()  # [n, new_max, g, k, d]
    # the keys that some new token of the request can see: all, or the first ones and the last window + new_max - 1
    tail = window + new_max - 1
    if not window or sinks + tail >= len_max:
        kpos = torch.arange(len_max, device="cuda").expand(n, -1)
    else:
        kpos = torch.cat([torch.arange(sinks, device="cuda").expand(n, -1), (length - tail).clamp(min=sinks)[:, None] + torch.arange(tail, device="cuda")], 1)
    there = kpos.clamp(max=(length - 1)[:, None])
    row = st["block_table"].gather(1, there // ps).long() * ps + there % ps  # [n, J]
    K = st["K_pages"].view(-1, g, d)[row].float().permute(0, 2, 3, 1)  # [n, g, d, J]
    V = st["V_pages"].view(-1, g, d)[row].float().permute(0, 2, 1, 3)  # [n, g, J, d]
    s = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(n, g, new_max * k, d) * d ** -0.5, K)
    seen = kpos[:, None] <= qpos[..., None]  # [n, new_max, J]
    if window:
        seen &= (kpos[:, None] > qpos[..., None] - window) | (kpos[:, None] < sinks)
    s = s.view(n, g, new_max, k, -1)
    s.masked_fill_(~seen[:, None, :, None], -math.inf)
    s -= s.amax(-1, keepdim=True)
    s.exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(n, g, new_max * k, -1), V).view(n, g, new_max, k, d) / total
    o = o.permute(0, 2, 1, 3, 4) * st["gate"][token][..., None]  # [n, new_max, g, k, d]
    out = st["O"]
    out[:rows] = 0
    at = token[held]
    out[at[:, None, None], idx[held]] = o[held].to(out.dtype)
    return {"O": out}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "append":
        out = {}
        rows = [i for i, x in enumerate(st["slots"].tolist()) if x >= 0]
        page, line = st["slots"][rows].long() // case["page_size"], st["slots"][rows].long() % case["page_size"]
        for x in "KV":
            out[x + "_pages"] = st[x + "_pages"].double()
            out[x + "_pages"][page, line] = st[x + "_new"][rows].double()
        return out
    g, k, d, ps, window, sinks = (case[x] for x in ("g", "k", "d_h", "page_size", "window", "sinks"))
    Q, Kp, Vp, table = st["Q"], st["K_pages"], st["V_pages"], st["block_table"]
    O = torch.zeros(Q.shape, dtype=torch.float64, device="cuda")
    cu, lengths = st["cu_new"].tolist(), st["lengths"].tolist()
    for b in range(case["n_seqs"]):
        t0, t1, L = cu[b], cu[b + 1], lengths[b]
        if t0 == t1:
            continue
        pos = torch.arange(L - (t1 - t0), L, device="cuda")[:, None]
        key = torch.arange(L, device="cuda")[None]
        hidden = key > pos
        if window:
            hidden = hidden | ((key <= pos - window) & (key >= sinks))
        pages = table[b, : _pages(L, ps)].long()
        for q in range(g):
            K = Kp[pages, :, q].reshape(-1, d)[:L].double()
            V = Vp[pages, :, q].reshape(-1, d)[:L].double()
            for r in range(k):
                head = st["idx"][t0:t1, q, r].long()
                t = torch.arange(t0, t1, device="cuda")
                score = Q[t, head].double() @ K.T / math.sqrt(d)
                score[hidden] = -math.inf
                weight = torch.exp(score - score.max(1, keepdim=True).values)
                weight = weight / weight.sum(1, keepdim=True)
                O[t, head] = st["gate"][t0:t1, q, r, None].double() * (weight @ V)
    return {"O": O}
