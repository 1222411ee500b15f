"""Plain implementations of the paged serving step, in Python integers and in
64-bit floats: the page plan, the append and the chunk attention.  They share
no code with the library."""
import math

import torch


class Refused(Exception):
    pass


def plan(page_size, num_pages, max_blocks, rows, lengths, new, free, table):
    """One step of the plan on Python lists.  free: the stack, top last; table:
    a list of lists (changed in place).  Returns (lengths, free, cu, slots, pushed)
    or raises Refused with the state untouched."""
    blocks = lambda n: -(-n // page_size)  # noqa: E731
    for n, a in zip(lengths, new):
        if n < 0 or a < -1 or n + max(a, 0) > page_size * max_blocks:
            raise Refused("arguments")
    pushed = [table[b][j] for b, a in enumerate(new) if a < 0 for j in range(blocks(lengths[b]))]
    if len(free) + len(pushed) > num_pages or sum(max(a, 0) for a in new) > rows:
        raise Refused("arguments")
    need = sum(blocks(n + a) - blocks(n) for n, a in zip(lengths, new) if a >= 0)
    if need > len(free) + len(pushed):
        raise Refused("pages")
    stack = free + pushed
    out, cu, slots = [], [0], []
    for b, (n, a) in enumerate(zip(lengths, new)):
        if a < 0:
            out.append(0)
            cu.append(cu[-1])
            continue
        for j in range(blocks(n), blocks(n + a)):
            table[b][j] = stack.pop()
        out.append(n + a)
        cu.append(cu[-1] + a)
        slots += [table[b][p // page_size] * page_size + p % page_size for p in range(n, n + a)]
    return out, stack, cu, slots + [-1] * (rows - len(slots)), pushed


def attention(Q, K_pages, V_pages, table, cu, lengths, window, sinks, idx, gate):
    """O [T, h, d] in float64 (rows past the last request NaN), and what its error
    is measured against: mag = gate * sum_s p_s |v_s| per element, and per
    element the bound on the relative error of a weight that fp32 scores give,
    2 * delta with |score error| <= delta = (d + 2) 2^-24 sum_i |q_i k_i| / sqrt(d)."""
    T, h, d = Q.shape
    g, k = idx.shape[-2:]
    ps = K_pages.shape[1]
    dev = Q.device
    O = torch.full((T, h, d), math.nan, dtype=torch.float64, device=dev)
    mag = torch.zeros_like(O)
    wob = torch.zeros_like(O)
    for b, L in enumerate(lengths):
        t0, t1 = cu[b], cu[b + 1]
        if t0 == t1:
            continue
        O[t0:t1] = 0
        pos = torch.arange(L - (t1 - t0), L, device=dev)
        key = torch.arange(L, device=dev)
        seen = key[None] <= pos[:, None]
        if window:
            seen &= (key[None] > pos[:, None] - window) | (key[None] < sinks)
        any_row = seen.any(0)
        pages = torch.tensor([p if any_row[j * ps:(j + 1) * ps].any() else 0 for j, p in
                              enumerate(table[b][: -(-L // ps)])], device=dev)
        t = torch.arange(t0, t1, device=dev)
        for q in range(g):
            Kq = K_pages[pages, :, q].reshape(-1, d)[:L].double()
            Vq = V_pages[pages, :, q].reshape(-1, d)[:L].double()
            Kq[~any_row] = 0  # rows that no token sees are not read
            Vq[~any_row] = 0
            for r in range(k):
                head = idx[t0:t1, q, r].long()
                x = Q[t, head].double()
                s = (x @ Kq.T / math.sqrt(d)).masked_fill(~seen, -math.inf)
                p = torch.exp(s - s.max(1, keepdim=True).values)
                p = p / p.sum(1, keepdim=True)
                gm = gate[t0:t1, q, r, None].double()
                O[t, head] = gm * torch.where(p[..., None] > 0, p[..., None] * Vq, 0.0).sum(1) if len(t) * L * d < 1 << 24 \
                    else gm * (p @ Vq)
                mag[t, head] = gm * (p @ Vq.abs())
                delta = ((x.abs() @ Kq.abs().T) / math.sqrt(d)).masked_fill(~seen, 0).max(1, keepdim=True).values
                wob[t, head] = (2 * (d + 2) * 2.0 ** -24 * delta).expand(-1, d)
    return O, mag, wob


def tolerance(O, mag, wob, dtype, longest):
    """Element-wise bound on |result - O|.  fp32 arithmetic: weights off by
    2 * delta (see `attention`) and 2^-21 (exp2), their sums over at most
    `longest` keys by longest * 2^-24 each, of numerator and denominator.  bf16:
    half a step, 2^-8, of the result, and on the tensor cores the same of every weight."""
    tol = mag * (wob + 2.0 ** -20 + longest * 2.0 ** -23) + 1e-30
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (mag + O.abs())
    return tol
