"""Plain 64-bit (or whole-number) forms of the paged-cache operators, for the tests: loops and
indexing from the definitions in include/mla_attn.h, nothing from the library."""
import random

import torch


def pages(n, page):
    return -(-n // page)


def plan_reference(ctx, new, table, free, head, page, T, parents=None):
    """(cu_q, kv_len, slots, positions, free_next, draft_mask, table) as lists, for lengths
    that fit.  table: rows of page ids, changed in a copy."""
    table = [list(r) for r in table]
    cu, kv, slots, pos, mask, at = [0], [], [], [], [], head
    for b, (c, n) in enumerate(zip(ctx, new)):
        kv.append(c + n)
        for k in range(pages(c, page), pages(c + n, page)):
            table[b][k] = free[at] if at < len(free) else -1
            at += 1
        bits, depth = [], []
        for i in range(n):
            p = -1 if parents is None else parents[cu[-1] + i]
            bits.append((bits[p] if p >= 0 else 0) | 1 << i)
            depth.append(i if parents is None else depth[p] + 1 if p >= 0 else 0)
            pg = table[b][(c + i) // page]
            slots.append(-1 if pg < 0 else pg * page + (c + i) % page)
            pos.append(c + depth[i])
            mask.append(bits[i] - (1 << 64) if bits[i] >> 63 else bits[i])
        cu.append(cu[-1] + n)
    pad = T - cu[-1]
    return (cu, kv, slots + [-1] * pad, pos + [0] * pad, min(at, len(free)),
            mask + [0] * pad, table)


def random_parents(r, n, roots=False):
    """A tree of n tokens (several with `roots`): each token hangs off one before it."""
    return [-1 if i == 0 or (roots and r.random() < 0.2) else r.randint(max(0, i - 6), i - 1)
            for i in range(n)]


def random_batch(seed, B, ctx, new, page, extra=2):
    """Lengths, a block table (-1 where nothing is held) and a free list of one pool."""
    r = random.Random(seed)
    c = [r.randint(*ctx) for _ in range(B)]
    n = [r.randint(*new) for _ in range(B)]
    width = max(1, max(pages(x + y, page) for x, y in zip(c, n)) + extra)
    held = [pages(x, page) for x in c]
    num = sum(pages(x + y, page) for x, y in zip(c, n)) + 3
    ids = list(range(num))
    r.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (width - h))
        at += h
    return r, c, n, table, ids[at:], num


def rotate64(x, table, positions):
    """Rotate-half of x [T, ..., 64] by the table rows of the positions, in 64 bits."""
    cs = table.double()[positions.long()]
    while cs.dim() < x.dim():
        cs = cs.unsqueeze(1)
    c, s = cs[..., :32], cs[..., 32:]
    lo, hi = x[..., :32].double(), x[..., 32:].double()
    return torch.cat((lo * c - hi * s, hi * c + lo * s), -1)
