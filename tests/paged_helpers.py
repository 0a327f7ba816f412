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


def tree_case(seed, B, H, ctx, new, page, tree, pad=0, dev="cuda"):
    """Inputs of mla_latent_tree_fwd.  Everything in the pool that no sequence holds is NaN, the
    rows behind a sequence's last one in its last page too; free table entries are -1."""
    r, c, n, table, free, num = random_batch(seed, B, ctx, new, page)
    g = torch.Generator("cpu").manual_seed(seed)
    mk = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    parents = [random_parents(r, k, roots=True) for k in n]
    flat = [x for p in parents for x in p]
    T = sum(n) + pad
    cu, kv, slots, _, _, mask, table = plan_reference(c, n, table, free, 0, page, T, flat)
    c_pages = torch.full((num, page, 512), float("nan"), dtype=torch.bfloat16)
    pe_pages = torch.full((num, page, 64), float("nan"), dtype=torch.bfloat16)
    for b, k in enumerate(kv):
        at = torch.tensor([table[b][p // page] * page + p % page for p in range(k)],
                          dtype=torch.int64)
        c_pages.view(-1, 512)[at] = mk(k, 512)
        pe_pages.view(-1, 64)[at] = mk(k, 64)
    i = lambda x, dt=torch.int32: torch.tensor(x, dtype=dt, device=dev)  # noqa: E731
    return dict(q_nope=mk(T, H, 128).to(dev), q_pe=mk(T, H, 64).to(dev), c_pages=c_pages.to(dev),
                pe_pages=pe_pages.to(dev), block_table=i(table), kv_len=i(kv), cu_q=i(cu),
                draft_mask=i(mask, torch.int64) if tree else None,
                w_kvb=mk(H * 256, 512).div(512 ** 0.5).to(dev))


def tree_reference(d, scale):
    """(out, spread, mixed) in 64 bits from the definition: each head's keys and values spelled
    out from the latent rows.  The scales of rounding errors: spread = sum_j p_j |v_j|, and for
    the latent mix, sum_l |W_V[l]| |mix_l|."""
    T, H = d["q_nope"].shape[:2]
    page = d["c_pages"].shape[1]
    cu, kv = d["cu_q"].tolist(), d["kv_len"].tolist()
    w = d["w_kvb"].double().view(H, 256, 512)
    out = torch.full((T, H, 128), float("nan"), dtype=torch.float64, device=w.device)
    spread, mixed = out.clone(), out.clone()
    for b, k in enumerate(kv):
        lo, hi = cu[b], cu[b + 1]
        if lo == hi:
            continue
        j = torch.arange(k, device=w.device)
        slot = d["block_table"][b].long()[j // page] * page + j % page
        c, pe = (d[x].view(-1, n)[slot].double() for x, n in (("c_pages", 512), ("pe_pages", 64)))
        new = j - (k - (hi - lo))
        i = torch.arange(hi - lo, device=w.device)
        if d["draft_mask"] is None:
            seen = new[None] <= i[:, None]
        else:
            seen = (new < 0) | ((d["draft_mask"][lo:hi, None] >> new.clamp(0, 63)) & 1).bool()
        keys = torch.einsum("jl,hdl->hjd", c, w[:, :128])
        vals = torch.einsum("jl,hdl->hjd", c, w[:, 128:])
        x = torch.einsum("ihd,hjd->hij", d["q_nope"][lo:hi].double(), keys)
        x = (x + torch.einsum("ihd,jd->hij", d["q_pe"][lo:hi].double(), pe)) * scale
        x = x.masked_fill(~seen, float("-inf"))
        top = x.amax(-1, keepdim=True).clamp(min=-1e300)
        e = (x - top).exp()
        total = e.sum(-1, keepdim=True)
        p = e / torch.where(total > 0, total, 1.0)
        out[lo:hi] = torch.einsum("hij,hjd->ihd", p, vals)
        spread[lo:hi] = torch.einsum("hij,hjd->ihd", p, vals.abs())
        mix = torch.einsum("hij,jl->ihl", p, c).abs()
        mixed[lo:hi] = torch.einsum("ihl,hdl->ihd", mix, w[:, 128:].abs())
    return out, spread, mixed
