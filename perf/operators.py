"""Serving operators of the MLA framework, measured: each in its plain form (elementary torch
operations) and, with ``own`` set, through the framework's entry points.

  plan    block tables, slots, positions and draft masks of a batch's new tokens
  append  the rotary step on the new rows, and their scatter into a paged latent cache
  tree    attention of drafted tokens (or of one new token each) over the paged latent cache
  prompt  causal attention over whole prompts of different lengths, packed in one buffer

Lengths and trees are drawn once per case from its "lens" number; the seed permutes them over
the batch and draws everything else, so the work of a case does not depend on the seed.
"""
import random

import torch

own = False

D_NOPE, D_ROPE, D_V, D_LAT = 128, 64, 128, 512
SCALE = (D_NOPE + D_ROPE) ** -0.5


# ---- cases ------------------------------------------------------------------------------

def listed():
    return [
        # one decode step's bookkeeping: 64 running requests, one new token each
        {"name": "plan_decode", "op": "plan", "B": 64, "ctx_lo": 512, "ctx_hi": 8192,
         "new_lo": 1, "new_hi": 1, "tree": False, "page": 64, "lens": 1},
        # a step with drafted trees of any size up to 64 tokens, many requests
        {"name": "plan_trees", "op": "plan", "B": 512, "ctx_lo": 1, "ctx_hi": 8192,
         "new_lo": 1, "new_hi": 64, "tree": True, "page": 64, "lens": 2},
        # a million prompt tokens admitted at once
        {"name": "plan_prompts", "op": "plan", "B": 256, "ctx_lo": 0, "ctx_hi": 0,
         "new_lo": 1, "new_hi": 8192, "tree": False, "page": 64, "lens": 3},
        # the new rows of a decode step of 64 requests
        {"name": "append_decode", "op": "append", "T": 64, "H": 64, "page": 64},
        # the rows of several packed prompts, an odd number of them
        {"name": "append_prompts", "op": "append", "T": 16411, "H": 64, "page": 64},
        # one request, 1000 cached keys and a small tree: latency
        {"name": "tree_one", "op": "tree", "B": 1, "H": 64, "ctx_lo": 1000, "ctx_hi": 1000,
         "new_lo": 8, "new_hi": 8, "tree": True, "page": 64, "lens": 4},
        # ordinary decode: one token per request over a ragged batch's pages
        {"name": "tree_decode", "op": "tree", "B": 64, "H": 64, "ctx_lo": 512, "ctx_hi": 8192,
         "new_lo": 1, "new_hi": 1, "tree": False, "page": 64, "lens": 5},
        # speculative decoding of the same batch with trees of 16 tokens
        {"name": "tree_batch", "op": "tree", "B": 64, "H": 64, "ctx_lo": 512, "ctx_hi": 8192,
         "new_lo": 16, "new_hi": 16, "tree": True, "page": 64, "lens": 6},
        # few long requests, the largest trees
        {"name": "tree_long", "op": "tree", "B": 8, "H": 64, "ctx_lo": 32768, "ctx_hi": 32768,
         "new_lo": 64, "new_hi": 64, "tree": True, "page": 64, "lens": 7},
        # a handful of short prompts
        {"name": "prompt_short", "op": "prompt", "B": 7, "H": 64, "Hkv": 64, "lo": 1, "hi": 200,
         "fused": True, "lens": 8},
        # an ordinary batch of prompts, read in place from the projections' outputs
        {"name": "prompt_batch", "op": "prompt", "B": 32, "H": 64, "Hkv": 64, "lo": 1,
         "hi": 1024, "fused": True, "lens": 9},
        # long prompts, heads in groups of four over fewer key/value heads
        {"name": "prompt_long", "op": "prompt", "B": 4, "H": 64, "Hkv": 16, "lo": 2048,
         "hi": 4096, "fused": False, "lens": 10},
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], its logarithm about uniform."""
    return max(lo, min(hi, int(lo * (hi / lo) ** rng.random() + rng.random())))


def draw(rng):
    op = rng.choice(("plan", "append", "tree", "tree", "prompt", "prompt"))
    lens = rng.randrange(1 << 30)
    if op == "plan":
        tree = rng.random() < 0.5
        prompts = not tree and rng.random() < 0.5
        return {"op": op, "B": _log_int(rng, 1, 250 if prompts else 512),
                "ctx_lo": 0, "ctx_hi": 0 if prompts else _log_int(rng, 1, 8192),
                "new_lo": 1, "new_hi": _log_int(rng, 1, 8192) if prompts else rng.randint(1, 64),
                "tree": tree, "page": rng.choice((16, 32, 64, 128)), "lens": lens}
    if op == "append":
        return {"op": op, "T": _log_int(rng, 1, 16411), "H": rng.choice((8, 16, 32, 64)),
                "page": rng.choice((16, 32, 64, 128))}
    if op == "tree":
        H, n = rng.choice((8, 16, 32, 64)), rng.randint(1, 64)
        ctx = _log_int(rng, 1, 32768)
        most = 8 * 64 * 64 * 32768 // (H * n * (ctx + n))
        return {"op": op, "B": _log_int(rng, 1, max(1, min(64, most))), "H": H,
                "ctx_lo": rng.randint(0, ctx), "ctx_hi": ctx, "new_lo": rng.randint(1, n),
                "new_hi": n, "tree": rng.random() < 0.7, "page": rng.choice((16, 32, 64, 128)),
                "lens": lens}
    Hkv, group = rng.choice((4, 8, 16)), rng.choice((1, 2, 4))
    hi = _log_int(rng, 1, 4000)
    most = 4 * 64 * 3000 ** 2 // (Hkv * group * hi * hi)
    return {"op": op, "B": _log_int(rng, 1, max(1, min(32, most))), "H": Hkv * group, "Hkv": Hkv,
            "lo": rng.randint(1, hi), "hi": hi, "fused": rng.random() < 0.5, "lens": lens}


def _batch(case):
    """The requests of a plan or tree case: (cached length, parents of the new tokens)."""
    r = random.Random(case["lens"])
    out = []
    for _ in range(case["B"]):
        ctx, n = r.randint(case["ctx_lo"], case["ctx_hi"]), r.randint(case["new_lo"], case["new_hi"])
        # token 0 is the root; the others hang off one of the eight tokens before them
        parents = [-1] + [r.randint(max(0, i - 8), i - 1) for i in range(1, n)] if case["tree"] \
            else [-1] * n
        out.append((ctx, parents))
    return out


def _prompt_lengths(case):
    r = random.Random(case["lens"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]


def _ancestors(parents):
    """Bit masks: bit j of token i is set where j is i or one of its ancestors."""
    bits = []
    for i, p in enumerate(parents):
        bits.append((bits[p] if p >= 0 else 0) | 1 << i)
    return bits


def _signed(x):
    return x - (1 << 64) if x >> 63 else x


def _pages(n, page):
    return -(-n // page)


def work(case):
    op = case["op"]
    if op == "plan":
        b = _batch(case)
        T = sum(len(p) for _, p in b)
        pg = case["page"]
        taken = sum(_pages(c + len(p), pg) - _pages(c, pg) for c, p in b)
        held = sum(1 for c, p in b if c % pg and p)
        return {"bytes": 16 * len(b) + 8 * taken + 4 * held + 8 * T + (12 * T if case["tree"] else 0),
                "flops": 0}
    if op == "append":
        T, H = case["T"], case["H"]
        return {"bytes": T * (2 * 2 * D_ROPE * H + 2 * 2 * (D_LAT + D_ROPE) + 8 + 4 * D_ROPE),
                "flops": T * (H + 1) * D_ROPE * 3}
    if op == "tree":
        b, H = _batch(case), case["H"]
        T = sum(len(p) for _, p in b)
        keys = sum(c + len(p) for c, p in b)
        if case["tree"]:
            pairs = sum(c * len(p) + sum(bin(m).count("1") for m in _ancestors(p)) for c, p in b)
        else:
            pairs = sum(c * len(p) + len(p) * (len(p) + 1) // 2 for c, p in b)
        return {"bytes": keys * (D_LAT + D_ROPE) * 2 + T * H * (D_NOPE + D_ROPE + D_V) * 2
                + H * (D_NOPE + D_V) * D_LAT * 2,
                "flops": pairs * H * 2 * (2 * D_LAT + D_ROPE) + T * H * 2 * (D_NOPE + D_V) * D_LAT}
    ns, H, Hkv = _prompt_lengths(case), case["H"], case["Hkv"]
    T = sum(ns)
    return {"bytes": T * 2 * (H * (D_NOPE + D_ROPE + D_V) + Hkv * (D_NOPE + D_V) + D_ROPE),
            "flops": H * 2 * (D_NOPE + D_ROPE + D_V) * sum(n * (n + 1) // 2 for n in ns)}


# ---- inputs -----------------------------------------------------------------------------

class _Draw:
    """Random device tensors of one seed."""

    def __init__(self, seed):
        self.host = random.Random(seed)
        self.gen = torch.Generator("cuda").manual_seed(seed)

    def normal(self, *shape, std=1.0):
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        return x.normal_(0.0, std, generator=self.gen)

    def permutation(self, n):
        return torch.randperm(n, generator=self.gen, device="cuda", dtype=torch.int32)

    def shuffled(self, items):
        items = list(items)
        self.host.shuffle(items)
        return items


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _offsets(ns):
    cu = [0]
    for n in ns:
        cu.append(cu[-1] + n)
    return cu


def _table(held, width, pages):
    """A block table [B, width] whose row b has the next held[b] of `pages`, then -1."""
    cu = _offsets(held)
    k = torch.arange(width, device="cuda")[None]
    held, first = _ints(held)[:, None], _ints(cu[:-1])[:, None]
    at = (first + k).clamp(max=pages.numel() - 1).long()
    return torch.where(k < held, pages[at], torch.full_like(at, -1, dtype=torch.int32))


def _rotary_table(rows):
    """cos | sin of p * 50000^(-2d/64), as the rotary step's table holds them."""
    f = 50000.0 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat((a.cos(), a.sin()), 1).float()


def prepare(case, seed):
    d = _Draw(seed)
    return {"plan": _prepare_plan, "append": _prepare_append, "tree": _prepare_tree,
            "prompt": _prepare_prompt}[case["op"]](case, d)


def _prepare_plan(case, d):
    b, pg = d.shuffled(_batch(case)), case["page"]
    ctx, new = [c for c, _ in b], [len(p) for _, p in b]
    held = [_pages(c, pg) for c in ctx]
    width = max(_pages(c + n, pg) for c, n in zip(ctx, new)) + 2
    need = sum(_pages(c + n, pg) for c, n in zip(ctx, new))
    pool = need + need // 4 + 8
    pages = d.permutation(pool)
    T = sum(new)
    s = {"op": "plan", "page": pg, "num_pages": pool, "ctx_len": _ints(ctx), "new_len": _ints(new),
         "block_table": _table(held, width, pages), "free_pages": pages[sum(held):].contiguous(),
         "free_head": _ints([0]), "tokens": _pages(T, 64) * 64, "most_new": max(new), "parent": None}
    # the buffers that a server fills anew every step: cu_q, kv_len, slots, positions, free_next
    # and the draft masks
    s["out"] = tuple(torch.empty(n, dtype=torch.int32, device="cuda")
                     for n in (len(b) + 1, len(b), s["tokens"], s["tokens"], 1))
    s["out"] += (torch.empty(s["tokens"], dtype=torch.int64, device="cuda") if case["tree"] else None,)
    if case["tree"]:
        flat = [x for _, p in b for x in p]
        s["parent"] = _ints(flat + [-1] * (s["tokens"] - T))
    return s


def _prepare_append(case, d):
    T, H, pg = case["T"], case["H"], case["page"]
    pool = _pages(T, pg) * 3 // 2 + 1
    t = torch.arange(T, device="cuda")
    rows = d.permutation(pool)[t // pg] * pg + (t % pg)
    first = d.host.randint(0, 8192)
    return {"op": "append", "c_new": d.normal(T, D_LAT), "k_pe_new": d.normal(T, D_ROPE),
            "q_pe": d.normal(T, H, D_ROPE), "slots": rows.to(torch.int32),
            "positions": (first + t % 8192).to(torch.int32), "table": _rotary_table(first + 8192),
            "c_pages": d.normal(pool, pg, D_LAT), "pe_pages": d.normal(pool, pg, D_ROPE),
            "q_pe_out": torch.empty((T, H, D_ROPE), dtype=torch.bfloat16, device="cuda")}


def _prepare_tree(case, d):
    b, pg, H = d.shuffled(_batch(case)), case["page"], case["H"]
    new = [len(p) for _, p in b]
    kv = [c + len(p) for c, p in b]
    held = [_pages(n, pg) for n in kv]
    pool = sum(held) + sum(held) // 8 + 1
    cu = _offsets(new)
    T = cu[-1]
    s = {"op": "tree", "q_nope": d.normal(T, H, D_NOPE), "q_pe": d.normal(T, H, D_ROPE),
         "c_pages": d.normal(pool, pg, D_LAT), "pe_pages": d.normal(pool, pg, D_ROPE),
         "block_table": _table(held, max(held), d.permutation(pool)), "kv_len": _ints(kv),
         "cu_q": _ints(cu), "draft_mask": None, "most_new": max(new), "most_kv": max(kv),
         "w_kvb": d.normal(H * (D_NOPE + D_V), D_LAT, std=D_LAT ** -0.5),
         "out": torch.empty((T, H, D_V), dtype=torch.bfloat16, device="cuda")}
    if case["tree"]:
        s["draft_mask"] = _ints([_signed(m) for _, p in b for m in _ancestors(p)], torch.int64)
    return s


def _prepare_prompt(case, d):
    ns, H, Hkv = d.shuffled(_prompt_lengths(case)), case["H"], case["Hkv"]
    T = sum(ns)
    if case["fused"]:  # slices of the query and key/value projections' outputs
        q, kv = d.normal(T, H, D_NOPE + D_ROPE), d.normal(T, Hkv, D_NOPE + D_V)
        q_nope, q_pe = q[..., :D_NOPE], q[..., D_NOPE:]
        k_nope, v = kv[..., :D_NOPE], kv[..., D_NOPE:]
    else:
        q_nope, q_pe = d.normal(T, H, D_NOPE), d.normal(T, H, D_ROPE)
        k_nope, v = d.normal(T, Hkv, D_NOPE), d.normal(T, Hkv, D_V)
    return {"op": "prompt", "q_nope": q_nope, "q_pe": q_pe, "k_nope": k_nope,
            "k_pe": d.normal(T, D_ROPE), "v": v, "cu_seqlens": _ints(_offsets(ns)),
            "most": max(ns), "out": torch.empty((T, H, D_V), dtype=torch.bfloat16, device="cuda")}


# ---- one pass ---------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"plan": _plain_plan, "append": _plain_append, "tree": _plain_tree,
            "prompt": _plain_prompt}[state["op"]](state)


def _run_own(s):
    import mla_causal_attention_gb300 as mla
    if s["op"] == "plan":
        p = mla.mla_paged_plan(s["ctx_len"], s["new_len"], s["block_table"], s["free_pages"],
                               s["free_head"], s["page"], s["num_pages"], s["tokens"],
                               parent=s["parent"], out=s["out"])
        return {"cu_q": p.cu_q, "kv_len": p.kv_len, "slots": p.slots, "positions": p.positions,
                "free_next": p.free_next, "block_table": s["block_table"],
                "draft_mask": p.draft_mask}
    if s["op"] == "append":
        mla.mla_latent_append(s["c_new"], s["k_pe_new"], s["slots"], s["c_pages"], s["pe_pages"],
                              positions=s["positions"], rope_table=s["table"], q_pe=s["q_pe"],
                              q_pe_out=s["q_pe_out"])
        return {"q_pe": s["q_pe_out"], "c_pages": s["c_pages"], "pe_pages": s["pe_pages"]}
    if s["op"] == "tree":
        return mla.mla_latent_tree_fwd(s["q_nope"], s["q_pe"], s["c_pages"], s["pe_pages"],
                                       s["block_table"], s["kv_len"], s["cu_q"], s["draft_mask"],
                                       s["w_kvb"], SCALE, out=s["out"])
    return mla.mla_attn_varlen_fwd(s["q_nope"], s["q_pe"], s["k_nope"], s["k_pe"], s["v"],
                                   s["cu_seqlens"], SCALE, out=s["out"])


def _rows(cu, T):
    """(sequence, row within it, whether there is one) of each packed row."""
    t = torch.arange(T, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    inside = b < cu.numel() - 1
    b = b.clamp(max=cu.numel() - 2)
    return b, t - cu[b], inside


def _plain_plan(s):
    pg, ctx, new, free = s["page"], s["ctx_len"].long(), s["new_len"].long(), s["free_pages"]
    kv = ctx + new
    before, after = (ctx + pg - 1) // pg, (kv + pg - 1) // pg
    taken = (after - before).cumsum(0)
    first = s["free_head"].long() + taken - (after - before)
    k = torch.arange(s["block_table"].shape[1], device="cuda")[None]
    at = (first[:, None] + k - before[:, None]).clamp(0, free.numel() - 1)
    fresh = (k >= before[:, None]) & (k < after[:, None])
    table = s["block_table"]
    table.copy_(torch.where(fresh, free[at], table))
    cu = torch.cat((new.new_zeros(1), new.cumsum(0)))
    b, i, inside = _rows(cu, s["tokens"])
    p = ctx[b] + i
    slots = table[b, (p // pg).clamp(max=table.shape[1] - 1)] * pg + p % pg
    out = {"cu_q": cu.int(), "kv_len": kv.int(),
           "slots": torch.where(inside, slots, -1).int(),
           "free_next": (s["free_head"] + taken[-1]).int(), "block_table": table,
           "draft_mask": None}
    depth = i
    if s["parent"] is not None:
        # reach[b, i, j]: j is i or an ancestor of i; paths of 1, 2, 4 .. 64 steps
        N = s["most_new"]
        parent = s["parent"].long()
        linked = inside & (parent >= 0)
        reach = torch.eye(N, device="cuda").repeat(ctx.numel(), 1, 1)
        reach.index_put_((b, i.clamp(max=N - 1), parent.clamp(min=0)), linked.float(), accumulate=True)
        for _ in range(6):
            reach = (reach @ reach).clamp(max=1.0)
        mine = reach[b, i.clamp(max=N - 1)] > 0
        mine &= inside[:, None]
        bit = torch.ones(N, dtype=torch.int64, device="cuda") << torch.arange(N, device="cuda")
        out["draft_mask"] = torch.where(mine, bit, torch.zeros_like(bit)).sum(1)
        depth = mine.sum(1) - 1
    out["positions"] = torch.where(inside, ctx[b] + depth, 0).int()
    return out


def _rotate(x, c, s):
    lo, hi = x[..., :32], x[..., 32:]
    return torch.cat((lo * c - hi * s, hi * c + lo * s), -1)


def _plain_append(s):
    at, slots = s["table"][s["positions"].long()], s["slots"].long()
    c, sn = at[:, :32], at[:, 32:]
    s["q_pe_out"].copy_(_rotate(s["q_pe"].float(), c[:, None], sn[:, None]))
    s["pe_pages"].view(-1, D_ROPE)[slots] = _rotate(s["k_pe_new"].float(), c, sn).bfloat16()
    s["c_pages"].view(-1, D_LAT)[slots] = s["c_new"]
    return {"q_pe": s["q_pe_out"], "c_pages": s["c_pages"], "pe_pages": s["pe_pages"]}


def _weights(scores, seen):
    """Softmax over the last axis of the seen scores; a row that sees nothing is all zeros."""
    scores = torch.where(seen, scores, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    e = (scores - torch.where(top == float("-inf"), 0.0, top)).exp()
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, 1.0)


def _plain_tree(s):
    T, H = s["q_nope"].shape[:2]
    pg, kv, N, S = s["c_pages"].shape[1], s["kv_len"].long(), s["most_new"], s["most_kv"]
    B = kv.numel()
    b, i, _ = _rows(s["cu_q"].long(), T)
    ctx = kv - (s["cu_q"][1:] - s["cu_q"][:-1])
    # the latent rows of each request, [B, S, 512 | 64], zeros past its end
    j = torch.arange(S, device="cuda")
    slot = s["block_table"][:, j // pg].clamp(min=0).long() * pg + j % pg
    held = (j < kv[:, None])[..., None]
    c = torch.where(held, s["c_pages"].view(-1, D_LAT)[slot].float(), 0.0)
    pe = torch.where(held, s["pe_pages"].view(-1, D_ROPE)[slot].float(), 0.0)
    # queries folded into the latent space
    w = s["w_kvb"].float().view(H, D_NOPE + D_V, D_LAT)
    q_lat = torch.zeros((B, N, H, D_LAT), device="cuda")
    q_pe = torch.zeros((B, N, H, D_ROPE), device="cuda")
    q_lat[b, i] = torch.einsum("thd,hdl->thl", s["q_nope"].float(), w[:, :D_NOPE])
    q_pe[b, i] = s["q_pe"].float()
    scores = (q_lat.view(B, N * H, D_LAT) @ c.mT + q_pe.view(B, N * H, D_ROPE) @ pe.mT) * SCALE
    # cached keys are seen by all, the new ones through the mask (or in order)
    off = j - ctx[:, None]
    seen = torch.zeros((B, N, S), dtype=torch.bool, device="cuda")
    if s["draft_mask"] is None:
        among = off[b] <= i[:, None]
    else:
        o = off[b]
        among = (o < 0) | ((s["draft_mask"][:, None] >> o.clamp(0, 63)) & 1).bool()
    seen[b, i] = among & (j < kv[b][:, None])
    weights = _weights(scores.view(B, N, H, S), seen[:, :, None])
    o_lat = (weights.view(B, N * H, S) @ c).view(B, N, H, D_LAT)[b, i]
    s["out"].copy_(torch.einsum("thl,hvl->thv", o_lat, w[:, D_NOPE:]))
    return s["out"]


def _plain_prompt(s):
    T, H = s["q_nope"].shape[:2]
    Hkv, L, B = s["k_nope"].shape[1], s["most"], s["cu_seqlens"].numel() - 1
    b, i, _ = _rows(s["cu_seqlens"].long(), T)

    def padded(*parts):
        x = torch.zeros((B, L) + parts[0].shape[1:-1] + (sum(p.shape[-1] for p in parts),),
                        device="cuda")
        x[b, i] = torch.cat([p.float() for p in parts], -1)
        return x

    q = padded(s["q_nope"], s["q_pe"]).view(B, L, Hkv, H // Hkv, D_NOPE + D_ROPE)
    k = padded(s["k_nope"], s["k_pe"][:, None].expand(T, Hkv, D_ROPE))
    v = padded(s["v"])
    scores = torch.einsum("bigrd,bjgd->bgrij", q, k) * SCALE
    order = torch.arange(L, device="cuda")
    weights = _weights(scores, order[None] <= order[:, None])
    del scores
    o = torch.einsum("bgrij,bjgd->bigrd", weights, v).reshape(B, L, H, D_V)
    s["out"].copy_(o[b, i])
    return s["out"]


# ---- from the definitions, in 64 bits ---------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "plan":
        return None
    if s["op"] == "append":
        row = s["table"].double().index_select(0, s["positions"].long())
        z = torch.complex(row[:, :32], row[:, 32:])

        def turn(x):
            x = x.double()
            y = torch.complex(x[..., :32], x[..., 32:]) * (z[:, None] if x.dim() == 3 else z)
            return torch.cat((y.real, y.imag), -1)

        pe = s["pe_pages"].double().view(-1, D_ROPE)
        pe.index_copy_(0, s["slots"].long(), turn(s["k_pe_new"]))
        return {"q_pe": turn(s["q_pe"]), "c_pages": None,
                "pe_pages": pe.view(s["pe_pages"].shape)}
    if s["op"] == "tree":
        return _exact_tree(s)
    cu = s["cu_seqlens"].tolist()
    group = s["q_nope"].shape[1] // s["k_nope"].shape[1]
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    for lo, hi in zip(cu, cu[1:]):
        hidden = torch.ones((hi - lo, hi - lo), dtype=torch.bool, device="cuda").triu(1)
        for h in range(s["q_nope"].shape[1]):
            q = torch.cat((s["q_nope"][lo:hi, h], s["q_pe"][lo:hi, h]), -1).double()
            k = torch.cat((s["k_nope"][lo:hi, h // group], s["k_pe"][lo:hi]), -1).double()
            p = (q @ k.T * SCALE).masked_fill(hidden, float("-inf")).softmax(-1)
            out[lo:hi, h] = p @ s["v"][lo:hi, h // group].double()
    return out


def _exact_tree(s):
    """Each head's keys and values spelled out from the latent rows, request by request."""
    H, pg = s["q_nope"].shape[1], s["c_pages"].shape[1]
    cu, kv = s["cu_q"].tolist(), s["kv_len"].tolist()
    w = s["w_kvb"].double().view(H, D_NOPE + D_V, D_LAT)
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    for r, n_keys in enumerate(kv):
        lo, hi = cu[r], cu[r + 1]
        pages = s["block_table"][r, :_pages(n_keys, pg)].long()
        c = s["c_pages"][pages].reshape(-1, D_LAT)[:n_keys].double()
        pe = s["pe_pages"][pages].reshape(-1, D_ROPE)[:n_keys].double()
        hidden = torch.ones((hi - lo, hi - lo), dtype=torch.bool, device="cuda").triu(1)
        if s["draft_mask"] is not None:
            at = torch.arange(hi - lo, device="cuda")
            hidden = (s["draft_mask"][lo:hi, None] >> at) & 1 == 0
        ctx = n_keys - (hi - lo)
        for h in range(H):
            k = c @ w[h, :D_NOPE].T
            x = s["q_nope"][lo:hi, h].double() @ k.T + s["q_pe"][lo:hi, h].double() @ pe.T
            x *= SCALE
            x[:, ctx:].masked_fill_(hidden, float("-inf"))
            out[lo:hi, h] = x.softmax(-1) @ (c @ w[h, D_NOPE:].T)
    return out
