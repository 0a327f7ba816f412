"""Operators of long-running requests, measured: each in its plain form (elementary torch operations)
and, with ``own`` set, through the framework's entry points.

  rope     the rotary step by itself: interleaved or half layout, slices of wider heads, inverse
  weights  the attention weight that every cached key receives from a step's tokens
  evict    which rows of each sequence's cache stay within a budget, and the pages that come free
  compact  the kept rows moved to the front of their sequence's pages

Lengths, budgets and trees are drawn once per case from its "lens" number; the seed permutes them
over the batch and draws everything else, so the work of a case does not depend on the seed.
"""
import random

import torch

own = False

D_NOPE, D_ROPE, D_V, D_LAT = 128, 64, 128, 512
SCALE = (D_NOPE + D_ROPE) ** -0.5
MOST_POS = 131072
TYPES = {"bf16": (torch.bfloat16, 2), "fp16": (torch.float16, 2), "fp32": (torch.float32, 4)}


# ---- cases ------------------------------------------------------------------------------

def listed():
    return [
        # a decode step's rotary queries, slices of the query projection's rows, from a
        # checkpoint whose rotary columns come in neighbouring pairs, into the cache's halves
        {"name": "rope_decode", "op": "rope", "T": 64, "H": 64, "R": 64, "W": 192, "type": "bf16",
         "layout": "interleaved", "out_layout": "half", "inverse": False, "in_place": False},
        # the same for the rows of several packed prompts, an odd number of them
        {"name": "rope_prompts", "op": "rope", "T": 16411, "H": 64, "R": 64, "W": 192,
         "type": "bf16", "layout": "interleaved", "out_layout": "half", "inverse": False,
         "in_place": False},
        # gradients (or cached keys) turned back where they are; a quarter of each head is rotary
        {"name": "rope_back", "op": "rope", "T": 4099, "H": 16, "R": 32, "W": 128, "type": "fp32",
         "layout": "half", "out_layout": "half", "inverse": True, "in_place": True},
        # one request, 1000 cached keys, one token: latency
        {"name": "weights_one", "op": "weights", "B": 1, "H": 64, "ctx_lo": 1000, "ctx_hi": 1000,
         "new_lo": 1, "new_hi": 1, "tree": False, "page": 64, "decay": 1.0, "lens": 1},
        # ordinary decode of a ragged batch, one token per request
        {"name": "weights_decode", "op": "weights", "B": 64, "H": 64, "ctx_lo": 512,
         "ctx_hi": 8192, "new_lo": 1, "new_hi": 1, "tree": False, "page": 64, "decay": 1.0,
         "lens": 2},
        # drafted trees of up to 16 tokens, fewer heads, older weight fading
        {"name": "weights_tree", "op": "weights", "B": 32, "H": 16, "ctx_lo": 512, "ctx_hi": 8192,
         "new_lo": 1, "new_hi": 16, "tree": True, "page": 32, "decay": 0.96875, "lens": 3},
        # the last 32 tokens of long prompts observe the whole prompt; nothing held before counts
        {"name": "weights_window", "op": "weights", "B": 16, "H": 64, "ctx_lo": 4096,
         "ctx_hi": 8160, "new_lo": 32, "new_hi": 32, "tree": False, "page": 64, "decay": 0.0,
         "lens": 4},
        # a ragged batch cut down to a budget
        {"name": "evict_batch", "op": "evict", "B": 64, "len_lo": 1024, "len_hi": 8192,
         "keep_lo": 2048, "keep_hi": 2048, "sinks": 4, "recent": 256, "page": 64, "lens": 5},
        # two very long requests
        {"name": "evict_long", "op": "evict", "B": 2, "len_lo": 400000, "len_hi": 500000,
         "keep_lo": 100000, "keep_hi": 131072, "sinks": 16, "recent": 4096, "page": 64, "lens": 6},
        # one request a little over its budget: latency
        {"name": "compact_one", "op": "compact", "B": 1, "len_lo": 2112, "len_hi": 2112,
         "keep_lo": 2048, "keep_hi": 2048, "sinks": 4, "recent": 256, "page": 64, "lens": 7},
        # the ragged batch's rows
        {"name": "compact_batch", "op": "compact", "B": 64, "len_lo": 1024, "len_hi": 8192,
         "keep_lo": 2048, "keep_hi": 2048, "sinks": 4, "recent": 256, "page": 64, "lens": 8},
        # one very long request
        {"name": "compact_long", "op": "compact", "B": 1, "len_lo": 262144, "len_hi": 262144,
         "keep_lo": 65536, "keep_hi": 65536, "sinks": 16, "recent": 4096, "page": 64, "lens": 9},
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], its logarithm about uniform."""
    return max(lo, min(hi, int(lo * (hi / lo) ** rng.random() + rng.random())))


def draw(rng):
    op = rng.choice(("rope", "weights", "weights", "evict", "compact"))
    lens, page = rng.randrange(1 << 30), rng.choice((16, 32, 64, 128))
    if op == "rope":
        R = rng.choice((32, 64, 64, 96, 128))
        in_place = rng.random() < 0.3
        layout = rng.choice(("half", "interleaved"))
        kind, H = rng.choice(("bf16", "bf16", "fp16", "fp32")), rng.choice((1, 8, 16, 64))
        most = 16411 * 64 * 128 // (H * R * TYPES[kind][1])
        return {"op": op, "T": _log_int(rng, 1, min(65536, most)), "H": H, "R": R,
                "W": rng.choice((R, 128 + R)), "type": kind, "layout": layout,
                "out_layout": rng.choice(("half", "interleaved")),
                "inverse": rng.random() < 0.5, "in_place": in_place}
    if op == "weights":
        H, n = rng.choice((8, 16, 32, 64)), rng.randint(1, 64)
        ctx = _log_int(rng, 1, 131072)
        most = 16 * 32 * 64 * 8192 // (H * n * (ctx + n))
        if most == 0:
            n, most = 1, 16 * 32 * 64 * 8192 // (H * (ctx + 1))
        return {"op": op, "B": _log_int(rng, 1, max(1, min(64, most))), "H": H,
                "ctx_lo": rng.randint(0, ctx), "ctx_hi": ctx, "new_lo": rng.randint(1, n),
                "new_hi": n, "tree": rng.random() < 0.5, "page": page,
                "decay": rng.choice((0.0, 1.0, 1.0, 0.875)), "lens": lens}
    if op == "evict":
        n = _log_int(rng, 128, 500000)
        B = _log_int(rng, 1, max(1, min(512, 1000000 // n)))
    else:
        n = _log_int(rng, 32, 262144)
        B = _log_int(rng, 1, max(1, min(256, 262144 // n)))
    # a single request is over its budget; of several, some may be within theirs
    keep = _log_int(rng, 16, n // 2 if B == 1 else n)
    return {"op": op, "B": B, "len_lo": rng.randint(n // 2, n), "len_hi": n,
            "keep_lo": rng.randint(16, keep), "keep_hi": keep, "sinks": rng.randint(0, 8),
            "recent": rng.randint(0, keep // 4), "page": page, "lens": lens}


def _batch(case):
    """The requests of a weights case: (cached length, parents of the new tokens)."""
    r = random.Random(case["lens"])
    out = []
    for _ in range(case["B"]):
        ctx, n = r.randint(case["ctx_lo"], case["ctx_hi"]), r.randint(case["new_lo"], case["new_hi"])
        # token 0 is the root; the others hang off one of the eight tokens before them
        parents = [-1] + [r.randint(max(0, i - 8), i - 1) for i in range(1, n)] if case["tree"] \
            else [-1] * n
        out.append((ctx, parents))
    return out


def _budgets(case):
    """The requests of an evict or compact case: (cached length, budget)."""
    r = random.Random(case["lens"])
    return [(r.randint(case["len_lo"], case["len_hi"]), r.randint(case["keep_lo"], case["keep_hi"]))
            for _ in range(case["B"])]


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
    if op == "rope":
        n = case["T"] * case["H"] * case["R"]
        return {"bytes": 2 * n * TYPES[case["type"]][1] + case["T"] * (4 + 4 * case["R"]),
                "flops": 3 * n}
    if op == "weights":
        b, H = _batch(case), case["H"]
        T = sum(len(p) for _, p in b)
        keys = sum(c + len(p) for c, p in b)
        old = sum(c for c, _ in b) if case["decay"] else 0
        if case["tree"]:
            pairs = sum(c * len(p) + sum(bin(m).count("1") for m in _ancestors(p)) for c, p in b)
        else:
            pairs = sum(c * len(p) + len(p) * (len(p) + 1) // 2 for c, p in b)
        return {"bytes": keys * ((D_LAT + D_ROPE) * 2 + 4) + old * 4
                + T * H * (D_NOPE + D_ROPE) * 2 + H * D_NOPE * D_LAT * 2,
                "flops": pairs * H * 2 * (D_LAT + D_ROPE) + T * H * 2 * D_NOPE * D_LAT}
    b, pg = _budgets(case), case["page"]
    if op == "evict":
        cut = [(n, k) for n, k in b if n > k]
        return {"bytes": sum(4 * n + 4 * _pages(n, pg) for n, _ in cut) + 12 * len(b)
                + sum(4 * min(n, k) for n, k in b)
                + sum(8 * (_pages(n, pg) - _pages(k, pg)) for n, k in cut), "flops": 0}
    moved = sum(max(k - case["sinks"], 0) for n, k in b if n > k)
    return {"bytes": moved * 2 * ((D_LAT + D_ROPE) * 2 + 4) + sum(4 * min(n, k) for n, k in b),
            "flops": 0}


# ---- inputs -----------------------------------------------------------------------------

class _Draw:
    """Random device tensors of one seed."""

    def __init__(self, seed):
        self.host = random.Random(seed)
        self.gen = torch.Generator("cuda").manual_seed(seed)

    def normal(self, *shape, std=1.0, dtype=torch.bfloat16):
        x = torch.empty(shape, dtype=dtype, device="cuda")
        return x.normal_(0.0, std, generator=self.gen)

    def uniform(self, *shape):
        return torch.rand(shape, generator=self.gen, device="cuda")

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


def _rotary_table(rows, R):
    """cos | sin of positions, the slower half of the frequencies scaled for a longer context."""
    d = torch.arange(R // 2, dtype=torch.float64, device="cuda")
    f = 50000.0 ** (-2.0 * d / R)
    f = torch.where(d < R // 4, f, f / 32.0)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat((a.cos(), a.sin()), 1).float()


def _held_weights(d, *shape):
    """Accumulated weights as a long decode leaves them: a few large ones, many small, some none."""
    w = d.normal(*shape, std=2.0, dtype=torch.float32).exp_()
    return torch.where(d.uniform(*shape) < 0.05, torch.zeros_like(w), w)


def prepare(case, seed):
    d = _Draw(seed)
    return {"rope": _prepare_rope, "weights": _prepare_weights, "evict": _prepare_evict,
            "compact": _prepare_compact}[case["op"]](case, d)


def _prepare_rope(case, d):
    T, H, R, W = case["T"], case["H"], case["R"], case["W"]
    x = d.normal(T, H, W, dtype=TYPES[case["type"]][0])[..., W - R:]
    first = d.host.randint(0, MOST_POS - 1)
    positions = (first + torch.arange(T, device="cuda")) % MOST_POS
    return {"op": "rope", "x": x, "positions": positions.to(torch.int32),
            "table": _rotary_table(MOST_POS, R), "layout": case["layout"],
            "out_layout": case["out_layout"], "inverse": case["inverse"],
            "out": x if case["in_place"] else torch.empty((T, H, R), dtype=x.dtype, device="cuda")}


def _prepare_weights(case, d):
    b, pg, H = d.shuffled(_batch(case)), case["page"], case["H"]
    new = [len(p) for _, p in b]
    kv = [c + len(p) for c, p in b]
    held = [_pages(n, pg) for n in kv]
    pool = sum(held) + sum(held) // 8 + 1
    cu = _offsets(new)
    T = cu[-1]
    s = {"op": "weights", "q_nope": d.normal(T, H, D_NOPE), "q_pe": d.normal(T, H, D_ROPE),
         "c_pages": d.normal(pool, pg, D_LAT), "pe_pages": d.normal(pool, pg, D_ROPE),
         "block_table": _table(held, max(held), d.permutation(pool)), "kv_len": _ints(kv),
         "cu_q": _ints(cu), "draft_mask": None, "most_new": max(new), "most_kv": max(kv),
         "w_kvb": d.normal(H * (D_NOPE + D_V), D_LAT, std=D_LAT ** -0.5), "decay": case["decay"],
         # one page more, which no table names; a prompt's first weights come into fresh pages
         "room": _held_weights(d, pool + 1, pg) if case["decay"] else
                 torch.zeros(pool + 1, pg, device="cuda")}
    s["weights"] = s["room"][:pool]
    if case["tree"]:
        s["draft_mask"] = _ints([_signed(m) for _, p in b for m in _ancestors(p)], torch.int64)
    return s


def _prepare_evict(case, d):
    b, pg = d.shuffled(_budgets(case)), case["page"]
    kv = [n for n, _ in b]
    held = [_pages(n, pg) for n in kv]
    width, pool = max(held), sum(held) + sum(held) // 8 + 1
    B, K = len(b), max(k for _, k in b)
    return {"op": "evict", "weights": _held_weights(d, pool, pg), "kv_len": _ints(kv),
            "block_table": _table(held, width, d.permutation(pool)), "most_kv": max(kv),
            "budget": _ints([k for _, k in b]), "sinks": case["sinks"], "recent": case["recent"],
            # the buffers that a server fills anew every time
            "out": (torch.full((B, K), -1, dtype=torch.int32, device="cuda"),
                    torch.empty(B, dtype=torch.int32, device="cuda"),
                    torch.full((B * width,), -1, dtype=torch.int32, device="cuda"),
                    torch.empty(1, dtype=torch.int32, device="cuda"))}


def _prepare_compact(case, d):
    b, pg = d.shuffled(_budgets(case)), case["page"]
    kv = [n for n, _ in b]
    held = [_pages(n, pg) for n in kv]
    pool = sum(held) + sum(held) // 8 + 1
    n, S = _ints(kv)[:, None], max(kv)
    k = torch.minimum(_ints([x for _, x in b])[:, None], n)
    # the first rows, the last ones, and any of the others
    j = torch.arange(S, device="cuda")[None]
    sinks = k.clamp(max=case["sinks"])
    recent = (k - sinks).clamp(max=case["recent"])
    rank = d.uniform(len(b), S)
    rank = torch.where((j < sinks) | (j >= n - recent), 2.0, rank)
    rank = torch.where(j < n, rank, -1.0)
    order = rank.argsort(1, descending=True)
    K = int(k.max())
    first = torch.where(j[:, :K] < k, order[:, :K], S).sort(1).values
    kept = torch.where(first < S, first, -1).to(torch.int32)
    # pools with one page more, which no table names
    s = {"op": "compact", "c_room": d.normal(pool + 1, pg, D_LAT),
         "pe_room": d.normal(pool + 1, pg, D_ROPE), "w_room": _held_weights(d, pool + 1, pg),
         "block_table": _table(held, max(held), d.permutation(pool)), "kept": kept,
         "kept_len": k[:, 0].to(torch.int32)}
    s["c_pages"], s["pe_pages"], s["weights"] = (s[x][:pool] for x in ("c_room", "pe_room", "w_room"))
    return s


# ---- one pass ---------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"rope": _plain_rope, "weights": _plain_weights, "evict": _plain_evict,
            "compact": _plain_compact}[state["op"]](state)


def _run_own(s):
    import mla_causal_attention_gb300 as mla
    if s["op"] == "rope":
        return mla.mla_rope_apply(s["x"], s["positions"], s["table"], layout=s["layout"],
                                  out_layout=s["out_layout"], inverse=s["inverse"], out=s["out"])
    if s["op"] == "weights":
        return mla.mla_latent_key_weights(s["q_nope"], s["q_pe"], s["c_pages"], s["pe_pages"],
                                          s["block_table"], s["kv_len"], s["cu_q"],
                                          s["draft_mask"], s["w_kvb"], SCALE, s["weights"],
                                          decay=s["decay"])
    if s["op"] == "evict":
        p = mla.mla_paged_evict(s["weights"], s["block_table"], s["kv_len"], s["budget"],
                                s["sinks"], s["recent"], out=s["out"])
        return {"kept": p.kept, "kept_len": p.kept_len, "freed": p.freed, "n_freed": p.n_freed}
    mla.mla_latent_compact(s["c_pages"], s["pe_pages"], s["block_table"], s["kept"], s["kept_len"],
                           weights=s["weights"])
    return {"c_pages": s["c_pages"], "pe_pages": s["pe_pages"], "weights": s["weights"]}


def _plain_rope(s):
    R = s["table"].shape[1]
    at = s["table"][s["positions"].long()][:, None]
    c, sn = at[..., :R // 2], at[..., R // 2:]
    if s["inverse"]:
        sn = -sn
    x = s["x"].float()
    if s["layout"] == "half":
        lo, hi = x[..., :R // 2], x[..., R // 2:]
    else:
        lo, hi = x[..., 0::2], x[..., 1::2]
    y = (lo * c - hi * sn, hi * c + lo * sn)
    s["out"].copy_(torch.cat(y, -1) if s["out_layout"] == "half" else torch.stack(y, -1).flatten(-2))
    return s["out"]


def _slots(table, j, page):
    """The slots [B, n] of positions j ([n] or [B, n]) in each row of a block table."""
    at = (j // page).clamp(max=table.shape[1] - 1)
    held = table[:, at] if j.dim() == 1 else table.gather(1, at)
    return held.clamp(min=0).long() * page + j % page


def _plain_weights(s):
    T, H = s["q_nope"].shape[:2]
    pg, kv, N, S = s["c_pages"].shape[1], s["kv_len"].long(), s["most_new"], s["most_kv"]
    B, cu = kv.numel(), s["cu_q"].long()
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    i = t - cu[b]
    ctx = kv - (cu[1:] - cu[:-1])
    # the latent rows of each request, [B, S, 512 | 64], zeros past its end
    j = torch.arange(S, device="cuda")
    slot, held = _slots(s["block_table"], j, pg), j < kv[:, None]
    c = torch.where(held[..., None], s["c_pages"].view(-1, D_LAT)[slot].float(), 0.0)
    pe = torch.where(held[..., None], s["pe_pages"].view(-1, D_ROPE)[slot].float(), 0.0)
    # queries folded into the latent space
    w = s["w_kvb"].float().view(H, D_NOPE + D_V, D_LAT)
    q_lat = torch.zeros((B, N, H, D_LAT), device="cuda")
    q_pe = torch.zeros((B, N, H, D_ROPE), device="cuda")
    q_lat[b, i] = torch.einsum("thd,hdl->thl", s["q_nope"].float(), w[:, :D_NOPE])
    q_pe[b, i] = s["q_pe"].float()
    x = (q_lat.view(B, N * H, D_LAT) @ c.mT + q_pe.view(B, N * H, D_ROPE) @ pe.mT) * SCALE
    # cached keys are seen by all, the new ones through the mask (or in order)
    off = (j - ctx[:, None])[b]
    seen = torch.zeros((B, N, S), dtype=torch.bool, device="cuda")
    if s["draft_mask"] is None:
        among = off <= i[:, None]
    else:
        among = (off < 0) | ((s["draft_mask"][:, None] >> off.clamp(0, 63)) & 1).bool()
    seen[b, i] = among & held[b]
    x = torch.where(seen[:, :, None], x.view(B, N, H, S), float("-inf"))
    top = x.amax(-1, keepdim=True)
    e = (x - torch.where(top == float("-inf"), 0.0, top)).exp()
    del x
    total = e.sum(-1, keepdim=True)
    got = torch.einsum("bnhs,bnh->bs", e, (1.0 / torch.where(total > 0, total, 1.0))[..., 0])
    # cached keys go on from what they hold, new ones begin
    room = s["room"].view(-1)
    got += torch.where(j < ctx[:, None], room[slot] * s["decay"], 0.0)
    room[torch.where(held, slot, room.numel() - 1)] = got
    return s["weights"]


def _plain_evict(s):
    pg, n, S = s["weights"].shape[1], s["kv_len"].long()[:, None], s["most_kv"]
    kept, kept_len, freed, n_freed = s["out"]
    table, K = s["block_table"], kept.shape[1]
    k = torch.minimum(s["budget"].long()[:, None], n)
    sinks = k.clamp(max=s["sinks"])
    recent = (k - sinks).clamp(max=s["recent"])
    j = torch.arange(S, device="cuda")[None]
    # the first rows, the last ones, then by weight; a stable order, so ties go to lower rows
    w = s["weights"].view(-1)[_slots(table, j[0], pg)]
    w = torch.where((j < sinks) | (j >= n - recent), float("inf"), w)
    order = torch.where(j < n, w, float("-inf")).sort(dim=1, descending=True, stable=True).indices
    stays = torch.zeros((n.numel(), S), dtype=torch.bool, device="cuda")
    stays.scatter_(1, order, j.expand_as(order) < k)
    at = stays.cumsum(1) - 1
    # a column more for the rows that go
    rows = torch.full((n.numel(), K + 1), -1, dtype=torch.int64, device="cuda")
    rows.scatter_(1, torch.where(stays, at, K), j.expand_as(at))
    kept.copy_(torch.where(torch.arange(K, device="cuda") < k, rows[:, :K], -1))
    kept_len.copy_(k[:, 0])
    # pages behind the kept rows, in order
    p = torch.arange(table.shape[1], device="cuda")[None]
    free = (p >= (k + pg - 1) // pg) & (p < (n + pg - 1) // pg)
    to = free.view(-1).cumsum(0) - 1
    n_freed.copy_(to[-1:] + 1)
    listed_pages = torch.cat((freed, freed[:1]))
    listed_pages[torch.where(free.view(-1), to, freed.numel())] = table.view(-1)
    freed.copy_(listed_pages[:-1])
    return {"kept": kept, "kept_len": kept_len, "freed": freed, "n_freed": n_freed}


def _plain_compact(s):
    pg, table, kept = s["c_pages"].shape[1], s["block_table"], s["kept"].long()
    i = torch.arange(kept.shape[1], device="cuda")
    real = i < s["kept_len"][:, None]
    spare = s["w_room"].numel() - 1
    src = torch.where(real, _slots(table, kept.clamp(min=0), pg), spare).view(-1)
    dst = torch.where(real, _slots(table, i, pg), spare).view(-1)
    c, pe, w = s["c_room"].view(-1, D_LAT), s["pe_room"].view(-1, D_ROPE), s["w_room"].view(-1)
    c[dst] = c[src]
    pe[dst] = pe[src]
    w[dst] = w[src]
    return {"c_pages": s["c_pages"], "pe_pages": s["pe_pages"], "weights": s["weights"]}


# ---- from the definitions, in 64 bits ---------------------------------------------------

def exact(case, seed):
    if case["op"] not in ("rope", "weights"):  # whole numbers and copied rows
        return None
    s = prepare(case, seed)
    if case["op"] == "weights":
        return _exact_weights(s)
    R = case["R"]
    row = s["table"].double().index_select(0, s["positions"].long())
    z = torch.complex(row[:, :R // 2], row[:, R // 2:])
    x = s["x"].double()
    if s["layout"] == "interleaved":
        x = torch.view_as_complex(x.unflatten(-1, (R // 2, 2)).contiguous())
    else:
        x = torch.complex(x[..., :R // 2], x[..., R // 2:])
    y = torch.view_as_real(x * (z.conj() if s["inverse"] else z)[:, None])
    return y.flatten(-2) if s["out_layout"] == "interleaved" else y.movedim(-1, -2).flatten(-2)


def _exact_weights(s):
    """Each head's keys spelled out from the latent rows, request by request."""
    H, pg = s["q_nope"].shape[1], s["c_pages"].shape[1]
    cu, kv = s["cu_q"].tolist(), s["kv_len"].tolist()
    w = s["w_kvb"].double().view(H, D_NOPE + D_V, D_LAT)
    out = s["weights"].double()
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
        got = torch.zeros(n_keys, dtype=torch.float64, device="cuda")
        for h in range(H):
            x = s["q_nope"][lo:hi, h].double() @ (c @ w[h, :D_NOPE].T).T
            x += s["q_pe"][lo:hi, h].double() @ pe.T
            x *= SCALE
            x[:, ctx:].masked_fill_(hidden, float("-inf"))
            got += x.softmax(-1).sum(0)
        mine = out[pages].view(-1)
        mine[:ctx] = mine[:ctx] * s["decay"] + got[:ctx]
        mine[ctx:n_keys] = got[ctx:]
        out[pages] = mine.view(-1, pg)
    return out
