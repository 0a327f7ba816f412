"""Bookkeeping and append of the paged latent cache (mla_paged_plan, mla_latent_append)
against plain forms: whole numbers equal, copied rows bit-identical, rotated rows within one
rounding of their 64-bit values."""
import random

import pytest
import torch

import mla_causal_attention_gb300 as mla
from mla_causal_attention_gb300 import binding
from paged_helpers import plan_reference, random_batch, random_parents, rotate64

pytestmark = pytest.mark.gpu

S = binding.MlaStatus


def _i(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def _plan(c, n, table, free, head, page, num, T, parents=None, **kw):
    t = _i(table)
    p = mla.mla_paged_plan(_i(c), _i(n), t, _i(free), _i([head]), page, num, T,
                           parent=None if parents is None else _i(parents + [-1] * (T - len(parents))),
                           **kw)
    torch.cuda.synchronize()
    return p, t


def _same(p, t, want):
    cu, kv, slots, pos, nxt, mask, table = want
    assert p.cu_q.tolist() == cu
    assert p.kv_len.tolist() == kv
    assert p.slots.tolist() == slots
    assert p.positions.tolist() == pos
    assert p.free_next.tolist() == [nxt]
    assert t.tolist() == table
    if p.draft_mask is not None:
        assert p.draft_mask.tolist() == mask


@pytest.mark.parametrize("B,ctx,new,page,tree", [
    (1, (0, 0), (1, 1), 16, False),          # the first token of the first request
    (1, (15, 15), (1, 1), 16, False),        # fills a page
    (1, (16, 16), (1, 1), 16, False),        # opens a page
    (64, (0, 300), (1, 1), 64, False),       # a decode step
    (5, (0, 0), (0, 700), 32, False),        # prompts, some empty
    (9, (0, 100), (0, 3), 16, False),        # sequences without new tokens among others
    (3, (0, 0), (0, 0), 16, False),          # nothing to do
    (300, (0, 40), (0, 64), 128, True),      # trees of every size
    (2, (63, 65), (64, 64), 64, True),       # the widest mask
    (1025, (0, 50), (0, 5), 16, True),       # one sequence past a scan's 1024
    (5000, (0, 20), (0, 3), 1024, False),    # several scans
    (7, (0, 5000), (1, 6000), 16, False),    # tokens of a sequence over many blocks
    (1500, (0, 50), (0, 200), 16, False),    # several scans, few and many pages per sequence
    (2, (0, 10), (20000, 30000), 16, False),  # a table row over many blocks
])
def test_plan(B, ctx, new, page, tree):
    r, c, n, table, free, num = random_batch(B + page, B, ctx, new, page)
    T = sum(n) + r.choice((0, 1, 5, 64))
    T = max(T, 1)
    par = [x for k in n for x in random_parents(r, k, roots=True)] if tree else None
    free = [0, 1] + free  # entries in front of free_head are not touched
    p, t = _plan(c, n, table, free, 2, page, num, T, par)
    _same(p, t, plan_reference(c, n, table, free, 2, page, T, par))
    assert mla.mla_attn_get_status() == 0


def test_plan_fills_given_buffers_and_replays():
    """A captured plan follows its inputs, and free_next feeds the next step's free_head."""
    page = 16
    r, c, n, table, free, num = random_batch(3, 20, (0, 90), (1, 4), page)
    free = free + list(range(num, num + 60))  # for a second step
    num += 60
    T = 128
    ctx, new, tab, head = _i(c), _i(n), _i(table), _i([0])
    out = mla.PagedPlan(_i([0] * 21), _i([0] * 20), _i([7] * T), _i([7] * T), _i([0]), None)
    g = torch.cuda.CUDAGraph()
    mla.mla_paged_plan(ctx, new, tab, _i(free), head, page, num, T, out=out)
    fl = _i(free)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        mla.mla_paged_plan(ctx, new, tab, fl, head, page, num, T, out=out)
    want = plan_reference(c, n, table, free, 0, page, T)
    _same(out, tab, want)
    # the second step: cached lengths and the head move on
    c2 = want[1]
    n2 = [r.randint(0, 6) for _ in c2]
    width = len(table[0])
    n2 = [k if x + k <= width * page else 0 for x, k in zip(c2, n2)]
    ctx.copy_(_i(c2)); new.copy_(_i(n2)); head.copy_(out.free_next)
    g.replay()
    torch.cuda.synchronize()
    _same(out, tab, plan_reference(c2, n2, want[6], free, want[4], page, T))
    assert mla.mla_attn_get_status() == 0


def test_plan_reports_what_only_the_device_sees():
    page = 16
    mla.mla_attn_get_status()
    # a free list that runs out: entries and slots -1, everything else as usual
    c, n, table = [0, 10], [40, 30], [[-1] * 4, [9] + [-1] * 3]
    p, t = _plan(c, n, table, [5, 6, 7, 8], 0, page, 10, 80)
    _same(p, t, plan_reference(c, n, table, [5, 6, 7, 8], 0, page, 80))
    assert mla.mla_attn_get_status() == S.ERR_PAGE
    # a free entry outside the pool
    p, t = _plan([0], [5], [[-1]], [10], 0, page, 10, 5)
    assert p.slots.tolist() == [-1] * 5 and t.tolist() == [[-1]]
    assert mla.mla_attn_get_status() == S.ERR_PAGE
    # a table entry outside the pool
    p, _ = _plan([3], [2], [[10]], [1], 0, page, 10, 2)
    assert p.slots.tolist() == [-1, -1]
    assert mla.mla_attn_get_status() == S.ERR_PAGE
    # lengths past the table, and below zero
    p, t = _plan([30, -4], [10, 2], [[3, 4], [-1, -1]], [1, 2], 0, page, 10, 12)
    assert p.kv_len.tolist() == [32, 2] and p.cu_q.tolist() == [0, 10, 12]
    assert p.slots.tolist() == [4 * 16 + 14, 4 * 16 + 15] + [-1] * 8 + [16, 17]
    assert mla.mla_attn_get_status() == S.ERR_KVLEN
    # more tokens than rows
    p, _ = _plan([0, 0], [3, 3], [[-1], [-1]], [1, 2], 0, page, 10, 4)
    assert p.cu_q.tolist() == [0, 3, 4] and p.slots.tolist() == [16, 17, 18, 32]
    assert mla.mla_attn_get_status() == S.ERR_KVLEN
    # a parent after its token, and 65 drafted tokens
    p, _ = _plan([4], [3], [[2]], [], 0, page, 10, 3, [-1, 1, 0])
    assert p.positions.tolist() == [4, 4, 5] and p.draft_mask.tolist() == [1, 2, 5]
    assert mla.mla_attn_get_status() == S.ERR_TREE
    p, _ = _plan([0], [65], [[-1] * 5], list(range(5)), 0, page, 10, 65, [-1] + list(range(64)))
    assert p.draft_mask.tolist()[62:] == [(1 << 63) - 1, -1, 0]
    assert mla.mla_attn_get_status() == S.ERR_TREE


def _append_case(seed, T, H, page, num, rope=True):
    g = torch.Generator("cpu").manual_seed(seed)
    mk = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    slots = torch.randperm(num * page, generator=g)[:T].to(torch.int32)
    d = dict(c=mk(T, 512), pe=mk(T, 64), slots=slots, c_pages=mk(num, page, 512),
             pe_pages=mk(num, page, 64), q=mk(T, H, 64) if H else None,
             pos=torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32) if rope else None)
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def _near(got, want):
    """bf16 results of 64-bit values: half a step of bf16 for the final rounding, and the fp32
    products and sum before it (two products and a sum, three roundings of 2^-24 of |x| + |y|
    <= 2 max|x| sqrt(2)), which can tip a value over to the next bf16: a whole step, and that."""
    err = (got.double() - want).abs()
    assert bool((err <= want.abs() * 2 ** -7 + want.abs().max() * 2 ** -20).all())
    assert float((err > want.abs() * 2 ** -8 + want.abs().max() * 2 ** -20).double().mean()) < 1e-3


@pytest.mark.parametrize("T,H,page,num", [
    (1, 64, 16, 1), (7, 3, 16, 2), (64, 64, 64, 40), (333, 16, 128, 5), (5000, 1, 32, 200),
])
def test_append_rotates_and_scatters(T, H, page, num):
    d = _append_case(T, T, H, page, num)
    table = mla.mla_rope_table(5000)
    d["slots"][T // 2] = -1 if T > 1 else d["slots"][0]
    keep = d["slots"] >= 0
    want_c, want_pe = d["c_pages"].clone(), d["pe_pages"].double()
    at = d["slots"][keep].long()
    want_c.view(-1, 512)[at] = d["c"][keep]
    untouched = torch.ones(num * page, dtype=torch.bool, device="cuda")
    untouched[at] = False
    before = d["pe_pages"].clone()
    out = torch.full_like(d["q"], 3.0)
    got = mla.mla_latent_append(d["c"], d["pe"], d["slots"], d["c_pages"], d["pe_pages"],
                                positions=d["pos"], rope_table=table, q_pe=d["q"], q_pe_out=out)
    assert got is out and mla.mla_attn_get_status() == 0
    assert torch.equal(d["c_pages"], want_c)
    assert torch.equal(d["pe_pages"].view(-1, 64)[untouched], before.view(-1, 64)[untouched])
    _near(d["pe_pages"].view(-1, 64)[at], rotate64(d["pe"], table, d["pos"])[keep])
    _near(out[keep], rotate64(d["q"], table, d["pos"])[keep])
    assert bool((out[~keep] == 3.0).all())  # a skipped row's query is left as it was
    # in place: the same values
    mla.mla_latent_append(d["c"], d["pe"], d["slots"], d["c_pages"], d["pe_pages"],
                          positions=d["pos"], rope_table=table, q_pe=d["q"], q_pe_out=d["q"])
    assert torch.equal(d["q"][keep], out[keep])


def test_append_copies_without_a_table_on_a_side_stream():
    d = _append_case(1, 100, 0, 16, 10, rope=False)
    want_c, want_pe = d["c_pages"].clone(), d["pe_pages"].clone()
    want_c.view(-1, 512)[d["slots"].long()] = d["c"]
    want_pe.view(-1, 64)[d["slots"].long()] = d["pe"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert mla.mla_latent_append(d["c"], d["pe"], d["slots"], d["c_pages"], d["pe_pages"],
                                 workspace=mla.Workspace(), stream=s) is None
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(d["c_pages"], want_c) and torch.equal(d["pe_pages"], want_pe)


def test_append_reports_bad_slots_and_positions():
    d = _append_case(2, 4, 1, 16, 2)
    table = mla.mla_rope_table(8)
    d["slots"].copy_(_i([3, 32, 5, -7]))
    d["pos"].copy_(_i([0, 1, 2, 3]))
    before = d["c_pages"].clone().view(-1, 512)
    before[3], before[5] = d["c"][0], d["c"][2]
    mla.mla_latent_append(d["c"], d["pe"], d["slots"], d["c_pages"], d["pe_pages"],
                          positions=d["pos"], rope_table=table, q_pe=d["q"])
    assert mla.mla_attn_get_status() == S.ERR_PAGE
    assert torch.equal(d["c_pages"].view(-1, 512), before)
    d["slots"].copy_(_i([0, 1, 2, 3]))
    d["pos"].copy_(_i([0, 8, -1, 7]))
    q = mla.mla_latent_append(d["c"], d["pe"], d["slots"], d["c_pages"], d["pe_pages"],
                              positions=d["pos"], rope_table=table, q_pe=d["q"])
    assert mla.mla_attn_get_status() == S.ERR_KVLEN
    _near(q, rotate64(d["q"], table, d["pos"].clamp(0, 7)))


def test_append_past_two_gigabytes():
    """Slots whose byte offset does not fit 32 bits."""
    page, num = 1024, 4200  # 4.4 GB of latent rows
    c_pages = torch.empty((num, page, 512), dtype=torch.bfloat16, device="cuda")
    pe_pages = torch.empty((num, page, 64), dtype=torch.bfloat16, device="cuda")
    slots = [num * page - 1, 2 ** 31 // 1024, 2 ** 32 // 1024 + 5, 0]
    g = torch.Generator("cpu").manual_seed(0)
    c, pe = (torch.randn(4, w, generator=g).to(torch.bfloat16).cuda() for w in (512, 64))
    mla.mla_latent_append(c, pe, _i(slots), c_pages, pe_pages)
    at = _i(slots, torch.int64)
    assert torch.equal(c_pages.view(-1, 512)[at], c)
    assert torch.equal(pe_pages.view(-1, 64)[at], pe)
    assert mla.mla_attn_get_status() == 0
