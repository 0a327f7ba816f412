"""Choice of a paged cache's rows within a budget (mla_paged_evict) and their compaction
(mla_latent_compact) against plain lists: whole numbers equal, rows bit-identical."""
import random

import pytest
import torch

import mla_causal_attention_gb300 as mla
from mla_causal_attention_gb300 import binding
from paged_helpers import pages

pytestmark = pytest.mark.gpu

S = binding.MlaStatus


def _i(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def keep_reference(w, n, budget, sinks, recent):
    """The kept rows of one sequence with weights w (a list)."""
    k = min(n, budget)
    if k == n:
        return list(range(n))
    s = min(sinks, k)
    r = min(recent, k - s)
    order = sorted(range(s, n - r), key=lambda j: (w[j] != w[j], -w[j] if w[j] == w[j] else 0, j))
    return list(range(s)) + sorted(order[:k - s - r]) + list(range(n - r, n))


def pool_of(lens, page, seed, extra=1, spare=3):
    """(block table as lists, pages of the pool)."""
    r = random.Random(seed)
    held = [pages(n, page) for n in lens]
    width = max(1, max(held)) + extra
    ids = list(range(sum(held) + spare))
    r.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (width - h))
        at += h
    return table, len(ids)


def slots_of(row, n, page):
    j = torch.arange(n)
    return torch.tensor(row)[j // page] * page + j % page


def _draw_weights(kind, n, seed):
    g = torch.Generator("cpu").manual_seed(seed)
    if kind == "plain":
        return torch.randn(n, generator=g).mul(2).exp()
    if kind == "ties":
        return torch.randint(0, 4, (n,), generator=g).float()
    if kind == "equal":
        return torch.zeros(n)
    w = torch.randn(n, generator=g)  # signed, with everything that floats have
    odd = [float("nan"), float("inf"), float("-inf"), 0.0, -0.0, 1e-42, -1e-42]
    pick = torch.randint(0, 4 * len(odd), (n,), generator=g)
    for k, x in enumerate(odd):
        w[pick == k] = x
    return w


def run_case(lens, budgets, sinks, recent, page, kind, seed, K=None, extra=1):
    table, num = pool_of(lens, page, seed, extra)
    per = [_draw_weights(kind, n, seed + b) for b, n in enumerate(lens)]
    pool = torch.full((num * page,), float("inf"))  # what no sequence holds would be heaviest
    for row, n, w in zip(table, lens, per):
        pool[slots_of(row, n, page)] = w
    kw = {} if K is None else {"max_keep": K}
    p = mla.mla_paged_evict(pool.view(num, page).cuda(), _i(table), _i(lens), _i(budgets), sinks,
                            recent, **kw)
    torch.cuda.synchronize()
    want = [keep_reference(w.tolist(), n, k, sinks, recent) for w, n, k in zip(per, lens, budgets)]
    assert p.kept_len.tolist() == [len(x) for x in want]
    kept = p.kept.cpu()
    for b, x in enumerate(want):
        assert kept[b, :len(x)].tolist() == x, b
        assert bool((kept[b, len(x):] == -1).all())
    free = [q for row, n, x in zip(table, lens, want)
            for q in row[pages(len(x), page):pages(n, page)]]
    assert int(p.n_freed) == len(free) and p.freed[:len(free)].tolist() == free
    assert mla.mla_attn_get_status() == 0
    return p


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "odd"])
@pytest.mark.parametrize("lens,budgets,sinks,recent,page", [
    ([1], [0], 0, 0, 16),                          # all of one row goes
    ([1], [1], 4, 4, 16),
    ([0, 5, 0], [3, 2, 0], 1, 1, 16),              # nothing held
    ([100], [99], 0, 0, 16),                       # one row goes
    ([100], [1], 4, 8, 16),                        # the first sink alone
    ([100], [6], 4, 8, 16),                        # sinks, then as many of the last as fit
    ([100], [50], 4, 46, 64),                      # ends fill the budget
    ([333, 1000, 64, 65, 2047], [64, 64, 64, 64, 64], 4, 16, 64),
    ([5000], [1234], 3, 77, 32),                   # a cluster of several CTAs
    ([40000], [33333], 16, 1000, 128),             # 16 of them
    ([3000, 3001, 2999], [10, 3001, 2998], 0, 0, 16),
])
def test_choice(lens, budgets, sinks, recent, page, kind):
    run_case(lens, budgets, sinks, recent, page, kind, len(lens) + lens[0])


@pytest.mark.parametrize("B", [70, 160, 1500])   # two CTAs per sequence, one, several waves
def test_choice_of_many(B):
    r = random.Random(B)
    lens = [r.randint(0, 4500 if B < 200 else 300) for _ in range(B)]
    budgets = [r.randint(0, 1 + n) for n in lens]
    run_case(lens, budgets, 2, 5, 16, "ties", B, K=max(1, max(map(min, lens, budgets))))


def test_choice_of_more_rows_than_shared_memory_holds():
    # 16 CTAs of 56251 rows, 49152 of them in shared memory
    run_case([900009], [300000], 4, 128, 1024, "ties", 1, K=300000)
    run_case([900009], [450000], 4, 128, 1024, "plain", 1, K=450000)


def test_lengths_far_below_the_table():
    run_case([40, 7], [20, 7], 1, 2, 16, "plain", 3, extra=60000, K=32)


def test_without_freed_pages_and_into_given_buffers():
    table, num = pool_of([50, 20], 16, 0)
    w = torch.rand(num, 16, device="cuda")
    kept, n = _i([[7] * 30] * 2), _i([0, 0])
    p = mla.mla_paged_evict(w, _i(table), _i([50, 20]), _i([30, 30]), 2, 2,
                            out=(kept, n, None, None))
    assert p.kept is kept and n.tolist() == [30, 20]
    assert kept[1].tolist() == list(range(20)) + [-1] * 10
    freed = _i([9] * (2 * len(table[0])))
    p = mla.mla_paged_evict(w, _i(table), _i([50, 20]), _i([10, 3]), 2, 2,
                            out=(kept, n, freed, _i([0])))
    got = table[0][1:4] + table[1][1:2]
    assert freed.tolist() == got + [9] * (len(freed) - len(got)) and int(p.n_freed) == 4


def test_choice_reports_what_only_the_device_sees():
    ws = mla.Workspace("cuda:0")
    table, num = pool_of([40, 40], 16, 5)
    w = torch.rand(num, 16, device="cuda")

    def call(table, lens, budgets, K=40, **kw):
        p = mla.mla_paged_evict(w, _i(table), _i(lens), _i(budgets), 0, 0, max_keep=K,
                                workspace=ws, **kw)
        torch.cuda.synchronize()
        return p, mla.mla_attn_get_status(ws)

    p, st = call(table, [-3, 40], [10, 10])
    assert st == S.ERR_KVLEN and p.kept_len.tolist() == [0, 10]
    p, st = call(table, [40, 5000], [10, 10])   # past the table: clamped to its 64 positions
    assert st == S.ERR_PAGE or st == S.ERR_KVLEN
    assert p.kept_len.tolist() == [10, 10]
    p, st = call(table, [40, 40], [-1, 40])
    assert st == S.ERR_KVLEN and p.kept_len.tolist() == [0, 40]
    p, st = call(table, [40, 40], [30, 20], K=25)
    assert st == S.ERR_KVLEN and p.kept_len.tolist() == [25, 20]
    bad = [list(r) for r in table]
    bad[0][1], bad[1][0] = num, -1              # rows of pages that do not exist go first
    p, st = call(bad, [40, 40], [24, 24])
    assert st == S.ERR_PAGE
    assert p.kept[0, :24].tolist() == list(range(16)) + list(range(32, 40))
    assert p.kept[1, :24].tolist() == list(range(16, 40))


# ---- compaction -------------------------------------------------------------------------

def _bits(*s, seed):
    g = torch.Generator("cpu").manual_seed(seed)
    return torch.randint(-2 ** 15, 2 ** 15, s, generator=g, dtype=torch.int32).to(torch.int16).view(
        torch.bfloat16)  # any pattern, NaN and infinities among them


def compact_case(lens, keep, page, seed, weights=True, extra=1):
    """keep: the kept rows of each sequence."""
    table, num = pool_of(lens, page, seed, extra)
    c, pe = _bits(num, page, 512, seed=seed), _bits(num, page, 64, seed=seed + 1)
    w = torch.randn(num, page)
    K = max(1, max(map(len, keep))) + 3
    kept = [list(x) + [-1] * (K - len(x)) for x in keep]
    dev = [c.cuda(), pe.cuda(), w.cuda()]
    mla.mla_latent_compact(dev[0], dev[1], _i(table), _i(kept), _i([len(x) for x in keep]),
                           weights=dev[2] if weights else None)
    torch.cuda.synchronize()
    assert mla.mla_attn_get_status() == 0
    for old, new, width in ((c, dev[0], 512), (pe, dev[1], 64), (w, dev[2], 1)):
        view = torch.int32 if width == 1 else torch.int16
        old, new = old.view(view).view(-1, width), new.cpu().view(view).view(-1, width)
        touched = torch.zeros(num * page, dtype=torch.bool)
        for row, n, x in zip(table, lens, keep):
            if width == 1 and not weights:
                continue
            s = slots_of(row, n, page) if n else torch.zeros(0, dtype=torch.int64)
            assert torch.equal(new[s[:len(x)]], old[s[torch.tensor(x, dtype=torch.int64)]])
            touched[s[:len(x)]] = True
        assert torch.equal(new[~touched], old[~touched])  # rows behind, other pages


def _some(r, n, k):
    return sorted(r.sample(range(n), k))


@pytest.mark.parametrize("lens,ks,page", [
    ([1], [0], 16), ([1], [1], 16), ([0, 40], [0, 17], 16),
    ([100], [99], 16), ([300], [256], 64), ([5000], [2500], 32), ([9000], [8999], 64),
    ([333, 1000, 64, 65, 2047], [64, 900, 64, 1, 1024], 64),
    ([4097] * 40, [2000] * 40, 128),   # slices of 128 bytes
    ([20000], [15000], 1024),          # many runs, overlapping sources and targets
])
def test_compaction(lens, ks, page):
    r = random.Random(sum(lens))
    compact_case(lens, [_some(r, n, k) for n, k in zip(lens, ks)], page, len(lens))


def test_compaction_of_shifted_runs():
    """Everything moves by a little: each row's target is another row's source."""
    for gap in (1, 2, 31, 255, 256, 1023, 1025):
        compact_case([6000], [list(range(gap, 6000))], 64, gap)
    compact_case([6000, 70], [list(range(6000)), list(range(70))], 64, 0)  # nothing moves
    compact_case([3000], [list(range(0, 3000, 2))], 16, 1, weights=False, extra=5000)


def test_compaction_of_many():
    r = random.Random(5)
    lens = [r.randint(0, 90) for _ in range(1500)]
    compact_case(lens, [_some(r, n, r.randint(0, n)) for n in lens], 16, 3)


def test_compaction_in_a_pool_past_4_gb():
    page, n, far = 64, 500, 80000
    pages_n = pages(n, page)
    c = torch.empty(far, page, 512, dtype=torch.bfloat16, device="cuda")
    pe = torch.empty(far, page, 64, dtype=torch.bfloat16, device="cuda")
    rows = [torch.randn(pages_n, page, k, device="cuda").bfloat16() for k in (512, 64)]
    c[-pages_n:], pe[-pages_n:] = rows
    table = torch.arange(far - pages_n, far, device="cuda", dtype=torch.int32)[None].contiguous()
    kept = list(range(0, n, 3))
    mla.mla_latent_compact(c, pe, table, _i([kept]), _i([len(kept)]))
    torch.cuda.synchronize()
    for pool, old in zip((c, pe), rows):
        old = old.view(-1, old.shape[-1])
        new = pool[-pages_n:].reshape(-1, old.shape[-1])
        assert torch.equal(new[:len(kept)], old[torch.tensor(kept, device="cuda")])
        assert torch.equal(new[len(kept):], old[len(kept):])


def test_calls_on_two_streams():
    """Two servers' compactions at once, each with a workspace of its own."""
    page, n = 64, 20000
    sets = []
    for k in range(2):
        table = torch.randperm(pages(n, page), device="cuda", dtype=torch.int32)[None].contiguous()
        c, pe = (torch.randn(pages(n, page), page, w, device="cuda").bfloat16() for w in (512, 64))
        kept = _some(random.Random(k), n, n - 3000 * (k + 1))
        sets.append((c, pe, table, _i([kept]), _i([len(kept)]), c.clone(), kept,
                     torch.cuda.Stream(), mla.Workspace("cuda:0")))
    torch.cuda.synchronize()
    for c, pe, table, kept, k, _, _, st, ws in sets:
        mla.mla_latent_compact(c, pe, table, kept, k, workspace=ws, stream=st)
    torch.cuda.synchronize()
    for c, pe, table, _, _, before, kept, st, ws in sets:
        s = slots_of(table[0].tolist(), n, page).cuda()
        at = torch.tensor(kept, device="cuda")
        assert torch.equal(c.view(-1, 512)[s[:len(kept)]], before.view(-1, 512)[s[at]])
        assert mla.mla_attn_get_status(ws, stream=st) == 0


def test_compaction_skips_what_is_no_such_list():
    ws = mla.Workspace("cuda:0")
    page = 16
    table, num = pool_of([40], page, 2)

    def call(kept, n, table=table):
        c, pe = torch.randn(num, page, 512).bfloat16().cuda(), torch.randn(num, page, 64).bfloat16().cuda()
        before = c.clone()
        mla.mla_latent_compact(c, pe, _i(table), _i([kept]), _i([n]), workspace=ws)
        torch.cuda.synchronize()
        s = slots_of([max(x, 0) for x in table[0]], 40, page)
        return c.view(-1, 512).cpu(), before.view(-1, 512).cpu(), s, mla.mla_attn_get_status(ws)

    new, old, s, st = call([0, 0, 5], 3)     # below its own index
    assert st == S.ERR_KVLEN
    assert torch.equal(new[s[:2]], old[s[:2]]) and torch.equal(new[s[2]], old[s[5]])
    new, old, s, st = call([0, 5000, 6], 3)  # past the table
    assert st == S.ERR_KVLEN and torch.equal(new[s[1]], old[s[1]]) and torch.equal(new[s[2]], old[s[6]])
    new, old, s, st = call([3, 5], 7)        # more than the list has
    assert st == S.ERR_KVLEN and torch.equal(new[s[1]], old[s[5]])
    new, old, s, st = call([3, 5], -1)
    assert st == S.ERR_KVLEN and torch.equal(new, old)
    bad = [list(table[0])]
    bad[0][1] = num
    new, old, s, st = call([3, 20, 35], 3, bad)
    assert st == S.ERR_PAGE
    s = slots_of([max(x, 0) for x in table[0]], 40, page)
    assert torch.equal(new[s[0]], old[s[3]]) and torch.equal(new[s[1]], old[s[1]])
    assert torch.equal(new[s[2]], old[s[35]])


def test_choice_and_compaction_replayed_on_another_stream():
    """A captured choice and compaction follow their inputs; each layer keeps its own rows."""
    page, lens = 16, [200, 90]
    table, num = pool_of(lens, page, 7)
    st = torch.cuda.Stream()
    ws = mla.Workspace("cuda:0")
    with torch.cuda.stream(st):
        w = torch.rand(num, page, device="cuda")
        c, pe = (torch.randn(num, page, n, device="cuda").bfloat16() for n in (512, 64))
        tab, kv, budget = _i(table), _i(lens), _i([64, 64])
        out = mla.mla_paged_evict(w, tab, kv, budget, 2, 8, max_keep=64, workspace=ws)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            mla.mla_paged_evict(w, tab, kv, budget, 2, 8, out=out, workspace=ws)
            mla.mla_latent_compact(c, pe, tab, out.kept, out.kept_len, weights=w, workspace=ws)
        for seed in (1, 2):
            torch.manual_seed(seed)
            w.copy_(torch.rand(num, page))
            c.copy_(torch.randn(num, page, 512))
            w0, c0 = w.view(-1).cpu().clone(), c.view(-1, 512).cpu().clone()
            g.replay()
            st.synchronize()
            for b, n in enumerate(lens):
                s = slots_of(table[b], n, page)
                x = keep_reference(w0[s].tolist(), n, 64, 2, 8)
                assert out.kept[b].tolist() == x
                assert torch.equal(c.view(-1, 512).cpu()[s[:64]], c0[s[x]])
                assert torch.equal(w.view(-1).cpu()[s[:64]], w0[s[x]])
        assert mla.mla_attn_get_status(ws, stream=st) == 0
