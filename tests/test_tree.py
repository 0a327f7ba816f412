"""Attention of new tokens over the paged latent cache (mla_latent_tree_fwd) against its
definition in 64 bits.  Every row of the pool that no sequence holds is NaN.

Tolerances.  The kernels round to bf16 four times on the way: the query folded into the latent
space, the softmax weights, the latent mix, the output.  Each rounding is off by at most half a
step, 2^-8 of the value, at most 2^-8 / sqrt(3) in the root of the mean square, and they are
independent: in the 2-norm the result is within 2 * 2^-8 / sqrt(3) = 0.0045 of the reference.
For one element: the weights err by at most 2^-8 of spread = sum_j p_j |v_j|, the output by 2^-8
of less, and the folded query moves every score by about 2^-8 of itself (scores here are
~N(0, 1): up to five), which is 5 * 2^-8 of the spread: 7 * 2^-8.  The mix is rounded in each of
its 512 latent columns, before the up-projection: column l by at most 2^-8 |mix_l|, so the output
by at most 2^-8 sum_l |W_V[l]| |mix_l|, which does not shrink where the sum over l cancels (a row
that sees two keys whose values nearly cancel in one of the 128 columns)."""
import pytest
import torch

import mla_causal_attention_gb300 as mla
from mla_causal_attention_gb300 import binding
from mla_causal_attention_gb300.workloads import softmax_scale_192
from paged_helpers import tree_case, tree_reference

pytestmark = pytest.mark.gpu

S = binding.MlaStatus
SCALE = softmax_scale_192()


def _run(d, **kw):
    out = mla.mla_latent_tree_fwd(d["q_nope"], d["q_pe"], d["c_pages"], d["pe_pages"],
                                  d["block_table"], d["kv_len"], d["cu_q"], d["draft_mask"],
                                  d["w_kvb"], SCALE, **kw)
    torch.cuda.synchronize()
    return out


def _close(got, d, rows=None):
    """rows: got's rows are these of the case."""
    used = int(d["cu_q"][-1]) if rows is None else len(rows)
    ref, spread, mixed = tree_reference(d, SCALE)
    if rows is not None:
        ref, spread, mixed = ref[rows], spread[rows], mixed[rows]
    err = (got.double() - ref).abs()[:used]
    if used == 0:
        return
    most = 2 ** -8 * (7 * spread + mixed)[:used] + 1e-30
    assert bool(torch.isfinite(got[:used]).all())
    rel = float(err.norm() / ref[:used].norm().clamp(min=1e-30))
    print(f"[tree] rel {rel:.2e} of the bound {float((err / most).max()):.2f}")
    assert rel <= 0.0045
    assert not bool((err > most).any())


CASES = [
    # B, H, cached, new, page, tree
    (1, 64, (0, 0), (1, 1), 64, False),         # a single key
    (1, 64, (1000, 1000), (8, 8), 64, True),
    (1, 64, (1000, 1000), (1, 1), 64, False),   # plain decode
    (5, 64, (0, 600), (0, 5), 16, True),        # sequences without new tokens among others
    (3, 16, (100, 900), (1, 64), 32, True),
    (2, 64, (0, 0), (64, 64), 64, True),        # no cached keys: the tree alone
    (2, 64, (63, 65), (63, 64), 64, False),     # tokens in order, tiles and pages end inside
    (4, 3, (0, 300), (1, 40), 16, True),        # head counts that fill no block of rows
    (3, 1, (0, 300), (1, 64), 128, True),
    (2, 5, (127, 129), (1, 3), 1024, False),
    (2, 128, (200, 300), (1, 3), 64, True),     # more heads than Kimi K2's 64
    (1, 8, (9000, 9000), (17, 17), 128, True),  # long: split over the keys
    (2, 64, (0, 10), (300, 400), 64, False),    # a chunk of a prompt, more than 64 tokens
    (150, 8, (0, 200), (1, 3), 16, True),       # more sequences than there are CTA pairs
    (40, 64, (1, 700), (1, 20), 64, True),
]


@pytest.mark.parametrize("B,H,ctx,new,page,tree", CASES)
def test_tree_matches_definition(B, H, ctx, new, page, tree):
    d = tree_case(B * 7 + H, B, H, ctx, new, page, tree, pad=3)
    out = torch.full((d["q_nope"].shape[0], H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    got = _run(d, out=out)
    assert got is out and mla.mla_attn_get_status() == 0
    _close(got, d)
    assert bool((got[int(d["cu_q"][-1]):] == 7.0).all())  # rows behind the last sequence


def test_tree_random_sweep():
    import random
    r = random.Random(11)
    for k in range(12):
        B, H = r.choice((1, 2, 9, 33)), r.choice((2, 7, 16, 48, 64))
        ctx, new = r.randint(0, 1500), r.randint(1, 64)
        page, tree = r.choice((16, 32, 64, 128, 256)), r.random() < 0.7
        d = tree_case(1000 + k, B, H, (0, ctx), (0, new), page, tree, pad=1)
        print(B, H, ctx, new, page, tree)
        _close(_run(d), d)
    assert mla.mla_attn_get_status() == 0


def test_any_mask_and_rows_that_see_nothing():
    """Bits of any kind; with nothing cached and no bit set a row is zero, and its neighbours
    in the same block of rows are as they would be."""
    d = tree_case(5, 3, 64, (0, 0), (20, 64), 16, True)
    g = torch.Generator("cpu").manual_seed(1)
    m = torch.randint(-2 ** 62, 2 ** 62, d["draft_mask"].shape, generator=g, dtype=torch.int64)
    m[::3] = 0
    m[4] = 1 << 40  # past the sequence's last key, or not: hidden either way if it is
    d["draft_mask"] = m.cuda()
    got = _run(d)
    _close(got, d)
    assert bool((got[::3] == 0).all())
    # with cached keys a zero mask leaves those
    d = tree_case(6, 2, 16, (50, 200), (5, 5), 16, True)
    d["draft_mask"].zero_()
    _close(_run(d), d)


def test_large_scores():
    """Scores of a few hundred: the running maximum moves by more than the type's range."""
    d = tree_case(8, 3, 64, (300, 900), (1, 20), 32, True)
    d["q_nope"] *= 24
    got = _run(d)
    ref, spread, _ = tree_reference(d, SCALE)
    # scores ~N(0, 20^2): the folded query's rounding moves them by up to 100 * 2^-8, so single
    # weights are off by a factor; what has to hold is that rows stay finite mixes of the values
    assert bool(torch.isfinite(got).all())
    assert bool((got.double() - ref).abs().mean() < 0.5 * spread.mean())


def test_equal_scores_average_the_values():
    """q = 0: every visible key has the same weight, and the mix is the mean."""
    d = tree_case(9, 2, 64, (700, 1500), (3, 9), 64, True)
    d["q_nope"].zero_()
    d["q_pe"].zero_()
    _close(_run(d), d)


def test_tree_runs_on_a_side_stream_and_under_a_graph():
    d = tree_case(10, 6, 64, (0, 900), (1, 12), 64, True, pad=5)
    e = tree_case(11, 6, 64, (0, 900), (1, 12), 64, True, pad=5)
    T = max(d["q_nope"].shape[0], e["q_nope"].shape[0])
    width = max(d["block_table"].shape[1], e["block_table"].shape[1])
    num = max(d["c_pages"].shape[0], e["c_pages"].shape[0])

    def fit(c):
        f = dict(c)
        for k, n in (("q_nope", T), ("q_pe", T), ("draft_mask", T), ("c_pages", num),
                     ("pe_pages", num)):
            f[k] = torch.zeros((n,) + c[k].shape[1:], dtype=c[k].dtype, device="cuda")
            f[k][:c[k].shape[0]] = c[k]
        f["block_table"] = torch.full((6, width), -1, dtype=torch.int32, device="cuda")
        f["block_table"][:, :c["block_table"].shape[1]] = c["block_table"]
        return f

    d, e = fit(d), fit(e)
    want = {k: _run(x).clone() for k, x in (("d", d), ("e", e))}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = _run(d, stream=s, workspace=mla.Workspace())
    used = int(d["cu_q"][-1])
    assert torch.equal(side[:used], want["d"][:used])
    st = {k: v.clone() for k, v in d.items()}
    out, ws = torch.empty_like(want["d"]), mla.Workspace()
    _run(st, out=out, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.mla_latent_tree_fwd(st["q_nope"], st["q_pe"], st["c_pages"], st["pe_pages"],
                                st["block_table"], st["kv_len"], st["cu_q"], st["draft_mask"],
                                st["w_kvb"], SCALE, out=out, workspace=ws)
    for name, c in (("e", e), ("d", d)):
        for k, v in c.items():
            st[k].copy_(v)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        n = int(c["cu_q"][-1])
        assert torch.equal(out[:n], want[name][:n])
        assert bool((out[n:] == 0).all())
    assert mla.mla_attn_get_status() == 0


def test_tree_reports_what_only_the_device_sees():
    mla.mla_attn_get_status()
    d = tree_case(12, 3, 16, (20, 60), (2, 4), 16, True)
    good = _run(d)
    cu = d["cu_q"].tolist()

    def other(**change):
        e = dict(d)
        e.update(change)
        return _run(e)

    kv = d["kv_len"].clone()
    kv[1] = 1 << 30
    out = other(kv_len=kv)
    st = mla.mla_attn_get_status()  # the clamped length may also meet entries that hold no page
    assert st in (S.ERR_KVLEN, S.ERR_PAGE)
    assert torch.equal(out[:cu[1]], good[:cu[1]]) and torch.equal(out[cu[2]:], good[cu[2]:])
    kv[1] = 1
    out = other(kv_len=kv)
    assert mla.mla_attn_get_status() == S.ERR_KVLEN
    assert torch.equal(out[cu[2]:], good[cu[2]:])
    table = d["block_table"].clone()
    table[0, 0] = d["c_pages"].shape[0]
    out = other(block_table=table)
    assert mla.mla_attn_get_status() == S.ERR_PAGE
    assert torch.equal(out[cu[1]:], good[cu[1]:])
    table[0, 0] = -1
    other(block_table=table)
    assert mla.mla_attn_get_status() == S.ERR_PAGE
    wide = tree_case(13, 1, 2, (5, 5), (70, 70), 16, False)
    wide["draft_mask"] = torch.ones(70, dtype=torch.int64, device="cuda")
    _run(wide)
    assert mla.mla_attn_get_status() == S.ERR_TREE
    cu_bad = d["cu_q"].clone()
    cu_bad[3] = 1000
    other(cu_q=cu_bad)
    assert mla.mla_attn_get_status() == S.ERR_KVLEN


def test_tree_agrees_with_the_dense_latent_decode():
    """One token per sequence is mla_latent_decode_fwd on the same rows laid end to end."""
    d = tree_case(14, 4, 64, (10, 500), (1, 1), 64, False)
    kv, page = d["kv_len"].tolist(), 64
    Tk = max(kv)
    c = torch.zeros((4, Tk, 512), dtype=torch.bfloat16, device="cuda")
    pe = torch.zeros((4, Tk, 64), dtype=torch.bfloat16, device="cuda")
    for b, k in enumerate(kv):
        j = torch.arange(k, device="cuda")
        slot = d["block_table"][b].long()[j // page] * page + j % page
        c[b, :k], pe[b, :k] = d["c_pages"].view(-1, 512)[slot], d["pe_pages"].view(-1, 64)[slot]
    dense = mla.mla_latent_decode_fwd(d["q_nope"], d["q_pe"], c, pe, d["w_kvb"], d["kv_len"], SCALE)
    _close(_run(d), d)
    _close(dense, d)


def test_a_pool_past_four_gigabytes():
    """Pages whose byte offset does not fit 32 bits."""
    page, num = 1024, 4300
    d = tree_case(15, 2, 16, (1500, 2500), (4, 9), page, True)
    big = {k: torch.empty((num, page, n), dtype=torch.bfloat16, device="cuda")
           for k, n in (("c_pages", 512), ("pe_pages", 64))}
    n_small = d["c_pages"].shape[0]
    far = torch.tensor([num - 1 - 7 * k for k in range(n_small)], device="cuda")
    for k in big:
        big[k][far] = d[k]
    table = torch.where(d["block_table"] >= 0, far[d["block_table"].clamp(min=0).long()].int(), -1)
    e = dict(d, block_table=table.contiguous(), **big)
    assert torch.equal(_run(e), _run(d))


def test_many_empty_sequences():
    """Tokens in the first and the last of 3000 sequences only."""
    d = tree_case(16, 2, 64, (200, 700), (3, 9), 64, True)
    B, width = 3000, d["block_table"].shape[1]
    n0 = int(d["cu_q"][1])
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    table[0], table[-1] = d["block_table"][0], d["block_table"][1]
    kv = torch.zeros(B, dtype=torch.int32, device="cuda")
    kv[0], kv[-1] = d["kv_len"][0], d["kv_len"][1]
    cu = torch.full((B + 1,), n0, dtype=torch.int32, device="cuda")
    cu[0], cu[-1] = 0, int(d["cu_q"][2])
    want = _run(d)
    assert torch.equal(_run(dict(d, block_table=table, kv_len=kv, cu_q=cu)), want)
    assert mla.mla_attn_get_status() == 0


@pytest.mark.parametrize("B", [1025, 8192, 8193, 20000])
def test_many_short_sequences(B):
    """Copies of six sequences, one of them without new tokens, as many as the partition's searches
    in shared memory take, and more."""
    d = tree_case(18, 6, 2, (0, 300), (1, 3), 16, True)
    cu = d["cu_q"].tolist()
    pick = [(5 * b + b // 7) % 6 for b in range(B)]
    none = 3  # its copies ask for nothing
    rows, cu_all, kv = [], [0], []
    for b in pick:
        n = 0 if b == none else cu[b + 1] - cu[b]
        rows += range(cu[b], cu[b] + n)
        cu_all.append(len(rows))
        kv.append(int(d["kv_len"][b]))
    rows = torch.tensor(rows, device="cuda")
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    e = dict(d, block_table=d["block_table"][pick].contiguous(), kv_len=i(kv), cu_q=i(cu_all))
    for k in ("q_nope", "q_pe", "draft_mask"):
        e[k] = d[k][rows].contiguous()
    _close(_run(e), d, rows)
    assert mla.mla_attn_get_status() == 0


def test_sequences_may_share_pages():
    """A common prefix held once: two sequences whose first pages are the same."""
    d = tree_case(17, 2, 16, (640, 640), (4, 4), 64, True)
    d["block_table"][1, :10] = d["block_table"][0, :10]
    _close(_run(d), d)


def test_many_calls_in_flight():
    """Calls of different sizes one behind the other on one workspace, without waiting."""
    cases = [tree_case(30 + k, B, H, (0, ctx), (1, new), 32, tree)
             for k, (B, H, ctx, new, tree) in enumerate(((1, 64, 900, 8, True), (9, 16, 300, 64, True),
                                                         (40, 64, 500, 1, False), (3, 8, 40, 5, True)))]
    want = [_run(d).clone() for d in cases]
    outs = [torch.empty_like(w) for w in want]
    for k in range(200):
        i = k % 4
        d = cases[i]
        mla.mla_latent_tree_fwd(d["q_nope"], d["q_pe"], d["c_pages"], d["pe_pages"],
                                d["block_table"], d["kv_len"], d["cu_q"], d["draft_mask"],
                                d["w_kvb"], SCALE, out=outs[i])
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert torch.equal(w, o)
    assert mla.mla_attn_get_status() == 0


def test_a_workspace_that_is_only_16_byte_aligned():
    d = tree_case(18, 5, 64, (0, 600), (1, 20), 16, True)
    want = _run(d)
    ws = mla.Workspace()
    T, H = d["q_nope"].shape[:2]
    n = binding.library().mla_latent_tree_workspace_bytes(T, H, 5)
    ws.buf = torch.zeros(n + 16, dtype=torch.uint8, device="cuda")[16:]
    assert torch.equal(_run(d, workspace=ws), want)


@pytest.mark.parametrize("T,H,rounds", [(2736, 64, 150), (5000, 16, 150), (288, 64, 150)])
def test_folded_queries_are_the_same_every_time(T, H, rounds):
    """Token counts whose last 128 end early, so that part of the warps have no row to write: every
    call's result is the first one's, whatever the workspace held before."""
    d = tree_case(50, 1, H, (0, 0), (T, T), 64, False)
    ws = mla.Workspace()
    want = _run(d, workspace=ws).clone()
    for k in range(rounds):
        if k % 3 == 0:
            ws.buf[256:].random_(0, 255)
        out = mla.mla_latent_tree_fwd(d["q_nope"], d["q_pe"], d["c_pages"], d["pe_pages"],
                                      d["block_table"], d["kv_len"], d["cu_q"], d["draft_mask"],
                                      d["w_kvb"], SCALE, workspace=ws)
        assert torch.equal(out, want), k


@pytest.mark.parametrize("new", [(1, 4), (20, 60)])  # merged in the up-projection, and apart
def test_some_of_a_batchs_sequences(new):
    """The last sequences of a batch in a call of their own: the rows in front are left alone."""
    d = tree_case(19, 4, 64, (100, 500), new, 32, True)
    cu = d["cu_q"].tolist()
    out = torch.full_like(d["q_nope"], 7.0)
    e = dict(d, cu_q=d["cu_q"][2:].contiguous(), kv_len=d["kv_len"][2:].contiguous(),
             block_table=d["block_table"][2:].contiguous())
    _run(e, out=out)
    assert mla.mla_attn_get_status() == 0
    assert bool((out[:cu[2]] == 7.0).all())
    _close(out[cu[2]:], d, list(range(cu[2], cu[4])))


@pytest.mark.parametrize("new", [(1, 4), (20, 60)])  # merged in the up-projection, and apart
def test_a_sequence_without_keys_is_zero(new):
    """New tokens whose sequence has no keys at all (a bad length): reported, and their rows see
    nothing; the other sequences come out as they would."""
    mla.mla_attn_get_status()
    d = tree_case(20, 4, 64, (100, 500), new, 32, True, pad=1)
    cu = d["cu_q"].tolist()
    kv = d["kv_len"].clone()
    kv[1], kv[2] = 0, -5
    out = torch.full_like(d["q_nope"], 7.0)
    _run(dict(d, kv_len=kv), out=out)
    assert mla.mla_attn_get_status() == S.ERR_KVLEN
    assert bool((out[cu[1]:cu[3]] == 0).all()) and bool((out[cu[4]:] == 7.0).all())
    rows = [*range(cu[1]), *range(cu[3], cu[4])]
    _close(out[rows], d, rows)
