"""The attention weight that each cached key receives (mla_latent_key_weights) against its definition
in 64 bits, each head's keys spelled out from the latent rows."""
import pytest
import torch

import mla_causal_attention_gb300 as mla
from mla_causal_attention_gb300 import binding
from mla_causal_attention_gb300.workloads import softmax_scale_192
from paged_helpers import tree_case

pytestmark = pytest.mark.gpu

S = binding.MlaStatus
SCALE = softmax_scale_192()


def reference(d, old, decay, scale=SCALE):
    """(weights, worst, held) in 64 bits: worst bounds the error of each weight that the roundings
    make; held marks the slots that are written."""
    H = d["q_nope"].shape[1]
    page = d["c_pages"].shape[1]
    cu, kv = d["cu_q"].tolist(), d["kv_len"].tolist()
    w = d["w_kvb"].double().view(H, 256, 512)
    out, worst = old.double().view(-1).clone(), torch.zeros(old.numel(), device=old.device).double()
    held = torch.zeros(old.numel(), device=old.device, dtype=torch.bool)
    for b, k in enumerate(kv):
        lo, hi = cu[b], cu[b + 1]
        if lo == hi:
            continue
        j = torch.arange(k, device=w.device)
        slot = d["block_table"][b].long()[j // page] * page + j % page
        c, pe = (d[x].view(-1, n)[slot].double() for x, n in (("c_pages", 512), ("pe_pages", 64)))
        new, i = j - (k - (hi - lo)), torch.arange(hi - lo, device=w.device)
        if d["draft_mask"] is None:
            seen = new[None] <= i[:, None]
        else:
            seen = (new < 0) | ((d["draft_mask"][lo:hi, None] >> new.clamp(0, 63)) & 1).bool()
            seen &= new < 64
        q = d["q_nope"][lo:hi].double()
        x = torch.einsum("ihd,hjd->hij", q, torch.einsum("jl,hdl->hjd", c, w[:, :128]))
        x = (x + torch.einsum("ihd,jd->hij", d["q_pe"][lo:hi].double(), pe)) * scale
        x = x.masked_fill(~seen, float("-inf"))
        e = (x - x.amax(-1, keepdim=True).clamp(min=-1e300)).exp()
        total = e.sum(-1, keepdim=True)
        p = e / torch.where(total > 0, total, 1.0)
        # The folded query is off by 2^-8 of 2^-8 of itself, and by fp32's rounding of a sum of 128;
        # a score adds 1088 products in fp32.  Both the score and its row's sum are off by as much.
        ql = torch.einsum("ihd,hdl->hil", q, w[:, :128]).abs()
        qs = torch.einsum("ihd,hdl->hil", q.abs(), w[:, :128].abs())
        size = torch.einsum("hil,jl->hij", ql * 2 ** -16 + qs * 2 ** -17, c.abs())
        size += torch.einsum("ihd,jd->hij", d["q_pe"][lo:hi].double().abs(), pe.abs()) * 2 ** -17
        far = size.masked_fill(~seen, 0.0) * scale
        far = far + far.amax(-1, keepdim=True) + 2 ** -19  # the sum's logarithm, ex2's own error
        got = p.sum((0, 1))
        base = torch.where(new < 0, out[slot] * decay, 0.0) if decay else torch.zeros_like(got)
        out[slot] = base + got
        held[slot] = True
        worst[slot] = (p * far.expm1()).sum((0, 1)) + 2 ** -21 * (got + base.abs())
    return out.view(old.shape), worst.view(old.shape), held.view(old.shape)


def call(d, old, decay, **kw):
    w = old.clone()
    got = mla.mla_latent_key_weights(d["q_nope"], d["q_pe"], d["c_pages"], d["pe_pages"],
                                     d["block_table"], d["kv_len"], d["cu_q"], d["draft_mask"],
                                     d["w_kvb"], SCALE, w, decay=decay, **kw)
    assert got is w
    return w


def check(d, decay, rms=True, old=None):
    if old is None:
        old = torch.rand(d["c_pages"].shape[:2], device="cuda")
    w = call(d, old, decay)
    torch.cuda.synchronize()
    want, worst, held = reference(d, old, decay)
    err = (w.double() - want).abs()
    assert bool((err <= worst).all()), (float(err.max()), float((err - worst).max()))
    assert torch.equal(w[~held], old[~held])  # other slots keep their bits
    if rms and not decay:
        # rounding errors of 512 columns in the 2-norm: 2^-16 / sqrt(3) of sqrt(sum (q_l c_l)^2) =
        # 0.5 sqrt(512), times the scale, for a score and again for its row's sum: 1.5e-5
        assert float((w.double() - want)[held].norm() / want[held].norm()) <= 1.5e-5
    return w


@pytest.mark.parametrize("B,H,ctx,new,page,tree,decay", [
    (1, 64, (0, 0), (1, 1), 16, False, 0.0),        # a single key
    (1, 64, (1000, 1000), (1, 1), 64, False, 1.0),  # one request, one token
    (1, 64, (255, 255), (1, 1), 64, False, 0.0),    # a key tile exactly full
    (1, 64, (256, 256), (1, 1), 64, False, 0.0),    # and one key more
    (64, 64, (0, 900), (1, 1), 32, False, 0.5),     # decode of a ragged batch
    (1, 1, (77, 77), (1, 1), 16, False, 0.0),       # one row
    (3, 5, (0, 400), (0, 7), 16, False, 1.0),       # odd heads; sequences without new tokens
    (2, 128, (100, 300), (2, 3), 128, False, 0.0),  # two row tiles per token
    (5, 16, (0, 300), (1, 64), 64, True, 0.875),    # trees of every size
    (1, 64, (500, 500), (64, 64), 1024, True, 0.0),  # 32 row tiles, few keys: shared key tiles
    (2, 16, (0, 0), (200, 300), 16, False, 0.0),    # whole prompts
    (1, 64, (3000, 3000), (40, 40), 64, False, 0.0),
    (40, 8, (0, 100), (0, 2), 16, True, -1.0),
    (1, 64, (20, 20), (3, 3), 16, False, 0.0),      # fewer steps than pairs
])
def test_matches_64_bits(B, H, ctx, new, page, tree, decay):
    d = tree_case(B + H + page, B, H, ctx, new, page, tree, pad=3)
    check(d, decay)
    assert mla.mla_attn_get_status() == 0


def test_decay_zero_reads_nothing_and_weights_sum_to_the_heads():
    d = tree_case(1, 3, 16, (100, 400), (5, 9), 32, False)
    old = torch.full(d["c_pages"].shape[:2], float("nan"), device="cuda")
    w = call(d, old, 0.0)
    page, total = 32, 0.0
    for b, k in enumerate(d["kv_len"].tolist()):
        j = torch.arange(k, device="cuda")
        s = w.view(-1)[d["block_table"][b].long()[j // page] * page + j % page]
        n = int(d["cu_q"][b + 1] - d["cu_q"][b])
        assert abs(float(s.double().sum()) - n * 16) <= n * 16 * 1e-4  # every row's weights sum to 1
        total += k
    assert int((~w.isnan()).sum()) == total


def test_rows_that_see_nothing_and_hidden_keys_that_are_no_numbers():
    d = tree_case(9, 2, 16, (40, 90), (6, 6), 16, True)
    cu, kv, page = d["cu_q"].tolist(), d["kv_len"].tolist(), 16
    mask = d["draft_mask"]
    for b in range(2):
        mask[cu[b]:cu[b + 1]] &= ~(1 << 3)          # new token 3 is hidden from every row
        j = kv[b] - 6 + 3
        slot = int(d["block_table"][b, j // page]) * page + j % page
        d["c_pages"].view(-1, 512)[slot] = float("nan")
        d["pe_pages"].view(-1, 64)[slot] = float("inf")
    old = torch.rand(d["c_pages"].shape[:2], device="cuda")
    w = call(d, old, 1.0)
    # the same with finite numbers in their place: they do not matter
    e = dict(d, c_pages=d["c_pages"].clone(), pe_pages=d["pe_pages"].clone())
    for b in range(2):
        j = kv[b] - 6 + 3
        slot = int(d["block_table"][b, j // page]) * page + j % page
        e["c_pages"].view(-1, 512)[slot] = 1.0
        e["pe_pages"].view(-1, 64)[slot] = 1.0
        assert float(w.view(-1)[slot]) == 0.0
    assert torch.equal(call(e, old, 1.0), w)
    check(e, 1.0)
    # no cached keys, and rows whose mask is empty: they give nothing, the others go on
    d = tree_case(10, 2, 16, (0, 0), (5, 5), 16, True)
    d["draft_mask"][1] = 0
    d["draft_mask"][5:] = 0
    w = check(d, 0.0, rms=False)
    slot = int(d["block_table"][1, 0]) * 16
    assert w.view(-1)[slot:slot + 5].tolist() == [0.0] * 5


def test_large_scores():
    """Weights of one and zero: scores far apart, maxima that rise from tile to tile."""
    d = tree_case(3, 1, 16, (700, 700), (2, 2), 64, False)
    k = int(d["kv_len"][0])
    j = torch.arange(k, device="cuda")
    slot = d["block_table"][0].long()[j // 64] * 64 + j % 64
    grow = torch.linspace(0.5, 12.0, k, device="cuda")[:, None]
    for name, n in (("c_pages", 512), ("pe_pages", 64)):
        x = d[name].view(-1, n)
        x[slot] = (x[slot].float() * grow).bfloat16()
    check(d, 0.0, rms=False)


def test_repeated_calls_give_the_same_bits():
    """Whatever the order in which the pairs of a shared key tile finish."""
    d = tree_case(4, 3, 64, (100, 700), (30, 60), 64, True)
    old = torch.rand(d["c_pages"].shape[:2], device="cuda")
    first = call(d, old, 1.0)
    for _ in range(20):
        assert torch.equal(call(d, old, 1.0), first)


def test_some_sequences_of_a_batch():
    d = tree_case(5, 4, 16, (50, 200), (1, 9), 16, True)
    part = dict(d, cu_q=d["cu_q"][1:4].contiguous(), kv_len=d["kv_len"][1:3].contiguous(),
                block_table=d["block_table"][1:3].contiguous())
    check(part, 0.0)


def test_long_cache():
    check(tree_case(6, 1, 16, (70000, 70000), (1, 1), 1024, False), 0.0)


def test_many_sequences():
    check(tree_case(12, 600, 4, (0, 60), (0, 3), 16, False), 1.0)


def test_scores_of_some_sequences_are_kept():
    """Four times 512 rows on 40000 keys: the store of 256 MB has room for three of them."""
    d = tree_case(13, 4, 64, (39000, 40000), (8, 8), 1024, True)
    check(d, 0.0)
    # in another order other ones are kept; nothing else changes
    order = torch.tensor([3, 1, 0, 2], device="cuda")
    T = d["q_nope"].shape[0]
    rows = (order[:, None] * 8 + torch.arange(8, device="cuda")).view(-1)
    assert T == 32
    e = dict(d, q_nope=d["q_nope"][rows].contiguous(), q_pe=d["q_pe"][rows].contiguous(),
             draft_mask=d["draft_mask"][rows].contiguous(),
             block_table=d["block_table"][order].contiguous(), kv_len=d["kv_len"][order].contiguous())
    check(e, 0.0)


@pytest.mark.parametrize("at", [16, 32, 64, 128])
@pytest.mark.parametrize("n", [(1, 1), (1, 9)])
def test_a_workspace_that_begins_anywhere(n, at):
    """16-byte alignment is enough; the kept scores' rows begin with a line of L2 or they do not.
    With 32 heads and 1 to 9 tokens a pair goes from sequences of half a unit to full ones and back."""
    d = tree_case(21, 200, 32, (1, 700), n, 16, False)
    old = torch.rand(d["c_pages"].shape[:2], device="cuda")
    want = check(d, 0.5, old=old)
    T, H = d["q_nope"].shape[:2]
    B, pages = d["block_table"].shape
    size = mla.binding.library().mla_latent_key_weights_workspace_bytes(T, H, B, pages * 16)
    ws = mla.Workspace("cuda:0")
    ws.buf = torch.zeros(size + at, dtype=torch.uint8, device="cuda")[at:]
    assert torch.equal(call(d, old, 0.5, workspace=ws), want)
    assert mla.mla_attn_get_status(ws) == 0


def test_pool_past_4_gb():
    """The pages of one sequence at the far end of a pool of 5 million rows."""
    d = tree_case(14, 1, 16, (300, 300), (2, 2), 64, False)
    pages, far = d["c_pages"].shape[0], 80000
    c = torch.empty(far, 64, 512, dtype=torch.bfloat16, device="cuda")
    pe = torch.empty(far, 64, 64, dtype=torch.bfloat16, device="cuda")
    c[-pages:], pe[-pages:] = d["c_pages"], d["pe_pages"]
    old = torch.rand(pages, 64, device="cuda")
    want = call(d, old, 1.0)
    w = torch.zeros(far, 64, device="cuda")
    w[-pages:] = old
    table = torch.where(d["block_table"] < 0, -1, d["block_table"] + far - pages)
    got = call(dict(d, c_pages=c, pe_pages=pe, block_table=table.to(torch.int32)), w, 1.0)
    assert torch.equal(got[-pages:], want) and not bool(got[:-pages].any())


def test_device_side_problems_are_reported():
    ws = mla.Workspace("cuda:0")
    d = tree_case(7, 2, 16, (100, 200), (3, 5), 16, True)
    old = torch.rand(d["c_pages"].shape[:2], device="cuda")

    def status(**change):
        call(dict(d, **change), old, 1.0, workspace=ws)  # d and old as they are by then
        return mla.mla_attn_get_status(ws)

    assert status() == 0
    long = d["kv_len"].clone()
    long[0] = 100000
    assert status(kv_len=long) in (S.ERR_KVLEN, S.ERR_PAGE)
    long[0] = -5
    assert status(kv_len=long) == S.ERR_KVLEN
    cu = d["cu_q"].clone()
    cu[1] = 10000
    assert status(cu_q=cu) == S.ERR_KVLEN
    bad = d["block_table"].clone()
    bad[0, 1] = d["c_pages"].shape[0]
    assert status(block_table=bad) == S.ERR_PAGE
    bad[0, 1] = -7
    assert status(block_table=bad) == S.ERR_PAGE
    d = tree_case(8, 1, 16, (10, 10), (70, 70), 16, False)
    old = torch.rand(d["c_pages"].shape[:2], device="cuda")
    assert status(draft_mask=torch.full((70,), -1, dtype=torch.int64, device="cuda")) == S.ERR_TREE


def test_on_another_stream_and_captured():
    d = tree_case(11, 3, 64, (100, 300), (1, 1), 64, False)
    st, ws = torch.cuda.Stream(), mla.Workspace("cuda:0")
    torch.cuda.synchronize()
    old = torch.rand(d["c_pages"].shape[:2], device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        want = call(d, old, 1.0, workspace=ws)
        w = old.clone()
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            mla.mla_latent_key_weights(d["q_nope"], d["q_pe"], d["c_pages"], d["pe_pages"],
                                       d["block_table"], d["kv_len"], d["cu_q"], None, d["w_kvb"],
                                       SCALE, w, workspace=ws)
        g.replay()
        st.synchronize()
        assert torch.equal(w, want)
        d["q_nope"].copy_(torch.randn_like(d["q_nope"]))
        w.copy_(old)
        g.replay()
        st.synchronize()
        want, worst, _ = reference(d, old, 1.0)
        assert bool(((w.double() - want).abs() <= worst).all())
