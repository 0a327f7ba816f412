"""The key weights' second pass takes one of three ways, by rows: scores kept and the rows' sums put
together where they are read (up to 512 rows in all), kept and read (up to 512 rows of a sequence), or
computed again.  What can go wrong in one of them is tested in each."""
import pytest
import torch

import mla_causal_attention_gb300 as mla
from paged_helpers import tree_case
from test_key_weights import SCALE, call, reference

pytestmark = pytest.mark.gpu

WAYS = ["merged", "kept", "computed", "both"]


def case(way, seed, ctx, page=16, tree=True, pad=1):
    B, H, new = {"merged": (2, 16, (6, 8)), "kept": (3, 64, (6, 8)), "computed": (2, 64, (9, 12)),
                 "both": (6, 64, (6, 12))}[way]
    d = tree_case(seed, B, H, ctx, new, page, tree, pad=pad)
    rows = [(int(d["cu_q"][b + 1]) - int(d["cu_q"][b])) * H for b in range(B)]
    if way == "merged":
        assert d["q_nope"].shape[0] * H <= 512
    else:
        assert d["q_nope"].shape[0] * H > 512
        assert any(r <= 512 for r in rows) == (way != "computed")
        assert any(r > 512 for r in rows) == (way != "kept")
    return d


def slots(d, b):
    """Slots of sequence b's keys."""
    page = d["c_pages"].shape[1]
    j = torch.arange(int(d["kv_len"][b]), device=d["kv_len"].device)
    return d["block_table"][b].long()[j // page] * page + j % page


def seen_by(d, b, i):
    """Which of sequence b's keys its new token i sees."""
    lo, k = int(d["cu_q"][b]), int(d["kv_len"][b])
    new = torch.arange(k, device=d["kv_len"].device) - (k - (int(d["cu_q"][b + 1]) - lo))
    if d["draft_mask"] is None:
        return new <= i
    return (new < 0) | ((d["draft_mask"][lo + i] >> new.clamp(0, 63)) & 1).bool()


def close(w, d, old, decay, but=None):
    """w against the 64-bit form, except where `but` says."""
    want, worst, held = reference(d, old, decay)
    ok = (w.double() - want).abs() <= worst
    if but is not None:
        ok |= but
    assert bool(ok.all())
    assert torch.equal(w[~held], old[~held])


@pytest.mark.parametrize("decay", [0.0, 0.5])
@pytest.mark.parametrize("what", ["query", "key"])
@pytest.mark.parametrize("way", WAYS)
def test_rows_that_are_no_numbers_leave_alone_what_they_do_not_see(way, what, decay):
    d = case(way, 31, (70, 300))
    B = d["kv_len"].shape[0]
    for b in range(B):  # token 1 sees itself alone, tokens 3 and 4 see 3, nothing else does
        lo, hi = int(d["cu_q"][b]), int(d["cu_q"][b + 1])
        d["draft_mask"][lo:hi] &= ~(2 | 8)
        d["draft_mask"][lo + 1] = 2
        d["draft_mask"][lo + 3:lo + 5] |= 8
    e = {k: x.clone() if x is not None else None for k, x in d.items()}
    lost = torch.zeros(d["c_pages"].shape[:2], dtype=torch.bool, device="cuda").view(-1)
    for b in range(0, B, 2):
        at = slots(d, b)
        if what == "query":
            d["q_nope"][int(d["cu_q"][b]) + 1, 3, 5] = float("nan")
            lost[at[seen_by(d, b, 1)]] = True
        else:
            n = int(d["cu_q"][b + 1] - d["cu_q"][b])
            d["c_pages"].view(-1, 512)[at[int(d["kv_len"][b]) - n + 3], 7] = float("nan")
            for i in (3, 4):
                lost[at[seen_by(d, b, i)]] = True
    lost = lost.view(d["c_pages"].shape[:2])
    old = torch.rand(lost.shape, device="cuda")
    w = call(d, old, decay)
    assert bool(w[lost].isnan().all()) and not bool(w[~lost].isnan().any())
    close(w, e, old, decay, but=lost)
    assert mla.mla_attn_get_status() == 0


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("way", WAYS)
def test_every_way_matches_64_bits(way, tree):
    d = case(way, 32, (0, 400), page=32, tree=tree)
    old = torch.rand(d["c_pages"].shape[:2], device="cuda")
    for decay in (0.0, 1.0, -0.5):
        close(call(d, old, decay), d, old, decay)


@pytest.mark.parametrize("way", WAYS)
def test_hidden_keys_that_are_no_numbers(way):
    d = case(way, 33, (40, 200))
    e = {k: x.clone() if x is not None else None for k, x in d.items()}
    hidden = []
    for b in range(d["kv_len"].shape[0]):  # new token 3 is hidden from every row
        lo, hi = int(d["cu_q"][b]), int(d["cu_q"][b + 1])
        for x in (d, e):
            x["draft_mask"][lo:hi] &= ~8
        at = slots(d, b)[int(d["kv_len"][b]) - (hi - lo) + 3]
        hidden.append(at)
        d["c_pages"].view(-1, 512)[at] = float("nan")
        d["pe_pages"].view(-1, 64)[at] = float("inf")
        e["c_pages"].view(-1, 512)[at] = 1.0
        e["pe_pages"].view(-1, 64)[at] = 1.0
    old = torch.rand(d["c_pages"].shape[:2], device="cuda")
    w = call(d, old, 0.5)
    assert w.view(-1)[torch.stack(hidden)].tolist() == [0.0] * len(hidden)
    assert torch.equal(call(e, old, 0.5), w)  # what stands there does not matter
    close(w, e, old, 0.5)


@pytest.mark.parametrize("way", WAYS)
def test_rows_that_see_nothing(way):
    d = case(way, 34, (0, 0))
    lo, hi = int(d["cu_q"][0]), int(d["cu_q"][1])
    d["draft_mask"][lo:hi] = 0         # no row of the first sequence sees anything
    d["draft_mask"][hi:hi + 2] = 0     # two tokens of the second
    old = torch.rand(d["c_pages"].shape[:2], device="cuda")
    w = call(d, old, 1.0)
    assert not bool(w.view(-1)[slots(d, 0)].any())
    close(w, d, old, 1.0)


@pytest.mark.parametrize("way", WAYS)
def test_decay_zero_reads_nothing(way):
    d = case(way, 35, (100, 400))
    old = torch.full(d["c_pages"].shape[:2], float("nan"), device="cuda")
    w = call(d, old, 0.0)
    H, total = d["q_nope"].shape[1], 0
    for b in range(d["kv_len"].shape[0]):
        at = slots(d, b)
        n = int(d["cu_q"][b + 1] - d["cu_q"][b])
        assert abs(float(w.view(-1)[at].double().sum()) - n * H) <= n * H * 1e-4
        total += len(at)
    assert int((~w.isnan()).sum()) == total


@pytest.mark.parametrize("way", WAYS)
def test_scores_far_apart(way):
    d = case(way, 36, (500, 700), page=64)
    for b in range(d["kv_len"].shape[0]):
        at = slots(d, b)
        grow = torch.linspace(0.5, 12.0, len(at), device="cuda")[:, None]
        for name, n in (("c_pages", 512), ("pe_pages", 64)):
            x = d[name].view(-1, n)
            x[at] = (x[at].float() * grow).bfloat16()
    old = torch.zeros(d["c_pages"].shape[:2], device="cuda")
    close(call(d, old, 0.0), d, old, 0.0)


@pytest.mark.parametrize("outside", [-7, -1, 1 << 20])
@pytest.mark.parametrize("way", WAYS)
def test_pages_outside_the_pool_count_as_zeros(way, outside):
    d = case(way, 37, (100, 300))
    ws = mla.Workspace("cuda:0")
    old = torch.rand(d["c_pages"].shape[:2], device="cuda")
    gone = d["block_table"][:, 2].long()  # positions 32 to 47 of every sequence
    e = dict(d, c_pages=d["c_pages"].clone(), pe_pages=d["pe_pages"].clone())
    e["c_pages"][gone] = 0.0
    e["pe_pages"][gone] = 0.0
    table = d["block_table"].clone()
    table[:, 2] = outside
    w = call(dict(d, block_table=table), old, 1.0, workspace=ws)
    assert mla.mla_attn_get_status(ws) == mla.binding.MlaStatus.ERR_PAGE
    assert torch.equal(w[gone], old[gone])  # nothing is written for them
    zeros = call(e, old, 1.0)
    zeros[gone] = old[gone]
    assert torch.equal(w, zeros)


@pytest.mark.parametrize("B,ctx,new", [(2, 35000, 5), (1, 70000, 10)])  # kept; computed again
def test_long_caches(B, ctx, new):
    d = tree_case(38, B, 64, (ctx, ctx + 100), (new, new), 1024, False)
    old = torch.rand(d["c_pages"].shape[:2], device="cuda")
    close(call(d, old, 0.0), d, old, 0.0)


@pytest.mark.parametrize("way", ["kept", "computed"])
def test_pools_past_4_gb(way):
    d = case(way, 39, (200, 300), page=64)
    pages, far = d["c_pages"].shape[0], 80000
    c = torch.empty(far, 64, 512, dtype=torch.bfloat16, device="cuda")
    pe = torch.empty(far, 64, 64, dtype=torch.bfloat16, device="cuda")
    c[-pages:], pe[-pages:] = d["c_pages"], d["pe_pages"]
    old = torch.rand(pages, 64, device="cuda")
    w = torch.zeros(far, 64, device="cuda")
    w[-pages:] = old
    table = torch.where(d["block_table"] < 0, -1, d["block_table"] + far - pages)
    got = call(dict(d, c_pages=c, pe_pages=pe, block_table=table.to(torch.int32)), w, 1.0)
    assert torch.equal(got[-pages:], call(d, old, 1.0)) and not bool(got[:-pages].any())


def test_a_captured_call_takes_the_way_of_its_replay():
    """Which sequences' scores are kept is decided on the device, at each replay."""
    d = batch(40, [700, 900, 300], [6, 12, 2], 64)
    st, ws = torch.cuda.Stream(), mla.Workspace("cuda:0")
    old = torch.rand(d["c_pages"].shape[:2], device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        call(d, old, 1.0, workspace=ws)
        w = old.clone()
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            mla.mla_latent_key_weights(*(d[k] for k in ("q_nope", "q_pe", "c_pages", "pe_pages",
                                                        "block_table", "kv_len", "cu_q", "draft_mask",
                                                        "w_kvb")), SCALE, w, workspace=ws)
        for cu, lens in (([0, 6, 18, 20], [700, 900, 300]), ([0, 8, 16, 20], [400, 900, 256]),
                         ([0, 9, 18, 20], [513, 10, 2]), ([0, 0, 20, 20], [90, 300, 0]),
                         ([0, 20, 20, 20], [640, 5, 0])):
            d["cu_q"].copy_(torch.tensor(cu, dtype=torch.int32))
            d["kv_len"].copy_(torch.tensor(lens, dtype=torch.int32))
            w.copy_(old)
            g.replay()
            st.synchronize()
            close(w, d, old, 1.0)
        assert mla.mla_attn_get_status(ws, stream=st) == 0


# ---- the store of kept scores -----------------------------------------------------------

ROOM = 1 << 26      # floats
UNTOUCHED = 0x7fc12345  # no score has these bits


def batch(seed, lens, new, H, page=64):
    """Sequences of `lens` keys, `new` of them new tokens, on the device."""
    g = torch.Generator("cuda").manual_seed(seed)
    held = [-(-n // page) for n in lens]
    ids = torch.randperm(sum(held), generator=g, device="cuda").tolist()
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (max(held) - h))
        at += h
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    return dict(q_nope=mk(cu[-1], H, 128), q_pe=mk(cu[-1], H, 64), c_pages=mk(at, page, 512),
                pe_pages=mk(at, page, 64), block_table=i(table), kv_len=i(lens), cu_q=i(cu),
                draft_mask=None, w_kvb=(mk(H * 256, 512) / 512 ** 0.5).bfloat16())


def kept_floats(lens, new, H):
    """In order, whoever finds room for its scores has it."""
    left = ROOM
    for n, k in zip(new, lens):
        own = n * H * (-(-k // 128) * 128)
        if n * H <= 512 and own <= left:
            left -= own
    return ROOM - left


def store_used(d):
    """Floats at the beginning of the store that a call writes (none behind them), and its weights."""
    T, H = d["q_nope"].shape[:2]
    B, width = d["block_table"].shape
    page = d["c_pages"].shape[1]
    ws = mla.Workspace("cuda:0")
    size = mla.binding.library().mla_latent_key_weights_workspace_bytes(T, H, B, width * page)
    ws.buf = torch.zeros(size, dtype=torch.uint8, device="cuda")
    store = ws.buf[size - 4 * ROOM:].view(torch.int32)
    store.fill_(UNTOUCHED)
    w = call(d, torch.zeros(d["c_pages"].shape[:2], device="cuda"), 0.0, workspace=ws)
    assert mla.mla_attn_get_status(ws) == 0
    written = store != UNTOUCHED
    n = int(written.sum())
    assert bool(written[:n].all())
    return n, w


@pytest.mark.parametrize("lens,new", [
    ([131201, 1000, 300], [8, 8, 1]),         # one request whose scores are more than the store holds
    ([1000, 300, 131201], [8, 1, 8]),         # the same, behind the others
    ([100000, 40000, 20000, 900, 11100], [8] * 5),  # behind the first, the third fits and the fourth
    ([131072, 100], [8, 1]),                  # all of it for one
    ([5000, 131072, 700], [9, 7, 1]),         # rows that are not kept anyway take nothing
])
def test_requests_without_room_leave_it_to_those_behind(lens, new):
    d = batch(len(lens), lens, new, 64)
    n, w = store_used(d)
    assert n == kept_floats(lens, new, 64)
    sums = torch.stack([w.view(-1)[slots(d, b)].double().sum() for b in range(len(lens))])
    for s, k in zip(sums.tolist(), new):
        assert abs(s - 64 * k) <= 64 * k * 1e-4  # every row's weights sum to 1


def test_many_requests_fill_the_store():
    g = torch.Generator("cpu").manual_seed(3)
    lens = torch.randint(4, 3001, (700,), generator=g).tolist()
    new = torch.randint(0, 5, (700,), generator=g).tolist()
    lens[5], new[5], lens[300], new[300] = 131500, 4, 140000, 4
    d = batch(3, lens, new, 128)
    n, w = store_used(d)
    want = kept_floats(lens, new, 128)
    assert n == want > ROOM - 128 * 128
    for b in range(0, 700, 7):
        s = float(w.view(-1)[slots(d, b)].double().sum())
        assert abs(s - 128 * new[b]) <= 128 * new[b] * 1e-4
