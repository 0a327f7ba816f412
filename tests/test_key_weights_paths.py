"""The key weights' second pass takes one of three ways, by rows: scores kept and the rows' sums put
together where they are read (up to 512 rows in all), kept and read (up to 512 rows of a sequence), or
computed again.  What can go wrong in one of them is tested in each."""
import pytest
import torch

import mla_causal_attention_gb300 as mla
from paged_helpers import tree_case
from test_key_weights import call, reference

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
