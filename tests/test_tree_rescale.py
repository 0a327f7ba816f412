"""The tree attention's running maximum: scores that rise along the keys, so that mixes and sums are
scaled down again and again within a segment and from one segment to the next.

The rotary part carries the rises: it is neither folded nor rounded, so large scores stay exact and
the bounds of test_tree.py hold.  Heads take turns (h % 4):
  0  a step of 7 in the exponent (10.1 in log2 units; the kernel rescales from 8 on) every two tiles
  1  a single key 9.6 above the others at 0.55 of the cache: about as heavy as all of them
  2  no rise
  3  a step of 8 every five tiles
Tolerance: that of test_tree.py, and for scores of up to 300 / SCALE = 4200 in the accumulator a
few fp32 sums, off by at most 2^-11 each, before the scale: 8 * 2^-11 * SCALE < 0.1 * 2^-8 of the
weights."""
import math

import pytest
import torch

import mla_causal_attention_gb300 as mla
from mla_causal_attention_gb300.workloads import softmax_scale_192
from paged_helpers import tree_case, tree_reference

SCALE = softmax_scale_192()


def _rising_case(seed, B, H, n, ctx, page=64, dev="cuda"):
    d = tree_case(seed, B, H, ctx, (n, n), page, True, dev=dev)
    kv = d["kv_len"].tolist()
    for b, k in enumerate(kv):
        p = torch.arange(k, device=dev)
        slot = d["block_table"][b].long()[p // page] * page + p % page
        rises = torch.stack((p // 256, p == int(0.55 * k), torch.zeros_like(p), p // 640), -1)
        d["pe_pages"].view(-1, 64)[slot, :4] = rises.to(torch.bfloat16)
    d["q_pe"][..., :4] = 0
    for h in range(H):
        d["q_pe"][:, h, h % 4] = (97, 133, 0, 111)[h % 4]
    return d


def _online(d, b, drop=None):
    """(result, rescales) of sequence b in 64 bits by tiles of 128 keys with a running maximum that
    moves when a score is more than 8 log2 units above it, as one segment; drop: the scaling of the
    mix ("o") or of the sum ("l") is left out."""
    page, H = d["c_pages"].shape[1], d["q_nope"].shape[1]
    lo, hi, k = *d["cu_q"][b:b + 2].tolist(), int(d["kv_len"][b])
    p = torch.arange(k)
    slot = d["block_table"][b].long()[p // page] * page + p % page
    c, pe = (d[x].view(-1, w)[slot].double() for x, w in (("c_pages", 512), ("pe_pages", 64)))
    w = d["w_kvb"].double().view(H, 256, 512)
    x = torch.einsum("ihd,hjd->hij", d["q_nope"][lo:hi].double(),
                     torch.einsum("jl,hdl->hjd", c, w[:, :128]))
    x = (x + torch.einsum("ihd,jd->hij", d["q_pe"][lo:hi].double(), pe)) * (SCALE / math.log(2))
    new = p - (k - (hi - lo))
    seen = (new < 0) | ((d["draft_mask"][lo:hi, None] >> new.clamp(0, 63)) & 1).bool()
    x = x.masked_fill(~seen, float("-inf"))
    m = torch.full(x.shape[:2], float("-inf"), dtype=torch.float64)
    l, rescales = torch.zeros_like(m), torch.zeros_like(m)
    o = torch.zeros(*m.shape, 512, dtype=torch.float64)
    for j in range(0, k, 128):
        t = x[..., j:j + 128]
        top = t.amax(-1)
        need = (top > m + 8) | (m.isinf() & ~top.isinf())
        alpha = torch.where(need, (m - top).exp2(), 1.0)
        rescales += need & ~m.isinf()
        m = torch.where(need, top, m)
        e = (t - m[..., None]).exp2()
        l = (l if drop == "l" else l * alpha) + e.sum(-1)
        o = (o if drop == "o" else o * alpha[..., None]) + e @ c[j:j + 128]
    return torch.einsum("hil,hdl->ihd", o / l[..., None], w[:, 128:]), rescales


def _errors(got, d):
    """(relative error of the norm per kind of head, largest share of the elements' bounds)."""
    ref, spread, mixed = tree_reference(d, SCALE)
    err = (got.double() - ref).abs()
    share = float((err / (2 ** -8 * (7.1 * spread + mixed) + 1e-30)).max())
    return [float(err[:, k::4].norm() / ref[:, k::4].norm()) for k in range(4)], share


def test_the_cases_need_the_rescaling():
    """On the CPU: these scores move the maximum over and over, and a form that leaves either
    scaling out is far outside the tolerance."""
    d = _rising_case(1, 1, 8, 4, (1500, 1500), dev="cpu")
    right, rescales = _online(d, 0)
    rel, share = _errors(right, d)
    assert max(rel) < 1e-10 and share < 1e-6
    assert bool((rescales[0::4] >= 4).all()) and bool((rescales[3::4] >= 2).all())
    assert float((rescales[1::4] >= 1).double().mean()) > 0.5
    for drop in ("o", "l"):
        rel, share = _errors(_online(d, 0, drop)[0], d)
        assert min(rel[0], rel[1], rel[3]) > 0.1 and share > 10, drop


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,n,ctx,page", [
    (1, 64, 64, (10000, 10000), 64),    # 32 units of 79 tiles shared out in ranges of 35
    (20, 16, 4, (2000, 3900), 16),      # a unit of half the rows per sequence, 8 tiles to a pair
    (100, 32, 4, (1500, 2500), 128),    # whole units first, then ranges
    (3, 64, 5, (2000, 6000), 64),       # up to 16 tokens: merged in the up-projection
])
def test_rising_scores(B, H, n, ctx, page):
    d = _rising_case(B * 100 + n, B, H, n, ctx, page)
    out = mla.mla_latent_tree_fwd(d["q_nope"], d["q_pe"], d["c_pages"], d["pe_pages"],
                                  d["block_table"], d["kv_len"], d["cu_q"], d["draft_mask"],
                                  d["w_kvb"], SCALE)
    assert mla.mla_attn_get_status() == 0
    assert bool(torch.isfinite(out).all())
    rel, share = _errors(out, d)
    print(f"[tree] rel {rel} of the bound {share:.2f}")
    assert max(rel) <= 0.0045 and share <= 1
