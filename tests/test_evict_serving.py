"""Requests that outgrow their budget, as a server runs them: queries and keys of a checkpoint with
paired rotary columns are rotated, planned, appended and attended to; the last tokens' attention is
accumulated per key; what is over the budget goes, the rest moves together, the pages come back; and
decoding goes on over what is left.  Beside the cache the test keeps plain lists of the rows that it
should hold, and compares every step with its definition over those."""
import random

import pytest
import torch

import mla_causal_attention_gb300 as mla
from mla_causal_attention_gb300.workloads import softmax_scale_192
from paged_helpers import pages
from test_evict import keep_reference

pytestmark = pytest.mark.gpu

SCALE = softmax_scale_192()
PAGE, WIDTH, POOL, B = 16, 24, 60, 3


def _i(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class _Server:
    def __init__(self, H, seed, layers=2):
        self.g = torch.Generator("cpu").manual_seed(seed)
        self.r = random.Random(seed)
        self.H, self.layers = H, layers
        self.free = list(range(POOL))
        self.r.shuffle(self.free)
        nan = lambda n: torch.full((POOL, PAGE, n), float("nan"), device="cuda")  # noqa: E731
        self.c = [nan(512).bfloat16() for _ in range(layers)]
        self.pe = [nan(64).bfloat16() for _ in range(layers)]
        self.weight = [nan(1)[..., 0].contiguous() for _ in range(layers)]
        self.w_kvb = [self.normal(H * 256, 512).div(512 ** 0.5) for _ in range(layers)]
        self.table = _i([[-1] * WIDTH] * B)
        self.rope = mla.mla_rope_table(4000)
        self.ctx = [0] * B      # rows of the cache
        self.dropped = [0] * B  # tokens that are no longer in it
        # what each layer's cache should hold: per sequence its rows' (latent, rotated key), weights
        self.rows = [[(torch.zeros(0, 512).cuda(), torch.zeros(0, 64).cuda())] * B for _ in range(layers)]

    def normal(self, *s):
        return torch.randn(*s, generator=self.g).to(torch.bfloat16).cuda()

    def step(self, new, decay):
        T = sum(new)
        p = mla.mla_paged_plan(_i(self.ctx), _i(new), self.table, _i(self.free), _i([0]), PAGE, POOL, T)
        used = int(p.free_next)
        self.free = self.free[used:]
        # positions go on behind the tokens that were dropped
        pos = p.positions + torch.repeat_interleave(_i(self.dropped), _i(new).long())
        kv = [x + n for x, n in zip(self.ctx, new)]
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        for L in range(self.layers):
            q = self.normal(T, self.H, 192)
            c_new, k_raw = self.normal(T, 512), self.normal(T, 64)
            q_pe = mla.mla_rope_apply(q[..., 128:], pos, self.rope, "interleaved", "half")
            k_pe = mla.mla_rope_apply(k_raw, pos, self.rope, "interleaved", "half")
            mla.mla_latent_append(c_new, k_pe, p.slots, self.c[L], self.pe[L])
            q_nope = q[..., :128].contiguous()
            args = (q_nope, q_pe, self.c[L], self.pe[L], self.table, p.kv_len, p.cu_q, None,
                    self.w_kvb[L], SCALE)
            out = mla.mla_latent_tree_fwd(*args)
            held = [self.held_weights(L, b, self.ctx[b]) for b in range(B)]
            mla.mla_latent_key_weights(*args, self.weight[L], decay=decay)
            torch.cuda.synchronize()
            # rotated pairs, in 64 bits
            turn = torch.view_as_complex(q[..., 128:].double().unflatten(-1, (32, 2)).contiguous())
            cs = self.rope.double()[pos.long()]
            turn = turn * torch.complex(cs[:, :32], cs[:, 32:])[:, None]
            want = torch.cat((turn.real, turn.imag), -1)
            assert bool(((q_pe.double() - want).abs() <= want.abs() * 2 ** -8 + 1e-5).all())
            for b in range(B):
                lo, hi = cu[b], cu[b + 1]
                c_old, pe_old = self.rows[L][b]
                c = torch.cat((c_old, c_new[lo:hi].float()))
                pe = torch.cat((pe_old, k_pe[lo:hi].float()))
                self.rows[L][b] = (c, pe)
                if lo == hi:
                    continue
                w = self.w_kvb[L].double().view(self.H, 256, 512)
                keys = torch.einsum("jl,hdl->hjd", c.double(), w[:, :128])
                vals = torch.einsum("jl,hdl->hjd", c.double(), w[:, 128:])
                x = torch.einsum("ihd,hjd->hij", q_nope[lo:hi].double(), keys)
                x = (x + torch.einsum("ihd,jd->hij", q_pe[lo:hi].double(), pe.double())) * SCALE
                j = torch.arange(kv[b], device="cuda")
                hidden = j[None] > self.ctx[b] + torch.arange(hi - lo, device="cuda")[:, None]
                prob = x.masked_fill(hidden, float("-inf")).softmax(-1)
                ref = torch.einsum("hij,hjd->ihd", prob, vals)
                err = (out[lo:hi].double() - ref).norm() / ref.norm()
                assert float(err) <= 0.0045  # four roundings to bf16
                # the weights go on from those of the rows that were kept
                total = prob.sum((0, 1))
                total[:self.ctx[b]] += decay * held[b].double() if decay else 0.0
                got = self.held_weights(L, b, kv[b]).double()
                # scores are exact to about 2^-16: 3e-4 for the largest, both here and in the sum
                assert float(((got - total).abs() / total).max()) <= 6e-4
        self.ctx = kv

    def slots(self, b, n):
        j = torch.arange(n, device="cuda")
        return self.table[b].long()[j // PAGE] * PAGE + j % PAGE

    def held_weights(self, L, b, n):
        return self.weight[L].view(-1)[self.slots(b, n)].clone()

    def cut(self, budget, sinks, recent):
        free_pages = None
        for L in range(self.layers):  # each layer keeps its own rows, and as many as the others
            w = [self.held_weights(L, b, self.ctx[b]).cpu() for b in range(B)]
            e = mla.mla_paged_evict(self.weight[L], self.table, _i(self.ctx), _i([budget] * B), sinks,
                                    recent, max_keep=budget)
            mla.mla_latent_compact(self.c[L], self.pe[L], self.table, e.kept, e.kept_len,
                                   weights=self.weight[L])
            torch.cuda.synchronize()
            for b in range(B):
                keep = keep_reference(w[b].tolist(), self.ctx[b], budget, sinks, recent)
                n = len(keep)
                assert e.kept[b, :n].tolist() == keep and int(e.kept_len[b]) == n
                at = torch.tensor(keep, dtype=torch.int64, device="cuda")
                c, pe = self.rows[L][b]
                self.rows[L][b] = (c[at], pe[at])
                assert torch.equal(self.held_weights(L, b, n).cpu(), w[b][at.cpu()])
                s = self.slots(b, n)
                assert torch.equal(self.c[L].view(-1, 512)[s].float(), c[at])
                assert torch.equal(self.pe[L].view(-1, 64)[s].float(), pe[at])
            free_pages = e.freed[:int(e.n_freed)].tolist()
        kept = [min(n, budget) for n in self.ctx]
        assert len(free_pages) == sum(pages(n, PAGE) - pages(k, PAGE) for n, k in zip(self.ctx, kept))
        self.free += free_pages
        self.dropped = [d + n - k for d, n, k in zip(self.dropped, self.ctx, kept)]
        self.ctx = kept
        held = sum(pages(n, PAGE) for n in self.ctx)
        assert sorted(self.free) == sorted(set(self.free)) and len(self.free) + held == POOL
        assert mla.mla_attn_get_status() == 0


@pytest.mark.parametrize("H,seed", [(16, 0), (64, 1)])
def test_requests_outgrow_their_budget(H, seed):
    s = _Server(H, seed)
    s.step([150, 20, 97], decay=0.0)      # prompts; fresh weights
    s.cut(budget=64, sinks=2, recent=10)
    for _ in range(3):
        for _ in range(4):
            s.step([1, 1, 1], decay=1.0)  # decoding
        s.step([5, 0, 17], decay=0.5)     # a continued prompt, a request that waits
        s.cut(budget=64, sinks=2, recent=10)
    s.cut(budget=20, sinks=0, recent=0)   # several times in a row
    s.cut(budget=20, sinks=0, recent=0)
    s.step([1, 3, 1], decay=1.0)
    assert sum(s.dropped) > 200
