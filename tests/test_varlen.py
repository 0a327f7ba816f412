"""Causal attention over packed prompts (mla_attn_varlen_fwd) against its definition in 64 bits.

Tolerances.  The softmax weights and the output are rounded to bf16, by at most half a step each,
2^-8 of the value: per element 2^-8 of spread = sum_j p_j |v_j| for the weights, 2^-8 of |out| <=
spread for the output, 2 * 2^-8 spread in all (and 2^-16 of it for fp32 sums over at most a few
thousand keys).  In the 2-norm the two are independent and at most 2^-8 / sqrt(3) each: 0.0032."""
import ctypes
import random

import pytest
import torch

import mla_causal_attention_gb300 as mla
from mla_causal_attention_gb300 import binding
from mla_causal_attention_gb300.build import build_test_variant
from mla_causal_attention_gb300.workloads import softmax_scale_192

pytestmark = pytest.mark.gpu

S = binding.MlaStatus
SCALE = softmax_scale_192()


def _case(seed, ns, H, Hkv, fused, pad=0):
    """Rows behind the last sequence are NaN."""
    g = torch.Generator("cpu").manual_seed(seed)
    T = sum(ns) + pad
    mk = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    q, kv, k_pe = mk(T, H, 192), mk(T, Hkv, 256), mk(T, 64)
    for x in (q, kv, k_pe):
        x[sum(ns):] = float("nan")
    d = dict(q_nope=q[..., :128], q_pe=q[..., 128:], k_nope=kv[..., :128], v=kv[..., 128:], k_pe=k_pe)
    if not fused:
        d = {k: x.contiguous() for k, x in d.items()}
    cu = [0]
    for n in ns:
        cu.append(cu[-1] + n)
    d["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    return d


def _run(d, **kw):
    out = mla.mla_attn_varlen_fwd(d["q_nope"], d["q_pe"], d["k_nope"], d["k_pe"], d["v"],
                                  d["cu_seqlens"], SCALE, **kw)
    torch.cuda.synchronize()
    return out


def _reference(d, seqs=None):
    """{sequence: (out, spread)}, head by head."""
    cu = d["cu_seqlens"].tolist()
    group = d["q_nope"].shape[1] // d["k_nope"].shape[1]
    res = {}
    for b in range(len(cu) - 1) if seqs is None else seqs:
        lo, hi = cu[b], cu[b + 1]
        q = torch.cat((d["q_nope"][lo:hi], d["q_pe"][lo:hi]), -1).double().transpose(0, 1)
        k = d["k_nope"][lo:hi].double().transpose(0, 1).repeat_interleave(group, 0)
        pe = d["k_pe"][lo:hi].double().expand(k.shape[0], -1, -1)
        v = d["v"][lo:hi].double().transpose(0, 1).repeat_interleave(group, 0)
        x = q @ torch.cat((k, pe), -1).transpose(1, 2) * SCALE
        x = x.masked_fill(torch.ones(hi - lo, hi - lo, dtype=torch.bool, device="cuda").triu(1),
                          float("-inf"))
        e = (x - x.amax(-1, keepdim=True)).exp() if hi > lo else x
        p = e / e.sum(-1, keepdim=True)
        res[b] = ((p @ v).transpose(0, 1), (p @ v.abs()).transpose(0, 1))
    return res


def _close(got, d, seqs=None):
    cu = d["cu_seqlens"].tolist()
    for b, (ref, spread) in _reference(d, seqs).items():
        if ref.numel() == 0:
            continue
        x = got[cu[b]:cu[b + 1]].double()
        err = (x - ref).abs()
        assert bool(torch.isfinite(x).all()), f"sequence {b}"
        rel = float(err.norm() / ref.norm())
        assert rel <= 0.0032, f"sequence {b} of length {len(ref)}: {rel}"
        assert not bool((err > spread * (2 * 2 ** -8 + 2 ** -16)).any()), f"sequence {b}"


@pytest.mark.parametrize("ns,H,Hkv,fused", [
    ([1], 64, 64, True),
    ([1, 1, 1], 2, 1, False),
    ([127, 128, 129], 4, 4, True),           # ends inside, on and behind a tile
    ([255, 256, 257, 1], 3, 1, False),       # the same for tile pairs; three heads on one
    ([0, 5, 0, 0, 300, 0], 8, 2, True),      # empty sequences
    ([17, 200, 3, 64, 90, 1, 150], 64, 64, True),
    ([700, 33, 1500], 16, 4, False),
    ([2100], 6, 2, True),
    ([64] * 40, 8, 8, False),
    ([1] * 300, 4, 2, True),                 # more sequences than CTAs
    ([0, 0], 4, 4, False),                   # nothing to do
    ([2, 0, 1] * 500, 2, 1, True),           # more sequences than threads that list their tiles
    ([3] * 40 + [1500] + [5, 0] * 600 + [1100, 700], 2, 2, False),  # long ones among them
])
def test_varlen_matches_definition(ns, H, Hkv, fused):
    d = _case(len(ns) * 100 + H, ns, H, Hkv, fused, pad=5)
    T = sum(ns) + 5
    out = torch.full((T, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    assert _run(d, out=out) is out
    assert mla.mla_attn_get_status() == 0
    _close(out, d)
    assert bool((out[sum(ns):] == 7.0).all())  # rows behind the last sequence


def test_varlen_random_sweep():
    r = random.Random(3)
    for k in range(12):
        Hkv, group = r.choice((1, 2, 5, 8)), r.choice((1, 2, 3, 8))
        ns = [r.choice((r.randint(0, 20), r.randint(0, 700))) for _ in range(r.randint(1, 20))]
        if sum(ns) == 0:
            ns[0] = 1
        d = _case(50 + k, ns, Hkv * group, Hkv, r.random() < 0.5)
        print(ns, Hkv, group)
        _close(_run(d), d)
    assert mla.mla_attn_get_status() == 0


def test_another_sequences_rows_never_reach_a_result():
    """Every second sequence NaN or infinite: the others come out as if it were not there."""
    ns = [130, 77, 300, 1, 250, 128, 5]
    d = _case(9, ns, 8, 4, False)
    want = _run(d).clone()
    cu = d["cu_seqlens"].tolist()
    for b in range(1, len(ns), 2):
        for k, bad in (("v", float("inf")), ("k_nope", float("nan")), ("q_nope", float("nan")),
                       ("k_pe", float("-inf"))):
            d[k][cu[b]:cu[b + 1]] = bad
    got = _run(d)
    for b in range(0, len(ns), 2):
        assert torch.equal(got[cu[b]:cu[b + 1]], want[cu[b]:cu[b + 1]]), b


def test_large_scores():
    d = _case(4, [300, 40], 4, 4, False)
    d["q_nope"] *= 30
    _close(_run(d), d)


def test_varlen_of_one_sequence_is_the_prefill():
    """One sequence with a key/value head per head: bit for bit mla_attn_fwd's result."""
    n, H = 777, 16
    d = _case(5, [n], H, H, False)
    got = _run(d)
    per_head = lambda x: x.transpose(0, 1).contiguous()[None]  # noqa: E731
    want = mla.mla_attn_fwd(per_head(d["q_nope"]), per_head(d["q_pe"]), per_head(d["k_nope"]),
                            d["k_pe"][None], per_head(d["v"]), None, 0, SCALE)
    assert torch.equal(got, want[0].transpose(0, 1))


def test_varlen_on_a_side_stream_and_under_a_graph():
    d = _case(6, [100, 300, 5], 8, 4, True, pad=300)
    e = _case(7, [1, 600, 50], 8, 4, True, pad=54)
    want = {k: _run(x).clone() for k, x in (("d", d), ("e", e))}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = _run(d, stream=s, workspace=mla.Workspace())
    assert torch.equal(side[:405], want["d"][:405])
    st = {k: v.clone() for k, v in d.items()}
    out, ws = torch.zeros_like(want["d"]), mla.Workspace()
    _run(st, out=out, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.mla_attn_varlen_fwd(st["q_nope"], st["q_pe"], st["k_nope"], st["k_pe"], st["v"],
                                st["cu_seqlens"], SCALE, out=out, workspace=ws)
    for name, c in (("e", e), ("d", d)):
        for k, v in c.items():
            st[k].copy_(v)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        n = int(c["cu_seqlens"][-1])
        assert torch.equal(out[:n], want[name][:n]) and bool((out[n:] == 0).all())


def test_varlen_reports_bad_offsets():
    mla.mla_attn_get_status()
    d = _case(8, [50, 60, 70], 4, 4, False)
    good = _run(d)
    for cu in ([0, 50, 110, 500], [0, 50, 40, 180], [-3, 50, 110, 180], [0, 180, 0, 180]):
        e = dict(d, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        out = _run(e)
        assert mla.mla_attn_get_status() == S.ERR_KVLEN
        if cu[:2] == [0, 50]:
            assert torch.equal(out[:40], good[:40])


def test_varlen_long_sequence_sampled():
    """5000 rows of one sequence between two others, heads in groups: three whole sequences'
    rows against the definition."""
    d = _case(10, [1000, 5000, 129], 8, 2, True)
    _close(_run(d), d)


def test_many_calls_in_flight():
    """Short prompts, one key tile per unit: the value tiles of successive units are on their way
    at the same time.  A few hundred calls without waiting in between, warm in L2."""
    d, e = (_case(s, [17, 200, 3, 64, 90, 1, 150, 33], 64, 64, True) for s in (20, 21))
    want = {k: _run(x).clone() for k, x in (("d", d), ("e", e))}
    outs = [torch.empty_like(want["d"]) for _ in range(4)]
    for k in range(300):
        c = d if k % 2 == 0 else e
        mla.mla_attn_varlen_fwd(c["q_nope"], c["q_pe"], c["k_nope"], c["k_pe"], c["v"],
                                c["cu_seqlens"], SCALE, out=outs[k % 4])
    torch.cuda.synchronize()
    for k in range(4):
        assert torch.equal(outs[k], want["d" if k % 2 == 0 else "e"])
    assert mla.mla_attn_get_status() == 0


def test_results_are_the_same_every_time():
    """Whatever the workspace held before, and in whatever order units of equal length run."""
    r = random.Random(5)
    for k in range(4):
        ns = [r.choice((1, 60, 128, 200, 300, 900)) for _ in range(24)]
        d = _case(70 + k, ns, 16, 4, True)
        ws = mla.Workspace()
        want = _run(d, workspace=ws).clone()
        for i in range(40):
            if i % 3 == 0:
                ws.buf[256:].random_(0, 255)
            assert torch.equal(_run(d, workspace=ws), want), (k, i)


def test_offsets_that_fall_over_and_over():
    """Sequences that overlap, with more pairs of query tiles together than rising offsets can have:
    the first ones count, as many as the list has room for."""
    mla.mla_attn_get_status()
    d = _case(11, [600], 4, 2, False)
    want = _run(d)
    e = dict(d, cu_seqlens=torch.tensor([0, 600] * 50, dtype=torch.int32, device="cuda"))
    ws = mla.Workspace()
    assert torch.equal(_run(e, workspace=ws), want)  # 50 sequences of the same rows
    assert mla.mla_attn_get_status(ws) == S.ERR_KVLEN
    # room for 600 // 256 + 99 = 101 pairs, three to a sequence
    assert int(ws.buf[256:260].view(torch.int32)) == 33 * 3
    assert torch.equal(_run(d, workspace=ws), want) and mla.mla_attn_get_status(ws) == 0


def test_more_pairs_than_32_bits_count():
    """2^23 sequences of 2^16 rows, the same ones: 2^31 pairs of query tiles if all were counted."""
    mla.mla_attn_get_status()
    T, B = 1 << 16, 1 << 24
    x = torch.zeros((T, 1, 128), dtype=torch.bfloat16, device="cuda")
    pe = torch.zeros((T, 1, 64), dtype=torch.bfloat16, device="cuda")
    v = torch.randn((1, 128), device="cuda").to(torch.bfloat16).repeat(T, 1)[:, None].contiguous()
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = T
    ws = mla.Workspace()
    out = mla.mla_attn_varlen_fwd(x, pe, x, pe[:, 0], v, cu, SCALE, workspace=ws)
    assert mla.mla_attn_get_status(ws) == S.ERR_KVLEN
    most = T // 256 + T
    assert int(ws.buf[256:260].view(torch.int32)) == most // 256 * 256
    # Every value row is the same and every weight 1, so each row's mean is that row: half a step of
    # bf16, 2^-8, and in fp32 at most 2^16 / 16 sums of a tensor instruction, off by 2^-23 each.
    assert bool(((out.float() - v.float()).abs() <= v.float().abs() * 2 ** -7).all())


def test_some_of_a_batchs_prompts():
    d = _case(12, [40, 300, 129, 5], 8, 4, True)
    want = _run(d)
    out = torch.full_like(want, 7.0)
    _run(dict(d, cu_seqlens=d["cu_seqlens"][2:4].contiguous()), out=out)
    assert mla.mla_attn_get_status() == 0
    assert torch.equal(out[340:469], want[340:469])
    assert bool((out[:340] == 7.0).all()) and bool((out[469:] == 7.0).all())


@pytest.mark.parametrize("packed", [True, False])
def test_waits_that_last_for_a_whole_unit(packed):
    """A prompt of 2049 key tiles whose last query tile pair has rows in one tile only, by a test
    build whose waits give up after 1 ms: the warps that wait for the whole unit, about 3 ms, do not
    take its length for a hang.  (The library gives up after a second, a unit of 2^26 keys.)"""
    lib = ctypes.CDLL(build_test_variant("wait_long", "prefill.cu", ["-DMLA_WAIT_LIMIT_NS=1000000ull"]))
    p, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.mla_attn_varlen_fwd.argtypes = [p, p, p, p, p, p, p, i, i, i, i, f, p, p, sz, p]
    lib.mla_attn_fwd.argtypes = [p, p, p, p, p, p, i, i, i, i, i, f, p, p, sz, p]
    lib.mla_attn_get_status.argtypes = [p, p]
    T = (1 << 18) + 100
    d = _case(13, [T], 1, 1, False)
    out = torch.zeros((T, 1, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(1 << 23, dtype=torch.uint8, device="cuda")
    at = [d[k].data_ptr() for k in ("q_nope", "q_pe", "k_nope", "k_pe", "v")]
    tail = [SCALE, out.data_ptr(), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream]
    torch.cuda.synchronize()
    if packed:
        rc = lib.mla_attn_varlen_fwd(*at, None, d["cu_seqlens"].data_ptr(), 1, T, 1, 1, *tail)
    else:
        rc = lib.mla_attn_fwd(*at, None, 1, 1, T, T, 0, *tail)
    assert rc == 0
    assert lib.mla_attn_get_status(ws.data_ptr(), tail[-1]) == 0
    torch.cuda.synchronize()
    assert torch.equal(out, _run(d))
