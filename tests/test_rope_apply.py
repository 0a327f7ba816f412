"""The rotary step by itself (mla_rope_apply) against complex arithmetic in 64 bits: layouts, types,
slices, in place, and its inverse as the gradient."""
import random

import pytest
import torch

import mla_causal_attention_gb300 as mla
from mla_causal_attention_gb300 import binding

pytestmark = pytest.mark.gpu

S = binding.MlaStatus
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
LAYOUTS = ("half", "interleaved")


def _positions(T, rows, seed=0):
    r = random.Random(seed)
    return torch.tensor([r.randrange(rows) for _ in range(T)], dtype=torch.int32, device="cuda")


def _pairs(x, layout):
    h = x.shape[-1] // 2
    return (x[..., :h], x[..., h:]) if layout == "half" else (x[..., 0::2], x[..., 1::2])


def _join(u, v, layout):
    return torch.cat((u, v), -1) if layout == "half" else torch.stack((u, v), -1).flatten(-2)


def reference(x, positions, table, layout, out_layout, inverse):
    """(y, |u c| + |v s|) in 64 bits."""
    cs = table.double()[positions.long()]
    while cs.dim() < x.dim():
        cs = cs.unsqueeze(1)
    h = x.shape[-1] // 2
    c, s = cs[..., :h], cs[..., h:] * (-1 if inverse else 1)
    u, v = _pairs(x.double(), layout)
    size = _join((u * c).abs() + (v * s).abs(), (v * c).abs() + (u * s).abs(), out_layout)
    return _join(u * c - v * s, v * c + u * s, out_layout), size


def check(y, x, positions, table, layout, out_layout, inverse=False):
    want, size = reference(x, positions, table, layout, out_layout, inverse)
    # two products and a sum, one of the products rounded: 2^-24 of it and of the sum; then the
    # rounding to the type, half a step (of fp16's smallest numbers: 2^-25)
    fp32 = 2 * 2 ** -24 * size
    tol = fp32 + (torch.finfo(y.dtype).eps / 2) * (want.abs() + fp32)
    if y.dtype == torch.float16:
        tol = tol + 2 ** -25
    err = (y.double() - want).abs()
    assert bool((err <= tol + 1e-37).all()), float((err - tol).max())


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("out_layout", LAYOUTS)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("T,H,R", [
    (1, 1, 64),      # a single key
    (7, 64, 64),     # queries: every head of a token by one warp
    (5, 3, 64),      # fewer heads than a warp has rows
    (33, 5, 32), (3, 17, 96), (2, 9, 128), (4, 3, 256),
    (300, 1, 64),    # keys of many tokens
    (6, 2, 2), (5, 3, 6), (2, 2, 250),  # widths that fill no 16-byte piece
])
def test_matches_64_bits(T, H, R, layout, out_layout, kind):
    g = torch.Generator("cuda").manual_seed(T + H + R)
    x = torch.randn(T, H, R, device="cuda", generator=g).to(TYPES[kind])
    table = mla.mla_rope_table(1000, dim=R)
    pos = _positions(T, 1000)
    for inverse in (False, True):
        y = mla.mla_rope_apply(x, pos, table, layout, out_layout, inverse)
        torch.cuda.synchronize()
        check(y, x, pos, table, layout, out_layout, inverse)
    assert mla.mla_attn_get_status() == 0


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("offset,step,row", [
    (128, 192, 0),   # the last 64 of a head's 192 columns
    (0, 64, 64),     # rows with room behind them
    (3, 71, 5),      # odd steps and an odd start: no 16-byte pieces
    (4, 72, 4),      # whole pieces for fp32 alone
])
def test_slices_and_in_place(offset, step, row, kind):
    T, H, R = 19, 12, 64
    wide = torch.randn(T, H * step + row + offset, device="cuda").to(TYPES[kind])
    x = wide[:, offset:offset + H * step].unflatten(-1, (H, step))[..., :R]
    table, pos = mla.mla_rope_table(5000, dim=R), _positions(T, 5000)
    before = wide.clone()
    bx = before[:, offset:offset + H * step].unflatten(-1, (H, step))[..., :R]
    y = mla.mla_rope_apply(x, pos, table, "interleaved", "half")
    check(y, bx, pos, table, "interleaved", "half")
    assert torch.equal(wide, before)
    for layout, to in (("interleaved", "half"), ("half", "interleaved"), ("half", "half")):
        wide.copy_(before)
        assert mla.mla_rope_apply(x, pos, table, layout, to, out=x) is x
        check(x, bx, pos, table, layout, to)
        x.copy_(bx)  # nothing beside the rows has changed
        assert torch.equal(wide, before)


def test_other_columns_of_the_same_rows():
    T, H, R = 11, 4, 64
    wide = torch.randn(T, H, 192, device="cuda").bfloat16()
    table, pos = mla.mla_rope_table(100), _positions(T, 100)
    x, to = wide[..., 128:], wide[..., 64:128]
    want = mla.mla_rope_apply(x, pos, table, "interleaved", "half")
    first = wide[..., :64].clone()
    mla.mla_rope_apply(x, pos, table, "interleaved", "half", out=to)
    assert torch.equal(to, want) and torch.equal(wide[..., :64], first)


def test_heads_before_rows_and_broadcast_rows():
    """[H, T, R] storage, and one row for all heads."""
    T, H, R = 40, 6, 64
    x = torch.randn(H, T, R, device="cuda").bfloat16().transpose(0, 1)
    table, pos = mla.mla_rope_table(300), _positions(T, 300)
    out = torch.zeros(H, T, R, device="cuda", dtype=torch.bfloat16).transpose(0, 1)
    mla.mla_rope_apply(x, pos, table, out=out)
    check(out, x, pos, table, "half", "half")
    one = torch.randn(T, 1, R, device="cuda").bfloat16().expand(T, H, R)
    check(mla.mla_rope_apply(one, pos, table), one, pos, table, "half", "half")


def test_two_dimensional_keys_match_the_append():
    """Half-layout keys come out as mla_latent_append writes them, bit for bit."""
    T, page = 50, 16
    k = torch.randn(T, 64, device="cuda").bfloat16()
    table, pos = mla.mla_rope_table(2000), _positions(T, 2000)
    slots = torch.arange(T, device="cuda", dtype=torch.int32)
    c = torch.zeros(4, page, 512, device="cuda", dtype=torch.bfloat16)
    pe = torch.zeros(4, page, 64, device="cuda", dtype=torch.bfloat16)
    mla.mla_latent_append(torch.zeros(T, 512, device="cuda", dtype=torch.bfloat16), k, slots, c, pe,
                          positions=pos, rope_table=table)
    assert torch.equal(mla.mla_rope_apply(k, pos, table), pe.view(-1, 64)[:T])
    paired = torch.stack((k[:, :32], k[:, 32:]), -1).flatten(-2)
    assert torch.equal(mla.mla_rope_apply(paired, pos, table, "interleaved", "half"),
                       pe.view(-1, 64)[:T])


@pytest.mark.parametrize("layout,out_layout", [(a, b) for a in LAYOUTS for b in LAYOUTS])
def test_inverse_is_the_gradient(layout, out_layout):
    """Against autograd through the formula in 64 bits, and against differences."""
    T, H, R = 4, 3, 32
    table = mla.mla_rope_table(500, mla.RopeConfig(mscale=2.0, mscale_all_dim=1.0), dim=R)
    pos = _positions(T, 500)
    x = torch.randn(T, H, R, device="cuda")
    dy = torch.randn(T, H, R, device="cuda")
    leaf = x.double().requires_grad_()
    reference(leaf, pos, table, layout, out_layout, False)[0].backward(dy.double())
    dx = mla.mla_rope_apply(dy, pos, table, out_layout, layout, inverse=True)
    size = reference(dy, pos, table, out_layout, layout, True)[1]
    assert bool(((dx.double() - leaf.grad).abs() <= 3 * 2 ** -24 * size).all())
    # the step is linear: <dy, f(x + e) - f(x - e)> / 2 = <dx, e> but for fp32's rounding
    e = torch.randn(T, H, R, device="cuda")
    up, down = (mla.mla_rope_apply(x + s * e, pos, table, layout, out_layout) for s in (1, -1))
    diff = float((dy.double() * (up.double() - down.double())).sum() / 2)
    got = float((dx.double() * e.double()).sum())
    # inputs and results of three roundings each, 2^-24 of |x| + |e| times the rotation's ratio
    most = float((dy.double().abs() * 2 * (x.abs() + e.abs()).double()).sum()) * 2.0
    assert abs(diff - got) <= 6 * 2 ** -24 * most


def test_inverse_undoes_the_step():
    x = torch.randn(64, 8, 64, device="cuda")
    table, pos = mla.mla_rope_table(131072), _positions(64, 131072)
    y = mla.mla_rope_apply(x, pos, table, "interleaved", "half")
    back = mla.mla_rope_apply(y, pos, table, "half", "interleaved", inverse=True)
    # c^2 + s^2 = 1 to 2 * 2^-24; every step adds three roundings of at most |u| + |v|
    assert float((back - x).abs().max()) <= 10 * 2 ** -24 * 2 * float(x.abs().max())


@pytest.mark.parametrize("dim", [2, 32, 96, 256])
def test_table_of_another_width(dim):
    f, ratio = mla.mla_rope_frequencies(dim=dim)
    assert len(f) == dim // 2
    table = mla.mla_rope_table(70000, dim=dim)
    p = torch.tensor([0, 1, 4095, 69999], device="cuda")
    a = p.double()[:, None] * torch.tensor(f, dtype=torch.float64, device="cuda")
    want = torch.cat((a.cos(), a.sin()), 1) * ratio
    # angles of up to 70000 in 64 bits: 2^-52 of them; then one rounding to fp32
    assert float((table[p].double() - want).abs().max()) <= 2 ** -24 + 70000 * 2 ** -51
    plain = mla.RopeConfig(rope_theta=10000.0, factor=1.0)
    f, ratio = mla.mla_rope_frequencies(plain, dim=dim)
    assert ratio == 1.0
    for d, x in enumerate(f):
        assert abs(x - 10000.0 ** (-2 * d / dim)) <= 1e-15


def test_positions_outside_the_table_are_reported():
    x = torch.randn(3, 2, 64, device="cuda")
    table = mla.mla_rope_table(10)
    ws = mla.Workspace("cuda:0")
    pos = torch.tensor([-1, 4, 10], dtype=torch.int32, device="cuda")
    y = mla.mla_rope_apply(x, pos, table, workspace=ws)
    check(y, x, pos.clamp(0, 9), table, "half", "half")
    assert mla.mla_attn_get_status(ws) == S.ERR_KVLEN
    assert mla.mla_attn_get_status(ws) == 0


def test_captured_step_follows_its_inputs():
    x = torch.randn(9, 4, 64, device="cuda").bfloat16()
    table, pos = mla.mla_rope_table(100), _positions(9, 100)
    y = mla.mla_rope_apply(x, pos, table)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mla.mla_rope_apply(x, pos, table, out=y)
    x.copy_(torch.randn(9, 4, 64)); pos.copy_(_positions(9, 100, 1))
    g.replay()
    torch.cuda.synchronize()
    check(y, x, pos, table, "half", "half")
