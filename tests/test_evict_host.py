"""What the rotary step, the eviction and the key weights refuse, before any launch (no GPU)."""
import ctypes

import pytest
import torch

import mla_causal_attention_gb300 as mla
from mla_causal_attention_gb300 import binding
from mla_causal_attention_gb300.build import build_library

S = binding.MlaStatus


@pytest.fixture(scope="module")
def lib():
    build_library()
    return binding.library()


@pytest.fixture(scope="module")
def base():
    buf = ctypes.create_string_buffer(1 << 16)
    base.keep = buf
    return (ctypes.addressof(buf) + 255) & ~255


def _accepted(status):
    """Past every check of the arguments: what is left to refuse is the missing device."""
    return torch.cuda.is_available() or status in (S.ERR_CUDA, S.ERR_DEVICE)


ROPE = ["x", "x_row", "x_head", "y", "y_row", "y_head", "type", "T", "H", "R", "positions", "table",
        "rows", "layout", "out_layout", "inverse", "workspace", "workspace_bytes", "stream"]


def _rope_args(base):
    a = dict(x=base, x_row=128, x_head=64, y=base + 8192, y_row=128, y_head=64, type=0, T=4, H=2,
             R=64, positions=base + 16384, table=base + 20480, rows=9, layout=1, out_layout=0,
             inverse=0, workspace=base + 32768, workspace_bytes=256, stream=None)
    return a


@pytest.mark.parametrize("change,want", [
    ({"x": None}, S.ERR_NULL), ({"y": None}, S.ERR_NULL), ({"positions": None}, S.ERR_NULL),
    ({"table": None}, S.ERR_NULL), ({"workspace": None}, S.ERR_WORKSPACE),
    ({"workspace_bytes": 255}, S.ERR_WORKSPACE),
    ({"T": 0}, S.ERR_SHAPE), ({"H": 0}, S.ERR_SHAPE), ({"R": 0}, S.ERR_SHAPE),
    ({"R": 63}, S.ERR_SHAPE), ({"R": 258}, S.ERR_SHAPE), ({"rows": 0}, S.ERR_SHAPE),
    ({"x_row": -1}, S.ERR_SHAPE), ({"y_head": -64}, S.ERR_SHAPE),
    ({"x_row": 1 << 41}, S.ERR_SHAPE), ({"T": 1 << 30, "H": 1 << 20}, S.ERR_SHAPE),
    ({"y_row": 0}, S.ERR_SHAPE), ({"y_head": 32}, S.ERR_SHAPE),      # rows of y that overlap
    ({"y_row": 64, "y_head": 64}, S.ERR_SHAPE), ({"y_row": 100}, S.ERR_SHAPE),
    ({"type": 3}, S.ERR_ARG), ({"type": -1}, S.ERR_ARG), ({"layout": 2}, S.ERR_ARG),
    ({"out_layout": -1}, S.ERR_ARG), ({"inverse": 2}, S.ERR_ARG),
])
def test_rope_refuses(lib, base, change, want):
    a = _rope_args(base)
    a.update(change)
    assert lib.mla_rope_apply(*[a[n] for n in ROPE]) == want


def test_rope_refuses_alignment_and_overlap(lib, base):
    for name, off in [("x", 1), ("y", 1), ("positions", 2), ("table", 8), ("workspace", 8)]:
        a = _rope_args(base)
        a[name] += off
        assert lib.mla_rope_apply(*[a[n] for n in ROPE]) == S.ERR_ALIGN, name
    for change in ({"y": base + 2}, {"y": base + 128}, {"y": base + 256, "y_row": 256},
                   {"y": base, "x_row": 256}, {"y": base + 16384 - 64}, {"y": base + 20480}):
        a = _rope_args(base)
        a.update(change)
        assert lib.mla_rope_apply(*[a[n] for n in ROPE]) == S.ERR_ARG, change
    if torch.cuda.is_available():
        return
    wide = {"x_row": 384, "x_head": 192, "y_row": 384, "y_head": 192}
    for change in ({}, {"y": base}, {"x": base + 2, "y": base + 8194},  # element-aligned
                   {**wide, "y": base + 128}, {**wide, "y": base + 256},  # other columns
                   {"x_row": 0, "x_head": 0}, {"y_row": 64, "y_head": 256}):
        a = _rope_args(base)
        a.update(change)
        assert _accepted(lib.mla_rope_apply(*[a[n] for n in ROPE])), change


EVICT = ["weights", "num_pages", "page_size", "block_table", "max_pages", "kv_len", "budget", "B",
         "sinks", "recent", "kept", "K", "kept_len", "freed", "n_freed", "workspace",
         "workspace_bytes", "stream"]


def _evict_args(base):
    a = {n: base + 1024 * i for i, n in enumerate(EVICT)}
    a.update(num_pages=8, page_size=16, max_pages=4, B=2, sinks=1, recent=1, K=9,
             workspace_bytes=256, stream=None)
    return a


@pytest.mark.parametrize("change,want", [
    ({"weights": None}, S.ERR_NULL), ({"block_table": None}, S.ERR_NULL),
    ({"kv_len": None}, S.ERR_NULL), ({"budget": None}, S.ERR_NULL), ({"kept": None}, S.ERR_NULL),
    ({"kept_len": None}, S.ERR_NULL), ({"freed": None}, S.ERR_NULL), ({"n_freed": None}, S.ERR_NULL),
    ({"workspace": None}, S.ERR_WORKSPACE), ({"workspace_bytes": 0}, S.ERR_WORKSPACE),
    ({"B": 0}, S.ERR_SHAPE), ({"B": 65536}, S.ERR_SHAPE), ({"K": 0}, S.ERR_SHAPE),
    ({"max_pages": 0}, S.ERR_SHAPE), ({"max_pages": 1 << 27}, S.ERR_SHAPE),
    ({"page_size": 24}, S.ERR_SHAPE), ({"num_pages": 0}, S.ERR_SHAPE),
    ({"sinks": -1}, S.ERR_ARG), ({"recent": -1}, S.ERR_ARG),
])
def test_evict_refuses(lib, base, change, want):
    a = _evict_args(base)
    a.update(change)
    assert lib.mla_paged_evict(*[a[n] for n in EVICT]) == want


def test_evict_refuses_alignment_and_overlap(lib, base):
    for name, off in [("weights", 2), ("kept", 1), ("freed", 2), ("workspace", 8), ("budget", 3)]:
        a = _evict_args(base)
        a[name] += off
        assert lib.mla_paged_evict(*[a[n] for n in EVICT]) == S.ERR_ALIGN, name
    for one, other in [("kept_len", "kv_len"), ("kept", "weights"), ("freed", "block_table"),
                       ("n_freed", "kept_len"), ("kept_len", "budget"), ("freed", "kept")]:
        a = _evict_args(base)
        a[one] = a[other]
        assert lib.mla_paged_evict(*[a[n] for n in EVICT]) == S.ERR_ARG, (one, other)
    if not torch.cuda.is_available():
        a = _evict_args(base)
        assert _accepted(lib.mla_paged_evict(*[a[n] for n in EVICT]))
        a.update(freed=None, n_freed=None)
        assert _accepted(lib.mla_paged_evict(*[a[n] for n in EVICT]))


COMPACT = ["c_pages", "pe_pages", "weights", "num_pages", "page_size", "block_table", "max_pages",
           "kept", "K", "kept_len", "B", "workspace", "workspace_bytes", "stream"]


def _compact_args(base):
    a = {n: base + 1024 * i for i, n in enumerate(COMPACT)}
    a.update(num_pages=8, page_size=16, max_pages=4, B=2, K=9, workspace_bytes=768, stream=None)
    return a


@pytest.mark.parametrize("change,want", [
    ({"c_pages": None}, S.ERR_NULL), ({"pe_pages": None}, S.ERR_NULL),
    ({"block_table": None}, S.ERR_NULL), ({"kept": None}, S.ERR_NULL),
    ({"kept_len": None}, S.ERR_NULL), ({"workspace": None}, S.ERR_WORKSPACE),
    ({"workspace_bytes": 767}, S.ERR_WORKSPACE), ({"B": 0}, S.ERR_SHAPE), ({"B": 65536}, S.ERR_SHAPE),
    ({"K": 0}, S.ERR_SHAPE), ({"max_pages": 0}, S.ERR_SHAPE), ({"page_size": 15}, S.ERR_SHAPE),
    ({"num_pages": 1 << 28}, S.ERR_SHAPE),
])
def test_compact_refuses(lib, base, change, want):
    a = _compact_args(base)
    a.update(change)
    assert lib.mla_latent_compact(*[a[n] for n in COMPACT]) == want


def test_compact_refuses_alignment(lib, base):
    for name, off in [("c_pages", 8), ("pe_pages", 8), ("weights", 2), ("kept", 2), ("workspace", 4)]:
        a = _compact_args(base)
        a[name] += off
        assert lib.mla_latent_compact(*[a[n] for n in COMPACT]) == S.ERR_ALIGN, name
    if not torch.cuda.is_available():
        a = _compact_args(base)
        a["weights"] = None
        assert lib.mla_latent_compact_workspace_bytes(2, 9) == 768
        assert lib.mla_latent_compact_workspace_bytes(0, 9) == 0
        assert _accepted(lib.mla_latent_compact(*[a[n] for n in COMPACT]))


WEIGHTS = ["q_nope", "q_pe", "c_pages", "pe_pages", "num_pages", "page_size", "block_table",
           "max_pages", "kv_len", "cu_q", "draft_mask", "w_kvb", "B", "T", "H", "scale", "decay",
           "weights", "workspace", "workspace_bytes", "stream"]


def _weights_args(lib, base):
    a = {n: base + 1024 * i for i, n in enumerate(WEIGHTS)}
    a.update(num_pages=8, page_size=16, max_pages=4, B=2, T=3, H=4, scale=0.1, decay=1.0,
             workspace_bytes=lib.mla_latent_key_weights_workspace_bytes(3, 4, 2, 64), stream=None)
    return a


@pytest.mark.parametrize("change,want", [
    ({"q_nope": None}, S.ERR_NULL), ({"q_pe": None}, S.ERR_NULL), ({"c_pages": None}, S.ERR_NULL),
    ({"pe_pages": None}, S.ERR_NULL), ({"block_table": None}, S.ERR_NULL),
    ({"kv_len": None}, S.ERR_NULL), ({"cu_q": None}, S.ERR_NULL), ({"w_kvb": None}, S.ERR_NULL),
    ({"weights": None}, S.ERR_NULL), ({"workspace": None}, S.ERR_WORKSPACE),
    ({"B": 0}, S.ERR_SHAPE), ({"T": 0}, S.ERR_SHAPE), ({"H": 0}, S.ERR_SHAPE),
    ({"H": 1025}, S.ERR_SHAPE), ({"T": (1 << 24) + 1}, S.ERR_SHAPE), ({"max_pages": 0}, S.ERR_SHAPE),
    ({"page_size": 20}, S.ERR_SHAPE), ({"num_pages": 0}, S.ERR_SHAPE),
    ({"scale": 0.0}, S.ERR_ARG), ({"scale": float("inf")}, S.ERR_ARG),
    ({"decay": float("nan")}, S.ERR_ARG), ({"decay": float("inf")}, S.ERR_ARG),
])
def test_weights_refuse(lib, base, change, want):
    a = _weights_args(lib, base)
    a.update(change)
    assert lib.mla_latent_key_weights(*[a[n] for n in WEIGHTS]) == want


def test_weights_refuse_alignment_and_small_workspaces(lib, base):
    for name, off in [("q_nope", 8), ("pe_pages", 8), ("weights", 2), ("draft_mask", 4), ("cu_q", 2)]:
        a = _weights_args(lib, base)
        a[name] += off
        assert lib.mla_latent_key_weights(*[a[n] for n in WEIGHTS]) == S.ERR_ALIGN, name
    size = lib.mla_latent_key_weights_workspace_bytes
    assert size(0, 4, 2, 64) == size(3, 0, 2, 64) == size(3, 1025, 2, 64) == size(3, 4, 0, 64) == 0
    assert size(3, 4, 2, 0) == 0
    assert size(3, 4, 2, 64) > 3 * 4 * (2048 + 4 + 128 * 4)
    # scores are kept up to 256 MB
    assert size(64, 64, 2, 1 << 30) - size(64, 64, 2, 128) == (1 << 28) - 64 * 64 * 512
    a = _weights_args(lib, base)
    if not torch.cuda.is_available():
        assert _accepted(lib.mla_latent_key_weights(*[a[n] for n in WEIGHTS]))
    else:
        a["workspace_bytes"] -= 1
        assert lib.mla_latent_key_weights(*[a[n] for n in WEIGHTS]) == S.ERR_WORKSPACE


def test_tables_refuse_other_widths(lib):
    for dim in (0, 1, 63, 258):
        with pytest.raises(mla.MlaAttnError):
            mla.mla_rope_frequencies(dim=dim)
    # the 64 columns of the cache's keys are the plain call's
    f = (ctypes.c_double * 32)()
    m = ctypes.c_double()
    cfg = mla.RopeConfig()
    assert lib.mla_rope_frequencies(ctypes.byref(cfg), f, ctypes.byref(m)) == 0
    assert (list(f), m.value) == mla.mla_rope_frequencies(dim=64)


def test_binding_refuses_cpu_tensors(lib):
    z = torch.zeros
    i = z(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        mla.mla_rope_apply(z(2, 1, 64), i, z(9, 64))
    with pytest.raises(ValueError):
        mla.mla_paged_evict(z(4, 16), z(2, 3, dtype=torch.int32), i, i)
    with pytest.raises(ValueError):
        mla.mla_latent_compact(z(4, 16, 512).bfloat16(), z(4, 16, 64).bfloat16(),
                               z(2, 3, dtype=torch.int32), z(2, 5, dtype=torch.int32), i)
