"""What the paged-cache entry points refuse, on the host and before any launch (no GPU)."""
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


def _no_device():
    return (S.ERR_CUDA, S.ERR_DEVICE)


PLAN = ["ctx_len", "new_len", "B", "block_table", "max_pages", "free_pages", "n_free", "free_head",
        "page_size", "num_pages", "parent", "T", "cu_q", "kv_len", "slots", "positions",
        "draft_mask", "free_next", "workspace", "workspace_bytes", "stream"]


def _plan_args(base):
    a = {n: base + 256 * i for i, n in enumerate(PLAN)}
    a.update(B=2, max_pages=4, n_free=3, page_size=16, num_pages=8, T=5, parent=None,
             draft_mask=None, workspace_bytes=256, stream=None)
    return a


@pytest.mark.parametrize("change,want", [
    ({"ctx_len": None}, S.ERR_NULL), ({"new_len": None}, S.ERR_NULL),
    ({"block_table": None}, S.ERR_NULL), ({"free_pages": None}, S.ERR_NULL),
    ({"free_head": None}, S.ERR_NULL), ({"cu_q": None}, S.ERR_NULL),
    ({"kv_len": None}, S.ERR_NULL), ({"slots": None}, S.ERR_NULL),
    ({"positions": None}, S.ERR_NULL), ({"free_next": None}, S.ERR_NULL),
    ({"draft_mask": 512}, S.ERR_NULL), ({"parent": 512}, S.ERR_NULL),
    ({"workspace": None}, S.ERR_WORKSPACE), ({"workspace_bytes": 255}, S.ERR_WORKSPACE),
    ({"B": 0}, S.ERR_SHAPE), ({"T": 0}, S.ERR_SHAPE), ({"max_pages": 0}, S.ERR_SHAPE),
    ({"n_free": -1}, S.ERR_SHAPE), ({"page_size": 8}, S.ERR_SHAPE),
    ({"page_size": 48}, S.ERR_SHAPE), ({"page_size": 2048}, S.ERR_SHAPE),
    ({"num_pages": 0}, S.ERR_SHAPE), ({"num_pages": 1 << 27}, S.ERR_SHAPE),
    ({"max_pages": 1 << 27}, S.ERR_SHAPE),
])
def test_plan_refuses(lib, base, change, want):
    a = _plan_args(base)
    a.update(change)
    assert lib.mla_paged_plan(*[a[n] for n in PLAN]) == want


def test_plan_refuses_alignment_and_alias(lib, base):
    for name, off in [("slots", 4), ("positions", 8), ("ctx_len", 2), ("block_table", 1),
                      ("free_next", 2), ("workspace", 4)]:
        a = _plan_args(base)
        a[name] += off
        assert lib.mla_paged_plan(*[a[n] for n in PLAN]) == S.ERR_ALIGN, name
    for out, read in (("free_next", "free_head"), ("kv_len", "ctx_len"), ("kv_len", "new_len")):
        a = _plan_args(base)
        a[out] = a[read]
        assert lib.mla_paged_plan(*[a[n] for n in PLAN]) == S.ERR_ARG
    if not torch.cuda.is_available():
        a = _plan_args(base)
        assert lib.mla_paged_plan(*[a[n] for n in PLAN]) in _no_device()


APPEND = ["c_kv_new", "k_pe_new", "slots", "T", "c_pages", "pe_pages", "num_pages", "page_size",
          "positions", "rope_table", "table_rows", "q_pe", "H", "q_pe_out", "workspace",
          "workspace_bytes", "stream"]


def _append_args(base):
    a = {n: base + 256 * i for i, n in enumerate(APPEND)}
    a.update(T=3, num_pages=2, page_size=16, table_rows=9, H=2, workspace_bytes=256, stream=None)
    return a


@pytest.mark.parametrize("change,want", [
    ({"c_kv_new": None}, S.ERR_NULL), ({"k_pe_new": None}, S.ERR_NULL),
    ({"slots": None}, S.ERR_NULL), ({"c_pages": None}, S.ERR_NULL),
    ({"pe_pages": None}, S.ERR_NULL), ({"positions": None}, S.ERR_NULL),
    ({"rope_table": None}, S.ERR_NULL),        # q_pe would stay unrotated
    ({"q_pe": None}, S.ERR_NULL), ({"q_pe_out": None}, S.ERR_NULL),
    ({"workspace": None}, S.ERR_WORKSPACE), ({"workspace_bytes": 0}, S.ERR_WORKSPACE),
    ({"T": 0}, S.ERR_SHAPE), ({"H": 0}, S.ERR_SHAPE), ({"table_rows": 0}, S.ERR_SHAPE),
    ({"page_size": 17}, S.ERR_SHAPE), ({"num_pages": -1}, S.ERR_SHAPE),
])
def test_append_refuses(lib, base, change, want):
    a = _append_args(base)
    a.update(change)
    assert lib.mla_latent_append(*[a[n] for n in APPEND]) == want


def test_append_refuses_alignment(lib, base):
    for name in ("c_kv_new", "k_pe_new", "c_pages", "pe_pages", "rope_table", "q_pe", "q_pe_out"):
        a = _append_args(base)
        a[name] += 8
        assert lib.mla_latent_append(*[a[n] for n in APPEND]) == S.ERR_ALIGN, name
    if not torch.cuda.is_available():
        a = _append_args(base)
        assert lib.mla_latent_append(*[a[n] for n in APPEND]) in _no_device()


def test_status_names(lib):
    assert lib.mla_status_string(10).decode().startswith("MLA_ERR_PAGE")
    assert lib.mla_status_string(11).decode().startswith("MLA_ERR_TREE")


def test_binding_refuses_cpu_tensors(lib):
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        mla.mla_paged_plan(i, i, i[None], i, i, 16, 1, 1)
    x = torch.zeros((1, 16, 512), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mla.mla_latent_append(x[0], x[0], i, x, x)


TREE = ["q_nope", "q_pe", "c_pages", "pe_pages", "num_pages", "page_size", "block_table",
        "max_pages", "kv_len", "cu_q", "draft_mask", "w_kvb", "B", "T", "H", "scale", "out",
        "workspace", "workspace_bytes", "stream"]


def _tree_args(base, lib):
    a = {n: base + 256 * i for i, n in enumerate(TREE)}
    a.update(num_pages=4, page_size=16, max_pages=2, B=2, T=3, H=4, scale=0.1, stream=None,
             workspace_bytes=lib.mla_latent_tree_workspace_bytes(3, 4, 2))
    return a


@pytest.mark.parametrize("change,want", [
    ({k: None}, S.ERR_NULL) for k in ("q_nope", "q_pe", "c_pages", "pe_pages", "block_table",
                                      "kv_len", "cu_q", "w_kvb", "out")
] + [
    ({"workspace": None}, S.ERR_WORKSPACE), ({"B": 0}, S.ERR_SHAPE), ({"T": 0}, S.ERR_SHAPE),
    ({"H": 0}, S.ERR_SHAPE), ({"H": 1025}, S.ERR_SHAPE), ({"page_size": 20}, S.ERR_SHAPE),
    ({"num_pages": 0}, S.ERR_SHAPE), ({"max_pages": 0}, S.ERR_SHAPE),
    ({"T": 1 << 27}, S.ERR_SHAPE), ({"scale": 0.0}, S.ERR_ARG), ({"scale": float("inf")}, S.ERR_ARG),
    ({"max_pages": (1 << 26) + 1}, S.ERR_SHAPE),
])
def test_tree_refuses(lib, base, change, want):
    a = _tree_args(base, lib)
    a.update(change)
    assert lib.mla_latent_tree_fwd(*[a[n] for n in TREE]) == want


def test_tree_refuses_alignment_and_small_workspaces(lib, base):
    for name in ("q_nope", "q_pe", "c_pages", "pe_pages", "w_kvb", "out", "workspace"):
        a = _tree_args(base, lib)
        a[name] += 8
        assert lib.mla_latent_tree_fwd(*[a[n] for n in TREE]) == S.ERR_ALIGN, name
    a = _tree_args(base, lib)
    a["draft_mask"] += 4
    assert lib.mla_latent_tree_fwd(*[a[n] for n in TREE]) == S.ERR_ALIGN
    assert lib.mla_latent_tree_workspace_bytes(0, 4, 2) == 0
    assert lib.mla_latent_tree_workspace_bytes(3, 1025, 2) == 0
    a = _tree_args(base, lib)
    a["workspace_bytes"] = 256
    want = (S.ERR_WORKSPACE,) if torch.cuda.is_available() else _no_device()
    assert lib.mla_latent_tree_fwd(*[a[n] for n in TREE]) in want


VARLEN = ["q_nope", "q_pe", "k_nope", "k_pe", "v", "strides", "cu_seqlens", "B", "T", "H", "Hkv",
          "scale", "out", "workspace", "workspace_bytes", "stream"]


def _varlen_args(base, lib, strides=None):
    a = {n: base + 256 * i for i, n in enumerate(VARLEN)}
    a.update(B=2, T=3, H=4, Hkv=2, scale=0.1, stream=None, strides=None,
             workspace_bytes=lib.mla_attn_varlen_workspace_bytes(3, 2))
    if strides is not None:
        a["strides"] = ctypes.addressof((ctypes.c_int64 * 9)(*strides))
    return a


@pytest.mark.parametrize("change,want", [
    ({k: None}, S.ERR_NULL) for k in ("q_nope", "q_pe", "k_nope", "k_pe", "v", "cu_seqlens", "out")
] + [
    ({"workspace": None}, S.ERR_WORKSPACE), ({"workspace_bytes": 256}, S.ERR_WORKSPACE),
    ({"B": 0}, S.ERR_SHAPE), ({"T": 0}, S.ERR_SHAPE), ({"H": 0}, S.ERR_SHAPE),
    ({"Hkv": 0}, S.ERR_SHAPE), ({"Hkv": 3}, S.ERR_SHAPE), ({"Hkv": 8}, S.ERR_SHAPE),
    ({"T": 1 << 27}, S.ERR_SHAPE), ({"scale": -1.0}, S.ERR_ARG),
])
def test_varlen_refuses(lib, base, change, want):
    a = _varlen_args(base, lib)
    a.update(change)
    assert lib.mla_attn_varlen_fwd(*[a[n] for n in VARLEN]) == want


def test_varlen_refuses_strides_and_alignment(lib, base):
    good = [4 * 192, 192, 4 * 192, 192, 512, 256, 64, 512, 256]
    for i in range(9):
        for bad in (0, 4, -8, good[i] + 1):
            keep = (ctypes.c_int64 * 9)(*(good[:i] + [bad] + good[i + 1:]))
            a = _varlen_args(base, lib)
            a["strides"] = ctypes.addressof(keep)
            assert lib.mla_attn_varlen_fwd(*[a[n] for n in VARLEN]) == S.ERR_SHAPE
    for name in ("q_nope", "q_pe", "k_nope", "k_pe", "v", "out", "workspace"):
        a = _varlen_args(base, lib)
        a[name] += 8
        assert lib.mla_attn_varlen_fwd(*[a[n] for n in VARLEN]) == S.ERR_ALIGN
    if not torch.cuda.is_available():
        a = _varlen_args(base, lib)
        assert lib.mla_attn_varlen_fwd(*[a[n] for n in VARLEN]) in _no_device()


def test_an_outgrown_workspace_is_kept():
    """A captured graph may still use it."""
    ws = binding.Workspace("cpu")
    first = ws.get(300)
    at = first.data_ptr()
    assert first.numel() == 300 and ws.get(200) is first
    del first
    second = ws.get(400)
    assert second.numel() == 600 and [b.data_ptr() for b in ws.outgrown] == [at]
    assert ws.get(10000).numel() == 10000 and ws.outgrown[1] is second


def test_plan_refuses_overlap(lib, base):
    """Every output with every input and every other output, from its first byte to its last."""
    size = dict(ctx_len=8, new_len=8, free_pages=12, free_head=4, parent=20, block_table=32, cu_q=12,
                kv_len=8, slots=20, positions=20, draft_mask=40, free_next=4)
    outs = ["block_table", "cu_q", "kv_len", "slots", "positions", "draft_mask", "free_next"]
    def call(**change):
        a = _plan_args(base)
        a.update(parent=base + 256 * 30, draft_mask=base + 256 * 31, **change)
        return a, lambda: lib.mla_paged_plan(*[a[n] for n in PLAN])

    for o in outs:
        for other in size:
            if other == o:
                continue
            a, run = call()
            align = 16 if o in ("slots", "positions", "draft_mask") else 4
            a[o] = a[other]
            assert run() == S.ERR_ARG, (o, other)
            # the output's first byte just inside the other's last word
            inside = (size[other] - 4) // align * align
            a[o] = a[other] + inside
            assert run() == S.ERR_ARG, (o, other, inside)
            if not torch.cuda.is_available():  # and just behind it: no call of this is run on a GPU
                a[o] = a[other] + -(-size[other] // align) * align
                assert run() in _no_device(), (o, other)


def test_outgrown_workspaces_are_given_back():
    import weakref
    ws = binding.Workspace("cpu")
    gone = weakref.ref(ws.get(300))
    kept = ws.get(400)
    assert gone() is not None
    ws.release_outgrown()
    assert gone() is None and ws.outgrown == [] and ws.get(400) is kept


def test_a_workspace_of_another_device_is_refused():
    ws = binding.Workspace("cpu")
    with pytest.raises(ValueError, match="workspace is on cpu"):
        ws.get(300)
        binding._buffer(ws, torch.device("cuda", 0), 300, None)
