"""The bounded waits of the key weights' CTA pairs and of the compaction, exercised without any GPU
fault: test builds with a 2 ms wait limit (the library proper sets neither define) in which one plain
arrival, or one flag, is withheld that starts no copy.  The waits for it run out, the kernels unwind, the
call returns with MLA_ERR_TIMEOUT in the status word, and the library itself then runs clean."""
import ctypes
import time

import pytest
import torch

import mla_causal_attention_gb300 as mla
from mla_causal_attention_gb300 import binding
from mla_causal_attention_gb300.build import build_test_variant
from mla_causal_attention_gb300.workloads import softmax_scale_192
from paged_helpers import tree_case

pytestmark = pytest.mark.gpu

SCALE = softmax_scale_192()


def _with(lib_path, names, run):
    """run() with the binding's library exchanged for the test build's functions `names`."""
    lib, real = ctypes.CDLL(lib_path), binding.library()
    for n in (*names, "mla_attn_get_status", "mla_status_string"):
        getattr(lib, n).argtypes = getattr(real, n).argtypes
        getattr(lib, n).restype = getattr(real, n).restype
    for n in ("mla_latent_key_weights_workspace_bytes", "mla_latent_compact_workspace_bytes"):
        getattr(lib, n).argtypes = getattr(real, n).argtypes
        getattr(lib, n).restype = getattr(real, n).restype
    binding._lib = lib
    try:
        t0 = time.perf_counter()
        status = run()
        assert time.perf_counter() - t0 < 5.0
        return status
    finally:
        binding._lib = real


# one token of 64 heads: the first pass alone has several tiles per pair; 16 tokens: more rows than are
# kept, so that the second pass computes scores too
@pytest.mark.parametrize("ctx,new", [(40000, 1), (6000, 16)])
def test_key_weights_wait_gives_up(ctx, new):
    d = tree_case(40, 2, 64, (ctx, ctx), (new, new), 64, False)
    old = torch.rand(d["c_pages"].shape[:2], device="cuda")

    def run(workspace=None):
        w = old.clone()
        mla.mla_latent_key_weights(d["q_nope"], d["q_pe"], d["c_pages"], d["pe_pages"],
                                   d["block_table"], d["kv_len"], d["cu_q"], None, d["w_kvb"], SCALE, w,
                                   workspace=workspace)
        torch.cuda.synchronize()
        return w

    want = run()
    path = build_test_variant("wait_timeout_weights", "key_weights.cu",
                              ["-DMLA_WAIT_LIMIT_NS=2000000ull", "-DMLA_TEST_DROP_S_FREE=1"])
    ws = mla.Workspace("cuda:0")

    def aborted():
        run(ws)
        return mla.mla_attn_get_status(ws)

    assert _with(path, ("mla_latent_key_weights",), aborted) == binding.MlaStatus.ERR_TIMEOUT
    assert mla.mla_attn_get_status(ws) == 0
    assert torch.equal(run(ws), want) and mla.mla_attn_get_status(ws) == 0


def test_waits_grow_with_the_rows():
    """A pair's keys stay in use for 312 tiles of rows, some 0.8 ms: longer than the limit of this build
    (0.2 ms), which the wait for them grows beyond."""
    d = tree_case(41, 1, 64, (19400, 19400), (600, 600), 64, False)
    old = torch.zeros(d["c_pages"].shape[:2], device="cuda")
    ws = mla.Workspace("cuda:0")

    def run():
        w = old.clone()
        mla.mla_latent_key_weights(d["q_nope"], d["q_pe"], d["c_pages"], d["pe_pages"],
                                   d["block_table"], d["kv_len"], d["cu_q"], None, d["w_kvb"], SCALE, w,
                                   workspace=ws)
        torch.cuda.synchronize()
        return w, mla.mla_attn_get_status(ws)

    want, status = run()
    assert status == 0
    path = build_test_variant("wait_long_weights", "key_weights.cu", ["-DMLA_WAIT_LIMIT_NS=200000ull"])
    got, status = _with(path, ("mla_latent_key_weights",), run)
    assert status == 0 and torch.equal(got, want)


def test_compaction_wait_gives_up():
    n, page = 4000, 64
    pages = -(-n // page)
    table = torch.randperm(pages, device="cuda", dtype=torch.int32)[None]
    kept = torch.arange(1, n, device="cuda", dtype=torch.int32)[None].contiguous()  # all move by one
    c0, pe0 = (torch.randn(pages, page, k, device="cuda").bfloat16() for k in (512, 64))

    def run(workspace=None):
        c, pe = c0.clone(), pe0.clone()
        mla.mla_latent_compact(c, pe, table, kept, torch.full((1,), n - 1, dtype=torch.int32,
                                                               device="cuda"), workspace=workspace)
        torch.cuda.synchronize()
        return c

    want = run()
    path = build_test_variant("wait_timeout_compact", "evict.cu",
                              ["-DMLA_WAIT_LIMIT_NS=2000000ull", "-DMLA_TEST_DROP_READ=1"])
    ws = mla.Workspace("cuda:0")

    def aborted():
        run(ws)
        return mla.mla_attn_get_status(ws)

    assert _with(path, ("mla_latent_compact",), aborted) == binding.MlaStatus.ERR_TIMEOUT
    assert torch.equal(run(ws), want) and mla.mla_attn_get_status(ws) == 0
