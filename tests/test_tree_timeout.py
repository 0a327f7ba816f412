"""The bounded waits of the tree attention's CTA pairs, exercised without any GPU fault: a test build
(tree.cu with MLA_TEST_DROP_P_READY and a 2 ms wait limit; the library proper sets neither) in which
one softmax warp of the first pair withholds one plain arrival that starts no copy.  The mix warp's
wait for it runs out, both CTAs of the pair unwind, the call returns with MLA_ERR_TIMEOUT in the
status word, and the library itself then runs clean on the same GPU."""
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


def test_tree_wait_gives_up_reports_timeout_and_device_stays_usable():
    # 4 sequences of 3000 cached keys: several tiles per pair, so the first pair has a second one
    d = tree_case(40, 4, 64, (3000, 3000), (8, 8), 64, True)
    scale = softmax_scale_192()

    def run():
        out = mla.mla_latent_tree_fwd(d["q_nope"], d["q_pe"], d["c_pages"], d["pe_pages"],
                                      d["block_table"], d["kv_len"], d["cu_q"], d["draft_mask"],
                                      d["w_kvb"], scale)
        torch.cuda.synchronize()
        return out

    want = run()
    path = build_test_variant("wait_timeout_tree", "tree.cu",
                              ["-DMLA_WAIT_LIMIT_NS=2000000ull", "-DMLA_TEST_DROP_P_READY=1"])
    lib = ctypes.CDLL(path)
    p, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.mla_latent_tree_workspace_bytes.restype = sz
    lib.mla_latent_tree_workspace_bytes.argtypes = [i, i, i]
    lib.mla_latent_tree_fwd.restype = i
    lib.mla_latent_tree_fwd.argtypes = [p, p, p, p, i, i, p, i, p, p, p, p, i, i, i, f, p, p, sz, p]
    lib.mla_attn_get_status.restype = i
    lib.mla_attn_get_status.argtypes = [p, p]
    T, H = d["q_nope"].shape[:2]
    n = lib.mla_latent_tree_workspace_bytes(T, H, 4)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(want)
    a = lambda t: t.data_ptr()  # noqa: E731
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    rc = lib.mla_latent_tree_fwd(a(d["q_nope"]), a(d["q_pe"]), a(d["c_pages"]), a(d["pe_pages"]),
                                 d["c_pages"].shape[0], 64, a(d["block_table"]),
                                 d["block_table"].shape[1], a(d["kv_len"]), a(d["cu_q"]),
                                 a(d["draft_mask"]), a(d["w_kvb"]), 4, T, H, scale, a(out), a(ws),
                                 n, stream)
    assert rc == 0
    st = lib.mla_attn_get_status(a(ws), stream)  # synchronises the stream
    elapsed = time.perf_counter() - t0
    assert st == binding.MlaStatus.ERR_TIMEOUT, f"status {st}"
    assert elapsed < 5.0, f"the aborted launch took {elapsed:.2f} s"
    assert lib.mla_attn_get_status(a(ws), stream) == 0
    assert torch.equal(run(), want) and mla.mla_attn_get_status() == 0
