"""ctypes binding of libmla_attn.so (argument marshalling only).

Every step of the attention core runs in the library's CUDA kernels; this module only
checks tensor dtypes/devices, passes raw device pointers, sizes and the current CUDA
stream, and turns status codes into exceptions.  There is no fallback: if the library is
missing, every call raises.
"""
from __future__ import annotations

import ctypes
import enum
import os
import threading
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libmla_attn.so")
_lock = threading.Lock()
_lib = None


class MlaStatus(enum.IntEnum):
    OK = 0
    ERR_NULL = 1
    ERR_SHAPE = 2
    ERR_ALIGN = 3
    ERR_WORKSPACE = 4
    ERR_DEVICE = 5
    ERR_CUDA = 6
    ERR_KVLEN = 7
    ERR_TIMEOUT = 8
    ERR_ARG = 9
    ERR_PAGE = 10
    ERR_TREE = 11


PATH_AUTO, PATH_PREFILL, PATH_DECODE = 0, 1, 2


class MlaAttnError(RuntimeError):
    def __init__(self, status: int, msg: str = ""):
        self.status = MlaStatus(status) if status in MlaStatus._value2member_map_ else status
        super().__init__(f"{msg}{self.status!r}: {_status_string(status)}")


class RopeConfig(ctypes.Structure):
    """mla_rope_config: YaRN rotary scaling (Kimi K2's values are the defaults)."""
    _fields_ = [("rope_theta", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_max_position", ctypes.c_double), ("beta_fast", ctypes.c_double),
                ("beta_slow", ctypes.c_double), ("mscale", ctypes.c_double),
                ("mscale_all_dim", ctypes.c_double)]

    def __init__(self, rope_theta=50000.0, factor=32.0, original_max_position=4096,
                 beta_fast=1.0, beta_slow=1.0, mscale=1.0, mscale_all_dim=1.0):
        super().__init__(float(rope_theta), float(factor), float(original_max_position),
                         float(beta_fast), float(beta_slow), float(mscale),
                         float(mscale_all_dim))


class _Options(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int), ("decode_chunk", ctypes.c_int),
                ("reserved", ctypes.c_int * 6)]


EXPORTED = ("mla_attn_workspace_bytes", "mla_attn_fwd", "mla_attn_fwd_ex",
            "mla_attn_get_status", "mla_status_string", "mla_attn_decode_plan",
            "mla_attn_append_fwd", "mla_rope_frequencies", "mla_rope_table",
            "mla_attn_rope_workspace_bytes", "mla_attn_rope_append_fwd",
            "mla_attn_masked_workspace_bytes", "mla_attn_masked_fwd",
            "mla_latent_workspace_bytes", "mla_latent_decode_fwd",
            "mla_oproj_workspace_bytes", "mla_oproj_fwd", "mla_paged_plan",
            "mla_attn_varlen_workspace_bytes", "mla_attn_varlen_fwd",
            "mla_latent_append", "mla_latent_tree_workspace_bytes", "mla_latent_tree_fwd")


def library():
    """Load libmla_attn.so (built in-tree by build.py); raise if it is not there."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise MlaAttnError(MlaStatus.ERR_CUDA,
                               f"{LIB_PATH} is not built (run python -m "
                               "mla_causal_attention_gb300.build); ")
        lib = ctypes.CDLL(LIB_PATH)
        p, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        fwd_args = [p, p, p, p, p, p, i, i, i, i, i, f, p, p, sz, p]
        lib.mla_attn_workspace_bytes.restype = sz
        lib.mla_attn_workspace_bytes.argtypes = [i, i, i, i]
        lib.mla_attn_fwd.restype = i
        lib.mla_attn_fwd.argtypes = fwd_args
        lib.mla_attn_fwd_ex.restype = i
        lib.mla_attn_fwd_ex.argtypes = fwd_args + [ctypes.POINTER(_Options)]
        lib.mla_attn_get_status.restype = i
        lib.mla_attn_get_status.argtypes = [p, p]
        lib.mla_status_string.restype = ctypes.c_char_p
        lib.mla_status_string.argtypes = [i]
        lib.mla_attn_decode_plan.restype = i
        lib.mla_attn_decode_plan.argtypes = [i, i, i, ctypes.POINTER(i), ctypes.POINTER(i)]
        lib.mla_attn_append_fwd.restype = i
        lib.mla_attn_append_fwd.argtypes = [p, p, p, p, p, p, p, p, p, i, i, i, i, i, f, p, p,
                                            sz, p]
        lib.mla_attn_masked_workspace_bytes.restype = sz
        lib.mla_attn_masked_workspace_bytes.argtypes = [i, i, i, i]
        lib.mla_attn_masked_fwd.restype = i
        lib.mla_attn_masked_fwd.argtypes = [p, p, p, p, p, p, p, i, i, i, i, i, f, p, p, sz, p]
        lib.mla_latent_workspace_bytes.restype = sz
        lib.mla_latent_workspace_bytes.argtypes = [i, i, i]
        lib.mla_latent_decode_fwd.restype = i
        lib.mla_latent_decode_fwd.argtypes = [p, p, p, p, p, p, i, i, i, f, p, p, sz, p]
        lib.mla_oproj_workspace_bytes.restype = sz
        lib.mla_oproj_workspace_bytes.argtypes = []
        lib.mla_oproj_fwd.restype = i
        lib.mla_oproj_fwd.argtypes = [p, p, i, i, i, i, p, p, sz, p]
        lib.mla_rope_frequencies.restype = i
        lib.mla_rope_frequencies.argtypes = [ctypes.POINTER(RopeConfig),
                                             ctypes.POINTER(ctypes.c_double),
                                             ctypes.POINTER(ctypes.c_double)]
        lib.mla_rope_table.restype = i
        lib.mla_rope_table.argtypes = [ctypes.POINTER(RopeConfig), i, p, p]
        lib.mla_attn_rope_workspace_bytes.restype = sz
        lib.mla_attn_rope_workspace_bytes.argtypes = [i, i, i, i]
        lib.mla_attn_rope_append_fwd.restype = i
        lib.mla_attn_rope_append_fwd.argtypes = [p, p, p, p, p, p, p, p, p, i, i, i, i, i, f,
                                                 p, i, p, p, sz, p]
        lib.mla_paged_plan.restype = i
        lib.mla_paged_plan.argtypes = [p, p, i, p, i, p, i, p, i, i, p, i, p, p, p, p, p, p, p,
                                       sz, p]
        lib.mla_latent_append.restype = i
        lib.mla_latent_append.argtypes = [p, p, p, i, p, p, i, i, p, p, i, p, i, p, p, sz, p]
        lib.mla_latent_tree_workspace_bytes.restype = sz
        lib.mla_latent_tree_workspace_bytes.argtypes = [i, i, i]
        lib.mla_latent_tree_fwd.restype = i
        lib.mla_latent_tree_fwd.argtypes = [p, p, p, p, i, i, p, i, p, p, p, p, i, i, i, f, p, p,
                                            sz, p]
        lib.mla_attn_varlen_workspace_bytes.restype = sz
        lib.mla_attn_varlen_workspace_bytes.argtypes = [i, i]
        lib.mla_attn_varlen_fwd.restype = i
        lib.mla_attn_varlen_fwd.argtypes = [p, p, p, p, p, p, p, i, i, i, i, f, p, p, sz, p]
        _lib = lib
        return lib


def _status_string(s: int) -> str:
    try:
        return library().mla_status_string(int(s)).decode()
    except Exception:  # pragma: no cover - library missing
        return "libmla_attn.so unavailable"


def mla_attn_workspace_bytes(B: int, H: int, Tq: int, Tk: int) -> int:
    return int(library().mla_attn_workspace_bytes(B, H, Tq, Tk))


def decode_plan(B: int, H: int, Tk: int):
    c, s = ctypes.c_int(), ctypes.c_int()
    rc = library().mla_attn_decode_plan(B, H, Tk, ctypes.byref(c), ctypes.byref(s))
    if rc != 0:
        raise MlaAttnError(rc)
    return c.value, s.value


class Workspace:
    """A zero-initialised device workspace sized for given shapes (grows on demand).

    A workspace serves one stream at a time: calls that may overlap on the GPU (on
    different streams) need workspaces of their own.  The default one, used when a call
    gets none, is shared by every call on its device.  A buffer that was outgrown is kept,
    since a captured graph may go on using it; growth is at least twofold, so that the kept
    ones together are smaller than the one in use.  A program without graphs of the smaller
    calls gives them back with release_outgrown().
    """

    def __init__(self, device=None):
        self.device = torch.device(device or "cuda")
        self.buf = None
        self.outgrown = []

    def get(self, nbytes: int, stream=None) -> torch.Tensor:
        """The buffer, at least nbytes long.  A new buffer is allocated and zero-filled on
        `stream` (the one the call launches on), so the fill precedes the call's kernels."""
        if self.buf is None or self.buf.numel() < nbytes:
            if self.buf is not None:
                self.outgrown.append(self.buf)
                nbytes = max(nbytes, 2 * self.buf.numel())
            with torch.cuda.stream(stream):
                self.buf = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=self.device)
        return self.buf

    def release_outgrown(self) -> None:
        """Frees the outgrown buffers, with what their status words hold.  Only once no captured
        graph or PreparedCall uses them and the calls on this workspace have completed."""
        self.outgrown.clear()


def _buffer(workspace, dev, nbytes, stream):
    """A call's workspace buffer, at least nbytes long and on the call's device."""
    ws = workspace or _default_workspace(dev)
    buf = ws.buf
    if buf is None or buf.numel() < nbytes:
        buf = ws.get(nbytes, stream=stream or torch.cuda.current_stream(dev))
    if buf.get_device() != dev.index:
        raise ValueError(f"the workspace is on {buf.device}, the call on {dev}")
    return buf


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t, name, dtype, shape, device):
    try:  # the usual case, in few steps
        if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
            return
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _addr(t):
    return None if t is None else t.data_ptr()


def _enqueue(name, dev, stream, workspace, ws_bytes, args):
    """Calls entry point `name` with args, then workspace, its size and the stream, with `dev`
    current.  For calls of a few microseconds the host side counts: no device context unless
    the device changes, and the stream's address without a Stream object."""
    fn = getattr(_lib or library(), name)
    index = dev.index
    s = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    buf = _buffer(workspace, dev, ws_bytes, stream)
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, buf.data_ptr(), buf.numel(), s)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, buf.data_ptr(), buf.numel(), s)
    if rc != 0:
        raise MlaAttnError(rc, name + ": ")


def _check_all(dev, dtype, named):
    """_check of several tensors of one type, (name, tensor, shape) each."""
    index = dev.index
    for name, t, shape in named:
        try:
            if (t.dtype is dtype and t.get_device() == index and t.shape == shape
                    and t.is_contiguous()):
                continue
        except AttributeError:
            pass
        _check(t, name, dtype, shape, dev)


class PreparedCall:
    """mla_attn_fwd with its tensors, workspace, stream and options fixed.

    Construction validates everything once; each call re-enqueues the attention core with
    one ctypes call (no per-call Python checks), which matters when the kernels themselves
    take only microseconds.  The tensors are kept alive by this object.
    """

    def __init__(self, q_nope, q_pe, k_nope, k_pe_shared, v, kv_len, past_len: int,
                 softmax_scale: float, out=None, workspace: "Workspace | None" = None,
                 stream=None, path: int = PATH_AUTO, decode_chunk: int = 0):
        lib = library()
        dev = q_nope.device
        if dev.type != "cuda":
            raise ValueError("inputs must be CUDA tensors")
        B, H, Tq = q_nope.shape[:3]
        Tk = k_nope.shape[2]
        bf = torch.bfloat16
        _check(q_nope, "q_nope", bf, (B, H, Tq, 128), dev)
        _check(q_pe, "q_pe", bf, (B, H, Tq, 64), dev)
        _check(k_nope, "k_nope", bf, (B, H, Tk, 128), dev)
        _check(k_pe_shared, "k_pe_shared", bf, (B, Tk, 64), dev)
        _check(v, "v", bf, (B, H, Tk, 128), dev)
        if kv_len is not None:
            _check(kv_len, "kv_len", torch.int32, (B,), dev)
        if out is None:
            out = torch.empty((B, H, Tq, 128), dtype=bf, device=dev)
        _check(out, "out", bf, (B, H, Tq, 128), dev)
        ws_bytes = lib.mla_attn_workspace_bytes(B, H, Tq, Tk)
        if decode_chunk:
            splits = -(-Tk // decode_chunk)
            ws_bytes = max(ws_bytes, 256 + (-(-B * H * splits * 8 // 256)) * 256
                           + B * H * splits * 512)
        s = stream if stream is not None else torch.cuda.current_stream(dev)
        ws = _buffer(workspace, dev, ws_bytes, s)
        self.out = out
        self.device = dev
        self._keep = (q_nope, q_pe, k_nope, k_pe_shared, v, kv_len, out, ws, s)
        self._opts = _Options(int(path), int(decode_chunk))
        self._fn = lib.mla_attn_fwd_ex
        self._args = (_ptr(q_nope), _ptr(q_pe), _ptr(k_nope), _ptr(k_pe_shared), _ptr(v),
                      _ptr(kv_len), B, H, Tq, Tk, int(past_len), float(softmax_scale),
                      _ptr(out), _ptr(ws), ws.numel(), ctypes.c_void_p(s.cuda_stream),
                      ctypes.byref(self._opts))

    def __call__(self):
        if torch.cuda.current_device() != self.device.index:
            with torch.cuda.device(self.device):
                rc = self._fn(*self._args)
        else:
            rc = self._fn(*self._args)
        if rc != 0:
            raise MlaAttnError(rc, "mla_attn_fwd: ")
        return self.out


def mla_attn_fwd(q_nope, q_pe, k_nope, k_pe_shared, v, kv_len, past_len: int,
                 softmax_scale: float, out=None, workspace: Workspace | None = None,
                 stream=None, path: int = PATH_AUTO, decode_chunk: int = 0):
    """out[B,H,Tq,128] (bf16) of the MLA causal-attention core on the current device.

    q_nope [B,H,Tq,128], q_pe [B,H,Tq,64], k_nope [B,H,Tk,128], k_pe_shared [B,Tk,64],
    v [B,H,Tk,128] (bf16, contiguous, CUDA); kv_len [B] int32 on the same device or None.
    Enqueued on ``stream`` (default: torch's current stream); returns ``out``.
    """
    return PreparedCall(q_nope, q_pe, k_nope, k_pe_shared, v, kv_len, past_len,
                        softmax_scale, out, workspace, stream, path, decode_chunk)()


def mla_attn_append_fwd(q_nope, q_pe, k_nope_new, k_pe_new, v_new, k_nope_cache,
                        k_pe_cache, v_cache, kv_len, past_len: int, softmax_scale: float,
                        out=None, workspace: "Workspace | None" = None, stream=None):
    """Append the new key/value rows at [past_len, past_len + Tq) of the caches, then
    attend over rows [0, past_len + Tq).  Caches: k_nope_cache / v_cache [B,H,T_cap,128],
    k_pe_cache [B,T_cap,64]; new rows [B,H,Tq,128] / [B,Tq,64] / [B,H,Tq,128]."""
    lib = library()
    dev = q_nope.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    B, H, Tq = q_nope.shape[:3]
    T_cap = k_nope_cache.shape[2]
    bf = torch.bfloat16
    _check(q_nope, "q_nope", bf, (B, H, Tq, 128), dev)
    _check(q_pe, "q_pe", bf, (B, H, Tq, 64), dev)
    _check(k_nope_new, "k_nope_new", bf, (B, H, Tq, 128), dev)
    _check(k_pe_new, "k_pe_new", bf, (B, Tq, 64), dev)
    _check(v_new, "v_new", bf, (B, H, Tq, 128), dev)
    _check(k_nope_cache, "k_nope_cache", bf, (B, H, T_cap, 128), dev)
    _check(k_pe_cache, "k_pe_cache", bf, (B, T_cap, 64), dev)
    _check(v_cache, "v_cache", bf, (B, H, T_cap, 128), dev)
    if kv_len is not None:
        _check(kv_len, "kv_len", torch.int32, (B,), dev)
    if out is None:
        out = torch.empty((B, H, Tq, 128), dtype=bf, device=dev)
    _check(out, "out", bf, (B, H, Tq, 128), dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    ws = _buffer(workspace, dev, lib.mla_attn_workspace_bytes(B, H, Tq, past_len + Tq), s)
    with torch.cuda.device(dev):
        rc = lib.mla_attn_append_fwd(_ptr(q_nope), _ptr(q_pe), _ptr(k_nope_new),
                                     _ptr(k_pe_new), _ptr(v_new), _ptr(k_nope_cache),
                                     _ptr(k_pe_cache), _ptr(v_cache), _ptr(kv_len), B, H, Tq,
                                     T_cap, int(past_len), float(softmax_scale), _ptr(out),
                                     _ptr(ws), ws.numel(), ctypes.c_void_p(s.cuda_stream))
    if rc != 0:
        raise MlaAttnError(rc, "mla_attn_append_fwd: ")
    return out


def mla_attn_masked_fwd(q_nope, q_pe, k_nope, k_pe_shared, v, kv_len, key_mask,
                        past_len: int, softmax_scale: float, out=None,
                        workspace: "Workspace | None" = None, stream=None):
    """Attention with a 2D padding mask on the keys: key_mask [B, Tk] (uint8 or bool CUDA
    tensor, nonzero = attend).  Rows that see no visible key get the mean of all value
    rows (uniform weights)."""
    lib = library()
    dev = q_nope.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    B, H, Tq = q_nope.shape[:3]
    Tk = k_nope.shape[2]
    bf = torch.bfloat16
    _check(q_nope, "q_nope", bf, (B, H, Tq, 128), dev)
    _check(q_pe, "q_pe", bf, (B, H, Tq, 64), dev)
    _check(k_nope, "k_nope", bf, (B, H, Tk, 128), dev)
    _check(k_pe_shared, "k_pe_shared", bf, (B, Tk, 64), dev)
    _check(v, "v", bf, (B, H, Tk, 128), dev)
    if kv_len is not None:
        _check(kv_len, "kv_len", torch.int32, (B,), dev)
    if key_mask.dtype == torch.bool:
        key_mask = key_mask.view(torch.uint8)
    _check(key_mask, "key_mask", torch.uint8, (B, Tk), dev)
    if out is None:
        out = torch.empty((B, H, Tq, 128), dtype=bf, device=dev)
    _check(out, "out", bf, (B, H, Tq, 128), dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    ws = _buffer(workspace, dev, lib.mla_attn_masked_workspace_bytes(B, H, Tq, Tk), s)
    with torch.cuda.device(dev):
        rc = lib.mla_attn_masked_fwd(_ptr(q_nope), _ptr(q_pe), _ptr(k_nope), _ptr(k_pe_shared),
                                     _ptr(v), _ptr(kv_len), _ptr(key_mask), B, H, Tq, Tk,
                                     int(past_len), float(softmax_scale), _ptr(out), _ptr(ws),
                                     ws.numel(), ctypes.c_void_p(s.cuda_stream))
    if rc != 0:
        raise MlaAttnError(rc, "mla_attn_masked_fwd: ")
    return out


def mla_latent_decode_fwd(q_nope, q_pe, c_kv, k_pe, w_kvb, kv_len, softmax_scale: float,
                          out=None, workspace: "Workspace | None" = None, stream=None):
    """Decode over the latent cache: q_nope [B,H,128], q_pe [B,H,64], c_kv [B,Tk,512],
    k_pe [B,Tk,64], w_kvb [H*256,512] (kv_b_proj weight), kv_len [B] int32 or None;
    returns out [B,H,128]."""
    lib = library()
    dev = q_nope.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    B, H = q_nope.shape[:2]
    Tk = c_kv.shape[1]
    bf = torch.bfloat16
    _check(q_nope, "q_nope", bf, (B, H, 128), dev)
    _check(q_pe, "q_pe", bf, (B, H, 64), dev)
    _check(c_kv, "c_kv", bf, (B, Tk, 512), dev)
    _check(k_pe, "k_pe", bf, (B, Tk, 64), dev)
    _check(w_kvb, "w_kvb", bf, (H * 256, 512), dev)
    if kv_len is not None:
        _check(kv_len, "kv_len", torch.int32, (B,), dev)
    if out is None:
        out = torch.empty((B, H, 128), dtype=bf, device=dev)
    _check(out, "out", bf, (B, H, 128), dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    ws = _buffer(workspace, dev, lib.mla_latent_workspace_bytes(B, H, Tk), s)
    with torch.cuda.device(dev):
        rc = lib.mla_latent_decode_fwd(_ptr(q_nope), _ptr(q_pe), _ptr(c_kv), _ptr(k_pe),
                                       _ptr(w_kvb), _ptr(kv_len), B, H, Tk,
                                       float(softmax_scale), _ptr(out), _ptr(ws), ws.numel(),
                                       ctypes.c_void_p(s.cuda_stream))
    if rc != 0:
        raise MlaAttnError(rc, "mla_latent_decode_fwd: ")
    return out


def mla_oproj_fwd(attn, w_o, out=None, workspace: "Workspace | None" = None, stream=None):
    """Output projection: attn [B,H,T,128], w_o [N, H*128] (bf16, device); returns y [B,T,N]
    with y[b,i] = w_o @ concat_h attn[b,h,i]."""
    lib = library()
    dev = attn.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    B, H, T = attn.shape[:3]
    N = w_o.shape[0]
    bf = torch.bfloat16
    _check(attn, "attn", bf, (B, H, T, 128), dev)
    _check(w_o, "w_o", bf, (N, H * 128), dev)
    if out is None:
        out = torch.empty((B, T, N), dtype=bf, device=dev)
    _check(out, "out", bf, (B, T, N), dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    ws = _buffer(workspace, dev, lib.mla_oproj_workspace_bytes(), s)
    with torch.cuda.device(dev):
        rc = lib.mla_oproj_fwd(_ptr(attn), _ptr(w_o), B, H, T, N, _ptr(out), _ptr(ws),
                               ws.numel(), ctypes.c_void_p(s.cuda_stream))
    if rc != 0:
        raise MlaAttnError(rc, "mla_oproj_fwd: ")
    return out


class PagedPlan(NamedTuple):
    """What mla_paged_plan lists: offsets of the sequences' new tokens [B + 1], cached lengths
    with them [B], per token its slot and position [T], the first free-list entry left [1], and
    for drafted trees the tokens' ancestor masks [T] (int64), else None."""
    cu_q: torch.Tensor
    kv_len: torch.Tensor
    slots: torch.Tensor
    positions: torch.Tensor
    free_next: torch.Tensor
    draft_mask: "torch.Tensor | None"


def mla_paged_plan(ctx_len, new_len, block_table, free_pages, free_head, page_size: int,
                   num_pages: int, num_tokens: int, parent=None, out=None,
                   workspace: "Workspace | None" = None, stream=None) -> PagedPlan:
    """Takes pages for a step's new tokens and lists where every token goes.

    ctx_len, new_len [B] int32 (cached and new tokens per sequence); block_table
    [B, max_pages] int32, updated in place; free_pages [n] int32, taken from entry
    free_head[0] (int32 [1]) on; parent [num_tokens] int32 for drafted trees (index within the
    sequence's new tokens, -1 for a root).  num_tokens: rows of the per-token outputs, at least
    the new tokens (rows behind them get slot -1).  ``out``: a PagedPlan (or a tuple like it)
    to fill instead of new tensors; none of them may overlap an input or another one."""
    dev = ctx_len.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    B, T, i32 = ctx_len.shape[0], int(num_tokens), torch.int32
    max_pages, n_free = block_table.shape[-1], free_pages.shape[0]
    if out is None:
        new = lambda n, dt=i32: torch.empty(n, dtype=dt, device=dev)  # noqa: E731
        out = PagedPlan(new(B + 1), new(B), new(T), new(T), new(1),
                        None if parent is None else new(T, torch.int64))
    elif not isinstance(out, PagedPlan):
        out = PagedPlan(*out)
    cu_q, kv_len, slots, positions, free_next, draft_mask = out
    _check_all(dev, i32, (
        ("ctx_len", ctx_len, (B,)), ("new_len", new_len, (B,)),
        ("block_table", block_table, (B, max_pages)), ("free_pages", free_pages, (n_free,)),
        ("free_head", free_head, (1,)), ("cu_q", cu_q, (B + 1,)), ("kv_len", kv_len, (B,)),
        ("slots", slots, (T,)), ("positions", positions, (T,)), ("free_next", free_next, (1,))))
    if parent is not None:
        _check(parent, "parent", i32, (T,), dev)
        _check(draft_mask, "draft_mask", torch.int64, (T,), dev)
    elif draft_mask is not None:
        raise ValueError("draft_mask is listed with parent only")
    _enqueue("mla_paged_plan", dev, stream, workspace, 256, (
        ctx_len.data_ptr(), new_len.data_ptr(), B, block_table.data_ptr(), max_pages,
        free_pages.data_ptr(), n_free, free_head.data_ptr(), int(page_size), int(num_pages),
        _addr(parent), T, cu_q.data_ptr(), kv_len.data_ptr(), slots.data_ptr(),
        positions.data_ptr(), _addr(draft_mask), free_next.data_ptr()))
    return out


def mla_latent_append(c_kv_new, k_pe_new, slots, c_pages, pe_pages, positions=None,
                      rope_table=None, q_pe=None, q_pe_out=None,
                      workspace: "Workspace | None" = None, stream=None):
    """Writes the rows c_kv_new [T,512], k_pe_new [T,64] to their slots [T] (int32; negative:
    skipped) of a paged latent cache c_pages [num_pages, page_size, 512] / pe_pages
    [num_pages, page_size, 64].  With rope_table (mla_rope_table) and positions [T] (int32)
    k_pe_new is rotated on its way, and so is q_pe [T,H,64] into q_pe_out (new if None; may be
    q_pe).  Returns q_pe_out (None without q_pe)."""
    dev = c_pages.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    T, bf, i32 = c_kv_new.shape[0], torch.bfloat16, torch.int32
    num_pages, page_size = c_pages.shape[:2]
    _check_all(dev, bf, (
        ("c_kv_new", c_kv_new, (T, 512)), ("k_pe_new", k_pe_new, (T, 64)),
        ("c_pages", c_pages, (num_pages, page_size, 512)),
        ("pe_pages", pe_pages, (num_pages, page_size, 64))))
    _check(slots, "slots", i32, (T,), dev)
    rows, H = 0, 0
    if rope_table is not None:
        rows = rope_table.shape[0]
        _check(rope_table, "rope_table", torch.float32, (rows, 64), dev)
        _check(positions, "positions", i32, (T,), dev)
        if q_pe is not None:
            H = q_pe.shape[1]
            _check(q_pe, "q_pe", bf, (T, H, 64), dev)
            if q_pe_out is None:
                q_pe_out = torch.empty_like(q_pe)
            _check(q_pe_out, "q_pe_out", bf, (T, H, 64), dev)
    elif q_pe is not None:
        raise ValueError("q_pe is rotated with rope_table only")
    if q_pe is None and q_pe_out is not None:
        raise ValueError("q_pe_out without q_pe")
    _enqueue("mla_latent_append", dev, stream, workspace, 256, (
        c_kv_new.data_ptr(), k_pe_new.data_ptr(), slots.data_ptr(), T, c_pages.data_ptr(),
        pe_pages.data_ptr(), num_pages, page_size, _addr(positions), _addr(rope_table), rows,
        _addr(q_pe), H, _addr(q_pe_out)))
    return q_pe_out


def mla_latent_tree_fwd(q_nope, q_pe, c_pages, pe_pages, block_table, kv_len, cu_q, draft_mask,
                        w_kvb, softmax_scale: float, out=None,
                        workspace: "Workspace | None" = None, stream=None):
    """Attention of a step's new tokens over the paged latent cache (their rows appended).

    q_nope [T,H,128], q_pe [T,H,64] packed by sequence; c_pages [num_pages, page_size, 512] /
    pe_pages [num_pages, page_size, 64]; block_table [B, max_pages], kv_len [B] (with the new
    tokens), cu_q [B+1] (int32, from mla_paged_plan); draft_mask [T] int64 for token trees, or
    None for tokens in order (one per sequence: plain decode); w_kvb [H*256,512].  Returns out
    [T,H,128]; rows in front of cu_q[0] and from cu_q[B] on are left as they were."""
    dev = q_nope.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    T, H = q_nope.shape[:2]
    num_pages, page_size = c_pages.shape[:2]
    B, max_pages = block_table.shape
    bf, i32 = torch.bfloat16, torch.int32
    if out is None:
        out = torch.empty((T, H, 128), dtype=bf, device=dev)
    _check_all(dev, bf, (
        ("q_nope", q_nope, (T, H, 128)), ("q_pe", q_pe, (T, H, 64)),
        ("c_pages", c_pages, (num_pages, page_size, 512)),
        ("pe_pages", pe_pages, (num_pages, page_size, 64)),
        ("w_kvb", w_kvb, (H * 256, 512)), ("out", out, (T, H, 128))))
    _check_all(dev, i32, (("block_table", block_table, (B, max_pages)),
                          ("kv_len", kv_len, (B,)), ("cu_q", cu_q, (B + 1,))))
    if draft_mask is not None:
        _check(draft_mask, "draft_mask", torch.int64, (T,), dev)
    nbytes = library().mla_latent_tree_workspace_bytes(T, H, B)
    _enqueue("mla_latent_tree_fwd", dev, stream, workspace, nbytes, (
        q_nope.data_ptr(), q_pe.data_ptr(), c_pages.data_ptr(), pe_pages.data_ptr(), num_pages,
        page_size, block_table.data_ptr(), max_pages, kv_len.data_ptr(), cu_q.data_ptr(),
        _addr(draft_mask), w_kvb.data_ptr(), B, T, H, float(softmax_scale), out.data_ptr()))
    return out


def _slices(t, name, shape, device):
    """(row, head) strides of a [T, heads, width] tensor that may be a slice of a larger one."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    st = t.stride()
    # a dimension of one element has no stride of its own
    head = st[-2] if len(shape) == 3 and shape[1] > 1 else shape[-1]
    row = st[0] if shape[0] > 1 else head * (shape[1] if len(shape) == 3 else 1)
    if st[-1] != 1 or row % 8 or head % 8 or row < 8 or head < 8:
        raise ValueError(f"{name}: the last dimension must be contiguous and the other strides "
                         f"positive multiples of 8, got {st}")
    return row, head


def mla_attn_varlen_fwd(q_nope, q_pe, k_nope, k_pe, v, cu_seqlens, softmax_scale: float, out=None,
                        workspace: "Workspace | None" = None, stream=None):
    """Causal attention over packed prompts: sequence b is rows cu_seqlens[b] .. of every tensor.

    q_nope [T,H,128], q_pe [T,H,64], k_nope / v [T,Hkv,128] (Hkv divides H), k_pe [T,64]
    (bf16; slices of larger tensors are read in place), cu_seqlens [B+1] int32.  Returns out
    [T,H,128]; rows in front of cu_seqlens[0] and from cu_seqlens[B] on are left as they were."""
    dev = q_nope.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    T, H = q_nope.shape[:2]
    Hkv, B = k_nope.shape[1], cu_seqlens.shape[0] - 1
    st = (*_slices(q_nope, "q_nope", (T, H, 128), dev), *_slices(q_pe, "q_pe", (T, H, 64), dev),
          *_slices(k_nope, "k_nope", (T, Hkv, 128), dev), _slices(k_pe, "k_pe", (T, 64), dev)[0],
          *_slices(v, "v", (T, Hkv, 128), dev))
    _check(cu_seqlens, "cu_seqlens", torch.int32, (B + 1,), dev)
    if out is None:
        out = torch.empty((T, H, 128), dtype=torch.bfloat16, device=dev)
    else:
        _check(out, "out", torch.bfloat16, (T, H, 128), dev)
    strides = (ctypes.c_int64 * 9)(*st)
    _enqueue("mla_attn_varlen_fwd", dev, stream, workspace,
             library().mla_attn_varlen_workspace_bytes(T, B), (
                 q_nope.data_ptr(), q_pe.data_ptr(), k_nope.data_ptr(), k_pe.data_ptr(),
                 v.data_ptr(), ctypes.addressof(strides), cu_seqlens.data_ptr(), B, T, H, Hkv,
                 float(softmax_scale), out.data_ptr()))
    return out


def mla_rope_frequencies(cfg: RopeConfig | None = None):
    """(inv_freq[32] as a list of floats, mscale ratio) computed by the library's host code."""
    cfg = cfg or RopeConfig()
    f = (ctypes.c_double * 32)()
    m = ctypes.c_double()
    rc = library().mla_rope_frequencies(ctypes.byref(cfg), f, ctypes.byref(m))
    if rc != 0:
        raise MlaAttnError(rc, "mla_rope_frequencies: ")
    return list(f), m.value


def mla_rope_table(max_pos: int, cfg: RopeConfig | None = None, device=None, stream=None):
    """Device float32 [max_pos, 64] cos|sin table (times the mscale ratio)."""
    cfg = cfg or RopeConfig()
    dev = torch.device(device or "cuda")
    table = torch.empty((max_pos, 64), dtype=torch.float32, device=dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    with torch.cuda.device(dev):
        rc = library().mla_rope_table(ctypes.byref(cfg), int(max_pos), _ptr(table),
                                      ctypes.c_void_p(s.cuda_stream))
    if rc != 0:
        raise MlaAttnError(rc, "mla_rope_table: ")
    return table


def mla_attn_rope_append_fwd(q_nope, q_pe_raw, k_nope_new, k_pe_new_raw, v_new, k_nope_cache,
                             k_pe_cache, v_cache, kv_len, past_len: int, softmax_scale: float,
                             rope_table, out=None, workspace: "Workspace | None" = None,
                             stream=None):
    """Rotate q_pe_raw / k_pe_new_raw at positions past_len + t (table from mla_rope_table),
    append the new rows (rotated rotary keys) at [past_len, past_len + Tq) of the caches,
    then attend over rows [0, past_len + Tq)."""
    lib = library()
    dev = q_nope.device
    if dev.type != "cuda":
        raise ValueError("inputs must be CUDA tensors")
    B, H, Tq = q_nope.shape[:3]
    T_cap = k_nope_cache.shape[2]
    bf = torch.bfloat16
    _check(q_nope, "q_nope", bf, (B, H, Tq, 128), dev)
    _check(q_pe_raw, "q_pe_raw", bf, (B, H, Tq, 64), dev)
    _check(k_nope_new, "k_nope_new", bf, (B, H, Tq, 128), dev)
    _check(k_pe_new_raw, "k_pe_new_raw", bf, (B, Tq, 64), dev)
    _check(v_new, "v_new", bf, (B, H, Tq, 128), dev)
    _check(k_nope_cache, "k_nope_cache", bf, (B, H, T_cap, 128), dev)
    _check(k_pe_cache, "k_pe_cache", bf, (B, T_cap, 64), dev)
    _check(v_cache, "v_cache", bf, (B, H, T_cap, 128), dev)
    _check(rope_table, "rope_table", torch.float32, (rope_table.shape[0], 64), dev)
    if kv_len is not None:
        _check(kv_len, "kv_len", torch.int32, (B,), dev)
    if out is None:
        out = torch.empty((B, H, Tq, 128), dtype=bf, device=dev)
    _check(out, "out", bf, (B, H, Tq, 128), dev)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    ws = _buffer(workspace, dev, lib.mla_attn_rope_workspace_bytes(B, H, Tq, past_len + Tq), s)
    with torch.cuda.device(dev):
        rc = lib.mla_attn_rope_append_fwd(
            _ptr(q_nope), _ptr(q_pe_raw), _ptr(k_nope_new), _ptr(k_pe_new_raw), _ptr(v_new),
            _ptr(k_nope_cache), _ptr(k_pe_cache), _ptr(v_cache), _ptr(kv_len), B, H, Tq, T_cap,
            int(past_len), float(softmax_scale), _ptr(rope_table), int(rope_table.shape[0]),
            _ptr(out), _ptr(ws), ws.numel(), ctypes.c_void_p(s.cuda_stream))
    if rc != 0:
        raise MlaAttnError(rc, "mla_attn_rope_append_fwd: ")
    return out


def mla_attn_get_status(workspace: Workspace | None = None, device=None, stream=None) -> int:
    """Synchronise and read/clear the device status word (0 = no device-side error)."""
    dev = torch.device(device or "cuda")
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    ws = workspace or _default_workspace(dev)
    bufs = [ws.get(256, stream=s), *ws.outgrown]  # each has a status word of its own
    with torch.cuda.device(dev):
        codes = [int(library().mla_attn_get_status(_ptr(b), ctypes.c_void_p(s.cuda_stream)))
                 for b in bufs]
    return next((c for c in codes if c != 0), 0)


_default_ws: dict = {}


def _default_workspace(dev) -> Workspace:
    # "cuda" and "cuda:0" are one workspace: a status is read where the calls recorded it
    key = dev.index if dev.index is not None else torch.cuda.current_device()
    ws = _default_ws.get(key)
    if ws is None:
        ws = _default_ws.setdefault(key, Workspace(torch.device("cuda", key)))
    return ws
