"""Thin ctypes binding of libswa_attn.so (include/swa_attn.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI.  There is no CPU fallback; if the library is
missing or was not built, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
SO_PATH = os.path.join(_PKG, "libswa_attn.so")

# names declared in include/swa_attn.h
EXPORTED = (
    "swa_attn_fwd_workspace_bytes",
    "swa_attn_fwd",
    "swa_attn_bwd_workspace_bytes",
    "swa_attn_bwd",
    "swa_attn_get_status",
    "swa_attn_strerror",
    "swa_attn_version",
    "swa_attn_profile_begin",
    "swa_attn_profile_end",
    "swa_attn_bwd_noalloc",
    "swa_attn_selftest_timeout",
    "swa_attn_fwd_workspace_bytes_ex",
    "swa_attn_bwd_workspace_bytes_ex",
    "swa_attn_fwd_ex",
    "swa_attn_bwd_ex",
    "swa_attn_fwd_workspace_bytes_prefix",
    "swa_attn_bwd_workspace_bytes_prefix",
    "swa_attn_fwd_prefix",
    "swa_attn_bwd_prefix",
    "swa_attn_add_rows_f32",
    "swa_attn_fwd_sinks",
    "swa_attn_bwd_sinks",
    "swa_attn_fwd_workspace_bytes_shared",
    "swa_attn_fwd_shared",
    "swa_attn_qk_rope_fwd",
    "swa_attn_qk_rope_bwd_workspace_bytes",
    "swa_attn_qk_rope_bwd",
)

_lock = threading.Lock()
_lib = None


class SwaError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {strerror(code)} ({code})")


def load(path: str | None = None) -> ctypes.CDLL:
    """Load the shared library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or SO_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                f"{p} not found: build the CUDA library first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(p)
        I, Z, P, F = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
        shape = [I, I, I, I, I, I]
        lib.swa_attn_fwd_workspace_bytes.argtypes = shape
        lib.swa_attn_fwd_workspace_bytes.restype = Z
        lib.swa_attn_bwd_workspace_bytes.argtypes = shape
        lib.swa_attn_bwd_workspace_bytes.restype = Z
        lib.swa_attn_fwd.argtypes = [P, P, P, P, P] + shape + [F, P, Z, P]
        lib.swa_attn_fwd.restype = I
        lib.swa_attn_bwd.argtypes = [P, P, P, P, P, P, P, P, P] + shape + [F, P, Z, P]
        lib.swa_attn_bwd.restype = I
        lib.swa_attn_get_status.argtypes = [P]
        lib.swa_attn_get_status.restype = I
        lib.swa_attn_strerror.argtypes = [I]
        lib.swa_attn_strerror.restype = ctypes.c_char_p
        lib.swa_attn_version.argtypes = []
        lib.swa_attn_version.restype = I
        lib.swa_attn_profile_begin.argtypes = []
        lib.swa_attn_profile_begin.restype = I
        lib.swa_attn_profile_end.argtypes = [P, I, ctypes.POINTER(I)]
        lib.swa_attn_profile_end.restype = I
        lib.swa_attn_bwd_noalloc.argtypes = [P, P, P, P, P, P, P, P, P] + shape + [F, P]
        lib.swa_attn_bwd_noalloc.restype = I
        lib.swa_attn_selftest_timeout.argtypes = [P]
        lib.swa_attn_selftest_timeout.restype = I
        shape_ex = [I, I, I, I, I, I, I, I]  # B, Hq, Hkv, Lq, Lk, D, window, causal
        lib.swa_attn_fwd_workspace_bytes_ex.argtypes = shape_ex
        lib.swa_attn_fwd_workspace_bytes_ex.restype = Z
        lib.swa_attn_bwd_workspace_bytes_ex.argtypes = shape_ex
        lib.swa_attn_bwd_workspace_bytes_ex.restype = Z
        lib.swa_attn_fwd_ex.argtypes = [P, P, P, P, P] + shape_ex + [F, P, Z, P]
        lib.swa_attn_fwd_ex.restype = I
        lib.swa_attn_bwd_ex.argtypes = [P, P, P, P, P, P, P, P, P] + shape_ex + [F, P, Z, P]
        lib.swa_attn_bwd_ex.restype = I
        shape_px = [I, I, I, I, I, I, I, I]  # B, Hq, Hkv, L, D, window, prompt_len, chosen_len
        lib.swa_attn_fwd_workspace_bytes_prefix.argtypes = shape_px
        lib.swa_attn_fwd_workspace_bytes_prefix.restype = Z
        lib.swa_attn_bwd_workspace_bytes_prefix.argtypes = shape_px
        lib.swa_attn_bwd_workspace_bytes_prefix.restype = Z
        lib.swa_attn_fwd_prefix.argtypes = [P, P, P, P, P] + shape_px + [F, P, Z, P]
        lib.swa_attn_fwd_prefix.restype = I
        lib.swa_attn_bwd_prefix.argtypes = [P, P, P, P, P, P, P, P, P] + shape_px + [F, P, Z, P]
        lib.swa_attn_bwd_prefix.restype = I
        lib.swa_attn_add_rows_f32.argtypes = [P, P, I, I, I, I, I, P]
        lib.swa_attn_add_rows_f32.restype = I
        # attention sinks: the sink logits after v; the backward adds dsinks after dv
        lib.swa_attn_fwd_sinks.argtypes = [P, P, P, P, P, P] + shape_ex + [F, P, Z, P]
        lib.swa_attn_fwd_sinks.restype = I
        lib.swa_attn_bwd_sinks.argtypes = [P, P, P, P, P, P, P, P, P, P, P] + shape_ex + [F, P, Z, P]
        lib.swa_attn_bwd_sinks.restype = I
        # shared prefix: B, Hq, Hkv, Lq, prefix_len, [prefix_rows,] own_rows, D, window
        lib.swa_attn_fwd_workspace_bytes_shared.argtypes = [I] * 8
        lib.swa_attn_fwd_workspace_bytes_shared.restype = Z
        lib.swa_attn_fwd_shared.argtypes = [P] * 9 + [I] * 9 + [F, P, Z, P]
        lib.swa_attn_fwd_shared.restype = I
        # per-head norm and rotation: B, Hq, Hkv, L, D, [kv_rows,] rot_dim, interleaved, pos0, eps, weight_offset
        LL = ctypes.c_longlong
        lib.swa_attn_qk_rope_fwd.argtypes = [P] * 3 + [LL] * 3 + [P] * 8 + [I] * 9 + [F, F, P]
        lib.swa_attn_qk_rope_fwd.restype = I
        lib.swa_attn_qk_rope_bwd_workspace_bytes.argtypes = [I, I, I]
        lib.swa_attn_qk_rope_bwd_workspace_bytes.restype = Z
        lib.swa_attn_qk_rope_bwd.argtypes = [P] * 2 + [LL] * 2 + [P] * 10 + [LL] * 3 + [P] * 2 + [I] * 8 + [F, F, P, Z, P]
        lib.swa_attn_qk_rope_bwd.restype = I
        _lib = lib
        return lib


class KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 48), ("launches", ctypes.c_longlong), ("total_ms", ctypes.c_double)]


def profile_begin() -> None:
    rc = load().swa_attn_profile_begin()
    if rc:
        raise SwaError(rc, "swa_attn_profile_begin")


def profile_end(max_entries: int = 32) -> dict:
    """Return {kernel name: (launches, total_ms)} recorded since profile_begin()."""
    buf = (KernelTime * max_entries)()
    n = ctypes.c_int(0)
    rc = load().swa_attn_profile_end(buf, max_entries, ctypes.byref(n))
    if rc:
        raise SwaError(rc, "swa_attn_profile_end")
    return {buf[i].name.decode(): (int(buf[i].launches), float(buf[i].total_ms)) for i in range(n.value)}


def strerror(code: int) -> str:
    return load().swa_attn_strerror(int(code)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream):
    if stream is None:
        import torch

        # the handle alone: torch.cuda.current_stream() builds a Stream object
        # around it, which took 2.9 us of a call's 10 to 20 on the GB300's host
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _dims(q, k, D=None):
    B, Hq, L, D_ = q.shape
    Hkv = k.shape[1]
    return B, Hq, Hkv, L, D_


def fwd_workspace_bytes(B, Hq, Hkv, L, D, window) -> int:
    return int(load().swa_attn_fwd_workspace_bytes(B, Hq, Hkv, L, D, window))


def bwd_workspace_bytes(B, Hq, Hkv, L, D, window) -> int:
    return int(load().swa_attn_bwd_workspace_bytes(B, Hq, Hkv, L, D, window))


def fwd_workspace_bytes_ex(B, Hq, Hkv, Lq, Lk, D, window, causal=True) -> int:
    return int(load().swa_attn_fwd_workspace_bytes_ex(B, Hq, Hkv, Lq, Lk, D, window, int(bool(causal))))


def bwd_workspace_bytes_ex(B, Hq, Hkv, Lq, Lk, D, window, causal=True) -> int:
    return int(load().swa_attn_bwd_workspace_bytes_ex(B, Hq, Hkv, Lq, Lk, D, window, int(bool(causal))))


def _dims_ex(q, k):
    B, Hq, Lq, D = q.shape
    return B, Hq, k.shape[1], Lq, k.shape[2], D


def swa_attn_fwd_ex(q, k, v, o, lse, window: int, causal: bool, scale: float, workspace=None, stream=None) -> None:
    """Forward through the C ABI for q [B,Hq,Lq,D] and k, v [B,Hkv,Lk,D]
    (Lq <= Lk; the queries are the last Lq key positions); o fp32
    [B,Hq,Lq,D] and lse fp32 [B,Hq,Lq] are caller-allocated outputs."""
    B, Hq, Hkv, Lq, Lk, D = _dims_ex(q, k)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().swa_attn_fwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, Lq, Lk, D, int(window),
                                int(bool(causal)), float(scale), _ptr(workspace), nbytes, _stream_ptr(stream))
    if rc:
        raise SwaError(rc, "swa_attn_fwd_ex")


def swa_attn_bwd_ex(q, k, v, o, lse, dO, dq, dk, dv, window: int, causal: bool, scale: float, workspace=None,
                    stream=None) -> None:
    """Backward through the C ABI for q, dO [B,Hq,Lq,D] and k, v [B,Hkv,Lk,D];
    dq, dk, dv are caller-allocated fp32 outputs."""
    B, Hq, Hkv, Lq, Lk, D = _dims_ex(q, k)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().swa_attn_bwd_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk),
                                _ptr(dv), B, Hq, Hkv, Lq, Lk, D, int(window), int(bool(causal)), float(scale),
                                _ptr(workspace), nbytes, _stream_ptr(stream))
    if rc:
        raise SwaError(rc, "swa_attn_bwd_ex")


def swa_attn_fwd_sinks(q, k, v, sinks, o, lse, window: int, causal: bool, scale: float, workspace=None,
                       stream=None) -> None:
    """swa_attn_fwd_ex with one sink logit per query head (sinks fp32 [Hq],
    CUDA; see include/swa_attn.h)."""
    B, Hq, Hkv, Lq, Lk, D = _dims_ex(q, k)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().swa_attn_fwd_sinks(_ptr(q), _ptr(k), _ptr(v), _ptr(sinks), _ptr(o), _ptr(lse), B, Hq, Hkv, Lq, Lk,
                                   D, int(window), int(bool(causal)), float(scale), _ptr(workspace), nbytes,
                                   _stream_ptr(stream))
    if rc:
        raise SwaError(rc, "swa_attn_fwd_sinks")


def swa_attn_bwd_sinks(q, k, v, sinks, o, lse, dO, dq, dk, dv, dsinks, window: int, causal: bool, scale: float,
                       workspace=None, stream=None) -> None:
    """Backward of swa_attn_fwd_sinks; dq, dk, dv and dsinks (fp32 [Hq]) are
    caller-allocated outputs."""
    B, Hq, Hkv, Lq, Lk, D = _dims_ex(q, k)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().swa_attn_bwd_sinks(_ptr(q), _ptr(k), _ptr(v), _ptr(sinks), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq),
                                   _ptr(dk), _ptr(dv), _ptr(dsinks), B, Hq, Hkv, Lq, Lk, D, int(window),
                                   int(bool(causal)), float(scale), _ptr(workspace), nbytes, _stream_ptr(stream))
    if rc:
        raise SwaError(rc, "swa_attn_bwd_sinks")


def fwd_workspace_bytes_prefix(B, Hq, Hkv, L, D, window, prompt_len, chosen_len) -> int:
    return int(load().swa_attn_fwd_workspace_bytes_prefix(B, Hq, Hkv, L, D, window, prompt_len, chosen_len))


def bwd_workspace_bytes_prefix(B, Hq, Hkv, L, D, window, prompt_len, chosen_len) -> int:
    return int(load().swa_attn_bwd_workspace_bytes_prefix(B, Hq, Hkv, L, D, window, prompt_len, chosen_len))


def swa_attn_fwd_prefix(q, k, v, o, lse, window: int, prompt_len: int, chosen_len: int, scale: float,
                        workspace=None, stream=None) -> None:
    """Forward over [prompt; chosen; rejected] with the shared-prefix mask
    (see include/swa_attn.h); q, k, v bf16 [B,H,L,D]; o, lse fp32 outputs."""
    B, Hq, Hkv, L, D = _dims(q, k)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().swa_attn_fwd_prefix(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, L, D, int(window),
                                    int(prompt_len), int(chosen_len), float(scale), _ptr(workspace), nbytes,
                                    _stream_ptr(stream))
    if rc:
        raise SwaError(rc, "swa_attn_fwd_prefix")


def swa_attn_bwd_prefix(q, k, v, o, lse, dO, dq, dk, dv, window: int, prompt_len: int, chosen_len: int,
                        scale: float, workspace=None, stream=None) -> None:
    """Backward of swa_attn_fwd_prefix; dq, dk, dv are caller-allocated fp32 outputs."""
    B, Hq, Hkv, L, D = _dims(q, k)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().swa_attn_bwd_prefix(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk),
                                    _ptr(dv), B, Hq, Hkv, L, D, int(window), int(prompt_len), int(chosen_len),
                                    float(scale), _ptr(workspace), nbytes, _stream_ptr(stream))
    if rc:
        raise SwaError(rc, "swa_attn_bwd_prefix")


def swa_attn_add_rows_f32(dst, src, row0: int, stream=None) -> None:
    """dst[:, :, row0 : row0 + n] += src through the C ABI, for fp32 CUDA
    tensors dst [B, H, dst_rows, D] and src [B, H, n, D] (contiguous)."""
    B, H, dst_rows, D = dst.shape
    n = src.shape[2]
    if tuple(src.shape) != (B, H, n, D) or not (dst.is_contiguous() and src.is_contiguous()):
        raise ValueError("src must be a contiguous [B, H, n, D] block of dst's heads")
    rc = load().swa_attn_add_rows_f32(_ptr(dst), _ptr(src), B * H, dst_rows, int(row0), n, D, _stream_ptr(stream))
    if rc:
        raise SwaError(rc, "swa_attn_add_rows_f32")


def swa_attn_fwd(q, k, v, o, lse, window: int, scale: float, workspace=None, stream=None) -> None:
    """Forward through the C ABI.  q,k,v: bf16 CUDA tensors [B,H,L,D]; o fp32
    [B,Hq,L,D] and lse fp32 [B,Hq,L] are caller-allocated outputs."""
    B, Hq, Hkv, L, D = _dims(q, k)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().swa_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, L, D, int(window),
                             float(scale), _ptr(workspace), nbytes, _stream_ptr(stream))
    if rc:
        raise SwaError(rc, "swa_attn_fwd")


def swa_attn_bwd(q, k, v, o, lse, dO, dq, dk, dv, window: int, scale: float, workspace=None, stream=None) -> None:
    """Backward through the C ABI; dq, dk, dv are caller-allocated fp32 outputs."""
    B, Hq, Hkv, L, D = _dims(q, k)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().swa_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk),
                             _ptr(dv), B, Hq, Hkv, L, D, int(window), float(scale), _ptr(workspace), nbytes,
                             _stream_ptr(stream))
    if rc:
        raise SwaError(rc, "swa_attn_bwd")


def swa_attn_bwd_noalloc(q, k, v, o, lse, dO, dq, dk, dv, window: int, scale: float, stream=None) -> None:
    """Backward without a workspace (fixed built-in scratch; see include/swa_attn.h)."""
    B, Hq, Hkv, L, D = _dims(q, k)
    rc = load().swa_attn_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk),
                                     _ptr(dv), B, Hq, Hkv, L, D, int(window), float(scale), _stream_ptr(stream))
    if rc:
        raise SwaError(rc, "swa_attn_bwd_noalloc")


def swa_attn_selftest_timeout(stream=None) -> None:
    """Launch the device-side timeout self-test (see include/swa_attn.h)."""
    rc = load().swa_attn_selftest_timeout(_stream_ptr(stream))
    if rc:
        raise SwaError(rc, "swa_attn_selftest_timeout")


def swa_attn_get_status(stream=None) -> int:
    return int(load().swa_attn_get_status(_stream_ptr(stream)))


# ---------------------------------------------------------------------------
# convenience wrappers: allocate outputs / workspace with torch, call the ABI


def _workspace(nbytes, device):
    import torch

    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def forward(q, k, v, window: int, scale: float, stream=None, causal: bool = True, prefix=None, sinks=None):
    """Return (o fp32, lse fp32) for bf16 CUDA tensors q [B,Hq,Lq,D], k/v
    [B,Hkv,Lk,D] (Lq <= Lk; Lq = Lk and causal is self-attention).
    prefix=(prompt_len, chosen_len): the shared-prefix mask over one
    [prompt; chosen; rejected] sequence (self-attention, causal).
    sinks: fp32 CUDA tensor [Hq], one sink logit per query head."""
    import torch

    B, Hq, Hkv, Lq, Lk, D = _dims_ex(q, k)
    o = torch.empty((B, Hq, Lq, D), dtype=torch.float32, device=q.device)
    lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device)
    if sinks is not None:
        if prefix is not None:
            raise ValueError("sinks are not combined with a shared-prefix plan")
        ws = _workspace(fwd_workspace_bytes_ex(B, Hq, Hkv, Lq, Lk, D, window, causal), q.device)
        swa_attn_fwd_sinks(q, k, v, sinks, o, lse, window, causal, scale, ws, stream)
    elif prefix is not None:
        ws = _workspace(fwd_workspace_bytes_prefix(B, Hq, Hkv, Lk, D, window, *prefix), q.device)
        swa_attn_fwd_prefix(q, k, v, o, lse, window, prefix[0], prefix[1], scale, ws, stream)
    elif Lq == Lk and causal:
        ws = _workspace(fwd_workspace_bytes(B, Hq, Hkv, Lk, D, window), q.device)
        swa_attn_fwd(q, k, v, o, lse, window, scale, ws, stream)
    else:
        ws = _workspace(fwd_workspace_bytes_ex(B, Hq, Hkv, Lq, Lk, D, window, causal), q.device)
        swa_attn_fwd_ex(q, k, v, o, lse, window, causal, scale, ws, stream)
    return o, lse


def backward(q, k, v, o, lse, dO, window: int, scale: float, stream=None, causal: bool = True, prefix=None,
             sinks=None):
    """Return (dq, dk, dv) fp32, and dsinks [Hq] too when sinks are given."""
    import torch

    B, Hq, Hkv, Lq, Lk, D = _dims_ex(q, k)
    dq = torch.empty((B, Hq, Lq, D), dtype=torch.float32, device=q.device)
    dk = torch.empty((B, Hkv, Lk, D), dtype=torch.float32, device=q.device)
    dv = torch.empty((B, Hkv, Lk, D), dtype=torch.float32, device=q.device)
    if sinks is not None:
        if prefix is not None:
            raise ValueError("sinks are not combined with a shared-prefix plan")
        dsinks = torch.empty((Hq,), dtype=torch.float32, device=q.device)
        ws = _workspace(bwd_workspace_bytes_ex(B, Hq, Hkv, Lq, Lk, D, window, causal), q.device)
        swa_attn_bwd_sinks(q, k, v, sinks, o, lse, dO, dq, dk, dv, dsinks, window, causal, scale, ws, stream)
        return dq, dk, dv, dsinks
    if prefix is not None:
        ws = _workspace(bwd_workspace_bytes_prefix(B, Hq, Hkv, Lk, D, window, *prefix), q.device)
        swa_attn_bwd_prefix(q, k, v, o, lse, dO, dq, dk, dv, window, prefix[0], prefix[1], scale, ws, stream)
    elif Lq == Lk and causal:
        ws = _workspace(bwd_workspace_bytes(B, Hq, Hkv, Lk, D, window), q.device)
        swa_attn_bwd(q, k, v, o, lse, dO, dq, dk, dv, window, scale, ws, stream)
    else:
        ws = _workspace(bwd_workspace_bytes_ex(B, Hq, Hkv, Lq, Lk, D, window, causal), q.device)
        swa_attn_bwd_ex(q, k, v, o, lse, dO, dq, dk, dv, window, causal, scale, ws, stream)
    return dq, dk, dv


# ---------------------------------------------------------------------------
# attention over a shared prefix and per-request caches; per-head norm and rotation
#
# A generation step calls these with tensors of a few KB, where the host's
# time is what counts: the calls that allocate their outputs go through
# csrc/marshal.cpp, which returns None for anything unusual; the path below then
# runs the call or says what is wrong with it.  Its checks are one pass over
# (name, tensor, type, shape), and workspace sizes are remembered by shape.


_fast = None  # csrc/marshal.cpp, once a call needs it


def _marshal():
    """The marshalling module, bound to the library that load() returned."""
    global _fast
    lib = load()
    with _lock:
        if _fast is None:
            import torch  # its libraries are the module's

            try:
                from . import _marshal as m
            except ImportError as e:
                raise RuntimeError("the binding's marshalling module is missing: build the CUDA library first "
                                   "(python -c 'import __graft_entry__ as g; g.build()')") from e
            m.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
                lib.swa_attn_fwd_workspace_bytes_shared, lib.swa_attn_fwd_shared, lib.swa_attn_qk_rope_fwd,
                lib.swa_attn_qk_rope_bwd_workspace_bytes, lib.swa_attn_qk_rope_bwd)), torch.OutOfMemoryError)
            _fast = m
        return _fast


def _check(device, specs):
    """Every tensor dense, on `device` (an index) and of its type and shape."""
    for name, t, dtype, shape in specs:
        if t is None:
            raise ValueError(f"{name} is missing: a {dtype} tensor of shape {tuple(shape)} is needed")
        if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, "
                             f"got {t.dtype} {tuple(t.shape)}{'' if t.is_contiguous() else ' (strided)'}")
        if t.get_device() != device:
            raise ValueError(f"{name} must be on the current CUDA device, like the other tensors (got {t.device})")


def _scratch_bytes(workspace, device) -> int:
    """Bytes of a caller's workspace on `device` (an index); none (0) is for the library to refuse."""
    if workspace is None:
        return 0
    if not workspace.is_contiguous() or workspace.get_device() != device:
        raise ValueError(f"workspace must be contiguous and on the current CUDA device, got {tuple(workspace.shape)} "
                         f"strides {workspace.stride()} on {workspace.device}")
    return workspace.numel() * workspace.element_size()


def _int32(name, v) -> int:
    """v as the int of a C argument (ctypes drops the bits above 32)."""
    v = int(v)
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{name} does not fit 32 bits: {v}")
    return v


def _current_device(t, name):
    import torch

    if not t.is_cuda or t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} must be on the current CUDA device (got {t.device})")
    return t.get_device()


@functools.lru_cache(maxsize=256)
def fwd_workspace_bytes_shared(B, Hq, Hkv, Lq, prefix_len, own_rows, D, window) -> int:
    return int(load().swa_attn_fwd_workspace_bytes_shared(B, Hq, Hkv, Lq, prefix_len, own_rows, D, window))


def _check_shared(q, k_prefix, v_prefix, k_own, v_own, own_len, sinks):
    import torch

    B, Hq, Lq, D = q.shape
    _, Hkv, own_rows, _ = k_own.shape
    if (k_prefix is None) != (v_prefix is None):
        raise ValueError("k_prefix and v_prefix are given together, or neither")
    prefix_rows = 0 if k_prefix is None else k_prefix.shape[1]
    dev, bf16 = _current_device(q, "q"), torch.bfloat16
    prefix, own = (Hkv, prefix_rows, D), (B, Hkv, own_rows, D)
    _check(dev, (("q", q, bf16, (B, Hq, Lq, D)), ("k_own", k_own, bf16, own), ("v_own", v_own, bf16, own),
                 ("own_len", own_len, torch.int32, (B,))))
    if k_prefix is not None:
        _check(dev, (("k_prefix", k_prefix, bf16, prefix), ("v_prefix", v_prefix, bf16, prefix)))
    if sinks is not None:
        _check(dev, (("sinks", sinks, torch.float32, (Hq,)),))
    return dev, B, Hq, Hkv, Lq, D, prefix_rows, own_rows


def _run_shared(dims, q, k_prefix, v_prefix, k_own, v_own, own_len, sinks, o, lse, window, scale, P, ws, nbytes,
                stream):
    _, B, Hq, Hkv, Lq, D, prefix_rows, own_rows = dims
    rc = load().swa_attn_fwd_shared(q.data_ptr(), _addr(k_prefix), _addr(v_prefix), k_own.data_ptr(),
                                    v_own.data_ptr(), own_len.data_ptr(), None if sinks is None else sinks.data_ptr(),
                                    o.data_ptr(), lse.data_ptr(), B, Hq, Hkv, Lq, P, prefix_rows, own_rows, D, window,
                                    scale, None if ws is None else ws.data_ptr(), nbytes, _stream_ptr(stream))
    if rc:
        raise SwaError(rc, "swa_attn_fwd_shared")


def swa_attn_fwd_shared(q, k_prefix, v_prefix, k_own, v_own, own_len, sinks, o, lse, window: int, scale: float,
                        prefix_len=None, workspace=None, stream=None) -> None:
    """Attention of a generation step over a prefix shared by the batch and
    each request's own cache (see include/swa_attn.h).  q bf16 [B,Hq,Lq,D];
    k_prefix, v_prefix bf16 [Hkv,prefix_rows,D] (prefix_len of the rows, all
    by default) or None for no prefix; k_own, v_own bf16 [B,Hkv,own_rows,D]; own_len int32 [B];
    sinks fp32 [Hq] or None; o bf16 like q and lse fp32 [B,Hq,Lq] are
    caller-allocated outputs."""
    import torch

    dims = _check_shared(q, k_prefix, v_prefix, k_own, v_own, own_len, sinks)
    _check(dims[0], (("o", o, torch.bfloat16, q.shape), ("lse", lse, torch.float32, q.shape[:3])))
    P = dims[6] if prefix_len is None else _int32("prefix_len", prefix_len)
    nbytes = _scratch_bytes(workspace, dims[0])
    _run_shared(dims, q, k_prefix, v_prefix, k_own, v_own, own_len, sinks, o, lse, _int32("window", window),
                float(scale), P, workspace, nbytes, stream)


def forward_shared(q, k_prefix, v_prefix, k_own, v_own, own_len, window: int, scale: float, prefix_len=None,
                   sinks=None, stream=None):
    """Return (o bf16 [B,Hq,Lq,D], lse fp32 [B,Hq,Lq]) of swa_attn_fwd_shared,
    allocated on the stream that the call runs on."""
    if stream is not None:
        import torch

        with torch.cuda.stream(stream):
            return forward_shared(q, k_prefix, v_prefix, k_own, v_own, own_len, window, scale, prefix_len, sinks)
    r = (_fast or _marshal()).forward_shared(q, k_prefix, v_prefix, k_own, v_own, own_len, window, scale, prefix_len,
                                             sinks)
    if r.__class__ is tuple:
        return r
    if r is not None:
        raise SwaError(r, "swa_attn_fwd_shared")
    import torch

    dims = _check_shared(q, k_prefix, v_prefix, k_own, v_own, own_len, sinks)
    dev, B, Hq, Hkv, Lq, D, prefix_rows, own_rows = dims
    P = prefix_rows if prefix_len is None else _int32("prefix_len", prefix_len)
    window = _int32("window", window)
    nbytes = fwd_workspace_bytes_shared(B, Hq, Hkv, Lq, P, own_rows, D, window)
    device = q.device
    o = torch.empty_like(q)
    lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=device)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    _run_shared(dims, q, k_prefix, v_prefix, k_own, v_own, own_len, sinks, o, lse, window, float(scale), P, ws,
                nbytes, None)
    return o, lse


def _token_rows(name, t, B, L, D, device):
    """(heads, elements between tokens) of a bf16 [B, L, H, D] tensor whose
    heads are dense within a token (a fused projection's slice)."""
    import torch

    shape = t.shape
    if t.dtype is not torch.bfloat16 or len(shape) != 4 or shape[0] != B or shape[1] != L or shape[3] != D:
        raise ValueError(f"{name} must be a bf16 tensor [{B}, {L}, heads, {D}], got {t.dtype} {tuple(shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on the current CUDA device, like the other tensors (got {t.device})")
    H = shape[2]
    sb, sl, sh, sd = t.stride()
    tok = sl if L > 1 else (sb if B > 1 else H * D)
    if sd != 1 or (H > 1 and sh != D) or (B > 1 and L > 1 and sb != L * sl) or tok < H * D or tok % 8:
        raise ValueError(f"{name} must hold each token's heads densely, with one stride (a multiple of 8 elements) "
                         f"between tokens; got strides {t.stride()} of shape {tuple(shape)}")
    return H, tok


def _rope_common(q, wq, wk, inv_freq, positions):
    import torch

    if q.dim() != 4:
        raise ValueError("q must be [B, L, heads, D]")
    dev = _current_device(q, "q")
    B, L, _, D = q.shape
    f32 = torch.float32
    _check(dev, [s for s in (("wq", wq, f32, (D,)), ("wk", wk, f32, (D,)),
                             ("inv_freq", inv_freq, torch.float64, None if inv_freq is None else inv_freq.shape[:1]),
                             ("positions", positions, torch.int32, (B, L))) if s[1] is not None])
    return dev, B, L, D, 0 if inv_freq is None else 2 * inv_freq.shape[0]


def _addr(t):
    return None if t is None else t.data_ptr()


def swa_attn_qk_rope_fwd(q, k, v, wq, wk, inv_freq, q_out, k_out, v_out, eps: float, positions=None, kv_len=None,
                         pos0: int = 0, weight_offset: float = 0.0, interleaved: bool = False, stream=None) -> None:
    """Per-head RMS norm, scale and rotation of q and k, and the layout change
    of v, through the C ABI (see include/swa_attn.h).  q, k, v: bf16
    [B,L,heads,D] (slices of a fused projection, or dense); k, v may be None.
    wq, wk fp32 [D] or None; inv_freq fp64 [rot_dim / 2] or None;
    q_out bf16 [B,Hq,L,D], k_out and v_out bf16 [B,Hkv,kv_rows,D]."""
    import torch

    dev, B, L, D, rot = _rope_common(q, wq, wk, inv_freq, positions)
    bf16 = torch.bfloat16
    Hq, q_tok = _token_rows("q", q, B, L, D, dev)
    outs = [("q_out", q_out, bf16, (B, Hq, L, D))]
    Hkv, k_tok, v_tok, rows = 1, 0, 0, L
    if (k is not None and k_out is None) or (v is not None and v_out is None):
        raise ValueError("k needs k_out and v needs v_out")
    if k is not None:
        Hkv, k_tok = _token_rows("k", k, B, L, D, dev)
        rows = k_out.shape[2]
        outs.append(("k_out", k_out, bf16, (B, Hkv, rows, D)))
    if v is not None:
        Hv, v_tok = _token_rows("v", v, B, L, D, dev)
        if k is not None and Hv != Hkv:
            raise ValueError(f"k has {Hkv} heads and v has {Hv}")
        Hkv = Hv
        rows = v_out.shape[2] if k is None else rows
        outs.append(("v_out", v_out, bf16, (B, Hkv, rows, D)))
    if kv_len is not None:
        outs.append(("kv_len", kv_len, torch.int32, (B,)))
    _check(dev, outs)
    rc = load().swa_attn_qk_rope_fwd(q.data_ptr(), _addr(k), _addr(v), q_tok, k_tok, v_tok, _addr(wq), _addr(wk),
                                     _addr(inv_freq), _addr(positions), _addr(kv_len), q_out.data_ptr(),
                                     None if k is None else k_out.data_ptr(), None if v is None else v_out.data_ptr(),
                                     B, Hq, Hkv, L, D, rows, rot, 1 if interleaved else 0, _int32("pos0", pos0),
                                     float(eps), float(weight_offset), _stream_ptr(stream))
    if rc:
        raise SwaError(rc, "swa_attn_qk_rope_fwd")


def qk_rope(q, k, v, wq, wk, inv_freq, eps: float, positions=None, pos0: int = 0, weight_offset: float = 0.0,
            interleaved: bool = False, stream=None):
    """Return (q [B,Hq,L,D], k [B,Hkv,L,D], v [B,Hkv,L,D]) for the attention
    from a projection's bf16 q, k, v [B,L,heads,D]: q and k normalised per
    head, scaled and rotated by position.  k and v may be None."""
    if stream is not None:
        import torch

        with torch.cuda.stream(stream):
            return qk_rope(q, k, v, wq, wk, inv_freq, eps, positions, pos0, weight_offset, interleaved)
    r = (_fast or _marshal()).qk_rope(q, k, v, wq, wk, inv_freq, None, None, None, eps, positions, pos0,
                                      weight_offset, interleaved)
    if r.__class__ is tuple:
        return r
    if r is not None:
        raise SwaError(r, "swa_attn_qk_rope_fwd")
    import torch

    B, L, _, D = q.shape
    dtype, device = q.dtype, q.device
    out = [None if t is None else torch.empty((B, t.shape[2], L, D), dtype=dtype, device=device) for t in (q, k, v)]
    swa_attn_qk_rope_fwd(q, k, v, wq, wk, inv_freq, *out, eps, positions, None, pos0, weight_offset, interleaved)
    return tuple(out)


def qk_rope_append(q, k, v, wq, wk, inv_freq, k_cache, v_cache, kv_len, eps: float, positions=None, pos0: int = 0,
                   weight_offset: float = 0.0, interleaved: bool = False, stream=None):
    """The same for a generation step: k and v go into rows kv_len[b] - L ..
    kv_len[b] - 1 of each request's cache [B,Hkv,kv_rows,D] (kv_len int32 [B]
    counts the step's tokens), which also give their positions, from pos0.
    Return q [B,Hq,L,D]."""
    if kv_len is None:
        raise ValueError("qk_rope_append needs kv_len, the lengths of the caches that it appends to")
    if stream is not None:
        import torch

        with torch.cuda.stream(stream):
            return qk_rope_append(q, k, v, wq, wk, inv_freq, k_cache, v_cache, kv_len, eps, positions, pos0,
                                  weight_offset, interleaved)
    r = (_fast or _marshal()).qk_rope(q, k, v, wq, wk, inv_freq, k_cache, v_cache, kv_len, eps, positions, pos0,
                                      weight_offset, interleaved)
    if r.__class__ is tuple:
        return r[0]
    if r is not None:
        raise SwaError(r, "swa_attn_qk_rope_fwd")
    import torch

    B, L, Hq, D = q.shape
    q_out = torch.empty((B, Hq, L, D), dtype=q.dtype, device=q.device)
    swa_attn_qk_rope_fwd(q, k, v, wq, wk, inv_freq, q_out, k_cache, v_cache, eps, positions, kv_len, pos0,
                         weight_offset, interleaved)
    return q_out


@functools.lru_cache(maxsize=256)
def qk_rope_bwd_workspace_bytes(B, L, D) -> int:
    return int(load().swa_attn_qk_rope_bwd_workspace_bytes(B, L, D))


def _check_rope_bwd(q, k, wq, wk, inv_freq, dq, dk, dv, positions):
    import torch

    dev, B, L, D, rot = _rope_common(q, wq, wk, inv_freq, positions)
    f32 = torch.float32
    Hq, q_tok = _token_rows("q", q, B, L, D, dev)
    grads = [("dq", dq, f32, (B, Hq, L, D))]
    Hkv, k_tok = 1, 0
    if k is not None:
        Hkv, k_tok = _token_rows("k", k, B, L, D, dev)
        grads.append(("dk", dk, f32, (B, Hkv, L, D)))
    if dv is not None:
        Hkv = dv.shape[1] if k is None else Hkv
        grads.append(("dv", dv, f32, (B, Hkv, L, D)))
    _check(dev, grads)
    return dev, B, L, D, rot, Hq, Hkv, q_tok, k_tok


def _run_rope_bwd(dims, q, k, wq, wk, inv_freq, dq, dk, dv, outs, toks, dwq, dwk, eps, positions, pos0,
                  weight_offset, interleaved, ws, nbytes, stream):
    """outs, toks: addresses of the q, k and v gradients' first rows and the elements between their tokens."""
    _, B, L, D, rot, Hq, Hkv, q_tok, k_tok = dims
    rc = load().swa_attn_qk_rope_bwd(q.data_ptr(), _addr(k), q_tok, k_tok, _addr(wq), _addr(wk), _addr(inv_freq),
                                     _addr(positions), dq.data_ptr(), None if k is None else dk.data_ptr(), _addr(dv),
                                     *outs, *toks, _addr(dwq), _addr(dwk), B, Hq, Hkv, L, D, rot,
                                     1 if interleaved else 0, _int32("pos0", pos0), float(eps), float(weight_offset),
                                     _addr(ws), nbytes, _stream_ptr(stream))
    if rc:
        raise SwaError(rc, "swa_attn_qk_rope_bwd")


def swa_attn_qk_rope_bwd(q, k, wq, wk, inv_freq, dq, dk, dv, dq_in, dk_in, dv_in, dwq, dwk, eps: float,
                         positions=None, pos0: int = 0, weight_offset: float = 0.0, interleaved: bool = False,
                         workspace=None, stream=None) -> None:
    """Backward of swa_attn_qk_rope_fwd (without kv_len): fp32 dq [B,Hq,L,D],
    dk, dv [B,Hkv,L,D] to bf16 dq_in, dk_in, dv_in [B,L,heads,D] (which may be
    slices of a fused buffer) and fp32 dwq, dwk [D] (None: not wanted)."""
    import torch

    dims = _check_rope_bwd(q, k, wq, wk, inv_freq, dq, dk, dv, positions)
    dev, B, L, D, _, Hq, Hkv, _, _ = dims
    outs, toks = [], []
    for name, t, H in (("dq_in", dq_in, Hq), ("dk_in", None if k is None else dk_in, Hkv),
                       ("dv_in", None if dv is None else dv_in, Hkv)):
        heads, tok = (H, 0) if t is None else _token_rows(name, t, B, L, D, dev)
        if heads != H:
            raise ValueError(f"{name} must have {H} heads, got {heads}")
        outs.append(_addr(t))
        toks.append(tok)
    _check(dev, [(n, w, torch.float32, (D,)) for n, w in (("dwq", dwq), ("dwk", dwk)) if w is not None])
    nbytes = _scratch_bytes(workspace, dev)
    _run_rope_bwd(dims, q, k, wq, wk, inv_freq, dq, dk, dv, outs, toks, dwq, dwk, eps, positions, pos0,
                  weight_offset, interleaved, workspace, nbytes, stream)


def qk_rope_backward(q, k, wq, wk, inv_freq, dq, dk, dv, eps: float, positions=None, pos0: int = 0,
                     weight_offset: float = 0.0, interleaved: bool = False, stream=None):
    """Return (d, dwq, dwk): d bf16 [B,L,Hq + Hkv + Hkv,D] is the gradient of
    the fused projection output (q, k and v heads in that order; the k or v
    part is left out with k or dv None), dwq and dwk fp32 [D] (None for a
    None weight)."""
    if stream is not None:
        import torch

        with torch.cuda.stream(stream):
            return qk_rope_backward(q, k, wq, wk, inv_freq, dq, dk, dv, eps, positions, pos0, weight_offset,
                                    interleaved)
    r = (_fast or _marshal()).qk_rope_backward(q, k, wq, wk, inv_freq, dq, dk, dv, eps, positions, pos0,
                                               weight_offset, interleaved)
    if r.__class__ is tuple:
        return r
    if r is not None:
        raise SwaError(r, "swa_attn_qk_rope_bwd")
    import torch

    dims = _check_rope_bwd(q, k, wq, wk, inv_freq, dq, dk, dv, positions)
    _, B, L, D, _, Hq, Hkv, _, _ = dims
    device = q.device
    Hk, Hv = (0 if k is None else Hkv), (0 if dv is None else Hkv)
    H = Hq + Hk + Hv
    d = torch.empty((B, L, H, D), dtype=torch.bfloat16, device=device)
    dwq = None if wq is None else torch.empty_like(wq)
    dwk = None if wk is None or k is None else torch.empty_like(wk)
    nbytes = qk_rope_bwd_workspace_bytes(B, L, D)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    at, row = d.data_ptr(), 2 * D  # bytes of a head's row
    outs = (at, at + Hq * row if Hk else None, at + (Hq + Hk) * row if Hv else None)
    _run_rope_bwd(dims, q, k, wq, wk, inv_freq, dq, dk, dv, outs, (H * D,) * 3, dwq, dwk, eps, positions, pos0,
                  weight_offset, interleaved, ws, nbytes, None)
    return d, dwq, dwk


def prefix_positions(B: int, L: int, prompt_len: int, chosen_len: int, device):
    """Positions int32 [B, L] of a shared-prefix sequence [prompt; chosen;
    rejected]: the rejected response starts again behind the prompt, as the
    window of swa_attn_fwd_prefix measures it."""
    import torch

    if prompt_len < 0 or chosen_len < 0 or prompt_len + chosen_len > L:
        raise ValueError("a shared-prefix sequence needs prompt_len >= 0, chosen_len >= 0 and prompt_len + chosen_len <= L, "
                         f"got {prompt_len}, {chosen_len}, {L}")
    p = torch.arange(L, dtype=torch.int32, device=device)
    if chosen_len > 0:
        p[prompt_len + chosen_len:] -= chosen_len
    return p.expand(B, L).contiguous()
