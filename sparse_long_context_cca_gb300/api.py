"""Thin Python binding of libcca.so (include/cca.h), argument marshalling only.

Every step of the computation runs in the library's CUDA kernels; this module
allocates outputs with torch (device memory is plumbing), checks that tensors
match the C ABI's layout, and forwards raw device pointers.  There is no
fallback: if the library is missing or a call fails, an exception is raised.

The rotary, paged and packed calls, of which a step makes many, are checked and
marshalled by the extension module _binding (csrc/binding.cpp), bound to the same
library.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

CCA_OK = 0
CCA_ERR_INVALID_ARG = -1
CCA_ERR_UNSUPPORTED = -2
CCA_ERR_CUDA = -3
CCA_ERR_TIMEOUT = -4
CCA_ERR_SCRATCH_LIMIT = -5
CCA_ERR_NO_PAGES = -6
CCA_BF16 = 0
CCA_F32 = 1

_DTYPE = {torch.bfloat16: CCA_BF16, torch.float32: CCA_F32}


class CcaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


class CcaParams(ctypes.Structure):
    """Mirror of cca_params_t."""
    _fields_ = [("B", ctypes.c_int32), ("Hq", ctypes.c_int32), ("Hkv", ctypes.c_int32),
                ("N", ctypes.c_int32), ("d", ctypes.c_int32), ("g", ctypes.c_int32),
                ("w", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("dev_status", ctypes.c_void_p), ("window_mode", ctypes.c_int32),
                ("pool_mode", ctypes.c_int32)]


class CcaRopeParams(ctypes.Structure):
    """Mirror of cca_rope_params_t."""
    _fields_ = [("B", ctypes.c_int32), ("N", ctypes.c_int32), ("d", ctypes.c_int32), ("rot", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("dtype", ctypes.c_int32), ("inverse", ctypes.c_int32),
                ("factor", ctypes.c_float), ("inv_freq", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("pos_stride", ctypes.c_int64), ("start", ctypes.c_int64)]


class CcaRopeTensor(ctypes.Structure):
    """Mirror of cca_rope_tensor_t."""
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("H", ctypes.c_int32),
                ("x_stride", ctypes.c_int64 * 3), ("y_stride", ctypes.c_int64 * 3)]


class CcaNormTensor(ctypes.Structure):
    """Mirror of cca_norm_tensor_t."""
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("dy", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("dweight", ctypes.c_void_p), ("H", ctypes.c_int32), ("weight_heads", ctypes.c_int32),
                ("x_stride", ctypes.c_int64 * 3), ("y_stride", ctypes.c_int64 * 3), ("dy_stride", ctypes.c_int64 * 3)]


class CcaNormParams(ctypes.Structure):
    """Mirror of cca_norm_params_t."""
    _fields_ = [("rope", CcaRopeParams), ("eps", ctypes.c_float), ("offset", ctypes.c_float),
                ("weight_dtype", ctypes.c_int32)]


class CcaPacked(ctypes.Structure):
    """Mirror of cca_packed_t."""
    _fields_ = [("plan", ctypes.c_void_p), ("plan_bytes", ctypes.c_uint64), ("S", ctypes.c_int32), ("T", ctypes.c_int32),
                ("g", ctypes.c_int32), ("w", ctypes.c_int32), ("window_mode", ctypes.c_int32)]


class CcaPackedRows(ctypes.Structure):
    """Mirror of cca_packed_rows_t."""
    _fields_ = [("p", ctypes.c_void_p), ("head_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64)]


class CcaPages(ctypes.Structure):
    """Mirror of cca_pages_t."""
    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("n_pages", ctypes.c_int32), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("layers", ctypes.c_int32)]


_lib = None
_fast = None    # the _binding module, bound to the library
_lock = threading.Lock()

EXPORTED = ["cca_pool", "cca_attn_fwd", "cca_attn_fwd_rows", "cca_decode_fwd", "cca_decode_workspace_size",
            "cca_decode_kernels", "cca_pool_group",
            "cca_decode_fwd_noalloc", "cca_prefill_bwd", "cca_prefill_bwd_workspace_size",
            "cca_prefill_host", "cca_prefill_host_workspace_size",
            "cca_rope", "cca_rope_append", "cca_tree_fwd", "cca_tree_workspace_size", "cca_pool_pages",
            "cca_pages_reserve", "cca_pages_reserve_workspace_size", "cca_pages_fork", "cca_pages_free",
            "cca_pages_copy", "cca_pages_compact",
            "cca_norm_rope", "cca_norm_rope_bwd", "cca_norm_rope_bwd_workspace_size", "cca_norm_rope_append",
            "cca_pack", "cca_pack_size", "cca_pack_positions_offset", "cca_pool_packed", "cca_attn_packed",
            "cca_packed_clear",
            "cca_packed_bwd", "cca_packed_bwd_workspace_size",
            "cca_status_string", "cca_abi_version", "cca_test_set_wait_limit_ns", "cca_test_skip_q_load",
            "cca_test_decode_path"]


def library_path() -> str:
    return os.environ.get("CCA_LIBRARY", _build.LIB)


def load_library():
    """Load libcca.so; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"libcca.so not found at {path}: build it first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        lib = ctypes.CDLL(path)
        vp = ctypes.c_void_p
        pp = ctypes.POINTER(CcaParams)
        lib.cca_pool.argtypes = [vp, vp, vp, vp, vp, pp, vp]
        lib.cca_pool.restype = ctypes.c_int
        lib.cca_attn_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, pp, vp]
        lib.cca_attn_fwd.restype = ctypes.c_int
        ci = ctypes.c_int
        lib.cca_attn_fwd_rows.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, pp, vp]
        lib.cca_attn_fwd_rows.restype = ctypes.c_int
        lib.cca_decode_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, ctypes.c_int, pp, vp, ctypes.c_uint64, vp]
        lib.cca_decode_fwd.restype = ctypes.c_int
        lib.cca_decode_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, ctypes.c_int, pp, vp]
        lib.cca_decode_fwd_noalloc.restype = ctypes.c_int
        lib.cca_prefill_bwd.argtypes = [vp] * 11 + [pp, vp, ctypes.c_uint64, vp]
        lib.cca_prefill_bwd.restype = ctypes.c_int
        lib.cca_prefill_bwd_workspace_size.argtypes = [pp]
        lib.cca_prefill_bwd_workspace_size.restype = ctypes.c_uint64
        lib.cca_prefill_host.argtypes = [vp] * 7 + [pp, vp, ctypes.c_uint64, vp]
        lib.cca_prefill_host.restype = ctypes.c_int
        lib.cca_prefill_host_workspace_size.argtypes = [pp]
        lib.cca_prefill_host_workspace_size.restype = ctypes.c_uint64
        lib.cca_decode_kernels.argtypes = [pp, ctypes.c_int]
        lib.cca_decode_kernels.restype = ctypes.c_int
        lib.cca_decode_workspace_size.argtypes = [pp]
        lib.cca_decode_workspace_size.restype = ctypes.c_uint64
        lib.cca_pool_group.argtypes = [vp, vp, vp, vp, vp, ctypes.c_int, pp, vp]
        lib.cca_pool_group.restype = ctypes.c_int
        u64 = ctypes.c_uint64
        rp, rt, pg, nt, np_, pk, pr = (ctypes.POINTER(x) for x in (CcaRopeParams, CcaRopeTensor, CcaPages, CcaNormTensor,
                                                                  CcaNormParams, CcaPacked, CcaPackedRows))
        for name, args, res in (
                ("cca_rope", [rt, ci, rp, vp], ci),
                ("cca_rope_append", [rt, rt, rt, pg, vp, vp, vp, vp, rp, vp], ci),
                ("cca_tree_fwd", [vp, pg, pg, vp, vp, ci, vp, vp, pp, vp, u64, vp], ci),
                ("cca_tree_workspace_size", [pp, ci], u64),
                ("cca_pool_pages", [vp, pg, pg, vp, vp, vp, ci, ci, pp, vp], ci),
                ("cca_pages_reserve", [vp, ci, vp, ci, ci, ci, vp, vp, vp, vp, u64, vp, vp], ci),
                ("cca_pages_reserve_workspace_size", [ci, ci], u64),
                ("cca_pages_fork", [vp, ci, vp, ci, ci, ci, vp, vp, ci, vp, vp, vp], ci),
                ("cca_pages_free", [vp, ci, vp, ci, ci, vp, vp, vp, vp], ci),
                ("cca_pages_copy", [pg, vp, ci, pp, vp], ci),
                ("cca_pages_compact", [pg, vp, vp, ci, vp, pp, vp], ci),
                ("cca_norm_rope", [nt, ci, np_, vp], ci),
                ("cca_norm_rope_bwd", [nt, ci, np_, vp, u64, vp], ci),
                ("cca_norm_rope_bwd_workspace_size", [nt, ci, np_], u64),
                ("cca_norm_rope_append", [nt, nt, rt, pg, vp, vp, vp, vp, np_, vp], ci),
                ("cca_pack_size", [ci, ci, ci], u64),
                ("cca_pack_positions_offset", [ci, ci, ci], u64),
                ("cca_pack", [vp, pk, vp, vp], ci),
                ("cca_pool_packed", [pr, pr, pr, vp, vp, pk, pp, vp], ci),
                ("cca_attn_packed", [pr, pr, pr, vp, vp, pr, vp, pk, pp, vp], ci),
                ("cca_packed_clear", [pr, ctypes.POINTER(ctypes.c_int32), ci, pk, pp, vp], ci),
                ("cca_packed_bwd", [pr, pr, pr, vp, vp, pr, vp, pr, pr, pr, pr, pk, pp, vp, u64, vp], ci),
                ("cca_packed_bwd_workspace_size", [pk, pp], u64)):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, res
        lib.cca_status_string.argtypes = [ctypes.c_int]
        lib.cca_status_string.restype = ctypes.c_char_p
        lib.cca_abi_version.argtypes = []
        lib.cca_abi_version.restype = ctypes.c_int
        lib.cca_test_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
        lib.cca_test_set_wait_limit_ns.restype = None
        lib.cca_test_skip_q_load.argtypes = [ctypes.c_int]
        lib.cca_test_skip_q_load.restype = None
        lib.cca_test_decode_path.argtypes = [ctypes.c_int]
        lib.cca_test_decode_path.restype = None
        _lib = lib
        return lib


def _bound():
    """The binding of the rotary, paged and packed calls (the others do without it); raises if it has not been
    built, or for another torch."""
    global _fast
    lib = load_library()
    with _lock:
        if _fast is None:
            if not _build.binding_is_for_this_torch():
                raise RuntimeError(f"{_build.BINDING} is not there or was built for another torch or Python: build it first "
                                   "(python -c 'import __graft_entry__ as g; g.build()')")
            from . import _binding
            _binding.bind(CcaError, {n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value
                                     for n in EXPORTED if not n.startswith("cca_test")})
            _fast = _binding
        return _fast


def status_string(status: int) -> str:
    return load_library().cca_status_string(int(status)).decode()


def make_params(B, Hq, Hkv, N, d, g, w, dtype, scale=0.0, dev_status=None, window_mode=0,
                pool_mode=0) -> CcaParams:
    return CcaParams(int(B), int(Hq), int(Hkv), int(N), int(d), int(g), int(w), int(dtype),
                     float(scale), dev_status, int(window_mode), int(pool_mode))


def _stream_handle(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _check(t: torch.Tensor, name: str, dtype, shape):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _dims(Q, K):
    if Q.dim() != 4 or K.dim() != 4:
        raise ValueError("Q and K must be [B, H, N, d]")
    B, Hq, N, d = Q.shape
    Hkv = K.shape[1]
    return B, Hq, Hkv, N, d


def cca_pool(Q, K, V, g: int, Kc=None, Vc=None, scale: float = 0.0, stream=None, pool_mode: int = 0):
    """Global-aware pooling: returns (Kc, Vc), each [B, Hkv, N/g, d].
    pool_mode 0: softmax weights of the group-last query (GQA: the r heads' logits averaged);
    1: mean; 2: element-wise max; 3: GQA pooling averaged after the softmax (each query head's
    own softmax weights, averaged over the r heads sharing the KV head; r <= 8)."""
    lib = load_library()
    B, Hq, Hkv, N, d = _dims(Q, K)
    if Q.dtype not in _DTYPE:
        raise ValueError(f"unsupported dtype {Q.dtype}")
    _check(Q, "Q", Q.dtype, (B, Hq, N, d))
    _check(K, "K", Q.dtype, (B, Hkv, N, d))
    _check(V, "V", Q.dtype, (B, Hkv, N, d))
    G = N // g if g > 0 else 0
    if Kc is None:
        Kc = torch.empty((B, Hkv, G, d), dtype=Q.dtype, device=Q.device)
    if Vc is None:
        Vc = torch.empty((B, Hkv, G, d), dtype=Q.dtype, device=Q.device)
    _check(Kc, "Kc", Q.dtype, (B, Hkv, G, d))
    _check(Vc, "Vc", Q.dtype, (B, Hkv, G, d))
    prm = make_params(B, Hq, Hkv, N, d, g, 1, _DTYPE[Q.dtype], scale, pool_mode=pool_mode)
    st = lib.cca_pool(Q.data_ptr(), K.data_ptr(), V.data_ptr(), Kc.data_ptr(), Vc.data_ptr(),
                      ctypes.byref(prm), _stream_handle(stream))
    if st != CCA_OK:
        raise CcaError(st, "cca_pool")
    return Kc, Vc


def cca_attn_fwd(Q, K, V, Kc, Vc, g: int, w: int, O=None, LSE=None, scale: float = 0.0,
                 dev_status=None, stream=None, window_mode: int = 0):
    """Fused core/local attention: returns (O [B,Hq,N,d], LSE [B,Hq,N] fp32).
    window_mode 1: the raw window starts at the group boundary g*(lo(i)//g)."""
    lib = load_library()
    B, Hq, Hkv, N, d = _dims(Q, K)
    if Q.dtype not in _DTYPE:
        raise ValueError(f"unsupported dtype {Q.dtype}")
    G = N // g if g > 0 else 0
    _check(Q, "Q", Q.dtype, (B, Hq, N, d))
    _check(K, "K", Q.dtype, (B, Hkv, N, d))
    _check(V, "V", Q.dtype, (B, Hkv, N, d))
    _check(Kc, "Kc", Q.dtype, (B, Hkv, G, d))
    _check(Vc, "Vc", Q.dtype, (B, Hkv, G, d))
    if O is None:
        O = torch.empty_like(Q)
    if LSE is None:
        LSE = torch.empty((B, Hq, N), dtype=torch.float32, device=Q.device)
    _check(O, "O", Q.dtype, (B, Hq, N, d))
    _check(LSE, "LSE", torch.float32, (B, Hq, N))
    status_ptr = None
    if dev_status is not None:
        _check(dev_status, "dev_status", torch.int32, (1,))
        status_ptr = dev_status.data_ptr()
    prm = make_params(B, Hq, Hkv, N, d, g, w, _DTYPE[Q.dtype], scale, status_ptr, window_mode=window_mode)
    st = lib.cca_attn_fwd(Q.data_ptr(), K.data_ptr(), V.data_ptr(), Kc.data_ptr(), Vc.data_ptr(),
                          O.data_ptr(), LSE.data_ptr(), ctypes.byref(prm), _stream_handle(stream))
    if st != CCA_OK:
        raise CcaError(st, "cca_attn_fwd")
    return O, LSE


def cca_attn_fwd_rows(Q, K, V, Kc, Vc, g: int, w: int, N: int, q_off: int, kv_off: int, O=None, LSE=None,
                      scale: float = 0.0, dev_status=None, stream=None, window_mode: int = 0):
    """Fused attention for the query rows [q_off, q_off + n_q) of an N-token sequence.
    Q [B,Hq,n_q,d] holds those rows, K, V [B,Hkv,n_kv,d] the raw tokens from kv_off on,
    Kc, Vc [B,Hkv,N/g,d] the whole sequence's core tokens.  Returns (O [B,Hq,n_q,d],
    LSE [B,Hq,n_q] fp32), equal to rows q_off .. q_off + n_q - 1 of cca_attn_fwd over N."""
    lib = load_library()
    B, Hq, n_q, d = Q.shape
    Hkv, n_kv = K.shape[1], K.shape[2]
    if Q.dtype not in _DTYPE:
        raise ValueError(f"unsupported dtype {Q.dtype}")
    G = N // g if g > 0 else 0
    _check(Q, "Q", Q.dtype, (B, Hq, n_q, d))
    _check(K, "K", Q.dtype, (B, Hkv, n_kv, d))
    _check(V, "V", Q.dtype, (B, Hkv, n_kv, d))
    _check(Kc, "Kc", Q.dtype, (B, Hkv, G, d))
    _check(Vc, "Vc", Q.dtype, (B, Hkv, G, d))
    if O is None:
        O = torch.empty_like(Q)
    if LSE is None:
        LSE = torch.empty((B, Hq, n_q), dtype=torch.float32, device=Q.device)
    _check(O, "O", Q.dtype, (B, Hq, n_q, d))
    _check(LSE, "LSE", torch.float32, (B, Hq, n_q))
    status_ptr = None
    if dev_status is not None:
        _check(dev_status, "dev_status", torch.int32, (1,))
        status_ptr = dev_status.data_ptr()
    prm = make_params(B, Hq, Hkv, N, d, g, w, _DTYPE[Q.dtype], scale, status_ptr, window_mode=window_mode)
    st = lib.cca_attn_fwd_rows(Q.data_ptr(), K.data_ptr(), V.data_ptr(), Kc.data_ptr(), Vc.data_ptr(),
                               O.data_ptr(), LSE.data_ptr(), int(q_off), int(n_q), int(kv_off), int(n_kv),
                               ctypes.byref(prm), _stream_handle(stream))
    if st != CCA_OK:
        raise CcaError(st, "cca_attn_fwd_rows")
    return O, LSE


def cca_prefill(Q, K, V, g: int, w: int, scale: float = 0.0, out=None, stream=None, pool_mode: int = 0,
                window_mode: int = 0):
    """Both steps of CCA prefill: pooling, then fused attention.
    Returns (O, LSE, Kc, Vc).  `out` may hold preallocated (O, LSE, Kc, Vc)."""
    O = LSE = Kc = Vc = None
    if out is not None:
        O, LSE, Kc, Vc = out
    Kc, Vc = cca_pool(Q, K, V, g, Kc, Vc, scale, stream, pool_mode=pool_mode)
    O, LSE = cca_attn_fwd(Q, K, V, Kc, Vc, g, w, O, LSE, scale, None, stream, window_mode=window_mode)
    return O, LSE, Kc, Vc


def causal_attention(Q, K, V, scale: float = 0.0, O=None, LSE=None, stream=None):
    """Full causal softmax attention through the same fused kernel: with g = 1 every
    token is its own core and with w >= N no core is visible, so the visible set of
    query i is exactly tokens [0, i] (the closed form the oracle is pinned to).
    K and V serve as their own core tensors (shape [B, Hkv, N/1, d])."""
    N = Q.shape[2]
    return cca_attn_fwd(Q, K, V, K, V, 1, N, O, LSE, scale, None, stream)


def decode_workspace_size(B, Hq, Hkv, Ncap, d, g, w, dtype) -> int:
    prm = make_params(B, Hq, Hkv, Ncap, d, g, w, _DTYPE[dtype])
    return int(load_library().cca_decode_workspace_size(ctypes.byref(prm)))


def decode_kernels(B, Hq, Hkv, Ncap, d, g, w, dtype, pos: int, window_mode: int = 0) -> int:
    """Kernels one cca_decode_fwd call at `pos` launches on the current device (1 or 2)."""
    prm = make_params(B, Hq, Hkv, Ncap, d, g, w, _DTYPE[dtype], window_mode=window_mode)
    n = int(load_library().cca_decode_kernels(ctypes.byref(prm), int(pos)))
    if n < 0:
        raise CcaError(n, "cca_decode_kernels")
    return n


def cca_decode_fwd(q, K, V, Kc, Vc, pos: int, g: int, w: int, O=None, LSE=None, workspace=None,
                   scale: float = 0.0, stream=None, window_mode: int = 0):
    """One decoding step: row `pos` of the fused attention over the caches.
    q [B, Hq, d]; K, V [B, Hkv, Ncap, d]; Kc, Vc [B, Hkv, Ncap/g, d].
    Returns (O [B, Hq, d], LSE [B, Hq])."""
    lib = load_library()
    if q.dim() != 3 or K.dim() != 4:
        raise ValueError("q must be [B, Hq, d] and K [B, Hkv, Ncap, d]")
    B, Hq, d = q.shape
    Hkv, Ncap = K.shape[1], K.shape[2]
    if q.dtype not in _DTYPE:
        raise ValueError(f"unsupported dtype {q.dtype}")
    G = Ncap // g if g > 0 else 0
    _check(q, "q", q.dtype, (B, Hq, d))
    _check(K, "K", q.dtype, (B, Hkv, Ncap, d))
    _check(V, "V", q.dtype, (B, Hkv, Ncap, d))
    _check(Kc, "Kc", q.dtype, (B, Hkv, G, d))
    _check(Vc, "Vc", q.dtype, (B, Hkv, G, d))
    if O is None:
        O = torch.empty_like(q)
    if LSE is None:
        LSE = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    _check(O, "O", q.dtype, (B, Hq, d))
    _check(LSE, "LSE", torch.float32, (B, Hq))
    prm = make_params(B, Hq, Hkv, Ncap, d, g, w, _DTYPE[q.dtype], scale, window_mode=window_mode)
    need = int(lib.cca_decode_workspace_size(ctypes.byref(prm)))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if not workspace.is_cuda or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be a CUDA buffer of at least {need} bytes")
    st = lib.cca_decode_fwd(q.data_ptr(), K.data_ptr(), V.data_ptr(), Kc.data_ptr(), Vc.data_ptr(),
                            O.data_ptr(), LSE.data_ptr(), int(pos), ctypes.byref(prm), workspace.data_ptr(),
                            workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if st != CCA_OK:
        raise CcaError(st, "cca_decode_fwd")
    return O, LSE


def cca_pool_group(q, K, V, Kc, Vc, j: int, g: int, scale: float = 0.0, stream=None, pool_mode: int = 0):
    """Pool the newly completed group j of the caches in place (Kc[:, :, j], Vc[:, :, j]),
    scored by q [B, Hq, d], the query of the group's last token."""
    lib = load_library()
    B, Hq, d = q.shape
    Hkv, Ncap = K.shape[1], K.shape[2]
    G = Ncap // g if g > 0 else 0
    _check(q, "q", q.dtype, (B, Hq, d))
    _check(K, "K", q.dtype, (B, Hkv, Ncap, d))
    _check(V, "V", q.dtype, (B, Hkv, Ncap, d))
    _check(Kc, "Kc", q.dtype, (B, Hkv, G, d))
    _check(Vc, "Vc", q.dtype, (B, Hkv, G, d))
    prm = make_params(B, Hq, Hkv, Ncap, d, g, 1, _DTYPE[q.dtype], scale, pool_mode=pool_mode)
    st = lib.cca_pool_group(q.data_ptr(), K.data_ptr(), V.data_ptr(), Kc.data_ptr(), Vc.data_ptr(), int(j),
                            ctypes.byref(prm), _stream_handle(stream))
    if st != CCA_OK:
        raise CcaError(st, "cca_pool_group")
    return Kc, Vc


def cca_prefill_bwd(Q, K, V, Kc, Vc, O, LSE, dO, g: int, w: int, scale: float = 0.0, pool_mode: int = 0,
                    window_mode: int = 0, dQ=None, dK=None, dV=None, workspace=None, stream=None,
                    dev_status=None):
    """Gradients (dQ, dK, dV), fp32, of sum(dO * O) for CCA prefill (pooling + attention).
    dev_status: optional int32 CUDA tensor of one element that receives CCA_ERR_TIMEOUT
    if a tensor-core kernel gives up waiting."""
    lib = load_library()
    B, Hq, Hkv, N, d = _dims(Q, K)
    G = N // g if g > 0 else 0
    for name, t, shape in (("Q", Q, (B, Hq, N, d)), ("K", K, (B, Hkv, N, d)), ("V", V, (B, Hkv, N, d)),
                           ("Kc", Kc, (B, Hkv, G, d)), ("Vc", Vc, (B, Hkv, G, d)), ("O", O, (B, Hq, N, d)),
                           ("dO", dO, (B, Hq, N, d))):
        _check(t, name, Q.dtype, shape)
    _check(LSE, "LSE", torch.float32, (B, Hq, N))
    dQ = torch.empty((B, Hq, N, d), dtype=torch.float32, device=Q.device) if dQ is None else dQ
    dK = torch.empty((B, Hkv, N, d), dtype=torch.float32, device=Q.device) if dK is None else dK
    dV = torch.empty((B, Hkv, N, d), dtype=torch.float32, device=Q.device) if dV is None else dV
    _check(dQ, "dQ", torch.float32, (B, Hq, N, d))
    _check(dK, "dK", torch.float32, (B, Hkv, N, d))
    _check(dV, "dV", torch.float32, (B, Hkv, N, d))
    status_ptr = None
    if dev_status is not None:
        _check(dev_status, "dev_status", torch.int32, (1,))
        status_ptr = dev_status.data_ptr()
    prm = make_params(B, Hq, Hkv, N, d, g, w, _DTYPE[Q.dtype], scale, status_ptr, window_mode=window_mode,
                      pool_mode=pool_mode)
    need = int(lib.cca_prefill_bwd_workspace_size(ctypes.byref(prm)))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=Q.device)
    nbytes = workspace.numel() * workspace.element_size()
    st = lib.cca_prefill_bwd(Q.data_ptr(), K.data_ptr(), V.data_ptr(), Kc.data_ptr(), Vc.data_ptr(), O.data_ptr(),
                             LSE.data_ptr(), dO.data_ptr(), dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(),
                             ctypes.byref(prm), workspace.data_ptr(), nbytes, _stream_handle(stream))
    if st != CCA_OK:
        raise CcaError(st, "cca_prefill_bwd")
    return dQ, dK, dV


def _check_host(t: torch.Tensor, name: str, dtype, shape):
    if not isinstance(t, torch.Tensor) or t.device.type != "cpu":
        raise ValueError(f"{name} must be a CPU tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def prefill_host_workspace_size(B, Hq, Hkv, N, d, g, w, dtype) -> int:
    prm = make_params(B, Hq, Hkv, N, d, g, w, _DTYPE[dtype])
    return int(load_library().cca_prefill_host_workspace_size(ctypes.byref(prm)))


def cca_prefill_host(Q, K, V, g: int, w: int, scale: float = 0.0, out=None, with_lse: bool = True,
                     with_cores: bool = False, workspace=None, device=None, stream=None, pool_mode: int = 0,
                     window_mode: int = 0):
    """The prefill step on HOST tensors (pinned for overlap): the library copies Q, K, V in,
    pools, attends and copies the outputs back, pipelined over slices of KV heads.
    Returns (O, LSE or None, Kc or None, Vc or None) as CPU tensors; `out` may hold them
    preallocated.  The outputs are valid once `stream` has been synchronised."""
    lib = load_library()
    B, Hq, Hkv, N, d = _dims(Q, K)
    if Q.dtype not in _DTYPE:
        raise ValueError(f"unsupported dtype {Q.dtype}")
    G = N // g if g > 0 else 0
    _check_host(Q, "Q", Q.dtype, (B, Hq, N, d))
    _check_host(K, "K", Q.dtype, (B, Hkv, N, d))
    _check_host(V, "V", Q.dtype, (B, Hkv, N, d))
    pin = Q.is_pinned()
    if out is None:
        O = torch.empty((B, Hq, N, d), dtype=Q.dtype, pin_memory=pin)
        LSE = torch.empty((B, Hq, N), dtype=torch.float32, pin_memory=pin) if with_lse else None
        Kc = torch.empty((B, Hkv, G, d), dtype=Q.dtype, pin_memory=pin) if with_cores else None
        Vc = torch.empty((B, Hkv, G, d), dtype=Q.dtype, pin_memory=pin) if with_cores else None
    else:
        O, LSE, Kc, Vc = out
    _check_host(O, "O", Q.dtype, (B, Hq, N, d))
    if LSE is not None:
        _check_host(LSE, "LSE", torch.float32, (B, Hq, N))
    if (Kc is None) != (Vc is None):
        raise ValueError("Kc and Vc must be given together")
    if Kc is not None:
        _check_host(Kc, "Kc", Q.dtype, (B, Hkv, G, d))
        _check_host(Vc, "Vc", Q.dtype, (B, Hkv, G, d))
    prm = make_params(B, Hq, Hkv, N, d, g, w, _DTYPE[Q.dtype], scale, window_mode=window_mode,
                      pool_mode=pool_mode)
    need = int(lib.cca_prefill_host_workspace_size(ctypes.byref(prm)))
    if workspace is None:
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    if not workspace.is_cuda or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"workspace must be a CUDA buffer of at least {need} bytes")
    ptr = (lambda t: None if t is None else t.data_ptr())
    with torch.cuda.device(workspace.device):
        st = lib.cca_prefill_host(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), ptr(LSE), ptr(Kc),
                                  ptr(Vc), ctypes.byref(prm), workspace.data_ptr(),
                                  workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if st != CCA_OK:
        raise CcaError(st, "cca_prefill_host")
    return O, LSE, Kc, Vc


class CcaAttentionFunction(torch.autograd.Function):
    """Autograd wrapper of the prefill step: forward = cca_prefill (pooling + fused
    attention), backward = cca_prefill_bwd.  Both run in the library's kernels; this
    class only saves tensors and casts the fp32 gradients to the inputs' dtype."""

    @staticmethod
    def forward(ctx, Q, K, V, g, w, scale, pool_mode, window_mode):
        Q, K, V = Q.contiguous(), K.contiguous(), V.contiguous()
        O, LSE, Kc, Vc = cca_prefill(Q, K, V, g, w, scale, pool_mode=pool_mode, window_mode=window_mode)
        ctx.save_for_backward(Q, K, V, Kc, Vc, O, LSE)
        ctx.cfg = (g, w, scale, pool_mode, window_mode)
        return O

    @staticmethod
    def backward(ctx, dO):
        if torch.cuda.is_current_stream_capturing() and _build.binding_is_for_this_torch():
            (_fast or _bound()).check_leaves()
        of = _CcaGradients.apply if torch.is_grad_enabled() else _cca_gradients
        return (*of(*ctx.saved_tensors, dO, ctx.cfg), None, None, None, None, None)


def _dense(x):
    """x, contiguous from a 16-byte boundary on."""
    x = x.contiguous()
    return x if x.data_ptr() % 16 == 0 else x.clone()


def _cca_gradients(Q, K, V, Kc, Vc, O, LSE, dO, cfg):
    g, w, scale, pool_mode, window_mode = cfg
    dQ, dK, dV = cca_prefill_bwd(Q, K, V, Kc, Vc, O, LSE, _dense(dO.to(Q.dtype)), g, w, scale,
                                 pool_mode=pool_mode, window_mode=window_mode)
    return dQ.to(Q.dtype), dK.to(K.dtype), dV.to(V.dtype)


class _CcaGradients(torch.autograd.Function):
    """The gradients as a function of what they depend on, where someone might differentiate them again:
    that is an error then, and not a term that is left out."""

    @staticmethod
    def forward(ctx, *args):
        return _cca_gradients(*args)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("cca_attention: its gradient cannot be differentiated again")


def _positioned(Q, K, q_weight, k_weight, norm, inv_freq, rotary):
    """Q and K normed and given their positions, as far as they are asked for."""
    if norm or q_weight is not None or k_weight is not None:
        return norm_rope(Q, K, q_weight, k_weight, inv_freq, **rotary)
    if inv_freq is not None:
        return rope(Q, K, inv_freq, **rotary)
    if rotary:
        raise ValueError(f"{sorted(rotary)} without inv_freq")
    return Q, K


def cca_attention(Q, K, V, g: int, w: int, scale: float = 0.0, pool_mode: int = 0, window_mode: int = 0,
                  inv_freq=None, q_weight=None, k_weight=None, norm: bool = False, **rotary):
    """CCA attention output O [B, Hq, N, d] with gradients for Q, K and V (prefill step).
    With inv_freq, Q and K are first given their positions by rope(Q, K, inv_freq, **rotary); with
    weights of their norms (or norm=True), by norm_rope(Q, K, q_weight, k_weight, inv_freq, **rotary).
    The gradients cannot be differentiated again: under create_graph they carry an error (RuntimeError)."""
    Q, K = _positioned(Q, K, q_weight, k_weight, norm, inv_freq, rotary)
    # copies are made outside the function, so that what it saves is what its gradients depend on
    Q, K, V = _dense(Q), _dense(K), _dense(V)
    return CcaAttentionFunction.apply(Q, K, V, g, w, scale, pool_mode, window_mode)


# ---------------------------------------------------------------- rotary positions

def rope_frequencies(rot: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original: int = 8192, low: float = 1.0, high: float | None = None, device="cuda"):
    """Frequencies of a rotary embedding, and the factor that goes with them: (inv_freq float64
    [rot/2] on `device`, attention factor).  inv_freq[i] = base**(-2i/rot), stretched for contexts
    `factor` times the `original` length by one of
      "linear"  every frequency / factor (positions interpolated)
      "ntk"     base * factor**(rot/(rot-2)): the slowest pair / factor, the fastest unchanged
      "bands"   by the turns a pair makes over `original` positions: above `high` (4 unless given)
                unchanged, below `low` / factor, between them the mean weighted linearly in the turns
      "yarn"    the same with the weight linear in the pair's index (`high` 32 unless given), and the
                attention factor 0.1 ln(factor) + 1."""
    import math
    if rot < 2 or rot % 2 or factor < 1.0 or scaling not in (None, "linear", "ntk", "bands", "yarn"):
        raise ValueError(f"rot {rot}, scaling {scaling!r}, factor {factor}")
    if high is None:
        high = 32.0 if scaling == "yarn" else 4.0
    if scaling == "ntk":
        if rot == 2:
            raise ValueError("ntk scaling needs more than one pair")
        base = base * factor ** (rot / (rot - 2))
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = base ** (-2.0 * i / rot)
    attention = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling in ("bands", "yarn"):
        if not 0.0 < low < high or original < 1:
            raise ValueError("bands and yarn need 0 < low < high and original >= 1")
        if scaling == "bands":
            keep = (f * (original / (2.0 * math.pi)) - low) / (high - low)
        else:
            def pair(turns):    # the (fractional) pair that makes so many turns over `original`
                return rot * math.log(original / (2.0 * math.pi * turns)) / (2.0 * math.log(base))
            a, z = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
            keep = 1.0 - (i - a) / max(z - a, 1e-3)
            attention = 0.1 * math.log(factor) + 1.0
        keep = keep.clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / factor)
    return f.to(device), attention


class _On:
    """The caller's stream as the current one, so that what a call allocates belongs to it too."""

    def __init__(self, t, stream):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError("the first tensor must be a CUDA tensor")
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=t.device)
        if stream.device != t.device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {t.device}")
        self.over = torch.cuda.stream(stream)

    def __enter__(self):
        self.over.__enter__()

    def __exit__(self, *exc):
        self.over.__exit__(*exc)


def cca_rope(Q, K, inv_freq, positions=None, start: int = 0, layout: str = "half", factor: float = 1.0,
             inverse: bool = False, out=None, stream=None):
    """Gives queries and keys their rotary positions, in one launch.  Q [B, Hq, N, d] and
    K [B, Hkv, N, d] (or None) may have any strides with contiguous, 16-byte aligned rows, e.g.
    the transposed view of a projection's output; the results are contiguous [B, H, N, d] (or
    `out`, a pair of such tensors, which may be Q and K themselves).  The first 2 * len(inv_freq)
    columns rotate.  Row n is at position start + n, or positions[n] / positions[b, n] (int32).
    inverse: rotate back (the gradient).  Returns (Q', K').  Autograd does not follow this call (rope()
    is the one with gradients): an `out` that requires a gradient is refused outside torch.no_grad(), and
    counts as modified in place, as whatever a call of this module is given to write."""
    if stream is not None:
        with _On(Q, stream):
            return cca_rope(Q, K, inv_freq, positions, start, layout, factor, inverse, out)
    q, k = (None, None) if out is None else out
    return (_fast or _bound()).rope(Q, K, inv_freq, positions, start, layout, factor, inverse, q, k)


def rope(Q, K, inv_freq, positions=None, start: int = 0, layout: str = "half", factor: float = 1.0):
    """cca_rope with gradients for Q and K (or Q alone, with K None): returns (Q', K').  The gradient is
    the rotation back, by the same kernel, and can be differentiated again.  Rows that cannot be read
    in place are copied first.  As with any autograd function, a backward pass is captured into a CUDA
    graph together with its forward pass, from leaves that no eager graph still holds on the default
    stream (RuntimeError where one does)."""
    return (_fast or _bound()).rope_grad(Q, K, inv_freq, positions, start, layout, factor)


def cca_norm_rope(Q, K, q_weight=None, k_weight=None, inv_freq=None, positions=None, start: int = 0, layout: str = "half",
                  factor: float = 1.0, eps: float = 1e-6, offset: float = 0.0, out=None, stream=None):
    """cca_rope of queries and keys that are first normed for each head, in one launch: every row is divided
    by its root mean square (sqrt(mean + eps)) and multiplied by offset + weight, weights [d] or
    [heads, d] in the inputs' type or fp32 (None: by nothing).  Without inv_freq nothing rotates.
    Everything else as cca_rope.  Returns (Q', K')."""
    if stream is not None:
        with _On(Q, stream):
            return cca_norm_rope(Q, K, q_weight, k_weight, inv_freq, positions, start, layout, factor, eps, offset, out)
    q, k = (None, None) if out is None else out
    return (_fast or _bound()).norm_rope(Q, K, inv_freq, positions, start, layout, factor, q_weight, k_weight, eps, offset, q, k)


def norm_rope(Q, K, q_weight=None, k_weight=None, inv_freq=None, positions=None, start: int = 0, layout: str = "half",
              factor: float = 1.0, eps: float = 1e-6, offset: float = 0.0):
    """cca_norm_rope with gradients for Q, K (or Q alone, with K None) and the weights: returns (Q', K').
    The gradient cannot be differentiated again (RuntimeError); captured backward passes as in rope()."""
    return (_fast or _bound()).norm_rope_grad(Q, K, inv_freq, positions, start, layout, factor, q_weight, k_weight, eps, offset)


# ---------------------------------------------------------------- packed sequences

class Packed:
    """A batch of packed sequences as cca_pack lays it out: `plan` (the device buffer that the packed
    calls read), `positions` (int32 [tokens], every token's position in its sequence, for rope),
    and the sizes that it was made for."""
    __slots__ = ("plan", "positions", "sequences", "tokens", "g", "w", "window_mode")

    def __init__(self, plan, positions, sequences, tokens, g, w, window_mode):
        self.plan, self.positions = plan, positions
        self.sequences, self.tokens, self.g, self.w, self.window_mode = sequences, tokens, g, w, window_mode

    def _args(self):
        return self.plan, self.sequences, self.tokens, self.g, self.w, self.window_mode

    @property
    def cores(self) -> bool:
        """Whether a sequence may be long enough to see core tokens."""
        return self.w < self.tokens and self.g <= self.tokens


def cca_pack(cu_seqlens, tokens: int, g: int = 16, w: int | None = None, window_mode: int = 0, plan=None, dev_status=None,
             stream=None) -> Packed:
    """Lays out a batch of sequences that lie one behind the other in [heads, tokens, d] tensors: sequence s
    holds rows cu_seqlens[s] .. cu_seqlens[s + 1] - 1 (int32 [S + 1] on the device, never read by the host;
    any sequence may be empty).  Made once for a batch and given to every packed call of every layer.
    w None: every earlier token of the sequence is seen (full causal attention, no core tokens).
    A captured call serves later lengths of the same cu_seqlens; `plan` may hold a buffer to use again."""
    if stream is not None:
        with _On(cu_seqlens, stream):
            return cca_pack(cu_seqlens, tokens, g, w, window_mode, plan, dev_status)
    w = tokens if w is None else w
    plan, positions = (_fast or _bound()).pack(cu_seqlens, tokens, g, w, window_mode, plan, dev_status)
    return Packed(plan, positions, cu_seqlens.shape[0] - 1, tokens, g, w, window_mode)


def cca_pool_packed(Q, K, V, packed: Packed, Kc=None, Vc=None, scale: float = 0.0, pool_mode: int = 0, dev_status=None,
                    stream=None):
    """Global-aware pooling of every whole group of every packed sequence: Q [Hq, tokens, d], K, V [Hkv, tokens, d]
    with any strides (contiguous, 16-byte aligned rows).  Returns (Kc, Vc), each [Hkv, tokens // g, d]:
    group j of the sequence that starts at row a is row a // g + j; rows of no group are zero.
    pool_mode 0 or 1 (see cca_pool)."""
    if stream is not None:
        with _On(Q, stream):
            return cca_pool_packed(Q, K, V, packed, Kc, Vc, scale, pool_mode, dev_status)
    return (_fast or _bound()).pool_packed(Q, K, V, *packed._args(), Kc, Vc, scale, pool_mode, dev_status)


def cca_attn_packed(Q, K, V, Kc, Vc, packed: Packed, O=None, LSE=None, scale: float = 0.0, dev_status=None, stream=None):
    """CCA attention of every row of every packed sequence over its own tokens and cores (Kc, Vc None where
    packed.w covers all tokens).  Strides as in cca_pool_packed, of O too.  Returns (O [Hq, tokens, d],
    LSE [Hq, tokens] fp32); rows of no sequence are left as they were."""
    if stream is not None:
        with _On(Q, stream):
            return cca_attn_packed(Q, K, V, Kc, Vc, packed, O, LSE, scale, dev_status)
    return (_fast or _bound()).attn_packed(Q, K, V, Kc, Vc, *packed._args(), O, LSE, scale, dev_status)


def cca_prefill_packed(Q, K, V, packed: Packed, scale: float = 0.0, pool_mode: int = 0, out=None, dev_status=None, stream=None):
    """Both steps of CCA prefill over packed sequences: pooling (where a core can be seen), then attention.
    Returns (O, LSE, Kc, Vc), Kc and Vc None without cores.  `out` may hold preallocated (O, LSE, Kc, Vc)."""
    if stream is not None:
        with _On(Q, stream):
            return cca_prefill_packed(Q, K, V, packed, scale, pool_mode, out, dev_status)
    O, LSE, Kc, Vc = (None,) * 4 if out is None else out
    if packed.cores:
        Kc, Vc = cca_pool_packed(Q, K, V, packed, Kc, Vc, scale, pool_mode, dev_status)
    else:
        Kc = Vc = None
    O, LSE = cca_attn_packed(Q, K, V, Kc, Vc, packed, O, LSE, scale, dev_status)
    return O, LSE, Kc, Vc


def cca_packed_bwd(Q, K, V, Kc, Vc, O, LSE, dO, packed: Packed, scale: float = 0.0, pool_mode: int = 0, dQ=None, dK=None,
                   dV=None, workspace=None, dev_status=None, stream=None):
    """Gradients (dQ, dK, dV) of sum(dO * O) for cca_prefill_packed, in the inputs' type.  Rows of no sequence
    are left as they were."""
    if stream is not None:
        with _On(Q, stream):
            return cca_packed_bwd(Q, K, V, Kc, Vc, O, LSE, dO, packed, scale, pool_mode, dQ, dK, dV, workspace, dev_status)
    return (_fast or _bound()).packed_bwd(Q, K, V, Kc, Vc, O, LSE, dO, *packed._args(), dQ, dK, dV, workspace, scale, pool_mode,
                                          dev_status)


def cca_packed_clear(packed: Packed, *tensors, stream=None):
    """Sets the rows of no sequence (before the first one, behind the last one) of up to four packed tensors
    [heads, tokens, d] to zero, in place; all rows where the lengths were refused."""
    if stream is not None:
        with _On(tensors[0], stream):
            return cca_packed_clear(packed, *tensors)
    (_fast or _bound()).packed_clear(*packed._args(), *(tensors + (None,) * (4 - len(tensors))))


def cca_attention_packed(Q, K, V, packed: Packed, scale: float = 0.0, pool_mode: int = 0, inv_freq=None, q_weight=None,
                         k_weight=None, norm: bool = False, dev_status=None, **rotary):
    """CCA attention output O [Hq, tokens, d] of packed sequences with gradients for Q, K and V; tokens of no
    sequence have output and gradients zero.  With inv_freq and weights of the norms (see cca_attention), Q and
    K are first normed and given their positions within their sequences.  The gradients cannot be differentiated
    again: under create_graph they carry an error (RuntimeError) for whoever tries.
    dev_status (int32 [1]) takes what the kernels report, of this call and of its backward pass: lengths that cca_pack
    has refused (output and gradients are zero then), and waits that ran out (rows may be unwritten then)."""
    if inv_freq is not None or norm or q_weight is not None or k_weight is not None:
        Q, K = _positioned(Q[None], K[None], q_weight, k_weight, norm, inv_freq, {"positions": packed.positions, **rotary})
        Q, K = Q[0], K[0]
    elif rotary:
        raise ValueError(f"{sorted(rotary)} without inv_freq")
    return (_fast or _bound()).attention_packed(Q, K, V, *packed._args(), scale, pool_mode, dev_status)


# ---------------------------------------------------------------- paged caches

def cca_rope_append(Q, K, V, Kp, Vp, table, lens, inv_freq=None, parents=None, counts=None, layout: str = "half",
                    factor: float = 1.0, out=None, dev_status=None, stream=None):
    """The new tokens of a step: rotates Q [B, Hq, T, d] and K [B, Hkv, T, d], and stores K and V
    into the raw pages at rows lens[b] + t.  Strides as in cca_rope.  parents [B, T] (int32): the
    tokens are a drafted tree (see cca_tree_fwd), node t at position lens[b] + depth; without, at
    lens[b] + t.  counts [B]: only the first counts[b] tokens are real.  Tokens that are not real are
    not stored and their query rows are zero.  Without inv_freq nothing rotates (core tokens of a
    prompt are stored that way, with Q None).  Returns the queries, contiguous [B, Hq, T, d]."""
    if stream is not None:
        with _On(K, stream):
            return cca_rope_append(Q, K, V, Kp, Vp, table, lens, inv_freq, parents, counts, layout, factor, out, dev_status)
    return (_fast or _bound()).rope_append(Q, K, V, Kp, Vp, table, lens, inv_freq, parents, counts, layout, factor, out, dev_status)


def cca_norm_rope_append(Q, K, V, Kp, Vp, table, lens, q_weight=None, k_weight=None, inv_freq=None, parents=None, counts=None,
                         layout: str = "half", factor: float = 1.0, eps: float = 1e-6, offset: float = 0.0, out=None,
                         dev_status=None, stream=None):
    """cca_rope_append of queries and keys that are first normed for each head (see cca_norm_rope), in one
    launch; values are stored as they are.  Returns the queries, contiguous [B, Hq, T, d]."""
    if stream is not None:
        with _On(K, stream):
            return cca_norm_rope_append(Q, K, V, Kp, Vp, table, lens, q_weight, k_weight, inv_freq, parents, counts, layout,
                                        factor, eps, offset, out, dev_status)
    return (_fast or _bound()).norm_rope_append(Q, K, V, Kp, Vp, table, lens, inv_freq, parents, counts, layout, factor, out,
                                                dev_status, q_weight, k_weight, eps, offset)


def tree_workspace_size(B, Hq, Hkv, T, d, g, w, dtype) -> int:
    """Bytes of workspace cca_tree_fwd needs on the current device."""
    prm = make_params(B, Hq, Hkv, 0, d, g, w, _DTYPE[dtype])
    return int(load_library().cca_tree_workspace_size(ctypes.byref(prm), int(T)))


def cca_tree_fwd(Q, Kp, Vp, table, Kcp, Vcp, core_table, lens, g: int, w: int, parents=None, O=None, LSE=None,
                 workspace=None, scale: float = 0.0, dev_status=None, stream=None, window_mode: int = 0):
    """CCA attention of drafted tokens over paged caches; T = 1 is plain decoding.
    Q [B, Hq, T, d]; raw pool Kp, Vp [pages, Hkv, rows, d] with table [B, columns]; core pool Kcp, Vcp
    with core_table; lens [B] committed tokens.  Node t's K and V lie in raw row lens[b] + t;
    parents [B, T] is the node before it, -1 for a child of the last committed token, anything else
    (-2) for padding, which needs no page; without parents the nodes are one chain.  Returns (O [B, Hq, T, d], LSE
    [B, Hq, T] fp32); padding nodes have O = 0 and LSE = -inf."""
    if stream is not None:
        with _On(Q, stream):
            return cca_tree_fwd(Q, Kp, Vp, table, Kcp, Vcp, core_table, lens, g, w, parents, O, LSE, workspace, scale,
                                dev_status, None, window_mode)
    return (_fast or _bound()).tree_fwd(Q, Kp, Vp, table, Kcp, Vcp, core_table, lens, g, w, parents, O, LSE, workspace, scale,
                                        dev_status, window_mode)


def cca_pool_pages(Q, Kp, Vp, table, Kcp, Vcp, core_table, lens, accepted, g: int, path=None, scale: float = 0.0,
                   dev_status=None, stream=None, pool_mode: int = 0):
    """Pools the groups that the accepted[b] tokens after lens[b] complete, from raw pages into core
    pages (in place).  Q [B, Hq, T, d] holds the step's queries; the i-th accepted token's is
    Q[b, :, path[b, i]] (path [B, A] int32), or Q[b, :, i] without a path.  Returns (Kcp, Vcp)."""
    if stream is not None:
        with _On(Q, stream):
            return cca_pool_pages(Q, Kp, Vp, table, Kcp, Vcp, core_table, lens, accepted, g, path, scale, dev_status, None,
                                  pool_mode)
    (_fast or _bound()).pool_pages(Q, Kp, Vp, table, Kcp, Vcp, core_table, lens, accepted, g, path, scale, dev_status, pool_mode)
    return Kcp, Vcp


def cca_pages_reserve(refs, table, lens, extra, rows: int, pairs=None, workspace=None, dev_status=None, stream=None):
    """Room for rows [lens[b], lens[b] + extra[b]) of every sequence: table [B, columns] and refs
    [pages] (int32, holders of each page) are updated in place.  Missing pages are the lowest free
    ones; a shared page is replaced by one of the row's own.  Returns pairs [B, 2], (old, new) pages
    for cca_pages_copy, (-1, -1) for none.  Too few free pages: nothing changes and dev_status
    becomes CCA_ERR_NO_PAGES."""
    if stream is not None:
        with _On(refs, stream):
            return cca_pages_reserve(refs, table, lens, extra, rows, pairs, workspace, dev_status)
    return (_fast or _bound()).pages_reserve(refs, table, lens, extra, rows, pairs, workspace, dev_status)


def cca_pages_fork(refs, table, src, dst, lens, rows: int, dev_status=None, stream=None):
    """Table rows dst [n] become second holders of the pages of rows src [n] (the first
    ceil(lens[src] / rows) entries), in place.  The dst rows must hold no pages."""
    if stream is not None:
        with _On(refs, stream):
            return cca_pages_fork(refs, table, src, dst, lens, rows, dev_status)
    (_fast or _bound()).pages_fork(refs, table, src, dst, lens, rows, dev_status)


def cca_pages_free(refs, table, first, last, dev_status=None, stream=None):
    """Entries [first[b], last[b]) of every table row give up their pages, in place."""
    if stream is not None:
        with _On(refs, stream):
            return cca_pages_free(refs, table, first, last, dev_status)
    (_fast or _bound()).pages_free(refs, table, first, last, dev_status)


def cca_pages_copy(Kp, Vp, pairs, dev_status=None, stream=None):
    """Copies page pairs[i, 0] to page pairs[i, 1] of the pools (every layer of a [layers, pages, ...]
    pool), in place; pairs with a negative entry are skipped."""
    if stream is not None:
        with _On(Kp, stream):
            return cca_pages_copy(Kp, Vp, pairs, dev_status)
    (_fast or _bound()).pages_copy(Kp, Vp, pairs, dev_status)
    return Kp, Vp


def cca_pages_compact(Kp, Vp, table, lens, path, accepted, dev_status=None, stream=None):
    """Keeps the accepted nodes of a drafted tree: raw row lens[b] + path[b, i] moves to row
    lens[b] + i for i < accepted[b], K and V, every layer, in place.  path [B, A] rises."""
    if stream is not None:
        with _On(Kp, stream):
            return cca_pages_compact(Kp, Vp, table, lens, path, accepted, dev_status)
    (_fast or _bound()).pages_compact(Kp, Vp, table, lens, path, accepted, dev_status)
    return Kp, Vp
