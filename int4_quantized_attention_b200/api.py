"""Thin Python binding of the C ABI in include/rotate_attn.h.

Argument marshalling only: every step of the path runs in the CUDA kernels of
``librotate_attn.so``.  PyTorch supplies device memory and the current CUDA
stream.  There is no fallback: if the library is missing or a call fails, a
``RotateAttnError`` is raised.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
# RA_LIBRARY=bounds loads the bounds-checked test build instead (the same
# ABI; every computed device index is checked, violations are reported as
# RA_ERR_DEVICE_BOUNDS by ra_check_device_error).
LIB_PATH = os.path.join(PKG, "librotate_attn_bounds.so" if os.environ.get("RA_LIBRARY") == "bounds"
                        else "librotate_attn.so")

RA_OK, RA_ERR_INVALID_ARG, RA_ERR_UNSUPPORTED, RA_ERR_WORKSPACE, RA_ERR_CUDA, \
    RA_ERR_DEVICE_TIMEOUT, RA_ERR_DEVICE_BOUNDS, RA_ERR_CACHE_FULL = range(8)
ROT = {"none": 0, "interleaved": 1, "half": 2, "full": 3, "blocks_interleaved": 4, "blocks_half": 5}
P_MODE = {"range": 0, "symmetric": 1}       # ra_p_mode
DTYPE_FP16, DTYPE_BF16 = 0, 1               # ra_dtype


class RotateAttnError(RuntimeError):
    def __init__(self, call: str, status: int, detail: str):
        super().__init__(f"{call}: {status_string(status)} ({detail})")
        self.status = status


class Problem(ctypes.Structure):
    """Mirror of ra_problem."""
    _fields_ = [("B", ctypes.c_int), ("H", ctypes.c_int), ("d", ctypes.c_int),
                ("F", ctypes.c_int), ("Hh", ctypes.c_int), ("W", ctypes.c_int),
                ("n_text", ctypes.c_int), ("split", ctypes.c_int * 3),
                ("theta", ctypes.c_double), ("rot", ctypes.c_int), ("p_mode", ctypes.c_int),
                ("v_rot", ctypes.c_int), ("blocks", ctypes.c_void_p)]


class Qkv4(ctypes.Structure):
    """Mirror of ra_qkv4 (device pointers)."""
    _fields_ = [("q4", ctypes.c_void_p), ("k4", ctypes.c_void_p), ("v4t", ctypes.c_void_p),
                ("sq", ctypes.c_void_p), ("sk", ctypes.c_void_p), ("sv", ctypes.c_void_p),
                ("vsum", ctypes.c_void_p)]


class Packed(ctypes.Structure):
    """Mirror of ra_packed."""
    _fields_ = [(n, ctypes.c_int) for n in ("n_seqs", "Hq", "Hkv", "d", "dtype", "causal", "total_q", "total_k")] + \
        [("scale", ctypes.c_double)] + \
        [(n, ctypes.c_longlong) for n in ("q_token", "q_head", "k_token", "k_head", "v_token", "v_head",
                                          "o_token", "o_head")]


class CacheProblem(ctypes.Structure):
    """Mirror of ra_cache_problem."""
    _fields_ = [(n, ctypes.c_int) for n in ("layers", "n_pages", "page_size", "Hkv", "d", "dtype", "max_seqs",
                                            "max_pages")]


class Cache(ctypes.Structure):
    """Mirror of ra_cache (device pointers)."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "refs", "lens", "table")]


class CacheAttn(ctypes.Structure):
    """Mirror of ra_cache_attn."""
    _fields_ = [(n, ctypes.c_int) for n in ("n_seqs", "Hq", "total_q", "layer", "shared")] + \
        [("scale", ctypes.c_double)] + \
        [(n, ctypes.c_longlong) for n in ("q_token", "q_head", "o_token", "o_head")]


_lib = None
_P = ctypes.POINTER(Problem)
_V = ctypes.c_void_p
_SZ = ctypes.c_size_t

_PK, _CP, _C, _CA = (ctypes.POINTER(t) for t in (Packed, CacheProblem, Cache, CacheAttn))
_I, _LL = ctypes.c_int, ctypes.c_longlong

_SIGNATURES = {
    "ra_seq_len": (ctypes.c_int, [_P]),
    "ra_seq_pad": (ctypes.c_int, [_P]),
    "ra_validate": (ctypes.c_int, [_P]),
    "ra_qkv4_bytes": (_SZ, [_P]),
    "ra_qkv4_bind": (ctypes.c_int, [_P, _V, _SZ, ctypes.POINTER(Qkv4)]),
    "ra_workspace_bytes": (_SZ, [_P, ctypes.c_int]),
    "ra_prepare": (ctypes.c_int, [_P, _V, _SZ, _V]),
    "ra_rotate_quantize_qkv": (ctypes.c_int, [_P, _V, _V, _V, ctypes.POINTER(Qkv4), _V, _SZ, _V]),
    "ra_int4_attention_fwd": (ctypes.c_int, [_P, ctypes.POINTER(Qkv4), _V, _V, _SZ, _V]),
    "ra_fp16_attention_fwd": (ctypes.c_int, [_P, _V, _V, _V, _V, _V, _SZ, _V]),
    "ra_check_device_error": (ctypes.c_int, [_V, _V]),
    "ra_host_staging_bytes": (_SZ, [_P, ctypes.c_int]),
    "ra_int4_attention_host": (ctypes.c_int, [_P, _V, _V, _V, _V, ctypes.c_int, _V, _SZ, _V]),
    "ra_host_chunks": (ctypes.c_int, [_P, ctypes.c_int, ctypes.POINTER(ctypes.c_int), ctypes.c_int]),
    "ra_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "ra_last_error_detail": (ctypes.c_char_p, []),
    "ra_tables_floats": (_SZ, [_P]),
    "ra_build_tables_host": (ctypes.c_int, [_P, _V, _SZ]),
    "ra_debug_int4_tile": (ctypes.c_int, [_P, ctypes.POINTER(Qkv4), ctypes.c_int, ctypes.c_int,
                                          ctypes.c_int, _V, _V, _V, _SZ, _V]),
    "ra_rotate_quantize_qkv_noalloc": (ctypes.c_int, [_P, _V, _V, _V, ctypes.POINTER(Qkv4), _V]),
    "ra_noalloc_check_device_error": (ctypes.c_int, [_V]),
    "ra_debug_set_wait_timeout_us": (None, [ctypes.c_uint32]),
    "ra_debug_timeout_probe": (ctypes.c_int, [_V, _SZ, _V]),
    "ra_measure_mma_i8": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int, _V, _SZ, _V]),
    "ra_debug_ex2": (ctypes.c_int, [_V, _V, ctypes.c_int, _V]),
    "ra_packed_workspace_bytes": (_SZ, [_PK]),
    "ra_packed_attention_fwd": (_I, [_PK, _V, _V, _V, _V, _V, _V, _V, _V, _SZ, _V]),
    "ra_cache_validate": (_I, [_CP]),
    "ra_cache_pool_bytes": (_SZ, [_CP]),
    "ra_cache_state_bytes": (_SZ, [_CP]),
    "ra_cache_bind": (_I, [_CP, _V, _SZ, _V, _SZ, _C]),
    "ra_cache_workspace_bytes": (_SZ, [_CP]),
    "ra_cache_init": (_I, [_CP, _C, _V]),
    "ra_cache_extend": (_I, [_CP, _C, _V, _V, _I, _V, _SZ, _V]),
    "ra_cache_write": (_I, [_CP, _C, _I, _V, _V, _I, _I, _V, _V, _LL, _LL, _LL, _LL, _V, _SZ, _V]),
    "ra_cache_fork": (_I, [_CP, _C, _V, _V, _I, _V, _SZ, _V]),
    "ra_cache_free": (_I, [_CP, _C, _V, _I, _V, _SZ, _V]),
    "ra_cache_compact": (_I, [_CP, _C, _V, _SZ, _V]),
    "ra_cache_attention_workspace_bytes": (_SZ, [_CP, _CA]),
    "ra_cache_attention_fwd": (_I, [_CP, _C, _CA, _V, _V, _V, _V, _V, _V, _SZ, _V]),
}


def lib():
    """Load librotate_attn.so (built in-tree by ``build.build()``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RotateAttnError("load", RA_ERR_CUDA,
                                  f"{LIB_PATH} is missing; run int4_quantized_attention_b200.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().ra_status_string(status).decode()


def _check(call: str, status: int) -> None:
    if status != RA_OK:
        raise RotateAttnError(call, status, lib().ra_last_error_detail().decode())


def problem(cfg, rot: Optional[str] = None) -> Problem:
    """ra_problem from any object with B, H, d, F, Hh, W, n_text, split, theta, rot."""
    p = Problem()
    p.B, p.H, p.d = cfg.B, cfg.H, cfg.d
    p.F, p.Hh, p.W, p.n_text = cfg.F, cfg.Hh, cfg.W, cfg.n_text
    p.split = (ctypes.c_int * 3)(*cfg.split)
    p.theta = float(cfg.theta)
    p.rot = ROT[rot if rot is not None else cfg.rot]
    p.p_mode = P_MODE[getattr(cfg, "p_mode", "range")]
    p.v_rot = int(getattr(cfg, "v_rot", 0))
    blocks = getattr(cfg, "blocks", None)
    if blocks is not None:
        arr = (ctypes.c_double * len(blocks))(*blocks)
        p._keep = arr                      # the array lives as long as the struct
        p.blocks = ctypes.cast(arr, ctypes.c_void_p)
    return p


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


# ---------------------------------------------------------------- C entry points

def seq_len(p: Problem) -> int:
    return lib().ra_seq_len(ctypes.byref(p))


def seq_pad(p: Problem) -> int:
    return lib().ra_seq_pad(ctypes.byref(p))


def validate(p: Problem) -> int:
    return lib().ra_validate(ctypes.byref(p))


def qkv4_bytes(p: Problem) -> int:
    return lib().ra_qkv4_bytes(ctypes.byref(p))


def qkv4_bind(p: Problem, buf) -> Qkv4:
    out = Qkv4()
    _check("ra_qkv4_bind", lib().ra_qkv4_bind(ctypes.byref(p), _ptr(buf), buf.numel() * buf.element_size(),
                                              ctypes.byref(out)))
    return out


def workspace_bytes(p: Problem, with_fp16_path: bool = True) -> int:
    return lib().ra_workspace_bytes(ctypes.byref(p), int(with_fp16_path))


def prepare(p: Problem, workspace, stream=None) -> None:
    _check("ra_prepare", lib().ra_prepare(ctypes.byref(p), _ptr(workspace), workspace.numel(), _stream(stream)))


def rotate_quantize_qkv(p: Problem, q, k, v, out: Qkv4, workspace, stream=None) -> None:
    _check("ra_rotate_quantize_qkv",
           lib().ra_rotate_quantize_qkv(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), ctypes.byref(out),
                                        _ptr(workspace), workspace.numel(), _stream(stream)))


def int4_attention_fwd(p: Problem, qkv4: Qkv4, o, workspace, stream=None) -> None:
    _check("ra_int4_attention_fwd",
           lib().ra_int4_attention_fwd(ctypes.byref(p), ctypes.byref(qkv4), _ptr(o), _ptr(workspace),
                                       workspace.numel(), _stream(stream)))


def fp16_attention_fwd(p: Problem, q, k, v, o, workspace, stream=None) -> None:
    _check("ra_fp16_attention_fwd",
           lib().ra_fp16_attention_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(workspace),
                                       workspace.numel(), _stream(stream)))


def host_staging_bytes(p: Problem, heads_per_chunk: int = 0) -> int:
    return lib().ra_host_staging_bytes(ctypes.byref(p), heads_per_chunk)


def host_chunks(p: Problem, heads_per_chunk: int = 0) -> list:
    """Heads per chunk, in order, of ra_int4_attention_host's pipeline."""
    n = lib().ra_host_chunks(ctypes.byref(p), heads_per_chunk, None, 0)
    if n < 0:
        _check("ra_host_chunks", RA_ERR_INVALID_ARG)
    out = (ctypes.c_int * max(n, 1))()
    lib().ra_host_chunks(ctypes.byref(p), heads_per_chunk, out, n)
    return list(out[:n])


def int4_attention_host(p: Problem, q, k, v, o, staging, heads_per_chunk: int = 0, stream=None) -> None:
    """The INT4 path from host q, k, v to host o (CPU tensors, page-locked for
    overlap); blocks until o is written."""
    _check("ra_int4_attention_host",
           lib().ra_int4_attention_host(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(o), heads_per_chunk,
                                        _ptr(staging), staging.numel(), _stream(stream)))


def rotate_quantize_qkv_noalloc(p: Problem, q, k, v, out: Qkv4, stream=None) -> None:
    """The prologue with its scratch in the library's fixed device array."""
    _check("ra_rotate_quantize_qkv_noalloc",
           lib().ra_rotate_quantize_qkv_noalloc(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), ctypes.byref(out),
                                                _stream(stream)))


def noalloc_check_device_error(stream=None) -> None:
    """Read and clear the error word of the allocation-free prologue's scratch."""
    _check("ra_noalloc_check_device_error", lib().ra_noalloc_check_device_error(_stream(stream)))


def check_device_error(workspace, stream=None) -> None:
    _check("ra_check_device_error", lib().ra_check_device_error(_ptr(workspace), _stream(stream)))


def build_tables_host(p: Problem):
    import numpy as np
    n = lib().ra_tables_floats(ctypes.byref(p))
    out = np.empty((n,), np.float32)
    _check("ra_build_tables_host",
           lib().ra_build_tables_host(ctypes.byref(p), out.ctypes.data_as(ctypes.c_void_p), n))
    return out.reshape(-1, 4)


def debug_int4_tile(p: Problem, qkv4: Qkv4, bh: int, q_tile: int, kv_tile: int, workspace, stream=None):
    """int32 S tile [128, 128] and int8 P codes [128, 128] of one (head, q tile, kv tile)."""
    import torch
    dev = workspace.device
    s_out = torch.zeros((128, 128), dtype=torch.int32, device=dev)
    p_out = torch.zeros((128, 128), dtype=torch.int8, device=dev)
    _check("ra_debug_int4_tile",
           lib().ra_debug_int4_tile(ctypes.byref(p), ctypes.byref(qkv4), bh, q_tile, kv_tile, _ptr(s_out),
                                    _ptr(p_out), _ptr(workspace), workspace.numel(), _stream(stream)))
    return s_out, p_out


def debug_ex2(x, stream=None):
    """The attention kernel's 2^x (ex2.approx) of a device float32 tensor."""
    import torch
    y = torch.empty_like(x)
    _check("ra_debug_ex2", lib().ra_debug_ex2(_ptr(x), _ptr(y), x.numel(), _stream(stream)))
    return y


def debug_set_wait_timeout_us(microseconds: int) -> None:
    lib().ra_debug_set_wait_timeout_us(microseconds)


def debug_timeout_probe(workspace, stream=None) -> None:
    _check("ra_debug_timeout_probe",
           lib().ra_debug_timeout_probe(_ptr(workspace), workspace.numel(), _stream(stream)))


def measure_mma_i8(n: int, iters: int, ctas: int, workspace, stream=None) -> None:
    """Enqueue the INT8 tensor-core rate probe (ctas * iters * 4 * 2 * 128 * n * 32 ops)."""
    _check("ra_measure_mma_i8", lib().ra_measure_mma_i8(n, iters, ctas, _ptr(workspace), workspace.numel(),
                                                        _stream(stream)))


def packed_workspace_bytes(p: Packed) -> int:
    return lib().ra_packed_workspace_bytes(ctypes.byref(p))


def packed_attention_fwd(p: Packed, q, k, v, cu_q, cu_k, o, lse, workspace, stream=None) -> None:
    _check("ra_packed_attention_fwd",
           lib().ra_packed_attention_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(cu_q), _ptr(cu_k), _ptr(o),
                                         _ptr(lse), _ptr(workspace), workspace.numel(), _stream(stream)))


def cache_validate(p: CacheProblem) -> int:
    return lib().ra_cache_validate(ctypes.byref(p))


def cache_pool_bytes(p: CacheProblem) -> int:
    return lib().ra_cache_pool_bytes(ctypes.byref(p))


def cache_state_bytes(p: CacheProblem) -> int:
    return lib().ra_cache_state_bytes(ctypes.byref(p))


def cache_bind(p: CacheProblem, pool, state) -> Cache:
    out = Cache()
    _check("ra_cache_bind", lib().ra_cache_bind(ctypes.byref(p), _ptr(pool), pool.numel() * pool.element_size(),
                                                _ptr(state), state.numel() * state.element_size(), ctypes.byref(out)))
    return out


def cache_workspace_bytes(p: CacheProblem) -> int:
    return lib().ra_cache_workspace_bytes(ctypes.byref(p))


def cache_init(p: CacheProblem, c: Cache, stream=None) -> None:
    _check("ra_cache_init", lib().ra_cache_init(ctypes.byref(p), ctypes.byref(c), _stream(stream)))


def cache_extend(p: CacheProblem, c: Cache, seqs, n_new, workspace, stream=None) -> None:
    _check("ra_cache_extend",
           lib().ra_cache_extend(ctypes.byref(p), ctypes.byref(c), _ptr(seqs), _ptr(n_new), seqs.numel(),
                                 _ptr(workspace), workspace.numel(), _stream(stream)))


def cache_write(p: CacheProblem, c: Cache, layer: int, seqs, cu_new, k, v, workspace, stream=None) -> None:
    """k, v: [tokens, Hkv, 128]."""
    _check("ra_cache_write",
           lib().ra_cache_write(ctypes.byref(p), ctypes.byref(c), layer, _ptr(seqs), _ptr(cu_new), seqs.numel(),
                                k.shape[0], _ptr(k), _ptr(v), k.stride(0), k.stride(1), v.stride(0), v.stride(1),
                                _ptr(workspace), workspace.numel(), _stream(stream)))


def cache_fork(p: CacheProblem, c: Cache, parents, children, workspace, stream=None) -> None:
    _check("ra_cache_fork",
           lib().ra_cache_fork(ctypes.byref(p), ctypes.byref(c), _ptr(parents), _ptr(children), children.numel(),
                               _ptr(workspace), workspace.numel(), _stream(stream)))


def cache_free(p: CacheProblem, c: Cache, seqs, workspace, stream=None) -> None:
    _check("ra_cache_free", lib().ra_cache_free(ctypes.byref(p), ctypes.byref(c), _ptr(seqs), seqs.numel(),
                                                _ptr(workspace), workspace.numel(), _stream(stream)))


def cache_compact(p: CacheProblem, c: Cache, workspace, stream=None) -> None:
    _check("ra_cache_compact", lib().ra_cache_compact(ctypes.byref(p), ctypes.byref(c), _ptr(workspace),
                                                      workspace.numel(), _stream(stream)))


def cache_attention_workspace_bytes(p: CacheProblem, a: CacheAttn) -> int:
    return lib().ra_cache_attention_workspace_bytes(ctypes.byref(p), ctypes.byref(a))


def cache_attention_fwd(p: CacheProblem, c: Cache, a: CacheAttn, q, seqs, cu_q, o, lse, workspace,
                        stream=None) -> None:
    _check("ra_cache_attention_fwd",
           lib().ra_cache_attention_fwd(ctypes.byref(p), ctypes.byref(c), ctypes.byref(a), _ptr(q), _ptr(seqs),
                                        _ptr(cu_q), _ptr(o), _ptr(lse), _ptr(workspace), workspace.numel(),
                                        _stream(stream)))


# ---------------------------------------------------------------- convenience

def _bad(call: str, detail: str):
    lib()
    return RotateAttnError(call, RA_ERR_INVALID_ARG, detail)


def _dtype(call: str, dtype) -> int:
    import torch
    if dtype not in (torch.float16, torch.bfloat16):
        raise _bad(call, f"dtype {dtype}: float16 or bfloat16")
    return DTYPE_FP16 if dtype == torch.float16 else DTYPE_BF16


def _rows(call: str, name: str, t, dtype, device, heads=None, tokens=None):
    """Checks a [tokens, heads, 128] tensor whose last dimension is contiguous."""
    shape = t.shape
    if len(shape) == 3 and shape[2] == 128 and t.dtype == dtype and t.device == device and \
            (t.stride(2) == 1 or not t.numel()) and (heads is None or shape[1] == heads) and \
            (tokens is None or shape[0] == tokens):
        return
    raise _bad(call, f"{name}: {tuple(shape)} {t.dtype} on {t.device}, strides {t.stride()}; want "
                     f"[{'tokens' if tokens is None else tokens}, {'heads' if heads is None else heads}, 128] "
                     f"{dtype} on {device} with a contiguous last dimension")


def _ints(call: str, name: str, t, device, n=None):
    import torch
    if t.dtype == torch.int32 and t.device == device and t.dim() == 1 and t.is_contiguous() and \
            (n is None or t.numel() == n):
        return
    raise _bad(call, f"{name}: a contiguous 1-D int32 tensor{'' if n is None else f' of {n}'} on {device}")


class _Workspace:
    """A workspace that grows with what it is asked for.  Buffers that were
    outgrown are kept, since a captured graph may still use them."""

    def __init__(self, device):
        self.device, self.buffers = device, []

    def current(self):
        return self.buffers[-1] if self.buffers else self.grow(256)

    def grow(self, need: int):
        import torch
        if torch.cuda.is_current_stream_capturing():   # its zeroing would wait for the first replay
            raise _bad("workspace", "make the first call of this size before capturing it")
        size = max(need, 2 * self.buffers[-1].numel()) if self.buffers else need
        self.buffers.append(torch.zeros((size,), dtype=torch.uint8, device=self.device))
        return self.buffers[-1]

    def check(self):
        with _on(self.device):
            for b in self.buffers:
                check_device_error(b)


class PackedAttention:
    """Attention over packed sequences of different lengths (ra_packed_attention_fwd):
    owns, through PyTorch, the workspace of one stream of calls and runs on the
    current stream.  Calls of one object must not overlap on the GPU."""

    def __init__(self, device="cuda"):
        import torch
        self.device = torch.empty(0, device=device).device
        self._ws = _Workspace(self.device)

    def forward(self, q, k, v, cu_q, cu_k, causal: bool = True, scale: float = 0.0, out=None, lse=None,
                return_lse: bool = False):
        """q [total_q, Hq, 128], k and v [total_k, Hkv, 128], fp16 or bf16, any
        token and head strides that are multiples of 8 elements; cu_q and cu_k
        int32 [n + 1] on the device.  Returns out, or (out, lse)."""
        call = "packed_attention"
        dtype = q.dtype
        code = _dtype(call, dtype)
        _rows(call, "q", q, dtype, self.device)
        _rows(call, "k", k, dtype, self.device)
        _rows(call, "v", v, dtype, self.device, k.shape[1], k.shape[0])
        _ints(call, "cu_q", cu_q, self.device)
        _ints(call, "cu_k", cu_k, self.device, cu_q.numel())
        total_q, Hq = q.shape[0], q.shape[1]
        if out is None:
            out = q.new_empty(q.shape)
        else:
            _rows(call, "out", out, dtype, self.device, Hq, total_q)
        lse = _lse(call, lse, return_lse, q)
        p = Packed(cu_q.numel() - 1, Hq, k.shape[1], 128, code, int(bool(causal)), total_q, k.shape[0], scale,
                   q.stride(0), q.stride(1), k.stride(0), k.stride(1), v.stride(0), v.stride(1),
                   out.stride(0), out.stride(1))
        ref = ctypes.byref(p)
        with _on(self.device) as stream:
            for last in (False, True):
                ws = self._ws.current()
                status = lib().ra_packed_attention_fwd(
                    ref, q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_q.data_ptr(), cu_k.data_ptr(), out.data_ptr(),
                    None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.numel(), stream)
                if last or status != RA_ERR_WORKSPACE:
                    break
                self._ws.grow(packed_workspace_bytes(p))
            _check("ra_packed_attention_fwd", status)
        return (out, lse) if lse is not None else out

    def check(self) -> None:
        """Synchronises and raises what the calls' kernels reported."""
        self._ws.check()


class _on:
    """Makes a tensor's device the current one for a call; gives its current stream."""
    __slots__ = ("index", "before")

    def __init__(self, device):
        self.index, self.before = device.index, None

    def __enter__(self):
        import torch
        now = torch.cuda.current_device()
        if now != self.index:
            self.before = now
            torch.cuda.set_device(self.index)
        return torch._C._cuda_getCurrentRawStream(self.index)

    def __exit__(self, *exc):
        if self.before is not None:
            import torch
            torch.cuda.set_device(self.before)


def _lse(call: str, lse, wanted: bool, q):
    import torch
    rows = q.shape[:2]
    if lse is None:
        return q.new_empty(rows, dtype=torch.float32) if wanted else None
    if lse.shape != rows or lse.dtype != torch.float32 or lse.device != q.device or not lse.is_contiguous():
        raise _bad(call, f"lse: a contiguous float32 {list(rows)} tensor on {q.device}")
    return lse


class PagedCache:
    """A paged key/value cache: pool [2, layers, n_pages, Hkv, page_size, 128]
    (keys, values) and int32 state, owned through PyTorch, with the page
    operations and the attention over it on the current stream.  Calls of one
    object must not overlap on the GPU.  `pool` and `state` may be given: a
    state that describes the pool's contents, e.g. a copy of `.state`.
    `.refs`, `.lens` and `.table` are views of the state."""

    def __init__(self, layers: int, n_pages: int, page_size: int, Hkv: int, max_seqs: int, max_pages: int,
                 dtype=None, device="cuda", pool=None, state=None):
        import torch
        call = "paged_cache"
        self.dtype = torch.float16 if dtype is None else dtype
        self.p = CacheProblem(layers, n_pages, page_size, Hkv, 128, _dtype(call, self.dtype), max_seqs, max_pages)
        _check("ra_cache_validate", cache_validate(self.p))
        self.device = torch.empty(0, device=device).device
        shape = (2, layers, n_pages, Hkv, page_size, 128)
        ints = cache_state_bytes(self.p) // 4
        if pool is None:
            pool = torch.empty(shape, dtype=self.dtype, device=self.device)
        if pool.shape != shape or pool.dtype != self.dtype or pool.device != self.device or not pool.is_contiguous():
            raise _bad(call, f"pool: a contiguous {self.dtype} tensor {shape} on {self.device}")
        fresh = state is None
        if fresh:
            state = torch.empty((ints,), dtype=torch.int32, device=self.device)
        _ints(call, "state", state, self.device, ints)
        self.pool, self.state = pool, state
        self.c = cache_bind(self.p, pool, state)
        at = lambda ptr: (ptr - state.data_ptr()) // 4   # noqa: E731
        self.refs = state[:n_pages]
        self.lens = state[at(self.c.lens):at(self.c.lens) + max_seqs]
        self.table = state[at(self.c.table):at(self.c.table) + max_seqs * max_pages].view(max_seqs, max_pages)
        self._work = torch.zeros((cache_workspace_bytes(self.p),), dtype=torch.uint8, device=self.device)
        self._ws = _Workspace(self.device)
        self._rp, self._rc = ctypes.byref(self.p), ctypes.byref(self.c)
        if fresh:
            with _on(self.device):
                cache_init(self.p, self.c)

    def _call(self, name: str, *args) -> None:
        with _on(self.device) as stream:
            _check(name, getattr(lib(), name)(self._rp, self._rc, *args, self._work.data_ptr(), self._work.numel(), stream))

    def extend(self, seqs, n_new) -> None:
        """Rows `seqs` grow by `n_new` tokens (int32 device lists; -1 rows are passed over).
        Writes behind a refused extend pass its rows over until check() has
        raised it or another call has given the row slots."""
        _ints("cache_extend", "seqs", seqs, self.device)
        _ints("cache_extend", "n_new", n_new, self.device, seqs.numel())
        self._call("ra_cache_extend", seqs.data_ptr(), n_new.data_ptr(), seqs.numel())

    def write(self, layer: int, seqs, k, v, cu_new=None) -> None:
        """The last tokens of rows `seqs` in one layer: k, v [tokens, Hkv, 128];
        row i gets tokens cu_new[i] to cu_new[i + 1], or token i.  Into pages
        that no other row shares."""
        call = "cache_write"
        _ints(call, "seqs", seqs, self.device)
        if cu_new is not None:
            _ints(call, "cu_new", cu_new, self.device, seqs.numel() + 1)
        _rows(call, "k", k, self.dtype, self.device, self.p.Hkv)
        _rows(call, "v", v, self.dtype, self.device, self.p.Hkv, k.shape[0])
        (kt, kh, _), (vt, vh, _) = k.stride(), v.stride()
        self._call("ra_cache_write", layer, seqs.data_ptr(), None if cu_new is None else cu_new.data_ptr(), seqs.numel(),
                   k.shape[0], k.data_ptr(), v.data_ptr(), kt, kh, vt, vh)

    def fork(self, parents, children) -> None:
        """Empty rows `children` become copies of rows `parents`, sharing their full pages."""
        _ints("cache_fork", "parents", parents, self.device)
        _ints("cache_fork", "children", children, self.device, parents.numel())
        self._call("ra_cache_fork", parents.data_ptr(), children.data_ptr(), children.numel())

    def free(self, seqs) -> None:
        """Rows `seqs` become empty."""
        _ints("cache_free", "seqs", seqs, self.device)
        self._call("ra_cache_free", seqs.data_ptr(), seqs.numel())

    def compact(self) -> None:
        """Moves the n live pages to the first n places."""
        self._call("ra_cache_compact")

    def attention(self, layer: int, q, seqs, cu_q=None, shared: int = 0, scale: float = 0.0, out=None, lse=None,
                  return_lse: bool = False):
        """The newest tokens q [total_q, Hq, 128] of rows `seqs` (token i, or
        tokens cu_q[i] to cu_q[i + 1] of row i) over their sequences, whose
        first `shared` tokens lie in the same pages.  Returns out, or (out, lse)."""
        call = "cache_attention"
        _rows(call, "q", q, self.dtype, self.device)
        _ints(call, "seqs", seqs, self.device)
        if cu_q is not None:
            _ints(call, "cu_q", cu_q, self.device, seqs.numel() + 1)
        total_q, Hq = q.shape[0], q.shape[1]
        if out is None:
            out = q.new_empty(q.shape)
        else:
            _rows(call, "out", out, self.dtype, self.device, Hq, total_q)
        lse = _lse(call, lse, return_lse, q)
        a = CacheAttn(seqs.numel(), Hq, total_q, layer, shared, scale, q.stride(0), q.stride(1), out.stride(0),
                      out.stride(1))
        ref = ctypes.byref(a)
        with _on(self.device) as stream:
            for last in (False, True):
                ws = self._ws.current()
                status = lib().ra_cache_attention_fwd(
                    self._rp, self._rc, ref, q.data_ptr(), seqs.data_ptr(), None if cu_q is None else cu_q.data_ptr(),
                    out.data_ptr(), None if lse is None else lse.data_ptr(), ws.data_ptr(), ws.numel(), stream)
                if last or status != RA_ERR_WORKSPACE:
                    break
                self._ws.grow(cache_attention_workspace_bytes(self.p, a))
            _check("ra_cache_attention_fwd", status)
        return (out, lse) if lse is not None else out

    def check(self) -> None:
        """Synchronises and raises what the calls' kernels reported."""
        with _on(self.device):
            check_device_error(self._work)
        self._ws.check()


class RotateAttention:
    """Owns (through PyTorch) the workspace and the quantised-QKV buffer of one
    problem and calls the C entry points on the current stream."""

    def __init__(self, cfg, device="cuda", fp16_path: bool = True):
        import torch
        self.cfg = cfg
        self.p = problem(cfg)
        _check("ra_validate", validate(self.p))
        self.N = seq_len(self.p)
        self.N_pad = seq_pad(self.p)
        self.device = torch.device(device)
        self.workspace = torch.empty((workspace_bytes(self.p, fp16_path),), dtype=torch.uint8, device=self.device)
        self.qkv4_buf = torch.empty((qkv4_bytes(self.p),), dtype=torch.uint8, device=self.device)
        self.qkv4 = qkv4_bind(self.p, self.qkv4_buf)
        prepare(self.p, self.workspace)

    def rotate_quantize(self, q, k, v) -> Qkv4:
        rotate_quantize_qkv(self.p, q, k, v, self.qkv4, self.workspace)
        return self.qkv4

    def int4_attention(self, out=None):
        import torch
        if out is None:
            out = torch.empty((self.cfg.B, self.cfg.H, self.N, self.cfg.d), dtype=torch.float16, device=self.device)
        int4_attention_fwd(self.p, self.qkv4, out, self.workspace)
        return out

    def fp16_attention(self, q, k, v, out=None):
        import torch
        if out is None:
            out = torch.empty_like(q)
        fp16_attention_fwd(self.p, q, k, v, out, self.workspace)
        return out

    def forward(self, q, k, v, path: str = "int4", out=None):
        if path == "int4":
            self.rotate_quantize(q, k, v)
            return self.int4_attention(out)
        if path == "fp16":
            return self.fp16_attention(q, k, v, out)
        raise ValueError(path)

    def forward_host(self, q, k, v, out, heads_per_chunk: int = 0):
        """INT4 path on host tensors (q, k, v, out on the CPU, page-locked for
        overlap): copies, kernels and copies back pipelined over head chunks
        by the library.  Returns once out is written."""
        import torch
        need = host_staging_bytes(self.p, heads_per_chunk)
        if getattr(self, "_staging", None) is None or self._staging.numel() < need:
            self._staging = torch.empty((need,), dtype=torch.uint8, device=self.device)
        int4_attention_host(self.p, q, k, v, out, self._staging, heads_per_chunk)
        return out

    def check(self) -> None:
        check_device_error(self.workspace)

    def unpack(self):
        """Host copies of the quantised tensors (int8 codes, unpacked), for tests."""
        import numpy as np
        import torch
        BH, Np = self.cfg.B * self.cfg.H, self.N_pad
        torch.cuda.synchronize()
        buf = self.qkv4_buf.cpu().numpy()
        base = self.qkv4_buf.data_ptr()

        def view(ptr, nbytes, dtype):
            off = ptr - base
            return buf[off:off + nbytes].view(dtype)

        packed = BH * Np * 64
        q4 = view(self.qkv4.q4, packed, np.uint8).reshape(BH, Np, 64)
        k4 = view(self.qkv4.k4, packed, np.uint8).reshape(BH, Np, 64)
        v4t = view(self.qkv4.v4t, packed, np.uint8).reshape(BH, Np // 128, 128, 64)
        sq = view(self.qkv4.sq, BH * (Np // 64) * 4, np.float32).reshape(BH, Np // 64)
        sk = view(self.qkv4.sk, BH * (Np // 64) * 4, np.float32).reshape(BH, Np // 64)
        sv = view(self.qkv4.sv, BH * 128 * 4, np.float32).reshape(BH, 128)
        vsum = view(self.qkv4.vsum, BH * (Np // 64) * 128 * 4, np.int32).reshape(BH, Np // 64, 128)
        return dict(qc=unpack_nibbles(q4), kc=unpack_nibbles(k4),
                    vc=np.ascontiguousarray(unpack_nibbles(v4t).transpose(0, 1, 3, 2).reshape(BH, Np, 128)),
                    qs=sq, ks=sk, sv=sv, colsum=vsum)


def unpack_nibbles(packed):
    """uint8 [..., n] with two's-complement nibbles -> int8 [..., 2n], low nibble first."""
    import numpy as np
    lo = (packed & 0x0F).astype(np.int8)
    hi = (packed >> 4).astype(np.int8)
    lo = np.where(lo > 7, lo - 16, lo).astype(np.int8)
    hi = np.where(hi > 7, hi - 16, hi).astype(np.int8)
    out = np.empty(packed.shape[:-1] + (packed.shape[-1] * 2,), np.int8)
    out[..., 0::2] = lo
    out[..., 1::2] = hi
    return out
