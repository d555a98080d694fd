"""ctypes binding of libfa.so: the C ABI of include/fa.h, same names.

Argument marshalling only -- every step of the computation runs in the CUDA
kernels.  There is no fallback: if the library has not been built, or a call
returns an error status, the call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "_build", "libfa.so")

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_WORKSPACE, FA_ERR_CUDA, FA_ERR_TIMEOUT = range(6)
FA_FP16, FA_BF16 = 0, 1

EXPORTS = (
    "fa_fwd", "fa_fwd_local", "fa_bwd_local", "fa_fwd_varlen", "fa_bwd_varlen", "fa_bwd_varlen_workspace_bytes",
    "fa_bwd", "fa_bwd_workspace_bytes", "fa_bwd_two_pass", "fa_bwd_two_pass_workspace_bytes",
    "fa_bwd_noalloc", "fa_hadamard_quant_fp8",
    "fa_hadamard_quant_workspace_bytes", "fa_fwd_fp8", "fa_get_device_status",
    "fa_selftest_bounded_wait", "fa_status_string", "fa_fwd_f32_out", "fa_probe_exp2", "fa_fwd_persistent",
    "fa_paged_tables", "fa_paged_append", "fa_fwd_paged", "fa_fwd_paged_prefix", "fa_fwd_paged_workspace_bytes",
    "fa_fwd_paged_tree", "fa_fwd_paged_tree_workspace_bytes", "fa_paged_fork", "fa_paged_copy", "fa_paged_compact", "fa_paged_free",
)

_lock = threading.Lock()
_lib = None


class FAError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed: {msg} ({status})")
        self.status = status


def load():
    """Load libfa.so (it must already be built: ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing "
                               "(run __graft_entry__.build()); there is no fallback path")
        lib = ctypes.CDLL(LIB_PATH)
        P, I, F, Z, L = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_long
        lib.fa_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, I, P]
        lib.fa_fwd_local.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, I, P]
        lib.fa_fwd_f32_out.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, I, P]
        lib.fa_fwd_persistent.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, I, P]
        lib.fa_bwd_local.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, I, P, Z, P]
        lib.fa_fwd_varlen.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, I, P]
        lib.fa_bwd_varlen.argtypes = [P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, I, I, P, Z, P]
        lib.fa_bwd_varlen_workspace_bytes.argtypes = [I, I, I, I]
        lib.fa_bwd_varlen_workspace_bytes.restype = Z
        lib.fa_bwd.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, P, Z, P]
        lib.fa_bwd_two_pass.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, P, Z, P]
        lib.fa_bwd_two_pass_workspace_bytes.argtypes = [I, I, I, I]
        lib.fa_bwd_two_pass_workspace_bytes.restype = Z
        lib.fa_bwd_noalloc.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, P]
        lib.fa_bwd_workspace_bytes.argtypes = [I, I, I, I]
        lib.fa_bwd_workspace_bytes.restype = Z
        lib.fa_hadamard_quant_fp8.argtypes = [P, P, P, P, L, I, P, Z, P]
        lib.fa_hadamard_quant_workspace_bytes.argtypes = [L, I]
        lib.fa_hadamard_quant_workspace_bytes.restype = Z
        lib.fa_fwd_fp8.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, P]
        lib.fa_paged_tables.argtypes = [P] * 9 + [I] * 6 + [P]
        lib.fa_paged_append.argtypes = [P] * 5 + [I] * 6 + [P]
        lib.fa_paged_fork.argtypes = [P] * 9 + [I] * 6 + [P]
        lib.fa_paged_copy.argtypes = [P] * 5 + [I] * 6 + [P]
        lib.fa_paged_compact.argtypes = [P] * 6 + [I] * 8 + [P]
        lib.fa_paged_free.argtypes = [P] * 7 + [I] * 5 + [P]
        lib.fa_fwd_paged.argtypes = [P] * 8 + [I] * 10 + [F, I, P, Z, P]
        lib.fa_fwd_paged_prefix.argtypes = [P] * 4 + [I] + [P] * 5 + [I] * 10 + [F, I, P, Z, P]
        lib.fa_fwd_paged_tree.argtypes = [P] * 9 + [I] * 10 + [F, I, P, Z, P]
        lib.fa_fwd_paged_tree_workspace_bytes.argtypes = [I] * 8
        lib.fa_fwd_paged_tree_workspace_bytes.restype = Z
        lib.fa_fwd_paged_workspace_bytes.argtypes = [I] * 9
        lib.fa_fwd_paged_workspace_bytes.restype = Z
        lib.fa_get_device_status.argtypes = [P]
        lib.fa_selftest_bounded_wait.argtypes = [I, P]
        lib.fa_probe_exp2.argtypes = [P, I, I, P]
        lib.fa_probe_exp2.restype = ctypes.c_longlong
        lib.fa_status_string.argtypes = [I]
        lib.fa_status_string.restype = ctypes.c_char_p
        for name in ("fa_fwd", "fa_fwd_local", "fa_fwd_f32_out", "fa_fwd_persistent", "fa_bwd_local", "fa_fwd_varlen", "fa_bwd_varlen",
                     "fa_bwd", "fa_bwd_two_pass", "fa_bwd_noalloc", "fa_hadamard_quant_fp8", "fa_fwd_fp8",
                     "fa_paged_tables", "fa_paged_append", "fa_fwd_paged", "fa_fwd_paged_prefix", "fa_fwd_paged_tree", "fa_paged_fork",
                     "fa_paged_copy", "fa_paged_compact", "fa_paged_free", "fa_get_device_status", "fa_selftest_bounded_wait"):
            getattr(lib, name).restype = I
        _lib = lib
        return lib


def _check(fn: str, status: int):
    if status != FA_OK:
        msg = load().fa_status_string(status).decode()
        raise FAError(fn, status, msg)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        # torch.cuda.current_stream().cuda_stream without the Stream object
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _handle(stream, dev: int) -> int | None:
    """_stream for a call whose tensors are known to be on the current device, `dev`."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return FA_BF16
    if t.dtype == torch.float16:
        return FA_FP16
    raise TypeError(f"unsupported element type {t.dtype}")


def _need(name, t, dtypes=()):
    """Refuses a tensor the C call cannot take: the library receives bare
    pointers, so a wrong element type or a strided view would be read as
    something else without any error."""
    if t is None:
        return
    if dtypes and t.dtype not in dtypes:
        raise TypeError(f"{name}: element type {t.dtype}, expected {' or '.join(str(x) for x in dtypes)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensor must be contiguous")


def _io16(q, lse=None, f32=(), **same):
    """Checks a 16-bit call's tensors (q's element type for `same`, fp32
    for lse and `f32`) and returns q's type code."""
    import torch
    code = _dtype_code(q)
    _need("q", q)
    for name, t in same.items():
        _need(name, t, (q.dtype,))
    for name, t in (("lse", lse),) + tuple(f32):
        _need(name, t, (torch.float32,))
    return code


def _dims(q, k):
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    return B, Hq, Hkv, N, d


def fa_fwd(q, k, v, o, lse, causal: bool, scale: float, stream=None):
    """O and LSE for q [B,Hq,N,d], k/v [B,Hkv,N,d] (contiguous CUDA tensors)."""
    B, Hq, Hkv, N, d = _dims(q, k)
    code = _io16(q, lse, k=k, v=v, o=o)
    _check("fa_fwd", load().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, N, d,
                                   int(causal), float(scale), code, _stream(stream)))


def fa_fwd_persistent(q, k, v, o, lse, causal: bool, scale: float, stream=None):
    """fa_fwd as the persistent kernel (dynamic block schedule); same results."""
    B, Hq, Hkv, N, d = _dims(q, k)
    code = _io16(q, lse, k=k, v=v, o=o)
    _check("fa_fwd_persistent", load().fa_fwd_persistent(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq,
                                                         Hkv, N, d, int(causal), float(scale), code,
                                                         _stream(stream)))


def fa_fwd_f32_out(q, k, v, o_f32, lse, causal: bool, scale: float, stream=None):
    """fa_fwd with O written in fp32 (o_f32 [B,Hq,N,d] float32): the
    normalised accumulator before rounding to the input type."""
    B, Hq, Hkv, N, d = _dims(q, k)
    code = _io16(q, lse, f32=(("o_f32", o_f32),), k=k, v=v)
    _check("fa_fwd_f32_out", load().fa_fwd_f32_out(_ptr(q), _ptr(k), _ptr(v), _ptr(o_f32), _ptr(lse), B, Hq, Hkv,
                                                   N, d, int(causal), float(scale), code, _stream(stream)))


def fa_fwd_local(q, k, v, o, lse, window: int, scale: float, stream=None):
    """Causal sliding-window forward: row r sees keys r - window + 1 .. r."""
    B, Hq, Hkv, N, d = _dims(q, k)
    code = _io16(q, lse, k=k, v=v, o=o)
    _check("fa_fwd_local", load().fa_fwd_local(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, Hq, Hkv, N, d,
                                               int(window), float(scale), code, _stream(stream)))


def fa_bwd_local(q, k, v, o, lse, dO, dq, dk, dv, window: int, scale: float, deterministic: bool, workspace,
                 stream=None):
    B, Hq, Hkv, N, d = _dims(q, k)
    code = _io16(q, lse, k=k, v=v, o=o, dO=dO, dq=dq, dk=dk, dv=dv)
    _need("workspace", workspace)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("fa_bwd_local", load().fa_bwd_local(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk), _ptr(dv), B, Hq, Hkv, N, d,
        int(window), float(scale), code, int(bool(deterministic)), _ptr(workspace), ws_bytes,
        _stream(stream)))


def fa_fwd_varlen(q, k, v, o, lse, cu_seqlens, max_seqlen: int, causal: bool, scale: float, window: int = 0,
                  stream=None):
    """Packed sequences: q/o [total,Hq,d], k/v [total,Hkv,d], lse [Hq,total],
    cu_seqlens int32 [B+1] on the device."""
    import torch
    total, Hq, d = q.shape
    Hkv = k.shape[1]
    B = cu_seqlens.numel() - 1
    code = _io16(q, lse, k=k, v=v, o=o)
    _need("cu_seqlens", cu_seqlens, (torch.int32,))
    _check("fa_fwd_varlen", load().fa_fwd_varlen(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(cu_seqlens), B, int(max_seqlen), total, Hq, Hkv, d,
        int(causal), int(window), float(scale), code, _stream(stream)))


def fa_bwd_varlen_workspace_bytes(total: int, Hq: int, d: int, deterministic: bool) -> int:
    return int(load().fa_bwd_varlen_workspace_bytes(total, Hq, d, int(bool(deterministic))))


def fa_bwd_varlen(q, k, v, o, lse, dO, dq, dk, dv, cu_seqlens, max_seqlen: int, causal: bool, scale: float,
                  deterministic: bool, workspace, window: int = 0, stream=None):
    import torch
    total, Hq, d = q.shape
    Hkv = k.shape[1]
    B = cu_seqlens.numel() - 1
    code = _io16(q, lse, k=k, v=v, o=o, dO=dO, dq=dq, dk=dk, dv=dv)
    _need("cu_seqlens", cu_seqlens, (torch.int32,))
    _need("workspace", workspace)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("fa_bwd_varlen", load().fa_bwd_varlen(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(cu_seqlens),
        B, int(max_seqlen), total, Hq, Hkv, d, int(causal), int(window), float(scale), code,
        int(bool(deterministic)), _ptr(workspace), ws_bytes, _stream(stream)))


def fa_bwd_workspace_bytes(B: int, Hq: int, N: int, d: int) -> int:
    return int(load().fa_bwd_workspace_bytes(B, Hq, N, d))


def fa_bwd(q, k, v, o, lse, dO, dq, dk, dv, causal: bool, scale: float, workspace, stream=None):
    B, Hq, Hkv, N, d = _dims(q, k)
    code = _io16(q, lse, k=k, v=v, o=o, dO=dO, dq=dq, dk=dk, dv=dv)
    _need("workspace", workspace)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("fa_bwd", load().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq),
                                   _ptr(dk), _ptr(dv), B, Hq, Hkv, N, d, int(causal), float(scale),
                                   code, _ptr(workspace), ws_bytes, _stream(stream)))


def fa_bwd_two_pass_workspace_bytes(B: int, Hq: int, N: int, d: int) -> int:
    return int(load().fa_bwd_two_pass_workspace_bytes(B, Hq, N, d))


def fa_bwd_two_pass(q, k, v, o, lse, dO, dq, dk, dv, causal: bool, scale: float, workspace, stream=None):
    """Deterministic backward: dQ from a second pass over Q tiles, no atomics."""
    B, Hq, Hkv, N, d = _dims(q, k)
    code = _io16(q, lse, k=k, v=v, o=o, dO=dO, dq=dq, dk=dk, dv=dv)
    _need("workspace", workspace)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("fa_bwd_two_pass", load().fa_bwd_two_pass(
        _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq), _ptr(dk), _ptr(dv), B, Hq, Hkv,
        N, d, int(causal), float(scale), code, _ptr(workspace), ws_bytes, _stream(stream)))


def fa_bwd_noalloc(q, k, v, o, lse, dO, dq, dk, dv, causal: bool, scale: float, stream=None):
    """fa_bwd using the library's built-in scratch buffer instead of a
    caller workspace: for callers that cannot allocate device memory.  Calls
    that may overlap on the GPU race on that buffer."""
    B, Hq, Hkv, N, d = _dims(q, k)
    code = _io16(q, lse, k=k, v=v, o=o, dO=dO, dq=dq, dk=dk, dv=dv)
    _check("fa_bwd_noalloc", load().fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO),
                                                   _ptr(dq), _ptr(dk), _ptr(dv), B, Hq, Hkv, N, d, int(causal),
                                                   float(scale), code, _stream(stream)))


def fa_hadamard_quant_workspace_bytes(rows: int, d: int) -> int:
    return int(load().fa_hadamard_quant_workspace_bytes(rows, d))


def _byte_types():
    import torch
    return (torch.float8_e4m3fn, torch.uint8)


def fa_hadamard_quant_fp8(x, signs, x8, descale, workspace, stream=None):
    """x bf16 (the only input type of the C call), x8 e4m3 bytes, signs and
    descale fp32."""
    import torch
    _need("x", x, (torch.bfloat16,))
    _need("signs", signs, (torch.float32,))
    _need("x8", x8, _byte_types())
    _need("descale", descale, (torch.float32,))
    _need("workspace", workspace)
    d = x.shape[-1]
    rows = x.numel() // d
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("fa_hadamard_quant_fp8", load().fa_hadamard_quant_fp8(
        _ptr(x), _ptr(signs), _ptr(x8), _ptr(descale), rows, d, _ptr(workspace), ws_bytes,
        _stream(stream)))


def fa_fwd_fp8(q8, k8, v8, q_descale, k_descale, v_descale, o, lse, causal: bool, scale: float,
               stream=None):
    import torch
    B, Hq, Hkv, N, d = _dims(q8, k8)
    for name, t in (("q8", q8), ("k8", k8), ("v8", v8)):
        _need(name, t, _byte_types())
    for name, t in (("q_descale", q_descale), ("k_descale", k_descale), ("v_descale", v_descale), ("lse", lse)):
        _need(name, t, (torch.float32,))
    _need("o", o, (torch.bfloat16,))
    _check("fa_fwd_fp8", load().fa_fwd_fp8(
        _ptr(q8), _ptr(k8), _ptr(v8), _ptr(q_descale), _ptr(k_descale), _ptr(v_descale), _ptr(o),
        _ptr(lse), B, Hq, Hkv, N, d, int(causal), float(scale), _stream(stream)))


def _refuse(name, t, device: int):
    import torch
    if device < 0 or t.get_device() != device:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{torch.cuda.current_device() if device < 0 else device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensor must be contiguous")
    raise TypeError(f"{name}: element type {t.dtype}")


def _need_all(*tensors) -> int:
    """Refuses what a paged call's pointers cannot take: (name, tensor, type)
    triples off the current device (where the library launches), of another
    type, or not contiguous.  None passes.  Returns the device's index."""
    import torch
    device = tensors[0][1].get_device()
    if device < 0:
        raise ValueError(f"{tensors[0][0]}: expected a CUDA tensor, got one on {tensors[0][1].device}")
    if device != torch.cuda.current_device():
        raise ValueError(f"tensors are on cuda:{device}, the current device is cuda:{torch.cuda.current_device()}")
    for name, t, dtype in tensors:
        if t is not None and (t.get_device() != device or t.dtype != dtype or not t.is_contiguous()):
            _refuse(name, t, device)
    return device


def _need_numel(**tensors):
    for name, (t, n) in tensors.items():
        if t is not None and t.numel() != n:
            raise ValueError(f"{name}: {t.numel()} elements, expected {n}")


def _need_int32(**values):
    # ctypes would pass the low 32 bits of a larger one
    for name, x in values.items():
        if not -0x80000000 <= x <= 0x7FFFFFFF:
            raise ValueError(f"{name}: {x} does not fit 32 bits")


def fa_paged_tables(cached_lens, new_lens, free_pages, free_start, block_table, seq_lens, cu_seqlens, slots, counts,
                    page_size: int, num_pages: int, stream=None):
    """Pages and slots for a step's new tokens; int32 tensors as in fa.h."""
    import torch
    B, max_pages = block_table.shape
    i32, dev = torch.int32, block_table.get_device()
    # the checks of _need_all and _need_numel in one expression: the kernel
    # takes some 4 us, so they would be a good part of a call
    if not (dev >= 0 and dev == torch.cuda.current_device() and block_table.dtype == i32 and block_table.is_contiguous()
            and cached_lens.get_device() == dev and cached_lens.dtype == i32 and cached_lens.is_contiguous()
            and new_lens.get_device() == dev and new_lens.dtype == i32 and new_lens.is_contiguous()
            and free_pages.get_device() == dev and free_pages.dtype == i32 and free_pages.is_contiguous()
            and seq_lens.get_device() == dev and seq_lens.dtype == i32 and seq_lens.is_contiguous()
            and cu_seqlens.get_device() == dev and cu_seqlens.dtype == i32 and cu_seqlens.is_contiguous()
            and slots.get_device() == dev and slots.dtype == i32 and slots.is_contiguous()
            and counts.get_device() == dev and counts.dtype == i32 and counts.is_contiguous()
            and (free_start is None or (free_start.get_device() == dev and free_start.dtype == i32
                                        and free_start.numel() == 1))
            and cached_lens.numel() == B and new_lens.numel() == B and seq_lens.numel() == B
            and cu_seqlens.numel() == B + 1 and counts.numel() == 2):
        _need_all(("block_table", block_table, i32), ("cached_lens", cached_lens, i32), ("new_lens", new_lens, i32),
                  ("free_pages", free_pages, i32), ("free_start", free_start, i32), ("seq_lens", seq_lens, i32),
                  ("cu_seqlens", cu_seqlens, i32), ("slots", slots, i32), ("counts", counts, i32))
        _need_numel(cached_lens=(cached_lens, B), new_lens=(new_lens, B), free_start=(free_start, 1),
                    seq_lens=(seq_lens, B), cu_seqlens=(cu_seqlens, B + 1), counts=(counts, 2))
    num_free, total = free_pages.numel(), slots.numel()
    # a tensor's sizes too: ctypes would pass their low 32 bits
    if not (0 < page_size <= 0x7FFFFFFF and 0 < num_pages <= 0x7FFFFFFF and B <= 0x7FFFFFFF
            and max_pages <= 0x7FFFFFFF and num_free <= 0x7FFFFFFF and total <= 0x7FFFFFFF):
        _need_int32(page_size=page_size, num_pages=num_pages, B=B, max_pages=max_pages, free_pages=num_free,
                    total=total)
    _check("fa_paged_tables", load().fa_paged_tables(
        cached_lens.data_ptr(), new_lens.data_ptr(), free_pages.data_ptr() if num_free else None, _ptr(free_start),
        block_table.data_ptr(), seq_lens.data_ptr(), cu_seqlens.data_ptr(), slots.data_ptr(), counts.data_ptr(), B,
        max_pages, int(page_size), int(num_pages), num_free, total, _stream(stream)))


def fa_paged_append(k, v, slots, k_cache, v_cache, stream=None):
    """Writes k, v [total,Hkv,d] into slots of the caches [pages,Hkv,page_size,d]."""
    import torch
    total, Hkv, d = k.shape
    shape = k_cache.shape
    num_pages, heads, page_size, dc = shape
    code, dtype, dev = _dtype_code(k), k.dtype, k.get_device()
    if not (dev >= 0 and dev == torch.cuda.current_device() and k.is_contiguous()
            and v.get_device() == dev and v.dtype == dtype and v.is_contiguous()
            and slots.get_device() == dev and slots.dtype == torch.int32 and slots.is_contiguous()
            and slots.numel() == total
            and k_cache.get_device() == dev and k_cache.dtype == dtype and k_cache.is_contiguous()
            and v_cache.get_device() == dev and v_cache.dtype == dtype and v_cache.is_contiguous()):
        _need_all(("k", k, dtype), ("v", v, dtype), ("slots", slots, torch.int32), ("k_cache", k_cache, dtype),
                  ("v_cache", v_cache, dtype))
        _need_numel(slots=(slots, total))
    if v.shape != k.shape or v_cache.shape != shape or heads != Hkv or dc != d:
        raise ValueError("k, v must be [total,Hkv,d] and the caches [pages,Hkv,page_size,d] of the same heads")
    _check("fa_paged_append", load().fa_paged_append(
        k.data_ptr(), v.data_ptr(), slots.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), total, Hkv, d, page_size,
        num_pages, code, _stream(stream)))


def fa_paged_fork(src, dst, seq_lens, block_table, free_pages, free_start, shares, copies, counts, page_size: int,
                  stream=None):
    """Table rows dst continue where rows src stand; int32 tensors as in fa.h."""
    import torch
    B, max_pages = block_table.shape
    F, num_pages, num_free = src.numel(), shares.numel(), free_pages.numel()
    i32, dev = torch.int32, block_table.get_device()
    # one expression, as for the tables: the kernel takes some 4 us
    if not (dev >= 0 and dev == torch._C._cuda_getDevice() and block_table.dtype == i32 and block_table.is_contiguous()
            and src.get_device() == dev and src.dtype == i32 and src.is_contiguous()
            and dst.get_device() == dev and dst.dtype == i32 and dst.is_contiguous()
            and seq_lens.get_device() == dev and seq_lens.dtype == i32 and seq_lens.is_contiguous()
            and free_pages.get_device() == dev and free_pages.dtype == i32 and free_pages.is_contiguous()
            and shares.get_device() == dev and shares.dtype == i32 and shares.is_contiguous()
            and copies.get_device() == dev and copies.dtype == i32 and copies.is_contiguous()
            and counts.get_device() == dev and counts.dtype == i32 and counts.is_contiguous()
            and (free_start is None or (free_start.get_device() == dev and free_start.dtype == i32
                                        and free_start.numel() == 1))
            and dst.numel() == F and seq_lens.numel() == B and copies.numel() == 3 * F and counts.numel() == 2):
        _need_all(("block_table", block_table, i32), ("src", src, i32), ("dst", dst, i32), ("seq_lens", seq_lens, i32),
                  ("free_pages", free_pages, i32), ("free_start", free_start, i32), ("shares", shares, i32),
                  ("copies", copies, i32), ("counts", counts, i32))
        _need_numel(dst=(dst, F), seq_lens=(seq_lens, B), copies=(copies, 3 * F), counts=(counts, 2),
                    free_start=(free_start, 1))
    if not (0 < page_size <= 0x7FFFFFFF and F <= 0x7FFFFFFF and B <= 0x7FFFFFFF and max_pages <= 0x7FFFFFFF
            and num_pages <= 0x7FFFFFFF and num_free <= 0x7FFFFFFF):
        _need_int32(page_size=page_size, src=F, B=B, max_pages=max_pages, shares=num_pages, free_pages=num_free)
    _check("fa_paged_fork", load().fa_paged_fork(
        src.data_ptr(), dst.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(),
        free_pages.data_ptr() if num_free else None, _ptr(free_start), shares.data_ptr(), copies.data_ptr(),
        counts.data_ptr(), F, B, max_pages, int(page_size), num_pages, num_free, _handle(stream, dev)))


def fa_paged_copy(src, dst, rows, k_cache, v_cache, stream=None):
    """Pages dst of the caches [pages,Hkv,page_size,d] get the first rows tokens of pages src."""
    import torch
    shape = k_cache.shape
    num_pages, Hkv, page_size, d = shape
    code, dtype, dev, i32, n = _dtype_code(k_cache), k_cache.dtype, k_cache.get_device(), torch.int32, src.numel()
    if not (dev >= 0 and dev == torch._C._cuda_getDevice() and k_cache.is_contiguous()
            and v_cache.get_device() == dev and v_cache.dtype == dtype and v_cache.is_contiguous()
            and src.get_device() == dev and src.dtype == i32 and src.is_contiguous()
            and dst.get_device() == dev and dst.dtype == i32 and dst.is_contiguous() and dst.numel() == n
            and (rows is None or (rows.get_device() == dev and rows.dtype == i32 and rows.is_contiguous()
                                  and rows.numel() == n))):
        _need_all(("k_cache", k_cache, dtype), ("v_cache", v_cache, dtype), ("src", src, i32), ("dst", dst, i32),
                  ("rows", rows, i32))
        _need_numel(dst=(dst, n), rows=(rows, n))
    if v_cache.shape != shape:
        raise ValueError("the caches must both be [pages,Hkv,page_size,d]")
    if n > 0x7FFFFFFF:
        _need_int32(src=n)
    _check("fa_paged_copy", load().fa_paged_copy(
        src.data_ptr(), dst.data_ptr(), _ptr(rows), k_cache.data_ptr(), v_cache.data_ptr(), n, Hkv, d, page_size,
        num_pages, code, _handle(stream, dev)))


def fa_paged_compact(keep, keep_lens, base_lens, block_table, k_cache, v_cache, stream=None):
    """Tokens base_lens + keep [B,max_keep] of the requests move to base_lens + 0, 1, .."""
    import torch
    B, max_pages = block_table.shape
    shape = k_cache.shape
    num_pages, Hkv, page_size, d = shape
    code, dtype, dev, i32 = _dtype_code(k_cache), k_cache.dtype, k_cache.get_device(), torch.int32
    if not (dev >= 0 and dev == torch._C._cuda_getDevice() and k_cache.is_contiguous()
            and v_cache.get_device() == dev and v_cache.dtype == dtype and v_cache.is_contiguous()
            and block_table.get_device() == dev and block_table.dtype == i32 and block_table.is_contiguous()
            and keep.get_device() == dev and keep.dtype == i32 and keep.is_contiguous()
            and keep_lens.get_device() == dev and keep_lens.dtype == i32 and keep_lens.is_contiguous()
            and base_lens.get_device() == dev and base_lens.dtype == i32 and base_lens.is_contiguous()):
        _need_all(("k_cache", k_cache, dtype), ("v_cache", v_cache, dtype), ("block_table", block_table, i32),
                  ("keep", keep, i32), ("keep_lens", keep_lens, i32), ("base_lens", base_lens, i32))
    if v_cache.shape != shape:
        raise ValueError("the caches must both be [pages,Hkv,page_size,d]")
    if keep.dim() != 2 or keep.shape[0] != B or keep_lens.numel() != B or base_lens.numel() != B:
        raise ValueError(f"keep must be [B,max_keep], keep_lens and base_lens [B], with the table's B = {B}")
    max_keep = keep.shape[1]
    if not (B <= 0x7FFFFFFF and max_keep <= 0x7FFFFFFF and max_pages <= 0x7FFFFFFF):
        _need_int32(B=B, max_keep=max_keep, max_pages=max_pages)
    _check("fa_paged_compact", load().fa_paged_compact(
        keep.data_ptr(), keep_lens.data_ptr(), base_lens.data_ptr(), block_table.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), B, max_keep, max_pages, Hkv, d, page_size, num_pages, code, _handle(stream, dev)))


def fa_paged_free(old_lens, new_lens, block_table, free_pages, free_start, shares, counts, page_size: int,
                  num_pages: int, stream=None):
    """Pages behind new_lens back to the free list; int32 tensors as in fa.h."""
    import torch
    B, max_pages = block_table.shape
    num_free = free_pages.numel()
    i32, dev = torch.int32, block_table.get_device()
    if not (dev >= 0 and dev == torch._C._cuda_getDevice() and block_table.dtype == i32 and block_table.is_contiguous()
            and old_lens.get_device() == dev and old_lens.dtype == i32 and old_lens.is_contiguous()
            and new_lens.get_device() == dev and new_lens.dtype == i32 and new_lens.is_contiguous()
            and free_pages.get_device() == dev and free_pages.dtype == i32 and free_pages.is_contiguous()
            and free_start.get_device() == dev and free_start.dtype == i32 and free_start.numel() == 1
            and counts.get_device() == dev and counts.dtype == i32 and counts.is_contiguous()
            and (shares is None or (shares.get_device() == dev and shares.dtype == i32 and shares.is_contiguous()
                                    and shares.numel() == num_pages))
            and old_lens.numel() == B and new_lens.numel() == B and counts.numel() == 2):
        _need_all(("block_table", block_table, i32), ("old_lens", old_lens, i32), ("new_lens", new_lens, i32),
                  ("free_pages", free_pages, i32), ("free_start", free_start, i32), ("shares", shares, i32),
                  ("counts", counts, i32))
        _need_numel(old_lens=(old_lens, B), new_lens=(new_lens, B), free_start=(free_start, 1), counts=(counts, 2),
                    shares=(shares, num_pages))
    if not (0 < page_size <= 0x7FFFFFFF and 0 < num_pages <= 0x7FFFFFFF and B <= 0x7FFFFFFF
            and max_pages <= 0x7FFFFFFF and num_free <= 0x7FFFFFFF):
        _need_int32(page_size=page_size, num_pages=num_pages, B=B, max_pages=max_pages, free_pages=num_free)
    _check("fa_paged_free", load().fa_paged_free(
        old_lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(), free_pages.data_ptr() if num_free else None,
        free_start.data_ptr(), _ptr(shares), counts.data_ptr(), B, max_pages, int(page_size), int(num_pages), num_free,
        _handle(stream, dev)))


@functools.lru_cache(maxsize=1024)  # a function of the sizes alone
def fa_fwd_paged_workspace_bytes(B: int, total: int, max_new: int, Hq: int, Hkv: int, d: int, max_pages: int,
                                 page_size: int, prefix_len: int = 0) -> int:
    return int(load().fa_fwd_paged_workspace_bytes(B, total, max_new, Hq, Hkv, d, max_pages, page_size, prefix_len))


def _paged_call(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens, o, lse, max_new, scale, workspace, window,
                prefix=None):
    """Checks shared by the paged forwards; returns the arguments that follow
    the tables in the C call, but for the stream."""
    import torch
    total, Hq, d = q.shape
    shape = k_cache.shape
    num_pages, Hkv, page_size, dc = shape
    B, max_pages = block_table.shape
    code, dtype, i32, dev = _dtype_code(q), q.dtype, torch.int32, q.get_device()
    # the checks of _need_all and _need_numel in one expression: a call is a
    # few microseconds of kernel at times, and this is part of every one
    if not (dev >= 0 and dev == torch.cuda.current_device() and q.is_contiguous()
            and k_cache.get_device() == dev and k_cache.dtype == dtype and k_cache.is_contiguous()
            and v_cache.get_device() == dev and v_cache.dtype == dtype and v_cache.is_contiguous()
            and block_table.get_device() == dev and block_table.dtype == i32 and block_table.is_contiguous()
            and seq_lens.get_device() == dev and seq_lens.dtype == i32 and seq_lens.is_contiguous()
            and o.get_device() == dev and o.dtype == dtype and o.is_contiguous()
            and lse.get_device() == dev and lse.dtype == torch.float32 and lse.is_contiguous()
            and seq_lens.numel() == B
            and (cu_seqlens is None or (cu_seqlens.get_device() == dev and cu_seqlens.dtype == i32
                                        and cu_seqlens.is_contiguous() and cu_seqlens.numel() == B + 1))
            and (prefix is None or (prefix.get_device() == dev and prefix.dtype == i32 and prefix.is_contiguous()))
            and (workspace is None or (workspace.get_device() == dev and workspace.dtype == torch.uint8
                                       and workspace.is_contiguous()))):
        _need_all(("q", q, dtype), ("k_cache", k_cache, dtype), ("v_cache", v_cache, dtype),
                  ("block_table", block_table, i32), ("seq_lens", seq_lens, i32), ("cu_seqlens", cu_seqlens, i32),
                  ("prefix_pages", prefix, i32), ("o", o, dtype), ("lse", lse, torch.float32),
                  ("workspace", workspace, torch.uint8))
        _need_numel(seq_lens=(seq_lens, B), cu_seqlens=(cu_seqlens, B + 1))
    if dc != d or v_cache.shape != shape:
        raise ValueError("the caches must both be [pages,Hkv,page_size,d] with q's d")
    if o.shape != q.shape or lse.shape != (Hq, total):
        raise ValueError("o must have q's shape and lse be [Hq,total]")
    # of the tensors' sizes the table's alone can pass 32 bits (a row of q or
    # of a cache has 128 bytes)
    if not (0 < max_new <= 0x7FFFFFFF and 0 <= window <= 0x7FFFFFFF and B <= 0x7FFFFFFF and max_pages <= 0x7FFFFFFF):
        _need_int32(max_new=max_new, window=window, B=B, max_pages=max_pages)
    return (o.data_ptr(), lse.data_ptr(), B, total, int(max_new), Hq, Hkv, d, max_pages, page_size, num_pages,
            int(window), float(scale), code, None if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel())


def fa_fwd_paged(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens, o, lse, max_new: int, scale: float,
                 workspace, window: int = 0, stream=None):
    """Attention of new rows q [total,Hq,d] to a paged cache (fa.h); the
    workspace is a uint8 tensor, or None where its size is 0."""
    rest = _paged_call(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens, o, lse, max_new, scale, workspace, window)
    _check("fa_fwd_paged", load().fa_fwd_paged(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
        _ptr(cu_seqlens), *rest, _stream(stream)))


def fa_fwd_paged_prefix(q, k_cache, v_cache, prefix_pages, prefix_len: int, block_table, seq_lens, cu_seqlens, o,
                        lse, max_new: int, scale: float, workspace, window: int = 0, stream=None):
    """fa_fwd_paged for requests that share their first prefix_len keys."""
    rest = _paged_call(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens, o, lse, max_new, scale, workspace, window,
                       prefix_pages)
    _need_int32(prefix_len=prefix_len)
    if prefix_pages.numel() * k_cache.shape[2] < prefix_len:
        raise ValueError(f"prefix_pages: {prefix_pages.numel()} pages of {k_cache.shape[2]} hold fewer than "
                         f"{prefix_len} tokens")
    _check("fa_fwd_paged_prefix", load().fa_fwd_paged_prefix(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), prefix_pages.data_ptr(), int(prefix_len),
        block_table.data_ptr(), seq_lens.data_ptr(), _ptr(cu_seqlens), *rest, _stream(stream)))


@functools.lru_cache(maxsize=1024)  # a function of the sizes alone
def fa_fwd_paged_tree_workspace_bytes(B: int, total: int, max_new: int, Hq: int, Hkv: int, d: int, max_pages: int,
                                      page_size: int) -> int:
    return int(load().fa_fwd_paged_tree_workspace_bytes(B, total, max_new, Hq, Hkv, d, max_pages, page_size))


def fa_fwd_paged_tree(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens, parents, o, lse, max_new: int,
                      scale: float, workspace, window: int = 0, stream=None):
    """fa_fwd_paged for trees of drafted tokens; parents int32 [total]."""
    rest = _paged_call(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens, o, lse, max_new, scale, workspace, window)
    import torch
    if not (parents.get_device() == q.get_device() and parents.dtype == torch.int32 and parents.is_contiguous()
            and parents.numel() == q.shape[0]):
        _need_all(("q", q, q.dtype), ("parents", parents, torch.int32))
        _need_numel(parents=(parents, q.shape[0]))
    _check("fa_fwd_paged_tree", load().fa_fwd_paged_tree(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
        _ptr(cu_seqlens), parents.data_ptr(), *rest, _stream(stream)))


def paged_tree_forward(q, k_cache, v_cache, block_table, seq_lens, cu_seqlens, parents, max_new: int, scale: float,
                       window: int, workspace):
    """fa_fwd_paged_tree on the current stream with outputs, and a workspace if
    none is given, that are made here: (O, LSE).  The checks of that and of
    _paged_call but for those outputs, in one place: of the 22 to 29 us of a
    call of few tokens 4 went to doing more."""
    import torch
    total, Hq, d = q.shape
    shape = k_cache.shape
    num_pages, Hkv, page_size, dc = shape
    B, max_pages = block_table.shape
    code, dtype, i32, dev = _dtype_code(q), q.dtype, torch.int32, q.get_device()
    if not (dev >= 0 and dev == torch._C._cuda_getDevice() and q.is_contiguous()
            and k_cache.get_device() == dev and k_cache.dtype == dtype and k_cache.is_contiguous()
            and v_cache.get_device() == dev and v_cache.dtype == dtype and v_cache.is_contiguous()
            and block_table.get_device() == dev and block_table.dtype == i32 and block_table.is_contiguous()
            and seq_lens.get_device() == dev and seq_lens.dtype == i32 and seq_lens.is_contiguous()
            and parents.get_device() == dev and parents.dtype == i32 and parents.is_contiguous()
            and (cu_seqlens is None or (cu_seqlens.get_device() == dev and cu_seqlens.dtype == i32
                                        and cu_seqlens.is_contiguous() and cu_seqlens.numel() == B + 1))
            and (workspace is None or (workspace.get_device() == dev and workspace.dtype == torch.uint8
                                       and workspace.is_contiguous()))
            and seq_lens.numel() == B and parents.numel() == total):
        _need_all(("q", q, dtype), ("k_cache", k_cache, dtype), ("v_cache", v_cache, dtype),
                  ("block_table", block_table, i32), ("seq_lens", seq_lens, i32), ("cu_seqlens", cu_seqlens, i32),
                  ("parents", parents, i32), ("workspace", workspace, torch.uint8))
        _need_numel(seq_lens=(seq_lens, B), cu_seqlens=(cu_seqlens, B + 1), parents=(parents, total))
    if dc != d or v_cache.shape != shape:
        raise ValueError("the caches must both be [pages,Hkv,page_size,d] with q's d")
    if not (0 < max_new <= 0x7FFFFFFF and 0 <= window <= 0x7FFFFFFF and B <= 0x7FFFFFFF and max_pages <= 0x7FFFFFFF):
        _need_int32(max_new=max_new, window=window, B=B, max_pages=max_pages)
    o, lse = torch.empty_like(q), q.new_empty((Hq, total), dtype=torch.float32)
    if workspace is None:
        n = fa_fwd_paged_tree_workspace_bytes(B, total, max_new, Hq, Hkv, d, max_pages, page_size)
        if n:
            workspace = q.new_empty(n, dtype=torch.uint8)
    else:
        n = workspace.numel()
    _check("fa_fwd_paged_tree", load().fa_fwd_paged_tree(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
        None if cu_seqlens is None else cu_seqlens.data_ptr(), parents.data_ptr(), o.data_ptr(), lse.data_ptr(), B, total,
        int(max_new), Hq, Hkv, d, max_pages, page_size, num_pages, int(window), float(scale), code,
        None if workspace is None else workspace.data_ptr(), n, torch._C._cuda_getCurrentRawStream(dev)))
    return o, lse


def fa_get_device_status(stream=None) -> int:
    """FA_OK, or FA_ERR_TIMEOUT if a bounded device wait ran out (clears it)."""
    return int(load().fa_get_device_status(_stream(stream)))


def fa_selftest_bounded_wait(timeout_us: int, stream=None):
    _check("fa_selftest_bounded_wait", load().fa_selftest_bounded_wait(int(timeout_us), _stream(stream)))


def fa_probe_exp2(sink, blocks: int, iters: int, stream=None) -> int:
    """Launches the exp2 throughput probe; returns the exp2 evaluations it
    performs.  sink: float32 CUDA tensor of at least blocks * 256 elements."""
    if sink.numel() < blocks * 256:
        raise ValueError("sink too small")
    n = load().fa_probe_exp2(_ptr(sink), int(blocks), int(iters), _stream(stream))
    if n < 0:
        raise FAError("fa_probe_exp2", FA_ERR_INVALID_ARG, "invalid arguments or launch failure")
    return int(n)
