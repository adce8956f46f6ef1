"""Thin ctypes binding over libmla_gb300.so (the C ABI in include/mla_decode.h).

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, their raw pointers and the current CUDA stream are handed to the
library, and every step of the decode runs in the library's kernels.  There
is no fallback: if the library is missing or a call fails, an error is raised.

stream: the stream of a call's kernels, None for the current one.  On another
stream than the current one, the caller's tensors have to be ready there and to
live until the kernels are done; what a call allocates itself (outputs and a
workspace that were not given) is that stream's memory.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import _build

MLA_OK = 0
_STATUS = {
    0: "MLA_OK", -1: "MLA_ERR_INVALID_ARG", -2: "MLA_ERR_UNSUPPORTED", -3: "MLA_ERR_WORKSPACE",
    -4: "MLA_ERR_CUDA", -5: "MLA_STATUS_BAD_PAGE", -6: "MLA_STATUS_TIMEOUT", -7: "MLA_STATUS_BAD_SEQ_LEN",
    -8: "MLA_STATUS_BAD_INDEX",
}

# Exported entry points and their C signatures (restype, argtypes).
_P = ctypes.c_void_p
_I = ctypes.c_int
_Z = ctypes.c_size_t
SIGNATURES = {
    "mla_workspace_size": (_I, [_I, _I, _I, _I, ctypes.POINTER(ctypes.c_size_t)]),
    "mla_decode_bf16": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P, _P,
                             ctypes.c_size_t, _P]),
    "mla_decode_bf16_noalloc": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P, _P,
                                     _P]),
    "mla_decode_fp8": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P, _P,
                            ctypes.c_size_t, _P]),
    "mla_decode_fp4": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P, _P,
                            ctypes.c_size_t, _P]),
    "mla_decode_fp8_v41": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P, _P,
                                ctypes.c_size_t, _P]),
    "mla_decode_fp4_v41": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P, _P,
                                ctypes.c_size_t, _P]),
    "mla_workspace_size_sparse": (_I, [_I, _I, _I, _I, _I, ctypes.POINTER(ctypes.c_size_t)]),
    "mla_decode_sparse_bf16": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P, _P,
                                    ctypes.c_size_t, _P]),
    "mla_up_project_wuv": (_I, [_P, _P, _I, _I, _I, _P, _P, ctypes.c_size_t, _P]),
    "mla_workspace_size_tree": (_I, [_I, _I, _I, _I, ctypes.POINTER(_Z)]),
    "mla_workspace_size_tree_widened": (_I, [_I, _I, _I, _I, _I, ctypes.POINTER(_Z)]),
    **{"mla_decode_tree_" + f: (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P, _P,
                                     _Z, _P])
       for f in ("bf16", "fp8", "fp4", "fp8_v41", "fp4_v41")},
    **{"mla_cache_append_" + f: (_I, [_P, _Z, _P, _Z, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _Z, _P])
       for f in ("bf16", "fp8", "fp4", "fp8_v41", "fp4_v41")},
    **{"mla_cache_gather_" + f: (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _Z, _P])
       for f in ("bf16", "fp8", "fp4", "fp8_v41", "fp4_v41")},
    "mla_expand_kv": (_I, [_P, _Z, _P, _P, _I, _I, _I, _P, _P, _P, _Z, _P]),
    "mla_workspace_size_prefill": (_I, [_I, _I, ctypes.POINTER(_Z)]),
    "mla_prefill_bf16": (_I, [_P, _P, _P, _P, _P, ctypes.POINTER(_Z), _P, _P, _I, _I, _I, _I, _I, ctypes.c_float, _P,
                              _P, _P, _Z, _P]),
    "mla_combine_splits": (_I, [_P, _P, _P, _I, _I, _P, _P, _P]),
    "mla_get_status": (_I, [_P, _P]),
    "mla_profile_next_decode": (_I, [_P, _P]),
    "mla_status_string": (ctypes.c_char_p, [_I]),
}

_lib = None


class MLAError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {status_string(code)} ({code})")
        self.code = code


def library_path() -> str:
    return _build.LIB_PATH


def load(path: str | None = None) -> ctypes.CDLL:
    """Load the compiled library (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _build.LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"CUDA library not built ({p} missing): run __graft_entry__.build()")
    lib = ctypes.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def status_string(code: int) -> str:
    try:
        return load().mla_status_string(int(code)).decode()
    except RuntimeError:
        return _STATUS.get(int(code), "MLA_UNKNOWN_STATUS")


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# the current stream's handle without building a Stream object (3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        if _raw_stream is not None:
            return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()))
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(t: torch.Tensor, name: str, dtype, shape=None):
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and (shape is None or t.shape == shape) and t.is_cuda
            and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _same_device(tensors: dict, current: int) -> None:
    """Every tensor of a call on one CUDA device, the calling thread's current
    one: the library launches its kernels on the current device, which then
    reads and writes these pointers."""
    devs = {name: t.device for name, t in tensors.items() if t is not None}
    first_name, first = next(iter(devs.items()))
    for name, d in devs.items():
        if d != first:
            raise ValueError(f"{name} is on {d} but {first_name} is on {first}")
    if first.index != current:
        raise ValueError(f"the tensors are on {first} but the current device is cuda:{current}; "
                         f"call under torch.cuda.device({first})")


def _status_workspace(device) -> torch.Tensor:
    return torch.zeros(256, dtype=torch.uint8, device=device)


def _new(stream, make, *args, **kwargs) -> torch.Tensor:
    """A tensor that a call allocates itself, for kernels that run on `stream`:
    its memory is that stream's, so that neither what a free block was last used
    for nor its next use after the call lies on another stream than they do, and
    a fill (a zeroed workspace) comes before them.  The caller's current stream may
    use the tensor as well (after it has waited for `stream`)."""
    if stream is None:
        return make(*args, **kwargs)
    current = torch.cuda.current_stream()
    if current.cuda_stream == stream.cuda_stream:
        return make(*args, **kwargs)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    with torch.cuda.stream(stream):
        t = make(*args, **kwargs)
    t.record_stream(current)
    return t


def mla_workspace_size(batch: int, sq: int, num_heads: int = 128, page_size: int = 64) -> int:
    n = ctypes.c_size_t(0)
    rc = load().mla_workspace_size(int(batch), int(sq), int(num_heads), int(page_size), ctypes.byref(n))
    if rc != MLA_OK:
        raise MLAError(rc, "mla_workspace_size")
    return int(n.value)


def alloc_workspace(batch: int, sq: int, device=None) -> torch.Tensor:
    """A zeroed workspace buffer (uint8) of the size the library asks for."""
    n = mla_workspace_size(batch, sq)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def _decode(fn_name, q_absorbed, q_rope, kv_cache, block_table, seq_lens, scale, out, lse, workspace, stream,
            kv_dtype, row_bytes):
    B, Sq, H, D = q_absorbed.shape
    _check(q_absorbed, "q_absorbed", torch.bfloat16, (B, Sq, H, 512))
    _check(q_rope, "q_rope", torch.bfloat16, (B, Sq, H, 64))
    _check(kv_cache, "kv_cache", kv_dtype)
    if kv_cache.dim() != 3 or kv_cache.shape[2] != row_bytes:
        raise ValueError(f"kv_cache must be [num_pages, page_size, {row_bytes}], got {tuple(kv_cache.shape)}")
    _check(block_table, "block_table", torch.int32)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_pages]")
    _check(seq_lens, "seq_lens", torch.int32, (B,))
    if out is None:
        out = _new(stream, torch.empty, (B, Sq, H, 512), dtype=torch.bfloat16, device=q_absorbed.device)
    if lse is None:
        lse = _new(stream, torch.empty, (B, Sq, H), dtype=torch.float32, device=q_absorbed.device)
    _check(out, "out", torch.bfloat16, (B, Sq, H, 512))
    _check(lse, "lse", torch.float32, (B, Sq, H))
    if workspace is None:
        workspace = _new(stream, alloc_workspace, B, Sq, q_absorbed.device)
    _check(workspace, "workspace", torch.uint8)
    _same_device(dict(q_absorbed=q_absorbed, q_rope=q_rope, kv_cache=kv_cache, block_table=block_table,
                      seq_lens=seq_lens, out=out, lse=lse, workspace=workspace), torch.cuda.current_device())
    rc = getattr(load(), fn_name)(
        _ptr(q_absorbed), _ptr(q_rope), _ptr(kv_cache), _ptr(block_table), _ptr(seq_lens),
        int(B), int(Sq), int(H), int(kv_cache.shape[0]), int(kv_cache.shape[1]), int(block_table.shape[1]),
        ctypes.c_float(float(scale)), _ptr(out), _ptr(lse), _ptr(workspace), ctypes.c_size_t(workspace.numel()),
        _stream(stream))
    if rc != MLA_OK:
        raise MLAError(rc, fn_name)
    return out, lse


def mla_decode_bf16(q_absorbed, q_rope, kv_cache, block_table, seq_lens, scale, out=None, lse=None,
                    workspace=None, stream=None):
    """MLA decode over a bf16 latent cache [num_pages, 64, 576]; returns (out, lse)."""
    return _decode("mla_decode_bf16", q_absorbed, q_rope, kv_cache, block_table, seq_lens, scale, out, lse,
                   workspace, stream, torch.bfloat16, 576)


def mla_decode_bf16_noalloc(q_absorbed, q_rope, kv_cache, block_table, seq_lens, scale, out=None, lse=None,
                            device_status=None, stream=None):
    """mla_decode_bf16 on the library's own static scratch (no workspace
    argument; the library allocates nothing).  At most 8192 query rows;
    calls that can overlap in time race on the shared scratch.
    `device_status`: optional int32 CUDA tensor of one element that receives
    the call's device status.  Returns (out, lse)."""
    B, Sq, H, D = q_absorbed.shape
    _check(q_absorbed, "q_absorbed", torch.bfloat16, (B, Sq, H, 512))
    _check(q_rope, "q_rope", torch.bfloat16, (B, Sq, H, 64))
    _check(kv_cache, "kv_cache", torch.bfloat16)
    if kv_cache.dim() != 3 or kv_cache.shape[2] != 576:
        raise ValueError(f"kv_cache must be [num_pages, page_size, 576], got {tuple(kv_cache.shape)}")
    _check(block_table, "block_table", torch.int32)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_pages]")
    _check(seq_lens, "seq_lens", torch.int32, (B,))
    if out is None:
        out = _new(stream, torch.empty, (B, Sq, H, 512), dtype=torch.bfloat16, device=q_absorbed.device)
    if lse is None:
        lse = _new(stream, torch.empty, (B, Sq, H), dtype=torch.float32, device=q_absorbed.device)
    _check(out, "out", torch.bfloat16, (B, Sq, H, 512))
    _check(lse, "lse", torch.float32, (B, Sq, H))
    if device_status is not None:
        _check(device_status, "device_status", torch.int32, (1,))
    _same_device(dict(q_absorbed=q_absorbed, q_rope=q_rope, kv_cache=kv_cache, block_table=block_table,
                      seq_lens=seq_lens, out=out, lse=lse, device_status=device_status),
                 torch.cuda.current_device())
    rc = load().mla_decode_bf16_noalloc(
        _ptr(q_absorbed), _ptr(q_rope), _ptr(kv_cache), _ptr(block_table), _ptr(seq_lens),
        int(B), int(Sq), int(H), int(kv_cache.shape[0]), int(kv_cache.shape[1]), int(block_table.shape[1]),
        ctypes.c_float(float(scale)), _ptr(out), _ptr(lse), _ptr(device_status), _stream(stream))
    if rc != MLA_OK:
        raise MLAError(rc, "mla_decode_bf16_noalloc")
    return out, lse


def mla_decode_fp8(q_absorbed, q_rope, kv_cache, block_table, seq_lens, scale, out=None, lse=None,
                   workspace=None, stream=None):
    """MLA decode over an FP8 latent cache [num_pages, 64, 594] (uint8 rows:
    576 e4m3 codes then 18 e8m0 scales); returns (out, lse)."""
    return _decode("mla_decode_fp8", q_absorbed, q_rope, kv_cache, block_table, seq_lens, scale, out, lse,
                   workspace, stream, torch.uint8, 594)


def mla_decode_fp4(q_absorbed, q_rope, kv_cache, block_table, seq_lens, scale, out=None, lse=None,
                   workspace=None, stream=None):
    """MLA decode over an FP4 latent cache [num_pages, 64, 324] (uint8 rows:
    576 e2m1 codes, two per byte with the even value in the low nibble, then
    36 e8m0 scales, one per 16 values); returns (out, lse)."""
    return _decode("mla_decode_fp4", q_absorbed, q_rope, kv_cache, block_table, seq_lens, scale, out, lse,
                   workspace, stream, torch.uint8, 324)


def mla_decode_fp8_v41(q_absorbed, q_rope, kv_cache, block_table, seq_lens, scale, out=None, lse=None,
                       workspace=None, stream=None):
    """MLA decode over an FP8 latent cache in the V4.1 row layout
    [num_pages, 64, 528] (uint8 rows: 512 e4m3 codes, 448 latent then 64
    RoPE, then 16 e8m0 scales, one per 32 codes); returns (out, lse) with
    out [..., 512] whose dims 448..511 are 0 (q_absorbed dims 448..511 are
    ignored)."""
    return _decode("mla_decode_fp8_v41", q_absorbed, q_rope, kv_cache, block_table, seq_lens, scale, out, lse,
                   workspace, stream, torch.uint8, 528)


def mla_decode_fp4_v41(q_absorbed, q_rope, kv_cache, block_table, seq_lens, scale, out=None, lse=None,
                       workspace=None, stream=None):
    """MLA decode over an FP4 latent cache in the 288-byte V4.1 row layout
    [num_pages, 64, 288] (uint8 rows: 512 e2m1 codes, two per byte, 448
    latent then 64 RoPE values, then 32 e8m0 scales, one per 16 values);
    returns (out, lse) as mla_decode_fp8_v41 does."""
    return _decode("mla_decode_fp4_v41", q_absorbed, q_rope, kv_cache, block_table, seq_lens, scale, out, lse,
                   workspace, stream, torch.uint8, 288)


def mla_workspace_size_sparse(batch: int, sq: int, topk: int, num_heads: int = 128, page_size: int = 64) -> int:
    n = ctypes.c_size_t(0)
    rc = load().mla_workspace_size_sparse(int(batch), int(sq), int(topk), int(num_heads), int(page_size),
                                          ctypes.byref(n))
    if rc != MLA_OK:
        raise MLAError(rc, "mla_workspace_size_sparse")
    return int(n.value)


def alloc_workspace_sparse(batch: int, sq: int, topk: int, device=None) -> torch.Tensor:
    """A zeroed workspace buffer (uint8) for the sparse decode."""
    n = mla_workspace_size_sparse(batch, sq, topk)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def mla_decode_sparse_bf16(q_absorbed, q_rope, kv_cache, token_slots, scale, out=None, lse=None,
                           workspace=None, stream=None):
    """Sparse top-k decode over a bf16 latent cache [num_pages, 64, 576]:
    query row (b, i) attends over the cache slots token_slots[b, i, :]
    (int32 [B, Sq, topk], slot = page * 64 + offset, -1 = no token).
    Returns (out, lse)."""
    B, Sq, H, D = q_absorbed.shape
    _check(q_absorbed, "q_absorbed", torch.bfloat16, (B, Sq, H, 512))
    _check(q_rope, "q_rope", torch.bfloat16, (B, Sq, H, 64))
    _check(kv_cache, "kv_cache", torch.bfloat16)
    if kv_cache.dim() != 3 or kv_cache.shape[2] != 576:
        raise ValueError(f"kv_cache must be [num_pages, page_size, 576], got {tuple(kv_cache.shape)}")
    _check(token_slots, "token_slots", torch.int32)
    if token_slots.dim() != 3 or tuple(token_slots.shape[:2]) != (B, Sq):
        raise ValueError("token_slots must be [B, Sq, topk]")
    topk = int(token_slots.shape[2])
    if out is None:
        out = _new(stream, torch.empty, (B, Sq, H, 512), dtype=torch.bfloat16, device=q_absorbed.device)
    if lse is None:
        lse = _new(stream, torch.empty, (B, Sq, H), dtype=torch.float32, device=q_absorbed.device)
    _check(out, "out", torch.bfloat16, (B, Sq, H, 512))
    _check(lse, "lse", torch.float32, (B, Sq, H))
    if workspace is None:
        workspace = _new(stream, alloc_workspace_sparse, B, Sq, topk, q_absorbed.device)
    _check(workspace, "workspace", torch.uint8)
    _same_device(dict(q_absorbed=q_absorbed, q_rope=q_rope, kv_cache=kv_cache, token_slots=token_slots, out=out,
                      lse=lse, workspace=workspace), torch.cuda.current_device())
    rc = load().mla_decode_sparse_bf16(
        _ptr(q_absorbed), _ptr(q_rope), _ptr(kv_cache), _ptr(token_slots), int(B), int(Sq), topk, int(H),
        int(kv_cache.shape[0]), int(kv_cache.shape[1]), ctypes.c_float(float(scale)), _ptr(out), _ptr(lse),
        _ptr(workspace), ctypes.c_size_t(workspace.numel()), _stream(stream))
    if rc != MLA_OK:
        raise MLAError(rc, "mla_decode_sparse_bf16")
    return out, lse


def mla_up_project_wuv(latent, w_uv, out=None, workspace=None, stream=None):
    """out[r, h] = w_uv[h] @ latent[r, h]: latent [..., 128, 512] bf16 (the
    decode's output), w_uv [128, 128, 512] bf16 -> [..., 128, 128] bf16."""
    lead = tuple(latent.shape[:-2])
    _check(latent, "latent", torch.bfloat16)
    if tuple(latent.shape[-2:]) != (128, 512):
        raise ValueError("latent must be [..., 128, 512]")
    _check(w_uv, "w_uv", torch.bfloat16, (128, 128, 512))
    rows = 1
    for x in lead:
        rows *= int(x)
    if out is None:
        out = _new(stream, torch.empty, lead + (128, 128), dtype=torch.bfloat16, device=latent.device)
    _check(out, "out", torch.bfloat16, lead + (128, 128))
    if workspace is None:
        workspace = _new(stream, _status_workspace, latent.device)
    _check(workspace, "workspace", torch.uint8)
    _same_device(dict(latent=latent, w_uv=w_uv, out=out, workspace=workspace), torch.cuda.current_device())
    rc = load().mla_up_project_wuv(_ptr(latent), _ptr(w_uv), rows, 128, 128, _ptr(out), _ptr(workspace),
                                   ctypes.c_size_t(workspace.numel()), _stream(stream))
    if rc != MLA_OK:
        raise MLAError(rc, "mla_up_project_wuv")
    return out


def _check_rows(t: torch.Tensor, name: str, tail: tuple, rows: int | None = None):
    """A bf16 tensor [rows, *tail] whose last dimension is contiguous and whose
    other strides and base are multiples of 16 bytes (it may be a view)."""
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()
            and t.shape[1:] == tail and (rows is None or t.shape[0] == rows) and t.data_ptr() % 16 == 0):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() != 1 + len(tail) or tuple(t.shape[1:]) != tuple(tail) or (rows is not None and t.shape[0] != rows):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [{'rows' if rows is None else rows}, "
                         f"{', '.join(map(str, tail))}]")
    if t.numel() and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    if any(t.shape[d] > 1 and (t.stride(d) <= 0 or t.stride(d) % 8) for d in range(t.dim() - 1)) or t.data_ptr() % 16:
        raise ValueError(f"{name} must start on 16 bytes with strides that are positive multiples of 16 bytes")


def _stride(t, dim: int, default: int) -> int:
    """Stride of a dimension; of one that holds a single entry, `default`."""
    return int(t.stride(dim)) if t.shape[dim] > 1 else default


# The two below pass an ordinary tensor with few attribute reads (a call's checks
# cost the host several times its launches); every other goes through
# _check_rows, which has the rules and the messages.
def _rows_arg(t, name: str, width: int, rows: int | None = None):
    """Address and row stride of a checked [rows, width] bf16 tensor or view."""
    if isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.is_cuda:
        shape = t.shape
        if len(shape) == 2 and shape[1] == width and shape[0] > 1 and (rows is None or shape[0] == rows):
            s0, s1 = t.stride()
            at = t.data_ptr()
            if s1 == 1 and s0 > 0 and s0 % 8 == 0 and at % 16 == 0:
                return at, s0
    _check_rows(t, name, (width,), rows)
    return t.data_ptr(), _stride(t, 0, width)


def _heads_arg(t, name: str, width: int, rows: int | None = None):
    """Address, row and head stride of a checked [rows, 128, width] bf16 tensor or view."""
    if isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.is_cuda:
        shape = t.shape
        if (len(shape) == 3 and shape[2] == width and shape[1] == 128 and shape[0] > 1
                and (rows is None or shape[0] == rows)):
            s0, s1, s2 = t.stride()
            at = t.data_ptr()
            if s2 == 1 and s0 > 0 and s1 > 0 and s0 % 8 == 0 and s1 % 8 == 0 and at % 16 == 0:
                return at, s0, s1
    _check_rows(t, name, (128, width), rows)
    return t.data_ptr(), _stride(t, 0, 128 * width), int(t.stride(1))


def _handle(stream, device: int) -> int:
    """The stream's handle, of the device's current stream for None."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(device)
    return (torch.cuda.current_stream() if stream is None else stream).cuda_stream


_ROW_WIDTH = {"bf16": 576, "fp8": 594, "fp4": 324, "fp8_v41": 528, "fp4_v41": 288}


def _check_cache(fmt, kv_cache, block_table, seq_lens, cu_rows):
    _check(kv_cache, "kv_cache", torch.bfloat16 if fmt == "bf16" else torch.uint8)
    if kv_cache.dim() != 3 or kv_cache.shape[2] != _ROW_WIDTH[fmt]:
        raise ValueError(f"kv_cache must be [num_pages, page_size, {_ROW_WIDTH[fmt]}], got {tuple(kv_cache.shape)}")
    _check(block_table, "block_table", torch.int32)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    batch = block_table.shape[0]
    _check(seq_lens, "seq_lens", torch.int32, (batch,))
    _check(cu_rows, "cu_rows", torch.int32, (batch + 1,))


def _append(fmt, c_kv, k_rope, kv_cache, block_table, seq_lens, cu_rows, workspace, stream):
    name = "mla_cache_append_" + fmt
    c_at, c_stride = _rows_arg(c_kv, "c_kv", 512)
    rows = c_kv.shape[0]
    r_at, r_stride = _rows_arg(k_rope, "k_rope", 64, rows)
    _check_cache(fmt, kv_cache, block_table, seq_lens, cu_rows)
    if workspace is None:
        workspace = _new(stream, _status_workspace, kv_cache.device)
    _check(workspace, "workspace", torch.uint8)
    dev = torch.cuda.current_device()
    if not (kv_cache.device == c_kv.device == k_rope.device == block_table.device == seq_lens.device == cu_rows.device
            == workspace.device and kv_cache.device.index == dev):
        _same_device(dict(kv_cache=kv_cache, c_kv=c_kv, k_rope=k_rope, block_table=block_table, seq_lens=seq_lens,
                          cu_rows=cu_rows, workspace=workspace), dev)
    batch, max_pages = block_table.shape
    pages, page_size, _ = kv_cache.shape
    rc = getattr(load(), name)(
        c_at, c_stride, r_at, r_stride, kv_cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
        cu_rows.data_ptr(), batch, rows, pages, page_size, max_pages, workspace.data_ptr(), workspace.numel(),
        _handle(stream, dev))
    if rc != MLA_OK and rows:       # empty tensors have null pointers: nothing to do
        raise MLAError(rc, name)
    return kv_cache


def _gather(fmt, kv_cache, block_table, seq_lens, cu_rows, n_rows, out, workspace, stream):
    name = "mla_cache_gather_" + fmt
    _check_cache(fmt, kv_cache, block_table, seq_lens, cu_rows)
    rows = int(n_rows)
    if rows < 0:
        raise ValueError("n_rows must not be negative")
    if out is None:
        out = _new(stream, torch.empty, (rows, 576), dtype=torch.bfloat16, device=kv_cache.device)
    else:
        _check(out, "out", torch.bfloat16, (rows, 576))
    if workspace is None:
        workspace = _new(stream, _status_workspace, kv_cache.device)
    _check(workspace, "workspace", torch.uint8)
    dev = torch.cuda.current_device()
    if not (kv_cache.device == block_table.device == seq_lens.device == cu_rows.device == out.device
            == workspace.device and kv_cache.device.index == dev):
        _same_device(dict(kv_cache=kv_cache, block_table=block_table, seq_lens=seq_lens, cu_rows=cu_rows, out=out,
                          workspace=workspace), dev)
    batch, max_pages = block_table.shape
    pages, page_size, _ = kv_cache.shape
    rc = getattr(load(), name)(
        kv_cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(), cu_rows.data_ptr(), batch, rows, pages,
        page_size, max_pages, out.data_ptr(), workspace.data_ptr(), workspace.numel(), _handle(stream, dev))
    if rc != MLA_OK and rows:
        raise MLAError(rc, name)
    return out


def mla_cache_append_bf16(c_kv, k_rope, kv_cache, block_table, seq_lens, cu_rows, workspace=None, stream=None):
    """Write packed new tokens (c_kv [n, 512], k_rope [n, 64] bf16, views with
    16-byte row strides allowed) into a bf16 cache [num_pages, 64, 576] in
    place: sequence b's rows [cu_rows[b], cu_rows[b+1]) are the last of its
    seq_lens[b] tokens.  Returns kv_cache."""
    return _append("bf16", c_kv, k_rope, kv_cache, block_table, seq_lens, cu_rows, workspace, stream)


def mla_cache_append_fp8(c_kv, k_rope, kv_cache, block_table, seq_lens, cu_rows, workspace=None, stream=None):
    """mla_cache_append_bf16 into an FP8 cache [num_pages, 64, 594]: e4m3 codes
    with the smallest power-of-two scale per 32 values that clips nothing."""
    return _append("fp8", c_kv, k_rope, kv_cache, block_table, seq_lens, cu_rows, workspace, stream)


def mla_cache_append_fp4(c_kv, k_rope, kv_cache, block_table, seq_lens, cu_rows, workspace=None, stream=None):
    """mla_cache_append_bf16 into an FP4 cache [num_pages, 64, 324]: e2m1 codes
    with the smallest power-of-two scale per 16 values that clips nothing."""
    return _append("fp4", c_kv, k_rope, kv_cache, block_table, seq_lens, cu_rows, workspace, stream)


def mla_cache_append_fp8_v41(c_kv, k_rope, kv_cache, block_table, seq_lens, cu_rows, workspace=None, stream=None):
    """mla_cache_append_fp8 into the V4.1 rows [num_pages, 64, 528]: the first
    448 latent values and the 64 RoPE values (c_kv[:, 448:] is ignored)."""
    return _append("fp8_v41", c_kv, k_rope, kv_cache, block_table, seq_lens, cu_rows, workspace, stream)


def mla_cache_append_fp4_v41(c_kv, k_rope, kv_cache, block_table, seq_lens, cu_rows, workspace=None, stream=None):
    """mla_cache_append_fp4 into the V4.1 rows [num_pages, 64, 288]: the first
    448 latent values and the 64 RoPE values (c_kv[:, 448:] is ignored)."""
    return _append("fp4_v41", c_kv, k_rope, kv_cache, block_table, seq_lens, cu_rows, workspace, stream)


def mla_cache_gather_bf16(kv_cache, block_table, seq_lens, cu_rows, n_rows, out=None, workspace=None, stream=None):
    """Read packed rows back: out [n_rows, 576] bf16, sequence b's rows
    [cu_rows[b], cu_rows[b+1]) being the last of its seq_lens[b] tokens (all of
    them where the difference is seq_lens[b]).  Rows past cu_rows[B] of `out`
    are left as they were."""
    return _gather("bf16", kv_cache, block_table, seq_lens, cu_rows, n_rows, out, workspace, stream)


def mla_cache_gather_fp8(kv_cache, block_table, seq_lens, cu_rows, n_rows, out=None, workspace=None, stream=None):
    """mla_cache_gather_bf16 from an FP8 cache [num_pages, 64, 594] (dequantised)."""
    return _gather("fp8", kv_cache, block_table, seq_lens, cu_rows, n_rows, out, workspace, stream)


def mla_cache_gather_fp4(kv_cache, block_table, seq_lens, cu_rows, n_rows, out=None, workspace=None, stream=None):
    """mla_cache_gather_bf16 from an FP4 cache [num_pages, 64, 324] (dequantised)."""
    return _gather("fp4", kv_cache, block_table, seq_lens, cu_rows, n_rows, out, workspace, stream)


def mla_cache_gather_fp8_v41(kv_cache, block_table, seq_lens, cu_rows, n_rows, out=None, workspace=None,
                             stream=None):
    """mla_cache_gather_bf16 from V4.1 rows [num_pages, 64, 528]; dims 448..511 are 0."""
    return _gather("fp8_v41", kv_cache, block_table, seq_lens, cu_rows, n_rows, out, workspace, stream)


def mla_cache_gather_fp4_v41(kv_cache, block_table, seq_lens, cu_rows, n_rows, out=None, workspace=None,
                             stream=None):
    """mla_cache_gather_bf16 from V4.1 rows [num_pages, 64, 288]; dims 448..511 are 0."""
    return _gather("fp4_v41", kv_cache, block_table, seq_lens, cu_rows, n_rows, out, workspace, stream)


def mla_workspace_size_tree(batch: int, nodes: int, num_heads: int = 128, page_size: int = 64) -> int:
    n = ctypes.c_size_t(0)
    rc = load().mla_workspace_size_tree(int(batch), int(nodes), int(num_heads), int(page_size), ctypes.byref(n))
    if rc != MLA_OK:
        raise MLAError(rc, "mla_workspace_size_tree")
    return int(n.value)


def mla_workspace_size_tree_widened(batch: int, nodes: int, max_pages: int, num_heads: int = 128,
                                    page_size: int = 64) -> int:
    n = ctypes.c_size_t(0)
    rc = load().mla_workspace_size_tree_widened(int(batch), int(nodes), int(num_heads), int(page_size),
                                                int(max_pages), ctypes.byref(n))
    if rc != MLA_OK:
        raise MLAError(rc, "mla_workspace_size_tree_widened")
    return int(n.value)


def alloc_workspace_tree(batch: int, nodes: int, device=None, max_pages: int = 0) -> torch.Tensor:
    """A zeroed workspace buffer (uint8) for the tree decode; with the width of
    the block table as max_pages, one in which a quantised cache's rows are
    widened to bf16 once for all nodes (faster, 72 KiB a page more)."""
    size = (mla_workspace_size_tree_widened(batch, nodes, max_pages) if max_pages
            else mla_workspace_size_tree(batch, nodes))
    return torch.zeros(size, dtype=torch.uint8, device=device or "cuda")


_WIDENED_PAGE = 64 * 576 * 2
_WIDENED_DEFAULT = 1 << 30   # a call without a workspace of its own takes up to this much for widened rows


def _tree(fmt, q_absorbed, q_rope, kv_cache, block_table, seq_lens, parents, scale, n_nodes, out, lse, workspace,
          stream):
    name = "mla_decode_tree_" + fmt
    B, T, H, _ = q_absorbed.shape
    _check(q_absorbed, "q_absorbed", torch.bfloat16, (B, T, H, 512))
    _check(q_rope, "q_rope", torch.bfloat16, (B, T, H, 64))
    _check(kv_cache, "kv_cache", torch.bfloat16 if fmt == "bf16" else torch.uint8)
    if kv_cache.dim() != 3 or kv_cache.shape[2] != _ROW_WIDTH[fmt]:
        raise ValueError(f"kv_cache must be [num_pages, page_size, {_ROW_WIDTH[fmt]}], got {tuple(kv_cache.shape)}")
    _check(block_table, "block_table", torch.int32)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_pages]")
    _check(seq_lens, "seq_lens", torch.int32, (B,))
    _check(parents, "parents", torch.int32, (B, T))
    if n_nodes is not None:
        _check(n_nodes, "n_nodes", torch.int32, (B,))
    if out is None:
        out = _new(stream, torch.empty, (B, T, H, 512), dtype=torch.bfloat16, device=q_absorbed.device)
    else:
        _check(out, "out", torch.bfloat16, (B, T, H, 512))
    if lse is None:
        lse = _new(stream, torch.empty, (B, T, H), dtype=torch.float32, device=q_absorbed.device)
    else:
        _check(lse, "lse", torch.float32, (B, T, H))
    max_pages = block_table.shape[1]
    if workspace is None:
        widen = fmt != "bf16" and T > 1 and B * max_pages * _WIDENED_PAGE <= _WIDENED_DEFAULT
        workspace = _new(stream, alloc_workspace_tree, B, T, q_absorbed.device, max_pages if widen else 0)
    _check(workspace, "workspace", torch.uint8)
    dev = torch.cuda.current_device()
    if not (q_absorbed.device == q_rope.device == kv_cache.device == block_table.device == seq_lens.device
            == parents.device == out.device == lse.device == workspace.device
            and (n_nodes is None or n_nodes.device == out.device) and out.device.index == dev):
        _same_device(dict(q_absorbed=q_absorbed, q_rope=q_rope, kv_cache=kv_cache, block_table=block_table,
                          seq_lens=seq_lens, parents=parents, n_nodes=n_nodes, out=out, lse=lse, workspace=workspace),
                     dev)
    if B == 0:
        return out, lse
    pages, page_size, _ = kv_cache.shape
    rc = getattr(load(), name)(
        q_absorbed.data_ptr(), q_rope.data_ptr(), kv_cache.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
        parents.data_ptr(), None if n_nodes is None else n_nodes.data_ptr(), B, T, H, pages, page_size, max_pages,
        float(scale), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel(), _handle(stream, dev))
    if rc != MLA_OK:
        raise MLAError(rc, name)
    return out, lse


def mla_decode_tree_bf16(q_absorbed, q_rope, kv_cache, block_table, seq_lens, parents, scale, n_nodes=None, out=None,
                         lse=None, workspace=None, stream=None):
    """Decode of a drafted tree over a bf16 latent cache [num_pages, 64, 576]:
    q_absorbed [B, T, 128, 512], q_rope [B, T, 128, 64]; sequence b's nodes are
    the last n_nodes[b] (None: T) of its seq_lens[b] cached tokens, parents
    [B, T] int32 names the node each node continues (-1: the context).  Node i
    sees the context, itself and its ancestors.  Returns (out, lse)."""
    return _tree("bf16", q_absorbed, q_rope, kv_cache, block_table, seq_lens, parents, scale, n_nodes, out, lse,
                 workspace, stream)


def mla_decode_tree_fp8(q_absorbed, q_rope, kv_cache, block_table, seq_lens, parents, scale, n_nodes=None, out=None,
                        lse=None, workspace=None, stream=None):
    """mla_decode_tree_bf16 over the cache mla_decode_fp8 reads, [num_pages, 64, 594]."""
    return _tree("fp8", q_absorbed, q_rope, kv_cache, block_table, seq_lens, parents, scale, n_nodes, out, lse,
                 workspace, stream)


def mla_decode_tree_fp4(q_absorbed, q_rope, kv_cache, block_table, seq_lens, parents, scale, n_nodes=None, out=None,
                        lse=None, workspace=None, stream=None):
    """mla_decode_tree_bf16 over the cache mla_decode_fp4 reads, [num_pages, 64, 324]."""
    return _tree("fp4", q_absorbed, q_rope, kv_cache, block_table, seq_lens, parents, scale, n_nodes, out, lse,
                 workspace, stream)


def mla_decode_tree_fp8_v41(q_absorbed, q_rope, kv_cache, block_table, seq_lens, parents, scale, n_nodes=None, out=None,
                        lse=None, workspace=None, stream=None):
    """mla_decode_tree_bf16 over the cache mla_decode_fp8_v41 reads, [num_pages, 64, 528]."""
    return _tree("fp8_v41", q_absorbed, q_rope, kv_cache, block_table, seq_lens, parents, scale, n_nodes, out, lse,
                 workspace, stream)


def mla_decode_tree_fp4_v41(q_absorbed, q_rope, kv_cache, block_table, seq_lens, parents, scale, n_nodes=None, out=None,
                        lse=None, workspace=None, stream=None):
    """mla_decode_tree_bf16 over the cache mla_decode_fp4_v41 reads, [num_pages, 64, 288]."""
    return _tree("fp4_v41", q_absorbed, q_rope, kv_cache, block_table, seq_lens, parents, scale, n_nodes, out, lse,
                 workspace, stream)


def mla_expand_kv(latent, w_uk, w_uv, k_nope=None, v=None, workspace=None, stream=None):
    """k_nope[t, h] = w_uk[h] @ latent[t], v[t, h] = w_uv[h] @ latent[t]:
    latent [n, 512] bf16 (a view with a 16-byte row stride, such as gathered
    rows' [:, :512]), w_uk, w_uv [128, 128, 512] bf16 -> two [n, 128, 128]."""
    at, stride = _rows_arg(latent, "latent", 512)
    _check(w_uk, "w_uk", torch.bfloat16, (128, 128, 512))
    _check(w_uv, "w_uv", torch.bfloat16, (128, 128, 512))
    n = latent.shape[0]
    if k_nope is None:
        k_nope = _new(stream, torch.empty, (n, 128, 128), dtype=torch.bfloat16, device=latent.device)
    else:
        _check(k_nope, "k_nope", torch.bfloat16, (n, 128, 128))
    if v is None:
        v = _new(stream, torch.empty, (n, 128, 128), dtype=torch.bfloat16, device=latent.device)
    else:
        _check(v, "v", torch.bfloat16, (n, 128, 128))
    if workspace is None:
        workspace = _new(stream, _status_workspace, latent.device)
    _check(workspace, "workspace", torch.uint8)
    dev = torch.cuda.current_device()
    if not (latent.device == w_uk.device == w_uv.device == k_nope.device == v.device == workspace.device
            and latent.device.index == dev):
        _same_device(dict(latent=latent, w_uk=w_uk, w_uv=w_uv, k_nope=k_nope, v=v, workspace=workspace), dev)
    rc = load().mla_expand_kv(at, stride, w_uk.data_ptr(), w_uv.data_ptr(), n, 128, 128, k_nope.data_ptr(),
                              v.data_ptr(), workspace.data_ptr(), workspace.numel(), _handle(stream, dev))
    if rc != MLA_OK and n:
        raise MLAError(rc, "mla_expand_kv")
    return k_nope, v


_Strides = ctypes.c_size_t * 9


def mla_workspace_size_prefill(batch: int, num_q: int) -> int:
    n = ctypes.c_size_t(0)
    rc = load().mla_workspace_size_prefill(int(batch), int(num_q), ctypes.byref(n))
    if rc != MLA_OK:
        raise MLAError(rc, "mla_workspace_size_prefill")
    return int(n.value)


def alloc_workspace_prefill(batch: int, num_q: int, device=None) -> torch.Tensor:
    """A zeroed workspace buffer (uint8) for the prefill of up to `batch`
    sequences with `num_q` queries together."""
    return torch.zeros(mla_workspace_size_prefill(batch, num_q), dtype=torch.uint8, device=device or "cuda")


def mla_prefill_bf16(q_nope, q_rope, k_nope, k_rope, v, cu_q, cu_k, scale, causal=True, out=None, lse=None,
                     workspace=None, stream=None):
    """Expanded-form attention over ragged sequences: q_nope [nq, 128, 128],
    q_rope [nq, 128, 64], k_nope [nk, 128, 128], k_rope [nk, 64], v [nk, 128,
    128] bf16 (views with 16-byte strides and a contiguous last dimension
    allowed), cu_q, cu_k int32 [B + 1].  causal: query i of a sequence's n_q
    sees keys j <= i + n_k - n_q.  Returns (out [nq, 128, 128] bf16, lse
    [nq, 128] fp32); rows past cu_q[B] are left as they were."""
    qn = _heads_arg(q_nope, "q_nope", 128)
    nq = q_nope.shape[0]
    qr = _heads_arg(q_rope, "q_rope", 64, nq)
    kn = _heads_arg(k_nope, "k_nope", 128)
    nk = k_nope.shape[0]
    kr = _rows_arg(k_rope, "k_rope", 64, nk)
    vv = _heads_arg(v, "v", 128, nk)
    _check(cu_q, "cu_q", torch.int32)
    if cu_q.dim() != 1 or cu_q.numel() < 1:
        raise ValueError("cu_q must be [B + 1]")
    B = cu_q.numel() - 1
    _check(cu_k, "cu_k", torch.int32, (B + 1,))
    if out is None:
        out = _new(stream, torch.empty, (nq, 128, 128), dtype=torch.bfloat16, device=q_nope.device)
    else:
        _check(out, "out", torch.bfloat16, (nq, 128, 128))
    if lse is None:
        lse = _new(stream, torch.empty, (nq, 128), dtype=torch.float32, device=q_nope.device)
    else:
        _check(lse, "lse", torch.float32, (nq, 128))
    if workspace is None:
        workspace = _new(stream, alloc_workspace_prefill, B, nq, q_nope.device)
    _check(workspace, "workspace", torch.uint8)
    dev = torch.cuda.current_device()
    if not (q_nope.device == q_rope.device == k_nope.device == k_rope.device == v.device == cu_q.device == cu_k.device
            == out.device == lse.device == workspace.device and q_nope.device.index == dev):
        _same_device(dict(q_nope=q_nope, q_rope=q_rope, k_nope=k_nope, k_rope=k_rope, v=v, cu_q=cu_q, cu_k=cu_k,
                          out=out, lse=lse, workspace=workspace), dev)
    if nq == 0:
        return out, lse
    strides = _Strides(qn[1], qn[2], qr[1], qr[2], kn[1], kn[2], kr[1], vv[1], vv[2])
    rc = load().mla_prefill_bf16(
        qn[0], qr[0], kn[0], kr[0], vv[0], strides, cu_q.data_ptr(), cu_k.data_ptr(), B, nq, nk, 128,
        1 if causal else 0, float(scale), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
        _handle(stream, dev))
    if rc != MLA_OK:
        raise MLAError(rc, "mla_prefill_bf16")
    return out, lse


def mla_combine_splits(partial_out, partial_lse, split_indptr, out=None, lse=None, stream=None):
    """Merge split partials: partial_out [n, 128, 512] fp32, partial_lse [n, 128] fp32,
    split_indptr [rows+1] int32 -> (out [rows, 128, 512] bf16, lse [rows, 128] fp32)."""
    _check(partial_out, "partial_out", torch.float32)
    if partial_out.dim() != 3 or partial_out.shape[2] != 512:
        raise ValueError(f"partial_out must be [n_parts, num_heads, 512], got {tuple(partial_out.shape)}")
    _check(partial_lse, "partial_lse", torch.float32, tuple(partial_out.shape[:2]))
    _check(split_indptr, "split_indptr", torch.int32)
    if split_indptr.dim() != 1 or split_indptr.numel() < 1:
        raise ValueError("split_indptr must be [rows + 1]")
    rows = split_indptr.numel() - 1
    H = partial_out.shape[1]
    if out is None:
        out = _new(stream, torch.empty, (rows, H, 512), dtype=torch.bfloat16, device=partial_out.device)
    if lse is None:
        lse = _new(stream, torch.empty, (rows, H), dtype=torch.float32, device=partial_out.device)
    _check(out, "out", torch.bfloat16, (rows, H, 512))
    _check(lse, "lse", torch.float32, (rows, H))
    _same_device(dict(partial_out=partial_out, partial_lse=partial_lse, split_indptr=split_indptr, out=out, lse=lse),
                 torch.cuda.current_device())
    rc = load().mla_combine_splits(_ptr(partial_out), _ptr(partial_lse), _ptr(split_indptr), int(rows), int(H),
                                   _ptr(out), _ptr(lse), _stream(stream))
    if rc != MLA_OK:
        raise MLAError(rc, "mla_combine_splits")
    return out, lse


def mla_profile_next_decode(before: torch.cuda.Event, after: torch.cuda.Event) -> None:
    """Have the next decode call record `before`/`after` around its attention
    kernel (on the call's stream)."""
    before.record() if before.cuda_event == 0 else None
    after.record() if after.cuda_event == 0 else None
    rc = load().mla_profile_next_decode(ctypes.c_void_p(before.cuda_event), ctypes.c_void_p(after.cuda_event))
    if rc != MLA_OK:
        raise MLAError(rc, "mla_profile_next_decode")


def mla_get_status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return int(load().mla_get_status(_ptr(workspace), _stream(stream)))
