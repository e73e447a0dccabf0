"""Thin ctypes binding of liblora_sgmv (argument marshalling only).

Every step of the shrink and expand runs in the CUDA library; this module
checks torch-side metadata (device, dtype, strides) on the host, takes
``data_ptr()`` of each tensor and the current CUDA stream, and calls the C
ABI declared in ``include/lora_sgmv.h``.  There is no fallback: if the
library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# LORA_SGMV_LIB may point at another build of the library (e.g. an installed copy)
LIB_PATH = os.environ.get("LORA_SGMV_LIB") or os.path.join(_HERE, "liblora_sgmv.so")

LORA_OK, LORA_ERR_INVALID_ARGUMENT, LORA_ERR_UNSUPPORTED, LORA_ERR_CUDA, LORA_ERR_BAD_VALUES = \
    range(5)
BAD_INDPTR, BAD_ADAPTER, BAD_PERMUTATION, BAD_SLICES = 2, 4, 8, 16
MAX_SLICES = 8

_P, _I, _L, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
_F = ctypes.c_float
_lib = None
_lock = threading.Lock()


class LoraError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """Loads liblora_sgmv.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with `python -m scatter_gemm_b200.build`")
            l = ctypes.CDLL(LIB_PATH)
            l.lora_shrink.argtypes = [_P, _L, _P, _P, _P, _P, _P, _L] + [_I] * 8 + [_P, _Z, _P]
            l.lora_shrink.restype = _I
            l.lora_expand.argtypes = [_P, _L, _P, _P, _P, _P, _P, _P, _P, _L] + [_I] * 7 + \
                [_P, _Z, _P]
            l.lora_expand.restype = _I
            l.lora_validate.argtypes = [_P, _P, _P, _P, _I, _I, _I, _I, _L, _P, _P, _Z, _P]
            l.lora_validate.restype = _I
            l.lora_workspace_size.argtypes = [_I, _I, _I]
            l.lora_workspace_size.restype = _Z
            l.lora_validate_workspace_size.argtypes = [_I]
            l.lora_validate_workspace_size.restype = _Z
            l.lora_status_string.argtypes = [_I]
            l.lora_status_string.restype = ctypes.c_char_p
            l.lora_launch_count.argtypes = []
            l.lora_launch_count.restype = ctypes.c_uint64
            l.lora_reset_launch_count.argtypes = []
            l.lora_reset_launch_count.restype = None
            l.lora_last_path.argtypes = []
            l.lora_last_path.restype = _I
            l.lora_device_error.argtypes = [_P, _I]
            l.lora_device_error.restype = _I
            l.lora_shrink_i64.argtypes = l.lora_shrink.argtypes
            l.lora_shrink_i64.restype = _I
            l.lora_expand_i64.argtypes = l.lora_expand.argtypes
            l.lora_expand_i64.restype = _I
            l.lora_index64_workspace_size.argtypes = [_I, _I]
            l.lora_index64_workspace_size.restype = _Z
            l.lora_shrink_expand.argtypes = [_P, _L, _P, _P, _P, _P, _P, _P, _P, _P, _L, _P, _L] + \
                [_I] * 8 + [_P, _Z, _P]
            l.lora_shrink_expand.restype = _I
            l.lora_base_expand.argtypes = [_P, _L, _P, _L, _P, _L, _P, _P, _P, _P, _P, _P, _P,
                                           _L] + [_I] * 8 + [_P]
            l.lora_base_expand.restype = _I
            l.lora_rmsnorm.argtypes = [_P, _L, _P, _L, _P, _L, _P, _F, _F, _P, _L, _P, _L, _P] + \
                [_I] * 3 + [_P]
            l.lora_rmsnorm.restype = _I
            l.lora_w4_project.argtypes = [_P, _L, _P, _P, _L, _P, _P, _L, _P, _L] + [_I] * 6 + \
                [_P, _Z, _P]
            l.lora_w4_workspace_size.argtypes = [_I] * 3
            l.lora_w4_workspace_size.restype = _Z
            l.lora_w4_copies_x.argtypes = [_I] * 2
            l.lora_w4_copies_x.restype = _I
            l.lora_w4_project.restype = _I
            l.lora_rope_append.argtypes = [_P, _L, _P, _I, _I, _P, _L, _I, _P, _P, _L, _I, _P, _P,
                                           _F, _F, _P, _L, _P, _P, _P, _P, _L, _I, _I, _F, _F, _P,
                                           _I, _I, _I, _P]
            l.lora_rope_append.restype = _I
            for name in ("lora_rmsnorm", "lora_w4_project", "lora_rope_append"):
                f = getattr(l, name + "_packed")
                f.argtypes = [ctypes.c_char_p]
                f.restype = _I
            _lib = l
    return _lib


def status_string(status: int) -> str:
    return lib().lora_status_string(status).decode()


def launch_count() -> int:
    return int(lib().lora_launch_count())


def reset_launch_count() -> None:
    lib().lora_reset_launch_count()


PATH_GENERAL, PATH_TENSOR, PATH_GROUPED, PATH_SPLITK, PATH_FUSED = 1, 2, 4, 8, 16


def last_path() -> int:
    """LORA_PATH_* bits of the last call's kernel path on this thread."""
    return int(lib().lora_last_path())


def device_error(clear: bool = True) -> int:
    """Reads (and clears) the device-side failure code of the bounded waits."""
    v = ctypes.c_int32(0)
    st = lib().lora_device_error(ctypes.byref(v), int(clear))
    if st != LORA_OK:
        raise LoraError("lora_device_error", st)
    return int(v.value)


def workspace_size(tok: int, nseg: int, num_adapters: int) -> int:
    return int(lib().lora_workspace_size(tok, nseg, num_adapters))


def make_workspace(tok: int, nseg: int, num_adapters: int, device=None) -> torch.Tensor:
    """Allocates (through torch) the optional scratch that lets the calls
    group many small segments by adapter."""
    n = workspace_size(tok, nseg, num_adapters)
    return torch.empty(max(n, 1), dtype=torch.uint8, device=device or "cuda")


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return 0
    if t.dtype == torch.float16:
        return 1
    raise TypeError(f"unsupported element type {t.dtype} (bf16 or fp16)")


def _row_major(t: torch.Tensor, name: str, dims: int = 2) -> int:
    if t.dim() != dims:
        raise ValueError(f"{name} must be {dims}-D, got {tuple(t.shape)}")
    if t.stride(-1) != 1:
        raise ValueError(f"{name} must have a unit inner stride")
    return t.stride(0) if dims == 2 else 0


def _table(t: Optional[torch.Tensor], name: str, allow_none: bool = False,
           dtype: torch.dtype = torch.int32):
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor")
    return t.data_ptr()


def _index_dtype(*tables: Optional[torch.Tensor]) -> torch.dtype:
    """int32 or int64: the one index type all given tables share."""
    kinds = {t.dtype for t in tables if t is not None}
    if len(kinds) != 1 or not kinds <= {torch.int32, torch.int64}:
        raise ValueError("index tables must all be int32 or all be int64")
    return kinds.pop()


def index64_workspace_size(tok: int, nseg: int) -> int:
    """Bytes at the front of an int64-table call's workspace (the narrowed tables)."""
    return int(lib().lora_index64_workspace_size(tok, nseg))


def _ws64(workspace: Optional[torch.Tensor], tok: int, nseg: int, num_adapters: int, device):
    """Workspace of an int64-table call: the caller's, or one allocated here
    (narrowed tables followed by the adapter-grouping scratch)."""
    if workspace is None:
        n = index64_workspace_size(tok, nseg) + workspace_size(tok, nseg, num_adapters)
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=device)
    return workspace, _ws(workspace)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ws(workspace: Optional[torch.Tensor]):
    if workspace is None:
        return None, 0
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _shrink_shapes(x: torch.Tensor, A_stack: torch.Tensor, out_r: torch.Tensor,
                   num_slices: int, rank: Optional[int]):
    """Host-side shape checks shared by the shrink entry points; returns
    (dtype code, ld_x, ld_out, tok, K, S, r, rs, L)."""
    dt = _dtype_code(x)
    if A_stack.dtype != x.dtype or out_r.dtype != x.dtype:
        raise TypeError("x, A_stack and out_r must share one element type")
    ld_x = _row_major(x, "x")
    ld_out = _row_major(out_r, "out_r")
    if not A_stack.is_contiguous():
        raise ValueError("A_stack must be contiguous")
    S = int(num_slices)
    if S < 1:
        raise ValueError("num_slices must be positive")
    if A_stack.dim() == 4:
        L, S4, rs, K = A_stack.shape
        if S4 != S:
            raise ValueError("A_stack slice dimension does not match num_slices")
    elif A_stack.dim() == 3:
        L, srs, K = A_stack.shape
        if srs % S:
            raise ValueError("A_stack rows are not a multiple of num_slices")
        rs = srs // S
    else:
        raise ValueError("A_stack must be [L, S*rs, K] or [L, S, rs, K]")
    tok, Kx = x.shape
    if Kx != K:
        raise ValueError(f"x has K={Kx}, A_stack has K={K}")
    r = rs if rank is None else int(rank)
    if out_r.shape[0] != tok:
        raise ValueError("out_r must have one row per token")
    if out_r.shape[1] < S * rs:
        raise ValueError(f"out_r must have at least S*rs = {S * rs} columns")
    return dt, ld_x, ld_out, tok, K, S, r, rs, L


def lora_shrink(x: torch.Tensor, A_stack: torch.Tensor, seg_indptr: torch.Tensor,
                weight_indices: torch.Tensor, permutation: Optional[torch.Tensor],
                out_r: torch.Tensor, *, num_slices: int, rank: Optional[int] = None,
                workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Shrink: out_r[i, q*rs+j] = sum_k x[perm[i], k] * A_stack[a, q*rs+j, k].

    x [tok, K] (unit inner stride), A_stack [L, S*rs, K] contiguous (or
    [L, S, rs, K]), out_r [tok, >= S*rs] (unit inner stride, sorted order).
    `rank` is the valid rank r <= rs (default rs).  The index tables are all
    int32, or all int64 (then lora_shrink_i64 runs, and a workspace is
    allocated when none is given)."""
    dt, ld_x, ld_out, tok, K, S, r, rs, L = _shrink_shapes(x, A_stack, out_r, num_slices, rank)
    nseg = seg_indptr.numel() - 1
    idt = _index_dtype(seg_indptr, weight_indices, permutation)
    if idt == torch.int64:
        # int64 tables: lora_shrink_i64 narrows them into the workspace first
        workspace, (ws, wsb) = _ws64(workspace, tok, nseg, L, x.device)
        fn, name = lib().lora_shrink_i64, "lora_shrink_i64"
    else:
        ws, wsb = _ws(workspace)
        fn, name = lib().lora_shrink, "lora_shrink"
    st = fn(x.data_ptr(), ld_x, A_stack.data_ptr(), _table(seg_indptr, "seg_indptr", dtype=idt),
            _table(weight_indices, "weight_indices", dtype=idt),
            _table(permutation, "permutation", True, dtype=idt), out_r.data_ptr(), ld_out,
            tok, K, S, r, rs, nseg, L, dt, ws, wsb, _stream(stream))
    if st != LORA_OK:
        raise LoraError(name, st)
    return out_r


def lora_expand(in_r: torch.Tensor, B_stack: torch.Tensor, seg_indptr: torch.Tensor,
                weight_indices: torch.Tensor, permutation: Optional[torch.Tensor],
                slice_offsets: Sequence[int], scalings: torch.Tensor, base_out: torch.Tensor,
                *, rank: Optional[int] = None, workspace: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """Expand: base_out[perm[i], c] += scalings[a] * sum_j in_r[i, q*rs+j] * B_stack[a, c-off0, j].

    in_r [tok, >= S*rs] (sorted order), B_stack [L, N_tot, rs] contiguous,
    slice_offsets: S+1 host integers, scalings [L] fp32 CUDA, base_out
    [tok, >= off[S]] updated in place.  Index tables: all int32, or all int64
    (lora_expand_i64, as for lora_shrink)."""
    dt = _dtype_code(base_out)
    if in_r.dtype != base_out.dtype or B_stack.dtype != base_out.dtype:
        raise TypeError("in_r, B_stack and base_out must share one element type")
    if scalings.dtype != torch.float32 or not scalings.is_cuda or not scalings.is_contiguous():
        raise ValueError("scalings must be a contiguous fp32 CUDA tensor")
    ld_in = _row_major(in_r, "in_r")
    ld_base = _row_major(base_out, "base_out")
    if B_stack.dim() != 3 or not B_stack.is_contiguous():
        raise ValueError("B_stack must be a contiguous [L, N_tot, rs] tensor")
    L, n_tot, rs = B_stack.shape
    off = [int(v) for v in (slice_offsets.tolist() if torch.is_tensor(slice_offsets)
                            else slice_offsets)]
    S = len(off) - 1
    if S < 1 or S > MAX_SLICES:
        raise ValueError(f"need 2..{MAX_SLICES + 1} slice offsets")
    if off[-1] - off[0] != n_tot:
        raise ValueError("slice_offsets span does not match B_stack rows")
    r = rs if rank is None else int(rank)
    tok = base_out.shape[0]
    if in_r.shape[0] != tok:
        raise ValueError("in_r must have one row per token")
    nseg = seg_indptr.numel() - 1
    off_arr = (ctypes.c_int32 * len(off))(*off)
    idt = _index_dtype(seg_indptr, weight_indices, permutation)
    if idt == torch.int64:
        # int64 tables: lora_expand_i64 narrows them into the workspace first
        workspace, (ws, wsb) = _ws64(workspace, tok, nseg, L, base_out.device)
        fn, name = lib().lora_expand_i64, "lora_expand_i64"
    else:
        ws, wsb = _ws(workspace)
        fn, name = lib().lora_expand, "lora_expand"
    st = fn(in_r.data_ptr(), ld_in, B_stack.data_ptr(),
            _table(seg_indptr, "seg_indptr", dtype=idt),
            _table(weight_indices, "weight_indices", dtype=idt),
            _table(permutation, "permutation", True, dtype=idt),
            ctypes.cast(off_arr, ctypes.c_void_p), scalings.data_ptr(),
            base_out.data_ptr(), ld_base, tok, S, r, rs, nseg, L, dt, ws, wsb,
            _stream(stream))
    if st != LORA_OK:
        raise LoraError(name, st)
    return base_out


def lora_shrink_expand(x: torch.Tensor, A_stack: torch.Tensor, B_stack: torch.Tensor,
                       seg_indptr: torch.Tensor, weight_indices: torch.Tensor,
                       permutation: Optional[torch.Tensor], slice_offsets: Sequence[int],
                       scalings: torch.Tensor, out_r: torch.Tensor, base_out: torch.Tensor, *,
                       rank: Optional[int] = None, workspace: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """The pair in one call: lora_shrink into out_r, then lora_expand of out_r
    into base_out (one fused launch for decode-sized batches).

    x [tok, K], A_stack [L, S*rs, K], B_stack [L, N_tot, rs], out_r
    [tok, >= S*rs] (written), base_out [tok, >= off[S]] (updated), int32 tables."""
    dt = _dtype_code(x)
    for t, n in ((A_stack, "A_stack"), (B_stack, "B_stack"), (out_r, "out_r"),
                 (base_out, "base_out")):
        if t.dtype != x.dtype:
            raise TypeError(f"{n} must have the element type of x")
    if scalings.dtype != torch.float32 or not scalings.is_cuda or not scalings.is_contiguous():
        raise ValueError("scalings must be a contiguous fp32 CUDA tensor")
    ld_x = _row_major(x, "x")
    ld_out = _row_major(out_r, "out_r")
    ld_base = _row_major(base_out, "base_out")
    if not A_stack.is_contiguous() or A_stack.dim() != 3:
        raise ValueError("A_stack must be a contiguous [L, S*rs, K] tensor")
    if B_stack.dim() != 3 or not B_stack.is_contiguous():
        raise ValueError("B_stack must be a contiguous [L, N_tot, rs] tensor")
    L, srs, K = A_stack.shape
    Lb, n_tot, rs = B_stack.shape
    off = [int(v) for v in (slice_offsets.tolist() if torch.is_tensor(slice_offsets)
                            else slice_offsets)]
    S = len(off) - 1
    if S < 1 or S > MAX_SLICES or srs != S * rs or Lb != L:
        raise ValueError("A_stack, B_stack and slice_offsets disagree on L, S or rs")
    if off[-1] - off[0] != n_tot:
        raise ValueError("slice_offsets span does not match B_stack rows")
    tok, Kx = x.shape
    if Kx != K or out_r.shape[0] != tok or base_out.shape[0] != tok:
        raise ValueError("x, out_r and base_out must have one row per token and K columns")
    r = rs if rank is None else int(rank)
    nseg = seg_indptr.numel() - 1
    off_arr = (ctypes.c_int32 * len(off))(*off)
    ws, wsb = _ws(workspace)
    st = lib().lora_shrink_expand(x.data_ptr(), ld_x, A_stack.data_ptr(), B_stack.data_ptr(),
                                  _table(seg_indptr, "seg_indptr"),
                                  _table(weight_indices, "weight_indices"),
                                  _table(permutation, "permutation", True),
                                  ctypes.cast(off_arr, ctypes.c_void_p), scalings.data_ptr(),
                                  out_r.data_ptr(), ld_out, base_out.data_ptr(), ld_base, tok,
                                  K, S, r, rs, nseg, L, dt, ws, wsb, _stream(stream))
    if st != LORA_OK:
        raise LoraError("lora_shrink_expand", st)
    return base_out


def lora_base_expand(x: torch.Tensor, W: torch.Tensor, in_r: torch.Tensor,
                     B_stack: torch.Tensor, seg_indptr: torch.Tensor,
                     weight_indices: torch.Tensor, permutation: Optional[torch.Tensor],
                     slice_offsets: Sequence[int], scalings: torch.Tensor, out: torch.Tensor, *,
                     rank: Optional[int] = None, stream=None) -> torch.Tensor:
    """The base projection with the expand folded in:
    out[perm[i], c] = rn(x[perm[i]] . W[c-off0] + s_a * in_r[i, q*rs:q*rs+r] . B_a[c-off0, :r])
    for the rows of every segment and the columns of the slices.

    x [tok, K], W [N_tot, >= K] (unit inner stride), in_r [tok, >= S*rs],
    B_stack [L, N_tot, rs], out [tok, >= off[S]] (written there only)."""
    dt = _dtype_code(x)
    for t, n in ((W, "W"), (in_r, "in_r"), (B_stack, "B_stack"), (out, "out")):
        if t.dtype != x.dtype:
            raise TypeError(f"{n} must have the element type of x")
    if scalings.dtype != torch.float32 or not scalings.is_cuda or not scalings.is_contiguous():
        raise ValueError("scalings must be a contiguous fp32 CUDA tensor")
    ld_x = _row_major(x, "x")
    ld_w = _row_major(W, "W")
    ld_in = _row_major(in_r, "in_r")
    ld_out = _row_major(out, "out")
    if B_stack.dim() != 3 or not B_stack.is_contiguous():
        raise ValueError("B_stack must be a contiguous [L, N_tot, rs] tensor")
    L, n_tot, rs = B_stack.shape
    off = [int(v) for v in (slice_offsets.tolist() if torch.is_tensor(slice_offsets)
                            else slice_offsets)]
    S = len(off) - 1
    if S < 1 or S > MAX_SLICES or off[-1] - off[0] != n_tot or W.shape[0] != n_tot:
        raise ValueError("slice_offsets, W and B_stack disagree on N_tot")
    tok, K = x.shape
    if W.shape[1] < K or in_r.shape[0] != tok or out.shape[0] != tok:
        raise ValueError("x, W, in_r and out disagree on tok or K")
    r = rs if rank is None else int(rank)
    nseg = seg_indptr.numel() - 1
    off_arr = (ctypes.c_int32 * len(off))(*off)
    st = lib().lora_base_expand(x.data_ptr(), ld_x, W.data_ptr(), ld_w, in_r.data_ptr(), ld_in,
                                B_stack.data_ptr(), _table(seg_indptr, "seg_indptr"),
                                _table(weight_indices, "weight_indices"),
                                _table(permutation, "permutation", True),
                                ctypes.cast(off_arr, ctypes.c_void_p), scalings.data_ptr(),
                                out.data_ptr(), ld_out, tok, K, S, r, rs, nseg, L, dt,
                                _stream(stream))
    if st != LORA_OK:
        raise LoraError("lora_base_expand", st)
    return out


# ----------------------------------------------------------------------------
# operators around the adapted projection
# ----------------------------------------------------------------------------

_CODES = {torch.bfloat16: 0, torch.float16: 1, torch.float8_e4m3fn: 2}


def _rows(t: torch.Tensor, name: str, dtype: torch.dtype, tok: int, width: int, dev: int) -> int:
    """Checks a [tok, >= width] tensor of unit inner stride on device `dev`;
    returns its row stride."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the device of the other tensors, got {t.device}")
    if t.dim() != 2 or t.shape[0] != tok or t.shape[1] < width:
        raise ValueError(f"{name} must be [{tok}, >= {width}], got {tuple(t.shape)}")
    ld, inner = t.stride()
    if inner != 1 and width > 1:
        raise ValueError(f"{name} must have a unit inner stride")
    if tok <= 1:  # the only row's stride says nothing
        return max(ld, width)
    if ld < width:
        raise ValueError(f"{name} must not have overlapping rows")
    return ld


def _ld(t: torch.Tensor, name: str, dtype: torch.dtype, shape, dev: int) -> int:
    """_rows for a tensor that should have exactly `shape`: the usual case in
    few steps, as these calls' time on the host is that of a small launch."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        ld, inner = t.stride()
        if inner == 1 and ld >= shape[1]:
            return ld
    return _rows(t, name, dtype, shape[0], shape[1], dev)


def _scratch(n: int, device: torch.device, stream) -> torch.Tensor:
    """n bytes that belong to the stream of the call, so that whoever gets them
    after the call waits for it."""
    if stream is None:
        return torch.empty(n, dtype=torch.uint8, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(n, dtype=torch.uint8, device=device)


def _flat(t: torch.Tensor, name: str, dtype: torch.dtype, n: int, dev: int) -> int:
    """Checks a contiguous 1-D tensor of n elements; returns its address."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{n}] tensor on the others' device")
    return t.data_ptr()


# The words of the packed entry points: q an integer or an address, d a float.
_WORDS = {
    "lora_rmsnorm": struct.Struct("=7q2d9q").pack,
    "lora_w4_project": struct.Struct("=19q").pack,
    "lora_rope_append": struct.Struct("=17q2d13q2d5q").pack,
}


_PACKED = {name: name + "_packed" for name in _WORDS}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call_on(dev: int, name: str, args, stream, tail: bytes = b"") -> None:
    """Calls a packed entry point with the tensors' device current, on the given
    stream or that device's current one."""
    if dev < 0:
        raise ValueError(f"{name} needs CUDA tensors")
    fn = getattr(_lib or lib(), _PACKED[name])
    raw = _raw_stream(dev) if stream is None else _stream(stream)
    words = _WORDS[name](*args, raw)
    if tail:
        words += tail
    if dev == _current_device():
        st = fn(words)
    else:
        with torch.cuda.device(dev):
            st = fn(words)
    if st != LORA_OK:
        raise LoraError(name, st)


def lora_rmsnorm(x: torch.Tensor, weight: torch.Tensor, out: Optional[torch.Tensor], *,
                 residual: Optional[torch.Tensor] = None,
                 residual_out: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 weight_offset: float = 0.0, out_q: Optional[torch.Tensor] = None,
                 out_scale: Optional[torch.Tensor] = None, stream=None):
    """RMS norm of h = x + residual: out = h * rsqrt(mean(h^2) + eps) * (weight + weight_offset).

    x, residual, out [tok, H] (unit inner stride) and weight [H] share bf16 or
    fp16; h is rounded and written to residual_out (default: residual, in
    place).  out_q [tok, H] (float8_e4m3fn) with out_scale [tok] (fp32) takes
    the 8-bit form, out = out_q * out_scale[:, None] within rounding; `out` may
    then be None.  Returns out, or out_q where out is None."""
    dt = _dtype_code(x)
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"x must be 2-D, got {tuple(shape)}")
    tok, H = shape
    dtype, dev = x.dtype, x.get_device()
    ld_x = _ld(x, "x", dtype, shape, dev)
    w = _flat(weight, "weight", dtype, H, dev)
    ptr_r = ptr_ro = ptr_o = ptr_q = ptr_s = 0
    ld_r = ld_ro = ld_o = ld_q = 0
    if residual is not None:
        ld_ro = ld_r = _ld(residual, "residual", dtype, shape, dev)
        ptr_ro = ptr_r = residual.data_ptr()
    if residual_out is not None:
        if residual is None:
            raise ValueError("residual_out needs a residual")
        ld_ro = _ld(residual_out, "residual_out", dtype, shape, dev)
        ptr_ro = residual_out.data_ptr()
    if out is not None:
        ld_o, ptr_o = _ld(out, "out", dtype, shape, dev), out.data_ptr()
    if (out_q is None) != (out_scale is None):
        raise ValueError("out_q and out_scale go together")
    if out_q is not None:
        ld_q, ptr_q = _ld(out_q, "out_q", torch.float8_e4m3fn, shape, dev), out_q.data_ptr()
        ptr_s = _flat(out_scale, "out_scale", torch.float32, tok, dev)
    elif out is None:
        raise ValueError("out or out_q is required")
    if tok:
        _call_on(dev, "lora_rmsnorm",
                 (x.data_ptr(), ld_x, ptr_r, ld_r, ptr_ro, ld_ro, w, weight_offset, eps, ptr_o,
                  ld_o, ptr_q, ld_q, ptr_s, tok, H, dt), stream)
    return out if out is not None else out_q


def lora_w4_project(x: torch.Tensor, w_packed: torch.Tensor, w_scales: torch.Tensor,
                    out: torch.Tensor, *, group_size: int,
                    w_zeros: Optional[torch.Tensor] = None,
                    x_scale: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Base projection with 4-bit weights: out = x @ W^T with
    W[n, k] = w_scales[k // group_size, n] * (q[n, k] - w_zeros[k // group_size, n]).

    x [tok, K] (unit inner stride) of out's element type, or float8_e4m3fn
    with x_scale [tok] (fp32); w_packed [N, >= ceil(K/32)*16] uint8 holds q as
    :func:`w4_pack` lays it out; w_scales [ceil(K/group_size), N] of out's
    type; w_zeros uint8 of the same shape (default: 8 everywhere); out [tok,
    >= N] is written in its first N columns.  Rows of x that are not 16-byte
    aligned are copied to the workspace first (:func:`w4_workspace_size` bytes)
    where there are more than 16 of them, or more than shared memory holds.  It
    is allocated when none is given, unless up to 16 rows are so long (K over
    94,080) that shared memory does not hold one: those need a given one."""
    dt = _dtype_code(out)
    x_shape, w_shape = x.shape, w_packed.shape
    if len(x_shape) != 2 or len(w_shape) != 2:
        raise ValueError("x and w_packed must be 2-D")
    tok, K = x_shape
    N = w_shape[0]
    dtype, x_dtype, dev = out.dtype, x.dtype, x.get_device()
    x_dt = _CODES.get(x_dtype, -1)
    if x_dt != 2 and x_dt != dt:
        raise TypeError(f"x must be {dtype} or float8_e4m3fn, got {x_dtype}")
    if group_size not in (32, 64, 128):
        raise ValueError("group_size must be 32, 64 or 128")
    if K < 1:
        raise ValueError("x must have at least one column")
    s_shape = (-(-K // group_size), N)
    ld_x = _ld(x, "x", x_dtype, x_shape, dev)
    ld_w = _rows(w_packed, "w_packed", torch.uint8, N, -(-K // 32) * 16, dev)
    ld_s = _ld(w_scales, "w_scales", dtype, s_shape, dev)
    if w_scales.shape != s_shape:
        raise ValueError(f"w_scales must be {s_shape}, got {tuple(w_scales.shape)}")
    ptr_z = ptr_sx = 0
    if w_zeros is not None:
        ld_z = _ld(w_zeros, "w_zeros", torch.uint8, s_shape, dev)
        if w_zeros.shape != s_shape or (ld_z != ld_s and s_shape[0] > 1):
            raise ValueError("w_zeros must have the shape and row stride of w_scales")
        ptr_z = w_zeros.data_ptr()
    if (x_scale is not None) != (x_dt == 2):
        raise ValueError("x_scale goes with an 8-bit x")
    if x_scale is not None:
        ptr_sx = _flat(x_scale, "x_scale", torch.float32, tok, dev)
    ld_o = _ld(out, "out", dtype, (tok, N), dev)
    ptr_x = x.data_ptr()
    ws = wsb = 0
    if dev >= 0 and (ptr_x | ld_x * x_dtype.itemsize) & 15 and \
            (tok > 16 or lib().lora_w4_copies_x(tok, K)):
        if workspace is not None:
            if workspace.get_device() != dev:
                raise ValueError("workspace must be on the device of the other tensors")
        elif tok > 16 or not lib().lora_w4_copies_x(1, K):
            workspace = _scratch(w4_workspace_size(tok, K, x_dtype), x.device, stream)
        if workspace is not None:
            ws, wsb = _ws(workspace)
    if tok and N:
        _call_on(dev, "lora_w4_project",
                 (ptr_x, ld_x, ptr_sx, w_packed.data_ptr(), ld_w, w_scales.data_ptr(),
                  ptr_z, ld_s, out.data_ptr(), ld_o, tok, K, N, group_size, x_dt, dt, ws, wsb),
                 stream)
    return out


def w4_workspace_size(tok: int, K: int, x_dtype: torch.dtype) -> int:
    """Bytes of workspace that lora_w4_project takes for rows of x that are not
    16-byte aligned."""
    return int(lib().lora_w4_workspace_size(tok, K, _CODES[x_dtype]))


# the place of value i of eight in a 32-bit word of packed weights
_W4_SHIFT = (0, 16, 4, 20, 8, 24, 12, 28)


def w4_pack(q: torch.Tensor) -> torch.Tensor:
    """Packs integers q [N, K] in 0..15 as lora_w4_project reads them: uint8
    [N, ceil(K/32)*16], the values behind K being 0."""
    if q.dim() != 2 or q.dtype.is_floating_point or q.dtype.is_complex or q.dtype == torch.bool:
        raise ValueError("q must be a 2-D integer tensor")
    if q.numel() and (int(q.min()) < 0 or int(q.max()) > 15):
        raise ValueError("4-bit values must be in 0..15")
    N, K = q.shape
    words = torch.zeros(N, -(-K // 32) * 32, dtype=torch.int64, device=q.device)
    words[:, :K] = q
    shift = torch.tensor(_W4_SHIFT, dtype=torch.int64, device=q.device)
    words = (words.view(N, -1, 8) << shift).sum(dim=2)
    bytes_ = (words[:, :, None] >> torch.arange(0, 32, 8, device=q.device)) & 255
    return bytes_.to(torch.uint8).reshape(N, -1)


def w4_unpack(w_packed: torch.Tensor, K: int) -> torch.Tensor:
    """The integers [N, K] (uint8) of weights packed by :func:`w4_pack`."""
    if w_packed.dim() != 2 or w_packed.dtype != torch.uint8 or w_packed.shape[1] % 4:
        raise ValueError("w_packed must be a 2-D uint8 tensor of whole 32-bit words a row")
    if not 0 <= K <= 2 * w_packed.shape[1]:
        raise ValueError(f"rows of {w_packed.shape[1]} bytes do not hold {K} values")
    b = w_packed.reshape(w_packed.shape[0], -1, 4)
    q = torch.stack([(b[:, :, s // 8] >> (s % 8)) & 15 for s in _W4_SHIFT], dim=2)
    return q.reshape(w_packed.shape[0], -1)[:, :K].contiguous()


def w4_quantize(W: torch.Tensor, group_size: int = 128, zeros: bool = False):
    """Rounds a weight W [N, K] (bf16 or fp16) to 4 bits in groups of
    group_size columns: returns (w_packed, w_scales [G, N], w_zeros [G, N] or
    None).  With `zeros` a group spans its smallest to its largest value (and
    0), without it q - 8 spans plus and minus its largest magnitude."""
    dt = W.dtype
    _dtype_code(W)
    if W.dim() != 2 or group_size not in (32, 64, 128):
        raise ValueError("W must be 2-D and group_size 32, 64 or 128")
    N, K = W.shape
    G = -(-K // group_size)
    Wf = torch.zeros(N, G * group_size, dtype=torch.float32, device=W.device)
    Wf[:, :K] = W
    Wg = Wf.view(N, G, group_size)
    if zeros:
        lo, hi = Wg.amin(2).clamp(max=0), Wg.amax(2).clamp(min=0)
        s = (hi - lo) / 15
    else:
        s = Wg.abs().amax(2) / 7
    s = s.to(dt)
    # the scale that is stored is the one that values are divided by
    sf = torch.where(s > 0, s.float(), 1.0)
    z = (-lo / sf).round().clamp(0, 15) if zeros else torch.full_like(sf, 8.0)
    q = ((Wg / sf[:, :, None]).round() + z[:, :, None]).clamp(0, 15).to(torch.uint8)
    return (w4_pack(q.reshape(N, -1)[:, :K]), s.T.contiguous(),
            z.to(torch.uint8).T.contiguous() if zeros else None)


def rope_axis_map(sections: Sequence[int], interleaved: bool = False) -> list:
    """The position axis of each frequency for :func:`lora_rope_append`.

    sections: frequencies of each axis (time, height, width, ...).  In order,
    an axis' frequencies are neighbours; interleaved, frequency i belongs to
    axis i % len(sections) as long as that axis has frequencies left, counted
    as i < len(sections) * sections[axis], and to axis 0 otherwise."""
    sec = [int(v) for v in sections]
    if not 1 <= len(sec) <= 4 or min(sec) < 0:
        raise ValueError("need 1 to 4 non-negative sections")
    if not interleaved:
        return [a for a, n in enumerate(sec) for _ in range(n)]
    m = len(sec)
    return [i % m if i < m * sec[i % m] else 0 for i in range(sum(sec))]


def _cache(t: torch.Tensor, name: str, shape, dev: int):
    """Checks a cache of the given shape and any strides but the last; returns them."""
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the device of the other tensors, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    strides = t.stride()
    if strides[3] != 1 and shape[3] > 1:
        raise ValueError(f"{name} must have a unit inner stride")
    return strides


def lora_rope_append(qkv: torch.Tensor, slice_offsets: Sequence[int], head_dim: int,
                     positions: torch.Tensor, cos_sin: torch.Tensor, k_cache: torch.Tensor,
                     v_cache: torch.Tensor, slots: torch.Tensor, *,
                     q_out: Optional[torch.Tensor] = None,
                     axis_map: Optional[Sequence[int]] = None, interleaved: bool = False,
                     q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                     weight_offset: float = 0.0, k_scale: float = 1.0, v_scale: float = 1.0,
                     stream=None) -> torch.Tensor:
    """Rotates the q and k slices of qkv, writes q to q_out and appends k and v
    to a paged cache.

    qkv [tok, >= off[3]] with the q, k, v slices at the host offsets
    slice_offsets[0..3], heads of head_dim columns; positions [tok], or
    [axes, tok] with axis_map (one axis number for each frequency, see
    :func:`rope_axis_map`); cos_sin [max_pos, R] fp32, R/2 cosines and R/2
    sines, R <= head_dim even; k_cache, v_cache [pages, page_size, Hkv,
    head_dim] of qkv's type or float8_e4m3fn (values times the fp32
    reciprocal of k_scale, v_scale), any strides but a unit inner one; slots [tok], negative = no
    cache entry.  positions and slots are both int32 or both int64.  q_weight
    and k_weight [head_dim] normalise each head first.  q_out [tok, Hq *
    head_dim] defaults to the q slice itself, in place."""
    dt = _dtype_code(qkv)
    shape = qkv.shape
    if len(shape) != 2:
        raise ValueError(f"qkv must be 2-D, got {tuple(shape)}")
    if len(slice_offsets) != 4:
        raise ValueError("slice_offsets needs 4 entries")
    o0, o1, o2, o3 = slice_offsets
    dtype, tok, dev, D = qkv.dtype, shape[0], qkv.get_device(), head_dim
    if not 0 <= o0 <= o1 <= o2 <= o3 or D < 1 or (o1 - o0) % D or (o2 - o1) % D or \
            o3 - o2 != o2 - o1:
        raise ValueError("slice_offsets must span whole heads, as many of k as of v")
    if o3 > shape[1]:
        raise ValueError(f"qkv must have at least {o3} columns, got {shape[1]}")
    ld = _ld(qkv, "qkv", dtype, shape, dev)
    idt = slots.dtype
    if idt not in (torch.int32, torch.int64) or positions.dtype is not idt:
        raise TypeError("positions and slots must both be int32 or both be int64")
    ptr_s = _flat(slots, "slots", idt, tok, dev)
    table = cos_sin.shape
    if len(table) != 2 or cos_sin.dtype is not torch.float32 or not cos_sin.is_contiguous() or \
            cos_sin.get_device() != dev:
        raise ValueError("cos_sin must be a contiguous fp32 [max_pos, R] tensor on qkv's device")
    max_pos, R = table
    if R > D or R % 2 or (R and max_pos < 1):
        raise ValueError("cos_sin must have 2 * frequencies <= head_dim columns and a row")
    axes, ld_pos, amap = 1, 0, b""
    if positions.dim() == 1:
        ptr_p = _flat(positions, "positions", idt, tok, dev)
        if axis_map is not None:
            raise ValueError("axis_map needs positions of [axes, tok]")
    else:
        axes = positions.shape[0]
        ld_pos = _rows(positions, "positions", idt, axes, tok, dev)
        ptr_p = positions.data_ptr()
        if positions.shape[1] != tok or not 1 <= axes <= 4:
            raise ValueError(f"positions must be [tok] or [1..4, {tok}]")
        if axis_map is not None:
            amap = bytes(axis_map)
            if len(amap) != R // 2 or (amap and max(amap) >= axes):
                raise ValueError(f"axis_map needs {R // 2} axis numbers below {axes}")
        elif axes > 1:
            raise ValueError("positions of several axes need an axis_map")
    hkv = (o2 - o1) // D
    c_shape, c_dtype = k_cache.shape, k_cache.dtype
    if len(c_shape) != 4 or c_shape[2] != hkv or c_shape[3] != D:
        raise ValueError(f"k_cache must be [pages, page_size, {hkv}, {D}], got {tuple(c_shape)}")
    kp, kl, kh, _ = _cache(k_cache, "k_cache", c_shape, dev)
    vp, vl, vh, _ = _cache(v_cache, "v_cache", c_shape, dev)
    if c_dtype is not v_cache.dtype:
        raise ValueError("k_cache and v_cache must share their element type")
    c_dt = _CODES.get(c_dtype, -1)
    if c_dt != dt and c_dt != 2:
        raise TypeError(f"the caches must be {dtype} or float8_e4m3fn, got {c_dtype}")
    if q_out is None:
        q_out = qkv[:, o0:o1]
    ld_q = _ld(q_out, "q_out", dtype, (tok, o1 - o0), dev)
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight go together")
    qw = kw = 0
    if q_weight is not None:
        qw = _flat(q_weight, "q_weight", dtype, D, dev)
        kw = _flat(k_weight, "k_weight", dtype, D, dev)
    if tok:
        _call_on(dev, "lora_rope_append",
                 (qkv.data_ptr(), ld, o0, o1, o2, o3, D, R, ptr_p, ld_pos, axes, 1 if amap else 0,
                  cos_sin.data_ptr(), max_pos, 1 if interleaved else 0, qw, kw, weight_offset,
                  eps, q_out.data_ptr(), ld_q, k_cache.data_ptr(), kp, kl, kh,
                  v_cache.data_ptr(), vp, vl, vh, c_shape[0] if c_shape[1] else 0,
                  c_shape[1] or 1, c_dt, k_scale, v_scale, ptr_s,
                  8 if idt is torch.int64 else 4, tok, dt), stream, amap)
    return q_out


def lora_validate(seg_indptr: torch.Tensor, weight_indices: torch.Tensor,
                  permutation: Optional[torch.Tensor], num_adapters: int, tok: int,
                  slice_offsets: Optional[Sequence[int]] = None, ld_base: int = 0,
                  stream=None) -> int:
    """Runs the device-side table checks and returns the LORA_BAD_* bitmask
    (0 = valid).  Synchronises the stream to read the result."""
    nseg = seg_indptr.numel() - 1
    dev = seg_indptr.device
    result = torch.empty(1, dtype=torch.int32, device=dev)
    ws = torch.empty(max(int(lib().lora_validate_workspace_size(tok)), 4), dtype=torch.uint8,
                     device=dev)
    if slice_offsets is not None:
        off = [int(v) for v in slice_offsets]
        S = len(off) - 1
        off_ptr = ctypes.cast((ctypes.c_int32 * len(off))(*off), ctypes.c_void_p)
    else:
        S, off_ptr = 1, None
    st = lib().lora_validate(_table(seg_indptr, "seg_indptr"), _table(weight_indices,
                                                                      "weight_indices"),
                             _table(permutation, "permutation", True), off_ptr, tok, nseg,
                             num_adapters, S, ld_base, result.data_ptr(), ws.data_ptr(),
                             ws.numel(), _stream(stream))
    if st != LORA_OK:
        raise LoraError("lora_validate", st)
    (torch.cuda.current_stream() if stream is None else stream).synchronize()
    return int(result.item())


STATIC_SCRATCH_BYTES = 1 << 20


def lora_shrink_static_scratch(x: torch.Tensor, A_stack: torch.Tensor, seg_indptr: torch.Tensor,
                               weight_indices: torch.Tensor, permutation: Optional[torch.Tensor],
                               out_r: torch.Tensor, *, num_slices: int,
                               rank: Optional[int] = None, stream=None) -> torch.Tensor:
    """lora_shrink for callers that cannot allocate device memory.

    Same arguments and result as :func:`lora_shrink` without a workspace: the
    library's own fixed 1 MiB device array holds the scratch.  Calls that
    overlap on the GPU race on that array, and problems whose workspace would
    exceed it raise LoraError (LORA_ERR_UNSUPPORTED)."""
    dt, ld_x, ld_out, tok, K, S, r, rs, L = _shrink_shapes(x, A_stack, out_r, num_slices, rank)
    f = lib().lora_shrink_static_scratch
    f.argtypes = [_P, _L, _P, _P, _P, _P, _P, _L] + [_I] * 8 + [_P]
    f.restype = _I
    st = f(x.data_ptr(), ld_x, A_stack.data_ptr(),
           _table(seg_indptr, "seg_indptr"), _table(weight_indices, "weight_indices"),
           _table(permutation, "permutation", True), out_r.data_ptr(), ld_out,
           tok, K, S, r, rs, seg_indptr.numel() - 1, L, dt, _stream(stream))
    if st != LORA_OK:
        raise LoraError("lora_shrink_static_scratch", st)
    return out_r


# ----------------------------------------------------------------------------
# identity-permutation ops of the same page (segments in token order)
# ----------------------------------------------------------------------------

def _fn(name, argtypes):
    f = getattr(lib(), name)
    f.argtypes = argtypes
    f.restype = _I
    return f


def _check(name, st):
    if st != LORA_OK:
        raise LoraError(name, st)


def sgemm_lora_a_fwd(x, A_stack, seg_indptr, weight_indices, out, *, num_slices=1, rank=None,
                     workspace=None, stream=None):
    """out[i, q*rs+j] = sum_k x[i, k] * A_stack[a, q*rs+j, k] (no permutation)."""
    L, srs, K = A_stack.shape
    S = int(num_slices)
    rs = srs // S
    r = rs if rank is None else int(rank)
    ws, wsb = _ws(workspace)
    f = _fn("lora_sgemm_a", [_P, _L, _P, _P, _P, _P, _L] + [_I] * 8 + [_P, _Z, _P])
    _check("lora_sgemm_a", f(x.data_ptr(), _row_major(x, "x"), A_stack.data_ptr(),
                             _table(seg_indptr, "seg_indptr"),
                             _table(weight_indices, "weight_indices"), out.data_ptr(),
                             _row_major(out, "out"), x.shape[0], K, S, r, rs,
                             seg_indptr.numel() - 1, L, _dtype_code(x), ws, wsb,
                             _stream(stream)))
    return out


def _expand_like(name, in_r, B_stack, seg_indptr, weight_indices, scalings, base_out, rank,
                 workspace, stream, extra_front=(), extra_types=(), n_arg=None):
    L, n_tot, rs = B_stack.shape
    r = rs if rank is None else int(rank)
    ws, wsb = _ws(workspace)
    types = [_P, _L, _P, _P, _P] + list(extra_types) + [_P, _P, _L, _I] + \
        ([_I] if n_arg is not None else []) + [_I] * 5 + [_P, _Z, _P]
    f = _fn(name, types)
    args = [in_r.data_ptr(), _row_major(in_r, "in_r"), B_stack.data_ptr(),
            _table(seg_indptr, "seg_indptr"), _table(weight_indices, "weight_indices")]
    args += list(extra_front)
    args += [scalings.data_ptr(), base_out.data_ptr(), _row_major(base_out, "base_out"),
             base_out.shape[0]]
    if n_arg is not None:
        args.append(n_arg)
    args += [r, rs, seg_indptr.numel() - 1, L, _dtype_code(base_out), ws, wsb, _stream(stream)]
    _check(name, f(*args))
    return base_out


def sgemm_lora_b_fwd(in_r, B_stack, seg_indptr, weight_indices, scalings, base_out, *, rank=None,
                     workspace=None, stream=None):
    """base_out[i, c] += scalings[a] * sum_j in_r[i, j] * B_stack[a, c, j] (one slice)."""
    return _expand_like("lora_sgemm_b", in_r, B_stack, seg_indptr, weight_indices, scalings,
                        base_out, rank, workspace, stream, n_arg=B_stack.shape[1])


def qkv_lora_b_fwd(in_r, B_stack, seg_indptr, weight_indices, qkv_offsets, scalings, base_out, *,
                   rank=None, workspace=None, stream=None):
    """Expand into three slices q, k, v at host column offsets qkv_offsets[0..3]."""
    off = [int(v) for v in qkv_offsets]
    if len(off) != 4:
        raise ValueError("qkv_offsets needs 4 entries")
    arr = (ctypes.c_int32 * 4)(*off)
    return _expand_like("lora_qkv_b", in_r, B_stack, seg_indptr, weight_indices, scalings,
                        base_out, rank, workspace, stream,
                        extra_front=[ctypes.cast(arr, ctypes.c_void_p)], extra_types=[_P])


def gate_up_lora_b_fwd(in_r, B_stack, seg_indptr, weight_indices, scalings, base_out, *,
                       rank=None, workspace=None, stream=None):
    """Expand into two equal slices (gate, up) at columns 0 and N."""
    return _expand_like("lora_gate_up_b", in_r, B_stack, seg_indptr, weight_indices, scalings,
                        base_out, rank, workspace, stream, n_arg=B_stack.shape[1] // 2)


def embedding_lora_a_fwd(ids, A_emb, seg_indptr, weight_indices, out, *, rank=None, stream=None):
    """out[i, j] = A_emb[a, j, ids[i]] for j < rank (A_emb [L, rs, V])."""
    L, rs, V = A_emb.shape
    r = rs if rank is None else int(rank)
    f = _fn("lora_embedding_a", [_P, _P, _P, _P, _P, _L] + [_I] * 7 + [_P])
    _check("lora_embedding_a", f(_table(ids, "ids"), A_emb.data_ptr(),
                                 _table(seg_indptr, "seg_indptr"),
                                 _table(weight_indices, "weight_indices"), out.data_ptr(),
                                 _row_major(out, "out"), ids.numel(), V, r, rs,
                                 seg_indptr.numel() - 1, L, _dtype_code(out), _stream(stream)))
    return out


# the chunked-SGMV pair under the names the pages use
chunked_sgmv_lora_shrink_fwd = lora_shrink
chunked_sgmv_lora_expand_fwd = lora_expand
