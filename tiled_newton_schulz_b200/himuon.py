"""Thin ctypes binding of libhimuon (argument marshalling only).

Every step of the path runs in the library's CUDA kernels; this module only
turns torch tensors into ``himuon_mat`` records, passes the current CUDA
stream, and allocates the caller-side workspace with torch when the caller
does not pass one.  Importing works without a GPU; any compute call without
the built library raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libhimuon.so")

BF16, FP16, FP32, I8 = 0, 1, 2, 3
OK = 0
OP_NS_TILED, OP_NS_FULL, OP_GRAM_NS, OP_MOMENTUM_STEP = 0, 1, 2, 3
EXPORTS = ("himuon_ns_tiled", "himuon_ns_full", "himuon_gram_ns", "himuon_momentum_step",
           "himuon_workspace_size", "himuon_get_device_status", "himuon_status_string",
           "himuon_version", "himuon_plan_tiles", "himuon_launch_count", "himuon_ns_static",
           "himuon_expert_product", "himuon_expert_gradient", "himuon_quantize", "himuon_expert_product_i8")
ERR_TOO_LARGE = -9
STATIC_SCRATCH_BYTES = 32 << 20


class Mat(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("ld", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class Split(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int32), ("nblocks", ctypes.c_int32), ("sizes", ctypes.POINTER(ctypes.c_int64))]


class Params(ctypes.Structure):
    _fields_ = [("tile", ctypes.c_int32), ("steps", ctypes.c_int32), ("coeffs", ctypes.POINTER(ctypes.c_float)),
                ("eps", ctypes.c_float), ("compute", ctypes.c_int32), ("safety", ctypes.c_float),
                ("n_restart", ctypes.c_int32), ("restart_at", ctypes.POINTER(ctypes.c_int32)),
                ("chunk_bytes", ctypes.c_int64), ("tiles", ctypes.POINTER(ctypes.c_int32))]


class HimuonError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {status_string(code)} ({code})")
        self.code = code


_lib = None


def load() -> ctypes.CDLL:
    """Load the in-tree libhimuon.so; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m tiled_newton_schulz_b200.build`")
        lib = ctypes.CDLL(LIB_PATH)
        P, vp, i32, i64 = ctypes.POINTER, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        ns_sig = [P(Mat), P(Mat), i32, P(Split), P(Params), vp, ctypes.c_size_t, vp]
        for name in ("himuon_ns_tiled", "himuon_ns_full", "himuon_gram_ns"):
            getattr(lib, name).argtypes = ns_sig
            getattr(lib, name).restype = ctypes.c_int
        lib.himuon_ns_static.argtypes = [P(Mat), P(Mat), i32, P(Split), P(Params), vp]
        lib.himuon_ns_static.restype = ctypes.c_int
        lib.himuon_momentum_step.argtypes = [P(Mat), P(Mat), P(Mat), i32, ctypes.c_float, ctypes.c_float, P(Split),
                                             P(Params), P(Mat), vp, ctypes.c_size_t, vp]
        lib.himuon_momentum_step.restype = ctypes.c_int
        lib.himuon_workspace_size.argtypes = [P(Mat), i32, P(Split), P(Params), i32]
        lib.himuon_workspace_size.restype = i64
        lib.himuon_get_device_status.argtypes = [vp]
        lib.himuon_get_device_status.restype = ctypes.c_int
        lib.himuon_status_string.argtypes = [ctypes.c_int]
        lib.himuon_status_string.restype = ctypes.c_char_p
        lib.himuon_version.restype = ctypes.c_int
        lib.himuon_launch_count.restype = i64
        lib.himuon_plan_tiles.argtypes = [P(Mat), i32, P(Split), i32, P(i64), i64]
        lib.himuon_plan_tiles.restype = i64
        f32 = ctypes.c_float
        lib.himuon_expert_product.argtypes = [P(Mat), vp, i32, vp, i32, P(Mat), vp]
        lib.himuon_expert_gradient.argtypes = [P(Mat), P(Mat), i32, vp, f32, f32, vp, vp, vp]
        lib.himuon_quantize.argtypes = [vp, i32, i32, vp, vp, vp]
        lib.himuon_expert_product_i8.argtypes = [P(Mat), P(Mat), vp, P(Mat), i32, vp, P(Mat), vp]
        for name in ("himuon_expert_product", "himuon_expert_gradient", "himuon_quantize",
                     "himuon_expert_product_i8"):
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
    return _lib


def status_string(code: int) -> str:
    return load().himuon_status_string(int(code)).decode()


def _check(code: int, what: str) -> None:
    if code != OK:
        raise HimuonError(code, what)


# ---------------------------------------------------------------- marshalling

_DTYPES: dict = {}


def _dtype_code(t) -> int:
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32, torch.int8: I8})
    return _DTYPES[t.dtype]


def mat(t) -> Mat:
    """himuon_mat of a 2-D tensor whose rows are contiguous (stride(1) == 1)."""
    stride = t.stride()
    if len(stride) != 2 or stride[1] != 1:
        raise ValueError("himuon needs 2-D tensors with unit column stride")
    rows, cols = t.shape
    return Mat(t.data_ptr(), rows, cols, stride[0], _dtype_code(t))


def _mats(ts) -> ctypes.Array:
    arr = (Mat * len(ts))()
    for i, t in enumerate(ts):
        arr[i] = mat(t)
    return arr


def _splits(splits, n):
    """splits: None or a list of n entries, each None or (dim, sizes)."""
    if splits is None:
        return None, []
    arr = (Split * n)()
    keep = []
    for i, s in enumerate(splits):
        if s is None:
            arr[i] = Split(0, 0, None)
            continue
        dim, sizes = s
        sz = (ctypes.c_int64 * len(sizes))(*sizes)
        keep.append(sz)
        arr[i] = Split(int(dim), len(sizes), ctypes.cast(sz, ctypes.POINTER(ctypes.c_int64)))
    return arr, keep


def params(tile: int, coeffs, steps: int | None = None, eps: float = 1e-7, compute: int = BF16,
           safety: float = 1.0, restart: Sequence[int] = (), chunk_bytes: int = 0,
           tiles: Sequence[int] | None = None):
    """himuon_ns_params.  `tiles`: None, or one T per matrix of the call (it
    then replaces `tile`; T <= 0 is the whole matrix), e.g. the output of a
    runtime tile-size schedule (``schedule.TileSchedule``, ``schedule.choose_tiles``)."""
    flat = [float(v) for tri in (coeffs if isinstance(coeffs[0], (list, tuple)) else [coeffs]) for v in tri]
    if steps is not None and len(flat) == 3:
        flat = flat * steps
    K = len(flat) // 3
    c = (ctypes.c_float * len(flat))(*flat)
    r = (ctypes.c_int32 * max(1, len(restart)))(*restart)
    p = Params(int(tile), K, ctypes.cast(c, ctypes.POINTER(ctypes.c_float)), float(eps), int(compute), float(safety),
               len(restart), ctypes.cast(r, ctypes.POINTER(ctypes.c_int32)), int(chunk_bytes), None)
    tl = None
    if tiles is not None:
        tl = (ctypes.c_int32 * max(1, len(tiles)))(*[int(t) for t in tiles])
        p.tiles = ctypes.cast(tl, ctypes.POINTER(ctypes.c_int32))
    p._keep = (c, r, tl)
    p._ntiles = None if tiles is None else len(tiles)
    return p


def _check_tiles(p: Params, n: int) -> None:
    """The library reads one tile size per matrix from p.tiles: the list must
    have exactly n entries (the C side cannot see its length)."""
    if _has_tiles(p) and getattr(p, "_ntiles", None) != n:
        raise ValueError(f"params.tiles has {getattr(p, '_ntiles', '?')} entries for {n} matrices")


def _stream(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def workspace_size(tensors, p: Params, op: int, splits=None) -> int:
    _check_tiles(p, len(tensors))
    m = _mats(tensors)
    sp, _keep = _splits(splits, len(tensors))
    n = load().himuon_workspace_size(m, len(tensors), sp, ctypes.byref(p), op)
    if n < 0:
        raise HimuonError(int(n), "himuon_workspace_size")
    return int(n)


def _workspace(tensors, p, op, splits, workspace):
    import torch
    if workspace is not None:
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    need = workspace_size(tensors, p, op, splits)
    if need == 0:
        return None, 0, None
    ws = torch.empty(need, dtype=torch.uint8, device=tensors[0].device)
    return ws.data_ptr(), need, ws


def _ns_call(fn_name, op, inputs, outputs, p, splits, workspace, stream):
    if len(inputs) != len(outputs):
        raise ValueError("inputs and outputs differ in length")
    _check_tiles(p, len(inputs))
    mi, mo = _mats(inputs), _mats(outputs)
    sp, _keep = _splits(splits, len(inputs))
    wp, wb, _ws = _workspace(inputs, p, op, splits, workspace)
    rc = getattr(load(), fn_name)(mi, mo, len(inputs), sp, ctypes.byref(p), wp, wb, _stream(stream))
    _check(rc, fn_name)
    return _ws


def _has_tiles(p: Params) -> bool:
    return bool(ctypes.cast(p.tiles, ctypes.c_void_p).value)


def ns_tiled(inputs, outputs, p: Params, splits=None, workspace=None, stream=None):
    op = OP_NS_TILED if (_has_tiles(p) or p.tile > 0) else OP_NS_FULL
    return _ns_call("himuon_ns_tiled", op, inputs, outputs, p, splits, workspace, stream)


def ns_full(inputs, outputs, p: Params, splits=None, workspace=None, stream=None):
    return _ns_call("himuon_ns_full", OP_NS_FULL, inputs, outputs, p, splits, workspace, stream)


def gram_ns(inputs, outputs, p: Params, splits=None, workspace=None, stream=None):
    return _ns_call("himuon_gram_ns", OP_GRAM_NS, inputs, outputs, p, splits, workspace, stream)


def ns_static(inputs, outputs, p: Params, splits=None, stream=None) -> int:
    """Staged NS with the library's own fixed device scratch (no workspace).

    For callers that cannot allocate device memory; returns the status code
    (ERR_TOO_LARGE when the call does not fit the 32 MiB array) instead of
    raising, so callers can fall back.
    """
    if len(inputs) != len(outputs):
        raise ValueError("inputs and outputs differ in length")
    mi, mo = _mats(inputs), _mats(outputs)
    sp, _keep = _splits(splits, len(inputs))
    return int(load().himuon_ns_static(mi, mo, len(inputs), sp, ctypes.byref(p), _stream(stream)))


def momentum_step(W, M, G, mu: float, lr: float, p: Params, splits=None, update_out=None, workspace=None,
                  stream=None):
    """M <- mu M + G; O = tiledNS(M); W <- W - lr O (W may be None); O to update_out."""
    n = len(M)
    _check_tiles(p, n)
    mw = _mats(W) if W is not None else None
    mm, mg = _mats(M), _mats(G)
    mo = _mats(update_out) if update_out is not None else None
    sp, _keep = _splits(splits, n)
    wp, wb, _ws = _workspace(M, p, OP_MOMENTUM_STEP, splits, workspace)
    rc = load().himuon_momentum_step(mw, mm, mg, n, float(mu), float(lr), sp, ctypes.byref(p), mo, wp, wb,
                                     _stream(stream))
    _check(rc, "himuon_momentum_step")
    return _ws


# ---------------------------------------------------------------- expert products
@functools.lru_cache(maxsize=256)
def _stack_layout(n: int, rows: int, cols: int, ld: int, dtype: int, step: int):
    """The records of n matrices `step` bytes apart as five 64-bit words each,
    the first matrix at address 0."""
    import numpy as np
    rec = np.empty((n, 5), np.int64)
    rec[:, 0] = np.arange(n) * step
    rec[:, 1:] = (rows, cols, ld, dtype)
    return rec


def _stack(ts):
    """(himuon_mat array, its address, n) of a list of 2-D tensors or of a 3-D
    tensor of stacked matrices (unit column stride)."""
    if isinstance(ts, (list, tuple)):
        arr = _mats(ts)
        return arr, ctypes.addressof(arr), len(ts)
    stride = ts.stride()
    if len(stride) != 3 or stride[2] != 1:
        raise ValueError("stacked matrices are a 3-D tensor with unit column stride")
    n, rows, cols = ts.shape
    rec = _stack_layout(n, rows, cols, stride[1], _dtype_code(ts), stride[0] * ts.element_size()).copy()
    rec[:, 0] += ts.data_ptr()
    return rec, rec.ctypes.data, n


def _row_vector(t) -> Mat:
    """himuon_mat of a contiguous 1-D tensor (a 1 x len matrix)."""
    if t.dim() != 1 or (t.shape[0] > 1 and t.stride(0) != 1):
        raise ValueError("scales are contiguous 1-D tensors")
    return Mat(t.data_ptr(), 1, t.shape[0], max(1, t.shape[0]), _dtype_code(t))


def _one_device(*operands) -> int:
    """The index of the CUDA device that every tensor of the operands (tensors,
    lists of them or None) is on."""
    devs = set()
    for op in operands:
        if isinstance(op, (list, tuple)):
            devs.update([t.get_device() for t in op])
        elif op is not None:
            devs.add(op.get_device())
    dev = devs.pop() if len(devs) == 1 else -1
    if dev < 0:
        raise ValueError("expert products need all their tensors on one CUDA device")
    return dev


def _offsets(offsets, n):
    if offsets is None:
        return None
    import torch
    if offsets.dtype is not torch.int32 or offsets.shape != (n + 1,) or not offsets.is_contiguous():
        raise ValueError(f"offsets are a contiguous int32 tensor of n + 1 = {n + 1} entries")
    return offsets.data_ptr()


def _on_device(dev, name, stream, *args):
    """Calls the entry point with the operands' device current, on `stream` or
    on that device's current stream."""
    import torch
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError("the stream is on another device than the tensors")
        raw = stream.cuda_stream
    else:
        raw = torch._C._cuda_getCurrentRawStream(dev)   # (current_stream builds an object: 2 us)
    fn = getattr(load(), name)
    if torch.cuda.current_device() == dev:
        code = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            code = fn(*args, raw)
    _check(code, name)


def expert_product(X, W, Y, offsets=None, w_trans: bool = False, stream=None) -> None:
    """Y[r] = X[r] W_e (W_e: K x N), or X[r] W_e^T with `w_trans` (W_e: N x K),
    for the rows r of every group e.

    X: rows x K, Y: rows x N; W: a list of n matrices or a 3-D tensor;
    `offsets`: int32 CUDA tensor of n + 1 row bounds (None: n = 1, all rows).
    Rows outside every group are left as they were.
    """
    dev = _one_device(X, W, Y, offsets)
    keep, w, n = _stack(W)
    _on_device(dev, "himuon_expert_product", stream, mat(X), w, n, _offsets(offsets, n), int(bool(w_trans)), mat(Y))


def expert_gradient(A, B, G, offsets=None, alpha: float = 1.0, beta: float = 0.0, C=None, stream=None) -> None:
    """G_e = alpha * A[rows of e]^T B[rows of e] + beta * C_e for every group e.

    A: rows x P, B: rows x Q; G and C: lists of n P x Q matrices or 3-D
    tensors (C may be G; not read with beta = 0).  An empty group gives
    beta * C_e.
    """
    dev = _one_device(A, B, G, C, offsets)
    keep, g, n = _stack(G)
    keep_c, c, nc = _stack(C) if C is not None else (None, None, n)
    if nc != n:
        raise ValueError("G and C differ in length")
    _on_device(dev, "himuon_expert_gradient", stream, mat(A), mat(B), n, _offsets(offsets, n), float(alpha),
               float(beta), c, g)


def quantize(inputs, codes, scales, dim: int = 0, stream=None) -> None:
    """8-bit codes of each matrix: one scale per row (dim 0), or per column
    with the codes transposed (dim 1).

    inputs: list of 2-D float tensors, or a 3-D tensor of stacked matrices;
    codes: int8, likewise (transposed shape for dim 1); scales: list of 1-D fp32
    tensors, or a 2-D tensor with a row per matrix.
    """
    if not len(inputs) == len(codes) == len(scales):
        raise ValueError("inputs, codes and scales differ in length")
    dev = _one_device(inputs, codes, scales)
    keep_i, i, n = _stack(inputs)
    keep_c, c, _ = _stack(codes)
    if isinstance(scales, (list, tuple)):
        keep_s = (Mat * max(1, n))(*[_row_vector(s) for s in scales])
        s = ctypes.addressof(keep_s)
    else:
        keep_s, s, _ = _stack(scales.unsqueeze(1))
    _on_device(dev, "himuon_quantize", stream, i, n, int(dim), c, s)


def expert_product_i8(X, x_scale, W, w_scale, Y, offsets=None, stream=None) -> None:
    """Y[r, c] = x_scale[r] * w_scale[e, c] * sum_k X[r, k] W_e[c, k] for the
    rows r of every group e, the sum exact in int32.

    X: int8 rows x K, x_scale: fp32 per row, W: n int8 matrices N x K (list or
    3-D tensor), w_scale: fp32 n x N, Y: rows x N.
    """
    dev = _one_device(X, x_scale, W, w_scale, Y, offsets)
    keep, w, n = _stack(W)
    _on_device(dev, "himuon_expert_product_i8", stream, mat(X), _row_vector(x_scale), w, mat(w_scale), n,
               _offsets(offsets, n), mat(Y))


def launch_count() -> int:
    """Kernels the library has enqueued since it was loaded (host counter)."""
    return int(load().himuon_launch_count())


def device_status(stream=None) -> int:
    return int(load().himuon_get_device_status(_stream(stream)))


def plan_tiles(shapes, splits=None, tile: int = 128):
    """Tile list the scheduler numbers, as (matrix, row0, col0, h, w) tuples.

    Host-only: the matrices are described by shape alone (a dummy pointer).
    """
    n = len(shapes)
    arr = (Mat * n)()
    for i, (r, c) in enumerate(shapes):
        arr[i] = Mat(0x1000, r, c, c, BF16)
    sp, _keep = _splits(splits, n)
    lib = load()
    total = lib.himuon_plan_tiles(arr, n, sp, int(tile), None, 0)
    if total < 0:
        raise HimuonError(int(total), "himuon_plan_tiles")
    rec = (ctypes.c_int64 * (5 * max(1, total)))()
    lib.himuon_plan_tiles(arr, n, sp, int(tile), rec, total)
    return [tuple(rec[5 * i:5 * i + 5]) for i in range(total)]
