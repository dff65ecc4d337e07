"""Thin Python binding of ``libpurlin.so`` (the C ABI in ``include/purlin.h``).

Argument marshalling only: every step of a collective runs in the library's
CUDA kernels.  There is no fallback: if the shared library is missing or
cannot be loaded, importing this package raises.

Buffers may be given as torch CUDA tensors or as integer device addresses.
Function names match the C ABI; a non-OK status raises :class:`PurlinError`.
"""
from __future__ import annotations

import ctypes
import os
from typing import Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpurlin.so")

PURLIN_MAX_RANKS = 64
PURLIN_MAX_GROUPS = 1024

PURLIN_F32, PURLIN_BF16, PURLIN_E4M3 = 0, 1, 2
PURLIN_COPY, PURLIN_SUM = 0, 1
PURLIN_PACKED, PURLIN_SCATTERED, PURLIN_TRANSPOSED = 0, 1, 2
PURLIN_WEIGHTS_NK, PURLIN_WEIGHTS_KN = 0, 1
PURLIN_GATE_COLUMNS, PURLIN_GATE_ROWS = 0, 1
PURLIN_SOFTMAX, PURLIN_SIGMOID = 0, 1

PURLIN_OK = 0
PURLIN_ERR_INVALID_ARG = 1
PURLIN_ERR_ALIGNMENT = 2
PURLIN_ERR_UNSUPPORTED = 3
PURLIN_ERR_ALIAS = 4
PURLIN_ERR_OOM = 5
PURLIN_ERR_CUDA = 6
PURLIN_ERR_TIMEOUT = 7

(PURLIN_OPT_VARIANT, PURLIN_OPT_CROSSOVER_BYTES, PURLIN_OPT_AR_MODE, PURLIN_OPT_CHUNK_BYTES,
 PURLIN_OPT_STAGES, PURLIN_OPT_CTAS, PURLIN_OPT_SPIN_TIMEOUT_NS, PURLIN_OPT_DROP_NOTIFY,
 PURLIN_OPT_LAT_CTAS, PURLIN_OPT_LAT_BLOCK, PURLIN_OPT_CONSUMER_WARPS,
 PURLIN_OPT_COPY_STORES) = range(12)

(PURLIN_COLL_ALL_REDUCE, PURLIN_COLL_REDUCE_SCATTER, PURLIN_COLL_ALL_GATHER,
 PURLIN_COLL_ALL_TO_ALL, PURLIN_COLL_ALL_GATHER_V, PURLIN_COLL_REDUCE_SCATTER_V,
 PURLIN_COLL_ALL_TO_ALL_V) = range(7)

# The one legal (op, layout) pair of each collective
# ("Purlin: Separating Orchestration from the Datapath of Collectives" §3.1).
LAYOUTS = {
    "all_reduce": (PURLIN_SUM, (PURLIN_SCATTERED, PURLIN_SCATTERED)),
    "reduce_scatter": (PURLIN_SUM, (PURLIN_SCATTERED, PURLIN_PACKED)),
    "all_gather": (PURLIN_COPY, (PURLIN_PACKED, PURLIN_SCATTERED)),
    "all_to_all": (PURLIN_COPY, (PURLIN_SCATTERED, PURLIN_TRANSPOSED)),
    "all_gather_v": (PURLIN_COPY, (PURLIN_PACKED, PURLIN_SCATTERED)),
    "reduce_scatter_v": (PURLIN_SUM, (PURLIN_SCATTERED, PURLIN_PACKED)),
    "all_to_all_v": (PURLIN_COPY, (PURLIN_SCATTERED, PURLIN_TRANSPOSED)),
}


class purlin_layout(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_int32), ("out", ctypes.c_int32)]


class purlin_launch_info(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int32), ("grid", ctypes.c_int32), ("block", ctypes.c_int32),
                ("stages", ctypes.c_int32), ("chunk_bytes", ctypes.c_int64),
                ("chunks", ctypes.c_int64), ("units", ctypes.c_int64),
                ("segments", ctypes.c_int64), ("smem_bytes", ctypes.c_int64),
                ("epoch", ctypes.c_uint64), ("epoch_next", ctypes.c_uint64)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class purlin_segment(ctypes.Structure):
    _fields_ = [("src_off", ctypes.c_uint64), ("dst_off", ctypes.c_uint64),
                ("bytes", ctypes.c_uint64), ("src_rank", ctypes.c_int32),
                ("dst_rank", ctypes.c_int32), ("skip_rank", ctypes.c_int32),
                ("src_is_dst", ctypes.c_int32), ("sync", ctypes.c_int32), ("tma", ctypes.c_int32),
                ("shift", ctypes.c_int32), ("head_bytes", ctypes.c_uint64), ("tail_bytes", ctypes.c_uint64),
                ("chunk_begin", ctypes.c_uint64), ("chunk_bytes", ctypes.c_uint64),
                ("unit_begin", ctypes.c_uint64)]

    def as_dict(self):
        return {name: getattr(self, name) for name, _ in self._fields_}


class purlin_device_coll(ctypes.Structure):
    """A collective compiled for device-side calls (include/purlin.h)."""
    _fields_ = [("src", ctypes.c_void_p * PURLIN_MAX_RANKS),
                ("dst", ctypes.c_void_p * PURLIN_MAX_RANKS),
                ("segs", ctypes.c_void_p), ("flags", ctypes.c_void_p),
                ("epochs", ctypes.c_void_p), ("err", ctypes.c_void_p),
                ("nchunks", ctypes.c_uint64), ("nunits", ctypes.c_uint64),
                ("epoch_inc", ctypes.c_uint64), ("timeout_ns", ctypes.c_int64),
                ("drop_notify", ctypes.c_int64), ("flag_slots", ctypes.c_uint32),
                ("stages", ctypes.c_uint32), ("slot_stride", ctypes.c_uint32),
                ("workspace_bytes", ctypes.c_uint32), ("nseg", ctypes.c_int32),
                ("R", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("vector_copies", ctypes.c_int32), ("blocks", ctypes.c_int32),
                ("threads", ctypes.c_int32), ("composed", ctypes.c_int32),
                ("coll", ctypes.c_int32), ("ragged", ctypes.c_int32),
                ("owner", ctypes.c_void_p)]


class purlin_router(ctypes.Structure):
    """How tokens are routed to experts (include/purlin.h).  Fields left out are
    0: one group, its value the largest choice, a scale of 1."""
    _fields_ = [("experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("scores", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("top_groups", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("renormalise", ctypes.c_int32), ("scale", ctypes.c_float)]


class purlin_packet_channel(ctypes.Structure):
    """A payload+flag packet channel between CTAs of one launch (include/purlin.h)."""
    _fields_ = [("staging", ctypes.c_void_p), ("state", ctypes.c_void_p),
                ("capacity", ctypes.c_uint64), ("timeout_ns", ctypes.c_int64),
                ("drop_unit", ctypes.c_int64), ("ctas", ctypes.c_int32),
                ("pad", ctypes.c_int32), ("owner", ctypes.c_void_p)]


class PurlinError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = int(status)
        super().__init__(f"{what}: {status_string(status)} (status {status})")


# Exported symbols and their C signatures (kept in step with include/purlin.h).
_VPP = ctypes.POINTER(ctypes.c_void_p)
_SZP = ctypes.POINTER(ctypes.c_size_t)
_VP, _SZ = ctypes.c_void_p, ctypes.c_size_t
_CTX = ctypes.c_void_p
_SIGNATURES = {
    "purlin_init": (ctypes.c_int, [ctypes.c_int, ctypes.c_void_p, ctypes.POINTER(_CTX)]),
    "purlin_finalize": (ctypes.c_int, [_CTX]),
    "purlin_set_stream": (ctypes.c_int, [_CTX, ctypes.c_void_p]),
    "purlin_all_reduce": (ctypes.c_int, [_CTX, _VPP, _VPP, ctypes.c_size_t, ctypes.c_int,
                                         ctypes.c_int, purlin_layout]),
    "purlin_reduce_scatter": (ctypes.c_int, [_CTX, _VPP, _VPP, ctypes.c_size_t, ctypes.c_int,
                                             ctypes.c_int, purlin_layout]),
    "purlin_all_gather": (ctypes.c_int, [_CTX, _VPP, _VPP, ctypes.c_size_t, ctypes.c_int,
                                         ctypes.c_int, purlin_layout]),
    "purlin_all_to_all": (ctypes.c_int, [_CTX, _VPP, _VPP, ctypes.c_size_t, ctypes.c_int,
                                         ctypes.c_int, purlin_layout]),
    "purlin_all_gather_v": (ctypes.c_int, [_CTX, _VPP, _VPP, _SZP, ctypes.c_int, ctypes.c_int,
                                           purlin_layout]),
    "purlin_reduce_scatter_v": (ctypes.c_int, [_CTX, _VPP, _VPP, _SZP, ctypes.c_int,
                                               ctypes.c_int, purlin_layout]),
    "purlin_all_to_all_v": (ctypes.c_int, [_CTX, _VPP, _VPP, _SZP, ctypes.c_int, ctypes.c_int,
                                           purlin_layout]),
    "purlin_all_gather_v_device_counts": (ctypes.c_int, [
        _CTX, _VPP, _VPP, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_size_t, ctypes.c_int,
        ctypes.c_int, purlin_layout]),
    "purlin_reduce_scatter_v_device_counts": (ctypes.c_int, [
        _CTX, _VPP, _VPP, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_size_t, ctypes.c_int,
        ctypes.c_int, purlin_layout]),
    "purlin_all_to_all_v_device_counts": (ctypes.c_int, [
        _CTX, _VPP, _VPP, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_size_t, ctypes.c_int,
        ctypes.c_int, purlin_layout]),
    "purlin_all_reduce_noalloc": (ctypes.c_int, [ctypes.c_int, _VPP, _VPP, ctypes.c_size_t,
                                                 ctypes.c_int, ctypes.c_int, purlin_layout,
                                                 ctypes.c_void_p]),
    "purlin_noalloc_check": (ctypes.c_int, [ctypes.c_void_p]),
    "purlin_rms_norm": (ctypes.c_int, [
        _CTX, _VP, _SZ, _VP, _SZ, _VP, _VP, _SZ, _VP, _SZ, _VP, _SZ, _SZ, ctypes.c_float,
        ctypes.c_int, ctypes.c_int]),
    "purlin_rms_norm_backward": (ctypes.c_int, [
        _CTX, _VP, _SZ, _VP, _SZ, _VP, _VP, _SZ, _VP, _SZ, _VP, _SZ, _SZ, ctypes.c_float,
        ctypes.c_int]),
    "purlin_grouped_matmul": (ctypes.c_int, [
        _CTX, _VP, _SZ, _VP, _SZ, _VP, _SZ, _VP, _VP, _VP, _VP, ctypes.c_int, _SZ, _SZ, _SZ,
        ctypes.c_int, ctypes.c_int]),
    "purlin_grouped_matmul_weight_grad": (ctypes.c_int, [
        _CTX, _VP, _SZ, _VP, _SZ, _VP, _SZ, _VP, _VP, ctypes.c_int, _SZ, _SZ, _SZ,
        ctypes.c_int]),
    "purlin_block_norm": (ctypes.c_int, [
        _CTX, _VP, _SZ, _VP, _VP, _SZ, ctypes.c_int, ctypes.c_float, _VP, _SZ, ctypes.c_float, _VP,
        _VP, _SZ, _VP, _SZ, _VP, _SZ, _SZ, ctypes.c_float, ctypes.c_int, ctypes.c_int]),
    "purlin_block_norm_backward": (ctypes.c_int, [
        _CTX, _VP, _SZ, _VP, _SZ, _VP, _SZ, _VP, _SZ, _VP, _VP, _SZ, ctypes.c_int, ctypes.c_float,
        ctypes.c_float, _VP, _VP, _SZ, _VP, _SZ, _VP, _VP, _SZ, _VP, _SZ, _SZ, ctypes.c_float,
        ctypes.c_int]),
    "purlin_route": (ctypes.c_int, [
        _CTX, _VP, _SZ, _VP, _VP, _VP, _SZ, ctypes.POINTER(purlin_router), ctypes.c_int]),
    "purlin_route_backward": (ctypes.c_int, [
        _CTX, _VP, _VP, _SZ, _VP, _VP, _SZ, _SZ, ctypes.POINTER(purlin_router), ctypes.c_int]),
    "purlin_expert_order": (ctypes.c_int, [
        _CTX, _VP, _VP, _VP, _VP, _SZ, ctypes.c_int, _SZ]),
    "purlin_dispatch_rows": (ctypes.c_int, [
        _CTX, _VP, _SZ, _VP, _VP, _VP, _SZ, _VP, _SZ, ctypes.c_int, _SZ, _SZ, ctypes.c_int]),
    "purlin_combine_rows": (ctypes.c_int, [
        _CTX, _VP, _SZ, _VP, _VP, _VP, _SZ, _VP, _SZ, _SZ, ctypes.c_int, _SZ, _SZ, ctypes.c_int]),
    "purlin_combine_rows_backward": (ctypes.c_int, [
        _CTX, _VP, _SZ, _VP, _SZ, _VP, _VP, _VP, _SZ, _VP, _SZ, ctypes.c_int, _SZ, _SZ,
        ctypes.c_int]),
    "purlin_empty_launch": (ctypes.c_int, [ctypes.c_void_p]),
    "purlin_touch_launch": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "purlin_check": (ctypes.c_int, [_CTX]),
    "purlin_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "purlin_set_option": (ctypes.c_int, [_CTX, ctypes.c_int, ctypes.c_int64]),
    "purlin_get_option": (ctypes.c_int, [_CTX, ctypes.c_int, ctypes.POINTER(ctypes.c_int64)]),
    "purlin_last_launch": (ctypes.c_int, [_CTX, ctypes.POINTER(purlin_launch_info)]),
    "purlin_plan_inspect": (ctypes.c_int, [
        ctypes.c_int, ctypes.c_int, _VPP, _VPP, ctypes.c_size_t, _SZP, ctypes.c_int, ctypes.c_int,
        purlin_layout, ctypes.c_int, ctypes.c_int, ctypes.c_uint64,
        ctypes.POINTER(purlin_segment), ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t),
        ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(ctypes.c_uint64)]),
    "purlin_device_prepare": (ctypes.c_int, [
        _CTX, ctypes.c_int, _VPP, _VPP, ctypes.c_size_t, _SZP, ctypes.c_int, ctypes.c_int,
        purlin_layout, ctypes.c_int, ctypes.c_uint32, ctypes.POINTER(purlin_device_coll)]),
    "purlin_device_check": (ctypes.c_int, [ctypes.POINTER(purlin_device_coll), ctypes.c_void_p]),
    "purlin_device_release": (ctypes.c_int, [_CTX, ctypes.POINTER(purlin_device_coll)]),
    "purlin_device_coll_size": (ctypes.c_size_t, []),
    "purlin_packet_channel_create": (ctypes.c_int, [_CTX, ctypes.c_size_t, ctypes.c_int,
                                                    ctypes.POINTER(purlin_packet_channel)]),
    "purlin_packet_channel_check": (ctypes.c_int, [ctypes.POINTER(purlin_packet_channel),
                                                   ctypes.c_void_p]),
    "purlin_packet_channel_release": (ctypes.c_int, [_CTX, ctypes.POINTER(purlin_packet_channel)]),
}


def _load_library():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it first (python -c 'import __graft_entry__ as g; "
            "g.build()'); this package has no fallback path")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


lib = _load_library()


def status_string(status: int) -> str:
    return lib.purlin_status_string(int(status)).decode()


def _ok(status: int, what: str):
    if status != PURLIN_OK:
        raise PurlinError(status, what)


def _addr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _ptr_array(bufs: Sequence):
    arr = (ctypes.c_void_p * max(1, len(bufs)))()
    for i, b in enumerate(bufs):
        arr[i] = _addr(b)
    return ctypes.cast(arr, _VPP), arr


def _size_array(xs):
    xs = [int(x) for x in xs]
    arr = (ctypes.c_size_t * max(1, len(xs)))(*xs)
    return ctypes.cast(arr, _SZP), arr


def _layout(layout):
    return purlin_layout(int(layout[0]), int(layout[1]))


def _stream_handle(stream) -> int:
    if stream is None:
        return 0
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


class Context:
    """Owns one ``purlin_ctx*``; calls ``purlin_finalize`` on close."""

    def __init__(self, handle: int, R: int, stream_handle: int = 0):
        self.handle = ctypes.c_void_p(handle)
        self.R = R
        self.stream_handle = stream_handle   # the cudaStream_t that calls launch on

    def close(self):
        if self.handle:
            _ok(lib.purlin_finalize(self.handle), "purlin_finalize")
            self.handle = ctypes.c_void_p(0)

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()
        return False


# ----------------------------------------------------------- C ABI names ---

def purlin_init(R: int, stream=None) -> Context:
    h = ctypes.c_void_p(0)
    _ok(lib.purlin_init(int(R), ctypes.c_void_p(_stream_handle(stream)), ctypes.byref(h)),
        "purlin_init")
    return Context(h.value, int(R), _stream_handle(stream))


def purlin_finalize(ctx: Context):
    ctx.close()


def purlin_set_stream(ctx: Context, stream):
    _ok(lib.purlin_set_stream(ctx.handle, ctypes.c_void_p(_stream_handle(stream))),
        "purlin_set_stream")
    ctx.stream_handle = _stream_handle(stream)


def _uniform(fn, name, ctx, src, dst, n, dtype, op, layout):
    dflt_op, dflt_layout = LAYOUTS[name]
    op = dflt_op if op is None else op
    layout = dflt_layout if layout is None else layout
    ps, _keep1 = _ptr_array(src)
    pd, _keep2 = _ptr_array(dst)
    _ok(fn(ctx.handle, ps, pd, int(n), int(dtype), int(op), _layout(layout)), f"purlin_{name}")


def _varlen(fn, name, ctx, src, dst, counts, dtype, op, layout):
    dflt_op, dflt_layout = LAYOUTS[name]
    op = dflt_op if op is None else op
    layout = dflt_layout if layout is None else layout
    ps, _keep1 = _ptr_array(src)
    pd, _keep2 = _ptr_array(dst)
    pc, _keep3 = _size_array(counts)
    _ok(fn(ctx.handle, ps, pd, pc, int(dtype), int(op), _layout(layout)), f"purlin_{name}")


def purlin_all_reduce(ctx, src, dst, n, dtype, op=None, layout=None):
    _uniform(lib.purlin_all_reduce, "all_reduce", ctx, src, dst, n, dtype, op, layout)


def purlin_reduce_scatter(ctx, src, dst, n, dtype, op=None, layout=None):
    _uniform(lib.purlin_reduce_scatter, "reduce_scatter", ctx, src, dst, n, dtype, op, layout)


def purlin_all_gather(ctx, src, dst, n, dtype, op=None, layout=None):
    _uniform(lib.purlin_all_gather, "all_gather", ctx, src, dst, n, dtype, op, layout)


def purlin_all_to_all(ctx, src, dst, n, dtype, op=None, layout=None):
    _uniform(lib.purlin_all_to_all, "all_to_all", ctx, src, dst, n, dtype, op, layout)


def purlin_all_gather_v(ctx, src, dst, counts, dtype, op=None, layout=None):
    _varlen(lib.purlin_all_gather_v, "all_gather_v", ctx, src, dst, counts, dtype, op, layout)


def purlin_reduce_scatter_v(ctx, src, dst, counts, dtype, op=None, layout=None):
    _varlen(lib.purlin_reduce_scatter_v, "reduce_scatter_v", ctx, src, dst, counts, dtype, op,
            layout)


def purlin_all_to_all_v(ctx, src, dst, counts, dtype, op=None, layout=None):
    """``counts``: R*R element counts, row s = source, column d = destination."""
    _varlen(lib.purlin_all_to_all_v, "all_to_all_v", ctx, src, dst, counts, dtype, op, layout)


def _device_counts(fn, name, ctx, src, dst, counts, in_capacity, out_capacity, dtype, op,
                   layout):
    dflt_op, dflt_layout = LAYOUTS[name]
    op = dflt_op if op is None else op
    layout = dflt_layout if layout is None else layout
    ps, _keep1 = _ptr_array(src)
    pd, _keep2 = _ptr_array(dst)
    _ok(fn(ctx.handle, ps, pd, ctypes.c_void_p(_addr(counts)), int(in_capacity),
           int(out_capacity), int(dtype), int(op), _layout(layout)),
        f"purlin_{name}_device_counts")


def purlin_all_gather_v_device_counts(ctx, src, dst, counts, in_capacity, out_capacity, dtype,
                                      op=None, layout=None):
    """AllGatherV with the R counts in device memory (a tensor of int64 or a
    device address)."""
    _device_counts(lib.purlin_all_gather_v_device_counts, "all_gather_v", ctx, src, dst, counts,
                   in_capacity, out_capacity, dtype, op, layout)


def purlin_reduce_scatter_v_device_counts(ctx, src, dst, counts, in_capacity, out_capacity,
                                          dtype, op=None, layout=None):
    _device_counts(lib.purlin_reduce_scatter_v_device_counts, "reduce_scatter_v", ctx, src, dst,
                   counts, in_capacity, out_capacity, dtype, op, layout)


def purlin_all_to_all_v_device_counts(ctx, src, dst, counts, in_capacity, out_capacity, dtype,
                                      op=None, layout=None):
    """AllToAllV with the R*R count matrix (row = source) in device memory."""
    _device_counts(lib.purlin_all_to_all_v_device_counts, "all_to_all_v", ctx, src, dst, counts,
                   in_capacity, out_capacity, dtype, op, layout)


def purlin_all_reduce_noalloc(R, src, dst, n, dtype, op=None, layout=None, stream=None):
    """AllReduce with no device allocation (static scratch inside the
    library); see include/purlin.h for its limits."""
    dflt_op, dflt_layout = LAYOUTS["all_reduce"]
    op = dflt_op if op is None else op
    layout = dflt_layout if layout is None else layout
    ps, _keep1 = _ptr_array(src)
    pd, _keep2 = _ptr_array(dst)
    _ok(lib.purlin_all_reduce_noalloc(int(R), ps, pd, int(n), int(dtype), int(op),
                                      _layout(layout), ctypes.c_void_p(_stream_handle(stream))),
        "purlin_all_reduce_noalloc")


def purlin_noalloc_check(stream=None):
    """Synchronize `stream` and raise if a device-side wait of an
    allocation-free AllReduce expired since the last check."""
    _ok(lib.purlin_noalloc_check(ctypes.c_void_p(_stream_handle(stream))), "purlin_noalloc_check")


# ------------------------------------------------------ layer operators ---

def purlin_rms_norm(ctx, x, weight, y, rows, hidden, eps, dtype, out_dtype=None, residual=None,
                    total=None, scales=None, ldx=0, ldr=0, ldy=0, ldt=0):
    """Norm of ``x + residual``; ``out_dtype`` (default ``dtype``) PURLIN_E4M3
    writes 8-bit rows and ``scales``.  Strides 0: contiguous rows."""
    st = lib.purlin_rms_norm(ctx.handle, _addr(x), ldx, _addr(residual), ldr, _addr(weight),
                             _addr(y), ldy, _addr(total), ldt, _addr(scales), rows, hidden, eps,
                             dtype, dtype if out_dtype is None else out_dtype)
    if st:
        _ok(st, "purlin_rms_norm")


def purlin_rms_norm_backward(ctx, dy, total, weight, dx, dweight, rows, hidden, eps, dtype,
                             dtotal=None, lddy=0, ldt=0, lddt=0, lddx=0):
    """Gradients of :func:`purlin_rms_norm` at ``total``; ``dweight`` is float32."""
    st = lib.purlin_rms_norm_backward(ctx.handle, _addr(dy), lddy, _addr(total), ldt,
                                      _addr(weight), _addr(dtotal), lddt, _addr(dx), lddx,
                                      _addr(dweight), rows, hidden, eps, dtype)
    if st:
        _ok(st, "purlin_rms_norm_backward")


def purlin_grouped_matmul(ctx, x, w, y, begin, count, groups, rows, n, k, dtype,
                          layout=PURLIN_WEIGHTS_NK, x_scales=None, w_scales=None, ldx=0, ldw=0,
                          ldy=0):
    """Products grouped by expert; ``begin`` and ``count`` are device int64
    arrays (tensors or addresses) of each group's first row and row count."""
    st = lib.purlin_grouped_matmul(ctx.handle, _addr(x), ldx, _addr(w), ldw, _addr(y), ldy,
                                   _addr(x_scales), _addr(w_scales), _addr(begin), _addr(count),
                                   groups, rows, n, k, dtype, layout)
    if st:
        _ok(st, "purlin_grouped_matmul")


def purlin_grouped_matmul_weight_grad(ctx, dy, x, dw, begin, count, groups, rows, n, k, dtype,
                                      lddy=0, ldx=0, lddw=0):
    """Weight gradient of :func:`purlin_grouped_matmul`: ``dw`` is groups x n x k."""
    st = lib.purlin_grouped_matmul_weight_grad(ctx.handle, _addr(dy), lddy, _addr(x), ldx,
                                               _addr(dw), lddw, _addr(begin), _addr(count),
                                               groups, rows, n, k, dtype)
    if st:
        _ok(st, "purlin_grouped_matmul_weight_grad")


def purlin_block_norm(ctx, x, weight, y, rows, hidden, eps, dtype, out_dtype=None, residual=None,
                      post_weight=None, gate=None, gate_layout=PURLIN_GATE_COLUMNS,
                      residual_scale=1.0, block_scale=1.0, total=None, scales=None, ldx=0, ldg=0,
                      ldr=0, ldy=0, ldt=0):
    """Norms after and before a block, with its gate and the residual's addition
    between them; ``out_dtype`` PURLIN_E4M3 writes ``scales``.  ``weight`` and
    ``y`` None: only ``total``."""
    st = lib.purlin_block_norm(ctx.handle, _addr(x), ldx, _addr(post_weight), _addr(gate), ldg,
                               gate_layout, block_scale, _addr(residual), ldr, residual_scale,
                               _addr(weight), _addr(y), ldy, _addr(total), ldt, _addr(scales),
                               rows, hidden, eps, dtype, dtype if out_dtype is None else out_dtype)
    if st:
        _ok(st, "purlin_block_norm")


def purlin_block_norm_backward(ctx, dy, x, total, weight, dx, dweight, rows, hidden, eps, dtype,
                               dtotal=None, post_weight=None, gate=None,
                               gate_layout=PURLIN_GATE_COLUMNS, residual_scale=1.0,
                               block_scale=1.0, dresidual=None, dpost_weight=None, dgate=None,
                               lddy=0, lddt=0, ldx=0, ldt=0, ldg=0, lddx=0, lddr=0, lddg=0):
    """Gradients of :func:`purlin_block_norm` at ``x`` and ``total``; ``dweight``,
    ``dpost_weight`` and a column gate's ``dgate`` are float32."""
    st = lib.purlin_block_norm_backward(
        ctx.handle, _addr(dy), lddy, _addr(dtotal), lddt, _addr(x), ldx, _addr(total), ldt,
        _addr(post_weight), _addr(gate), ldg, gate_layout, block_scale, residual_scale,
        _addr(weight), _addr(dx), lddx, _addr(dresidual), lddr, _addr(dpost_weight), _addr(dgate),
        lddg, _addr(dweight), rows, hidden, eps, dtype)
    if st:
        _ok(st, "purlin_block_norm_backward")


def purlin_route(ctx, logits, weights, chosen, tokens, router, dtype, bias=None, ld=0):
    """Each token's ``top_k`` experts (int32, falling) and their weights (float32)
    from its logits; ``router`` is a :class:`purlin_router`."""
    st = lib.purlin_route(ctx.handle, _addr(logits), ld, _addr(bias), _addr(weights),
                          _addr(chosen), tokens, ctypes.byref(router), dtype)
    if st:
        _ok(st, "purlin_route")


def purlin_route_backward(ctx, dweights, logits, chosen, dlogits, tokens, router, dtype, ld=0,
                          ldd=0):
    """Gradient of :func:`purlin_route`'s weights with respect to the logits."""
    st = lib.purlin_route_backward(ctx.handle, _addr(dweights), _addr(logits), ld, _addr(chosen),
                                   _addr(dlogits), ldd, tokens, ctypes.byref(router), dtype)
    if st:
        _ok(st, "purlin_route_backward")


def purlin_expert_order(ctx, chosen, place, begin, count, slots, groups, capacity=0):
    """The row of each slot in the order of the experts, packed or in buffers of
    ``capacity`` rows (-1 past it), and the experts' first rows and counts (int64)."""
    st = lib.purlin_expert_order(ctx.handle, _addr(chosen), _addr(place), _addr(begin),
                                 _addr(count), slots, groups, capacity)
    if st:
        _ok(st, "purlin_expert_order")


def purlin_dispatch_rows(ctx, x, place, out, tokens, top_k, cols, out_rows, dtype, scales=None,
                         out_scales=None, ldx=0, ldo=0):
    """A copy of each token's row (and scale) at each of its places."""
    st = lib.purlin_dispatch_rows(ctx.handle, _addr(x), ldx, _addr(scales), _addr(place),
                                  _addr(out), ldo, _addr(out_scales), tokens, top_k, cols,
                                  out_rows, dtype)
    if st:
        _ok(st, "purlin_dispatch_rows")


def purlin_combine_rows(ctx, rows, place, y, tokens, top_k, cols, n_rows, dtype, weights=None,
                        shared=None, ldr=0, lds=0, ldy=0):
    """The weighted sum of the rows at a token's places, on ``shared`` if given."""
    st = lib.purlin_combine_rows(ctx.handle, _addr(rows), ldr, _addr(weights), _addr(place),
                                 _addr(shared), lds, _addr(y), ldy, tokens, top_k, cols, n_rows,
                                 dtype)
    if st:
        _ok(st, "purlin_combine_rows")


def purlin_combine_rows_backward(ctx, dy, rows, place, weights, drows, dweights, tokens, top_k,
                                 cols, n_rows, dtype, lddy=0, ldr=0, lddr=0):
    """Gradients of :func:`purlin_combine_rows`: of the rows, and float32 of the weights."""
    st = lib.purlin_combine_rows_backward(ctx.handle, _addr(dy), lddy, _addr(rows), ldr,
                                          _addr(weights), _addr(place), _addr(drows), lddr,
                                          _addr(dweights), tokens, top_k, cols, n_rows, dtype)
    if st:
        _ok(st, "purlin_combine_rows_backward")


def purlin_empty_launch(stream=None):
    _ok(lib.purlin_empty_launch(ctypes.c_void_p(_stream_handle(stream))), "purlin_empty_launch")


def purlin_touch_launch(src_ptr: int, dst_ptr: int, stream=None):
    _ok(lib.purlin_touch_launch(ctypes.c_void_p(src_ptr), ctypes.c_void_p(dst_ptr),
                                ctypes.c_void_p(_stream_handle(stream))), "purlin_touch_launch")


def purlin_check(ctx) -> int:
    """Synchronise and return the device status (raises on non-OK)."""
    _ok(lib.purlin_check(ctx.handle), "purlin_check")
    return PURLIN_OK


def purlin_check_status(ctx) -> int:
    """Like :func:`purlin_check` but returns the status instead of raising."""
    return int(lib.purlin_check(ctx.handle))


def purlin_set_option(ctx, opt: int, value: int):
    _ok(lib.purlin_set_option(ctx.handle, int(opt), int(value)), "purlin_set_option")


def purlin_get_option(ctx, opt: int) -> int:
    v = ctypes.c_int64(0)
    _ok(lib.purlin_get_option(ctx.handle, int(opt), ctypes.byref(v)), "purlin_get_option")
    return v.value


def purlin_last_launch(ctx) -> dict:
    info = purlin_launch_info()
    _ok(lib.purlin_last_launch(ctx.handle, ctypes.byref(info)), "purlin_last_launch")
    return info.as_dict()


def purlin_plan_inspect(coll: int, R: int, src, dst, n: int, counts, dtype: int, op: int,
                        layout, variant: int, ar_mode: int = 0, chunk_bytes: int = 0,
                        cap: int = 8192):
    """Validate + compile one call on the host.  Returns
    ``(status, segments, nchunks, nunits)``; never touches a GPU."""
    ps, _k1 = _ptr_array(src)
    pd, _k2 = _ptr_array(dst)
    if counts is None:
        pc, _k3 = None, None
    else:
        pc, _k3 = _size_array(counts)
    segs = (purlin_segment * cap)()
    nseg = ctypes.c_size_t(0)
    nch = ctypes.c_uint64(0)
    nun = ctypes.c_uint64(0)
    st = lib.purlin_plan_inspect(int(coll), int(R), ps, pd, int(n), pc, int(dtype), int(op),
                                 _layout(layout), int(variant), int(ar_mode), int(chunk_bytes),
                                 segs, cap, ctypes.byref(nseg), ctypes.byref(nch),
                                 ctypes.byref(nun))
    out = [segs[i].as_dict() for i in range(min(nseg.value, cap))] if st == PURLIN_OK else []
    return int(st), out, nch.value, nun.value


# ------------------------------------------------------ device-side API ---

COLL_NAMES = ["all_reduce", "reduce_scatter", "all_gather", "all_to_all", "all_gather_v",
              "reduce_scatter_v", "all_to_all_v"]


def purlin_device_prepare(ctx, coll: int, src, dst, n: int = 0, counts=None, dtype: int = 0,
                          op=None, layout=None, blocks: int = 1,
                          max_workspace_bytes: int = 0) -> purlin_device_coll:
    """Compile a collective for kernels that call it themselves; returns the
    descriptor to pass to them (see include/purlin.h)."""
    dflt_op, dflt_layout = LAYOUTS[COLL_NAMES[int(coll)]]
    op = dflt_op if op is None else op
    layout = dflt_layout if layout is None else layout
    ps, _k1 = _ptr_array(src)
    pd, _k2 = _ptr_array(dst)
    pc, _k3 = (None, None) if counts is None else _size_array(counts)
    d = purlin_device_coll()
    _ok(lib.purlin_device_prepare(ctx.handle, int(coll), ps, pd, int(n), pc, int(dtype), int(op),
                                  _layout(layout), int(blocks), int(max_workspace_bytes),
                                  ctypes.byref(d)), "purlin_device_prepare")
    return d


def purlin_device_check(desc: purlin_device_coll, stream=None) -> int:
    """Wait for the stream, then read and clear the descriptor's error word
    (returns the status; does not raise)."""
    return int(lib.purlin_device_check(ctypes.byref(desc),
                                       ctypes.c_void_p(_stream_handle(stream))))


def purlin_device_release(ctx, desc: purlin_device_coll):
    _ok(lib.purlin_device_release(ctx.handle, ctypes.byref(desc)), "purlin_device_release")


def purlin_packet_channel_create(ctx, capacity_bytes: int, ctas: int) -> purlin_packet_channel:
    ch = purlin_packet_channel()
    _ok(lib.purlin_packet_channel_create(ctx.handle, int(capacity_bytes), int(ctas),
                                         ctypes.byref(ch)), "purlin_packet_channel_create")
    return ch


def purlin_packet_channel_check(ch: purlin_packet_channel, stream=None) -> int:
    """Wait for the stream, then read and clear the channel's error word
    (returns the status; does not raise)."""
    return int(lib.purlin_packet_channel_check(ctypes.byref(ch),
                                               ctypes.c_void_p(_stream_handle(stream))))


def purlin_packet_channel_release(ctx, ch: purlin_packet_channel):
    _ok(lib.purlin_packet_channel_release(ctx.handle, ctypes.byref(ch)),
        "purlin_packet_channel_release")
