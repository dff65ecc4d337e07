"""Tensor-level calls in the shape of the "Purlin" project README's Python API
("Using Purlin", Python: ``initialize``, ``all_reduce(x, out, handle,
stream)``, ``finalize``; "Deterministic Reduction": ``reduction_mode``).

One GPU holds all R ranks here, so ``x`` and ``out`` are sequences of R
tensors (rank r's input and output), not one tensor per process.  Sizes and
dtypes are read from the tensors; everything else is the C ABI through the
ctypes binding, so this module only marshals arguments.

    h = initialize(8, stream=torch.cuda.current_stream())
    all_reduce(xs, outs, h)                  # every outs[r] = sum over s of xs[s]
    finalize(h)

The layer operators that follow the collectives take one rank's tensors:
``rms_norm``, ``grouped_matmul`` and their gradients.  They run on the handle's
stream (or on ``stream``), and so do the allocation and the zeroing of results
that are not passed in.  Where that is not torch's current stream, order the two
as for any stream's results: the inputs before the call, the results after it.
"""
from __future__ import annotations

import enum
from typing import Sequence

from . import (PURLIN_BF16, PURLIN_E4M3, PURLIN_F32, PURLIN_WEIGHTS_KN, PURLIN_WEIGHTS_NK, Context,
               _stream_handle, purlin_all_gather, purlin_all_gather_v, purlin_all_reduce,
               purlin_all_to_all, purlin_all_to_all_v, purlin_check, purlin_finalize,
               purlin_grouped_matmul, purlin_grouped_matmul_weight_grad, purlin_init,
               purlin_reduce_scatter, purlin_reduce_scatter_v, purlin_rms_norm,
               purlin_rms_norm_backward, purlin_set_stream)


class ReductionMode(enum.Enum):
    """The README's reduction modes.  Only the deterministic one exists on one
    GPU (no NVLink SHARP): sums are taken in rank order in binary32 and
    rounded once."""
    DETERMINISTIC = "deterministic"
    NON_DETERMINISTIC = "non_deterministic"


def _dtype_of(tensors: Sequence) -> int:
    import torch

    kinds = {t.dtype for t in tensors}
    if len(kinds) != 1:
        raise TypeError(f"all rank tensors must share one dtype, got {sorted(map(str, kinds))}")
    dt = kinds.pop()
    if dt == torch.float32:
        return PURLIN_F32
    if dt in (torch.bfloat16, torch.int16):   # bf16, or its raw bits
        return PURLIN_BF16
    raise TypeError(f"unsupported dtype {dt}: float32, bfloat16 (or its int16 bits)")


def _check(xs: Sequence, outs: Sequence, handle: Context):
    if len(xs) != handle.R or len(outs) != handle.R:
        raise ValueError(f"expected {handle.R} input and output tensors, got {len(xs)} and "
                         f"{len(outs)}")
    for t in list(xs) + list(outs):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("rank tensors must be contiguous CUDA tensors")
    d = _dtype_of(list(xs) + list(outs))
    return d


def _uniform_numel(xs: Sequence) -> int:
    n = {int(t.numel()) for t in xs}
    if len(n) != 1:
        raise ValueError("every rank's input must hold the same number of elements")
    return n.pop()


def _on(handle: Context, stream):
    """Switch the handle to `stream` if it names another stream (the switch
    waits for the previous stream, so it is skipped when nothing changes)."""
    if stream is None:
        return
    if _stream_handle(stream) != handle.stream_handle:
        purlin_set_stream(handle, stream)


def initialize(R: int, stream=None) -> Context:
    """A context for R rank buffers on the current CUDA device."""
    return purlin_init(R, stream)


def finalize(handle: Context, stream=None):
    _on(handle, stream)
    purlin_finalize(handle)


def check(handle: Context) -> None:
    """Wait for the handle's stream and raise if a device-side wait expired."""
    purlin_check(handle)


def all_reduce(xs, outs, handle, stream=None, reduction_mode=ReductionMode.DETERMINISTIC):
    if reduction_mode is not ReductionMode.DETERMINISTIC:
        raise NotImplementedError("only the deterministic reduction exists on one GPU")
    d = _check(xs, outs, handle)
    n = _uniform_numel(xs)
    if any(int(o.numel()) != n for o in outs):
        raise ValueError("AllReduce outputs hold as many elements as the inputs")
    _on(handle, stream)
    purlin_all_reduce(handle, xs, outs, n, d)


def reduce_scatter(xs, outs, handle, stream=None, reduction_mode=ReductionMode.DETERMINISTIC):
    if reduction_mode is not ReductionMode.DETERMINISTIC:
        raise NotImplementedError("only the deterministic reduction exists on one GPU")
    d = _check(xs, outs, handle)
    n = _uniform_numel(xs)
    if n % handle.R or any(int(o.numel()) != n // handle.R for o in outs):
        raise ValueError("ReduceScatter: inputs of n elements (n divisible by R), outputs of n/R")
    _on(handle, stream)
    purlin_reduce_scatter(handle, xs, outs, n, d)


def all_gather(xs, outs, handle, stream=None):
    d = _check(xs, outs, handle)
    n = _uniform_numel(xs)
    if any(int(o.numel()) != handle.R * n for o in outs):
        raise ValueError("AllGather outputs hold R times the input elements")
    _on(handle, stream)
    purlin_all_gather(handle, xs, outs, n, d)


def all_to_all(xs, outs, handle, stream=None):
    d = _check(xs, outs, handle)
    n = _uniform_numel(xs)
    if n % handle.R or any(int(o.numel()) != n for o in outs):
        raise ValueError("AllToAll: inputs and outputs of n elements, n divisible by R")
    _on(handle, stream)
    purlin_all_to_all(handle, xs, outs, n, d)


def all_gather_v(xs, outs, handle, stream=None):
    """Rank r contributes xs[r] (any length); every output holds all of them."""
    d = _check(xs, outs, handle)
    counts = [int(t.numel()) for t in xs]
    if any(int(o.numel()) != sum(counts) for o in outs):
        raise ValueError("AllGatherV outputs hold the sum of the input lengths")
    _on(handle, stream)
    purlin_all_gather_v(handle, xs, outs, counts, d)


def reduce_scatter_v(xs, outs, handle, stream=None, reduction_mode=ReductionMode.DETERMINISTIC):
    """outs[r] receives the rank-order sum of block r; block lengths are the
    output lengths, and every input holds their total."""
    if reduction_mode is not ReductionMode.DETERMINISTIC:
        raise NotImplementedError("only the deterministic reduction exists on one GPU")
    d = _check(xs, outs, handle)
    counts = [int(o.numel()) for o in outs]
    if any(int(t.numel()) != sum(counts) for t in xs):
        raise ValueError("ReduceScatterV inputs hold the sum of the output lengths")
    _on(handle, stream)
    purlin_reduce_scatter_v(handle, xs, outs, counts, d)


def all_to_all_v(xs, outs, counts, handle, stream=None):
    """counts: R x R element counts (row = source, column = destination), as a
    nested sequence or a flat one of R*R entries."""
    d = _check(xs, outs, handle)
    R = handle.R
    flat = [int(c) for row in counts for c in (row if hasattr(row, "__iter__") else [row])]
    if len(flat) != R * R:
        raise ValueError(f"AllToAllV needs {R * R} counts")
    for s in range(R):
        if int(xs[s].numel()) < sum(flat[s * R:(s + 1) * R]):
            raise ValueError(f"input {s} is shorter than its row of counts")
    for dd in range(R):
        if int(outs[dd].numel()) < sum(flat[s * R + dd] for s in range(R)):
            raise ValueError(f"output {dd} is shorter than its column of counts")
    _on(handle, stream)
    purlin_all_to_all_v(handle, xs, outs, flat, d)


# ------------------------------------------------------- layer operators ---

def _new(handle, stream, device, shape, dtype, zero=False):
    """A result for a call to write, of the stream that the call launches on.  Memory
    of another stream may still be in use there, and a fill there could land after
    the kernel."""
    import torch

    make = torch.zeros if zero else torch.empty
    current = torch.cuda.current_stream(device)
    h = handle.stream_handle if stream is None else _stream_handle(stream)
    if h == current.cuda_stream:
        return make(shape, device=device, dtype=dtype)
    launch = torch.cuda.ExternalStream(h, device) if h else torch.cuda.default_stream(device)
    with torch.cuda.stream(launch):
        t = make(shape, device=device, dtype=dtype)
    t.record_stream(current)   # the caller's: not to be reused while it reads
    return t


def _pitch(t, rows, stride):
    """Row stride to pass on for `rows` rows.  A single row's may be anything; it is
    rounded up to 16 bytes, which the products ask of a matrix's rows."""
    if rows > 1:
        return stride
    per = 16 // t.element_size()
    return (t.shape[-1] + per - 1) // per * per


def _rows(name, t, dtypes, cols=None):
    """(rows, cols, row stride) of a CUDA matrix whose rows are contiguous."""
    if not t.is_cuda or t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a CUDA matrix with contiguous rows")
    # (an expanded view's stride of 0 would read as "contiguous" below)
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}: its rows overlap (strides {t.stride()}); expanded views need a copy")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if cols is not None and t.shape[1] != cols:
        raise ValueError(f"{name} has {t.shape[1]} columns, expected {cols}")
    return t.shape[0], t.shape[1], _pitch(t, t.shape[0], t.stride(0))


def _vector(name, t, n, dtype):
    if not t.is_cuda or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{name} must hold {n} contiguous values on the GPU")
    if t.dtype != dtype:
        raise TypeError(f"{name}: {t.dtype}, expected {dtype}")


def _same_rows(name, t, like):
    if t.shape != like.shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(like.shape)}")
    return _rows(name, t, (like.dtype,))[2]


def rms_norm(x, weight, handle, residual=None, out=None, total=None, scales=None, eps=1e-5,
             quantize=False, stream=None):
    """Norm of the rows of ``x`` (+ ``residual``) times ``weight``.  Returns
    ``out``, or ``(out, scales)`` with ``quantize`` (e4m3 rows, a float32 scale
    a row); ``total``, if given, receives ``x + residual``.  Outputs are
    allocated unless passed in."""
    import torch

    rows, hidden, ldx = _rows("x", x, (torch.float32, torch.bfloat16))
    d = PURLIN_F32 if x.dtype == torch.float32 else PURLIN_BF16
    _vector("weight", weight, hidden, x.dtype)
    ldr = _same_rows("residual", residual, x) if residual is not None else 0
    ldt = _same_rows("total", total, x) if total is not None else 0
    kind = torch.float8_e4m3fn if quantize else x.dtype
    if out is None:
        out = _new(handle, stream, x.device, (rows, hidden), kind)
    if out.shape != x.shape:
        raise ValueError("out has the shape of x")
    ldy = _rows("out", out, (kind,))[2]
    if quantize and scales is None:
        scales = _new(handle, stream, x.device, (rows,), torch.float32)
    if scales is not None:
        if not quantize:
            raise ValueError("scales belong to a quantized output")
        _vector("scales", scales, rows, torch.float32)
    _on(handle, stream)
    purlin_rms_norm(handle, x, weight, out, rows, hidden, eps, d, PURLIN_E4M3 if quantize else d,
                    residual=residual, total=total, scales=scales, ldx=ldx, ldr=ldr, ldy=ldy,
                    ldt=ldt)
    return (out, scales) if quantize else out


def rms_norm_backward(dy, total, weight, handle, dtotal=None, dx=None, dweight=None, eps=1e-5,
                      stream=None):
    """Gradients of :func:`rms_norm` at ``total`` (``x + residual``): returns
    ``(dx, dweight)``, dx that of x and of the residual, dweight in float32.
    ``dtotal``: the gradient that reaches ``total`` from elsewhere."""
    import torch

    rows, hidden, ldt = _rows("total", total, (torch.float32, torch.bfloat16))
    d = PURLIN_F32 if total.dtype == torch.float32 else PURLIN_BF16
    _vector("weight", weight, hidden, total.dtype)
    lddy = _same_rows("dy", dy, total)
    lddt = _same_rows("dtotal", dtotal, total) if dtotal is not None else 0
    dx = _new(handle, stream, dy.device, (rows, hidden), dy.dtype) if dx is None else dx
    lddx = _same_rows("dx", dx, total)
    if dweight is None:
        dweight = _new(handle, stream, dy.device, (hidden,), torch.float32)
    _vector("dweight", dweight, hidden, torch.float32)
    _on(handle, stream)
    purlin_rms_norm_backward(handle, dy, total, weight, dx, dweight, rows, hidden, eps, d,
                             dtotal=dtotal, lddy=lddy, ldt=ldt, lddt=lddt, lddx=lddx)
    return dx, dweight


def _stack(name, t, dtypes):
    """(groups, rows, cols, row stride) of matrices that lie one after another."""
    if not t.is_cuda or t.dim() != 3 or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"{name} must be CUDA matrices with contiguous rows")
    row = t.stride(1) if t.shape[1] > 1 else t.stride(0)   # one row a matrix: from group to group
    if t.shape[0] > 1 and t.stride(0) != t.shape[1] * row:
        raise ValueError(f"{name} must be CUDA matrices with contiguous rows, one after another")
    if t.shape[0] * t.shape[1] > 1 and row < t.shape[2]:
        raise ValueError(f"{name}: its rows overlap (strides {t.stride()}); expanded views need a copy")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    return (*t.shape, _pitch(t, t.shape[0] * t.shape[1], row))


def _groups(begin, count, groups):
    import torch

    _vector("begin", begin, groups, torch.int64)
    _vector("count", count, groups, torch.int64)


def grouped_matmul(x, w, begin, count, handle, out=None, x_scales=None, w_scales=None,
                   transposed=False, stream=None):
    """Rows ``begin[g]`` to ``begin[g] + count[g]`` of ``x`` times the transpose
    of ``w[g]`` (``w``: groups x n x k), or times ``w[g]`` itself (groups x k x
    n) with ``transposed``, which with the output's gradient in place of ``x``
    is the gradient of x.  bf16, or e4m3 with a scale a row of x and a channel
    of w.  Rows of ``out`` in no group are left as they are (zero where it is
    allocated here)."""
    import torch

    kinds = (torch.bfloat16, torch.float8_e4m3fn)
    groups, wr, wc, ldw = _stack("w", w, kinds)
    n, k = (wc, wr) if transposed else (wr, wc)
    rows, _, ldx = _rows("x", x, (w.dtype,), k)
    _groups(begin, count, groups)
    if out is None:
        out = _new(handle, stream, x.device, (rows, n), torch.bfloat16, zero=True)
    out_rows, _, ldy = _rows("out", out, (torch.bfloat16,), n)
    if out_rows != rows:
        raise ValueError("out holds as many rows as x")
    e4m3 = w.dtype == torch.float8_e4m3fn
    if (x_scales is not None) != e4m3 or (w_scales is not None) != e4m3:
        raise ValueError("e4m3 operands, and only they, come with x_scales and w_scales")
    if e4m3:
        _vector("x_scales", x_scales, rows, torch.float32)
        _vector("w_scales", w_scales, groups * n, torch.float32)
    _on(handle, stream)
    purlin_grouped_matmul(handle, x, w, out, begin, count, groups, rows, n, k,
                          PURLIN_E4M3 if e4m3 else PURLIN_BF16,
                          PURLIN_WEIGHTS_KN if transposed else PURLIN_WEIGHTS_NK,
                          x_scales=x_scales, w_scales=w_scales, ldx=ldx, ldw=ldw, ldy=ldy)
    return out


def grouped_matmul_weight_grad(dy, x, begin, count, handle, out=None, stream=None):
    """groups x n x k gradients of the weights of :func:`grouped_matmul`."""
    import torch

    rows, n, lddy = _rows("dy", dy, (torch.bfloat16,))
    x_rows, k, ldx = _rows("x", x, (torch.bfloat16,))
    if x_rows != rows:
        raise ValueError("dy and x hold the same rows")
    groups = int(count.numel())
    _groups(begin, count, groups)
    if out is None:
        out = _new(handle, stream, x.device, (groups, n, k), torch.bfloat16)
    og, on, ok, lddw = _stack("out", out, (torch.bfloat16,))
    if (og, on, ok) != (groups, n, k):
        raise ValueError(f"out has shape {(og, on, ok)}, expected {(groups, n, k)}")
    _on(handle, stream)
    purlin_grouped_matmul_weight_grad(handle, dy, x, out, begin, count, groups, rows, n, k,
                                      PURLIN_BF16, lddy=lddy, ldx=ldx, lddw=lddw)
    return out
