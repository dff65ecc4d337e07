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
``rms_norm``, ``block_norm``, ``route``, ``expert_order``, ``dispatch_rows``,
``combine_rows``, ``grouped_matmul`` and their gradients.  They run on the handle's
stream (or on ``stream``), and so do the allocation and the zeroing of results
that are not passed in.  Where that is not torch's current stream, order the two
as for any stream's results: the inputs before the call, the results after it.
"""
from __future__ import annotations

import enum
from typing import Sequence

from . import (PURLIN_BF16, PURLIN_E4M3, PURLIN_F32, PURLIN_GATE_COLUMNS, PURLIN_GATE_ROWS,
               PURLIN_SIGMOID, PURLIN_SOFTMAX, PURLIN_WEIGHTS_KN, PURLIN_WEIGHTS_NK, Context,
               _stream_handle, purlin_all_gather, purlin_all_gather_v, purlin_all_reduce,
               purlin_all_to_all, purlin_all_to_all_v, purlin_block_norm,
               purlin_block_norm_backward, purlin_check, purlin_combine_rows,
               purlin_combine_rows_backward, purlin_dispatch_rows, purlin_expert_order,
               purlin_finalize, purlin_grouped_matmul, purlin_grouped_matmul_weight_grad,
               purlin_init, purlin_reduce_scatter, purlin_reduce_scatter_v, purlin_rms_norm,
               purlin_rms_norm_backward, purlin_route, purlin_route_backward, purlin_router,
               purlin_set_stream)


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


def _gate(gate, like):
    """(layout, row stride) of a gate: a value a column, or one an element."""
    if gate is None:
        return PURLIN_GATE_COLUMNS, 0
    if gate.dim() == 1:
        _vector("gate", gate, like.shape[1], like.dtype)
        return PURLIN_GATE_COLUMNS, 0
    return PURLIN_GATE_ROWS, _same_rows("gate", gate, like)


def block_norm(x, weight, handle, residual=None, post_weight=None, gate=None, residual_scale=1.0,
               block_scale=1.0, out=None, total=None, scales=None, eps=1e-5, quantize=False,
               stream=None):
    """Norm of ``t = residual_scale * residual + block_scale * gate * u`` times
    ``weight``, where ``u`` is the block's output ``x``, or its norm times
    ``post_weight``.  ``gate``: a value a column, or as many as ``x`` has.  Returns
    ``(out, total)``, or ``(out, total, scales)`` with ``quantize`` (e4m3 rows, a
    float32 scale a row); ``total`` is ``t``.  ``weight`` None: only ``total``, and
    ``out`` is None.  Outputs are allocated unless passed in."""
    import torch

    rows, hidden, ldx = _rows("x", x, (torch.float32, torch.bfloat16))
    d = PURLIN_F32 if x.dtype == torch.float32 else PURLIN_BF16
    for name, v in (("weight", weight), ("post_weight", post_weight)):
        if v is not None:
            _vector(name, v, hidden, x.dtype)
    layout, ldg = _gate(gate, x)
    ldr = _same_rows("residual", residual, x) if residual is not None else 0
    if weight is None and (quantize or out is not None):
        raise ValueError("without a weight there is no norm to write")
    total = _new(handle, stream, x.device, (rows, hidden), x.dtype) if total is None else total
    ldt = _same_rows("total", total, x)
    kind = torch.float8_e4m3fn if quantize else x.dtype
    ldy = 0
    if weight is not None:
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
    purlin_block_norm(handle, x, weight, out, rows, hidden, eps, d, PURLIN_E4M3 if quantize else d,
                      residual=residual, post_weight=post_weight, gate=gate, gate_layout=layout,
                      residual_scale=residual_scale, block_scale=block_scale, total=total,
                      scales=scales, ldx=ldx, ldg=ldg, ldr=ldr, ldy=ldy, ldt=ldt)
    return (out, total, scales) if quantize else (out, total)


def block_norm_backward(dy, x, total, weight, handle, dtotal=None, post_weight=None, gate=None,
                        residual_scale=1.0, block_scale=1.0, eps=1e-5, stream=None):
    """Gradients of :func:`block_norm` at ``x`` and ``total``: a dict of ``dx``,
    ``dresidual``, and those of ``dweight``, ``dpost_weight`` and ``dgate`` whose
    inputs are given (vectors in float32).  ``dtotal``: the gradient that reaches
    ``total`` from elsewhere.  ``dy``, ``total`` and ``weight`` None: the forward
    pass wrote ``total`` alone."""
    import torch

    rows, hidden, ldx = _rows("x", x, (torch.float32, torch.bfloat16))
    d = PURLIN_F32 if x.dtype == torch.float32 else PURLIN_BF16
    for name, v in (("weight", weight), ("post_weight", post_weight)):
        if v is not None:
            _vector(name, v, hidden, x.dtype)
    layout, ldg = _gate(gate, x)
    ld = {name: _same_rows(name, t, x) if t is not None else 0
          for name, t in (("dy", dy), ("total", total), ("dtotal", dtotal))}

    def new(shape, dtype):
        return _new(handle, stream, x.device, shape, dtype)

    got = {"dx": new((rows, hidden), x.dtype), "dresidual": new((rows, hidden), x.dtype)}
    if weight is not None:
        got["dweight"] = new((hidden,), torch.float32)
    if post_weight is not None:
        got["dpost_weight"] = new((hidden,), torch.float32)
    if gate is not None:
        got["dgate"] = new((rows, hidden), x.dtype) if layout == PURLIN_GATE_ROWS else \
            new((hidden,), torch.float32)
    _on(handle, stream)
    purlin_block_norm_backward(handle, dy, x, total, weight, got["dx"], got.get("dweight"), rows,
                               hidden, eps, d, dtotal=dtotal, post_weight=post_weight, gate=gate,
                               gate_layout=layout, residual_scale=residual_scale,
                               block_scale=block_scale, dresidual=got["dresidual"],
                               dpost_weight=got.get("dpost_weight"), dgate=got.get("dgate"),
                               lddy=ld["dy"], lddt=ld["dtotal"], ldx=ldx, ldt=ld["total"], ldg=ldg)
    return got


def router(experts, top_k, scores="softmax", groups=1, top_groups=1, group_top=1,
           renormalise=False, scale=1.0):
    """How :func:`route` chooses: see ``purlin_router`` in include/purlin.h."""
    kinds = {"softmax": PURLIN_SOFTMAX, "sigmoid": PURLIN_SIGMOID}
    if scores not in kinds:
        raise ValueError(f"scores are 'softmax' or 'sigmoid', got {scores!r}")
    if scale == 0:
        raise ValueError("a scale of 0 would read as 1")
    return purlin_router(experts=experts, top_k=top_k, scores=kinds[scores], groups=groups,
                         top_groups=top_groups, group_top=group_top, renormalise=int(renormalise),
                         scale=scale)


def route(logits, config, handle, bias=None, stream=None):
    """Each token's experts (int32, falling) and their weights (float32), both
    tokens x top_k, from its row of ``logits``; ``config`` is a :func:`router`.
    Returns ``(weights, experts)``; an expert of -1 is none."""
    import torch

    tokens, _, ld = _rows("logits", logits, (torch.float32, torch.bfloat16), config.experts)
    d = PURLIN_F32 if logits.dtype == torch.float32 else PURLIN_BF16
    if bias is not None:
        _vector("bias", bias, config.experts, torch.float32)
    weights = _new(handle, stream, logits.device, (tokens, config.top_k), torch.float32)
    chosen = _new(handle, stream, logits.device, (tokens, config.top_k), torch.int32)
    _on(handle, stream)
    purlin_route(handle, logits, weights, chosen, tokens, config, d, bias=bias, ld=ld)
    return weights, chosen


def _slots(name, t, tokens, top_k, dtype):
    if not t.is_cuda or not t.is_contiguous() or tuple(t.shape) != (tokens, top_k):
        raise ValueError(f"{name} must be {tokens} x {top_k} contiguous values on the GPU")
    if t.dtype != dtype:
        raise TypeError(f"{name}: {t.dtype}, expected {dtype}")


def route_backward(dweights, logits, experts, config, handle, stream=None):
    """Gradient of :func:`route`'s weights with respect to ``logits``."""
    import torch

    tokens, cols, ld = _rows("logits", logits, (torch.float32, torch.bfloat16), config.experts)
    d = PURLIN_F32 if logits.dtype == torch.float32 else PURLIN_BF16
    _slots("dweights", dweights, tokens, config.top_k, torch.float32)
    _slots("experts", experts, tokens, config.top_k, torch.int32)
    out = _new(handle, stream, logits.device, (tokens, cols), logits.dtype)
    _on(handle, stream)
    purlin_route_backward(handle, dweights, logits, experts, out, tokens, config, d, ld=ld)
    return out


def expert_order(experts, groups, handle, capacity=0, stream=None):
    """The row of each slot of ``experts`` (int32, as :func:`route` gives them) in
    the order of the experts, packed or in buffers of ``capacity`` rows (-1 past
    it).  Returns ``(place, begin, count)``: int32 in the shape of ``experts``, and
    int64 first rows and counts as :func:`grouped_matmul` takes them."""
    import torch

    if not experts.is_cuda or not experts.is_contiguous():
        raise ValueError("experts must be contiguous values on the GPU")
    if experts.dtype != torch.int32:
        raise TypeError(f"experts: {experts.dtype}, expected {torch.int32}")
    place = _new(handle, stream, experts.device, tuple(experts.shape), torch.int32)
    begin = _new(handle, stream, experts.device, (groups,), torch.int64)
    count = _new(handle, stream, experts.device, (groups,), torch.int64)
    _on(handle, stream)
    purlin_expert_order(handle, experts, place, begin, count, int(experts.numel()), groups,
                        capacity)
    return place, begin, count


def dispatch_rows(x, place, handle, out_rows=None, scales=None, out=None, out_scales=None,
                  stream=None):
    """``out[place[t, j]] = x[t]`` (and its scale) for every token and choice.
    ``out_rows``: rows of ``out``, as many as slots unless given.  Rows that no place
    names are left as they are (zero where ``out`` is allocated here).  Returns
    ``out``, or ``(out, out_scales)`` with ``scales``."""
    import torch

    kinds = {torch.float32: PURLIN_F32, torch.bfloat16: PURLIN_BF16,
             torch.float8_e4m3fn: PURLIN_E4M3}
    tokens, cols, ldx = _rows("x", x, tuple(kinds))
    top_k = place.shape[-1]
    _slots("place", place, tokens, top_k, torch.int32)
    if out is None:
        rows = tokens * top_k if out_rows is None else out_rows
        out = _new(handle, stream, x.device, (rows, cols), torch.uint8 if x.dtype ==
                   torch.float8_e4m3fn else x.dtype, zero=True)
        out = out.view(x.dtype)
    rows, _, ldo = _rows("out", out, (x.dtype,), cols)
    if out_rows is not None and rows != out_rows:
        raise ValueError(f"out has {rows} rows, expected {out_rows}")
    if scales is not None:
        _vector("scales", scales, tokens, torch.float32)
        if out_scales is None:
            out_scales = _new(handle, stream, x.device, (rows,), torch.float32, zero=True)
        _vector("out_scales", out_scales, rows, torch.float32)
    elif out_scales is not None:
        raise ValueError("out_scales are copies of scales")
    _on(handle, stream)
    purlin_dispatch_rows(handle, x, place, out, tokens, top_k, cols, rows, kinds[x.dtype],
                         scales=scales, out_scales=out_scales, ldx=ldx, ldo=ldo)
    return out if scales is None else (out, out_scales)


def combine_rows(rows, place, handle, weights=None, shared=None, out=None, stream=None):
    """For each token the sum of ``weights[t, j] * rows[place[t, j]]`` (on
    ``shared[t]``, if given); with ``weights`` None the gradient of
    :func:`dispatch_rows`' ``x`` from that of its output."""
    import torch

    n_rows, cols, ldr = _rows("rows", rows, (torch.float32, torch.bfloat16))
    d = PURLIN_F32 if rows.dtype == torch.float32 else PURLIN_BF16
    tokens, top_k = place.shape
    _slots("place", place, tokens, top_k, torch.int32)
    if weights is not None:
        _slots("weights", weights, tokens, top_k, torch.float32)
    out = _new(handle, stream, rows.device, (tokens, cols), rows.dtype) if out is None else out
    out_rows, _, ldy = _rows("out", out, (rows.dtype,), cols)
    if out_rows != tokens:
        raise ValueError(f"out has {out_rows} rows, expected {tokens}")
    lds = _same_rows("shared", shared, out) if shared is not None else 0
    _on(handle, stream)
    purlin_combine_rows(handle, rows, place, out, tokens, top_k, cols, n_rows, d, weights=weights,
                        shared=shared, ldr=ldr, lds=lds, ldy=ldy)
    return out


def combine_rows_backward(dy, rows, place, weights, handle, stream=None):
    """Gradients of :func:`combine_rows`: ``(drows, dweights)``.  Rows of drows that
    no place names are zero."""
    import torch

    n_rows, cols, ldr = _rows("rows", rows, (torch.float32, torch.bfloat16))
    d = PURLIN_F32 if rows.dtype == torch.float32 else PURLIN_BF16
    tokens, _, lddy = _rows("dy", dy, (rows.dtype,), cols)
    top_k = place.shape[-1]
    _slots("place", place, tokens, top_k, torch.int32)
    _slots("weights", weights, tokens, top_k, torch.float32)
    drows = _new(handle, stream, rows.device, (n_rows, cols), rows.dtype, zero=True)
    dweights = _new(handle, stream, rows.device, (tokens, top_k), torch.float32)
    _on(handle, stream)
    purlin_combine_rows_backward(handle, dy, rows, place, weights, drows, dweights, tokens, top_k,
                                 cols, n_rows, d, lddy=lddy, ldr=ldr)
    return drows, dweights


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
