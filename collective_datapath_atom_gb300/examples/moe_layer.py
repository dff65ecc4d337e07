"""A mixture-of-experts layer around the collectives, on R rank buffers of one
GPU, with nothing of a token's path on the host:

    ReduceScatter of the attention's partial sums
    -> residual's addition and RMS norm, to 8 bits with a scale a token
    -> AllToAllV of the rows and of their scales to the tokens' experts
    -> each expert's product, grouped, where the dispatch left the rows
    -> AllToAllV back.

Rank r holds expert r.  The routing stays on the device: the count matrix goes
to the collectives as device counts, its column sums to the grouped product.

    python -m collective_datapath_atom_gb300.examples.moe_layer
"""
from __future__ import annotations

import collective_datapath_atom_gb300 as purlin


def moe_layer(ctx, partials, residual, norm_weight, experts, expert_scales, destination,
              eps=1e-5, capacity=None):
    """``partials``: R tensors of T x H bf16, the ranks' partial sums; rank r
    owns tokens r T / R and on.  ``residual``: T x H.  ``experts``: R x N x H
    e4m3 with ``expert_scales`` R x N.  ``destination``: int64 of T, each
    token's expert.  ``capacity``: tokens an expert can take (default: all T).
    T / R and the capacity are multiples of 4, H and N of 16; the context's
    stream is torch's current one.

    Returns a dict: ``y`` (T x N bf16), ``total`` (T x H, the residual stream),
    and the 8-bit rows ``q`` with their ``scales``.
    """
    import torch

    R = ctx.R
    T, H = residual.shape
    N = experts.shape[1]
    rows = T // R
    cap = T if capacity is None else capacity
    dev = residual.device
    bf16, e4m3 = torch.bfloat16, torch.float8_e4m3fn

    def ranks(t, n):
        return [t[r * n:(r + 1) * n] for r in range(R)]

    # the ranks' shards lie one after another: one norm for all of them
    shard = torch.empty(T, H, device=dev, dtype=bf16)
    purlin.purlin_reduce_scatter(ctx, partials, ranks(shard, rows), T * H, purlin.PURLIN_BF16)
    q = torch.empty(T, H, device=dev, dtype=e4m3)
    total = torch.empty_like(shard)
    scales = torch.empty(T, device=dev)
    purlin.purlin_rms_norm(ctx, shard, norm_weight, q, T, H, eps, purlin.PURLIN_BF16,
                           purlin.PURLIN_E4M3, residual=residual, total=total, scales=scales)

    # each rank's tokens in the order of their experts, and the count matrix
    dest = destination.view(R, rows)
    start = torch.arange(R, device=dev)[:, None] * rows
    order = (dest.argsort(dim=1, stable=True) + start).reshape(-1)
    tokens = torch.zeros(R, R, device=dev, dtype=torch.int64)
    tokens.scatter_add_(1, dest, torch.ones_like(dest))

    # 8-bit rows travel as pairs
    sent, sent_scales = q.view(torch.uint8)[order], scales[order]
    got = torch.empty(R, cap, H, device=dev, dtype=torch.uint8)
    got_scales = torch.empty(R, cap, device=dev)
    purlin.purlin_all_to_all_v_device_counts(
        ctx, ranks(sent, rows), list(got), tokens * (H // 2), rows * H // 2, cap * H // 2,
        purlin.PURLIN_BF16)
    purlin.purlin_all_to_all_v_device_counts(
        ctx, ranks(sent_scales, rows), list(got_scales), tokens, rows, cap, purlin.PURLIN_F32)

    begin = torch.arange(R, device=dev) * cap
    out = torch.empty(R, cap, N, device=dev, dtype=bf16)
    purlin.purlin_grouped_matmul(ctx, got, experts, out, begin, tokens.sum(0), R, R * cap, N, H,
                                 purlin.PURLIN_E4M3, x_scales=got_scales, w_scales=expert_scales)

    back = torch.empty(T, N, device=dev, dtype=bf16)
    purlin.purlin_all_to_all_v_device_counts(
        ctx, list(out), ranks(back, rows), tokens.t().contiguous() * N, cap * N, rows * N,
        purlin.PURLIN_BF16)
    y = torch.empty_like(back)
    y[order] = back
    return {"y": y, "total": total, "q": q, "scales": scales}


def main(R=8, tokens=2048, hidden=7168, width=2048):
    import torch

    g = torch.Generator(device="cuda").manual_seed(3)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    ctx = purlin.purlin_init(R, torch.cuda.current_stream())
    try:
        partials = [randn(tokens, hidden).bfloat16() for _ in range(R)]
        residual = randn(tokens, hidden).bfloat16()
        experts = randn(R, width, hidden).to(torch.float8_e4m3fn)
        expert_scales = torch.full((R, width), hidden ** -0.5, device="cuda")
        share = torch.arange(1, R + 1, device="cuda").float() ** -1.2
        destination = torch.multinomial(share, tokens, replacement=True, generator=g)
        args = (ctx, partials, residual, torch.ones(hidden, device="cuda").bfloat16(), experts,
                expert_scales, destination)
        moe_layer(*args)
        purlin.purlin_check(ctx)
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        r = moe_layer(*args)
        b.record()
        purlin.purlin_check(ctx)
        print(f"{R} ranks, {tokens} tokens x {hidden}, experts {width}: "
              f"{a.elapsed_time(b) * 1e3:.0f} us, y {tuple(r['y'].shape)}, "
              f"rms {float(r['y'].float().square().mean().sqrt()):.3f}")
    finally:
        ctx.close()


if __name__ == "__main__":
    main()
