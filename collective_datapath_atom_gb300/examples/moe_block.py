"""A mixture-of-experts block between two residual additions, on R rank buffers of
one GPU, every token to its top_k experts and with nothing of its path on the host:

    ReduceScatter of the attention's partial sums
    -> the norm after the attention, its gate, the residual, the norm before the experts
    -> router: a product, sigmoid scores with a balance bias, the top_k, their weights
    -> each rank's slots in the order of their experts, the rows copied there
    -> AllToAllV of the rows with device counts
    -> each expert's two products, grouped, where the dispatch left the rows
    -> AllToAllV back, and each token's weighted sum
    -> the norm after the experts, their gate, the residual, the next block's norm.

Rank r holds expert r.

    python -m collective_datapath_atom_gb300.examples.moe_block
"""
from __future__ import annotations

import collective_datapath_atom_gb300 as purlin


def moe_block(ctx, partials, residual, norms, router_weight, router_bias, up, down, top_k=2,
              residual_scale=1.0, block_scale=1.0, eps=1e-5):
    """``partials``: R tensors of T x H bf16, the ranks' partial sums; rank r owns
    tokens r T / R and on.  ``residual``: T x H.  ``norms``: a pair of dicts, for the
    attention and for the experts, of H-vectors ``post`` (the norm after the block),
    ``gate`` and ``weight`` (the norm before the next one).  ``router_weight``: R x H
    bf16, ``router_bias``: R float32 (it decides the choice alone).  ``up``: R x N x H,
    ``down``: R x H x N bf16.  H and N are multiples of 8, T / R of 4; the context's
    stream is torch's current one.

    Returns a dict: ``y`` (T x H, the next block's input), ``total`` (the residual
    stream), ``load`` (tokens of each expert), and of the middle ``hidden`` (the
    experts' input), ``experts`` and ``weights`` (T x top_k).
    """
    import torch

    R = ctx.R
    T, H = residual.shape
    N = up.shape[1]
    rows, slots = T // R, T // R * top_k
    cap = T * top_k               # every slot may go to one expert
    dev, bf16 = residual.device, torch.bfloat16
    code = purlin.PURLIN_BF16

    def new(*shape, dtype=bf16):
        return torch.empty(*shape, device=dev, dtype=dtype)

    def ranks(t, n):
        return [t[r * n:(r + 1) * n] for r in range(R)]

    def norm(x, before, n):
        y, total = new(T, H), new(T, H)
        purlin.purlin_block_norm(ctx, x, n["weight"], y, T, H, eps, code, residual=before,
                                 post_weight=n["post"], gate=n["gate"], total=total,
                                 residual_scale=residual_scale, block_scale=block_scale)
        return y, total

    # the ranks' shards lie one after another: one norm, one router for all of them
    shard = new(T, H)
    purlin.purlin_reduce_scatter(ctx, partials, ranks(shard, rows), T * H, code)
    hidden, total = norm(shard, residual, norms[0])

    pitch = (R + 7) // 8 * 8
    logits = new(T, pitch)
    one = torch.tensor([0, T], device=dev)
    purlin.purlin_grouped_matmul(ctx, hidden, router_weight, logits, one[:1], one[1:], 1, T, R, H,
                                 code, ldy=pitch)
    config = purlin.purlin_router(experts=R, top_k=top_k, scores=purlin.PURLIN_SIGMOID,
                                  renormalise=1)
    weights, experts = new(T, top_k, dtype=torch.float32), new(T, top_k, dtype=torch.int32)
    purlin.purlin_route(ctx, logits, weights, experts, T, config, code, bias=router_bias, ld=pitch)

    # each rank's slots in the order of their experts, and its row of the count matrix
    place = new(T, top_k, dtype=torch.int32)
    begin, count = new(R, R, dtype=torch.int64), new(R, R, dtype=torch.int64)
    sent = new(T * top_k, H)
    for r in range(R):
        mine = slice(r * rows, (r + 1) * rows)
        purlin.purlin_expert_order(ctx, experts[mine], place[mine], begin[r], count[r], slots, R)
        purlin.purlin_dispatch_rows(ctx, hidden[mine], place[mine],
                                    sent[r * slots:(r + 1) * slots], rows, top_k, H, slots, code)

    got = new(R, cap, H)
    purlin.purlin_all_to_all_v_device_counts(ctx, ranks(sent, slots), list(got), count * H,
                                             slots * H, cap * H, code)
    first, load = torch.arange(R, device=dev) * cap, count.sum(0)
    inner, outer = new(R * cap, N), new(R, cap, H)
    purlin.purlin_grouped_matmul(ctx, got, up, inner, first, load, R, R * cap, N, H, code)
    inner.relu_()
    purlin.purlin_grouped_matmul(ctx, inner, down, outer, first, load, R, R * cap, H, N, code)

    back = new(T * top_k, H)
    purlin.purlin_all_to_all_v_device_counts(ctx, list(outer), ranks(back, slots),
                                             count.t().contiguous() * H, cap * H, slots * H, code)
    block = new(T, H)
    for r in range(R):
        mine = slice(r * rows, (r + 1) * rows)
        purlin.purlin_combine_rows(ctx, back[r * slots:(r + 1) * slots], place[mine], block[mine],
                                   rows, top_k, H, slots, code, weights=weights[mine])
    y, total = norm(block, total, norms[1])
    return {"y": y, "total": total, "load": load, "hidden": hidden, "experts": experts,
            "weights": weights}


def main(R=8, tokens=2048, hidden=4096, width=1024, top_k=2):
    import torch

    g = torch.Generator(device="cuda").manual_seed(5)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).bfloat16()

    def vector():
        return (1 + 0.1 * torch.randn(hidden, device="cuda", generator=g)).bfloat16()

    ctx = purlin.purlin_init(R, torch.cuda.current_stream())
    try:
        norms = [{"post": vector(), "gate": vector(), "weight": vector()} for _ in range(2)]
        args = (ctx, [randn(tokens, hidden) for _ in range(R)], randn(tokens, hidden), norms,
                randn(R, hidden, scale=hidden ** -0.5), torch.zeros(R, device="cuda"),
                randn(R, width, hidden, scale=hidden ** -0.5),
                randn(R, hidden, width, scale=width ** -0.5), top_k)
        moe_block(*args)
        purlin.purlin_check(ctx)
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        r = moe_block(*args)
        b.record()
        purlin.purlin_check(ctx)
        print(f"{R} ranks, {tokens} tokens x {hidden}, {top_k} experts each of {width}: "
              f"{a.elapsed_time(b) * 1e3:.0f} us, load {r['load'].tolist()}, "
              f"rms {float(r['y'].float().square().mean().sqrt()):.3f}")
    finally:
        ctx.close()


if __name__ == "__main__":
    main()
