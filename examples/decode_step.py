"""One decode step around the output projection, as a serving loop would run it.

Latent attention over a paged cache (requests with a few drafted tokens each, in
a tree), the absorbed products around it, and the publishing MXFP8 projection
with a low-rank adapter per request, captured in one CUDA graph and replayed.
With --experts a layer of routed experts in MXFP4 follows on the projection's rows.
Synthetic weights and activations.

    python examples/decode_step.py [--context 4096] [--heads 128] [--experts 64] [--steps 50]
"""
import argparse
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parents[1]))
import mxfp8_gemm_mailbox_gb300 as mx  # noqa: E402

ROPE, PAGE = 64, 64


def bf16(*shape, std=1.0):
    return (torch.randn(*shape, device="cuda") * std).to(torch.bfloat16)


def mxfp8(rows, k):
    """Random MXFP8 rows: E4M3 elements and E8M0 scales of 2^-4 .. 2^2."""
    x = torch.randn(rows, k, device="cuda").to(torch.float8_e4m3fn)
    return x, torch.randint(123, 130, (rows, k // 32), dtype=torch.uint8, device="cuda")


def mxfp4(experts, rows, k):
    """Random MXFP4 matrices of outputs of the order of one."""
    x = torch.randn(experts, rows, k, device="cuda") * k ** -0.5
    return mx.quantize(x, "mxfp4")


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--context", type=int, default=4096)
    ap.add_argument("--heads", type=int, default=128)
    ap.add_argument("--requests", type=int, default=2)
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--hidden", type=int, default=7168)
    ap.add_argument("--rank", type=int, default=32)
    ap.add_argument("--experts", type=int, default=0)
    ap.add_argument("--choices", type=int, default=4)
    ap.add_argument("--inner", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=50)
    args = ap.parse_args()
    torch.manual_seed(0)
    latent, nope, value, heads = 512, 128, 128, args.heads
    width, rows = latent + ROPE, args.requests * args.drafts

    # What a model holds: the absorbed matrices, the projection, the adapters.
    w_query = bf16(heads, latent, nope, std=nope ** -0.5)
    w_value = bf16(heads, value, latent, std=latent ** -0.5)
    mailbox = mx.Mailbox(8, args.hidden)
    gemm = mx.PublishGemm(*mxfp8(args.hidden, heads * value), mailbox)
    adapters = mx.Adapters(bf16(args.requests, args.rank, heads * value, std=0.01),
                           bf16(args.requests, args.hidden, args.rank))
    attention = mx.LatentAttention(heads, latent)
    if args.experts:
        w_route = bf16(args.hidden, args.experts, std=args.hidden ** -0.5)
        first = mx.ExpertProduct(*mxfp4(args.experts, 2 * args.inner, args.hidden), gated=True)
        second = mx.ExpertProduct(*mxfp4(args.experts, args.hidden, args.inner),
                                  workspace=first.workspace)

    # What a serving loop holds: the pool of pages, who owns which, the lengths.
    pages = -(-(args.context + args.drafts + args.steps) // PAGE)
    pool = torch.zeros((args.requests * pages, PAGE, width), dtype=torch.bfloat16, device="cuda")
    table = torch.randperm(pool.shape[0], device="cuda").view(args.requests, pages).int()
    for b in range(args.requests):
        pool[table[b].long()] = bf16(pages, PAGE, width)
    context = torch.full((args.requests,), args.context, dtype=torch.int32, device="cuda")
    lengths = context + args.drafts
    begin = torch.arange(args.requests + 1, dtype=torch.int32, device="cuda") * args.drafts
    which = torch.arange(args.requests, device="cuda").repeat_interleave(args.drafts).int()
    # Two branches off the first draft: 0 -> 1 -> 3, 0 -> 2 (and a chain from there on).
    masks = []
    for j in range(args.drafts):
        parent = {1: 0, 2: 0, 3: 1}.get(j, j - 1)
        masks.append((masks[parent] if j else 0) | 1 << j)
    tree = torch.tensor(masks * args.requests, dtype=torch.int64, device="cuda")

    # The step's inputs, in fixed buffers that the graph reads.
    q_nope, q_rope = bf16(rows, heads, nope), bf16(rows, heads, ROPE)
    new = bf16(args.requests, args.drafts, width)
    out = torch.empty((rows, args.hidden), dtype=torch.bfloat16, device="cuda")
    draft = torch.arange(args.drafts, device="cuda")

    def step():
        at = context[:, None].long() + draft  # the drafts' places in the cache
        pool[table.gather(1, at // PAGE).long(), at % PAGE] = new
        q = mx.latent_query(q_nope, q_rope, w_query)
        o = attention.run(q, pool, table, lengths, begin, (nope + ROPE) ** -0.5, tree=tree)
        x, x_scale = mx.latent_values(o, w_value)
        gemm.run_adapted(x, x_scale, adapters, which)
        mailbox.consume(rows, out)
        if args.experts:
            routing = mx.route(out @ w_route, args.choices)
            h, h_scale = mx.quantize(out, "mxfp8", rows=routing.row)
            h, h_scale = first.run(h, h_scale, routing.begin, format="mxfp8")
            y = second.run(h, h_scale, routing.begin)
            mx.combine(y, routing.weight, routing.slot, add=out, out=out)

    step()  # once outside the capture
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        step()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    with torch.cuda.stream(stream):
        graph.replay()
        start.record()
        for _ in range(args.steps):
            graph.replay()
            context.add_(1)  # one draft accepted a step; lengths are read on the device
            lengths.add_(1)
        end.record()
    torch.cuda.synchronize()
    status, words = mailbox.status()
    assert status == mx.OK and attention.status() == 0, (status, words)
    assert torch.isfinite(out).all()
    if args.experts:
        assert first.status() == 0 and second.status() == 0
    layer = f", {args.choices} of {args.experts} experts" if args.experts else ""
    print(f"{args.requests} requests x {args.drafts} drafts, {heads} heads, context "
          f"{args.context}{layer}: {start.elapsed_time(end) / args.steps * 1e3:.1f} us a step")


if __name__ == "__main__":
    main()
