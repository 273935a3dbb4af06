"""What a mixture-of-experts model trains on, and its gradients: routing with its
balance loss, cross entropy over a vocabulary, both without keeping anything of
their size, on one stream with the products between them.

    python examples/expert_losses.py [tokens]

hidden X [tokens, HIDDEN], router R [EXPERTS, HIDDEN], head W [VOCAB, HIDDEN]:
loss = mean cross entropy of X W^T + 0.01 * balance(X R^T) + 0.001 * mean lse^2
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_multiply_gb300 as tg  # noqa: E402

HIDDEN, VOCAB, EXPERTS, TOP_K = 512, 16000, 32, 4


def main(tokens: int = 256) -> tuple[float, ...]:
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape, std):
        return (torch.randn(*shape, device="cuda", generator=g) * std).to(torch.bfloat16)

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    ctx = tg.Context(torch.cuda.current_device())
    stream = tg.Stream(ctx, torch.cuda.current_stream())          # the library joins torch's stream
    X, R, W = normal(tokens, HIDDEN, std=1.0), normal(EXPERTS, HIDDEN, std=HIDDEN ** -0.5), normal(VOCAB, HIDDEN, std=HIDDEN ** -0.5)
    y = torch.randint(0, VOCAB, (tokens,), device="cuda", generator=g)
    valid = torch.arange(tokens, device="cuda") < max(1, tokens - tokens // 8)     # the rest is padding
    y[~valid] = -100
    weights_of = torch.tensor([0.01, 0.001], device="cuda")

    logits, dlogits = empty(tokens, EXPERTS), empty(tokens, EXPERTS)
    ids, p = empty(tokens, TOP_K, dtype=torch.int32), empty(tokens, TOP_K)
    counts, losses = empty(EXPERTS + 1, dtype=torch.int32), empty(2)
    loss, lse, dX, dW, dR = empty(1), empty(tokens), empty(tokens, HIDDEN), empty(VOCAB, HIDDEN), empty(EXPERTS, HIDDEN)

    # forward
    tg.gemm(ctx, X, R, logits, transpose_b=True, stream=stream)
    route = tg.PreparedRoute(ctx, tg.make_route_desc(tokens, EXPERTS, TOP_K), logits, ids, counts, stream, valid=valid,
                             weights=p, losses=losses, grad_losses=weights_of, dlogits=dlogits)
    head = tg.PreparedXent(ctx, tg.make_xent_desc(tokens, HIDDEN, VOCAB, "bf16", "f32"), X, W, y, lse, stream, loss=loss,
                           grad=torch.ones(1, device="cuda"), dX=dX, dW=dW)
    route.enqueue()
    head.enqueue()
    # backward: the router's part of dX is added to the head's
    head.enqueue_backward()
    route.enqueue_backward()
    d16 = dlogits.to(torch.bfloat16)
    tg.gemm(ctx, d16, R, dX, beta=1.0, stream=stream)
    tg.gemm(ctx, d16, X, dR, transpose_a=True, stream=stream)
    stream.sync()

    # the same in 64 bits, by automatic differentiation
    x, r, w = (t.double().requires_grad_() for t in (X, R, W))
    rl = x @ r.t()
    probs, n = torch.softmax(rl[valid], 1), int(valid.sum())
    f = counts[:EXPERTS].double() / (n * TOP_K)
    total = torch.nn.functional.cross_entropy(x @ w.t(), y, ignore_index=-100)
    total = total + weights_of[0].double() * EXPERTS * (f * probs.mean(0)).sum()
    total = total + weights_of[1].double() * (torch.logsumexp(rl[valid], 1) ** 2).mean()
    total.backward()
    mine = float(loss) + float((losses * weights_of).sum())
    off = tuple(float((a.double() - b.grad).norm() / b.grad.norm()) for a, b in ((dX, x), (dW, w), (dR, r)))
    print(f"{tokens} tokens, {n} of them counted: loss {mine:.5f} ({float(total.detach()):.5f} in 64 bits), gradients of X, W, "
          f"R off by {off[0]:.1e}, {off[1]:.1e}, {off[2]:.1e}; busiest expert {int(counts[:EXPERTS].max())} of {n * TOP_K}")
    return (abs(mine - float(total.detach())),) + off


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 256)
