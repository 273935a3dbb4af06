"""A decoding step's weights in 4 bits, end to end: quantise a projection and a
layer of experts, run both for a few tokens on one stream, and compare with the
same formulas in fp32 over the values the codes stand for.

    python examples/q4_block.py [tokens]

y = x + P x;  out = y + experts(y), with P [hidden, hidden] and the experts'
gate, up and down matrices as tc_q4_weight (groups of 64, zero points for the
experts).
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import matrix_multiply_gb300 as tg  # noqa: E402

HIDDEN, INTER, EXPERTS, TOP_K = 1024, 512, 8, 2


def quantised(ctx, stream, W, zeros):
    q = tg.Q4Weight.empty(*W.shape, 64, zeros=zeros)
    tg.tc_quantize_q4_async(ctx, W, q, stream)
    return q


def values(ctx, stream, q):
    V = torch.empty(q.N, q.K, device="cuda")
    tg.tc_dequantize_q4_async(ctx, q, V, stream)
    return V


def main(tokens: int = 4) -> float:
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape, std):
        return (torch.randn(*shape, device="cuda", generator=g) * std).to(torch.bfloat16)

    ctx = tg.Context(torch.cuda.current_device())
    stream = tg.Stream(ctx, torch.cuda.current_stream())          # the library joins torch's stream
    x = normal(tokens, HIDDEN, std=1.0)
    router = normal(EXPERTS, HIDDEN, std=HIDDEN ** -0.5).float()
    P = quantised(ctx, stream, normal(HIDDEN, HIDDEN, std=HIDDEN ** -0.5), zeros=False)
    W1 = quantised(ctx, stream, normal(EXPERTS * 2 * INTER, HIDDEN, std=HIDDEN ** -0.5), zeros=True)
    W2 = quantised(ctx, stream, normal(EXPERTS * HIDDEN, INTER, std=INTER ** -0.5), zeros=True)

    y = x.clone()
    moe_out = torch.empty(tokens, HIDDEN, device="cuda")
    ids = torch.empty(tokens, TOP_K, dtype=torch.int32, device="cuda")
    d = tg.make_desc(tokens, HIDDEN, HIDDEN, "bf16", "bf16", b_dtype="i4", transpose_b=True, beta=1.0)
    project = tg.PreparedGemm(ctx, d, x, P, y, stream)            # y = x P^T + y, the residual in the same call
    layer = tg.PreparedMoe(ctx, tg.make_moe_desc(tokens, HIDDEN, INTER, EXPERTS, TOP_K, "bf16", "f32"), y, router, W1, W2,
                           moe_out, stream, ids=ids)
    project.enqueue()
    layer.enqueue()
    out = y.float() + moe_out
    stream.sync()

    # the same in fp32 over the values the codes stand for
    want_y = (x.float() + x.float() @ values(ctx, stream, P).t()).to(torch.bfloat16)
    v1, v2 = values(ctx, stream, W1).reshape(EXPERTS, 2, INTER, HIDDEN), values(ctx, stream, W2).reshape(EXPERTS, HIDDEN, INTER)
    p = torch.softmax(y.float() @ router.t(), -1)
    top, chosen = p.topk(TOP_K)
    top = top / top.sum(-1, keepdim=True)
    assert torch.equal(chosen.to(torch.int32), ids)
    want = y.float()
    for t in range(tokens):
        for j in range(TOP_K):
            gate, up = v1[chosen[t, j]] @ y[t].float()
            want[t] += top[t, j] * (v2[chosen[t, j]] @ (torch.nn.functional.silu(gate) * up))
    err = float((out - want).norm() / want.norm())
    print(f"{tokens} tokens through {ctx.last_kernel}: projection differs by "
          f"{float((y.float() - want_y.float()).norm() / want_y.float().norm()):.1e}, experts by {err:.1e}")
    return err


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 4)
