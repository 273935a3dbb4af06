"""Routing of tokens to experts with its losses and gradient, on the GPU against
the formulas in 64 bits."""
from __future__ import annotations

import math

import pytest
import torch

from route_ref import DT, Case
from xent_ref import within

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import matrix_multiply_gb300 as tg
else:  # collected on CPU only to be deselected
    tg = None


@pytest.fixture(scope="module")
def ctx():
    c = tg.Context(0)
    yield c
    c.close()


def forward(ctx, c):
    ids = torch.full((c.T, c.k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((c.T, c.k), math.nan, device="cuda")
    counts = torch.full((c.E + 1,), -7, dtype=torch.int32, device="cuda")
    losses = torch.full((2,), math.nan, device="cuda")
    torch.cuda.synchronize()
    tg.tc_moe_route(ctx, c.desc(tg), c.l, ids, w, counts, losses, valid=c.valid)
    return ids, w, counts, losses


def backward(ctx, c, ids, counts, pad=0, **kw):
    full = torch.full((c.T + 2, c.E + pad), 123.0, dtype=DT[c.grad], device="cuda")
    dl = full[1:1 + c.T, :c.E]
    kw = {"grad_weights": c.gw, "grad_losses": c.gl, **kw}
    torch.cuda.synchronize()
    tg.tc_moe_route_backward(ctx, c.desc(tg, ld_dlogits=c.E + pad), c.l, ids, counts, dl, valid=c.valid, **kw)
    out = dl.clone()
    dl.fill_(123.0)
    assert bool((full == 123.0).all())
    return out


def check(ctx, c, pad=0):
    ids, w, ew, counts, losses, el = c.forward()
    got = forward(ctx, c)
    assert torch.equal(got[0], ids), ctx.last_kernel
    assert torch.equal(got[2], counts)
    within(got[1], w, ew, f"weights {ctx.last_kernel}")
    within(got[3], losses, el, f"losses {ctx.last_kernel}")
    within(backward(ctx, c, ids, counts, pad), *c.backward(ids, counts), "all gradients")
    within(backward(ctx, c, ids, counts, pad, grad_weights=None), *c.backward(ids, counts, with_weights=False), "losses'")
    within(backward(ctx, c, ids, counts, pad, grad_losses=None), *c.backward(ids, counts, with_losses=False), "weights'")


@pytest.mark.parametrize("E,k", [(1, 1), (2, 1), (7, 7), (13, 3), (16, 16), (31, 2), (32, 8), (33, 5), (60, 4), (64, 8),
                                 (100, 6), (128, 8), (129, 1), (255, 16), (256, 8), (257, 9), (384, 8), (511, 16), (512, 16)])
@pytest.mark.parametrize("T", [1, 5, 64, 65, 700])
def test_sizes(ctx, E, k, T):
    dtype = ("f32", "bf16", "f16")[(E + T) % 3]
    check(ctx, Case(T, E, k, dtype, renorm=(E + T) % 2 == 0, padded=T % 2 == 1 and T > 1, seed=1))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("grad", [None, "f32"])
@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("E", [24, 64, 120, 256, 300])
def test_types_and_strides(ctx, dtype, grad, pad, E):
    check(ctx, Case(170, E, 4, dtype, grad=grad, pad=pad, padded=True, seed=2), pad=pad)


@pytest.mark.parametrize("E", [8, 60, 256, 512])
def test_many_tokens(ctx, E):
    check(ctx, Case(20011, E, 8, "f32", padded=True, seed=3))


@pytest.mark.parametrize("E,k", [(9, 4), (64, 8), (100, 16), (256, 8), (512, 16)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ties_go_to_the_lowest_index(ctx, E, k, dtype):
    """Logits that are whole numbers, 0 of either sign among them."""
    check(ctx, Case(333, E, k, dtype, ties=True, seed=4))


def test_all_equal(ctx):
    c = Case(40, 256, 16, seed=5)
    c.l.fill_(-0.25)
    ids, w, counts, losses = forward(ctx, c)
    assert torch.equal(ids, torch.arange(16, device="cuda", dtype=torch.int32).expand(40, 16))
    # f = 1/16 for 16 experts, P = 1/256: the loss is 256 * 16 * (1/16) (1/256) = 1
    assert abs(float(losses[0]) - 1) < 1e-5


@pytest.mark.parametrize("E,k", [(5, 3), (40, 8), (256, 8), (400, 16)])
@pytest.mark.parametrize("renorm", [False, True])
def test_masked_experts(ctx, E, k, renorm):
    """Tokens that keep fewer experts than they would choose, or none."""
    c = Case(300, E, k, "f32", renorm=renorm, masked=0.9, padded=True, seed=6)
    c.l[7] = -math.inf
    c.l[8] = -math.inf
    c.l[8, E - 1] = 1.0
    c.valid[7:9] = 1
    ids = c.choice()
    assert int(ids[8, 0]) == E - 1 and bool((ids[8, 1:] == -1).all()) and bool((ids[7] == -1).all())
    check(ctx, c)


def test_lowest_value_is_not_masked(ctx):
    """The type's lowest value is a logit like others: chosen once nothing larger is left."""
    c = Case(20, 40, 5, "bf16", seed=7)
    c.l[:, 2:] = torch.finfo(torch.bfloat16).min
    ids, w, counts, losses = forward(ctx, c)
    assert torch.equal(ids, c.choice().to(torch.int32)) and int(ids.min()) >= 0
    assert bool((w[:, 2:] == 0).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_nan_and_inf(ctx, bad):
    """A NaN counts as the largest (either sign); the token's numbers are NaN, its choice and the counts are not."""
    c = Case(50, 100, 6, "f32", seed=8)
    c.l[3, 70] = bad
    c.l[3, 20] = math.copysign(bad, -1.0) if math.isnan(bad) else 5.0
    ids, w, counts, losses = forward(ctx, c)
    want = c.choice().to(torch.int32)
    assert torch.equal(ids, want)
    assert int(counts[-1]) == 50 and int(counts[:-1].sum()) == 300
    keep = torch.arange(50, device="cuda") != 3
    assert bool(w[3].isnan().any()) and not bool(w[keep].isnan().any())
    g = backward(ctx, c, ids, counts)
    assert not bool(g[keep].isnan().any())


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_padding_is_not_seen(ctx, bad):
    c = Case(90, 64, 8, "f32", padded=True, seed=9)
    want = forward(ctx, c)
    g = backward(ctx, c, want[0], want[2])
    c.l[c.valid == 0] = bad
    got = forward(ctx, c)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert torch.equal(g, backward(ctx, c, got[0], got[2]))
    assert bool((got[0][c.valid == 0] == -1).all()) and bool((g[c.valid == 0] == 0).all())


def test_no_token_counts(ctx):
    for T in (3, 500):
        c = Case(T, 64, 8, "f32", padded=True, seed=10)
        c.valid.zero_()
        ids, w, counts, losses = forward(ctx, c)
        assert bool((ids == -1).all()) and bool((w == 0).all()) and bool((counts == 0).all()) and bool((losses == 0).all())
        assert bool((backward(ctx, c, ids, counts) == 0).all())


def test_bool_mask(ctx):
    c = Case(77, 64, 8, "f32", padded=True, seed=11)
    want = forward(ctx, c)
    c.valid = c.valid.bool()
    assert all(torch.equal(a, b) for a, b in zip(want, forward(ctx, c)))


def test_ids_out_of_range_are_no_choice(ctx):
    """Also an index met twice: its gradients add up."""
    c = Case(30, 64, 4, "f32", renorm=False, seed=12)
    ids, _, _, counts, _, _ = c.forward()
    ids[0, 1], ids[1, 2], ids[2, 0] = 64, -5, 2 ** 31 - 1
    ids[3, 1] = ids[3, 0]
    cut = torch.where((ids < 0) | (ids >= 64), -1, ids)
    within(backward(ctx, c, ids, counts), *c.backward(cut, counts))


def test_gradient_against_differences(ctx):
    """Sum of weights times numbers, plus the losses, by differences of the 64-bit forms."""
    for renorm in (False, True):
        c = Case(6, 10, 3, "f32", renorm=renorm, seed=13)
        ids, w, counts, losses = forward(ctx, c)
        got = backward(ctx, c, ids, counts).double()
        f = counts[:-1].double() / (6 * 3)

        def value(l):
            p = torch.softmax(l, 1)
            w = p.gather(1, ids.long())
            w = w / w.sum(1, True) if renorm else w
            balance = 10 * (f * p.mean(0)).sum()
            return (c.gw.double() * w).sum() + c.gl[0].double() * balance + c.gl[1].double() * (torch.logsumexp(l, 1) ** 2).mean()

        l, h = c.l.double(), 1e-5
        for t, e in ((0, 0), (2, 5), (5, 9), (3, int(ids[3, 0])), (4, int(ids[4, 2]))):
            up, down = l.clone(), l.clone()
            up[t, e] += h
            down[t, e] -= h
            assert abs(float((value(up) - value(down)) / (2 * h)) - float(got[t, e])) < 1e-5


def test_repeats_bit_for_bit(ctx):
    c = Case(30000, 256, 8, "f32", padded=True, seed=14)
    first = forward(ctx, c)
    g = backward(ctx, c, first[0], first[2])
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, forward(ctx, c)))
        assert torch.equal(g, backward(ctx, c, first[0], first[2]))


def test_same_choice_as_the_experts_layer(ctx):
    """tc_moe_q4 chooses for the same logits the same experts, with the same weights."""
    T, H, E, k = 20, 128, 24, 5
    g = torch.Generator().manual_seed(15)
    X = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    R = (torch.randn(E, H, generator=g) / H ** 0.5).to(torch.bfloat16).cuda()
    q = [tg.Q4Weight.empty(*s, 32) for s in ((E * 2 * 32, H), (E * H, 32))]
    for w in q:
        W = torch.randn(w.N, w.K, generator=g).cuda()
        torch.cuda.synchronize()
        tg.tc_quantize_q4(ctx, W, w)
    Y, ids, p = torch.empty(T, H, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    tg.tc_moe_q4(ctx, tg.make_moe_desc(T, H, 32, E, k, "bf16", "f32", router_dtype="bf16"), X, R, *q, Y, ids=ids, weights=p)
    c = Case(T, E, k, "f32", seed=15)
    c.l = torch.empty(T, E, device="cuda")
    tg.tc_gemm(ctx, tg.make_desc(T, E, H, "bf16", "f32", transpose_b=True), X, R, c.l)
    got = forward(ctx, c)
    assert torch.equal(got[0], ids)
    # both logits are fp32 sums of 128 products: 2^-16 of the sum of their sizes, twice for the difference to the largest
    assert bool(((got[1] - p).abs() <= 2.0 ** -16 * 4 * 40 * p).all())
