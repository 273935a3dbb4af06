"""Softmax cross entropy against a vocabulary, forward and backward, on the GPU
against the formulas in 64 bits."""
from __future__ import annotations

import math

import pytest
import torch

from xent_ref import DT, Case, within

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


GUARD = 12345.0


def framed(rows, cols, dtype, pad):
    """A matrix inside a larger one, whose frame must stay as it is."""
    full = torch.full((rows + 2, cols + pad), GUARD, dtype=dtype, device="cuda")
    return full, full[1:1 + rows, :cols]


def frame_kept(full, rows, cols):
    inner = full.clone()
    inner[1:1 + rows, :cols] = GUARD
    return bool((inner == torch.full_like(inner, GUARD)).all())


def forward(ctx, c):
    loss = torch.full((c.T if c.reduction == "none" else 1,), math.nan, device="cuda")
    lse = torch.full((c.T,), math.nan, device="cuda")
    torch.cuda.synchronize()
    tg.tc_linear_xent(ctx, c.desc(tg), c.X, c.W, c.y, loss, lse)
    return loss, lse


def backward(ctx, c, lse, want=("dX", "dW"), pad=0):
    fx, dX = framed(c.T, c.H, DT[c.grad], pad)
    fw, dW = framed(c.V, c.H, DT[c.grad], pad)
    torch.cuda.synchronize()
    tg.tc_linear_xent_backward(ctx, c.desc(tg, lddx=c.H + pad, lddw=c.H + pad), c.X, c.W, c.y, lse, c.g,
                               dX if "dX" in want else None, dW if "dW" in want else None)
    assert frame_kept(fx, c.T, c.H) and frame_kept(fw, c.V, c.H)
    return dX, dW


def check(ctx, c, pad=0):
    loss, eloss, lse, elf = c.forward()
    got = forward(ctx, c)
    within(got[1], lse, elf, f"lse {ctx.last_kernel}")
    within(got[0], loss, eloss, f"loss {ctx.last_kernel}")
    lse32 = c.lse32()
    dX, ex, dW, ew = c.backward(lse32)
    gx, gw = backward(ctx, c, lse32, pad=pad)
    within(gx, dX, ex, f"dX {ctx.last_kernel}")
    within(gw, dW, ew, f"dW {ctx.last_kernel}")


@pytest.mark.parametrize("T", [1, 2, 9, 128, 129, 300])
@pytest.mark.parametrize("V", [1, 31, 256, 1000, 4099])
def test_sizes(ctx, T, V):
    check(ctx, Case(T, 72, V, ("bf16", "f16")[(T + V) % 2], z=0.01, ignored=0.2, wide=T % 2 == 0, seed=1))


@pytest.mark.parametrize("H", [1, 8, 63, 64, 65, 257, 1001])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_hidden(ctx, H, dtype):
    check(ctx, Case(70, H, 515, dtype, reduction="mean", ignored=0.1, seed=2))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("grad", ["own", "f32"])
@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_kinds(ctx, dtype, grad, reduction, pad):
    c = Case(150, 200, 777, dtype, reduction=reduction, grad=None if grad == "own" else "f32", pad=pad, scale=0.7,
             z=0.003, ignored=0.3, wide=pad == 3, seed=3)
    check(ctx, c, pad=pad)


@pytest.mark.parametrize("grad", [None, "f32"])
def test_pair_tiles(ctx, monkeypatch, grad):
    """Enough rows and columns for the paired tiles (fp32 gradients are planned in
    smaller ones there); a vocabulary that ends inside one."""
    if grad:
        monkeypatch.setenv("TC_FORCE_VARIANT", "bn=256 cg=2")
    c = Case(1270, 320, 20011, "bf16", reduction="mean", ignored=0.1, grad=grad, seed=4)
    check(ctx, c)
    assert "pair" in ctx.last_kernel


@pytest.mark.parametrize("dtype,grad,pad", [("bf16", None, 0), ("f16", None, 1), ("bf16", "f32", 0)])
def test_pieces(ctx, dtype, grad, pad):
    """G of more than one piece of the vocabulary: dX is summed over them."""
    c = Case(4100, 72, 40000 if grad is None else 20000, dtype, reduction="mean", ignored=0.1, grad=grad, pad=pad, seed=5)
    check(ctx, c)
    assert ctx.last_kernel.endswith("_p2")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("H", [64, 129])
def test_bases_off_16_bytes(ctx, dtype, H):
    """Every operand begins one element behind an aligned address."""
    c = Case(70, H, 600, dtype, reduction="mean", ignored=0.2, seed=17)

    def behind(t):
        full = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        out = full[1:].view(t.shape)
        out.copy_(t)
        return out

    c.X, c.W, c.y, c.g = behind(c.X), behind(c.W), behind(c.y), behind(c.g)
    loss, eloss, lse, elf = c.forward()
    out = [behind(torch.zeros(n, device="cuda")) for n in (1, c.T)]
    torch.cuda.synchronize()
    tg.tc_linear_xent(ctx, c.desc(tg), c.X, c.W, c.y, *out)
    within(out[0], loss, eloss)
    within(out[1], lse, elf)
    lse32 = behind(c.lse32())
    dX, ex, dW, ew = c.backward(lse32)
    gx, gw = behind(torch.zeros_like(c.X)), behind(torch.zeros_like(c.W))
    torch.cuda.synchronize()
    tg.tc_linear_xent_backward(ctx, c.desc(tg), c.X, c.W, c.y, lse32, c.g, gx, gw)
    within(gx, dX, ex)
    within(gw, dW, ew)


@pytest.mark.parametrize("T", [1, 31, 32, 33, 64, 65, 128, 129])
@pytest.mark.parametrize("dtype,grad", [("bf16", None), ("f16", None), ("bf16", "f32"), ("f16", "f32")])
def test_parts_of_g(ctx, T, dtype, grad):
    """The parts of G around whole warps and tiles, with a vocabulary long enough
    for the cluster split that adds them up, and a hidden size of several segments."""
    check(ctx, Case(T, 1100, 2100, dtype, reduction="none", z=0.001, ignored=0.1, grad=grad, seed=18))


@pytest.mark.parametrize("T", [20, 200])
@pytest.mark.parametrize("dtype,grad", [("bf16", None), ("f16", None), ("bf16", "f32")])
@pytest.mark.parametrize("reduction", ["sum", "mean"])
@pytest.mark.parametrize("g", [float("inf"), float("nan")])
def test_gradient_that_is_no_number(ctx, T, dtype, grad, reduction, g):
    """It reaches the rows that count and no other; where none counts, nothing."""
    c = Case(T, 130, 600, dtype, reduction=reduction, ignored=0.3, grad=grad, seed=19)
    c.g.fill_(g)
    lse32 = c.lse32()
    out = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype] if grad is None else torch.float32
    counted = (c.y >= 0) & (c.y < 600)
    assert 0 < int(counted.sum()) < T
    for none in (False, True):
        if none:
            c.y.fill_(-100)
            counted = counted & False
        dX, dW = torch.ones(c.X.shape, dtype=out, device="cuda"), torch.ones(c.W.shape, dtype=out, device="cuda")
        torch.cuda.synchronize()
        tg.tc_linear_xent_backward(ctx, c.desc(tg), c.X, c.W, c.y, lse32, c.g, dX, dW)
        assert bool((dX[~counted] == 0).all())
        assert not bool(torch.isfinite(dX[counted]).any())
        assert bool((dW == 0).all()) if none else not bool(torch.isfinite(dW).all())


def test_frozen(ctx):
    c = Case(40, 64, 500, seed=6)
    lse = c.lse32()
    both = backward(ctx, c, lse)
    only = backward(ctx, c, lse, ("dX",))
    assert torch.equal(only[0], both[0]) and bool((only[1] == GUARD).all())
    only = backward(ctx, c, lse, ("dW",))
    assert torch.equal(only[1], both[1]) and bool((only[0] == GUARD).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_no_row_counts(ctx, dtype, reduction):
    c = Case(33, 64, 300, dtype, reduction=reduction, ignored=1.1, seed=7)
    loss, lse = forward(ctx, c)
    assert bool((loss == 0).all())
    within(lse, c.forward()[2], c.forward()[3])
    dX, dW = backward(ctx, c, lse)
    assert bool((dX == 0).all()) and bool((dW == 0).all())


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_does_not_count_is_not_seen(ctx, bad):
    """A padding row may hold anything: its loss is 0 and no gradient sees it."""
    c = Case(60, 64, 300, "bf16", reduction="mean", ignored=0.4, z=0.01, seed=8)
    clean, rows = c.X.clone(), ~c.counted()
    c.X[rows] = bad
    loss, lse = forward(ctx, c)
    dX, dW = backward(ctx, c, lse)
    c.X = clean
    want = forward(ctx, c)
    assert torch.equal(loss, want[0]) and torch.equal(lse[~rows], want[1][~rows])
    gx, gw = backward(ctx, c, want[1])
    assert torch.equal(dX, gx) and torch.equal(dW, gw) and bool((dX[rows] == 0).all())


def test_nan_row_stays_its_own_in_the_loss(ctx):
    c = Case(20, 64, 300, "bf16", seed=9)
    want = forward(ctx, c)
    c.X[3, 5] = math.nan
    loss, lse = forward(ctx, c)
    keep = torch.arange(20, device="cuda") != 3
    assert bool(loss[3].isnan()) and bool(lse[3].isnan())
    assert torch.equal(loss[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])


def test_wide_logits(ctx):
    """Logits in the thousands: nothing overflows, the largest decides."""
    c = Case(50, 64, 700, "bf16", lift=6.0, seed=10)
    c.X *= 500
    check(ctx, c)


@pytest.mark.parametrize("size", [1e-12, 1e12])
def test_size_of_the_gradient(ctx, size):
    """f16 gradients of any size: fp32 outputs show what the rounding to 16 bits on the way kept."""
    c = Case(50, 64, 700, "f16", grad="f32", seed=11)
    c.g *= size
    check(ctx, c)


def test_gradient_against_differences(ctx):
    """The backward call against differences of the forward call, both the library's."""
    c = Case(12, 24, 40, "f16", reduction="sum", z=0.02, grad="f32", ignored=0.2, seed=12)
    c.g.fill_(1.0)
    loss, lse = forward(ctx, c)
    dX, dW = backward(ctx, c, lse)
    for name, t, d in (("X", c.X, dX), ("W", c.W, dW)):
        for i, j in ((0, 0), (3, 7), (11, 23)):
            old = t[i, j].clone()
            step = []
            for sign in (1, -1):
                t[i, j] = old + sign * 0.0625
                step.append((float(t[i, j]), float(forward(ctx, c)[0])))
            t[i, j] = old
            diff = (step[0][1] - step[1][1]) / (step[0][0] - step[1][0])
            # the third derivative times h^2 / 6, and two losses of 2^-21 relative error over 2 h
            assert abs(diff - float(d[i, j])) <= 0.0625 ** 2 * 2 + abs(step[0][1]) * 2.0 ** -20 / 0.125, (name, i, j)


def test_repeats_bit_for_bit(ctx):
    c = Case(300, 200, 5000, "f16", reduction="mean", ignored=0.1, seed=13)
    first, lse = forward(ctx, c), c.lse32()
    grads = [t.clone() for t in backward(ctx, c, lse)]
    for _ in range(3):
        again = forward(ctx, c)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        assert all(torch.equal(a, b) for a, b in zip(grads, backward(ctx, c, lse)))


@pytest.mark.parametrize("bn,cg", [(256, 2), (256, 1), (128, 1)])
def test_every_tile_shape(ctx, monkeypatch, bn, cg):
    monkeypatch.setenv("TC_FORCE_VARIANT", f"bn={bn} cg={cg}")
    c = Case(300, 130, 3001, "bf16", reduction="sum", ignored=0.2, grad="f32", seed=14)
    loss, eloss, lse, elf = c.forward()
    got = forward(ctx, c)
    assert f"{128 * cg}x{bn}" in ctx.last_kernel
    within(got[1], lse, elf)
    within(got[0], loss, eloss)
    monkeypatch.setenv("TC_FORCE_VARIANT", f"cg={cg}")      # (the gradient's products have all widths)
    lse32 = c.lse32()
    dX, ex, dW, ew = c.backward(lse32)
    gx, gw = backward(ctx, c, lse32)
    within(gx, dX, ex)
    within(gw, dW, ew)


def off(out, want):
    return float((out.double() - want).norm() / want.norm())


@pytest.mark.parametrize("H", [512, 2000, 4096])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_fp32_results_are_fp32(ctx, H, dtype):
    """Long sums do not lose what the tensor core truncates: a segment of 512
    products loses at most (512 / 16) 2^-24 = 1.9e-6 of their sizes' sum, half of
    it on average, and an exponential of a few tenths less errs by a few 1e-7."""
    c = Case(200, H, 6000, dtype, grad="f32", seed=16)
    loss, _, lse, _ = c.forward()
    got = forward(ctx, c)
    assert off(got[1], lse) < 1e-6 and off(got[0], loss) < 2e-6
    dX, _, dW, _ = c.backward(c.lse32())
    gx, gw = backward(ctx, c, c.lse32())
    # G in two parts: half a step of bf16, squared, is 2^-16 at most, a third of it on average
    limit = 1e-5 if dtype == "bf16" else 4e-6
    assert off(gx, dX) < limit and off(gw, dW) < limit
