"""The mixture-of-experts layer over 4-bit weights on GB300 against its
formulas in 64 bits; the bound is derived there (q4_ref.moe)."""
from __future__ import annotations

import pytest
import torch

import q4_ref
from q4_ref import DT, Weight, ulp, within

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


def problem(T, H, I, E, k, x="bf16", r="f32", group=32, zeros=True, scale="f16", seed=0, **kw):
    g = torch.Generator().manual_seed(seed + T * H + I)
    X = (torch.randn(T, H, generator=g) * torch.where(torch.rand(H, generator=g) < 0.02, 8.0, 1.0)).to(DT[x])
    R = (torch.randn(E, H, generator=g) / H ** 0.5).to(DT[r])
    w1 = Weight(E * 2 * I, H, group, zeros, scale, seed + 1, std=H ** -0.5, **kw)
    w2 = Weight(E * H, I, group, zeros, scale, seed + 2, std=I ** -0.5, **kw)
    return X, R, w1, w2


def layer(ctx, X, R, w1, w2, I, E, k, y="f32", renorm=True, stream=None, q=None, **ld):
    T, H = X.shape
    x = {torch.float16: "f16", torch.bfloat16: "bf16"}[X.dtype]
    r = {torch.float16: "f16", torch.bfloat16: "bf16", torch.float32: "f32"}[R.dtype]
    Y = torch.full((T, H), float("nan"), dtype=DT[y], device="cuda")
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    p = torch.full((T, k), float("nan"), device="cuda")
    d = tg.make_moe_desc(T, H, I, E, k, x, y, router_dtype=r, renormalize=renorm, **ld)
    q1, q2 = q or (w1.cuda(tg), w2.cuda(tg))
    torch.cuda.synchronize()                               # the library's stream does not wait for torch's
    if stream is None:
        tg.tc_moe_q4(ctx, d, X, R, q1, q2, Y, ids, p)
    else:
        tg.tc_moe_q4_async(ctx, d, X, R, q1, q2, Y, stream, ids, p)
        stream.sync()
    return Y, ids, p


def check(Y, ids, p, X, R, w1, w2, I, k, y, renorm, what=""):
    want, wids, wp, b, dp = q4_ref.moe(X, R, w1, w2, I, k, renorm)
    assert torch.equal(ids.cpu().long(), wids), what
    within(p.cpu(), wp, wp * dp[:, None], what + " p")
    within(Y.cpu(), want, b + (ulp(want, y) if y != "f32" else 2.0 ** -23 * want.abs()), what)


SHAPES = [(1, 64, 32, 4, 1), (1, 256, 128, 8, 2), (2, 100, 33, 5, 5), (3, 520, 264, 9, 3), (5, 1000, 333, 13, 3),
          (8, 512, 96, 16, 8), (16, 384, 200, 12, 4), (17, 129, 77, 3, 2), (32, 256, 64, 6, 2), (1, 1, 1, 1, 1),
          (32, 300, 40, 1, 1), (4, 2048, 768, 8, 4), (2, 96, 40, 512, 16), (9, 31, 7, 40, 6)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("x,y,r", [("bf16", "bf16", "f32"), ("f16", "f32", "f16"), ("bf16", "f32", "bf16")])
@pytest.mark.parametrize("group,zeros,renorm", [(32, True, True), (128, False, False), (64, True, True)])
def test_layer(ctx, shape, x, y, r, group, zeros, renorm):
    T, H, I, E, k = shape
    X, R, w1, w2 = problem(T, H, I, E, k, x, r, group, zeros, "bf16" if zeros else "f16")
    out = layer(ctx, X.cuda(), R.cuda(), w1, w2, I, E, k, y, renorm)
    check(*out, X, R, w1, w2, I, k, y, renorm, f"{shape} {x}->{y} {ctx.last_kernel}")


@pytest.mark.parametrize("shape", [(2, 6000, 40, 3, 2), (9, 9100, 24, 3, 1), (3, 72, 5000, 3, 2), (20, 5200, 70, 12, 3)])
def test_long_axes(ctx, shape):
    """hidden beyond one slab per warp and one panel of rows, inter beyond one
    slab, more than 8 tokens to an expert."""
    T, H, I, E, k = shape
    X, R, w1, w2 = problem(T, H, I, E, k, group=64)
    out = layer(ctx, X.cuda(), R.cuda(), w1, w2, I, E, k)
    check(*out, X, R, w1, w2, I, k, "f32", True, f"{shape}")


@pytest.mark.parametrize("shape", [(1, 256, 128, 8, 2), (3, 520, 264, 9, 3), (16, 384, 200, 12, 4), (32, 256, 64, 6, 2),
                                   (32, 5000, 40, 3, 2), (20, 4000, 72, 5, 2), (9, 9100, 24, 3, 1), (2, 72, 5000, 3, 2)])
@pytest.mark.parametrize("x", ["bf16", "f16"])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, True), (128, False)])
def test_tall_pieces(ctx, monkeypatch, shape, x, group, zeros):
    """Pieces of two units and 32 rows: odd numbers of units, panels of 8 to 32
    rows, several panels, several slabs to a warp."""
    monkeypatch.setenv("TC_FORCE_VARIANT", "tail=1")
    T, H, I, E, k = shape
    X, R, w1, w2 = problem(T, H, I, E, k, x, "f32", group, zeros)
    out = layer(ctx, X.cuda(), R.cuda(), w1, w2, I, E, k, x)
    assert ctx.last_kernel.endswith("_tall")
    check(*out, X, R, w1, w2, I, k, x, True, f"{shape}")


@pytest.mark.parametrize("x", ["bf16", "f16"])
def test_fp32_outputs_keep_24_bits(ctx, x):
    """One expert, one column of inter, one element of x per token: nothing is
    summed, so a factor's error is an output's.  Fewer than 16 roundings of
    2^-24 (scales, the exponential's two units, the sigmoid, the products)."""
    T, H = 32, 64
    g = torch.Generator().manual_seed(5)
    X = torch.zeros(T, H, dtype=DT[x])
    X[torch.arange(T), torch.randperm(H, generator=g)[:T]] = (torch.rand(T, generator=g) * 3 + 1).to(DT[x])
    w1, w2 = Weight(2, H, 32, False, "f16", 6), Weight(H, 1, 32, False, "f16", 7)
    R = torch.ones(1, H)
    Y, ids, p = layer(ctx, X.cuda(), R.cuda(), w1, w2, 1, 1, 1, "f32")
    gate, up = (X.double() @ w1.values.t()).unbind(1)
    want = (gate / (1 + torch.exp(-gate)) * up)[:, None] * w2.values[:, 0]
    within(Y.cpu(), want, 2.0 ** -20 * want.abs())
    assert bool((want != 0).any()) and p.cpu().tolist() == [[1.0]] * T


def test_ties_go_to_the_lowest_index(ctx):
    T, H, I, E, k = 3, 64, 32, 70, 5
    X, R, w1, w2 = problem(T, H, I, E, k)
    R[:] = 0
    R[40] = R[33] = X[0].float() * 0.01                    # two equal ones on top for token 0
    out = layer(ctx, X.cuda(), R.cuda(), w1, w2, I, E, k)
    assert out[1][0].tolist() == [33, 40, 0, 1, 2]
    check(*out, X, R, w1, w2, I, k, "f32", True)


def test_all_tokens_to_one_expert_and_none_to_others(ctx):
    T, H, I, E, k = 32, 128, 72, 20, 2
    X, R, w1, w2 = problem(T, H, I, E, k)
    X = X.abs()
    R[:] = R.abs() * 1e-3
    R[7], R[19] = 0.05, 0.04                               # two experts take every token
    out = layer(ctx, X.cuda(), R.cuda(), w1, w2, I, E, k)
    assert (out[1].cpu() == torch.tensor([7, 19], dtype=torch.int32)).all()
    check(*out, X, R, w1, w2, I, k, "f32", True)


def test_not_finite(ctx):
    """A token whose activations hold a NaN, or whose logits overflow, gets
    distinct experts in range and no finite output; the other tokens are as
    they would be without it."""
    T, H, I, E, k = 4, 96, 40, 10, 3
    X, R, w1, w2 = problem(T, H, I, E, k)
    base = layer(ctx, X.cuda(), R.cuda(), w1, w2, I, E, k)
    bad = X.clone()
    bad[1, 3] = float("nan")
    bad[2] = 3e38
    out = layer(ctx, bad.cuda(), R.cuda(), w1, w2, I, E, k)
    for t in range(T):
        ids = out[1][t].tolist()
        assert len(set(ids)) == k and min(ids) >= 0 and max(ids) < E
    assert out[1][1].tolist() == [0, 1, 2]                 # every logit NaN: a tie
    assert torch.isnan(out[0][1]).all() and not torch.isfinite(out[0][2]).any()
    for t in (0, 3):
        assert torch.equal(out[0][t], base[0][t]) and torch.equal(out[1][t], base[1][t])


def test_large_activations_stay_finite(ctx):
    """h far above the largest f16: it is not rounded to the activations' type."""
    T, H, I, E, k = 3, 128, 64, 4, 2
    X, R, w1, w2 = problem(T, H, I, E, k, x="f16", r="f16")
    X = (X.float() * 2000).to(torch.float16)
    R = (R.float() * 1e-3).to(torch.float16)
    out = layer(ctx, X.cuda(), R.cuda(), w1, w2, I, E, k)
    assert float(out[0].abs().max()) > 65504
    check(*out, X, R, w1, w2, I, k, "f32", True)


def test_strides_and_optional_outputs(ctx):
    T, H, I, E, k = 5, 200, 48, 7, 2
    X, R, w1, w2 = problem(T, H, I, E, k, ldw=256, lds=up_to(max(7 * 96, 7 * 200), 16) + 16)
    Xb = torch.full((T * (H + 3) + 1,), float("nan"), dtype=torch.bfloat16, device="cuda")
    Xv = Xb[1:].view(T, H + 3)[:, :H]
    Xv.copy_(X)
    Rb = torch.full((E, H + 5), float("nan"), device="cuda")
    Rb[:, :H] = R.cuda()
    Yb = torch.full((T * (H + 1) + 1,), 5.0, dtype=torch.bfloat16, device="cuda")
    Yv = Yb[1:].view(T, H + 1)[:, :H]
    d = tg.make_moe_desc(T, H, I, E, k, "bf16", "bf16", ldx=H + 3, ld_router=H + 5, ldy=H + 1)
    torch.cuda.synchronize()
    tg.tc_moe_q4(ctx, d, Xv, Rb[:, :H], w1.cuda(tg), w2.cuda(tg), Yv)
    want = layer(ctx, X.cuda(), R.cuda(), w1, w2, I, E, k, "bf16")
    assert torch.equal(Yv, want[0])
    assert float(Yb[0]) == 5.0 and (Yb[1:].view(T, H + 1)[:, H] == 5.0).all()


def up_to(x, m):
    return (x + m - 1) // m * m


def test_deterministic_on_two_streams(ctx):
    """Repeated calls give the same bits, also while another stream's calls
    run beside them in workspaces of their own."""
    T, H, I, E, k = 6, 1024, 512, 16, 4
    a, b = problem(T, H, I, E, k), problem(T, H, I, E, k, seed=9)
    sides = [tg.Stream(ctx), tg.Stream(ctx)]
    calls = []
    for (X, R, w1, w2), s in zip((a, b), sides):
        Y = torch.zeros(T, H, device="cuda")
        d = tg.make_moe_desc(T, H, I, E, k, "bf16", "f32")
        calls.append((tg.PreparedMoe(ctx, d, X.cuda(), R.cuda(), w1.cuda(tg), w2.cuda(tg), Y, s), Y))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, _y in calls:
            c.enqueue()
    for s in sides:
        s.sync()
    for (X, R, w1, w2), (_c, Y) in zip((a, b), calls):
        assert torch.equal(Y, layer(ctx, X.cuda(), R.cuda(), w1, w2, I, E, k)[0])
    for s in sides:
        s.close()


def test_refusals_launch_nothing(ctx):
    T, H, I, E, k = 2, 64, 32, 4, 2
    X, R, w1, w2 = problem(T, H, I, E, k)
    q1, q2 = w1.cuda(tg), w2.cuda(tg)
    Xc, Rc = X.cuda(), R.cuda()
    Y = torch.zeros(T, H, device="cuda")
    before = ctx.launch_count
    for args, want in [((T, H, I, E, 5), tg.TC_ERR_DIM), ((T, H, I + 1, E, k), tg.TC_ERR_DIM)]:
        with pytest.raises(tg.TcError) as err:
            tg.tc_moe_q4(ctx, tg.make_moe_desc(*args, "bf16", "f32"), Xc, Rc, q1, q2, Y)
        assert err.value.status == want
    d = tg.make_moe_desc(T, H, I, E, k, "bf16", "f32")
    with pytest.raises(ValueError):
        tg.tc_moe_q4(ctx, d, Xc[:1].clone(), Rc, q1, q2, Y)
    with pytest.raises(ValueError):
        tg.tc_moe_q4(ctx, d, Xc, Rc, q1, q2, Y, torch.zeros(T, k, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        tg.PreparedMoe(ctx, d, Xc, Rc, q1, q2, Y).enqueue()
    assert ctx.launch_count == before
