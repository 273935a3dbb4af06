"""Large and small bf16 activations through the 4-bit operators: bf16 reaches
as far as fp32, so a group's sum of products with codes must neither overflow
before its scale brings it down nor vanish."""
from __future__ import annotations

import pytest
import torch

import q4_ref
from q4_ref import Weight, unit, within

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


def scaled(w, e):
    """w with its scales times 2^e."""
    w.scales = (w.scales.double() * 2.0 ** e).to(w.scales.dtype)
    w.values = w.values * 2.0 ** e
    return w


def product(ctx, X, w):
    M = X.shape[0]
    C = torch.full((M, w.N), float("nan"), device="cuda")
    d = tg.make_desc(M, w.N, w.K, "bf16", "f32", b_dtype="i4", transpose_b=True)
    Xc, q = X.cuda(), w.cuda(tg)
    torch.cuda.synchronize()
    tg.tc_gemm_q4_weight(ctx, d, Xc, q, C)
    return C.cpu()


# streaming (16- and 32-row blocks, a cluster), tensor cores whole, in a
# cluster and cut
PLANS = [(1, 300, 700, ""), (3, 5000, 2304, ""), (12, 300, 4096, ""), (3, 300, 9000, ""), (40, 300, 700, ""),
         (100, 300, 4096, "bn=64 split=4"), (150, 1300, 2304, "bn=128 tail=1")]


@pytest.mark.parametrize("M,N,K,spec", PLANS)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_products_of_large_activations(ctx, monkeypatch, M, N, K, spec, group):
    """Whole numbers up to 4 times 2^125 (bf16's largest is below 2^128), all
    of one sign in the first row: sums of a group reach 2^135 and more, results
    stay below 2^24 and exact."""
    if spec:
        monkeypatch.setenv("TC_FORCE_VARIANT", spec)
    w = Weight(N, K, group, True, "bf16", seed=N + group, kind="pow2")
    X = torch.randint(-4, 5, (M, K), generator=torch.Generator().manual_seed(M)).double()
    X[0] = X[0].abs()
    want = X @ w.values.t()
    assert float(want.abs().max()) * 4 < 2 ** 24
    out = product(ctx, (X * 2.0 ** 125).to(torch.bfloat16), scaled(w, -121))
    assert torch.equal(out.double(), want * 2.0 ** 4), ctx.last_kernel


@pytest.mark.parametrize("M,N,K,spec", PLANS)
def test_products_of_the_largest_activations(ctx, monkeypatch, M, N, K, spec):
    """Every activation bf16's largest, every code 15 from its zero point."""
    if spec:
        monkeypatch.setenv("TC_FORCE_VARIANT", spec)
    w = Weight(N, K, 128, True, "bf16", seed=1)
    w.codes.fill_(255)
    w.zeros.zero_()
    w.values = 15.0 * q4_ref.spread(w.scales.double(), N, K, 128)
    w = scaled(w, -30)
    X = torch.full((M, K), torch.finfo(torch.bfloat16).max, dtype=torch.bfloat16)
    want = X.double() @ w.values.t()
    assert torch.isfinite(want.float()).all()
    within(product(ctx, X, w), want, unit(K) * want, ctx.last_kernel)


@pytest.mark.parametrize("M,N,K,spec", PLANS)
def test_products_of_small_activations(ctx, monkeypatch, M, N, K, spec):
    """Near 2^-115 results keep fp32's relative bound; below, 2^-137 per
    group's sum."""
    if spec:
        monkeypatch.setenv("TC_FORCE_VARIANT", spec)
    w = Weight(N, K, 64, True, "f16", seed=2, kind="pow2")
    X = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).to(torch.bfloat16)
    for e in (-100, -124):
        x = (X.double() * 2.0 ** e).to(torch.bfloat16)
        want, T = x.double() @ w.values.t(), x.double().abs() @ w.values.abs().t()
        within(product(ctx, x, w), want, unit(K) * T + (K / 64 + 1) * 2.0 ** -137, ctx.last_kernel)


@pytest.mark.parametrize("T,H,I,E,k", [(1, 512, 96, 8, 2), (9, 300, 72, 4, 2), (32, 256, 64, 4, 2)])
@pytest.mark.parametrize("tall", [0, 1])
@pytest.mark.parametrize("y", ["bf16", "f32"])
def test_layer_of_large_activations(ctx, monkeypatch, T, H, I, E, k, tall, y):
    """x times 2^123 and the router's and gate_up's values times 2^-123: every
    sum is the same to the bit.  Gate and up are near 32, their groups' sums
    near 2^129."""
    monkeypatch.setenv("TC_FORCE_VARIANT", f"tail={tall}")
    g = torch.Generator().manual_seed(T)
    X = torch.randn(T, H, generator=g).clamp(-7, 7).to(torch.bfloat16)
    R = torch.randint(-8, 9, (E, H), generator=g) / 8
    outs = []
    for e in (0, 123):
        w1 = scaled(Weight(E * 2 * I, H, 128, True, "bf16", seed=3, std=32 * H ** -0.5), -e)
        w2 = Weight(E * H, I, 128, True, "bf16", seed=4, std=I ** -0.5)
        assert float(w1.scales[:, : w1.N].double().min()) >= 2.0 ** -126       # normal: no bits lost
        Y = torch.full((T, H), float("nan"), device="cuda", dtype=q4_ref.DT[y])
        d = tg.make_moe_desc(T, H, I, E, k, "bf16", y)
        args = (X.double() * 2.0 ** e).to(torch.bfloat16).cuda(), (R.double() * 2.0 ** -e).float().cuda(), w1.cuda(tg), w2.cuda(tg)
        torch.cuda.synchronize()
        tg.tc_moe_q4(ctx, d, *args, Y)
        outs.append(Y.cpu())
    assert torch.isfinite(outs[0]).all() and torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("x", ["bf16", "f16"])
@pytest.mark.parametrize("y", ["x", "f32"])
def test_layer_with_large_h(ctx, x, y):
    """h near fp32's largest, whatever the activations' type: one expert whose
    down product brings it back."""
    T, H, I = 3, 128, 96
    g = torch.Generator().manual_seed(11)
    X = torch.randn(T, H, generator=g).to(q4_ref.DT[x])
    w1 = scaled(Weight(2 * I, H, 128, True, "bf16", seed=5), 64)    # gate and up near 2^62, h up to 2^127
    w2 = scaled(Weight(H, I, 128, True, "bf16", seed=6), -110)
    d = tg.make_moe_desc(T, H, I, 1, 1, x, "f32" if y == "f32" else x)
    Y = torch.full((T, H), float("nan"), device="cuda", dtype=torch.float32 if y == "f32" else q4_ref.DT[x])
    R = torch.zeros(1, H)
    args = X.cuda(), R.cuda(), w1.cuda(tg), w2.cuda(tg)
    torch.cuda.synchronize()
    tg.tc_moe_q4(ctx, d, *args, Y)
    gate, up = (X.double() @ w1.values.t()).split(I, 1)
    h = gate * torch.sigmoid(gate) * up
    assert 2.0 ** 120 < float(h.abs().max()) < 2.0 ** 127
    want, _ids, _p, b, _dp = q4_ref.moe(X, R, w1, w2, I, 1, True)
    within(Y.cpu(), want, b + (q4_ref.ulp(want, x) if y == "x" else 2.0 ** -23 * want.abs()))
