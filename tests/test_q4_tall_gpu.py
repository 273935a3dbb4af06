"""The streaming 4-bit product in blocks of 32 rows, which calls of at most 8
rows take where a CTA has more than 16 rows of W and K has more than 8 slabs
of 256: reached here with few CTAs, so that small weights have long ranges."""
from __future__ import annotations

import pytest
import torch

from q4_ref import DT, Weight, ulp, unit, up, within

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


# M, N, K, CTAs: ranges of 75 rows in blocks of 32, 32, 11; one block of 20; 33
# (the second block one row); 6 blocks in two phases, the last CTA short; two
# and three slabs to a warp
SHAPES = [(8, 300, 2304, 4, "b3x32"), (1, 100, 2999, 5, "b1x20"), (5, 330, 4096, 10, "b2x32"), (3, 499, 2100, 3, "b6x32"),
          (8, 300, 5000, 4, "b3x32"), (2, 77, 9001, 2, "b2x32")]


def run(ctx, monkeypatch, w, X, c, grid, alpha=1.0, beta=0.0, C=None):
    M = X.shape[0]
    monkeypatch.setenv("TC_FORCE_VARIANT", f"gemv_ks=1 gemv_grid={grid}")
    x = {torch.float16: "f16", torch.bfloat16: "bf16"}[X.dtype]
    C = torch.full((M, w.N), float("nan"), dtype=DT[c], device="cuda") if C is None else C
    d = tg.make_desc(M, w.N, w.K, x, c, b_dtype="i4", transpose_b=True, alpha=alpha, beta=beta,
                     lda=X.stride(0) if M > 1 else 0, ldc=C.stride(0) if M > 1 else 0)
    q = w.cuda(tg)
    torch.cuda.synchronize()
    tg.tc_gemm_q4_weight(ctx, d, X, q, C)
    return C


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("x,c", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
def test_product(ctx, monkeypatch, shape, x, c, group, zeros):
    M, N, K, grid, name = shape
    w = Weight(N, K, group, zeros, "f16" if x == "bf16" else "bf16", seed=M + N)
    g = torch.Generator().manual_seed(K)
    X = (torch.randn(M, K, generator=g) * torch.where(torch.rand(K, generator=g) < 0.05, 20.0, 1.0)).to(DT[x])
    old = torch.rand(M, N, generator=g).to(DT[c])
    out = run(ctx, monkeypatch, w, X.cuda(), c, grid, 0.75, -0.5, old.cuda()).cpu()
    assert ctx.last_kernel.endswith(name), ctx.last_kernel
    xd = X.double()
    want = 0.75 * (xd @ w.values.t()) - 0.5 * old.double()
    T = 0.75 * (xd.abs() @ w.values.abs().t()) + 0.5 * old.double()
    within(out, want, unit(K) * T + (ulp(want, c) if c != "f32" else 0), ctx.last_kernel)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("x", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_whole_numbers_bit_for_bit(ctx, monkeypatch, shape, x, group):
    M, N, K, grid, name = shape
    w = Weight(N, K, group, True, seed=M + N, kind="pow2")
    X = torch.randint(-4, 5, (M, K), generator=torch.Generator().manual_seed(M)).to(DT[x])
    out = run(ctx, monkeypatch, w, X.cuda(), "f32", grid)
    assert ctx.last_kernel.endswith(name), ctx.last_kernel
    want = X.double() @ w.values.t()
    assert float(want.abs().max()) * 4 < 2 ** 24
    assert torch.equal(out.cpu().double(), want)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("pad", [1, 2, 8])
def test_strides_and_alignment(ctx, monkeypatch, shape, pad):
    """Padded rows of every tensor, X and C off any alignment."""
    M, N, K, grid, name = shape
    w = Weight(N, K, 32, True, "bf16", seed=K, ldw=up(K, 32) + 64, lds=up(N, 16) + 32)
    X = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).to(torch.float16)
    buf = torch.full((M * (K + pad) + 1,), float("nan"), dtype=torch.float16, device="cuda")
    Xv = buf[1:].view(M, K + pad)[:, :K]
    Xv.copy_(X)
    cbuf = torch.full((M * (N + pad) + 1,), 5.0, dtype=torch.float16, device="cuda")
    Cv = cbuf[1:].view(M, N + pad)[:, :N]
    run(ctx, monkeypatch, w, Xv, "f16", grid, C=Cv)
    assert ctx.last_kernel.endswith(name), ctx.last_kernel
    x = X.double()
    want = x @ w.values.t()
    within(Cv.cpu(), want, unit(K) * (x.abs() @ w.values.abs().t()) + ulp(want, "f16"), ctx.last_kernel)
    assert float(cbuf[0]) == 5.0 and (cbuf[1:].view(M, N + pad)[:, N:] == 5.0).all()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("group", [32, 128])
def test_not_finite(ctx, monkeypatch, shape, group):
    """A NaN or an infinity stays in its row of X or its row of W; C's old NaN
    is not read when beta is 0."""
    M, N, K, grid, name = shape
    w = Weight(N, K, group, False, seed=M)
    w.scales[2, 13], w.scales[1, N - 1] = float("inf"), float("nan")
    X = torch.randn(M, K, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    clean = torch.ones(M, N, dtype=torch.bool)
    clean[:, 13] = clean[:, N - 1] = False
    if M > 1:
        X[M - 1, 7], X[0, K - 1] = float("nan"), float("inf")
        clean[M - 1] = clean[0] = False
    out = run(ctx, monkeypatch, w, X.cuda(), "f32", grid).cpu()
    assert ctx.last_kernel.endswith(name), ctx.last_kernel
    assert not torch.isfinite(out[:, 13]).any() and torch.isnan(out[:, N - 1]).all()
    if M > 1:
        assert torch.isnan(out[M - 1]).all() and not torch.isfinite(out[0]).all()
    x = torch.where(torch.isfinite(X), X, 0).double()
    v = torch.where(torch.isfinite(w.scales.double())[:, :N].t().repeat_interleave(group, 1)[:, :K],
                    w.values, torch.zeros((), dtype=torch.float64))
    T = x.abs() @ v.abs().t()
    # a row of X that is clean: its sums are those of the finite weights
    assert ((out.double() - x @ v.t()).abs() <= unit(K) * T)[clean].all()


@pytest.mark.parametrize("M,N,K", [(1, 5000, 2304), (8, 4099, 4096), (4, 9001, 5001)])
def test_as_planned(ctx, M, N, K):
    """The same without any forcing, on weights that have such ranges."""
    w = Weight(N, K, 32, True, "f16", seed=M, kind="pow2")
    X = torch.randint(-2, 3, (M, K), generator=torch.Generator().manual_seed(M)).to(torch.float16)
    C = torch.full((M, N), float("nan"), device="cuda")
    Xc, q = X.cuda(), w.cuda(tg)
    torch.cuda.synchronize()
    tg.tc_gemm_q4_weight(ctx, tg.make_desc(M, N, K, "f16", "f32", b_dtype="i4", transpose_b=True), Xc, q, C)
    block = int(ctx.last_kernel.rsplit("x", 1)[1])
    assert 16 < block <= 32, ctx.last_kernel
    assert torch.equal(C.cpu().double(), X.double() @ w.values.t())
