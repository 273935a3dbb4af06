"""The 4-bit weight operators on GB300 against their 64-bit forms: quantising
(bit for bit), giving values back (bit for bit), and the product."""
from __future__ import annotations

import pytest
import torch

import q4_ref
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


# ------------------------------------------------------------------ quantise

QSHAPES = [(1, 1, 32), (3, 31, 32), (17, 33, 32), (5, 64, 64), (33, 100, 64), (16, 127, 128), (7, 129, 128),
           (100, 1000, 32), (257, 2999, 64), (130, 4096, 128), (4099, 96, 32)]


@pytest.mark.parametrize("shape", QSHAPES)
@pytest.mark.parametrize("w", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("zeros", [False, True])
def test_quantise_bits(ctx, shape, w, zeros):
    N, K, group = shape
    scale = "bf16" if (N + K) % 2 else "f16"
    g = torch.Generator().manual_seed(N * K)
    pad = N % 3                                            # rows off any alignment
    full = (torch.randn(N, K + pad, generator=g) * 0.05).to(DT[w])
    if K > 64:
        full[0, :64] = 0                                   # a group of zeros
        full[-1, 1:64] = full[-1, 1:64].abs()              # one sign only
    W = full[:, :K]
    code, s, z = q4_ref.quantise(W, group, zeros, scale)
    q = tg.Q4Weight.empty(N, K, group, scale_dtype=DT[scale], zeros=zeros)
    for t in (q.codes, q.scales, q.zeros):
        if t is not None:
            t.fill_(77)
    dev = full.cuda()
    torch.cuda.synchronize()                               # the library's stream does not wait for torch's
    tg.tc_quantize_q4(ctx, dev[:, :K], q)
    assert torch.equal(q.scales.cpu()[:, :N].view(torch.int16), s.contiguous().view(torch.int16))
    if zeros:
        assert torch.equal(q.zeros.cpu()[:, :N].float(), z)
    got = q4_ref.unpack(q.codes.cpu(), up(K, 32)).float()
    assert torch.equal(got[:, :K], code[:, :K])
    # what lies past K stands for 0 where its group exists
    kp = min(up(K, 32), -(-K // group) * group)
    zz = q4_ref.spread(z if zeros else torch.full_like(s.float(), 8.0), N, kp, group)
    assert torch.equal(got[:, K:kp], zz[:, K:kp])
    # padding columns of the scales are left alone
    assert (q.scales.cpu()[:, N:].float() == 77).all()
    # values: the fp32 product, rounded once; within half a step of the weight
    for v in ("f32", "f16", "bf16"):
        V = torch.full((N, K + 3), 9.0, dtype=DT[v], device="cuda")
        torch.cuda.synchronize()
        tg.tc_dequantize_q4(ctx, q, V[:, :K])
        step = q4_ref.spread(s.float(), N, K, group)
        want = (code[:, :K] - zz[:, :K]) * step
        assert torch.equal(V.cpu()[:, :K], want.to(DT[v]))
        assert (V[:, K:] == 9.0).all()
    # half a step, and what the scale's own rounding (2^-8, or a subnormal f16
    # step 2^-25) leaves beyond the last code
    lim = step.double() * 0.5 + 15 * torch.maximum(step.double() * 2.0 ** -8, torch.tensor(2.0 ** -25).double())
    if zeros:
        lim = lim + step.double() * 0.5                   # the zero point is rounded too
    assert ((want.double() - W.double()).abs() <= lim).all()


def test_quantise_not_finite_and_extremes(ctx):
    """A group with a NaN or an infinity reads back as no finite number; its
    neighbours are untouched; tiny groups read back as 0."""
    for zeros in (False, True):
        W = torch.randn(4, 128) * 0.1
        W[0, 5], W[1, 40], W[2, 70] = float("nan"), float("inf"), -float("inf")
        W[3, :32] = 1e-12                                  # its scale is 0 in f16
        W[3, 32:64] = 1e7                                  # its scale is infinite in f16
        q = tg.Q4Weight.empty(4, 128, 32, zeros=zeros)
        tg.tc_quantize_q4(ctx, W.cuda(), q)
        V = torch.empty(4, 128, device="cuda")
        tg.tc_dequantize_q4(ctx, q, V)
        V = V.cpu()
        for r, gr in ((0, 0), (1, 1), (2, 2), (3, 1)):
            assert not torch.isfinite(V[r, 32 * gr: 32 * gr + 32]).any()
        assert (V[3, :32] == 0).all()
        fine = torch.isfinite(V)
        assert int(fine.sum()) == 4 * 128 - 4 * 32


# ------------------------------------------------------------------- product

def run(ctx, X, w, c, alpha=1.0, beta=0.0, C=None, q=None, stream=None, M=None):
    q = q or w.cuda(tg)
    M = X.shape[0]
    C = torch.full((M, w.N), float("nan"), dtype=DT[c], device="cuda") if C is None else C
    x = {torch.float16: "f16", torch.bfloat16: "bf16"}[X.dtype]
    d = tg.make_desc(M, w.N, w.K, x, c, b_dtype="i4", transpose_b=True, alpha=alpha, beta=beta,
                     lda=X.stride(0) if M > 1 else 0, ldc=C.stride(0) if M > 1 else 0)
    torch.cuda.synchronize()                               # the library's stream does not wait for torch's
    if stream is None:
        tg.tc_gemm_q4_weight(ctx, d, X, q, C)
    else:
        tg.tc_gemm_q4_weight_async(ctx, d, X, q, C, stream)
        stream.sync()
    return C


def check(out, X, w, c, alpha=1.0, beta=0.0, old=None, what=""):
    x = X.cpu().double()
    want, T = alpha * (x @ w.values.t()), abs(alpha) * (x.abs() @ w.values.abs().t())
    if beta:
        want, T = want + beta * old.double(), T + abs(beta) * old.double().abs()
    b = unit(w.K) * T + (ulp(want, c) if c != "f32" else 0)
    within(out.cpu(), want, b, what)


SHAPES = [(1, 1, 1), (1, 16, 32), (1, 1000, 77), (2, 17, 4096), (3, 24, 255), (4, 300, 2999), (5, 8, 257),
          (7, 129, 1000), (8, 1000, 64), (9, 33, 100), (12, 4099, 130), (16, 513, 2049), (16, 64, 11008),
          (17, 300, 700), (31, 1001, 129), (40, 260, 1500), (64, 128, 128), (65, 127, 255), (129, 200, 333),
          (200, 1001, 515), (300, 640, 1024)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("x,c", [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True), (128, False), (32, False), (64, True)])
def test_product(ctx, shape, x, c, group, zeros):
    M, N, K = shape
    w = Weight(N, K, group, zeros, "f16" if x == "bf16" else "bf16", seed=M + 3 * N + K)
    g = torch.Generator().manual_seed(K)
    X = (torch.randn(M, K, generator=g) * torch.where(torch.rand(K, generator=g) < 0.05, 20.0, 1.0)).to(DT[x])
    old = torch.rand(M, N, generator=g).to(DT[c])
    out = run(ctx, X.cuda(), w, c, 0.75, -0.5, C=old.cuda())
    check(out, X, w, c, 0.75, -0.5, old, f"{shape} {x}->{c} g{group} {ctx.last_kernel}")


@pytest.mark.parametrize("M", [1, 2, 3, 4, 7, 8, 9, 15, 16, 17, 24, 32, 33, 48, 64, 65, 100, 128, 129, 256, 257])
@pytest.mark.parametrize("x", ["f16", "bf16"])
def test_whole_numbers_bit_for_bit(ctx, M, x):
    """Whole activations and scales that are powers of two: every partial sum
    is exact in fp32, so any order of the sums gives the same bits."""
    for N, K, group, zeros in [(1000, 4096, 32, True), (40, 515, 64, False), (300, 1000, 128, True)]:
        w = Weight(N, K, group, zeros, seed=M + N, kind="pow2")
        X = torch.randint(-4, 5, (M, K), generator=torch.Generator().manual_seed(M)).to(DT[x])
        out = run(ctx, X.cuda(), w, "f32")
        assert torch.equal(out.cpu().double(), X.double() @ w.values.t()), (M, N, K, ctx.last_kernel)


@pytest.mark.parametrize("shape", [(3, 100, 40000), (16, 33, 33000), (4, 20000, 5000), (9, 9001, 9000), (3, 130001, 256),
                                   (2, 70000, 700), (16, 40000, 1030), (17, 100, 40000), (33, 3001, 9000), (1, 5, 100000)])
def test_long_axes(ctx, shape):
    """K beyond one slab per warp and one cluster, more blocks of rows than are
    held at once, K slices on the tensor cores."""
    M, N, K = shape
    w = Weight(N, K, 64, True, "f16", seed=N, kind="pow2")
    X = torch.randint(-2, 3, (M, K), generator=torch.Generator().manual_seed(M)).to(torch.bfloat16)
    out = run(ctx, X.cuda(), w, "f32")
    want = X.double() @ w.values.t()
    assert float(want.abs().max()) * 4 < 2 ** 24           # exact: quarter steps below 2^22
    assert torch.equal(out.cpu().double(), want), ctx.last_kernel


@pytest.mark.parametrize("M", [1, 6, 16, 40, 200])
def test_strides_and_alignment(ctx, M):
    """Padded rows of every tensor, X and C off any alignment."""
    for N, K, pad in [(301, 999, 1), (48, 640, 8), (77, 1001, 3)]:
        w = Weight(N, K, 64, True, "bf16", seed=K, ldw=up(K, 32) + 64, lds=up(N, 16) + 32)
        X = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).to(torch.float16)
        buf = torch.full((M * (K + pad) + 1,), float("nan"), dtype=torch.float16, device="cuda")
        Xv = buf[1:].view(M, K + pad)[:, :K]
        Xv.copy_(X)
        cbuf = torch.full((M * (N + pad) + 1,), 5.0, dtype=torch.float16, device="cuda")
        Cv = cbuf[1:].view(M, N + pad)[:, :N]
        run(ctx, Xv, w, "f16", C=Cv)
        check(Cv, X, w, "f16", what=f"{M}x{N}x{K} {ctx.last_kernel}")
        rest = cbuf[1:].view(M, N + pad)[:, N:]
        assert float(cbuf[0]) == 5.0 and (rest == 5.0).all()


@pytest.mark.parametrize("M", [1, 5, 16, 33, 130])
def test_not_finite(ctx, M):
    """A NaN or infinity in one row of X, or in one row's scale, stays in its
    row or column; C's old NaN is not read when beta is 0."""
    N, K = 70, 300
    w = Weight(N, K, 64, False, seed=M)
    w.scales[2, 13] = float("inf")
    X = torch.randn(M, K, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    clean = torch.ones(M, N, dtype=torch.bool)
    clean[:, 13] = False
    if M > 1:
        X[M - 1, 7], X[0, K - 1] = float("nan"), float("inf")
        clean[M - 1] = clean[0] = False
    out = run(ctx, X.cuda(), w, "f32").cpu()
    assert torch.isfinite(out[clean]).all()
    assert not torch.isfinite(out[:, 13]).any()
    if M > 1:
        assert torch.isnan(out[M - 1]).all()
        assert not torch.isfinite(out[0]).all()
    want = (torch.where(torch.isfinite(X), X, 0).double() @ torch.where(torch.isfinite(w.values), w.values, 0.0).t())
    T = torch.where(torch.isfinite(X), X, 0).double().abs() @ torch.where(torch.isfinite(w.values), w.values, 0.0).abs().t()
    assert ((out.double() - want).abs() <= unit(K) * T)[clean].all()


@pytest.mark.parametrize("M,N,K", [(150, 1300, 9000), (66, 5000, 2900), (290, 6000, 700), (1200, 5000, 400), (130, 130, 40000)])
def test_cut_tiles(ctx, monkeypatch, M, N, K):
    """Tiles cut along K where a range of work ends: exact sums, so any cut
    gives the same bits; then sums that round, the same in every run."""
    monkeypatch.setenv("TC_FORCE_VARIANT", "bn=128 tail=1")
    w = Weight(N, K, 64, True, "f16", seed=N, kind="pow2")
    X = torch.randint(-2, 3, (M, K), generator=torch.Generator().manual_seed(M)).to(torch.bfloat16)
    out = run(ctx, X.cuda(), w, "f32")
    assert ctx.last_kernel.endswith("_cut")
    want = X.double() @ w.values.t()
    assert float(want.abs().max()) * 4 < 2 ** 24
    assert torch.equal(out.cpu().double(), want), ctx.last_kernel
    old = torch.rand(M, N, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    X = torch.randn(M, K, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    q, Xc = w.cuda(tg), X.cuda()
    outs = [run(ctx, Xc, w, "bf16", 0.75, -0.5, C=old.cuda(), q=q) for _ in range(3)]
    assert torch.equal(outs[1], outs[0]) and torch.equal(outs[2], outs[0])
    check(outs[0], X, w, "bf16", 0.75, -0.5, old, ctx.last_kernel)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (4, 4096, 11008), (16, 11008, 4096), (200, 4096, 4096)])
def test_deterministic_and_async(ctx, M, N, K):
    w = Weight(N, K, 128, True, seed=71)
    X = torch.randn(M, K, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    q = w.cuda(tg)
    outs = [run(ctx, X, w, "f32", q=q).clone() for _ in range(4)]
    stream = tg.Stream(ctx)
    torch.cuda.synchronize()
    outs.append(run(ctx, X, w, "f32", q=q, stream=stream))
    stream.close()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    check(outs[0], X, w, "f32")


def test_back_to_back_chain(ctx):
    """Products that consume each other's outputs on one stream without waiting."""
    w = [Weight(512, 512, 32, False, seed=i, std=0.05) for i in range(2)]
    q = [v.cuda(tg) for v in w]
    X = torch.randn(3, 512, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    side = torch.cuda.Stream()
    bufs = [X.cuda(), torch.zeros(3, 512, dtype=torch.bfloat16, device="cuda")]
    torch.cuda.synchronize()
    stream = tg.Stream(ctx, side)
    d = tg.make_desc(3, 512, 512, "bf16", "bf16", b_dtype="i4", transpose_b=True)
    calls = [tg.PreparedGemm(ctx, d, bufs[0], q[0], bufs[1], stream), tg.PreparedGemm(ctx, d, bufs[1], q[1], bufs[0], stream)]
    for _ in range(10):
        calls[0].enqueue()
        calls[1].enqueue()
    stream.sync()
    y = X.cuda()
    for _ in range(10):
        for v, qq in zip(w, q):
            y = run(ctx, y, v, "bf16", q=qq)
    assert torch.equal(bufs[0], y)
    stream.close()


def test_past_32_bits(ctx):
    """Rows of codes, of X and of C that start past 2^32 bytes."""
    N, K = 300_000, 32768
    free, _ = torch.cuda.mem_get_info()
    if free < 30 << 30:
        pytest.skip("needs 30 GB of free device memory")
    codes = torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda")
    w = Weight(32, K, 128, False, seed=5)
    codes[-32:] = w.codes.cuda()
    scales = torch.zeros(K // 128, up(N, 16), dtype=torch.float16, device="cuda")
    scales[:, N - 32:N] = w.scales[:, :32].cuda()
    q = tg.Q4Weight(N, K, 128, codes, scales)
    for M in (3, 20):
        ldc = (2 ** 32 // 4 + 4096) // (M - 1) // 8 * 8 + 8
        cbuf = torch.empty((M - 1) * ldc + N, dtype=torch.float32, device="cuda")
        C = torch.as_strided(cbuf, (M, N), (ldc, 1))
        ldx = (2 ** 32 // 2 + 4096) // (M - 1) // 8 * 8 + 8
        xbuf = torch.zeros((M - 1) * ldx + K, dtype=torch.float16, device="cuda")
        X = torch.as_strided(xbuf, (M, K), (ldx, 1))
        X.copy_(torch.randn(M, K, generator=torch.Generator().manual_seed(M)).to(torch.float16))
        d = tg.make_desc(M, N, K, "f16", "f32", b_dtype="i4", transpose_b=True, lda=ldx, ldc=ldc)
        torch.cuda.synchronize()
        tg.tc_gemm_q4_weight(ctx, d, X, q, C)
        check(C[:, -32:].contiguous(), X, w, "f32", what=f"M={M} {ctx.last_kernel}")
        assert (C[:, : N - 32] == 0).all()
        del C, cbuf, X, xbuf


def test_refusals_launch_nothing(ctx):
    w = Weight(64, 96, 32, False)
    q = w.cuda(tg)
    X = torch.zeros(4, 96, dtype=torch.float16, device="cuda")
    C = torch.zeros(4, 64, dtype=torch.float16, device="cuda")
    before = ctx.launch_count
    for kw, want in [({"transpose_b": False}, tg.TC_ERR_LAYOUT), ({"b_dtype": "i8"}, tg.TC_ERR_DTYPE),
                     ({"ldb": 64}, tg.TC_ERR_LD)]:
        d = tg.make_desc(4, 64, 96, "f16", "f16", **{"b_dtype": "i4", "transpose_b": True, **kw})
        with pytest.raises(tg.TcError) as err:
            tg.tc_gemm_q4_weight(ctx, d, X, q, C)
        assert err.value.status == want
    d = tg.make_desc(4, 64, 96, "f16", "f16", b_dtype="i4", transpose_b=True)
    with pytest.raises(ValueError):
        tg.tc_gemm_q4_weight(ctx, d, X[:3].clone(), q, C)
    with pytest.raises(ValueError):
        tg.tc_gemm_q4_weight(ctx, d, X, q, C[:3].clone())
    with pytest.raises(ValueError):
        tg.tc_quantize_q4(ctx, X, q)
    with pytest.raises(ValueError):
        tg.Q4Weight(65, 96, 32, q.codes, q.scales)
    with pytest.raises(ValueError):
        tg.Q4Weight(64, 128, 32, q.codes, q.scales)
    assert ctx.launch_count == before


def test_quantised_weight_multiplies(ctx):
    """Quantise, multiply and compare with the product of the values read back."""
    N, K, M = 384, 1100, 9
    W = (torch.randn(N, K, generator=torch.Generator().manual_seed(8)) * 0.05).to(torch.bfloat16).cuda()
    X = torch.randn(M, K, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).cuda()
    torch.cuda.synchronize()
    for zeros in (False, True):
        q = tg.Q4Weight.empty(N, K, 64, zeros=zeros)
        tg.tc_quantize_q4(ctx, W, q)
        V = torch.empty(N, K, device="cuda")
        tg.tc_dequantize_q4(ctx, q, V)
        C = torch.empty(M, N, device="cuda")
        d = tg.make_desc(M, N, K, "bf16", "f32", b_dtype="i4", transpose_b=True)
        tg.tc_gemm_q4_weight(ctx, d, X, q, C)
        v, x = V.double().cpu(), X.double().cpu()
        within(C.cpu(), x @ v.t(), unit(K) * (x.abs() @ v.abs().t()))
