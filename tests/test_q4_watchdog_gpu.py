"""Every wait of the 4-bit kernels is bounded: a copy that does not complete,
or an arrival that does not come (flags that nothing sets), ends in
TC_ERR_DEVICE_TIMEOUT after a short limit, and the next calls on the same
stream -- which rely on the words such a kernel leaves behind -- are right."""
from __future__ import annotations

import time

import pytest
import torch

from q4_ref import Weight, unit, within

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import matrix_multiply_gb300 as tg
else:  # collected on CPU only to be deselected
    tg = None


@pytest.fixture
def ctx():
    c = tg.Context(0)
    yield c
    c.close()


def expires(monkeypatch, call, spec):
    """The call reports the expired wait, and does so in time: one limit of
    0.2 s, then at most eight of 0.2 s for the copies under way."""
    monkeypatch.setenv("TC_FORCE_VARIANT", f"{spec} debug_timeout_ms=200")
    t0 = time.monotonic()
    with pytest.raises(tg.TcError) as err:
        call()
    assert err.value.status == tg.TC_ERR_DEVICE_TIMEOUT
    assert time.monotonic() - t0 < 3.5
    monkeypatch.delenv("TC_FORCE_VARIANT")
    torch.cuda.synchronize()                               # the device answers


class Product:
    def __init__(self, ctx, M, N, K):
        self.w = Weight(N, K, 64, True, seed=M)
        x = torch.randn(M, K, generator=torch.Generator().manual_seed(N)).to(torch.bfloat16)
        X, self.C, q = x.cuda(), torch.zeros(M, N, device="cuda"), self.w.cuda(tg)
        d = tg.make_desc(M, N, K, "bf16", "f32", b_dtype="i4", transpose_b=True)
        torch.cuda.synchronize()
        self.call = lambda: tg.tc_gemm_q4_weight(ctx, d, X, q, self.C)
        x = x.double()
        self.want, self.bound = x @ self.w.values.t(), unit(K) * (x.abs() @ self.w.values.abs().t())

    def check(self):
        self.C.zero_()
        torch.cuda.synchronize()
        self.call()
        within(self.C.cpu(), self.want, self.bound)


class Layer:
    def __init__(self, ctx, T, H, I, E, k, y):
        g = torch.Generator().manual_seed(T)
        q = [w.cuda(tg) for w in (Weight(E * 2 * I, H, 64, True, seed=1, std=H ** -0.5),
                                  Weight(E * H, I, 64, True, seed=2, std=I ** -0.5))]
        X, R = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda(), torch.randn(E, H, generator=g).cuda()
        self.Y = torch.zeros(T, H, device="cuda", dtype={"f32": torch.float32, "bf16": torch.bfloat16}[y])
        d = tg.make_moe_desc(T, H, I, E, k, "bf16", y)
        torch.cuda.synchronize()
        self.call = lambda: tg.tc_moe_q4(ctx, d, X, R, *q, self.Y)
        other = tg.Context(0)                              # a stream and words of its own
        tg.tc_moe_q4(other, d, X, R, *q, self.Y)
        other.close()
        self.want = self.Y.clone()

    def check(self):
        self.Y.zero_()
        torch.cuda.synchronize()
        self.call()
        assert torch.equal(self.Y, self.want)


@pytest.mark.parametrize("M,N,K,kernel", [(3, 5000, 4096, "b2x32"), (12, 5000, 4096, "gemv_x12"), (3, 512, 11008, "x3_b"),
                                          (2, 300, 9000, "gemv_x2")])
def test_streaming_product(ctx, monkeypatch, M, N, K, kernel):
    p = Product(ctx, M, N, K)
    expires(monkeypatch, p.call, "debug_drop=1")
    assert kernel in ctx.last_kernel, ctx.last_kernel
    p.check()


@pytest.mark.parametrize("M,N,K,spec,kernel", [
    (100, 300, 1024, "bn=64 split=1 tail=0", "128x64_g64_s1"), (300, 20000, 640, "bn=128 split=1 tail=0", "128x128_g64_s1"),
    (100, 300, 4096, "bn=64 split=4", "128x64_g64_s4"), (40, 128, 8192, "bn=32 split=8", "128x32_g64_s8"),
    (200, 11008, 4096, "bn=128 tail=1", "_cut"), (66, 5000, 2900, "bn=128 tail=1", "_cut")])
def test_tensor_core_product(ctx, monkeypatch, M, N, K, spec, kernel):
    p, cut, layer = Product(ctx, M, N, K), Product(ctx, 200, 11008, 4096), Layer(ctx, 3, 256, 96, 8, 2, "f32")
    expires(monkeypatch, p.call, f"{spec} debug_drop=1")
    assert kernel in ctx.last_kernel, ctx.last_kernel
    monkeypatch.setenv("TC_FORCE_VARIANT", spec)
    p.check()
    monkeypatch.delenv("TC_FORCE_VARIANT")
    cut.check()
    assert ctx.last_kernel.endswith("_cut")
    layer.check()
    p.check()


@pytest.mark.parametrize("drop", [1, 2])
@pytest.mark.parametrize("shape,spec", [((8, 512, 200, 16, 4, "f32"), ""), ((8, 512, 200, 16, 4, "bf16"), "tail=1"),
                                        ((1, 2048, 768, 8, 4, "bf16"), "")])
def test_layer(ctx, monkeypatch, drop, shape, spec):
    layer, cut = Layer(ctx, *shape), Product(ctx, 200, 11008, 4096)
    if spec:                                               # the same pieces throughout
        monkeypatch.setenv("TC_FORCE_VARIANT", spec)
        layer.call()
        layer.want = layer.Y.clone()
    expires(monkeypatch, layer.call, f"{spec} debug_drop={drop}")
    if spec:
        monkeypatch.setenv("TC_FORCE_VARIANT", spec)
    for _ in range(3):
        layer.check()
    monkeypatch.delenv("TC_FORCE_VARIANT", raising=False)
    cut.check()
    assert ctx.last_kernel.endswith("_cut")
