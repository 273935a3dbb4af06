"""The joining of tiles that the 4-bit product cuts along K, call after call."""
from __future__ import annotations

import pytest
import torch

from q4_ref import Weight

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import matrix_multiply_gb300 as tg
else:  # collected on CPU only to be deselected
    tg = None


@pytest.mark.parametrize("M,N,K", [(200, 11008, 4096), (66, 5000, 2900), (1200, 5000, 400)])
def test_cut_products_back_to_back(monkeypatch, M, N, K):
    """Two activations in turn over one workspace and one set of counts, no
    waiting between the calls: sums that are exact, so a part of another
    call's, or one read too early, would show."""
    monkeypatch.setenv("TC_FORCE_VARIANT", "bn=128 tail=1")
    ctx = tg.Context(0)
    stream = tg.Stream(ctx)
    w = Weight(N, K, 128, True, "f16", seed=K, kind="pow2")
    q = w.cuda(tg)
    xs = [torch.randint(-2, 3, (M, K), generator=torch.Generator().manual_seed(i)).to(torch.bfloat16) for i in range(2)]
    outs = [torch.zeros(M, N, device="cuda") for _ in range(8)]
    d = tg.make_desc(M, N, K, "bf16", "f32", b_dtype="i4", transpose_b=True)
    calls = [tg.PreparedGemm(ctx, d, xs[i % 2].cuda(), q, outs[i], stream) for i in range(8)]
    torch.cuda.synchronize()
    for _ in range(10):
        for c in calls:
            c.enqueue()
    assert ctx.last_kernel.endswith("_cut")
    stream.sync()
    for i in range(2):
        want = xs[i].double() @ w.values.t()
        assert float(want.abs().max()) * 4 < 2 ** 24
        for o in outs[i::2]:
            assert torch.equal(o.cpu().double(), want)
    stream.close()
    ctx.close()
