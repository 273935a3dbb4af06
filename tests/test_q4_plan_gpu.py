"""The 4-bit product's split of K over clusters: as many slices as leave every
tile's cluster resident at once."""
from __future__ import annotations

import pytest
import torch

from q4_ref import Weight, unit, within

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import matrix_multiply_gb300 as tg
else:  # collected on CPU only to be deselected
    tg = None


@pytest.mark.parametrize("M,N,K", [(32, 512, 8192), (32, 2048, 4096), (17, 2048, 8192), (24, 2432, 4096), (32, 2560, 7168),
                                   (64, 1024, 4096)])
def test_clusters_are_resident_at_once(monkeypatch, M, N, K):
    """Clusters beyond those that fit wait for a second wave: nearly twice the
    time of a smaller split (how many fit depends on the GPU's own layout).
    The planned split is within 30% of the best."""
    ctx = tg.Context(0)
    stream = tg.Stream(ctx)
    w = Weight(N, K, 128, False, seed=M)
    X = torch.randn(M, K, generator=torch.Generator().manual_seed(N)).to(torch.bfloat16)
    C = torch.full((M, N), float("nan"), device="cuda")
    d = tg.make_desc(M, N, K, "bf16", "f32", b_dtype="i4", transpose_b=True)
    call = tg.PreparedGemm(ctx, d, X.cuda(), w.cuda(tg), C, stream)
    torch.cuda.synchronize()
    call.enqueue()
    stream.sync()
    x = X.double()
    within(C.cpu(), x @ w.values.t(), unit(K) * (x.abs() @ w.values.abs().t()), ctx.last_kernel)
    bn = ctx.last_kernel.split("128x")[1].split("_")[0]
    side = torch.cuda.ExternalStream(stream.handle)

    def best():
        t = []
        for _ in range(7):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record(side)
            for _ in range(50):
                call.enqueue()
            b.record(side)
            stream.sync()
            t.append(a.elapsed_time(b))
        return min(t)

    best()                                                 # clocks and caches as they stay
    planned, others = best(), {}
    for split in range(3, 9):
        monkeypatch.setenv("TC_FORCE_VARIANT", f"bn={bn} split={split} tail=0")
        others[split] = best()
    monkeypatch.delenv("TC_FORCE_VARIANT")
    planned = min(planned, best())
    assert planned <= 1.3 * min(others.values()), (ctx.last_kernel, planned, others)
    stream.close()
    ctx.close()
