"""4-bit operators under stream capture: what a call needs of the stream was
taken by an earlier one, and a call that would still have to allocate is
refused without a trace."""
from __future__ import annotations

import pytest
import torch

from q4_ref import Weight, unit, within

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import matrix_multiply_gb300 as tg
else:  # collected on CPU only to be deselected
    tg = None


@pytest.fixture
def place():
    ctx, side = tg.Context(0), torch.cuda.Stream()
    stream = tg.Stream(ctx, side)
    yield ctx, side, stream
    torch.cuda.synchronize()
    stream.close()
    ctx.close()


class Product:
    def __init__(self, place, M, N, K, pad=0):
        ctx, self.side, stream = place
        self.ctx, self.w = ctx, Weight(N, K, 128, True, seed=M)
        g = torch.Generator().manual_seed(M + N)
        self.x = torch.randn(M, K, generator=g).to(torch.bfloat16)
        self.X = torch.zeros(M, K + pad, dtype=torch.bfloat16, device="cuda")[:, :K]
        self.X.copy_(self.x)
        self.C = torch.zeros(M, N, device="cuda")
        d = tg.make_desc(M, N, K, "bf16", "f32", b_dtype="i4", transpose_b=True, lda=K + pad)
        self.call = tg.PreparedGemm(ctx, d, self.X, self.w.cuda(tg), self.C, stream)
        torch.cuda.synchronize()

    def enqueue(self):
        self.call.enqueue()
        return self.ctx.last_kernel

    def check(self):
        x, v = self.x.double(), self.w.values
        torch.cuda.synchronize()
        within(self.C.cpu(), x @ v.t(), unit(self.w.K) * (x.abs() @ v.abs().t()))
        self.C.zero_()
        torch.cuda.synchronize()


class Layer:
    def __init__(self, place, T=4, H=256, I=96, E=8, k=2):
        ctx, self.side, stream = place
        g = torch.Generator().manual_seed(T)
        w = Weight(E * 2 * I, H, 32, True, seed=1, std=H ** -0.5), Weight(E * H, I, 32, True, seed=2, std=I ** -0.5)
        X, R = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda(), torch.randn(E, H, generator=g).cuda()
        self.Y = torch.zeros(T, H, device="cuda")
        want = torch.zeros(T, H, device="cuda")
        d = tg.make_moe_desc(T, H, I, E, k, "bf16", "f32")
        q = [v.cuda(tg) for v in w]
        self.call = tg.PreparedMoe(ctx, d, X, R, *q, self.Y, stream)
        torch.cuda.synchronize()
        other = tg.Context(0)
        tg.tc_moe_q4(other, d, X, R, *q, want)              # on a stream of its own
        other.close()
        self.want = want.clone()

    def enqueue(self):
        self.call.enqueue()

    def check(self):
        torch.cuda.synchronize()
        assert torch.equal(self.Y, self.want)
        self.Y.zero_()
        torch.cuda.synchronize()


def capture(place, *calls):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=place[1]):
        for c in calls:
            c.enqueue()
    return graph


def test_larger_whole_call_then_captured_cut_one(place):
    """The larger call's tiles are taken whole, the captured one's last tiles
    are cut: its workspace and counts were there before."""
    whole, cut, layer = Product(place, 1216, 4096, 512), Product(place, 200, 11008, 4096), Layer(place)
    assert not whole.enqueue().endswith("_cut")
    whole.check()
    graph = capture(place, cut)
    assert place[0].last_kernel.endswith("_cut")
    for _ in range(3):
        graph.replay()
        cut.check()
    # calls outside the graph find the words as they expect them
    cut.enqueue()
    cut.check()
    layer.enqueue()
    layer.check()
    graph.replay()
    cut.check()


def test_captured_layer(place):
    layer, cut = Layer(place), Product(place, 200, 11008, 4096)
    cut.enqueue()
    cut.check()
    layer.enqueue()
    layer.check()
    graph = capture(place, layer, cut, layer)
    for _ in range(2):
        graph.replay()
        layer.check()
        cut.check()
    layer.enqueue()
    layer.check()


@pytest.mark.parametrize("make", [Layer, lambda p: Product(p, 40, 300, 512), lambda p: Product(p, 200, 11008, 4096),
                                  lambda p: Product(p, 40, 300, 999, pad=2)])
def test_first_call_under_capture_is_refused(place, make):
    call = make(place)
    before = place[0].launch_count
    graph = torch.cuda.CUDAGraph()
    mark = torch.zeros(4, device="cuda")
    with torch.cuda.graph(graph, stream=place[1]):
        with pytest.raises(tg.TcError) as err:
            call.enqueue()
        mark += 1
    assert err.value.status == tg.TC_ERR_CUDA and place[0].launch_count == before
    graph.replay()
    torch.cuda.synchronize()
    assert mark.tolist() == [1.0] * 4                      # the capture itself is unharmed
    call.enqueue()
    call.check()
    graph = capture(place, call)
    graph.replay()
    call.check()


def test_more_rows_to_copy_are_refused(place):
    """A copy of X larger than any before it."""
    small, large = Product(place, 40, 300, 999, pad=2), Product(place, 2000, 300, 999, pad=2)
    small.enqueue()
    small.check()
    graph = torch.cuda.CUDAGraph()
    mark = torch.zeros(1, device="cuda")
    with torch.cuda.graph(graph, stream=place[1]):
        with pytest.raises(tg.TcError):
            large.enqueue()
        small.enqueue()
        mark += 1
    graph.replay()
    small.check()
