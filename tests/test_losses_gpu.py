"""The training losses in use: together on one stream, captured and replayed,
on several streams, after expired waits, past 32-bit offsets."""
from __future__ import annotations

import gc
import time

import pytest
import torch

import route_ref
import xent_ref
from xent_ref import within

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


class Xent:
    """Both calls on a stream, their outputs and what they should be."""

    def __init__(self, place, *args, **kw):
        ctx, _, stream = place
        self.c = xent_ref.Case(*args, **kw)
        c = self.c
        self.loss = torch.zeros(c.T if c.reduction == "none" else 1, device="cuda")
        self.lse = torch.zeros(c.T, device="cuda")
        self.dX = torch.zeros(c.T, c.H, dtype=xent_ref.DT[c.grad], device="cuda")
        self.dW = torch.zeros(c.V, c.H, dtype=xent_ref.DT[c.grad], device="cuda")
        self.call = tg.PreparedXent(ctx, c.desc(tg), c.X, c.W, c.y, self.lse, stream, loss=self.loss, grad=c.g, dX=self.dX,
                                    dW=self.dW)
        torch.cuda.synchronize()

    def enqueue(self):
        self.call.enqueue()
        self.call.enqueue_backward()

    def clear(self):
        for t in (self.loss, self.lse, self.dX, self.dW):
            t.fill_(float("nan"))
        torch.cuda.synchronize()

    def check(self):
        torch.cuda.synchronize()
        loss, eloss, lse, elf = self.c.forward()
        within(self.lse, lse, elf, "lse")
        within(self.loss, loss, eloss, "loss")
        dX, ex, dW, ew = self.c.backward(self.lse)
        within(self.dX, dX, ex, "dX")
        within(self.dW, dW, ew, "dW")
        self.clear()


class Route:
    def __init__(self, place, *args, **kw):
        ctx, _, stream = place
        self.c = route_ref.Case(*args, **kw)
        c = self.c
        self.ids = torch.zeros(c.T, c.k, dtype=torch.int32, device="cuda")
        self.w = torch.zeros(c.T, c.k, device="cuda")
        self.counts = torch.zeros(c.E + 1, dtype=torch.int32, device="cuda")
        self.losses = torch.zeros(2, device="cuda")
        self.dl = torch.zeros(c.T, c.E, dtype=route_ref.DT[c.grad], device="cuda")
        self.call = tg.PreparedRoute(ctx, c.desc(tg), c.l, self.ids, self.counts, stream, valid=c.valid, weights=self.w,
                                     losses=self.losses, grad_weights=c.gw, grad_losses=c.gl, dlogits=self.dl)
        torch.cuda.synchronize()

    def enqueue(self):
        self.call.enqueue()
        self.call.enqueue_backward()

    def check(self):
        torch.cuda.synchronize()
        ids, w, ew, counts, losses, el = self.c.forward()
        assert torch.equal(self.ids, ids) and torch.equal(self.counts, counts)
        within(self.w, w, ew)
        within(self.losses, losses, el)
        within(self.dl, *self.c.backward(ids, counts))
        for t in (self.ids, self.counts):
            t.fill_(-3)
        for t in (self.w, self.losses, self.dl):
            t.fill_(float("nan"))
        torch.cuda.synchronize()


def capture(place, *calls):
    gc.collect()                                           # a graph freed during a capture would end it
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=place[1]):
        for c in calls:
            c.enqueue()
    return graph


MAKE = [lambda p: Xent(p, 20, 130, 1500, "bf16", reduction="mean", ignored=0.2),
        lambda p: Xent(p, 300, 131, 3001, "f16", reduction="sum", z=0.01, pad=3, grad="f32"),
        lambda p: Xent(p, 700, 256, 20000, "bf16", reduction="none"),
        lambda p: Route(p, 40, 64, 8, padded=True), lambda p: Route(p, 3000, 100, 5, "bf16", renorm=False)]


@pytest.mark.parametrize("make", MAKE)
def test_capture_and_replay(place, make):
    call = make(place)
    call.enqueue()
    call.check()
    graph = capture(place, call, call)
    for _ in range(3):
        graph.replay()
        call.check()
    # other data in the same buffers
    c = call.c
    for t in ("X", "l", "g", "gw"):
        if hasattr(c, t):
            setattr(c, t, getattr(c, t).mul_(0.75))
    torch.cuda.synchronize()
    graph.replay()
    call.check()
    call.enqueue()
    call.check()


@pytest.mark.parametrize("make", MAKE)
def test_first_call_under_capture_is_refused(place, make):
    call = make(place)
    before = place[0].launch_count
    gc.collect()
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


def test_larger_call_then_captured_smaller_ones(place):
    calls = [m(place) for m in MAKE]
    for c in calls:
        c.enqueue()
    torch.cuda.synchronize()
    graph = capture(place, *calls)
    graph.replay()
    for c in calls:
        c.check()


def test_capture_of_kernels_that_have_not_run(place):
    """What a capture needs of the stream is memory: a larger call of another kind has taken it."""
    large = Xent(place, 900, 320, 30000, "bf16", reduction="mean")
    large.enqueue()
    large.check()
    calls = [Xent(place, 20, 130, 1500, "f16", reduction="mean", ignored=0.2, grad="f32"),
             Xent(place, 150, 1040, 2003, "bf16", reduction="sum", grad="f32"), Route(place, 70, 200, 6, "f16")]
    graph = capture(place, *calls)
    for _ in range(2):
        graph.replay()
        for c in calls:
            c.check()


def test_two_streams(place):
    ctx = place[0]
    sides = [torch.cuda.Stream() for _ in range(3)]
    places = [(ctx, s, tg.Stream(ctx, s)) for s in sides]
    calls = [[Xent(p, 200 + 50 * i, 256, 8000, "bf16", reduction="mean", seed=i), Route(p, 2000 + i, 128, 8, seed=i)]
             for i, p in enumerate(places)]
    for _ in range(4):
        for pair in calls:
            for c in pair:
                c.enqueue()
    for pair in calls:
        for c in pair:
            c.check()
    for p in places:
        p[2].close()


def test_inputs_made_on_the_same_stream_just_before(place):
    """Ordinary work on the stream, then the calls, then ordinary work: in that order."""
    ctx, side, _ = place
    call = Xent(place, 90, 256, 4000, "bf16", reduction="mean")
    route = Route(place, 500, 64, 8)
    x, l = call.c.X.clone(), route.c.l.clone()
    call.enqueue()
    route.enqueue()
    call.check()
    route.check()
    with torch.cuda.stream(side):
        for _ in range(5):
            call.c.X.zero_()
            route.c.l.zero_()
            torch.mm(torch.ones(2048, 2048, device="cuda"), torch.ones(2048, 2048, device="cuda"))
            call.c.X.copy_(x)
            route.c.l.copy_(l)
            call.enqueue()
            route.enqueue()
            kept = [t.clone() for t in (call.loss, call.dX, call.dW, route.dl)]
            call.c.X.zero_()
            route.c.l.zero_()
    torch.cuda.synchronize()
    call.c.X.copy_(x)
    route.c.l.copy_(l)
    for t, k in zip((call.loss, call.dX, call.dW, route.dl), kept):
        t.copy_(k)
    call.check()
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,H,V", [(10, 128, 600), (300, 256, 5000), (600, 64, 40000)])
def test_waits_are_bounded(place, monkeypatch, T, H, V):
    """An accumulator that is never announced ends in TC_ERR_DEVICE_TIMEOUT after a
    short limit, forward and backward, and the next calls are right."""
    ctx, _, _ = place
    call = Xent(place, T, H, V, "bf16", reduction="mean")
    c = call.c
    for fn, args in ((tg.tc_linear_xent, (call.loss, call.lse)), (tg.tc_linear_xent_backward, (call.lse, c.g, call.dX, call.dW))):
        monkeypatch.setenv("TC_FORCE_VARIANT", "debug_drop=1 debug_timeout_ms=100")
        t0 = time.monotonic()
        with pytest.raises(tg.TcError) as err:
            fn(ctx, c.desc(tg), c.X, c.W, c.y, *args)
        assert err.value.status == tg.TC_ERR_DEVICE_TIMEOUT and time.monotonic() - t0 < 5
        monkeypatch.delenv("TC_FORCE_VARIANT")
        torch.cuda.synchronize()                           # the device answers
    call.clear()
    call.enqueue()
    call.check()


def test_offsets_beyond_32_bits(place):
    """A vocabulary of more than 2^31 values, whose last rows are looked at."""
    ctx = place[0]
    T, H, V = 3, 32768, 66000
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    W = torch.randn(V, H, device="cuda", generator=g, dtype=torch.bfloat16).mul_(H ** -0.5)
    y = torch.tensor([V - 1, 5, V - 70], device="cuda")
    loss, lse = torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda")
    dX, dW = torch.zeros(T, H, device="cuda", dtype=torch.bfloat16), torch.zeros(V, H, device="cuda", dtype=torch.bfloat16)
    grad = torch.ones(T, device="cuda")
    d = tg.make_xent_desc(T, H, V, "bf16", reduction="none")
    torch.cuda.synchronize()
    tg.tc_linear_xent(ctx, d, X, W, y, loss, lse)
    tg.tc_linear_xent_backward(ctx, d, X, W, y, lse, grad, dX, dW)
    x = X.double()
    l = torch.cat([x @ W[a:a + 4000].double().t() for a in range(0, V, 4000)], 1)
    want = torch.logsumexp(l, 1)
    # a logit's products have sizes of about 0.64 sqrt(H) = 116 in all; a segment of 1024 loses up to 64 2^-24 of its share,
    # 32 of them are added: 4.4e-4 + 2.2e-4
    assert bool(((lse - want).abs() < 1e-3).all())
    assert bool(((loss - (want - l.gather(1, y[:, None])[:, 0])).abs() < 2e-3).all())
    G = torch.exp(l - lse.double()[:, None])
    G[torch.arange(T), y] -= 1
    rows = torch.tensor([V - 1, V - 70, V - 2, 5, 40000], device="cuda")
    wantW = G[:, rows].t() @ x
    # bf16 outputs: half a step, and G in two parts with 1e-3 of error in its logits
    assert bool(((dW[rows].double() - wantW).abs() <= wantW.abs() * 2.0 ** -8 + 2e-3 * (G[:, rows].abs().t() @ x.abs()) + 1e-30).all())
    wantX = sum(G[:, a:a + 4000] @ W[a:a + 4000].double() for a in range(0, V, 4000))
    size = sum(G[:, a:a + 4000].abs() @ W[a:a + 4000].double().abs() for a in range(0, V, 4000))
    assert bool(((dX.double() - wantX).abs() <= wantX.abs() * 2.0 ** -8 + 3e-3 * size).all())


def test_whole_step(place):
    """The ends of a mixture-of-experts model's training step on one stream: router
    logits, choice and balance loss, cross entropy, and all gradients down to the
    hidden rows, the router and the head, against a 64-bit automatic derivative."""
    ctx, side, stream = place
    T, H, V, E, k = 400, 192, 3000, 24, 3
    g = torch.Generator().manual_seed(3)
    X = torch.randn(T, H, generator=g).bfloat16().cuda()
    R = (torch.randn(E, H, generator=g) * H ** -0.5).bfloat16().cuda()
    W = (torch.randn(V, H, generator=g) * H ** -0.5).bfloat16().cuda()
    y = torch.randint(0, V, (T,), generator=g).cuda()
    valid = torch.ones(T, dtype=torch.bool, device="cuda")
    valid[350:] = False
    y[~valid] = -100
    gw = torch.randn(T, k, generator=g).cuda() / T           # what a layer of experts would send back
    coef = torch.tensor([0.01, 0.001], device="cuda")
    one = torch.ones(1, device="cuda")

    def zeros(*s, dt=torch.float32):
        return torch.zeros(*s, dtype=dt, device="cuda")

    l, dl = zeros(T, E), zeros(T, E, dt=torch.float32)
    dl16 = zeros(T, E, dt=torch.bfloat16)
    ids, w, counts, losses = zeros(T, k, dt=torch.int32), zeros(T, k), zeros(E + 1, dt=torch.int32), zeros(2)
    loss, lse = zeros(1), zeros(T)
    dX, dW, dR = zeros(T, H), zeros(V, H), zeros(E, H)
    logits = tg.PreparedGemm(ctx, tg.make_desc(T, E, H, "bf16", "f32", transpose_b=True), X, R, l, stream)
    route = tg.PreparedRoute(ctx, tg.make_route_desc(T, E, k), l, ids, counts, stream, valid=valid, weights=w, losses=losses,
                             grad_weights=gw, grad_losses=coef, dlogits=dl)
    xent = tg.PreparedXent(ctx, tg.make_xent_desc(T, H, V, "bf16", "f32", z_weight=1e-3), X, W, y, lse, stream, loss=loss,
                           grad=one, dX=dX, dW=dW)
    more = tg.PreparedGemm(ctx, tg.make_desc(T, H, E, "bf16", "f32", beta=1.0), dl16, R, dX, stream)
    dr = tg.PreparedGemm(ctx, tg.make_desc(E, H, T, "bf16", "f32", transpose_a=True), dl16, X, dR, stream)

    def step():
        logits.enqueue()
        route.enqueue()
        xent.enqueue()
        xent.enqueue_backward()
        route.enqueue_backward()
        dl16.copy_(dl)
        more.enqueue()
        dr.enqueue()

    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    first = [t.clone() for t in (loss, losses, dX, dW, dR)]
    gc.collect()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for t in (loss, losses, dX, dW, dR):
        t.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (loss, losses, dX, dW, dR)))

    x, r, v = (t.double().requires_grad_() for t in (X, R, W))
    rl = x @ r.t()
    p = torch.softmax(rl, 1)[valid]
    chosen = p.gather(1, ids[valid].long())
    chosen = chosen / chosen.sum(1, keepdim=True)
    n = int(valid.sum())
    f = counts[:E].double() / (n * k)
    balance = E * (f * p.mean(0)).sum()
    z = (torch.logsumexp(rl[valid], 1) ** 2).mean()
    vl = x @ v.t()
    ce = torch.nn.functional.cross_entropy(vl, y, ignore_index=-100) + 1e-3 * (torch.logsumexp(vl[valid], 1) ** 2).mean()
    total = ce + coef[0].double() * balance + coef[1].double() * z + (gw[valid].double() * chosen).sum()
    total.backward()
    assert abs(float(loss) - float(ce.detach())) < 1e-5 * float(ce.detach())
    assert abs(float(losses[0]) - float(balance.detach())) < 1e-5 and abs(float(losses[1]) - float(z.detach())) < 1e-4

    def off(a, b):
        return float((a.double() - b).norm() / b.norm())

    # dl is rounded to bf16 on its way into two products: half a step is 2^-8; the head's gradient is fp32 throughout
    assert off(dW, v.grad) < 1e-4 and off(dR, r.grad) < 2.0 ** -8 and off(dX, x.grad) < 2.0 ** -9
