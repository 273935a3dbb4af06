"""Softmax cross entropy against a vocabulary in 64 bits, with bounds on what
the kernels may be off.

Bounds, per logit l = scale x . w:
  the product      el = scale (H + 8) 2^-23 sum |x w|  (fp32 sums; tensor cores may truncate)
  the exponential  its argument is one fused multiply-add of |l| log2(e) at most, rounded, its own error 2^-22:
                   an exponential is off by r = el + (|l| + |lse|) 2^-22 + 2^-21 of its value
  a row's sum      joined from half tiles of at most 128 columns, each in 4 chains of 32 additions with 4 rescalings,
                   the half tiles by rescaled additions: 2^-21 for each step at most
  lse              max r + (64 + 2 V / 128) 2^-21 + |lse| 2^-23
  G                |G| half a step of the 16-bit type (its square in two parts), the factor of the probability r off;
                   f16 is held at a scale that makes the largest 2^13 at least: absolute half steps 2^-25 / 2^13 of it;
                   the exponential instruction gives 0 for results below 2^-126 (ftz): 2^-126 of the probability's factor
  dX, dW           the error of G through the product, fp32 sums, half a step of the output
"""
from __future__ import annotations

import torch

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def unit(K):
    return (K + 8) * 2.0 ** -23


def half(dtype):
    return torch.finfo(DT[dtype]).eps / 2


class Case:
    def __init__(self, T, H, V, dtype="bf16", *, reduction="none", scale=1.0, z=0.0, ignored=0.0, grad=None, pad=0,
                 wide=True, seed=0, lift=6.0, device="cuda"):
        self.T, self.H, self.V, self.dtype, self.reduction = T, H, V, dtype, reduction
        self.scale, self.z, self.grad, self.pad = scale, z, grad or dtype, pad
        g = torch.Generator().manual_seed(1000 * seed + T + H + V)

        def rows(n):
            t = torch.full((n, H + pad), 7.0)
            t[:, :H] = torch.randn(n, H, generator=g)
            return t

        w, x = rows(V), rows(T)
        w[:, :H] /= H ** 0.5
        self.y = torch.randint(0, V, (T,), generator=g)
        x[:, :H] = x[:, :H] / scale + lift / scale * torch.rand(T, 1, generator=g) * w[self.y][:, :H]
        off = torch.rand(T, generator=g) < ignored
        self.y[off] = torch.tensor([-100, V, -1, V + 5])[torch.arange(int(off.sum())) % 4]
        self.target_dtype = "i64" if wide else "i32"
        if not wide:
            self.y = self.y.to(torch.int32)
        self.X, self.W = (t.to(DT[dtype]).to(device)[:, :H] for t in (x, w))
        self.y = self.y.to(device)
        n = T if reduction == "none" else 1
        self.g = (0.5 + torch.rand(n, generator=g)).to(device)

    def desc(self, tg, **kw):
        return tg.make_xent_desc(self.T, self.H, self.V, self.dtype, self.grad, reduction=self.reduction,
                                 scale=self.scale, z_weight=self.z, target_dtype=self.target_dtype,
                                 ldx=self.X.stride(0), ldw=self.W.stride(0), **kw)

    def logits(self):
        x, w = self.X.double(), self.W.double()
        return self.scale * (x @ w.t()), self.scale * unit(self.H) * (x.abs() @ w.abs().t())

    def counted(self):
        y = self.y.long()
        return (y >= 0) & (y < self.V)

    def forward(self):
        """(loss, its bound, lse, its bound)"""
        l, el = self.logits()
        lse = torch.logsumexp(l, 1)
        r = (el + (l.abs() + lse.abs()[:, None]) * 2.0 ** -22 + 2.0 ** -21).amax(1)
        elf = r + (64 + 2 * self.V / 128) * 2.0 ** -21 + lse.abs() * 2.0 ** -23
        on = self.counted()
        at = torch.where(on, self.y.long(), 0)[:, None]
        ly, ey = l.gather(1, at)[:, 0], el.gather(1, at)[:, 0]
        loss = torch.where(on, lse - ly + self.z * lse * lse, 0.0)
        eloss = torch.where(on, elf + ey + (ly.abs() + lse.abs() + loss.abs()) * 2.0 ** -22
                            + self.z * (2 * lse.abs() * elf + elf * elf + lse * lse * 2.0 ** -22), 0.0)
        if self.reduction != "none":
            n = int(on.sum()) if self.reduction == "mean" else 1
            loss, eloss = loss.sum().reshape(1) / max(n, 1), eloss.sum().reshape(1) / max(n, 1)
            eloss = eloss + loss.abs() * 2.0 ** -23
        return loss, eloss, lse, elf

    def lse32(self):
        return torch.logsumexp(self.logits()[0], 1).float()

    def backward(self, lse32):
        """(dX, its bound, dW, its bound) from a given lse"""
        l, el = self.logits()
        lse = lse32.double()[:, None]
        on, y = self.counted(), torch.where(self.counted(), self.y.long(), 0)
        g = self.g.double().expand(self.T) / (max(int(on.sum()), 1) if self.reduction == "mean" else 1)
        g = torch.where(on, g, 0.0)[:, None]
        p = torch.exp(l - lse)
        cp = g * (1 + 2 * self.z * lse)
        hot = torch.zeros_like(l)
        hot[torch.arange(self.T, device=l.device), y] = 1.0
        G = torch.where(on[:, None], cp * p - g * hot, 0.0)
        r = el + (l.abs() + lse.abs()) * 2.0 ** -22 + 2.0 ** -20
        u = half(self.dtype) ** (2 if self.grad == "f32" else 1)
        eg = torch.where(on[:, None], (cp * p).abs() * r * (1 + u) + G.abs() * (u + 2.0 ** -23), 0.0)
        eg = eg + torch.where(on[:, None], cp.abs() * 2.0 ** -126, 0.0)
        top = torch.maximum(cp.abs(), g.abs()).max()
        if self.dtype == "f16":
            eg = eg + top * 2.0 ** -38
        x, w = self.X.double(), self.W.double()
        x = torch.where(on[:, None], x, 0.0)
        out = []
        for A, E, B, K in ((G, eg, w, self.V), (G.t(), eg.t(), x, self.T)):
            v = self.scale * (A @ B)
            # a second part's sums are added to the first's
            b = self.scale * ((E + unit(K) * A.abs()) @ B.abs())
            least = torch.finfo(DT[self.grad]).smallest_normal * half(self.grad)
            out += [v, b + (v.abs() + b) * half(self.grad) + least]
        return out


def within(out, want, bound, what=""):
    out = out.double()
    err = (out - want).abs()
    bad = ~(err <= bound)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bound; first {i}: got {float(out[i])!r} "
                             f"want {float(want[i])!r} bound {float(bound[i]):.3g}")
