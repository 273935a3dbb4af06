"""Routing of tokens to experts in 64 bits, with bounds on what the kernels may
be off.

Bounds: an exponential's argument (l - max) log2(e) is a rounded difference times
a rounded constant, rounded: 3 half steps of at most 1.5 |l - max|; the
exponential itself errs by 2^-22, the sum over E values in 32 lanes by E / 32 + 5
additions, its inverse by one: a probability by
    r = (5 |l - max| + 2 + E / 32 + 8) 2^-23 of its value.
"""
from __future__ import annotations

import math

import torch

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def half(dtype):
    return torch.finfo(DT[dtype]).eps / 2


class Case:
    def __init__(self, T, E, k, dtype="f32", *, renorm=True, grad=None, padded=False, masked=0.0, pad=0, seed=0, ties=False):
        self.T, self.E, self.k, self.dtype, self.renorm, self.grad = T, E, k, dtype, renorm, grad or dtype
        g = torch.Generator().manual_seed(1000 * seed + 7 * T + E + k)
        l = torch.randn(T, E, generator=g) * 1.5 + torch.randn(E, generator=g)
        if ties:
            l = torch.round(l)
            l = torch.where(l == 0, torch.where(torch.rand(T, E, generator=g) < 0.5, 0.0, -0.0), l)
        if masked:
            l = torch.where(torch.rand(T, E, generator=g) < masked * torch.rand(T, 1, generator=g) * 1.5, -math.inf, l)
        full = torch.full((T, E + pad), 99.0)
        full[:, :E] = l
        self.l = full.to(DT[dtype]).cuda()[:, :E]
        self.valid = (torch.rand(T, generator=g) < 0.7).to(torch.uint8).cuda() if padded else None
        self.gw = torch.randn(T, k, generator=g).cuda()
        self.gl = torch.randn(2, generator=g).cuda()

    def desc(self, tg, **kw):
        return tg.make_route_desc(self.T, self.E, self.k, self.dtype, self.grad, renormalize=self.renorm,
                                  ld_logits=self.l.stride(0) if self.T > 1 else 0, **kw)

    def counted(self):
        on = (self.l > -math.inf).any(1) | self.l.isnan().any(1)
        return on if self.valid is None else on & self.valid.bool()

    def choice(self):
        """ids [T, k] with -1, from a loop over the definition: the largest that is left, the lowest index of equal ones."""
        left = torch.where(self.l.isnan(), math.inf, self.l.double())
        left = torch.where(self.l == math.inf, torch.finfo(torch.float64).max, left)
        index = torch.arange(self.E, device=left.device)
        ids = torch.full((self.T, self.k), -1, dtype=torch.int64, device=left.device)
        on = self.counted()
        for j in range(self.k):
            best = left.amax(1, True)
            e = torch.where(left == best, index, self.E).amin(1)
            got = on & (best[:, 0] > -math.inf)
            ids[:, j] = torch.where(got, e, -1)
            left[torch.arange(self.T), e] = -math.inf
        return ids

    def softmax(self):
        """(p, r, lse, its bound); rows of nothing are 0."""
        l, on = self.l.double(), self.counted()[:, None]
        l = torch.where(on, l, 0.0)
        lse = torch.logsumexp(l, 1, True)
        p = torch.where(on, torch.exp(l - lse), 0.0)
        d = torch.where(l == -math.inf, 0.0, (l - l.amax(1, True)).abs())
        r = (5 * d + 2 + self.E / 32 + 8) * 2.0 ** -23
        e = (p * r).sum(1, True) + lse.abs() * 2.0 ** -22 + 2.0 ** -22
        return p, r + 2.0 ** -126 / torch.clamp(p, min=2.0 ** -140), torch.where(on, lse, 0.0), e

    def weights(self, ids):
        p, r, _, _ = self.softmax()
        at = ids.clamp(min=0)
        w = torch.where(ids >= 0, p.gather(1, at), 0.0)
        e = w * torch.where(ids >= 0, r.gather(1, at), 0.0)
        if self.renorm:
            s = w.sum(1, True).clamp(min=1e-300)
            e = (e + w * (e.sum(1, True) / s + 8 * 2.0 ** -24)) / s
            w = w / s
        return w, e + 2.0 ** -126

    def forward(self):
        ids = self.choice()
        w, ew = self.weights(ids)
        p, r, lse, el = self.softmax()
        on = self.counted()
        n = max(int(on.sum()), 1)
        c = torch.bincount(ids[ids >= 0].flatten(), minlength=self.E)
        f = c.double() / (n * self.k)
        depth = (self.T / 32 + 64) * 2.0 ** -24         # additions of a lane's sum and of a block's
        losses = torch.stack([self.E * (f * p.sum(0) / n).sum(), (lse ** 2).sum() / n])
        bound = torch.stack([self.E * (f * (p * (r + depth)).sum(0) / n).sum(),
                             ((2 * lse.abs() * el + el * el) * on[:, None] + lse ** 2 * depth).sum() / n])
        counts = torch.cat([c, on.sum()[None]]).to(torch.int32)
        return ids.to(torch.int32), w, ew, counts, losses, bound + losses.abs() * 2.0 ** -23

    def backward(self, ids, counts, with_weights=True, with_losses=True):
        p, r, lse, el = self.softmax()
        on, ids = self.counted()[:, None], ids.long()
        n = max(int(counts[-1]), 1)
        f = counts[:-1].double() / (n * self.k)
        gb, gz = (self.gl.double() if with_losses else torch.zeros(2, dtype=torch.float64, device=p.device))
        gw = self.gw.double() if with_weights else torch.zeros_like(self.gw, dtype=torch.float64)
        w, _ = self.weights(ids)
        at = ids.clamp(min=0)
        gb = gb * self.E / n
        gz = gz * 2 / n
        mean = (f * p).sum(1, True)
        out = gb * p * (f - mean) + gz * lse * p
        big = p * (gb.abs() * (f + mean) + gz.abs() * (lse.abs() + el))
        gw = torch.where(ids >= 0, gw, 0.0)
        dot, adot = (gw * w).sum(1, True), (gw.abs() * w).sum(1, True)
        if self.renorm:
            out = out.scatter_add(1, at, torch.where(ids >= 0, w * (gw - dot), 0.0))
            big = big.scatter_add(1, at, torch.where(ids >= 0, w * (gw.abs() + adot), 0.0))
        else:
            out = out.scatter_add(1, at, w * gw) - p * dot
            big = big.scatter_add(1, at, w * gw.abs()) + p * adot
        # every factor of a term is off by at most the largest r of its row, a term has three of them; a dozen roundings
        rel = 3 * (torch.where(p > 2.0 ** -100, r, 0.0).amax(1, True)) + 16 * 2.0 ** -23
        least = torch.finfo(DT[self.grad]).smallest_normal * half(self.grad)
        bound = big * rel + gz.abs() * el * p + 2.0 ** -120 * (big.amax() + gw.abs().amax()) + least
        out = torch.where(on, out, 0.0)
        return out, torch.where(on, bound + (out.abs() + bound) * half(self.grad), 0.0)
