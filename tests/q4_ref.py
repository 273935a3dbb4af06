"""Plain 64-bit forms of the 4-bit weight operators, and inputs for them (CPU)."""
from __future__ import annotations

import torch

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
NIBBLE = [0, 4, 1, 5, 2, 6, 3, 7]          # element j of a word's eight sits at this nibble


def up(x, m):
    return (x + m - 1) // m * m


def pack(code, ldw):
    """Whole numbers [N, K] -> uint8 [N, ldw / 2]; elements past K hold 15."""
    N, K = code.shape
    full = torch.full((N, ldw), 15, dtype=torch.uint8)
    full[:, :K] = code
    word = full.reshape(N, -1, 8)
    nib = torch.empty_like(word)
    for j, p in enumerate(NIBBLE):
        nib[:, :, p] = word[:, :, j]
    nib = nib.reshape(N, -1, 2)
    return (nib[:, :, 0] | (nib[:, :, 1] << 4)).reshape(N, ldw // 2).contiguous()


def unpack(codes, K):
    nib = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1, 8)
    return nib[:, :, NIBBLE].reshape(codes.shape[0], -1)[:, :K]


def spread(t, N, K, group):
    """[groups, >= N] -> [N, K]"""
    return t[:, :N].t().repeat_interleave(group, 1)[:, :K]


class Weight:
    """A random 4-bit weight on the CPU and its values in 64 bits.  The
    padding holds values that would show: codes 15, scales NaN, zeros 255."""

    def __init__(self, N, K, group, zeros, scale="f16", seed=0, kind="normal", ldw=0, lds=0, std=0.02):
        g = torch.Generator().manual_seed(seed)
        self.N, self.K, self.group = N, K, group
        ng, lds, ldw = -(-K // group), lds or up(N, 16), ldw or up(K, 32)
        code = torch.randint(0, 16, (N, K), generator=g, dtype=torch.uint8)
        s = torch.full((ng, lds), float("nan"))
        if kind == "pow2":      # every sum of whole numbers times these is exact in fp32
            s[:, :N] = 2.0 ** torch.randint(-2, 3, (ng, N), generator=g)
        else:
            s[:, :N] = (0.5 + torch.rand(ng, N, generator=g)) * (std / 4.6)
        self.scales = s.to(DT[scale])
        self.zeros = None
        z = torch.full((N, K), 8.0, dtype=torch.float64)
        if zeros:
            self.zeros = torch.full((ng, lds), 255, dtype=torch.uint8)
            self.zeros[:, :N] = torch.randint(0, 16, (ng, N), generator=g, dtype=torch.uint8)
            z = spread(self.zeros.double(), N, K, group)
        self.codes = pack(code, ldw)
        self.values = (code.double() - z) * spread(self.scales.double(), N, K, group)

    def cuda(self, tg):
        return tg.Q4Weight(self.N, self.K, self.group, self.codes.cuda(), self.scales.cuda(),
                           None if self.zeros is None else self.zeros.cuda())


def unit(K):
    """Relative bound on an fp32 sum of K products against sum |a b|: each of
    at most K + 8 additions (and the scales) errs by at most 2^-23 (tensor
    cores may truncate), never above the library's 1e-4."""
    return min(1e-4, (K + 8) * 2.0 ** -23)


def ulp(y, dtype):
    frac, least = {"bf16": (7, -133), "f16": (10, -24), "f32": (23, -149)}[dtype]
    a = y.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a))))
    return torch.clamp(torch.where(a > 0, 2.0 ** (e - frac), torch.zeros_like(a)), min=2.0 ** least)


def within(out, want, bound, what=""):
    err = (out.double() - want).abs()
    bad = ~(err <= bound)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bound; first {i}: got "
                             f"{float(out[i])!r} want {float(want[i])!r} bound {float(bound[i]):.3g}")


def quantise(W, group, zeros, scale):
    """The header's formulas in fp32: (codes [N, K up 32], scales, zeros or None)."""
    N, K = W.shape
    ng, kp = -(-K // group), up(K, 32)
    w = torch.nn.functional.pad(W.float(), (0, ng * group - K)).reshape(N, ng, group)
    lo, hi = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
    s = (hi - lo) / 15.0 if zeros else torch.maximum(hi, -lo) / 7.0
    s = torch.where(torch.isfinite(w).all(-1), s, torch.nan).to(DT[scale])
    f = s.float()
    none = f == 0
    z = torch.full_like(f, 8.0)
    if zeros:
        z = torch.where(none, z, torch.round(-lo / f).clamp(0, 15))
    code = (torch.round(w / f[:, :, None]) + z[:, :, None]).clamp(0, 15)
    code = torch.where(none[:, :, None], z[:, :, None], code).reshape(N, -1)
    code = torch.nn.functional.pad(code, (0, max(0, kp - code.shape[1])))[:, :kp]
    return code, s.t(), z.t() if zeros else None


def moe(X, R, w1, w2, I, k, renorm):
    """(y, ids, p, bound on |y - computed|) in 64 bits; the bound carries the
    fp32 sums' errors (unit), 2^-15 of h for its 16 bits of significand, and
    4e-6 for the exponentials through the formulas' slopes."""
    T, H = X.shape
    x, r = X.double(), R.double()
    l = x @ r.t()
    e = torch.exp(l - l.max(1, keepdim=True).values)
    p = e / e.sum(1, keepdim=True)
    ids = torch.argsort(l, dim=1, descending=True, stable=True)[:, :k]
    val = p.gather(1, ids)
    if renorm:
        val = val / val.sum(1, keepdim=True)
    dl = unit(H) * (x.abs() @ r.abs().t())
    dp = 2 * (dl.max(1).values + 4e-6)          # relative: softmax of logits off by dl
    y, b = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    W1, W2 = w1.values.reshape(-1, 2 * I, H), w2.values.reshape(-1, H, I)
    u1, u2 = unit(H), unit(I)
    for t in range(T):
        for j in range(k):
            a, d = W1[ids[t, j]], W2[ids[t, j]]
            gu, tgu = a @ x[t], a.abs() @ x[t].abs()
            g, u, tg_, tu = gu[:I], gu[I:], tgu[:I], tgu[I:]
            si = g * torch.sigmoid(g)
            h = si * u
            dh = 1.1 * u1 * tg_ * (u.abs() + u1 * tu) + si.abs() * u1 * tu + (4e-6 + 2.0 ** -15) * h.abs()
            y[t] += val[t, j] * (d @ h)
            b[t] += val[t, j] * (d.abs() @ dh + (u2 + dp[t]) * (d.abs() @ h.abs()))
    return y, ids, val, b, dp
