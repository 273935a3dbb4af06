"""What is measured of the 4-bit weight operators: quantising a weight matrix to
4 bits with group scales (and giving its values back), the product of activations
with such a weight, and a whole mixture-of-experts layer over such weights.

A 4-bit weight W[N, K] is three tensors:
  codes   uint8 [N, L / 2], L = K rounded up to 32 elements: row-major, eight
          consecutive elements e0..e7 in four bytes, nibble order
          (low first) e0 e2 | e4 e6 | e1 e3 | e5 e7;
  scales  f16 or bf16 [ceil(K / G), Ns], Ns = N rounded up to 16: one scale for
          G consecutive k of a row, G in {32, 64, 128};
  zeros   uint8, the scales' shape, values 0..15, or none (then 8 everywhere);
and stands for W[n, k] = (code - zero) * scale.

Formulas:
  quantise   no zeros: s = round16(max|w| / 7), code = clamp(round(w / s) + 8, 0, 15)
             zeros:    lo = min(w, 0), hi = max(w, 0) over the group,
                       s = round16((hi - lo) / 15), z = clamp(round(-lo / s), 0, 15),
                       code = clamp(round(w / s) + z, 0, 15)
             (s = 0: code = zero = 8); round is to nearest even
  product    C[m, n] = alpha * sum_k X[m, k] W[n, k]
  experts    p = softmax(X router^T); the top_k experts of a token by p, ties to
             the lowest index, their p renormalised to one where asked;
             y = sum_j p_j * Wdown_e(j) (silu(Wgate_e(j) x) * (Wup_e(j) x))
"""
import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
# element j of eight sits at nibble NIBBLE[j] of its 32-bit word
NIBBLE = [0, 4, 1, 5, 2, 6, 3, 7]


def up(x, m):
    return (x + m - 1) // m * m


# ------------------------------------------------------------------- cases

def product(M, N, K, x, c, group, zeros, scale="f16", alpha=1.0, pad=0):
    return {"kind": "product", "M": M, "N": N, "K": K, "x": x, "c": c, "group": group, "zeros": zeros,
            "scale": scale, "alpha": alpha, "pad": pad}


def quantise(N, K, w, v, group, zeros, scale="f16", pad=0):
    return {"kind": "quantise", "N": N, "K": K, "w": w, "v": v, "group": group, "zeros": zeros, "scale": scale,
            "pad": pad}


def experts(T, H, I, E, k, x, y, group, zeros, scale="f16", renorm=True, router="f32"):
    return {"kind": "experts", "T": T, "H": H, "I": I, "E": E, "k": k, "x": x, "y": y, "group": group,
            "zeros": zeros, "scale": scale, "renorm": renorm, "router": router}


def listed():
    return [
        # one token through a square projection: the call whose latency is a decoding step's
        dict(product(1, 4096, 4096, "bf16", "bf16", 128, False), name="product 1x4096x4096"),
        # four sequences decoding together through a feed-forward block's second matrix
        dict(product(4, 4096, 11008, "f16", "f16", 64, True), name="product 4x4096x11008 zeros"),
        # sixteen through its first matrix, the finest groups, fp32 outputs
        dict(product(16, 11008, 4096, "bf16", "f32", 32, False, scale="bf16"), name="product 16x11008x4096"),
        # nothing a multiple of anything, padded activations, a scalar
        dict(product(7, 1001, 2999, "f16", "f32", 32, True, alpha=0.5, pad=3), name="product 7x1001x2999 ragged"),
        # a short prompt, not a multiple of a tile
        dict(product(200, 11008, 4096, "bf16", "bf16", 128, True, scale="bf16"), name="product 200x11008x4096"),
        # a long prompt
        dict(product(4096, 11008, 4096, "f16", "f16", 128, False), name="product 4096x11008x4096"),
        # one projection's weight on its way into 4 bits
        dict(quantise(4096, 4096, "bf16", "bf16", 128, False), name="quantise 4096x4096"),
        # ragged, from fp32, with zero points
        dict(quantise(1001, 2999, "f32", "f32", 32, True, scale="bf16", pad=5), name="quantise 1001x2999 ragged"),
        # all experts of a layer in one call
        dict(quantise(65536, 4096, "f16", "f16", 64, True), name="quantise 65536x4096"),
        # one token through small experts: a decoding step's latency
        dict(experts(1, 2048, 768, 64, 8, "bf16", "bf16", 128, False), name="experts 1 token"),
        # sixteen sequences decoding together through wider ones
        dict(experts(16, 4096, 1408, 64, 8, "f16", "f16", 64, True), name="experts 16 tokens"),
        # odd widths, an odd number of experts, a router in the activations' type, no renormalising
        dict(experts(5, 1000, 333, 13, 3, "bf16", "f32", 32, True, scale="bf16", renorm=False, router="bf16"),
             name="experts 5 tokens ragged"),
    ]


def log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def size(rng, lo, hi):
    """Spread over the logarithm; a third of them odd, the others multiples of 64 or of 8."""
    v = log_between(rng, lo, hi)
    how = rng.randrange(3)
    v = v | 1 if how == 0 else up(v, 64) if how == 1 else up(v, 8)
    v = max(lo, min(hi, v))
    return v + 8 if v == 3072 else v


def draw(rng):
    kind = rng.choice(["product", "product", "quantise", "experts"])
    group, zeros, scale = rng.choice([32, 64, 128]), rng.random() < 0.5, rng.choice(["f16", "bf16"])
    x = rng.choice(["f16", "bf16"])
    if kind == "product":
        M = rng.randint(1, 16) if rng.random() < 0.6 else log_between(rng, 17, 4096)
        N, K = size(rng, 64, 11008), size(rng, 64, 11008)
        while M * N * K > 4096 * 11008 * 4096:
            M = max(17, M // 2)
        return product(M, N, K, x, rng.choice([x, "f32"]), group, zeros, scale, rng.choice([1.0, 0.5, -2.0]),
                       rng.choice([0, 0, 1, 8]))
    if kind == "quantise":
        N, K, w = size(rng, 64, 32768), size(rng, 64, 4096), rng.choice(["f16", "bf16", "f32"])
        return quantise(N, K, w, w, group, zeros, scale, rng.choice([0, 0, 1, 8]))
    E = log_between(rng, 4, 64)
    return experts(log_between(rng, 1, 16), size(rng, 256, 4096), size(rng, 128, 1408), E,
                   rng.randint(1, min(8, E)), x, rng.choice([x, "f32"]), group, zeros, scale, rng.random() < 0.5,
                   rng.choice(["f32", x]))


# ------------------------------------------------------------------- inputs

def make_q4(N, K, group, zeros, scale, g, std=0.02):
    """Codes, scales and zeros of an [N, K] weight of about the given standard deviation."""
    dev = "cuda"
    codes = torch.randint(0, 256, (N, up(K, 32) // 2), dtype=torch.uint8, device=dev, generator=g)
    ng, ns = -(-K // group), up(N, 16)
    # a uniform code is 4.6 scales off its middle on average
    s = (0.5 + torch.rand(ng, ns, device=dev, generator=g)) * (std / 4.6)
    z = torch.randint(6, 11, (ng, ns), dtype=torch.uint8, device=dev, generator=g) if zeros else None
    return {"codes": codes, "scales": s.to(DT[scale]), "zeros": z, "N": N, "K": K, "group": group}


def make_x(M, K, x, pad, g):
    """Activations: normal, one channel in a hundred twenty times the others; rows `pad` elements apart."""
    full = torch.randn(M, K + pad, device="cuda", generator=g)
    full *= torch.where(torch.rand(K + pad, device="cuda", generator=g) < 0.01, 20.0, 1.0)
    return full.to(DT[x])[:, :K]


_user = []


def user():
    """The context and the stream that a user's program keeps."""
    import matrix_multiply_gb300 as tg
    if not _user:
        ctx = tg.Context(torch.cuda.current_device())
        _user.extend([tg, ctx, tg.Stream(ctx, torch.cuda.current_stream())])
    return _user


def handle(tg, q):
    return tg.Q4Weight(q["N"], q["K"], q["group"], q["codes"], q["scales"], q["zeros"])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, dev = case, "cuda"
    st = {"case": c}
    if c["kind"] == "product":
        st["X"] = make_x(c["M"], c["K"], c["x"], c["pad"], g)
        st["q"] = make_q4(c["N"], c["K"], c["group"], c["zeros"], c["scale"], g)
        if own:
            tg, ctx, stream = user()
            st["C"] = torch.empty(c["M"], c["N"], dtype=DT[c["c"]], device=dev)
            d = tg.make_desc(c["M"], c["N"], c["K"], c["x"], c["c"], b_dtype="i4", transpose_b=True,
                             alpha=c["alpha"], lda=st["X"].stride(0))
            st["call"] = tg.PreparedGemm(ctx, d, st["X"], handle(tg, st["q"]), st["C"], stream)
    elif c["kind"] == "quantise":
        full = torch.randn(c["N"], c["K"] + c["pad"], device=dev, generator=g).mul_(0.02)
        st["W"] = full.to(DT[c["w"]])[:, :c["K"]]
        if own:
            tg, ctx, stream = user()
            ng, ns = -(-c["K"] // c["group"]), up(c["N"], 16)
            st["scales"] = torch.zeros(ng, ns, dtype=DT[c["scale"]], device=dev)
            q = tg.Q4Weight(c["N"], c["K"], c["group"],
                            torch.empty(c["N"], up(c["K"], 32) // 2, dtype=torch.uint8, device=dev), st["scales"],
                            torch.zeros(ng, ns, dtype=torch.uint8, device=dev) if c["zeros"] else None)
            st["V"] = torch.empty(c["N"], c["K"], dtype=DT[c["v"]], device=dev)
            st["call"] = (tg, ctx, stream, q)
    else:
        T, H, I, E = c["T"], c["H"], c["I"], c["E"]
        st["X"] = make_x(T, H, c["x"], 0, g)
        st["router"] = (torch.randn(E, H, device=dev, generator=g) / math.sqrt(H)).to(DT[c["router"]])
        st["gate_up"] = make_q4(E * 2 * I, H, c["group"], c["zeros"], c["scale"], g, 1 / math.sqrt(H))
        st["down"] = make_q4(E * H, I, c["group"], c["zeros"], c["scale"], g, 1 / math.sqrt(I))
        if own:
            tg, ctx, stream = user()
            st["Y"] = torch.empty(T, H, dtype=DT[c["y"]], device=dev)
            st["ids"] = torch.empty(T, c["k"], dtype=torch.int32, device=dev)
            st["p"] = torch.empty(T, c["k"], dtype=torch.float32, device=dev)
            d = tg.make_moe_desc(T, H, I, E, c["k"], c["x"], c["y"], router_dtype=c["router"],
                                 renormalize=c["renorm"])
            st["call"] = tg.PreparedMoe(ctx, d, st["X"], st["router"], handle(tg, st["gate_up"]),
                                        handle(tg, st["down"]), st["Y"], stream, ids=st["ids"], weights=st["p"])
    return st


# --------------------------------------------------------------- plain form

def unpack(codes, K):
    """uint8 codes [N, L / 2] -> whole numbers [N, K] in 32-bit floats."""
    nib = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1, 8)
    return nib[:, :, NIBBLE].reshape(codes.shape[0], -1)[:, :K].float()


def over_rows(t, q):
    """A scale or a zero for each weight: [groups, Ns] -> [N, K]."""
    return t[:, :q["N"]].float().t().repeat_interleave(q["group"], 1)[:, :q["K"]]


def plain_values(q):
    code = unpack(q["codes"], q["K"])
    code -= 8.0 if q["zeros"] is None else over_rows(q["zeros"], q)
    code *= over_rows(q["scales"], q)
    return code


def plain_quantise(c, W):
    """(codes as whole numbers, scales, zeros) per weight, group by group: [N, groups, G] and [N, groups, 1]."""
    N, K, G = c["N"], c["K"], c["group"]
    ng = -(-K // G)
    w = torch.nn.functional.pad(W.float(), (0, ng * G - K)).reshape(N, ng, G)
    if c["zeros"]:
        lo, hi = w.amin(-1, True).clamp(max=0.0), w.amax(-1, True).clamp(min=0.0)
        s = ((hi - lo) / torch.full_like(hi, 15.0)).to(DT[c["scale"]]).float()
        none = s == 0
        z = torch.where(none, 8.0, torch.round(-lo / torch.where(none, 1.0, s)).clamp(0, 15))
    else:
        big = w.abs().amax(-1, True)
        s = (big / torch.full_like(big, 7.0)).to(DT[c["scale"]]).float()
        none = s == 0
        z = torch.full_like(s, 8.0)
    code = torch.where(none, z, (torch.round(w / torch.where(none, 1.0, s)) + z).clamp(0, 15))
    return code, s, z


def plain_experts(c, st):
    T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    x = st["X"].float()
    p = x @ st["router"].float().t()
    p = torch.exp(p - p.amax(-1, True))
    p = p / p.sum(-1, keepdim=True)
    # a stable sort keeps equal ones in the order of their index
    val, ids = torch.sort(p, dim=-1, descending=True, stable=True)
    val, ids = val[:, :k], ids[:, :k]
    if c["renorm"]:
        val = val / val.sum(-1, keepdim=True)
    per = torch.zeros(T, E, device=x.device).scatter_(1, ids, val)
    gu = (x @ plain_values(st["gate_up"]).t()).reshape(T, E, 2, I)
    gate, lin = gu[:, :, 0], gu[:, :, 1]
    h = gate / (1 + torch.exp(-gate)) * lin * per[:, :, None]
    h = torch.where(per[:, :, None] != 0, h, 0.0)
    y = h.reshape(T, E, I).transpose(0, 1) @ plain_values(st["down"]).reshape(E, H, I).transpose(1, 2)
    return {"y": y.sum(0).to(DT[c["y"]]), "ids": ids.to(torch.int32), "p": val}


def run(state):
    c, st = state["case"], state
    if c["kind"] == "product":
        if own:
            st["call"].enqueue()
            return st["C"]
        out = st["X"].float() @ plain_values(st["q"]).t()
        return (out * c["alpha"]).to(DT[c["c"]])
    if c["kind"] == "quantise":
        if own:
            tg, ctx, stream, q = st["call"]
            tg.tc_quantize_q4_async(ctx, st["W"], q, stream)
            tg.tc_dequantize_q4_async(ctx, q, st["V"], stream)
            return {"scales": st["scales"], "values": st["V"]}
        code, s, z = plain_quantise(c, st["W"])
        scales = torch.zeros(s.shape[1], up(c["N"], 16), dtype=DT[c["scale"]], device=s.device)
        scales[:, :c["N"]] = s[:, :, 0].t()
        values = ((code - z) * s).reshape(c["N"], -1)[:, :c["K"]]
        return {"scales": scales, "values": values.to(DT[c["v"]])}
    if own:
        st["call"].enqueue()
        return {"y": st["Y"], "ids": st["ids"], "p": st["p"]}
    return plain_experts(c, st)


# -------------------------------------------------------------------- work

def q4_bytes(rows, K, group, zeros):
    return rows * K / 2 + rows * -(-K // group) * (3 if zeros else 2)


def work(case):
    c, es = case, {"f16": 2, "bf16": 2, "f32": 4}
    if c["kind"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": q4_bytes(N, K, c["group"], c["zeros"]) + 2 * M * K + es[c["c"]] * M * N,
                "flops": 2.0 * M * N * K}
    if c["kind"] == "quantise":  # into 4 bits, and the values back from them
        N, K = c["N"], c["K"]
        return {"bytes": N * K * (es[c["w"]] + es[c["v"]]) + 2 * q4_bytes(N, K, c["group"], c["zeros"]), "flops": 0.0}
    T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    used = E * (1 - (1 - k / E) ** T)  # experts that at least one token goes to, for a router that spreads them
    each = q4_bytes(2 * I, H, c["group"], c["zeros"]) + q4_bytes(H, I, c["group"], c["zeros"])
    return {"bytes": used * each + es[c["router"]] * E * H + T * H * (2 + es[c["y"]]) + 8 * T * k,
            "flops": 2.0 * T * k * 3 * H * I + 2.0 * T * E * H}


# ---------------------------------------------------- the definition, 64 bits

def exact_weight(q, rows):
    """The rows' weights in 64 bits, from shifts of whole 32-bit words."""
    words = q["codes"][rows].to(torch.int64).reshape(-1, q["codes"].shape[1] // 4, 4)
    word = words[..., 0] + (words[..., 1] << 8) + (words[..., 2] << 16) + (words[..., 3] << 24)
    k = torch.arange(q["K"], device=word.device)
    e = k % 8
    nib = (word[:, k // 8] >> (4 * (e // 2 + 4 * (e % 2)))) & 15
    at = k // q["group"]
    s = q["scales"][at][:, rows].double().t()
    z = 8.0 if q["zeros"] is None else q["zeros"][at][:, rows].double().t()
    return (nib.double() - z) * s


def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["kind"] == "product":
        X, out = st["X"].double(), []
        for n in range(0, c["N"], 2048):
            rows = torch.arange(n, min(c["N"], n + 2048), device=X.device)
            out.append(c["alpha"] * (X @ exact_weight(st["q"], rows).t()))
        return torch.cat(out, 1)
    if c["kind"] == "quantise":
        N, K, G = c["N"], c["K"], c["group"]
        ng = -(-K // G)
        scales = torch.zeros(ng, up(N, 16), dtype=torch.float64, device="cuda")
        values = torch.empty(N, K, dtype=torch.float64, device="cuda")
        for i in range(ng):
            w = st["W"][:, i * G:(i + 1) * G].double()
            if c["zeros"]:
                lo, hi = torch.clamp(w.min(1).values, max=0), torch.clamp(w.max(1).values, min=0)
                s = ((hi - lo) / 15).to(DT[c["scale"]]).double()
                z = torch.where(s > 0, torch.clamp(torch.round(-lo / s), 0, 15), 8.0)
            else:
                s = (w.abs().max(1).values / 7).to(DT[c["scale"]]).double()
                z = torch.full_like(s, 8.0)
            code = torch.clamp(torch.round(w / s[:, None]) + z[:, None], 0, 15)
            values[:, i * G:(i + 1) * G] = torch.where(s[:, None] > 0, (code - z[:, None]) * s[:, None], 0.0)
            scales[i, :N] = s
        return {"scales": scales, "values": values}
    T, H, I, k = c["T"], c["H"], c["I"], c["k"]
    X = st["X"].double()
    logits = X @ st["router"].double().t()
    e = torch.exp(logits - logits.max(1, keepdim=True).values)
    p = e / e.sum(1, keepdim=True)
    val, ids = torch.topk(p, k, dim=1)
    if c["renorm"]:
        val = val / val.sum(1, keepdim=True)
    y = torch.zeros(T, H, dtype=torch.float64, device=X.device)
    for x in sorted(set(ids.flatten().tolist())):
        t, j = (ids == x).nonzero(as_tuple=True)
        W1 = exact_weight(st["gate_up"], torch.arange(x * 2 * I, (x + 1) * 2 * I, device=X.device))
        W2 = exact_weight(st["down"], torch.arange(x * H, (x + 1) * H, device=X.device))
        gate, lin = X[t] @ W1[:I].t(), X[t] @ W1[I:].t()
        y.index_add_(0, t, ((gate * torch.sigmoid(gate) * lin) @ W2.t()) * val[t, j][:, None])
    return {"y": y, "ids": None, "p": val}
