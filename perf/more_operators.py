"""What is measured of the training losses: softmax cross entropy of hidden rows
against a large vocabulary, straight from the two matrices and with its
gradients, and the routing of tokens to experts with its balance loss, its
counts and its gradient.

Formulas, X [T, H] hidden rows, W [V, H] the vocabulary's rows, y targets:
  l[t, v]  = scale * sum_h X[t, h] W[v, h]
  lse[t]   = log sum_v exp(l[t, v])
  loss[t]  = lse[t] - l[t, y_t] + z * lse[t]^2, 0 for a row whose target is outside [0, V) (it is not counted);
             reduced: none, the sum, or the mean over the counted rows (0 without any)
  g[t]     = the gradient that arrives at loss[t] (of a sum the one value, of a mean that over the counted rows)
  G[t, v]  = g[t] * ((1 + 2 z lse[t]) exp(l[t, v] - lse[t]) - [v = y_t]), 0 for rows not counted
  dX = scale * G W,  dW = scale * G^T X

and with l [T, E] the router's logits, a token counting where it is valid and any of its logits is above -inf:
  p = softmax(l[t]);  the top_k experts e_j of a token by l, ties to the lowest index, -1 once only -inf is left;
  w_j = p[e_j], divided by their sum where asked (0 for id -1; ids -1 and weights 0 of tokens not counted)
  n = the counted tokens, c[e] the tokens that chose e, f[e] = c[e] / (n k), P[e] = mean p[t, e]
  losses = E sum_e f[e] P[e], mean lse[t]^2   (0 without counted tokens)
  dl[t, e] = gb (E / n) p[e] (f[e] - sum_j f[j] p[j]) + gz (2 / n) lse[t] p[e]
             + the gradient through the weights: p[e] ([e = e_j] gw_j - sum_i gw_i w_i), or, where they were divided by
             their sum, w_j (gw_j - sum_i gw_i w_i) at e = e_j;   0 for tokens not counted
"""
import math

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ES = {"f16": 2, "bf16": 2, "f32": 4}


# ------------------------------------------------------------------- cases

def xent(kind, T, H, V, x, reduction, scale=1.0, z=0.0, ignored=0.0, wide=False, grad=None, pad=0):
    return {"kind": kind, "T": T, "H": H, "V": V, "x": x, "reduction": reduction, "scale": scale, "z": z,
            "ignored": ignored, "wide": wide, "grad": grad or x, "pad": pad}


def route(kind, T, E, k, x, renorm=True, padded=False, masked=False, grad=None, pad=0):
    return {"kind": kind, "T": T, "E": E, "k": k, "x": x, "renorm": renorm, "padded": padded, "masked": masked,
            "grad": grad or x, "pad": pad}


def listed():
    return [
        # one token scored against a vocabulary: the call is the stream of the weight
        dict(xent("loss", 1, 2048, 32000, "bf16", "none"), name="loss 1x2048x32000"),
        # a few short sequences with prompts that do not count, nothing a multiple of anything, padded rows, the z term
        dict(xent("loss", 300, 1001, 10007, "f16", "sum", 0.5, 1e-3, 0.4, True, pad=3), name="loss 300x1001x10007 ragged"),
        # the evaluation of a long batch over a large vocabulary
        dict(xent("loss", 4096, 4096, 131072, "bf16", "mean", ignored=0.05, wide=True), name="loss 4096x4096x131072"),
        # a small model's step, where launches count
        dict(xent("gradients", 64, 512, 2000, "bf16", "mean", ignored=0.1, wide=True), name="gradients 64x512x2000"),
        # ragged, a gradient for each row, gradients in 32 bits for an optimiser's sums
        dict(xent("gradients", 300, 1001, 10007, "f16", "none", 0.5, 1e-3, 0.4, grad="f32", pad=3),
             name="gradients 300x1001x10007 ragged"),
        # a training step's last layer
        dict(xent("gradients", 2048, 2048, 32000, "bf16", "mean", z=1e-4, wide=True), name="gradients 2048x2048x32000"),
        # the same of a large model, in the type whose range is narrow
        dict(xent("gradients", 4096, 4096, 65536, "f16", "mean", ignored=0.05), name="gradients 4096x4096x65536"),
        # one token's choice of experts: a decoding step's latency
        dict(route("route", 1, 64, 8, "f32"), name="route 1x64"),
        # odd numbers of tokens and experts, padded batch, experts that a token may not take, logits in 16 bits
        dict(route("route", 1001, 13, 3, "f16", False, True, True, pad=3), name="route 1001x13 ragged"),
        # a long batch over many experts
        dict(route("route", 65536, 256, 8, "f32", padded=True), name="route 65536x256"),
        # a training step's gradient over a middling number of experts, some padding
        dict(route("route gradients", 8192, 60, 4, "bf16", False, True, grad="f32"), name="route gradients 8192x60"),
        # and that of the long batch
        dict(route("route gradients", 65536, 256, 8, "f32", padded=True), name="route gradients 65536x256"),
    ]


def size(rng, lo, hi):
    """Spread over the logarithm; a third of them odd, the others multiples of 64 or of 8."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    how = rng.randrange(3)
    v = v | 1 if how == 0 else -(-v // 64) * 64 if how == 1 else -(-v // 8) * 8
    return max(lo, min(hi, v))


def draw(rng):
    kind = rng.choice(["loss", "gradients", "gradients", "route", "route gradients"])
    x = rng.choice(["f16", "bf16"])
    pad = rng.choice([0, 0, 1, 8])
    if kind in ("loss", "gradients"):
        T, H, V = size(rng, 1, 4096), size(rng, 64, 4096), size(rng, 1000, 131072)
        while kind == "gradients" and T * H * V > 4096 * 4096 * 65536:
            V = max(1000, V // 2 + 1)
        return xent(kind, T, H, V, x, rng.choice(["none", "sum", "mean"]), rng.choice([1.0, 0.5]),
                    rng.choice([0.0, 1e-4, 1e-2]), rng.choice([0.0, 0.1, 0.6]), rng.random() < 0.5,
                    rng.choice([x, x, "f32"]), pad)
    E = size(rng, 4, 256)
    return route(kind, size(rng, 1, 65536), E, rng.randint(1, min(8, E)), rng.choice(["f32", "f32", x]),
                 rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.3, rng.choice([None, "f32"]), pad)


# ------------------------------------------------------------------- inputs

_user = []


def user():
    """The context and the stream that a user's program keeps."""
    import matrix_multiply_gb300 as tg
    if not _user:
        ctx = tg.Context(torch.cuda.current_device())
        _user.extend([tg, ctx, tg.Stream(ctx, torch.cuda.current_stream())])
    return _user


def padded_rows(t, dt, pad):
    """t in type dt, its rows `pad` elements apart."""
    full = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=dt, device=t.device)
    full[:, :t.shape[1]] = t
    return full[:, :t.shape[1]]


def pieces(n, each):
    return [(i, min(n, i + each)) for i in range(0, n, each)]


def make_lse(c, st):
    """The forward pass's lse, which a backward pass is given."""
    out = []
    w = st["W"].float()
    for a, b in pieces(c["T"], 1024):
        out.append(torch.logsumexp(c["scale"] * (st["X"][a:b].float() @ w.t()), 1))
    return torch.cat(out)


def prepare_xent(c, g):
    T, H, V, dev = c["T"], c["H"], c["V"], "cuda"
    st = {"case": c}
    w = torch.randn(V, H, device=dev, generator=g).div_(math.sqrt(H))
    y = torch.randint(0, V, (T,), device=dev, generator=g)
    # a model that has learned something: the target's logit stands out, by up to 14
    lift = torch.rand(T, 1, device=dev, generator=g) * (14.0 / c["scale"])
    st["X"] = padded_rows(torch.randn(T, H, device=dev, generator=g) / c["scale"] + lift * w[y], DT[c["x"]], c["pad"])
    st["W"] = padded_rows(w, DT[c["x"]], c["pad"])
    del w
    y = torch.where(torch.rand(T, device=dev, generator=g) < c["ignored"], -100, y)
    st["y"] = y if c["wide"] else y.to(torch.int32)
    if c["kind"] == "gradients":
        st["lse"] = make_lse(c, st)
        st["g"] = (0.5 + torch.rand(T, device=dev, generator=g)) / T if c["reduction"] == "none" else \
            0.5 + torch.rand(1, device=dev, generator=g)
        if c["grad"] == "f16":
            st["g"] *= 1024.0  # the loss scale that training in this type comes with
    if own:
        tg, ctx, stream = user()
        d = tg.make_xent_desc(T, H, V, c["x"], c["grad"], reduction=c["reduction"], scale=c["scale"], z_weight=c["z"],
                              target_dtype="i64" if c["wide"] else "i32", ldx=st["X"].stride(0), ldw=st["W"].stride(0))
        if c["kind"] == "loss":
            st["loss"] = torch.empty(T if c["reduction"] == "none" else 1, device=dev)
            st["lse"] = torch.empty(T, device=dev)
            st["call"] = tg.PreparedXent(ctx, d, st["X"], st["W"], st["y"], st["lse"], stream, loss=st["loss"])
        else:
            st["dX"] = torch.empty(T, H, dtype=DT[c["grad"]], device=dev)
            st["dW"] = torch.empty(V, H, dtype=DT[c["grad"]], device=dev)
            st["call"] = tg.PreparedXent(ctx, d, st["X"], st["W"], st["y"], st["lse"], stream, grad=st["g"],
                                         dX=st["dX"], dW=st["dW"])
    return st


def plain_choice(c, l, valid):
    """ids [T, k], weights [T, k], softmax [T, E], lse [T] and the tokens that count, from logits in 32 bits."""
    big = l.amax(1, True)
    counted = (big[:, 0] > -math.inf) if valid is None else (big[:, 0] > -math.inf) & (valid != 0)
    e = torch.exp(l - torch.where(big == -math.inf, 0.0, big))
    s = e.sum(1, keepdim=True)
    p = e / torch.where(s == 0, 1.0, s)
    lse = big[:, 0] + torch.log(s[:, 0])
    # a stable sort keeps equal ones in the order of their index
    val, ids = torch.sort(l, dim=1, descending=True, stable=True)
    val, ids = val[:, :c["k"]], ids[:, :c["k"]]
    none = (val == -math.inf) | ~counted[:, None]
    w = torch.where(none, 0.0, p.gather(1, ids))
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total == 0, 1.0, total)
    return torch.where(none, -1, ids).to(torch.int32), w, p, torch.where(counted, lse, 0.0), counted


def plain_counts(c, ids, counted):
    counts = torch.zeros(c["E"] + 1, dtype=torch.int32, device=ids.device)
    counts.scatter_add_(0, torch.where(ids < 0, c["E"], ids).flatten().long(),
                        torch.ones(ids.numel(), dtype=torch.int32, device=ids.device))
    counts[c["E"]] = counted.sum()
    return counts


def prepare_route(c, g):
    T, E, k, dev = c["T"], c["E"], c["k"], "cuda"
    st = {"case": c}
    # logits of a router that favours some experts
    l = torch.randn(T, E, device=dev, generator=g) * 1.5 + torch.randn(E, device=dev, generator=g) * 0.7
    if c["masked"]:
        # experts that a token may not take; some tokens keep fewer than k, a few none
        share = torch.rand(T, 1, device=dev, generator=g) * 1.1
        l = torch.where(torch.rand(T, E, device=dev, generator=g) < share - 0.1, -math.inf, l)
    st["l"] = padded_rows(l, DT[c["x"]], c["pad"])
    st["valid"] = None
    if c["padded"]:
        # sequences of 512 whose ends are padding
        ends = torch.randint(256, 513, (-(-T // 512),), device=dev, generator=g)
        at = torch.arange(T, device=dev)
        st["valid"] = (at % 512 < ends[at // 512]).to(torch.uint8)
    if c["kind"] == "route gradients":
        st["ids"], _, _, _, counted = plain_choice(c, st["l"].float(), st["valid"])
        st["counts"] = plain_counts(c, st["ids"], counted)
        st["gw"] = torch.randn(T, k, device=dev, generator=g) / T
        st["gl"] = torch.tensor([1e-2, 1e-3], device=dev) * (0.5 + torch.rand(2, device=dev, generator=g))
    if own:
        tg, ctx, stream = user()
        d = tg.make_route_desc(T, E, k, c["x"], c["grad"], renormalize=c["renorm"], ld_logits=st["l"].stride(0))
        if c["kind"] == "route":
            st["ids"] = torch.empty(T, k, dtype=torch.int32, device=dev)
            st["w"] = torch.empty(T, k, device=dev)
            st["counts"] = torch.empty(E + 1, dtype=torch.int32, device=dev)
            st["losses"] = torch.empty(2, device=dev)
            st["call"] = tg.PreparedRoute(ctx, d, st["l"], st["ids"], st["counts"], stream, valid=st["valid"],
                                          weights=st["w"], losses=st["losses"])
        else:
            st["dl"] = torch.empty(T, E, dtype=DT[c["grad"]], device=dev)
            st["call"] = tg.PreparedRoute(ctx, d, st["l"], st["ids"], st["counts"], stream, valid=st["valid"],
                                          grad_weights=st["gw"], grad_losses=st["gl"], dlogits=st["dl"])
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (prepare_xent if case["kind"] in ("loss", "gradients") else prepare_route)(case, g)


# --------------------------------------------------------------- plain form

def plain_loss(c, st):
    l = c["scale"] * (st["X"].float() @ st["W"].float().t())
    big = l.amax(1)
    lse = big + torch.log(torch.exp(l - big[:, None]).sum(1))
    y = st["y"].long()
    counted = (y >= 0) & (y < c["V"])
    at = l.gather(1, torch.where(counted, y, 0)[:, None])[:, 0]
    loss = torch.where(counted, lse - at + c["z"] * lse * lse, 0.0)
    if c["reduction"] != "none":
        loss = loss.double().sum().reshape(1)
        if c["reduction"] == "mean":
            loss = loss / counted.sum().clamp(min=1)
    return {"loss": loss.float(), "lse": lse}


def plain_gradients(c, st):
    x, w, lse = st["X"].float(), st["W"].float(), st["lse"]
    y = st["y"].long()
    counted = (y >= 0) & (y < c["V"])
    g = st["g"] / counted.sum().clamp(min=1) if c["reduction"] == "mean" else st["g"]
    g = torch.where(counted, g, 0.0)
    G = torch.exp(c["scale"] * (x @ w.t()) - lse[:, None])
    G *= (1 + 2 * c["z"] * lse)[:, None]
    G[torch.arange(c["T"], device=x.device), torch.where(counted, y, 0)] -= 1.0
    G = torch.where(counted[:, None], G * g[:, None], 0.0)
    dX, dW = c["scale"] * (G @ w), c["scale"] * (G.t() @ x)
    return {"dX": dX.to(DT[c["grad"]]), "dW": dW.to(DT[c["grad"]])}


def plain_route(c, st):
    ids, w, p, lse, counted = plain_choice(c, st["l"].float(), st["valid"])
    counts = plain_counts(c, ids, counted)
    n = counted.sum().clamp(min=1)
    mean = torch.where(counted[:, None], p, 0.0).double().sum(0) / n
    balance = c["E"] * (counts[:-1] / (n * c["k"]) * mean).sum()
    z = (lse.double() ** 2).sum() / n
    return {"ids": ids, "weights": w, "counts": counts, "losses": torch.stack([balance, z]).float()}


def plain_route_gradients(c, st):
    _, w, p, lse, counted = plain_choice(c, st["l"].float(), st["valid"])
    n = st["counts"][-1].clamp(min=1)
    f = st["counts"][:-1] / (n * c["k"]).float()
    dl = st["gl"][0] * (c["E"] / n) * p * (f - (f * p).sum(1, keepdim=True)) + st["gl"][1] * (2 / n) * lse[:, None] * p
    ids, gw = st["ids"].long(), st["gw"]
    taken = ids >= 0
    dot = (gw * w).sum(1, keepdim=True)
    if c["renorm"]:
        dl.scatter_add_(1, ids.clamp(min=0), torch.where(taken, w * (gw - dot), 0.0))
    else:
        dl.scatter_add_(1, ids.clamp(min=0), torch.where(taken, w * gw, 0.0))
        dl -= p * dot
    return torch.where(counted[:, None], dl, 0.0).to(DT[c["grad"]])


def run(state):
    c, st = state["case"], state
    kind = c["kind"]
    if not own:
        return {"loss": plain_loss, "gradients": plain_gradients, "route": plain_route,
                "route gradients": plain_route_gradients}[kind](c, st)
    if kind in ("loss", "route"):
        st["call"].enqueue()
    else:
        st["call"].enqueue_backward()
    if kind == "loss":
        return {"loss": st["loss"], "lse": st["lse"]}
    if kind == "gradients":
        return {"dX": st["dX"], "dW": st["dW"]}
    if kind == "route":
        return {"ids": st["ids"], "weights": st["w"], "counts": st["counts"], "losses": st["losses"]}
    return st["dl"]


# -------------------------------------------------------------------- work

def work(case):
    c = case
    if c["kind"] in ("loss", "gradients"):
        T, H, V = c["T"], c["H"], c["V"]
        read = 2 * H * (T + V) + T * (8 if c["wide"] else 4) + 4 * T
        if c["kind"] == "loss":
            return {"bytes": read + 4 * T, "flops": 2.0 * T * H * V}
        # the logits again, as none are kept, and one product for each gradient
        return {"bytes": read + ES[c["grad"]] * H * (T + V), "flops": 6.0 * T * H * V}
    T, E, k = c["T"], c["E"], c["k"]
    move = T * E * ES[c["x"]] + 8 * T * k + (T if c["padded"] else 0) + 4 * E
    return {"bytes": move + (T * E * ES[c["grad"]] if c["kind"] == "route gradients" else 0), "flops": 6.0 * T * E}


# ---------------------------------------------------- the definition, 64 bits

def exact_xent(c, st):
    T, V, k = c["T"], c["V"], c["scale"]
    y = st["y"].to(torch.int64)
    rows = torch.nonzero((y >= 0) & (y < V))[:, 0]
    if c["kind"] == "loss":
        best = torch.full((T,), -math.inf, dtype=torch.float64, device=y.device)
        total, X = torch.zeros_like(best), st["X"].double()
        for a, b in pieces(V, 8192):
            l = k * torch.mm(X, st["W"][a:b].double().t())
            new = torch.maximum(best, l.max(1).values)
            total = total * torch.exp(best - new) + torch.exp(l - new[:, None]).sum(1)
            best = new
        lse = best + torch.log(total)
        loss = torch.zeros_like(lse)
        at = k * (X[rows] * st["W"].index_select(0, y[rows]).double()).sum(1)
        loss[rows] = lse[rows] - at + c["z"] * lse[rows] ** 2
        if c["reduction"] == "sum":
            loss = loss.sum(0, keepdim=True)
        elif c["reduction"] == "mean":
            loss = loss.sum(0, keepdim=True) / max(1, rows.numel())
        return {"loss": loss, "lse": lse}
    # only the counted rows take part
    X, lse, hot = st["X"][rows].double(), st["lse"][rows].double(), y[rows]
    g = st["g"].double()
    g = g[rows] if c["reduction"] == "none" else g.expand(rows.numel()) / (rows.numel() if c["reduction"] == "mean" else 1)
    dX = torch.zeros_like(X)
    dW = torch.empty(V, c["H"], dtype=torch.float64, device=y.device)
    for a, b in pieces(V, 8192):
        W = st["W"][a:b].double()
        G = torch.exp(k * torch.mm(X, W.t()) - lse[:, None]) * (g * (1 + 2 * c["z"] * lse))[:, None]
        here = torch.nonzero((hot >= a) & (hot < b))[:, 0]
        G[here, hot[here] - a] -= g[here]
        dX += k * torch.mm(G, W)
        dW[a:b] = k * torch.mm(G.t(), X)
    out = torch.zeros(T, c["H"], dtype=torch.float64, device=y.device)
    out[rows] = dX
    return {"dX": out, "dW": dW}


def exact_route(c, st):
    T, E, k = c["T"], c["E"], c["k"]
    l = st["l"].double()
    counted = (l > -math.inf).any(1)
    if st["valid"] is not None:
        counted &= st["valid"].bool()
    rows = torch.nonzero(counted)[:, 0]
    n = max(1, rows.numel())
    l = l[rows]
    lse = torch.logsumexp(l, 1)
    p = torch.exp(l - lse[:, None])
    if c["kind"] == "route":
        # the rank of an expert: those above it, and equal ones before it
        w = torch.zeros(T, k, dtype=torch.float64, device=l.device)
        counts = torch.zeros(E, dtype=torch.float64, device=l.device)
        left, some = l.clone(), []
        for j in range(k):
            e = left.argmax(1)
            got = left.gather(1, e[:, None])[:, 0] > -math.inf
            some.append(torch.where(got, p.gather(1, e[:, None])[:, 0], 0.0))
            counts += torch.bincount(e[got], minlength=E)
            left.scatter_(1, e[:, None], -math.inf)
        some = torch.stack(some, 1)
        w[rows] = some / some.sum(1, keepdim=True) if c["renorm"] else some
        balance = E * (counts / (n * k) * p.sum(0) / n).sum()
        return {"ids": None, "weights": w, "counts": None, "losses": torch.stack([balance, (lse ** 2).sum() / n])}
    f = st["counts"][:E].double() / (n * k)
    gb, gz = st["gl"].double()
    ids, gw = st["ids"][rows].to(torch.int64), st["gw"][rows].double()
    # the derivative of the sum of gw w, through a [tokens, experts] matrix of the arriving gradients
    hit = torch.nn.functional.one_hot(ids.clamp(min=0), E).double() * (ids >= 0)[..., None] if rows.numel() * k * E < 4e8 \
        else None
    if hit is not None:
        at, mask = (hit * gw[..., None]).sum(1), hit.sum(1)
    else:
        at, mask = torch.zeros_like(p), torch.zeros_like(p)
        for j in range(k):
            ok = torch.nonzero(ids[:, j] >= 0)[:, 0]
            at[ok, ids[ok, j]] += gw[ok, j]
            mask[ok, ids[ok, j]] = 1.0
    q = p * mask
    if c["renorm"]:
        q = q / q.sum(1, keepdim=True)
        through = q * (at - (q * at).sum(1, keepdim=True))
    else:
        through = p * (at - (p * at).sum(1, keepdim=True))
    mean = (f[None, :] * p).sum(1, keepdim=True)
    out = torch.zeros(T, E, dtype=torch.float64, device=l.device)
    out[rows] = through + gb * E / n * p * (f[None, :] - mean) + gz * 2 / n * lse[:, None] * p
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return (exact_xent if case["kind"] in ("loss", "gradients") else exact_route)(case, st)
