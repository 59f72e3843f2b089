"""Timed cases of what a training step needs around the experts' MLP: the router
that feeds it, the layer norm in front of it, and the update of its weights.

  router  softmax over the experts, the top_k of a token and their weights, how many
          slots each expert gets and the balance loss; the logits' gradient
  norm    layer norm of x (+ residual), and its gradients
  ortho   an update made orthogonal by Newton-Schulz products: X = G / |G|, then
          X <- a X + (b A + c A A) X with A = X X^T, `steps` times

`own` picks the library's kernels; otherwise `run` computes the same in
elementary torch operations in fp32, rounded once at the end.
"""
import math

import torch

own = False

BF = torch.bfloat16
F32 = torch.float32
TYPES = {"bf16": BF, "fp32": F32}
COEFFS = (3.4445, -4.7750, 2.0315)
EPS_NORM, EPS_ORTHO = 1e-5, 1e-7
LOSS_SCALE = 0.01  # the balance loss's share in a model's loss


def listed():
    return [
        # one token's routing in a model with many narrow experts: latency
        dict(name="router_one_token", op="router", T=1, E=64, k=8, t="bf16", w="fp32", renorm=True,
             pad=0.0, block=0.0, train=False),
        # a serving batch
        dict(name="router_serving", op="router", T=48, E=64, k=4, t="fp32", w="fp32", renorm=False,
             pad=0.0, block=0.0, train=False),
        # an odd batch with padding tokens, balance loss and gradient
        dict(name="router_padded", op="router", T=4099, E=60, k=4, t="bf16", w="bf16", renorm=True,
             pad=0.2, block=0.0, train=True),
        # a large training batch over many experts, balance loss and gradient
        dict(name="router_train", op="router", T=131072, E=256, k=8, t="fp32", w="fp32",
             renorm=True, pad=0.0, block=0.0, train=True),
        # one token between two layers: latency
        dict(name="norm_one_token", op="norm", M=1, H=4096, t="bf16", w="bf16", residual=True,
             bias=True, train=False),
        # a ragged prompt of a 2048-wide model
        dict(name="norm_prompt", op="norm", M=777, H=2048, t="bf16", w="fp32", residual=False,
             bias=True, train=False),
        # a training batch of a 4096-wide model, residual sum in front, every gradient
        dict(name="norm_train", op="norm", M=8192, H=4096, t="bf16", w="fp32", residual=True,
             bias=True, train=True),
        # an fp32 residual stream of an odd width, no bias, every gradient
        dict(name="norm_fp32", op="norm", M=4097, H=4872, t="fp32", w="fp32", residual=False,
             bias=False, train=True),
        # the update of a router's weights
        dict(name="ortho_router", op="ortho", B=1, m=64, n=2048, t="bf16", out="bf16", steps=5),
        # the updates of a layer's experts, a stack, from fp32 momenta
        dict(name="ortho_experts", op="ortho", B=16, m=1408, n=2048, t="fp32", out="bf16", steps=5),
        # a tall fc1, with an fp32 update
        dict(name="ortho_tall", op="ortho", B=1, m=4864, n=2048, t="fp32", out="fp32", steps=5),
        # the widest model's down projection
        dict(name="ortho_largest", op="ortho", B=1, m=4096, n=14336, t="bf16", out="bf16", steps=5),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    return max(lo, _log_int(rng, lo, hi) // 8 * 8)


def draw(rng):
    op = rng.choice(["router", "norm", "ortho"])
    train = rng.random() < 0.6
    t = rng.choice(["bf16", "fp32"])
    while True:
        if op == "router":
            E = rng.choice([4, 8, 16, 60, 64, 128, 160, 256, 384])
            c = dict(op=op, T=_log_int(rng, 1, 131072), E=E, k=rng.randint(1, min(8, E)), t=t,
                     w=rng.choice(["bf16", "fp32"]), renorm=rng.random() < 0.6,
                     pad=rng.choice([0.0, 0.0, 0.3]), block=rng.choice([0.0, 0.0, 0.5]),
                     train=train)
            fits = c["T"] * E <= 131072 * 256
        elif op == "norm":
            c = dict(op=op, M=_log_int(rng, 1, 16384), H=_width(rng, 64, 14336), t=t,
                     w="fp32" if t == "fp32" else rng.choice(["bf16", "fp32"]),
                     residual=rng.random() < 0.5, bias=rng.random() < 0.7, train=train)
            fits = c["M"] * c["H"] * (2 if t == "bf16" else 4) <= 8192 * 4096 * 2
        else:
            c = dict(op=op, B=rng.choice([1, 1, 1, 4, 8]), m=_width(rng, 64, 8192),
                     n=_width(rng, 64, 14336), t=t, out=rng.choice(["bf16", "bf16", "fp32"]),
                     steps=5)
            fits = work(c)["flops"] <= 1.5e12
        if fits:
            return c


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rn = lambda *z: torch.randn(z, generator=gen, device=dev, dtype=F32)  # noqa: E731
    s = dict(case)
    dt = TYPES[case["t"]]
    if case["op"] == "router":
        T, E, k = case["T"], case["E"], case["k"]
        logits = 1.2 * rn(T, E) + 0.6 * rn(1, E)
        if case["block"]:  # experts that a token may not use (often fewer than k are left)
            logits[torch.rand((T, E), generator=gen, device=dev) < case["block"]] = -math.inf
        s["logits"] = logits.to(dt)
        s["mask"] = None
        if case["pad"]:
            s["mask"] = torch.rand((T,), generator=gen, device=dev) >= case["pad"]
        s["dweights"] = rn(T, k).to(TYPES[case["w"]]) if case["train"] else None
        s["dloss"] = torch.full((1,), LOSS_SCALE, device=dev) if case["train"] else None
        return s
    if case["op"] == "norm":
        M, H = case["M"], case["H"]
        wt = TYPES[case["w"]]
        s["x"] = (rn(M, H) * 1.5 + 0.25 * rn(M, 1)).to(dt)
        s["r"] = rn(M, H).to(dt) if case["residual"] else None
        s["weight"] = (1 + 0.2 * rn(H)).to(wt)
        s["bias"] = (0.2 * rn(H)).to(wt) if case["bias"] else None
        s["dy"] = rn(M, H).to(dt) if case["train"] else None
        s["dh"] = rn(M, H).to(dt) if case["train"] and case["residual"] else None
        return s
    B, m, n = case["B"], case["m"], case["n"]
    r = max(1, min(m, n) // 8)  # a momentum: a few strong directions over noise
    low = torch.bmm(rn(B, m, r) * torch.logspace(0, -1.5, r, device=dev), rn(B, r, n))
    s["G"] = (1e-3 * (low / math.sqrt(r) + 0.3 * rn(B, m, n))).to(dt)
    return s


# ---------------------------------------------------------------- run

def run(s):
    if s["op"] == "router":
        return _own_router(s) if own else _router(s)
    if s["op"] == "norm":
        return _own_norm(s) if own else _norm(s)
    return _own_ortho(s) if own else _ortho(s)


def _own_router(s):
    import activated_mlp_gemms_gb300 as m
    logits, T, E, k = s["logits"], s["T"], s["E"], s["k"]
    dev, wt = logits.device, TYPES[s["w"]]
    p = m.router(T, E, k, s["renorm"], logits_dtype=logits.dtype, weights_dtype=wt)
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    weights = torch.empty((T, k), dtype=wt, device=dev)
    if not s["train"]:
        m.mlp_moe_router_fwd(p, logits, s["mask"], ids, weights)
        return {"ids": ids, "weights": weights}
    counts = torch.empty((E,), dtype=torch.int32, device=dev)
    balance = torch.empty((E + 1,), dtype=F32, device=dev)
    dlogits = torch.empty_like(logits)
    m.mlp_moe_router_fwd(p, logits, s["mask"], ids, weights, counts, balance)
    m.mlp_moe_router_bwd(p, logits, s["mask"], ids, balance, s["dweights"], s["dloss"], dlogits)
    return {"ids": ids, "weights": weights, "counts": counts, "loss": balance[:1],
            "dlogits": dlogits}


def _own_norm(s):
    import activated_mlp_gemms_gb300 as m
    x, r, w, b, M, H = s["x"], s["r"], s["weight"], s["bias"], s["M"], s["H"]
    p = m.layernorm(M, H, EPS_NORM, dtype=x.dtype, weight_dtype=w.dtype)
    y = torch.empty_like(x)
    h = torch.empty_like(x) if r is not None else None
    if not s["train"]:
        m.mlp_layernorm_fwd(p, x, r, w, b, y, h)
        return {"y": y, "h": h}
    mean = torch.empty((M,), dtype=F32, device=x.device)
    rstd = torch.empty_like(mean)
    m.mlp_layernorm_fwd(p, x, r, w, b, y, h, mean, rstd)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    db = torch.empty_like(b) if b is not None else None
    m.mlp_layernorm_bwd(p, s["dy"], x if h is None else h, w, mean, rstd, s["dh"], dx, dw, db)
    return {"y": y, "h": h, "dx": dx, "dw": dw, "db": db}


def _own_ortho(s):
    import activated_mlp_gemms_gb300 as m
    G = s["G"]
    p = m.ortho(s["m"], s["n"], s["B"], steps=s["steps"], coeffs=COEFFS, eps=EPS_ORTHO,
                dtype=G.dtype, out_dtype=TYPES[s["out"]])
    out = torch.empty(G.shape, dtype=TYPES[s["out"]], device=G.device)
    m.mlp_orthogonalize(p, G, out)
    return {"out": out}


# ---------------------------------------------------------------- plain forms (fp32)

def _router(s):
    T, E, k = s["T"], s["E"], s["k"]
    raw, wt = s["logits"], TYPES[s["w"]]
    l = raw.float()
    top = l.max(1, keepdim=True)[0]
    routed = (top > -math.inf).squeeze(1)
    if s["mask"] is not None:
        routed = routed & s["mask"]
    row = routed.unsqueeze(1)
    e = torch.exp(l - torch.where(top > -math.inf, top, 0.0)) * row
    p = e / torch.where(row, e.sum(1, keepdim=True), 1.0)
    best, ids = torch.sort(l, dim=1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k]
    taken = row & (best > -math.inf)
    pick = torch.gather(p, 1, ids) * taken
    total = pick.sum(1, keepdim=True)
    w = pick / torch.where(row, total, 1.0) if s["renorm"] else pick
    res = {"ids": torch.where(taken, ids, -1).to(torch.int32), "weights": w.to(wt)}
    if not s["train"]:
        return res
    counts = torch.zeros((E + 1,), dtype=torch.int64, device=l.device)
    slot = torch.where(taken, ids, E)
    counts.scatter_add_(0, slot.reshape(-1), torch.ones_like(slot).reshape(-1))
    counts = counts[:E]
    N = routed.sum().double().clamp(min=1)
    coef = (E * counts.double() / (k * N * N)).float()
    loss = (coef.double() * p.sum(0, dtype=torch.float64)).sum().float().reshape(1)
    # gradient
    dw = s["dweights"].float() * taken
    g = (coef * s["dloss"]).expand(T, E)
    if s["renorm"]:
        dl = p * (g - (p * g).sum(1, keepdim=True))
        dl = dl.scatter_add(1, ids, w * (dw - (w * dw).sum(1, keepdim=True)))
    else:
        g = g.scatter_add(1, ids, dw)
        dl = p * (g - (p * g).sum(1, keepdim=True))
    res.update(counts=counts.to(torch.int32), loss=loss, dlogits=dl.to(raw.dtype))
    return res


def _norm(s):
    x, r, H = s["x"], s["r"], s["H"]
    w, b = s["weight"].float(), s["bias"]
    h = None if r is None else (x.float() + r.float()).to(x.dtype)
    z = (x if h is None else h).float()
    mean = z.sum(1, keepdim=True) / H
    d = z - mean
    rstd = 1 / torch.sqrt((d * d).sum(1, keepdim=True) / H + EPS_NORM)
    xhat = d * rstd
    y = xhat * w if b is None else xhat * w + b.float()
    res = {"y": y.to(x.dtype), "h": h}
    if not s["train"]:
        return res
    dy = s["dy"].float()
    g = dy * w
    dx = rstd * (g - g.sum(1, keepdim=True) / H - xhat * ((g * xhat).sum(1, keepdim=True) / H))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    res.update(dx=dx.to(x.dtype), dw=(dy * xhat).sum(0).to(s["weight"].dtype),
               db=None if b is None else dy.sum(0).to(b.dtype))
    return res


def _ortho(s):
    a, b, c = COEFFS
    X = s["G"].float()
    tall = s["m"] > s["n"]
    if tall:
        X = X.transpose(1, 2)
    X = X / (torch.sqrt((X * X).sum((1, 2), keepdim=True)) + EPS_ORTHO)
    for _ in range(s["steps"]):
        A = torch.bmm(X, X.transpose(1, 2))
        X = a * X + torch.bmm(b * A + c * torch.bmm(A, A), X)
    if tall:
        X = X.transpose(1, 2)
    return {"out": X.to(TYPES[s["out"]]).contiguous()}


# ---------------------------------------------------------------- work

def work(case):
    size = {"bf16": 2, "fp32": 4}
    tb = size[case["t"]]
    if case["op"] == "router":
        T, E, k = case["T"], case["E"], case["k"]
        io = T * E * tb + T * k * (4 + size[case["w"]]) + (T if case["pad"] else 0)
        flops = 5.0 * T * E
        if case["train"]:  # dweights in; dlogits, counts, loss out
            io += T * k * size[case["w"]] + T * E * tb + 4 * E + 8
            flops += 6.0 * T * E
        return {"bytes": io, "flops": flops}
    if case["op"] == "norm":
        M, H = case["M"], case["H"]
        mh, hw = M * H * tb, H * size[case["w"]]
        vecs = hw * (2 if case["bias"] else 1)
        io = mh * (4 if case["residual"] else 2) + vecs
        flops = 8.0 * M * H
        if case["train"]:  # dy, dh in; dx, dw, db out
            io += mh * (3 if case["residual"] else 2) + vecs
            flops += 14.0 * M * H
        return {"bytes": io, "flops": flops}
    B, m, n = case["B"], min(case["m"], case["n"]), max(case["m"], case["n"])
    # X X^T and A A are symmetric: half of each
    return {"bytes": B * m * n * (tb + size[case["out"]]),
            "flops": float(B) * case["steps"] * (3.0 * m * m * n + 1.0 * m ** 3)}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_router(s, case):
    T, E, k = case["T"], case["E"], case["k"]
    z = s["logits"].double()
    dev = z.device
    keep = torch.isfinite(z).any(1)
    if s["mask"] is not None:
        keep &= s["mask"]
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    p[~keep] = 0
    # the best expert left, the first of equals, k times
    left = z.clone()
    left[~keep] = -math.inf
    number = torch.arange(E, device=dev).expand(T, E)
    ids = torch.full((T, k), -1, dtype=torch.int64, device=dev)
    for j in range(k):
        m = left.amax(1)
        some = m > -math.inf
        first = torch.where(left == m[:, None], number, E).amin(1)
        ids[:, j] = torch.where(some, first, -1)
        left.scatter_(1, first.clamp(max=E - 1)[:, None], -math.inf)
    has = ids >= 0
    chosen = torch.zeros((T, E), dtype=torch.bool, device=dev)
    t, j = torch.nonzero(has, as_tuple=True)
    chosen[t, ids[t, j]] = True
    scale = torch.ones((T, 1), dtype=torch.float64, device=dev)
    if case["renorm"]:
        scale = (p * chosen).sum(1, keepdim=True).reciprocal()
        scale[~keep] = 0
    full = p * chosen * scale  # weights laid out by expert
    w = torch.zeros((T, k), dtype=torch.float64, device=dev)
    w[t, j] = full[t, ids[t, j]]
    res = {"ids": ids.to(torch.int32), "weights": w}
    if not case["train"]:
        return res
    counts = chosen.sum(0)
    N = max(int(keep.sum()), 1)
    f, P = counts.double() / (k * N), p.sum(0) / N
    # gradient through the softmax's Jacobian, by the chain rule over probabilities
    dfull = torch.zeros((T, E), dtype=torch.float64, device=dev)
    dfull[t, ids[t, j]] = s["dweights"].double()[t, j]
    dp = float(s["dloss"]) * E * f[None, :] / N + torch.zeros_like(p)
    if case["renorm"]:
        dp = dp + chosen * scale * (dfull - (dfull * full).sum(1, keepdim=True))
    else:
        dp = dp + dfull
    dz = p * dp - p * (p * dp).sum(1, keepdim=True)
    res.update(counts=counts.to(torch.int32), loss=(E * (f * P).sum()).reshape(1), dlogits=dz)
    return res


def _exact_norm(s, case):
    # (the sum that is normed is the stored one, in x's type)
    h = None
    z = s["x"].double()
    if s["r"] is not None:
        h = z + s["r"].double()
        z = (s["x"].float() + s["r"].float()).to(s["x"].dtype).double()
    z.requires_grad_(case["train"])
    w = s["weight"].double().requires_grad_(case["train"])
    b = None if s["bias"] is None else s["bias"].double().requires_grad_(case["train"])
    var, mean = torch.var_mean(z, 1, unbiased=False, keepdim=True)
    y = (z - mean) * torch.rsqrt(var + EPS_NORM) * w
    if b is not None:
        y = y + b
    res = {"y": y.detach(), "h": h}
    if case["train"]:
        leaves = [z, w] + ([] if b is None else [b])
        g = torch.autograd.grad(y, leaves, s["dy"].double())
        res.update(dx=g[0] if s["dh"] is None else g[0] + s["dh"].double(), dw=g[1],
                   db=g[2] if b is not None else None)
    return res


def _exact_ortho(s, case):
    a, b, c = COEFFS
    outs = []
    for G in s["G"]:
        X = G.double()
        X = X / (torch.linalg.norm(X) + EPS_ORTHO)
        for _ in range(case["steps"]):
            if case["m"] <= case["n"]:
                A = X @ X.t()
                X = a * X + (b * A + c * (A @ A)) @ X
            else:
                A = X.t() @ X
                X = a * X + X @ (b * A + c * (A @ A))
        outs.append(X)
    return {"out": torch.stack(outs)}


def exact(case, seed):
    s = prepare(case, seed)
    f = {"router": _exact_router, "norm": _exact_norm, "ortho": _exact_ortho}[case["op"]]
    return f(s, case)
