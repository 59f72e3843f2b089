"""Timed cases of the linear layer with its epilogue, of the token sort by
expert, and of the mixture-of-experts MLP built on both.

  linear   out = act(x W^T + bias) + resid_scale * residual, and its gradients
  tokens   tokens sorted by expert (every expert's rows begin at a multiple of
           16), gathered, and summed back with their routing weights; its
           gradient (dy, dweights, dx)
  experts  the whole mixture-of-experts MLP: sort, gather, each expert's MLP
           over its own rows, weighted sum back; its gradients

`own` picks the library's kernels; otherwise `run` computes the same in
elementary torch operations in fp32, rounded once at the end.
"""
import math

import torch

own = False

BF = torch.bfloat16
ROW_ALIGN = 16
GATED = ("swiglu", "reglu", "geglu", "glu")


def listed():
    return [
        # one token through a wide bias + GELU layer: a weight stream
        dict(name="linear_one_token", op="linear", M=1, N=14336, K=4096, act="gelu_tanh_approx",
             bias=True, residual=False, train=False),
        # the smallest call: a few tokens through a square output layer with its residual
        dict(name="linear_smallest", op="linear", M=3, N=768, K=768, act="none", bias=True,
             residual=True, train=False),
        # a ragged prompt through fc1 of a 2048-wide model
        dict(name="linear_prompt", op="linear", M=777, N=4864, K=2048, act="relu_sq", bias=True,
             residual=False, train=False),
        # the widest model's output projection with bias and residual, a full training batch
        dict(name="linear_largest", op="linear", M=8192, N=4096, K=14336, act="none", bias=True,
             residual=True, train=False),
        # a training step of a biased GELU fc1 with every gradient
        dict(name="linear_train", op="linear", M=8192, N=4864, K=2048, act="gelu_tanh_approx",
             bias=True, residual=False, train=True),
        # a serving batch's tokens to 64 experts and back
        dict(name="tokens_serving", op="tokens", T=16, E=64, k=8, H=2048, drop=0.0, w="fp32",
             residual=True, train=False),
        # an odd prompt with slots dropped over capacity, forward and gradient
        dict(name="tokens_dropped", op="tokens", T=4099, E=8, k=2, H=4096, drop=0.1, w="bf16",
             residual=False, train=True),
        # a training batch over many experts, forward and gradient
        dict(name="tokens_train", op="tokens", T=8192, E=64, k=8, H=2048, drop=0.0, w="fp32",
             residual=False, train=True),
        # one token of a model with many narrow experts
        dict(name="experts_one_token", op="experts", T=1, E=64, k=8, H=2048, I=1408, act="swiglu",
             skew=0.5, w="fp32", train=False),
        # a serving batch: nearly every expert is touched by a few tokens
        dict(name="experts_serving", op="experts", T=48, E=64, k=4, H=4096, I=1792, act="swiglu",
             skew=0.5, w="fp32", train=False),
        # a long prompt over a few wide experts
        dict(name="experts_prompt", op="experts", T=4097, E=8, k=2, H=4096, I=14336, act="swiglu",
             skew=0.3, w="fp32", train=False),
        # a training step with an uneven load and every gradient
        dict(name="experts_train", op="experts", T=8192, E=16, k=2, H=2048, I=4864, act="swiglu",
             skew=0.5, w="bf16", train=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    return max(lo, _log_int(rng, lo, hi) // 8 * 8)


def draw(rng):
    op = rng.choice(["linear", "tokens", "experts"])
    train = rng.random() < 0.4
    while True:
        if op == "linear":
            c = dict(op=op, M=_log_int(rng, 1, 8192), N=_width(rng, 256, 14336),
                     K=_width(rng, 256, 14336),
                     act=rng.choice(["none", "relu", "relu_sq", "gelu_tanh_approx", "silu"]),
                     bias=rng.random() < 0.8, residual=rng.random() < 0.4, train=train)
            fits = work(c)["flops"] <= 2.0 * 8192 * 4096 * 14336
        elif op == "tokens":
            E = rng.choice([4, 8, 16, 60, 64, 128])
            c = dict(op=op, T=_log_int(rng, 1, 8192), E=E, k=rng.randint(1, min(8, E)),
                     H=_width(rng, 256, 4096), drop=rng.choice([0.0, 0.0, 0.1, 0.5]),
                     w=rng.choice(["fp32", "bf16"]), residual=rng.random() < 0.5, train=train)
            fits = work(c)["bytes"] <= 1.4e9
        else:
            E = rng.choice([4, 8, 16, 60, 64])
            c = dict(op=op, T=_log_int(rng, 1, 8192), E=E, k=rng.randint(1, min(8, E)),
                     H=_width(rng, 256, 4096), I=_width(rng, 256, 4864),
                     act=rng.choice(["swiglu", "swiglu", "reglu", "geglu", "relu_sq",
                                     "gelu_tanh_approx"]),
                     skew=rng.choice([0.0, 0.5, 1.5]), w="bf16" if train else "fp32", train=train)
            fits = (work(c)["flops"] <= 2.8e12 and E * c["H"] * c["I"] <= 5e8)
        if fits:
            return c


# ---------------------------------------------------------------- inputs

def _routes(gen, T, E, k, skew, drop, dev):
    """Distinct experts per token from skewed logits, best first, and their softmax weights."""
    logits = torch.randn((T, E), generator=gen, device=dev)
    logits += skew * torch.randn((1, E), generator=gen, device=dev)
    top, ids = torch.topk(logits, k, dim=-1)
    ids = ids.to(torch.int32)
    if drop:
        ids = torch.where(torch.rand((T, k), generator=gen, device=dev) < drop, -1, ids)
    return ids.contiguous(), torch.softmax(top, -1)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=gen, device=dev, dtype=torch.float32)  # noqa: E731

    def uni(fan_in, *s):
        return ((torch.rand(s, generator=gen, device=dev) * 2 - 1) / math.sqrt(fan_in)).to(BF)

    s = dict(case)
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = rn(M, K).to(BF)
        s["W"] = uni(K, N, K)
        s["b"] = uni(K, N) if case["bias"] else None
        s["r"] = rn(M, N).to(BF) if case["residual"] else None
        s["dout"] = rn(M, N).to(BF) if case["train"] else None
        return s
    T, E, k, H = case["T"], case["E"], case["k"], case["H"]
    ids, w = _routes(gen, T, E, k, case.get("skew", 0.5), case.get("drop", 0.0), dev)
    s["ids"], s["weights"] = ids, (w.to(BF) if case["w"] == "bf16" else w).contiguous()
    s["x"] = rn(T, H).to(BF)
    s["dout"] = rn(T, H).to(BF) if case["train"] else None
    if case["op"] == "tokens":
        rows = _rows(T, E, k)
        s["y"] = rn(rows, H).to(BF)      # the experts' outputs
        s["r"] = rn(T, H).to(BF) if case["residual"] else None
        s["dxs"] = rn(rows, H).to(BF) if case["train"] else None  # the gathered rows' gradient
        return s
    inner = case["I"]
    s["Wg"] = uni(H, E, inner, H)
    s["Wu"] = uni(H, E, inner, H) if case["act"] in GATED else None
    s["Wd"] = uni(inner, E, H, inner)
    return s


def _rows(T, E, k):
    """Rows of the sorted layout: every expert's rows rounded up to 16, at most."""
    n = T * k
    return (n + min(E, n) * (ROW_ALIGN - 1)) // ROW_ALIGN * ROW_ALIGN


# ---------------------------------------------------------------- run

def run(s):
    if s["op"] == "linear":
        return _own_linear(s) if own else _linear(s)
    if s["op"] == "tokens":
        return _own_tokens(s) if own else _tokens(s)
    return _own_experts(s) if own else _experts(s)


def _own_linear(s):
    import activated_mlp_gemms_gb300 as m
    x, W = s["x"], s["W"]
    M, N, K = s["M"], s["N"], s["K"]
    lin = m.linear(M, N, K, s["act"])
    out = torch.empty((M, N), dtype=BF, device=x.device)
    if not s["train"]:
        m.mlp_linear_fwd(lin, x, W, s["b"], s["r"], out)
        return {"out": out}
    pre = torch.empty_like(out) if s["act"] != "none" else None
    m.mlp_linear_fwd(lin, x, W, s["b"], s["r"], out, pre_save=pre)
    dx, dW = torch.empty_like(x), torch.empty_like(W)
    db = torch.empty_like(s["b"]) if s["b"] is not None else None
    m.mlp_linear_bwd(lin, s["dout"], x, W, pre, dx, dW, db)
    return {"out": out, "dx": dx, "dW": dW, "db": db}


def _own_tokens(s):
    import activated_mlp_gemms_gb300 as m
    T, H = s["T"], s["H"]
    x, y, dev = s["x"], s["y"], s["x"].device
    moe = m.moe(T, s["E"], s["k"], H, weights_dtype=s["weights"].dtype)
    plan = m.alloc_moe_plan(moe, dev)
    m.mlp_moe_sort(moe, s["ids"], plan)
    view = m.moe_plan_views(moe, plan)
    xs = torch.empty((m.mlp_moe_rows(moe), H), dtype=BF, device=dev)
    m.mlp_moe_dispatch(moe, plan, x, xs)
    out = torch.empty((T, H), dtype=BF, device=dev)
    m.mlp_moe_combine(moe, plan, y, s["weights"], s["r"], out)
    res = {"offsets": view["offsets"], "pos": view["pos"], "xs": xs, "out": out}
    if s["train"]:
        dy, dw, dx = torch.empty_like(y), torch.empty_like(s["weights"]), torch.empty_like(x)
        m.mlp_moe_combine_bwd(moe, plan, s["dout"], y, s["weights"], dy, dw)
        m.mlp_moe_dispatch_bwd(moe, plan, s["dxs"], dx)
        res.update(dy=dy, dweights=dw, dx=dx)
    return res


def _own_experts(s):
    import activated_mlp_gemms_gb300 as m
    T, E, k, H, inner = s["T"], s["E"], s["k"], s["H"], s["I"]
    x, w, Wg, Wu, Wd, dev = s["x"], s["weights"], s["Wg"], s["Wu"], s["Wd"], s["x"].device
    moe = m.moe(T, E, k, H, inner, s["act"], weights_dtype=w.dtype)
    out = torch.empty((T, H), dtype=BF, device=dev)
    if not s["train"]:
        m.mlp_moe_fwd_infer(moe, x, s["ids"], w, Wg, Wu, Wd, None, out)
        return {"out": out}
    rows = m.mlp_moe_rows(moe)
    new = lambda *z: torch.empty(z, dtype=BF, device=dev)  # noqa: E731
    plan = m.alloc_moe_plan(moe, dev)
    m.mlp_moe_sort(moe, s["ids"], plan)
    xs, y, G = new(rows, H), new(rows, H), new(rows, inner)
    U = new(rows, inner) if Wu is not None else None
    m.mlp_moe_dispatch(moe, plan, x, xs)
    m.mlp_moe_experts_fwd(moe, plan, xs, Wg, Wu, Wd, y, G, U)
    m.mlp_moe_combine(moe, plan, y, w, None, out)
    dy, dw, dxs, dx = new(rows, H), torch.empty_like(w), new(rows, H), new(T, H)
    m.mlp_moe_combine_bwd(moe, plan, s["dout"], y, w, dy, dw)
    dWg, dWd = torch.empty_like(Wg), torch.empty_like(Wd)
    dWu = torch.empty_like(Wu) if Wu is not None else None
    m.mlp_moe_experts_bwd(moe, plan, dy, xs, Wg, Wu, Wd, G, U, dxs, dWg, dWu, dWd)
    m.mlp_moe_dispatch_bwd(moe, plan, dxs, dx)
    return {"out": out, "dx": dx, "dweights": dw, "dWg": dWg, "dWu": dWu, "dWd": dWd}


# ---------------------------------------------------------------- plain forms (fp32)

def _act_grad(name, z):
    """act(z) and its derivative."""
    if name in ("silu", "swiglu"):
        q = 1 / (1 + torch.exp(-z))
        return z * q, q * (1 + z * (1 - q))
    if name == "glu":
        q = 1 / (1 + torch.exp(-z))
        return q, q * (1 - q)
    if name in ("relu", "reglu"):
        return z.clamp(min=0), (z > 0).to(z.dtype)
    if name == "relu_sq":
        r = z.clamp(min=0)
        return r * r, 2 * r
    if name in ("gelu_tanh_approx", "geglu"):
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 0.134145 * z * z)
    return z, torch.ones_like(z)


def _linear(s):
    x, W = s["x"].float(), s["W"].float()
    z = x @ W.t()
    if s["b"] is not None:
        z = z + s["b"].float()
    a, da = _act_grad(s["act"], z)
    out = (a if s["r"] is None else a + s["r"].float()).to(BF)
    if not s["train"]:
        return {"out": out}
    dz = s["dout"].float() * da
    return {"out": out, "dx": (dz @ W).to(BF), "dW": (dz.t() @ x).to(BF),
            "db": dz.sum(0).to(BF) if s["b"] is not None else None}


def _sorted(ids, E):
    """(row of each slot, or -1 where it is dropped; first row of each expert)."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    counts = torch.zeros(E + 1, dtype=torch.long, device=ids.device)
    counts.scatter_add_(0, key, torch.ones_like(key))
    padded = (counts[:E] + ROW_ALIGN - 1) // ROW_ALIGN * ROW_ALIGN
    offsets = torch.cat([torch.zeros_like(counts[:1]), torch.cumsum(padded, 0)])
    order = torch.argsort(key, stable=True)
    first = torch.cumsum(counts, 0) - counts
    by = key[order]
    row = offsets[by] + torch.arange(n, device=ids.device) - first[by]
    pos = torch.empty_like(row)
    pos[order] = torch.where(by < E, row, -1)
    return pos, offsets


def _gather(x, pos, k, rows):
    """The token rows at their places, zeros elsewhere (row `rows` takes the dropped slots)."""
    xs = torch.zeros((rows + 1, x.shape[1]), dtype=x.dtype, device=x.device)
    xs[torch.where(pos < 0, rows, pos)] = x.repeat_interleave(k, 0)
    xs[rows] = 0
    return xs


def _back(ys, pos, k):
    """Each slot's row ([T, k, H]), zeros where it is dropped."""
    got = ys[pos.clamp(min=0)] * (pos >= 0).unsqueeze(1).to(ys.dtype)
    return got.view(-1, k, ys.shape[1])


def _tokens(s):
    T, E, k, H = s["T"], s["E"], s["k"], s["H"]
    rows = _rows(T, E, k)
    w = s["weights"].float()
    pos, offsets = _sorted(s["ids"], E)
    xs = _gather(s["x"].float(), pos, k, rows)[:rows].to(BF)
    picked = _back(s["y"].float(), pos, k)
    out = (w.unsqueeze(2) * picked).sum(1)
    if s["r"] is not None:
        out = out + s["r"].float()
    res = {"offsets": offsets.to(torch.int32), "pos": pos.to(torch.int32).view(T, k), "xs": xs,
           "out": out.to(BF)}
    if s["train"]:
        dout = s["dout"].float()
        scaled = (w.unsqueeze(2) * dout.unsqueeze(1)).view(-1, H)
        dy = torch.zeros((rows + 1, H), device=dout.device)
        dy[torch.where(pos < 0, rows, pos)] = scaled
        res.update(dy=dy[:rows].to(BF),
                   dweights=(dout.unsqueeze(1) * picked).sum(2).to(s["weights"].dtype),
                   dx=_back(s["dxs"].float(), pos, k).sum(1).to(BF))
    return res


def _experts(s):
    T, E, k, H = s["T"], s["E"], s["k"], s["H"]
    x, w, act = s["x"].float(), s["weights"].float(), s["act"]
    gated = act in GATED
    flat = s["ids"].reshape(-1).long()
    n = T * k
    if not s["train"] and n <= E:
        # few tokens: every slot's weights, one product each
        Wg, Wd = s["Wg"][flat].float(), s["Wd"][flat].float()
        xe = x.repeat_interleave(k, 0).unsqueeze(2)
        h = _act_grad(act, torch.bmm(Wg, xe))[0]
        if gated:
            h = h * torch.bmm(s["Wu"][flat].float(), xe)
        y = torch.bmm(Wd, h).view(T, k, H)
        return {"out": (w.unsqueeze(2) * y).sum(1).to(BF)}
    # a box of as many rows for each expert as the fullest one has
    counts = torch.bincount(flat, minlength=E)
    cap = int(counts.max())
    order = torch.argsort(flat, stable=True)
    first = torch.cumsum(counts, 0) - counts
    rank = torch.empty_like(flat)
    rank[order] = torch.arange(n, device=x.device) - first[flat[order]]
    at = flat * cap + rank
    xe = torch.zeros((E * cap, H), device=x.device)
    xe[at] = x.repeat_interleave(k, 0)
    xe = xe.view(E, cap, H)
    Wg, Wd = s["Wg"].float(), s["Wd"].float()
    g = torch.bmm(xe, Wg.transpose(1, 2))
    a, da = _act_grad(act, g)
    u = torch.bmm(xe, s["Wu"].float().transpose(1, 2)) if gated else None
    h = a * u if gated else a
    y = torch.bmm(h, Wd.transpose(1, 2)).view(E * cap, H)[at].view(T, k, H)
    out = (w.unsqueeze(2) * y).sum(1).to(BF)
    if not s["train"]:
        return {"out": out}
    dout = s["dout"].float()
    dy = torch.zeros((E * cap, H), device=x.device)
    dy[at] = (w.unsqueeze(2) * dout.unsqueeze(1)).view(n, H)
    dy = dy.view(E, cap, H)
    dh = torch.bmm(dy, Wd)
    dg = dh * da * u if gated else dh * da
    dxe = torch.bmm(dg, Wg)
    res = {"out": out, "dweights": (dout.unsqueeze(1) * y).sum(2).to(s["weights"].dtype),
           "dWg": torch.bmm(dg.transpose(1, 2), xe).to(BF), "dWu": None,
           "dWd": torch.bmm(dy.transpose(1, 2), h).to(BF)}
    if gated:
        du = dh * a
        dxe = dxe + torch.bmm(du, s["Wu"].float())
        res["dWu"] = torch.bmm(du.transpose(1, 2), xe).to(BF)
    res["dx"] = dxe.view(E * cap, H)[at].view(T, k, H).sum(1).to(BF)
    return res


# ---------------------------------------------------------------- work

def work(case):
    b = 2  # bytes of a bf16 value
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        mn, mk, nk = M * N * b, M * K * b, N * K * b
        io = mk + nk + mn + (N * b if case["bias"] else 0) + (mn if case["residual"] else 0)
        flops = 2.0 * M * N * K
        if case["train"]:  # dout in; dx, dW, db out
            io += mn + mk + nk + (N * b if case["bias"] else 0)
            flops *= 3
        return {"bytes": io, "flops": flops}
    T, E, k, H = case["T"], case["E"], case["k"], case["H"]
    wb = 2 if case["w"] == "bf16" else 4
    if case["op"] == "tokens":
        n, rows = T * k * (1 - case["drop"]), _rows(T, E, k)
        th = T * H * b
        io = T * k * (4 + wb + 4) + th + rows * H * b + n * H * b + th
        io += th if case["residual"] else 0
        flops = 2.0 * n * H
        if case["train"]:  # dout, y, dxs in; dy, dweights, dx out
            io += th + n * H * b + rows * H * b + n * H * b + th + 2 * T * k * wb
            flops *= 3
        return {"bytes": io, "flops": flops}
    inner, mats = case["I"], 3 if case["act"] in GATED else 2
    touched = E * (1 - (1 - k / E) ** T) if case["k"] < E else E
    weights = mats * H * inner * b
    io = 2 * T * H * b + T * k * (4 + wb) + touched * weights
    flops = 2.0 * T * k * H * inner * mats
    if case["train"]:  # dout in; dx, dweights and every expert's gradients out
        io += 2 * T * H * b + T * k * wb + E * weights
        flops *= 3
    return {"bytes": io, "flops": flops}


# ---------------------------------------------------------------- the definition in 64 bits

def _f(name, z):
    if name in ("swiglu", "silu"):
        return z * torch.sigmoid(z)
    if name == "glu":
        return torch.sigmoid(z)
    if name in ("reglu", "relu"):
        return torch.relu(z)
    if name == "relu_sq":
        return torch.relu(z).square()
    if name in ("geglu", "gelu_tanh_approx"):
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z.pow(3))))
    return z


def exact(case, seed):
    s = prepare(case, seed)
    f64 = lambda t: None if t is None else t.double()  # noqa: E731
    if case["op"] == "linear":
        leaf = [t.requires_grad_(True) for t in (f64(s["x"]), f64(s["W"]))]
        b = f64(s["b"])
        z = torch.nn.functional.linear(leaf[0], leaf[1])
        if b is not None:
            leaf.append(b.requires_grad_(True))
            z = z + b
        out = _f(case["act"], z)
        if s["r"] is not None:
            out = out + f64(s["r"])
        if not case["train"]:
            return {"out": out.detach()}
        g = torch.autograd.grad(out, leaf, f64(s["dout"]))
        return {"out": out.detach(), "dx": g[0], "dW": g[1], "db": g[2] if len(g) > 2 else None}
    T, E, k, H = case["T"], case["E"], case["k"], case["H"]
    ids = s["ids"].cpu().tolist()
    w = f64(s["weights"])
    if case["op"] == "tokens":
        lists = [[] for _ in range(E)]
        for t, row in enumerate(ids):
            for j, e in enumerate(row):
                if 0 <= e < E:
                    lists[e].append((t, j))
        offsets, pos, src = [0], [[-1] * k for _ in range(T)], []
        for e in range(E):
            for t, j in lists[e]:
                pos[t][j] = len(src)
                src.append((t, j))
            src += [None] * (-len(src) % ROW_ALIGN)
            offsets.append(len(src))
        dev, rows = s["x"].device, _rows(T, E, k)
        real = [(r, t, j) for r, tj in enumerate(src) if tj is not None for t, j in [tj]]
        r, t, j = (torch.tensor(c, dtype=torch.long, device=dev) for c in
                   (zip(*real) if real else ([], [], [])))
        xs = torch.zeros((rows, H), dtype=torch.float64, device=dev).index_copy_(0, r, f64(s["x"])[t])
        out = torch.zeros((T, H), dtype=torch.float64, device=dev)
        out.index_add_(0, t, w[t, j].unsqueeze(1) * f64(s["y"])[r])
        if s["r"] is not None:
            out += f64(s["r"])
        res = {"offsets": torch.tensor(offsets, dtype=torch.int32),
               "pos": torch.tensor(pos, dtype=torch.int32).view(T, k), "xs": xs, "out": out}
        if case["train"]:
            dout = f64(s["dout"])
            dy = torch.zeros_like(xs).index_copy_(0, r, w[t, j].unsqueeze(1) * dout[t])
            dw = torch.zeros_like(w)
            dw[t, j] = (dout[t] * f64(s["y"])[r]).sum(1)
            dx = torch.zeros_like(out).index_add_(0, t, f64(s["dxs"])[r])
            res.update(dy=dy, dweights=dw, dx=dx)
        return res
    # each expert over its own tokens, differentiated by autograd
    gated = case["act"] in GATED
    x = f64(s["x"]).requires_grad_(case["train"])
    w.requires_grad_(case["train"])
    ids_t, dev = s["ids"].long(), s["x"].device
    out = torch.zeros((T, H), dtype=torch.float64, device=dev)
    dx, dw = torch.zeros_like(out), torch.zeros_like(w)
    grads = {n: [] for n in ("dWg", "dWu", "dWd")}
    for e in range(E):
        t, j = torch.nonzero(ids_t == e, as_tuple=True)
        Ws = [f64(s[n][e]).requires_grad_(case["train"]) for n in ("Wg", "Wu", "Wd")
              if s[n] is not None]
        h = _f(case["act"], x[t] @ Ws[0].t())
        if gated:
            h = h * (x[t] @ Ws[1].t())
        part = w[t, j].unsqueeze(1) * (h @ Ws[-1].t())
        out.index_add_(0, t, part.detach())
        if case["train"]:
            g = torch.autograd.grad(part, [x, w] + Ws, f64(s["dout"])[t])
            dx += g[0]
            dw += g[1]
            grads["dWg"].append(g[2].float())
            grads["dWd"].append(g[-1].float())
            if gated:
                grads["dWu"].append(g[3].float())
    if not case["train"]:
        return {"out": out.detach()}
    res = {"out": out.detach(), "dx": dx, "dweights": dw.detach()}
    res.update({n: torch.stack(v).double() if v else None for n, v in grads.items()})
    return res
