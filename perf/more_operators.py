"""Cases of the operators on either side of a training step's products: their inputs, their plain forms, the framework's
calls, and their values in 64 bits.

  norm        h = x + residual, y = (h - mean) rstd w + b over each row, and its gradients (layer_norm, layer_norm_bwd)
  orthogonal  a weight's update, or a stack of them, made orthogonal by five Newton-Schulz steps (newton_schulz)

x, w, b, y, h and the gradients are bf16, mean and rstd fp32; an update is bf16 or fp32, the orthogonal one bf16.
"""
import math

import torch

own = False

BF16 = torch.bfloat16
EPS = 1e-5                   # added to a row's variance
TINY = 1e-7                  # added to an update's norm
STEPS = ((3.4445, -4.7750, 2.0315),) * 5
MOST_ELEMENTS = 8192 * 14336     # of a drawn case: no more than the largest listed one of its operator
MOST_FLOPS = 4.2e12


# ---------------------------------------------------------------------------------------------- cases
def _norm(name, do, rows, width, residual, keep=False):
    """residual: x arrives with a residual stream to add (fwd), or the gradient of that stream is added to dx (bwd);
    keep: the statistics are kept for the backward pass."""
    return {"name": name, "op": "norm", "do": do, "rows": rows, "width": width, "residual": residual, "keep": keep}


def _orthogonal(name, E, R, C, dtype, idle=0):
    """idle: that many of the stack's updates are zero, as those of experts that no row went to."""
    return {"name": name, "op": "orthogonal", "E": E, "R": R, "C": C, "dtype": dtype, "idle": idle}


def listed():
    return [
        # one new token before a projection, the last block's output added to its residual stream
        _norm("norm_token", "fwd", 1, 4096, True),
        # a batch of tokens being decoded, the square workload's width
        _norm("norm_decode_batch", "fwd", 48, 8192, True),
        # a ragged prompt of odd width, before the head
        _norm("norm_prompt_odd", "fwd", 500, 1003, False),
        # training on the MLP-up workload's rows: the sum and the statistics are kept
        _norm("norm_train", "fwd", 16384, 4096, True, True),
        # its gradients, the residual stream's added in
        _norm("norm_train_bwd", "bwd", 16384, 4096, True),
        # gradients over a short sequence
        _norm("norm_short_bwd", "bwd", 33, 1024, True),
        # gradients at the widest rows, an MLP's hidden ones
        _norm("norm_wide_bwd", "bwd", 8192, 14336, False),
        # the update of the example's hidden layer
        _orthogonal("orthogonal_small", 1, 512, 256, "bf16"),
        # a projection of odd extents, its momentum in fp32
        _orthogonal("orthogonal_odd", 1, 1003, 1500, "fp32"),
        # a layer of experts, one of which no row went to
        _orthogonal("orthogonal_experts", 16, 2048, 1024, "bf16", 1),
        # a square projection, its momentum in fp32
        _orthogonal("orthogonal_square", 1, 4096, 4096, "fp32"),
        # the MLP-up workload's weight
        _orthogonal("orthogonal_mlp_up", 1, 14336, 4096, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        do = rng.choice(["fwd", "bwd"])
        rows, width = _log_int(rng, 1, 16384), _log_int(rng, 64, 14336)
        if rng.random() < 0.5:
            width = max(8, width // 8 * 8)
        rows = min(rows, MOST_ELEMENTS // width)
        case = _norm("", do, rows, width, rng.random() < 0.6, do == "fwd" and rng.random() < 0.5)
    else:
        E = rng.choice([1, 1, _log_int(rng, 2, 32)])
        R, C = _log_int(rng, 64, 8192), _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            R, C = (R + 4) // 8 * 8, (C + 4) // 8 * 8
        case = _orthogonal("", E, R, C, rng.choice(["bf16", "fp32"]), rng.choice([0, 1]) if E > 1 else 0)
        while work(case)["flops"] > MOST_FLOPS:
            if case["E"] > 1:
                case["E"] //= 2
            elif case["R"] >= case["C"]:
                case["R"] = case["R"] * 3 // 4
            else:
                case["C"] = case["C"] * 3 // 4
        case["idle"] = case["idle"] if case["E"] > 1 else 0
    del case["name"]
    return case


# --------------------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=BF16):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(dtype)

    s = {"case": case}
    if case["op"] == "norm":
        T, W = case["rows"], case["width"]
        s["w"], s["b"] = normal(W, std=0.1, mean=1.0), normal(W, std=0.1)
        # a residual stream's channels differ in scale and offset, and so do its rows
        x = normal(T, W, dtype=torch.float32) * normal(W, std=0.5, dtype=torch.float32).exp() + normal(W, std=0.3, dtype=torch.float32)
        x *= normal(T, 1, std=0.5, dtype=torch.float32).exp()
        if case["do"] == "fwd":
            s["x"] = x.to(BF16)
            s["residual"] = normal(T, W, std=2.0) if case["residual"] else None
            return s
        s["h"], s["dy"] = x.to(BF16), normal(T, W)
        s["dh"] = normal(T, W) if case["residual"] else None
        # what the forward pass kept
        v, m = torch.var_mean(s["h"].double(), 1, correction=0)
        s["mean"], s["rstd"] = m.float(), (v + EPS).rsqrt().float()
        return s
    E, R, C = case["E"], case["R"], case["C"]
    # a momentum: some directions that many gradients shared, falling off, and what is left of the others
    rank = min(64, R, C)
    fall = torch.arange(1, rank + 1, device="cuda", dtype=torch.float32) ** -1.0
    G = torch.empty(E, R, C, device="cuda")
    for e in range(E):
        torch.addmm(normal(R, C, std=0.05, dtype=torch.float32), normal(R, rank, dtype=torch.float32) * fall,
                    normal(rank, C, dtype=torch.float32), out=G[e])
    G *= 1e-3
    if case["idle"]:
        G[1:1 + case["idle"]] = 0
    G = G.to(BF16 if case["dtype"] == "bf16" else torch.float32)
    s["G"] = G if E > 1 else G[0]
    return s


# ---------------------------------------------------------------------------------------- plain forms
def _plain_norm(s):
    c, w, b = s["case"], s["w"].float(), s["b"].float()
    if c["do"] == "fwd":
        out = {}
        h = s["x"].float()
        if c["residual"]:
            out["h"] = (h + s["residual"].float()).to(BF16)
            h = out["h"].float()
        mean = h.mean(1, keepdim=True)
        d = h - mean
        rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
        out["y"] = (d * rstd * w + b).to(BF16)
        if c["keep"]:
            out["mean"], out["rstd"] = mean.squeeze(1), rstd.squeeze(1)
        return out
    rstd, dy = s["rstd"].unsqueeze(1), s["dy"].float()
    xh = (s["h"].float() - s["mean"].unsqueeze(1)) * rstd
    g = dy * w
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    if c["residual"]:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(BF16), "dw": (dy * xh).sum(0).to(BF16), "db": dy.sum(0).to(BF16)}


def _plain_orthogonal(s):
    X = s["G"].float()
    tall = X.shape[-2] > X.shape[-1]
    if tall:
        X = X.mT
    X = X / (torch.sqrt((X * X).sum((-2, -1), keepdim=True)) + TINY)
    for a, b, c in STEPS:
        A = X @ X.mT
        X = a * X + (b * A + c * (A @ A)) @ X
    return {"out": (X.mT if tall else X).to(BF16).contiguous()}


# --------------------------------------------------------------------------------- the framework's calls
def _own_norm(s):
    import allgather_gemm_amd as ag
    c = s["case"]
    if c["do"] == "bwd":
        dx, dw, db = ag.layer_norm_bwd(s["dy"], s["h"], s["mean"], s["rstd"], weight=s["w"], dh=s["dh"])
        return {"dx": dx, "dw": dw, "db": db}
    out = {}
    if c["residual"]:
        out["h"] = torch.empty_like(s["x"])
    if c["keep"]:
        out["mean"], out["rstd"] = s["x"].new_empty((2, c["rows"]), dtype=torch.float32)
    out["y"] = ag.layer_norm(s["x"], weight=s["w"], bias=s["b"], eps=EPS, residual=s["residual"], **out)
    return out


def _own_orthogonal(s):
    import allgather_gemm_amd as ag
    return {"out": ag.newton_schulz(s["G"], coefficients=STEPS, eps=TINY)}


def run(state):
    norm = state["case"]["op"] == "norm"
    if own:
        return _own_norm(state) if norm else _own_orthogonal(state)
    return _plain_norm(state) if norm else _plain_orthogonal(state)


# ----------------------------------------------------------------------------------- what it cannot do without
def work(case):
    if case["op"] == "norm":
        T, W = case["rows"], case["width"]
        if case["do"] == "fwd":
            return {"bytes": 2 * T * W * (2 + 2 * case["residual"]) + 4 * W + 8 * T * case["keep"], "flops": 8 * T * W}
        return {"bytes": 2 * T * W * (3 + case["residual"]) + 6 * W + 8 * T, "flops": 14 * T * W}
    E, m, n = case["E"] - case["idle"], min(case["R"], case["C"]), max(case["R"], case["C"])
    # X X^T and A A are symmetric: half of each
    flops = E * len(STEPS) * (m * (m + 1) * n + m * (m + 1) * m + 2 * m * m * n)
    return {"bytes": case["E"] * m * n * ((2 if case["dtype"] == "bf16" else 4) + 2), "flops": flops}


# ------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The normalisation and its derivative by torch in float64; the steps on the Gram matrix alone: with
    X_k = Q_k X_0, all that changes is Q_k, a polynomial of X_0 X_0^T."""
    s = prepare(case, seed)
    if case["op"] == "norm":
        W = case["width"]
        w, b = s["w"].double().requires_grad_(True), s["b"].double().requires_grad_(True)
        if case["do"] == "fwd":
            out, x = {}, s["x"].double()
            if case["residual"]:
                out["h"] = x + s["residual"].double()
                x = (s["x"].float() + s["residual"].float()).to(BF16).double()     # the stored sum is what is normalised
            out["y"] = torch.nn.functional.layer_norm(x, (W,), w, b, EPS).detach()
            if case["keep"]:
                v, out["mean"] = torch.var_mean(x, 1, correction=0)
                out["rstd"] = (v + EPS) ** -0.5
            return out
        x = s["h"].double().requires_grad_(True)
        with torch.enable_grad():
            y = torch.nn.functional.layer_norm(x, (W,), w, b, EPS)
            dx, dw, db = torch.autograd.grad(y, (x, w, b), s["dy"].double())
        return {"dx": dx + s["dh"].double() if case["residual"] else dx, "dw": dw, "db": db}
    G = s["G"] if case["E"] > 1 else s["G"][None]
    out = torch.empty(G.shape, dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        x = G[e].double()
        wide = x.shape[0] <= x.shape[1]
        x = x / (torch.linalg.vector_norm(x) + TINY)
        gram = torch.mm(x, x.T) if wide else torch.mm(x.T, x)
        eye = torch.eye(gram.shape[0], dtype=torch.float64, device="cuda")
        Q, N = eye.clone(), gram
        for a, b, c in STEPS:
            P = a * eye + b * N + c * torch.mm(N, N)       # X' = P X and X' X'^T = P N P; all of them commute
            Q, N = torch.mm(P, Q), torch.mm(torch.mm(P, N), P)
        out[e] = torch.mm(Q, x) if wide else torch.mm(x, Q)
    return {"out": out if case["E"] > 1 else out[0]}
