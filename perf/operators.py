"""Cases of the language-model operators around the gathered product: their inputs, their plain forms, the
framework's calls, and their values in 64 bits.

  linear   C = act(A B^T + bias) + residual, and its gradients (gemm_bias_act, gemm_bias_act_bwd)
  grouped  rows sorted by expert, each times its expert's weight, and its gradients (gemm_grouped, gemm_grouped_bwd)
  xent     cross entropy of the logits A B^T, which are not kept, and its gradients (gemm_xent, gemm_xent_bwd)

A is (rows, K), a weight is (outputs, K), everything bf16 but the loss, its gradient and the logarithm of the
sums (fp32), the targets (int64) and the groups' ends (int32).
"""
import math
import random

import torch

own = False

BF16 = torch.bfloat16
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
MOST_FLOPS = 1.9e12          # of a drawn case: no more than the largest listed one


# ---------------------------------------------------------------------------------------------- cases
def _linear(name, do, M, K, Nc, act, bias, residual, keep_pre=False):
    return {"name": name, "op": "linear", "do": do, "M": M, "K": K, "Nc": Nc, "act": act, "bias": bias,
            "residual": residual, "keep_pre": keep_pre}


def _grouped(name, do, M, K, Nc, E, skew, load, spare=0):
    return {"name": name, "op": "grouped", "do": do, "M": M, "K": K, "Nc": Nc, "E": E, "skew": skew,
            "load": load, "spare": spare}


def _xent(name, do, T, K, V, ignored):
    return {"name": name, "op": "xent", "do": do, "T": T, "K": K, "V": V, "ignored": ignored}


def listed():
    return [
        # one new token through an output projection: the residual stream comes back added
        _linear("linear_token", "fwd", 1, 4096, 4096, "none", True, True),
        # a batch of tokens being decoded through an MLP's first projection
        _linear("linear_decode_batch", "fwd", 48, 4096, 14336, "silu", False, False),
        # a ragged prompt, outputs that are not a multiple of any tile
        _linear("linear_prompt_odd", "fwd", 500, 8192, 1003, "relu", True, True),
        # the MLP-up workload of this repository in training: the pre-activation is kept for the backward pass
        _linear("linear_mlp_up", "fwd", 16384, 4096, 14336, "silu", True, False, True),
        # the gradients of the square workload with a GELU behind it
        _linear("linear_square_bwd", "bwd", 8192, 8192, 8192, "gelu", True, False),
        # a step of decoding: few rows, most experts with one or none
        _grouped("grouped_decode", "fwd", 32, 4096, 2048, 16, 1.0, 3),
        # a prompt's rows over many experts, unevenly
        _grouped("grouped_prompt", "fwd", 16384, 4096, 2048, 32, 2.0, 5),
        # training: both gradients, some experts empty, the buffer longer than what is routed
        _grouped("grouped_train_bwd", "bwd", 8192, 2048, 4096, 24, 4.0, 7, 200),
        # the log-probability of the next token for a batch of sequences
        _xent("xent_score_tokens", "fwd", 8, 4096, 32000, 0),
        # the loss of a batch of sequences, evaluation only
        _xent("xent_eval", "fwd", 8192, 4096, 32768, 100),
        # a training step over a vocabulary of odd size, some tokens without a target
        _xent("xent_train", "step", 4096, 2048, 50257, 300),
        # a training step over a short sequence
        _xent("xent_train_short", "step", 33, 1024, 32000, 2),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "grouped", "xent"])
    if op == "linear":
        do = rng.choice(["fwd", "fwd", "bwd"])
        M, K, Nc = _log_int(rng, 1, 16384), 8 * _log_int(rng, 16, 1024), _log_int(rng, 64, 14336)
        case = _linear("", do, M, K, Nc, rng.choice(ACTS), rng.random() < 0.6, do == "fwd" and rng.random() < 0.5,
                       do == "fwd" and rng.random() < 0.3)
        rows = "M"
    elif op == "grouped":
        do = rng.choice(["fwd", "fwd", "bwd"])
        M, K, Nc = _log_int(rng, 1, 16384), 8 * _log_int(rng, 16, 512), 8 * _log_int(rng, 16, 512)
        case = _grouped("", do, M, K, Nc, _log_int(rng, 2, 64), rng.uniform(0.5, 4.0), rng.randrange(1 << 20),
                        rng.choice([0, 0, rng.randrange(1, 300)]))
        rows = "M"
    else:
        do = rng.choice(["fwd", "step"])
        T, K, V = _log_int(rng, 1, 8192), 8 * _log_int(rng, 32, 512), _log_int(rng, 1000, 65536)
        case = _xent("", do, T, K, V, rng.choice([0, T // 8]))
        rows = "T"
    del case["name"]
    most = MOST_FLOPS / 1.02
    if work(case)["flops"] > most:
        case[rows] = int(case[rows] * most / work(case)["flops"])
        if op == "xent":
            case["ignored"] = min(case["ignored"], case["T"] // 8)
    return case


# --------------------------------------------------------------------------------------------- inputs
def _sizes(case):
    """Rows of each expert, drawn with weights that fall off the more the larger the skew."""
    rng = random.Random(case["load"])
    weight = [rng.random() ** case["skew"] for _ in range(case["E"])]
    sizes = [0] * case["E"]
    for e in rng.choices(range(case["E"]), weight, k=case["M"]):
        sizes[e] += 1
    return sizes


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF16)

    s = {"case": case}
    if case["op"] == "linear":
        M, K, Nc = case["M"], case["K"], case["Nc"]
        s["A"], s["B"] = normal(M, K), normal(Nc, K, std=0.02)
        s["bias"] = normal(Nc, std=0.1) if case["bias"] else None
        if case["do"] == "fwd":
            s["residual"] = normal(M, Nc) if case["residual"] else None
        else:
            s["dC"] = normal(M, Nc)
            s["pre"] = normal(M, Nc, std=0.02 * math.sqrt(K)) if case["act"] != "none" else None
    elif case["op"] == "grouped":
        rows, K, Nc, E = case["M"] + case["spare"], case["K"], case["Nc"], case["E"]
        s["sizes"] = _sizes(case)                # a plain program splits by sizes that the host knows
        s["ends"] = torch.tensor(s["sizes"], dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
        s["A"], s["B"] = normal(rows, K), normal(E, Nc, K, std=0.02)
        if case["do"] == "bwd":
            s["dC"] = normal(rows, Nc)
    else:
        T, K, V = case["T"], case["K"], case["V"]
        s["A"], s["B"] = normal(T, K), normal(V, K, std=0.02)
        y = torch.randint(0, V, (T,), generator=g, device="cuda")
        if case["ignored"]:
            y[torch.randperm(T, generator=g, device="cuda")[:case["ignored"]]] = -100
        s["targets"] = y
        # the mean over the tokens that have a target
        s["dloss"] = torch.full((T,), 1.0 / max(1, T - case["ignored"]), device="cuda")
    return s


# ---------------------------------------------------------------------------------------- plain forms
def _act(x, act):
    if act == "relu":
        return torch.clamp(x, min=0)
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _act_slope(x, act):
    if act == "relu":
        return (x > 0).float()
    if act == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s * (1 + x * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (x + 0.044715 * x * x * x))
        return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * c * (1 + 3 * 0.044715 * x * x)
    return torch.ones_like(x)


def _plain_linear(s):
    c = s["case"]
    a, b = s["A"].float(), s["B"].float()
    if c["do"] == "fwd":
        pre = a @ b.t()
        if s["bias"] is not None:
            pre = pre + s["bias"].float()
        out = _act(pre, c["act"])
        if s["residual"] is not None:
            out = out + s["residual"].float()
        return {"C": out.to(BF16), "pre": pre.to(BF16)} if c["keep_pre"] else {"C": out.to(BF16)}
    d = s["dC"].float()
    if c["act"] != "none":
        d = d * _act_slope(s["pre"].float(), c["act"])
    out = {"dA": (d @ b).to(BF16), "dB": (d.t() @ a).to(BF16)}
    if c["bias"]:
        out["dbias"] = d.sum(0).to(BF16)
    return out


def _plain_grouped(s):
    c, sizes = s["case"], s["sizes"]
    used = sum(sizes)
    a = s["A"].float()
    b = s["B"].float()
    if c["do"] == "fwd":
        C = torch.zeros(a.shape[0], c["Nc"], device="cuda")
        C[:used] = torch.cat([x @ w.t() for x, w in zip(a[:used].split(sizes), b)])
        return {"C": C.to(BF16)}
    d = s["dC"].float()
    dA = torch.zeros_like(a)
    dA[:used] = torch.cat([x @ w for x, w in zip(d[:used].split(sizes), b)])
    dB = torch.stack([x.t() @ y for x, y in zip(d[:used].split(sizes), a[:used].split(sizes))])
    return {"dA": dA.to(BF16), "dB": dB.to(BF16)}


def _plain_xent(s):
    c, y = s["case"], s["targets"]
    a, b = s["A"].float(), s["B"].float()
    logits = a @ b.t()
    top = logits.amax(1, keepdim=True)
    lse = (torch.log(torch.exp(logits - top).sum(1, keepdim=True)) + top).squeeze(1)
    has = y >= 0
    hit = torch.where(has, y, 0).unsqueeze(1)
    loss = torch.where(has, lse - logits.gather(1, hit).squeeze(1), 0.0)
    if c["do"] == "fwd":
        return {"loss": loss, "lse": lse}
    p = torch.exp(logits - lse.unsqueeze(1))
    p.scatter_add_(1, hit, torch.full_like(hit, -1, dtype=torch.float32))
    p = p * torch.where(has, s["dloss"], 0.0).unsqueeze(1)
    return {"loss": loss, "dA": (p @ b).to(BF16), "dB": (p.t() @ a).to(BF16)}


# --------------------------------------------------------------------------------- the framework's calls
def _own_linear(s):
    import allgather_gemm_amd as ag
    c = s["case"]
    if c["do"] == "fwd":
        if c["keep_pre"]:
            pre = torch.empty(c["M"], c["Nc"], dtype=BF16, device="cuda")
            C = ag.gemm_bias_act(s["A"], s["B"], bias=s["bias"], act=c["act"], residual=s["residual"], pre=pre)
            return {"C": C, "pre": pre}
        return {"C": ag.gemm_bias_act(s["A"], s["B"], bias=s["bias"], act=c["act"], residual=s["residual"])}
    dA, dB, dbias = ag.gemm_bias_act_bwd(s["dC"], s["A"], s["B"], act=c["act"], pre=s["pre"], need_dbias=c["bias"])
    return {"dA": dA, "dB": dB, "dbias": dbias} if c["bias"] else {"dA": dA, "dB": dB}


def _own_grouped(s):
    import allgather_gemm_amd as ag
    if s["case"]["do"] == "fwd":
        return {"C": ag.gemm_grouped(s["A"], s["B"], s["ends"])}
    dA, dB = ag.gemm_grouped_bwd(s["dC"], s["A"], s["B"], s["ends"])
    return {"dA": dA, "dB": dB}


def _own_xent(s):
    import allgather_gemm_amd as ag
    loss, lse = ag.gemm_xent(s["A"], s["B"], s["targets"])
    if s["case"]["do"] == "fwd":
        return {"loss": loss, "lse": lse}
    dA, dB = ag.gemm_xent_bwd(s["dloss"], s["A"], s["B"], s["targets"], lse)
    return {"loss": loss, "dA": dA, "dB": dB}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"linear": _own_linear, "grouped": _own_grouped, "xent": _own_xent}[op](state)
    return {"linear": _plain_linear, "grouped": _plain_grouped, "xent": _plain_xent}[op](state)


# ----------------------------------------------------------------------------------- what it cannot do without
def work(case):
    if case["op"] == "linear":
        M, K, Nc = case["M"], case["K"], case["Nc"]
        if case["do"] == "fwd":
            return {"bytes": 2 * (M * K + Nc * K + Nc * case["bias"] + M * Nc * (1 + case["residual"] + case["keep_pre"])),
                    "flops": 2 * M * Nc * K}
        return {"bytes": 2 * (M * Nc * (1 + (case["act"] != "none")) + 2 * M * K + 2 * Nc * K + Nc * case["bias"]),
                "flops": 4 * M * Nc * K}
    if case["op"] == "grouped":
        M, K, Nc, E = case["M"], case["K"], case["Nc"], case["E"]
        used = sum(1 for n in _sizes(case) if n)
        out = M + case["spare"]
        if case["do"] == "fwd":
            return {"bytes": 2 * (M * K + used * Nc * K + out * Nc) + 4 * E, "flops": 2 * M * Nc * K}
        return {"bytes": 2 * (M * Nc + M * K + used * Nc * K + out * K + E * Nc * K) + 4 * E, "flops": 4 * M * Nc * K}
    T, K, V = case["T"], case["K"], case["V"]
    if case["do"] == "fwd":
        return {"bytes": 2 * (T * K + V * K) + 16 * T, "flops": 2 * T * V * K}
    # the loss; then the logits again (they are not kept) and the two gradients
    return {"bytes": 2 * (2 * T * K + 2 * V * K) + 16 * T, "flops": 8 * T * V * K}


# ------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """From the definitions: sigmoids, error functions and softmaxes of torch in float64 on whole matrices."""
    s = prepare(case, seed)
    f = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    if case["op"] == "linear":
        def phi(x):                                   # act(x) = x * gate(x) for the smooth ones
            if case["act"] == "silu":
                return torch.sigmoid(x)
            if case["act"] == "gelu":
                return torch.special.ndtr(x)
            if case["act"] == "gelu_tanh":            # (1 + tanh u) / 2 = sigmoid(2u)
                return torch.sigmoid(math.sqrt(8 / math.pi) * (x + 0.044715 * x ** 3))
            return (x > 0).double() if case["act"] == "relu" else torch.ones_like(x)
        if case["do"] == "fwd":
            pre = torch.mm(f["A"], f["B"].T)
            if case["bias"]:
                pre += f["bias"][None, :]
            C = pre * phi(pre)
            if case["residual"]:
                C += f["residual"]
            return {"C": C, "pre": pre} if case["keep_pre"] else {"C": C}
        d = f["dC"]
        if case["act"] != "none":
            x = f["pre"].detach().requires_grad_(True)
            with torch.enable_grad():
                # the derivative of x * gate(x), by differentiation
                (d,) = torch.autograd.grad(x * phi(x), x, grad_outputs=d)
        out = {"dA": torch.mm(d, f["B"]), "dB": torch.mm(f["A"].T, d).T.contiguous()}
        if case["bias"]:
            out["dbias"] = torch.mv(d.T, torch.ones(d.shape[0], dtype=torch.float64, device="cuda"))
        return out
    if case["op"] == "grouped":
        ends = s["ends"].tolist()
        spans = list(zip([0] + ends[:-1], ends))
        if case["do"] == "fwd":
            C = torch.zeros(f["A"].shape[0], case["Nc"], dtype=torch.float64, device="cuda")
            for e, (lo, hi) in enumerate(spans):
                torch.mm(f["A"][lo:hi], f["B"][e].T, out=C[lo:hi])
            return {"C": C}
        dA = torch.zeros_like(f["A"])
        dB = torch.zeros_like(f["B"])
        for e, (lo, hi) in enumerate(spans):
            torch.mm(f["dC"][lo:hi], f["B"][e], out=dA[lo:hi])
            dB[e] = torch.mm(f["A"][lo:hi].T, f["dC"][lo:hi]).T
        return {"dA": dA, "dB": dB}
    z = torch.mm(f["B"], f["A"].T)                     # (V, T)
    lse = torch.logsumexp(z, 0)
    rows = torch.nonzero(s["targets"] != -100).flatten()
    y = s["targets"][rows]
    loss = torch.zeros(case["T"], dtype=torch.float64, device="cuda")
    loss[rows] = lse[rows] - z[y, rows]
    if case["do"] == "fwd":
        return {"loss": loss, "lse": lse}
    w = torch.zeros_like(loss)
    w[rows] = f["dloss"][rows]
    q = torch.softmax(z, 0)
    q[y, rows] -= 1
    q *= w
    return {"loss": loss, "dA": torch.mm(q.T, f["B"]), "dB": torch.mm(q, f["A"])}
