"""The operators of a tensor-parallel transformer block beside the plain MLP, as cases to be measured: the gated
feed-forward block (tp_glu), the matrix product with bias, activation and residual (tp_linear), and the global gradient
norm with clipping (GradGroup). Every tensor is laid out as the framework lays it out: one buffer per virtual rank.

``run`` computes a case in plain torch operations in float32, rounded once at the end, or, with ``own`` true, through the
package's public entry points."""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
WEIGHT_STD = 0.02  # the framework's own benchmark draws its MLP weights from N(0, 0.02) and X from N(0, 1)


def _glu(name, dir, M, K, F, N, P, act="silu", residual=True):
    return {"name": name, "op": "glu", "dir": dir, "M": M, "K": K, "F": F, "N": N, "P": P, "act": act,
            "residual": residual}


def _linear(name, dir, split, M, K, N, P, act="none", bias=True, residual=True):
    return {"name": name, "op": "linear", "dir": dir, "split": split, "M": M, "K": K, "N": N, "P": P, "act": act,
            "bias": bias, "residual": residual}


def _clip(name, layers, K, F, P, dtype, max_norm=1.0):
    return {"name": name, "op": "clip", "layers": layers, "K": K, "F": F, "P": P, "dtype": dtype, "max_norm": max_norm}


def listed():
    return [
        # serving: one token through the block of the framework's MLP configuration; reading the weights is the time
        _glu("glu 1 token", "forward", 1, 4096, 16384, 4096, 8),
        # serving: a small batch of decoded tokens through a small layer on two ranks; launches and latency count
        _glu("glu 37 tokens small", "forward", 37, 2048, 5632, 2048, 2),
        # a ragged prompt: no extent a multiple of a tile
        _glu("glu prompt ragged", "forward", 1021, 2056, 5648, 2056, 2, act="gelu_tanh"),
        # the Llama-70B MLP shape of the framework's overlap configuration, gated
        _glu("glu forward 4096x8192x28672", "forward", 4096, 8192, 28672, 8192, 8),
        # training forward at the framework's MLP configuration: keeps both pre-activations
        _glu("glu train forward 8192", "train", 8192, 4096, 16384, 4096, 8),
        # its backward pass: gradients of X and of all three weight sets
        _glu("glu backward 8192", "backward", 8192, 4096, 16384, 4096, 8),
        # serving: a few tokens through a row-parallel projection with bias and residual
        _linear("linear row 5 tokens", "forward", "row", 5, 16384, 4096, 8),
        # a prompt through a column-parallel projection with bias on four ranks
        _linear("linear column 777", "forward", "column", 777, 4096, 6144, 4, residual=False),
        # training forward of a row-parallel projection: bias and residual, all ranks summed
        _linear("linear row 8192", "forward", "row", 8192, 16384, 4096, 8),
        # backward of a column-parallel layer with GELU: the pre-activation kept by its forward is an input
        _linear("linear column backward", "backward", "column", 4096, 4096, 16384, 8, act="gelu", residual=False),
        # clipping after one step of a small layer: many small tensors, latency counts
        _clip("clip small bf16", 2, 256, 1024, 4, "bf16", 0.05),
        # clipping the float32 gradients of one block of the MLP configuration's sizes on eight ranks
        _clip("clip block f32", 1, 4096, 16384, 8, "f32"),
    ]


# ---- drawing cases ---------------------------------------------------------------------------------------------

MOST_FLOPS = 2 * 2 * 8192 * 3 * 4096 * 16384  # the listed backward pass


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["glu", "glu", "linear", "linear", "clip"])
    P = rng.choice([1, 2, 3, 4, 8])
    if op == "clip":
        P = rng.choice([1, 2, 4, 8])
        c = _clip("", 1 if P == 8 else rng.choice([1, 2, 3]), _log(rng, 128, 4096), P * _log(rng, 64, 16384 // P), P,
                  rng.choice(["bf16", "f32", "mixed"]), rng.choice([0.01, 0.3, 1.0, 1e6]))
        while sum(_grad_sizes(c)) > sum(_grad_sizes(_clip("", 1, 4096, 16384, 8, "f32"))):
            c["K"] = max(1, c["K"] // 2)
    else:
        K, N = _log(rng, 512, 8192, 8), _log(rng, 512, 8192, 8)
        M = _log(rng, 1, 8192)
        act = rng.choice(["silu", "gelu", "gelu_tanh", "relu"])
        dir = rng.choice(["forward", "forward", "train", "backward"])
        if dir != "forward":
            M = max(M, 256)
        if op == "glu":
            c = _glu("", dir, M, K, P * _log(rng, 512 // P, 28672 // P, 8), N, P, act, rng.random() < 0.7)
        else:
            split = rng.choice(["column", "row"])
            if split == "column":
                N = P * _log(rng, 256, 16384 // P, 8)
            else:
                K = P * _log(rng, 256, 16384 // P, 8)
            act = rng.choice(["none", "none", act])
            dir = "backward" if dir == "backward" else "forward"
            c = _linear("", dir, split, M, K, N, P, act, rng.random() < 0.8, dir == "forward" and rng.random() < 0.6)
        while work(c)["flops"] > MOST_FLOPS:
            c["M"] = c["M"] // 2 + 1
    del c["name"]
    return c


# ---- inputs ----------------------------------------------------------------------------------------------------

def _grad_sizes(c):
    """Elements of each gradient piece: per layer P ranks of three weight shards, and P replicas of a norm weight."""
    Fp = c["F"] // c["P"]
    return (([c["K"] * Fp] * 2 + [Fp * c["K"]]) * c["P"] + [c["K"]] * c["P"]) * c["layers"]


def _grad_counted(c):
    """The norm weight is replicated: only rank 0's copy counts."""
    return ([True] * (3 * c["P"]) + [True] + [False] * (c["P"] - 1)) * c["layers"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(shape, std=1.0, dtype=BF16):
        return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)

    s = {"case": case}
    if case["op"] == "clip":
        kinds = {"bf16": [BF16], "f32": [F32], "mixed": [BF16, F32]}[case["dtype"]]
        s["counted"] = _grad_counted(case)
        s["grads"] = [normal((n,), 1e-3 * (1 + i % 5), kinds[i % len(kinds)])
                      for i, n in enumerate(_grad_sizes(case))]
        for i, counted in enumerate(s["counted"]):  # a replica holds what rank 0 holds
            if not counted:
                s["grads"][i] = s["grads"][i - 1].to(s["grads"][i].dtype)
        if own:
            import resharding_tensor_parallelism_gb300 as rtp
            # a training program keeps its gradient buffers, and so the group over them and the clipped copies
            s["group"] = rtp.GradGroup(s["grads"], counted=s["counted"])
            s["clipped"] = [torch.empty_like(g) for g in s["grads"]]
        return s

    M, K, N, P, dir = (case[k] for k in ("M", "K", "N", "P", "dir"))
    if case["op"] == "glu":
        Fp = case["F"] // P
        s["X"] = normal((M, K))
        s["Ag"] = [normal((K, Fp), WEIGHT_STD) for _ in range(P)]
        s["Au"] = [normal((K, Fp), WEIGHT_STD) for _ in range(P)]
        s["B"] = [normal((Fp, N), WEIGHT_STD) for _ in range(P)]
        if dir == "backward":
            std = WEIGHT_STD * math.sqrt(K)  # the spread that X A has
            s["Hg"] = [normal((M, Fp), std) for _ in range(P)]
            s["Hu"] = [normal((M, Fp), std) for _ in range(P)]
            s["Y"] = [(_act(case["act"], g.float()) * u.float()).to(BF16) for g, u in zip(s["Hg"], s["Hu"])]
            s["dZ"] = normal((M, N), 1e-2)
        else:
            s["R"] = normal((M, N)) if case["residual"] else None
        return s

    row = case["split"] == "row"
    Kp, Np = (K // P, N) if row else (K, N // P)
    outs = 1 if row else P  # buffers of the output: one that sums the ranks, or one per rank
    s["X"] = [normal((M, Kp)) for _ in range(P if row else 1)]
    s["W"] = [normal((Kp, Np), WEIGHT_STD) for _ in range(P)]
    if dir == "backward":
        s["H"] = [normal((M, Np), WEIGHT_STD * math.sqrt(K)) for _ in range(outs)] if case["act"] != "none" else None
        s["dOut"] = [normal((M, Np), 1e-2) for _ in range(outs)]
    else:
        s["b"] = [normal((Np,), 0.1) for _ in range(outs)] if case["bias"] else None
        s["R"] = [normal((M, Np)) for _ in range(outs)] if case["residual"] else None
    return s


# ---- the plain form --------------------------------------------------------------------------------------------

def _phi(x):
    return 0.5 * (1 + torch.erf(x * math.sqrt(0.5)))


def _act(act, x):
    if act == "none":
        return x
    if act == "relu":
        return x * (x > 0)
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return x * _phi(x)
    return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))  # gelu_tanh


def _act_grad(act, x):
    if act == "none":
        return torch.ones_like(x)
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "silu":
        sig = 1 / (1 + torch.exp(-x))
        return sig * (1 + x * (1 - sig))
    if act == "gelu":
        return _phi(x) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    t = torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x))  # gelu_tanh
    return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * x * x)


def _wide(shards, dim):
    return torch.cat(shards, dim).float() if len(shards) > 1 else shards[0].float()


def _narrow(t, P, dim, dtype=BF16):
    return list(torch.chunk(t.to(dtype), P, dim))


def _plain_glu(c, s):
    P, act = c["P"], c["act"]
    X, B = s["X"].float(), _wide(s["B"], 0)
    if c["dir"] == "backward":
        hg, hu, dZ = _wide(s["Hg"], 1), _wide(s["Hu"], 1), s["dZ"].float()
        dY = dZ @ B.T
        dhg, dhu = dY * hu * _act_grad(act, hg), dY * _act(act, hg)
        dX = dhg @ _wide(s["Ag"], 1).T + dhu @ _wide(s["Au"], 1).T
        return {"dX": dX.to(BF16), "dAg": _narrow(X.T @ dhg, P, 1), "dAu": _narrow(X.T @ dhu, P, 1),
                "dB": _narrow(_wide(s["Y"], 1).T @ dZ, P, 0)}
    hg, hu = X @ _wide(s["Ag"], 1), X @ _wide(s["Au"], 1)
    y = _act(act, hg) * hu
    Z = y @ B
    if s["R"] is not None:
        Z = Z + s["R"].float()
    if c["dir"] == "forward":
        return Z.to(BF16)
    return {"Z": Z.to(BF16), "Y": _narrow(y, P, 1), "Hg": _narrow(hg, P, 1), "Hu": _narrow(hu, P, 1)}


def _plain_linear(c, s):
    row, P = c["split"] == "row", c["P"]
    X, W = _wide(s["X"], 1), _wide(s["W"], 0 if row else 1)
    if c["dir"] == "backward":
        dH = _wide(s["dOut"], 1)
        if s["H"] is not None:
            dH = dH * _act_grad(c["act"], _wide(s["H"], 1))
        dX, dW = dH @ W.T, X.T @ dH
        got = {"dX": _narrow(dX, P if row else 1, 1), "dW": _narrow(dW, P, 0 if row else 1)}
        if c["bias"]:
            got["db"] = _narrow(dH.sum(0), 1 if row else P, 0, F32)
        return got
    out = X @ W
    if s["b"] is not None:
        out = out + _wide(s["b"], 0)
    out = _act(c["act"], out)
    if s["R"] is not None:
        out = out + _wide(s["R"], 1)
    return _narrow(out, 1 if row else P, 1)


def _plain_clip(c, s):
    wide = [g.float() for g in s["grads"]]
    norm = torch.stack([g.square().sum() for g, counted in zip(wide, s["counted"]) if counted]).sum().sqrt()
    coef = (c["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    return {"norm": norm, "grads": [(g * coef).to(h.dtype) for g, h in zip(wide, s["grads"])]}


# ---- one pass --------------------------------------------------------------------------------------------------

def run(state):
    c, s = state["case"], state
    if not own:
        return {"glu": _plain_glu, "linear": _plain_linear, "clip": _plain_clip}[c["op"]](c, s)
    import resharding_tensor_parallelism_gb300 as rtp
    if c["op"] == "clip":
        norm, grads = s["group"].clip(c["max_norm"], out=s["clipped"])
        return {"norm": norm, "grads": grads}
    if c["op"] == "glu":
        if c["dir"] == "forward":
            return rtp.tp_glu(s["X"], s["Ag"], s["Au"], s["B"], act=c["act"], residual=s["R"])
        if c["dir"] == "train":
            Z, Y, Hg, Hu = rtp.tp_glu_train_forward(s["X"], s["Ag"], s["Au"], s["B"], act=c["act"], residual=s["R"])
            return {"Z": Z, "Y": Y, "Hg": Hg, "Hu": Hu}
        dX, dAg, dAu, dB = rtp.tp_glu_backward(s["X"], s["Ag"], s["Au"], s["B"], s["Hg"], s["Hu"], s["Y"], s["dZ"],
                                               act=c["act"])
        return {"dX": dX, "dAg": dAg, "dAu": dAu, "dB": dB}
    if c["dir"] == "forward":
        return rtp.tp_linear(s["X"], s["W"], split=c["split"], bias=s["b"], act=c["act"], residual=s["R"])
    dX, dW, db = rtp.tp_linear_backward(s["X"], s["W"], s["dOut"], split=c["split"], H=s["H"], act=c["act"],
                                        bias_grad=c["bias"])
    return {"dX": dX, "dW": dW, "db": db} if c["bias"] else {"dX": dX, "dW": dW}


def work(case):
    """Bytes and operations that a pass cannot do without: each input read once, each output written once."""
    if case["op"] == "clip":
        size = {"bf16": 2, "f32": 4, "mixed": 3}[case["dtype"]]
        n = sum(_grad_sizes(case))
        return {"bytes": 2 * n * size, "flops": 3 * n}
    M, K, N, back = case["M"], case["K"], case["N"], case["dir"] == "backward"
    if case["op"] == "glu":
        F = case["F"]
        weights, product = 2 * K * F + F * N, 2 * M * (2 * K * F + F * N)
        if back:  # reads X, weights, Hg, Hu, Y, dZ; writes dX and the weights' gradients
            return {"bytes": 2 * (2 * weights + 2 * M * K + 3 * M * F + M * N), "flops": 2 * product}
        kept = 3 * M * F if case["dir"] == "train" else 0
        return {"bytes": 2 * (M * K + weights + M * N * (2 if case["residual"] else 1) + kept), "flops": product}
    bias = N * bool(case["bias"])
    if back:
        kept = M * N * (2 if case["act"] != "none" else 1)
        return {"bytes": 2 * (2 * K * N + 2 * M * K + kept) + 4 * bias, "flops": 4 * M * K * N}
    return {"bytes": 2 * (M * K + K * N + M * N * (2 if case["residual"] else 1) + bias), "flops": 2 * M * K * N}


# ---- the definition in 64 bits ---------------------------------------------------------------------------------

def _wide64(parts):
    return [p.double() for p in parts]


def _act64(act, x):
    """(act(x), act'(x)) of a float64 tensor."""
    if act == "none":
        return x, torch.ones_like(x)
    if act == "relu":
        return x.clamp(min=0), (x > 0).double()
    if act == "silu":
        e = torch.special.expit(x)
        return x * e, e + x * e * torch.special.expit(-x)
    if act == "gelu":
        cdf = torch.special.ndtr(x)
        return x * cdf, cdf + x * (x * x / -2).exp() / math.sqrt(2 * math.pi)
    k = math.sqrt(8 / math.pi)  # 0.5 (1 + tanh(a)) is expit(2 a)
    e = torch.special.expit(k * (x + 0.044715 * x ** 3))
    return x * e, e + x * e * (1 - e) * k * (1 + 0.134145 * x ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        total = sum(float((g.double() ** 2).sum()) for g, counted in zip(s["grads"], s["counted"]) if counted)
        norm = math.sqrt(total)
        coef = min(1.0, case["max_norm"] / (norm + 1e-6))
        return {"norm": torch.tensor(norm, dtype=torch.float64, device="cuda"),
                "grads": [g.double() * coef for g in s["grads"]]}
    act = case["act"]
    if case["op"] == "glu":
        X = s["X"].double()
        if case["dir"] == "backward":
            dZ, dX = s["dZ"].double(), 0
            got = {"dAg": [], "dAu": [], "dB": []}
            for Ag, Au, B, Hg, Hu, Y in zip(*(s[k] for k in ("Ag", "Au", "B", "Hg", "Hu", "Y"))):
                a, da = _act64(act, Hg.double())
                dY = dZ.matmul(B.double().t())
                dg, du = dY * Hu.double() * da, dY * a
                dX = dX + dg.matmul(Ag.double().t()) + du.matmul(Au.double().t())
                got["dAg"].append(X.t().matmul(dg))
                got["dAu"].append(X.t().matmul(du))
                got["dB"].append(Y.double().t().matmul(dZ))
            return {"dX": dX, **got}
        Z = s["R"].double() if s["R"] is not None else 0
        got = {"Y": [], "Hg": [], "Hu": []}
        for Ag, Au, B in zip(s["Ag"], s["Au"], s["B"]):
            hg, hu = X.matmul(Ag.double()), X.matmul(Au.double())
            y = _act64(act, hg)[0] * hu
            Z = Z + y.matmul(B.double())
            for k, v in (("Y", y), ("Hg", hg), ("Hu", hu)):
                got[k].append(v)
        return Z if case["dir"] == "forward" else {"Z": Z, **got}
    row, P = case["split"] == "row", case["P"]
    W = _wide64(s["W"])
    X = _wide64(s["X"]) if row else _wide64(s["X"]) * P
    if case["dir"] == "backward":
        dH = _wide64(s["dOut"])
        if s["H"] is not None:
            dH = [d * _act64(act, h.double())[1] for d, h in zip(dH, s["H"])]
        db = [d.sum(0) for d in dH]
        dH = dH * P if row else dH
        dX = [d.matmul(w.t()) for d, w in zip(dH, W)]
        dW = [x.t().matmul(d) for x, d in zip(X, dH)]
        got = {"dX": dX if row else [sum(dX)], "dW": dW}
        return {**got, "db": db} if case["bias"] else got
    out = [x.matmul(w) for x, w in zip(X, W)]
    out = [sum(out)] if row else out
    if s["b"] is not None:
        out = [o + b.double() for o, b in zip(out, s["b"])]
    out = [_act64(act, o)[0] for o in out]
    if s["R"] is not None:
        out = [o + r.double() for o, r in zip(out, s["R"])]
    return out
