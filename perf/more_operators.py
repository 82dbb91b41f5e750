"""The two ends of a tensor-parallel training step, as cases to be measured: the softmax cross entropy of an output layer
whose vocabulary is split over the virtual ranks, with its gradients (tp_cross_entropy, tp_cross_entropy_train), and the
AdamW step over many rank pieces with moments in 32 or 8 bits (AdamWGroup). Every tensor is laid out as the framework lays
it out: one buffer per virtual rank.

``run`` computes a case in plain torch operations in float32, rounded once at the end, or, with ``own`` true, through the
package's public entry points."""
import math

import torch

own = False

BF16, F32, I64 = torch.bfloat16, torch.float32, torch.int64
WEIGHT_STD = 0.02  # the framework's own benchmark draws its MLP weights from N(0, 0.02) and X from N(0, 1)
IGNORE = -100
BETA1, BETA2, EPS, LR, DECAY, SEED = 0.9, 0.95, 1e-8, 1e-3, 0.1, 17
BLOCK = 128  # elements of a block of 8-bit moments that share a power of two


def _loss(name, dir, M, K, V, P, vocab=None, weights=False, ignored=0.05):
    return {"name": name, "op": "loss", "dir": dir, "M": M, "K": K, "V": V, "P": P, "vocab": V if vocab is None else vocab,
            "weights": weights, "ignored": ignored}


def _adam(name, layers, K, F, P, param, grad, states, clip=True):
    """param: f32, bf16 (rounded at random) or master (bf16 and a float32 copy); an odd F leaves odd sizes everywhere."""
    return {"name": name, "op": "adam", "layers": layers, "K": K, "F": F, "P": P, "param": param, "grad": grad,
            "states": states, "clip": clip}


def listed():
    return [
        # scoring one decoded token at the framework's hidden size: reading the output layer's weights is the time
        _loss("loss 1 token", "forward", 1, 4096, 131072, 8, ignored=0.0),
        # scoring a few tokens with a small model's output layer: launches and latency count
        _loss("loss 37 tokens small", "forward", 37, 512, 8192, 2),
        # evaluating a ragged prompt, a padded vocabulary on four ranks
        _loss("loss prompt ragged", "forward", 1021, 2056, 50016, 4, vocab=50011),
        # evaluation at the framework's MLP configuration (8192 tokens, hidden 4096) with a large vocabulary
        _loss("loss 8192", "forward", 8192, 4096, 131072, 8),
        # a training step of a small model: launches and latency count
        _loss("train small", "train", 256, 512, 8192, 2),
        # fine-tuning on a ragged batch with a weight per token, most of the prompt ignored
        _loss("train ragged weighted", "train", 777, 2056, 50016, 4, vocab=50011, weights=True, ignored=0.6),
        # many tokens through a narrow model: the rows are taken in pieces and the weights' gradients summed over them
        _loss("train 16384 narrow", "train", 16384, 1024, 32768, 2),
        # the training step of the framework's MLP configuration with a large vocabulary
        _loss("train 8192", "train", 8192, 4096, 131072, 8),
        # a small layer's many tensors in float32: latency counts
        _adam("adamw small f32", 2, 256, 1024, 4, "f32", "f32", 32),
        # one block of the MLP configuration's sizes: bf16 weights with float32 copies, bf16 gradients
        _adam("adamw block master", 1, 4096, 16384, 8, "master", "bf16", 32),
        # odd sizes, bf16 weights without copies, 8-bit moments
        _adam("adamw ragged 8 bit", 2, 777, 4 * 1021, 4, "bf16", "mixed", 8),
        # one block of the MLP configuration's sizes with 8-bit moments
        _adam("adamw block 8 bit", 1, 4096, 16384, 8, "master", "bf16", 8),
    ]


# ---- drawing cases ---------------------------------------------------------------------------------------------

MOST_FLOPS = 6 * 8192 * 4096 * 131072  # the listed training step
MOST_ELEMENTS = 3 * 4096 * 16384       # the listed blocks


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    P = rng.choice([1, 2, 3, 4, 8])
    if rng.random() < 0.4:
        c = _adam("", rng.choice([1, 2, 3]), _log(rng, 64, 4096), P * _log(rng, 64, 16384 // P), P,
                  rng.choice(["f32", "bf16", "master"]), rng.choice(["f32", "bf16", "mixed"]), rng.choice([8, 32]),
                  rng.random() < 0.7)
        while sum(_sizes(c)) > MOST_ELEMENTS:
            c["K"] = max(1, c["K"] // 2)
    else:
        dir = rng.choice(["forward", "train"])
        M, K, V = _log(rng, 1, 16384), _log(rng, 256, 8192, 8), P * _log(rng, 4096 // P // 8 * 8, 131072 // P, 8)
        c = _loss("", dir, M, K, V, P, V - rng.choice([0, 0, 1, 5, 77]), dir == "train" and rng.random() < 0.5,
                  rng.choice([0.0, 0.05, 0.5]))
        while work(c)["flops"] > MOST_FLOPS:
            c["M"] = c["M"] // 2 + 1
    del c["name"]
    return c


# ---- inputs ----------------------------------------------------------------------------------------------------

def _sizes(c):
    """Elements of each parameter piece: per layer P ranks of three weight shards, and a norm weight."""
    Fp = c["F"] // c["P"]
    return ([c["K"] * Fp] * (3 * c["P"]) + [c["K"]]) * c["layers"]


def _starts(sizes):
    """(where each tensor begins in a flat buffer of whole blocks, the buffer's elements)"""
    at = [0]
    for n in sizes:
        at.append(at[-1] + (n + BLOCK - 1) // BLOCK * BLOCK)
    return at[:-1], at[-1]


def _kinds(c):
    """The gradients' types."""
    kinds = {"bf16": [BF16], "f32": [F32], "mixed": [BF16, F32]}[c["grad"]]
    return [kinds[i % len(kinds)] for i in range(len(_sizes(c)))]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(shape, std=1.0, dtype=BF16):
        return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)

    s = {"case": case}
    if case["op"] == "loss":
        M, K, V, P = case["M"], case["K"], case["V"], case["P"]
        s["X"] = normal((M, K))
        s["W"] = [normal((K, V // P), WEIGHT_STD) for _ in range(P)]
        s["targets"] = torch.randint(0, case["vocab"], (M,), generator=gen, device="cuda")
        ignored = torch.rand((M,), generator=gen, device="cuda") < case["ignored"]
        ignored[0] = False  # a batch holds one token to learn from
        s["targets"][ignored] = IGNORE
        s["weights"] = torch.rand((M,), generator=gen, device="cuda").add_(0.5) if case["weights"] else None
        return s

    # a program's flat buffers, of which its tensors are views that begin at whole blocks; zeros between them
    sizes = _sizes(case)
    starts, total = _starts(sizes)
    s["index"] = torch.full((total,), -1, dtype=torch.int32, device="cuda")  # of each element in its tensor
    s["owner"] = torch.zeros((total,), dtype=torch.int32, device="cuda")     # and its tensor
    for i, (at, n) in enumerate(zip(starts, sizes)):
        s["index"][at:at + n] = torch.arange(n, dtype=torch.int32, device="cuda")
        s["owner"][at:at + n] = i
    used = s["index"] >= 0

    def views(flat):
        return [flat[at:at + n] for at, n in zip(starts, sizes)]

    wide = normal((total,), WEIGHT_STD, F32).mul_(used)
    s["p"] = wide if case["param"] == "f32" else wide.to(BF16)
    s["master"] = wide if case["param"] == "master" else None
    kinds = _kinds(case)
    grads = {kind: normal((total,), 1e-3, kind) for kind in set(kinds)}
    s["g"] = [views(grads[kind])[i] for i, kind in enumerate(kinds)]
    for kind, g in grads.items():
        g.mul_(used & torch.tensor([k is kind for k in kinds], device="cuda")[s["owner"]])
    s["g_flat"] = list(grads.values())
    # as after some hundred steps: the moments of gradients that still move
    s["m"] = normal((total,), 3e-4, F32).mul_(used)
    s["v"] = normal((total,), 1e-3, F32).square_().add_(1e-7).mul_(used)
    s["step"] = 300
    s["norm"] = torch.rand((), generator=gen, device="cuda").add_(1.0) if case["clip"] else None
    if case["states"] == 8:
        half = torch.full((), 0.5, device="cuda")
        (s["m"], mt), (s["v"], vt) = _encode(s["m"], half, 4), _encode(s["v"], half, 5)
        s["scales"] = torch.stack([mt, vt], 1)  # per block: m's exponent, v's
    if own:
        import resharding_tensor_parallelism_gb300 as rtp
        # a training program keeps its optimizer, here with the state of an earlier step
        s["group"] = rtp.AdamWGroup(views(s["p"]), lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY,
                                    states=case["states"], seed=SEED,
                                    masters=None if s["master"] is None else views(s["master"]))
        kept = {"step": s["step"], "exp_avg": s["m"], "exp_avg_sq": s["v"]}
        s["group"].load_state_dict({**kept, "scales": s["scales"]} if case["states"] == 8 else kept)
    return s


# ---- the plain form --------------------------------------------------------------------------------------------

def _plain_loss(c, s):
    X, W, t = s["X"].float(), torch.cat(s["W"], 1).float() if c["P"] > 1 else s["W"][0].float(), s["targets"]
    logits = X @ W
    logits[:, c["vocab"]:] = -math.inf
    top = logits.max(1, keepdim=True).values
    p = torch.exp(logits - top)
    total = p.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    counted = t != IGNORE
    at = t.clamp(min=0)[:, None]
    loss = torch.where(counted, lse - logits.gather(1, at)[:, 0], 0.0)
    if c["dir"] == "forward":
        return {"loss": loss, "lse": lse}
    del logits
    w = (torch.ones_like(loss) if s["weights"] is None else s["weights"]) * counted
    g = (w / w.sum().clamp(min=1e-30))[:, None]
    d = p.mul_(g / total)
    d.scatter_add_(1, at, -g)
    dX, dW = d @ W.T, X.T @ d
    return {"total": (loss * g[:, 0]).sum(), "loss": loss, "dX": dX.to(BF16), "dW": list(torch.chunk(dW.to(BF16), c["P"], 1))}


# 8-bit floats with 3 bits of mantissa and, behind a sign, 4 of exponent (m), or 5 without a sign (v): code = E * 8 + M is
# (1 + M/8) 2^(E-bias), or M/8 2^(1-bias) where E = 0, times a power of two for its block, in which the largest absolute
# value has the exponent 7 (m) or 15 (v).
BIAS = {4: 7, 5: 15}


def _power(e):
    """2^e of an integer tensor, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(F32)


def _encode(x, u, exp_bits):
    """(codes, exponents of the blocks' largest) of whole blocks, rounded up where the lost part is over 1 - u; u in [0, 1)."""
    bias, x = BIAS[exp_bits], x.view(-1, BLOCK)
    top = x.abs().amax(1).view(torch.int32).bitwise_right_shift(23).clamp(27)
    z = x.abs() * _power(142 - top if exp_bits == 5 else 134 - top)[:, None]
    low = z < 2.0 ** (1 - bias)
    z = torch.where(low, z + 2.0 ** (1 - bias), z)
    up = (u * 2 ** 20).to(torch.int32).expand(x.numel()).view(-1, BLOCK)
    code = ((z.view(torch.int32) + up) >> 20) - ((127 - bias) << 3) - 8 * low.to(torch.int32)
    code = torch.maximum(code, (x > 0).to(torch.int32)) if exp_bits == 5 else code | ((x < 0).to(torch.int32) << 7)
    return code.to(torch.uint8).view(-1), top.to(torch.uint8)


def _decode(code, top, exp_bits):
    """Values of whole blocks of codes."""
    bias, code = BIAS[exp_bits], code.to(torch.int32).view(-1, BLOCK)
    size = code if exp_bits == 5 else code & 127
    z = (size << 20).view(F32) * 2.0 ** (127 - bias) * _power(top.to(torch.int32) - (142 if exp_bits == 5 else 134))[:, None]
    return (z if exp_bits == 5 else torch.where(code > 127, -z, z)).view(-1)


def _pcg(x):
    """A 32-bit hash (the output function of O'Neill's PCG-RXS-M-XS on one step of its state), of integers in int64."""
    x = (x * 747796405 + 2891336453) & 0xFFFFFFFF
    w = (((x >> ((x >> 28) + 4)) ^ x) * 277803737) & 0xFFFFFFFF
    return (w >> 22) ^ w


def _noise(s, step):
    """32 random bits for each element: a hash of the seed, the tensor, the step (the first is 1) and its index."""
    tensors = torch.arange(len(s["g"]), device="cuda")
    key = _pcg(_pcg(_pcg(SEED) + tensors & 0xFFFFFFFF) + step & 0xFFFFFFFF)
    return _pcg(key[s["owner"]] + s["index"] & 0xFFFFFFFF)


def _rounded_at_random(x, r):
    """float32 to bf16, up where the lost 16 bits and the 16 random ones carry."""
    return (((x.view(torch.int32) + r.to(torch.int32)) >> 16) << 16).view(F32).to(BF16)


def _moments(c, s):
    """What is held of the moments, as float32 values."""
    if c["states"] == 32:
        return s["m"], s["v"]
    return _decode(s["m"], s["scales"][:, 0], 4), _decode(s["v"], s["scales"][:, 1], 5)


def _plain_adam(c, s):
    s["step"] += 1
    t, p = s["step"], s["p"]
    m, v = _moments(c, s)
    g = s["g_flat"][0].float() if len(s["g_flat"]) == 1 else s["g_flat"][0].float() + s["g_flat"][1].float()
    if s["norm"] is not None:
        g = g * (1.0 / (s["norm"] + 1e-6)).clamp(max=1.0)
    m, v = BETA1 * m + (1 - BETA1) * g, BETA2 * v + (1 - BETA2) * g * g
    wide = p.float() if s["master"] is None else s["master"]
    wide = wide * (1 - LR * DECAY) - LR * (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS)
    noise = _noise(s, t) if c["states"] == 8 or c["param"] == "bf16" else None
    if c["param"] == "bf16":
        p.copy_(_rounded_at_random(wide, _pcg(noise) & 0xFFFF))
    else:
        p.copy_(wide)
    got = {"p": p}
    if s["master"] is not None:
        got["master"] = s["master"].copy_(wide)
    if c["states"] == 32:
        return {**got, "m": s["m"].copy_(m), "v": s["v"].copy_(v)}
    m8, mt = _encode(m, ((noise & 0xFFFF) + 0.5) / 2 ** 16, 4)
    v8, vt = _encode(v, ((noise >> 16) + 0.5) / 2 ** 16, 5)
    s["m"].copy_(m8)
    s["v"].copy_(v8)
    s["scales"].copy_(torch.stack([mt, vt], 1))
    m, v = _moments(c, s)
    return {**got, "m": m.to(BF16), "v": v.to(BF16)}  # 4 significant bits and a power of two: exact


# ---- one pass --------------------------------------------------------------------------------------------------

def run(state):
    c, s = state["case"], state
    if not own:
        return {"loss": _plain_loss, "adam": _plain_adam}[c["op"]](c, s)
    import resharding_tensor_parallelism_gb300 as rtp
    if c["op"] == "loss":
        if c["dir"] == "forward":
            loss, lse = rtp.tp_cross_entropy(s["X"], s["W"], s["targets"], vocab=c["vocab"], ignore_index=IGNORE)
            return {"loss": loss, "lse": lse}
        total, loss, dX, dW = rtp.tp_cross_entropy_train(s["X"], s["W"], s["targets"], weights=s["weights"], vocab=c["vocab"],
                                                         ignore_index=IGNORE, reduction="mean")
        return {"total": total, "loss": loss, "dX": dX, "dW": dW}
    group = s["group"]
    group.step(s["g"], norm=s["norm"], max_norm=1.0) if c["clip"] else group.step(s["g"])
    m, v = group.moments()  # flat, each tensor from a whole block on
    got = {"p": s["p"], "m": m, "v": v}
    return got if s["master"] is None else {**got, "master": s["master"]}


def work(case):
    """Bytes and operations that a pass cannot do without: each input read once, each output written once."""
    if case["op"] == "loss":
        M, K, V = case["M"], case["K"], case["V"]
        rows = 8 * M + 4 * M * bool(case["weights"])  # targets and weights
        if case["dir"] == "forward":
            return {"bytes": 2 * (M * K + K * V) + rows + 8 * M, "flops": 2 * M * K * V}
        return {"bytes": 4 * (M * K + K * V) + rows + 4 * M, "flops": 6 * M * K * V}
    param = {"f32": 8, "bf16": 4, "master": 10}[case["param"]]
    # the moments read and written; 8-bit ones with two exponents a block, and given back as bf16 values
    moments = 16 if case["states"] == 32 else 4 + 4 / BLOCK + 4
    grads = sum(n * (2 if kind is BF16 else 4) for n, kind in zip(_sizes(case), _kinds(case)))
    n = sum(_sizes(case))
    return {"bytes": n * (param + moments) + grads, "flops": 16 * n}


# ---- the definition in 64 bits ---------------------------------------------------------------------------------

def _exact_loss(case, s):
    M, vocab = case["M"], case["vocab"]
    flops = work(case)["flops"]
    if flops > 12e12:  # over some 20 seconds in 64 bits
        return None
    X = s["X"].double()
    pieces = [X.matmul(w.double()) for w in s["W"]]
    wide = torch.cat(pieces, 1)[:, :vocab]
    del pieces
    lse = torch.logsumexp(wide, 1)
    rows = (s["targets"] != IGNORE).nonzero()[:, 0]
    cols = s["targets"][rows]
    loss = torch.zeros(M, dtype=torch.float64, device="cuda")
    loss[rows] = lse[rows] - wide[rows, cols]
    if case["dir"] == "forward":
        return {"loss": loss, "lse": lse}
    w = torch.zeros_like(loss)
    w[rows] = 1.0 if s["weights"] is None else s["weights"].double()[rows]
    if rows.numel():
        w /= w.sum()
    prob = (wide - lse[:, None]).exp_()
    del wide
    prob[rows, cols] -= 1
    prob *= w[:, None]
    prob = torch.nn.functional.pad(prob, (0, case["V"] - vocab))
    dX, dW = 0, []
    for d, W in zip(prob.chunk(case["P"], 1), s["W"]):
        dX = dX + d.matmul(W.double().t())
        dW.append(X.t().matmul(d))
    return {"total": w.dot(loss), "loss": loss, "dX": dX, "dW": dW}


def _pow64(e):
    """2^e of an integer tensor in 64 bits, exactly."""
    return ((e.to(I64) + 1023) << 52).view(torch.float64)


def _held64(x, top, u, sign):
    """Values that blocks of 8-bit floats hold of x (rows), u their random numbers; `top`: exponent of a block's largest."""
    mag = x.abs()
    least = top[:, None] - (13 if sign else 29)  # exponent of the smallest normal value
    step = _pow64(torch.maximum(torch.frexp(mag)[1] - 1, least) - 3)
    held = torch.floor(mag / step + u) * step
    if not sign:  # what is not zero stays so
        held = torch.where((mag > 0) & (held == 0), step, held)
    return held * torch.sign(x)


def _exact_adam(case, s):
    t = s["step"] + 1
    coef = 1.0 if s["norm"] is None else min(1.0, 1.0 / (float(s["norm"]) + 1e-6))
    m, v = (x.double() for x in _moments(case, s))
    g = sum(x.double() for x in s["g_flat"]) * coef
    m, v = m + (g - m) * (1 - BETA1), v + (g ** 2 - v) * (1 - BETA2)
    w = s["p"].double() if s["master"] is None else s["master"].double()
    w = w - LR * (DECAY * w + m / (1 - BETA1 ** t) / ((v / (1 - BETA2 ** t)) ** 0.5 + EPS))
    got = {"p": w}
    if s["master"] is not None:
        got["master"] = w
    r = _noise(s, t) if case["states"] == 8 or case["param"] == "bf16" else None
    if case["param"] == "bf16":
        ulp = _pow64(torch.frexp(w)[1].clamp(min=-125) - 8)
        up = torch.floor(w.abs() / ulp + (_pcg(r) % 65536).double() / 65536)
        got["p"] = up * ulp * torch.sign(w)
    for k, x, sign in (("m", m, True), ("v", v, False)):
        got[k] = x
        if case["states"] == 8:
            rows, u = x.view(-1, BLOCK), ((r % 65536 if sign else r // 65536).double() + 0.5) / 65536
            top = torch.frexp(rows.abs().amax(1))[1] - 1
            got[k] = _held64(rows, top.clamp(min=-100), u.view(-1, BLOCK), sign).reshape(-1)
    return got


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_loss(case, s) if case["op"] == "loss" else _exact_adam(case, s)
