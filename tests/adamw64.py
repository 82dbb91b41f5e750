"""Plain float64 form of the AdamW step and of the 8-bit moments, with the bounds that the kernels are held to."""
import torch

EPS = 2.0 ** -24  # half a step of float32
BLOCK = 128


def pcg(x):
    """The output function of PCG-RXS-M-XS 32/32 on one step of its state, of integers (or int64 tensors) below 2^32."""
    x = (x * 747796405 + 2891336453) % 2 ** 32
    w = (((x >> ((x >> 28) + 4)) ^ x) * 277803737) % 2 ** 32
    return (w >> 22) ^ w


def noise(n, seed, tensor, step, device):
    key = pcg((pcg((pcg(seed) + tensor) % 2 ** 32) + step) % 2 ** 32)
    return pcg((torch.arange(n, device=device) + key) % 2 ** 32)


def pow2(e):
    """2^e of integers as float64, exactly (torch.ldexp is not, on a GPU)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _blocks(x):
    return torch.nn.functional.pad(x, (0, -x.numel() % BLOCK)).view(-1, BLOCK)


def quantise(x, u, signed):
    """(code, exponent byte per block, distance of each value's fraction from where it would round the other way, in steps):
    8-bit floats of blocks of x, rounded up where fraction + u >= 1."""
    rows, u = _blocks(x.double()), _blocks(u.double())
    top = (torch.frexp(rows.abs().amax(1))[1] - 1).clamp(min=-100)
    bias, most = (7, 7) if signed else (15, 15)
    z = rows.abs() * pow2(most - top)[:, None]
    e = torch.where(z > 0, torch.frexp(z)[1] - 1, -1000).clamp(min=1 - bias)
    steps = z * pow2(3 - e)
    whole = torch.floor(steps + u)
    near = (steps + u - torch.round(steps + u)).abs()
    code = whole + torch.where(e > 1 - bias, (e + bias - 1) * 8, torch.zeros_like(e))
    if signed:
        code = code + 128 * (rows < 0)
    else:
        code = torch.where((rows > 0) & (code == 0), torch.ones_like(code), code)
    n = x.numel()
    return code.to(torch.int64).view(-1)[:n], (top + 127).to(torch.int64), near.view(-1)[:n]


def values(code, top, signed):
    """What codes stand for."""
    n, code = code.numel(), _blocks(code.to(torch.int64))
    bias, most = (7, 7) if signed else (15, 15)
    size = code % 128 if signed else code
    e, frac = size // 8, (size % 8).double()
    z = torch.where(e > 0, 1 + frac / 8, frac / 8) * pow2(e.clamp(min=1) - bias)
    z = z * pow2(top.to(torch.int64).clamp(min=27) - 127 - most)[:, None]
    z[top.to(torch.int64) == 255] = float("nan")
    return torch.where(code >= 128, -z, z).view(-1)[:n] if signed else z.view(-1)[:n]


def step(p, g, m, v, t, lr, betas, eps, decay, norm=None, max_norm=1.0):
    """(p, m, v, bound of p, bound of m, bound of v) after step t (the first is 1), before any rounding: float64 of what the
    kernel starts from. Bounds: its float32 operations, and 2^-20 of the quotient."""
    b1, b2 = betas
    c = 1.0 if norm is None else min(1.0, max_norm / (float(norm) + 1e-6))
    p, g, m, v = p.double(), g.double() * c, m.double(), v.double()
    m1, v1 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    em = EPS * (3 * (b1 * m).abs() + 10 * ((1 - b1) * g).abs())
    ev = EPS * (3 * b2 * v + 18 * (1 - b2) * g * g)
    denom = (v1 / (1 - b2 ** t)).sqrt() + eps
    rate = lr / (1 - b1 ** t)
    upd = rate * m1 / denom
    new = p * (1 - lr * decay) - upd
    # sqrt halves v's relative error
    ep = EPS * (4 * p.abs() + new.abs()) + rate * em / denom + upd.abs() * (2.0 ** -20 + 8 * EPS + ev / v1.clamp(min=1e-300))
    return new, m1, v1, ep, em + EPS * m1.abs(), ev + EPS * v1
