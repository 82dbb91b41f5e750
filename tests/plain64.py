"""Plain float64 forms of the linear layer and the gated block (torch on the GPU), and the bounds their kernels are
held to.

Bounds, from the arithmetic of the kernels (bf16 operands, whose products are exact in float32):
  * a sum of n products in float32 is off by at most 1.2 n 2^-24 sum |terms| (n - 1 roundings in any order, the 1.2
    for the tensor core's alignment of its addends), the form of the MLP tests' bound;
  * an activation is Lipschitz with constant 1.13 (GELU's largest slope 1.1290, SiLU's 1.0998, the others less) and is
    evaluated to 2^-18 of max(|act|, |x| 2^-4) (expf to 1 ulp on arguments up to 88, the quotient to 2 ulp);
  * one rounding to bf16 is at most 2^-8 of the value (half a spacing, doubled for a value on a boundary); to float32
    2^-23."""
import math

import torch

BF16_REL = 2.0 ** -8
LIP = 1.13


def acc_bound(n, abs_sum):
    return 1.2 * max(n, 1) * 2.0 ** -24 * abs_sum


def act(name, x):
    if name == "none":
        return x.clone()
    if name == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if name == "silu":
        return x * torch.special.expit(x)
    if name == "gelu":
        return x * torch.special.ndtr(x)
    z = math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    return x * torch.special.expit(2 * z)


def act_grad(name, x):
    if name == "none":
        return torch.ones_like(x)
    if name == "relu":
        return (x > 0).double()
    if name == "silu":
        s = torch.special.expit(x)
        return s + x * s * torch.special.expit(-x)
    if name == "gelu":
        return torch.special.ndtr(x) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    z = math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    s = torch.special.expit(2 * z)
    return s + x * s * torch.special.expit(-2 * z) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * x * x)


def act_eval_bound(a, x):
    return 2.0 ** -18 * torch.maximum(a.abs(), x.abs() / 16)


def product(A, B):
    """(A B, float32 accumulation bound) in float64."""
    A, B = A.double(), B.double()
    return A @ B, acc_bound(A.shape[1], A.abs() @ B.abs())


def check(what, got, ref, err, rel):
    """Every element of got within err of ref plus its rounding (rel of the value)."""
    bound = err + rel * (ref.abs() + err) + 1e-37
    bad = ~((got.double() - ref).abs() <= bound)
    if bool(bad.any()):
        i = int(torch.nonzero(bad.reshape(-1))[0])
        raise AssertionError("%s: %d of %d elements outside the bound; first at %d: got %r, exact %r, bound %r" % (
            what, int(bad.sum()), bad.numel(), i, float(got.reshape(-1)[i]), float(ref.reshape(-1)[i]),
            float(bound.reshape(-1)[i])))


def rel_of(dtype):
    return BF16_REL if dtype == torch.bfloat16 else 2.0 ** -23
