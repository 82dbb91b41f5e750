"""GPU parity of the activations alone: every bf16 number of a range goes through a product that leaves it as it is
(one column of ones in the weight), so that the output is the activation of it, rounded once."""
import pytest
import torch

import plain64 as p64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
TINY = 2.0 ** -125  # exponentials below 2^-126 count as zero, and bf16 is spaced 2^-133 there
rtp = None


@pytest.fixture(scope="module", autouse=True)
def lib():
    global rtp
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from resharding_tensor_parallelism_gb300 import _build
    _build.build()
    import resharding_tensor_parallelism_gb300 as m
    rtp = m
    yield
    assert m.device_error() == 0


def _bf16_numbers(lo, hi):
    """Every bf16 number in [lo, hi], in one column."""
    bits = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16)
    x = bits.view(BF16)
    x = x[x.isfinite() & (x >= lo) & (x <= hi)]
    return x.cuda()


def _through(x, act, M, call):
    """x, padded to a multiple of M rows and cut into calls of M rows (one K column holds x, the weight ones)."""
    pad = torch.cat([x, x[:1].expand(-len(x) % M)]).view(-1, M)
    got = []
    for part in pad:
        X = torch.zeros((M, 8), dtype=BF16, device="cuda")
        X[:, 0] = part
        got.append(call(X, act))
    return torch.cat(got)[:len(x)]


def _linear(out_dtype):
    W = torch.zeros((8, 8), dtype=BF16, device="cuda")
    W[0] = 1
    return lambda X, act: rtp.tp_linear(X, [W], act=act, out_dtype=out_dtype)[0][:, 3]


def _glu(X, act):
    """act(x) * 1: the up projection picks a column of ones."""
    X[:, 1] = 1
    Ag, Au = (torch.zeros((8, 8), dtype=BF16, device="cuda") for _ in range(2))
    Ag[0], Au[1] = 1, 1
    return rtp.tp_glu(X, [Ag], [Au], [torch.eye(8, dtype=BF16, device="cuda")], act=act)[:, 3]


def _exact(act, x):
    """The activation in float64, accurate relative to itself in the tails (ndtr is (1 + erf) / 2, which is not)."""
    return 0.5 * x * torch.erfc(-x * 0.5 ** 0.5) if act == "gelu" else p64.act(act, x)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M", [128, 256])  # the few-row kernel, the pair kernel
@pytest.mark.parametrize("what", ["linear", "glu"])
def test_bf16_outputs_are_rounded_once(act, M, what):
    """Each output is the rounding to bf16 of a value within 2^-13 of the exact one, tails included: the exponent, at
    most 88, is off by at most 5 roundings of 2^-24 (2^-15.7 of the value; tanh's argument, of more steps, by twice
    that), the rest by a few roundings (5e-6 at most). Rounding is monotonous, so the output lies between the rounded
    ends of that interval. A product by one, or by the identity, adds nothing."""
    x = _bf16_numbers(-13.0 if act == "gelu" else -6.5 if act == "gelu_tanh" else -84.0, 40.0)
    ref = _exact(act, x.double())
    got = _through(x, act, M, _linear(BF16) if what == "linear" else _glu)
    err = 2.0 ** -13 * ref.abs() + TINY
    bad = ~((got >= (ref - err).to(BF16)) & (got <= (ref + err).to(BF16)))
    assert not bool(bad.any()), (act, float(x[bad][0]), float(got[bad][0]), float(ref[bad][0]), int(bad.sum()))
