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


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M,K,form", [(128, 8, "few"), (256, 8, "whole"), (256, 2056, 4)])
def test_float32_outputs_keep_float32(act, M, K, form):
    """Relative to the value, tails included: e^u is off by at most one unit (2^-23), or twice as much where it is
    multiplied in as two halves, the reciprocal by one unit, and three roundings of 2^-24 follow: 3.5 2^-23, held to
    2^-21. tanh's argument u is off by at most 8 roundings of 2^-24 first: |u| 2^-21 more. GELU's polynomial is within
    8e-7 with its roundings and its quotient's, the exponential within 3 2^-24, two roundings follow: 1.1e-6, held to
    2^-19. Below 2^-126 numbers are spaced 2^-149. The bias gives the numbers between bf16's."""
    x = _bf16_numbers(-13.5 if act == "gelu" else -10.0 if act == "gelu_tanh" else -100.0, 40.0)
    bias = torch.tensor([0, 1, -1, 3, -5, 7, 11, -13], device="cuda").mul(2.0 ** -12).to(BF16)
    W = torch.zeros((K, 8), dtype=BF16, device="cuda")
    W[0] = 1

    def call(X, act):
        wide = torch.zeros((M, K), dtype=BF16, device="cuda")
        wide[:, 0] = X[:, 0]
        rtp.product_launches()
        got = rtp.tp_linear(wide, [W], act=act, bias=[bias], out_dtype=F32)[0]
        assert rtp.product_launches()[form] == 1
        return got

    got = _through(x, act, M, call).double()
    x = (x.float()[:, None] + bias.float()).double()  # one float32 addition, as the kernel's
    ref = _exact(act, x)
    u = 2 * (2 / torch.pi) ** 0.5 * (x + 0.044715 * x ** 3)
    rel = 2.0 ** -19 if act == "gelu" else 2.0 ** -21 * (1 + u.abs()) if act == "gelu_tanh" else 2.0 ** -21
    bad = ~((got - ref).abs() <= rel * ref.abs() + 2.0 ** -140)
    assert not bool(bad.any()), (act, float(x[bad][0]), float(got[bad][0]), float(ref[bad][0]), int(bad.sum()))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M", [16, 256])
def test_special_values(dtype, M):
    """NaN stays, +inf stays, 0 stays, and numbers far out give x or 0, in every activation."""
    x = torch.tensor([float("nan"), float("inf"), 0.0, -0.0, 3e38, -3e38, 1e25, -1e25, 200.0, -200.0], device="cuda").to(BF16)
    for act in ("gelu", "gelu_tanh", "silu", "relu"):
        got = _through(x, act, M, _linear(dtype))
        assert bool(got[0].isnan()) and float(got[1]) == float("inf") and not bool(got[2:4].any())
        assert got[4:].tolist() == [v if v > 0 else 0.0 for v in x[4:].tolist()], act
