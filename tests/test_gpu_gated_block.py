"""The gated block example: the linear layers, the gated feed-forward block, their backward passes, resharding and
gradient clipping run together as a training step and as decoding."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from resharding_tensor_parallelism_gb300 import _build
    _build.build()
    spec = importlib.util.spec_from_file_location("gated_block", os.path.join(ROOT, "examples", "gated_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_training_lowers_the_loss(example):
    losses = example.main(width=256, hidden=512, ranks=4, rows=300, steps=12, decode=3)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_step_against_plain_autograd(example, rows):
    """Every gradient of one step against torch autograd in float64 on the same bf16 weights. The step rounds seven
    intermediate tensors to bf16 (h, Y, Hg, Hu, out, d_out, dH's, dh), each at most 2^-8 of its values at random signs, so
    a gradient's error is within 7 * 2^-8 of its norm; 2^-4 leaves room for the few-row cases' small sums."""
    D, F, P = 256, 512, 2
    block = example.GatedBlock(D, F, P, seed=3)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    X = torch.randn((rows, D), generator=gen, device="cuda").to(BF16)
    target = torch.randn((rows, D), generator=gen, device="cuda").to(BF16)
    wide = {k: torch.cat([w.double() for w in ws], dim).requires_grad_() for k, ws, dim in (
        ("Wi", block.Wi, 1), ("Ag", block.Ag, 1), ("Au", block.Au, 1), ("B", block.B, 0), ("Wo", block.Wo, 0),
        ("bi", block.bi, 0), ("bo", [block.bo], 0))}
    h = X.double() @ wide["Wi"] + wide["bi"]
    g = h @ wide["Ag"]
    out = h + (g * torch.sigmoid(g) * (h @ wide["Au"])) @ wide["B"]
    Z = out @ wide["Wo"] + wide["bo"] + X.double()
    loss = 0.5 * (Z - target.double()).square().mean()
    loss.backward()
    norm = torch.sqrt(sum(w.grad.square().sum() for w in wide.values()))
    got_loss, got_norm = block.step(X, target, lr=0.0, max_norm=1e9)
    want = float(loss.detach())
    assert abs(float(got_loss) - want) <= 2.0 ** -6 * want
    assert abs(float(got_norm) - float(norm)) <= 2.0 ** -4 * float(norm)
    grads = block.grads
    for i, (k, dim) in enumerate((("Wi", 1), ("Ag", 1), ("Au", 1), ("B", 0), ("Wo", 0), ("bi", 0))):
        got = torch.cat(grads[i * P:(i + 1) * P], dim).double()
        ref = wide[k].grad
        assert float((got - ref).norm()) <= 2.0 ** -4 * float(ref.norm()), k
    assert float((grads[6 * P].double() - wide["bo"].grad).norm()) <= 2.0 ** -4 * float(wide["bo"].grad.norm())
