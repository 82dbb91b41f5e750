"""The training step example: gated block, loss, their gradients, the norm and AdamW run together."""
import importlib.util
import os

import pytest
import torch

import adamw64

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from resharding_tensor_parallelism_gb300 import _build
    _build.build()
    spec = importlib.util.spec_from_file_location("training_step", os.path.join(ROOT, "examples", "training_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_it_runs(example):
    losses = example.main(width=128, hidden=256, vocab=1003, ranks=4, rows=300, steps=4)
    assert len(losses) == 4 and all(torch.isfinite(torch.tensor(losses)))


def _inputs(rows, D, vocab, seed=4):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    X = torch.randn((rows, D), generator=gen, device="cuda").to(BF16)
    t = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    if rows > 1:
        t[::4] = -100
    return X, t


@pytest.mark.parametrize("states", [8, 32])
@pytest.mark.parametrize("rows", [1, 40, 300])
def test_step_against_plain_autograd(example, rows, states):
    """Gradients of one step against torch autograd in float64 on the same bf16 weights, and the update against its formula
    on the step's own gradients. Six intermediate tensors are rounded to bf16 (h, Hg, Hu, Y, exponentials, scaled rows, dh,
    dHg and dHu), each within 2^-8 of its values at random signs: 2^-4 of a gradient's norm leaves room for few rows."""
    D, F, V, P = 256, 512, 1000, 2
    model = example.NextToken(D, F, V - 3, P, seed=3, states=states)
    X, t = _inputs(rows, D, V - 3)
    wide = {k: torch.cat([w.double() for w in ws], dim).requires_grad_() for k, ws, dim in (
        ("Ag", model.Ag, 1), ("Au", model.Au, 1), ("B", model.B, 0), ("W", model.W, 1))}
    x = X.double()
    g = x @ wide["Ag"]
    h = x + (g * torch.sigmoid(g) * (x @ wide["Au"])) @ wide["B"]
    loss = torch.nn.functional.cross_entropy((h @ wide["W"])[:, :V - 3], t, ignore_index=-100)
    loss.backward()
    group, before = model.optimizer, [m.double().clone() for m in model.optimizer.masters]
    # a counted row may be the only one: rows[0] is ignored where there are several
    got, norm = model.step(X, t, max_norm=0.5)
    want = float(loss.detach())
    assert abs(float(got) - want) <= 2.0 ** -6 * want
    for i, (k, dim) in enumerate((("Ag", 1), ("Au", 1), ("B", 0), ("W", 1))):
        have = torch.cat(model.grads[i * P:(i + 1) * P], dim).double()
        assert float((have - wide[k].grad).norm()) <= 2.0 ** -4 * float(wide[k].grad.norm()), k
    total = torch.sqrt(sum(v.double().square().sum() for v in model.grads))
    assert abs(float(norm) - float(total)) <= 2.0 ** -22 * float(total)
    for i, (p, m, b, grad) in enumerate(zip(model.params, group.masters, before, model.grads)):
        zero = torch.zeros_like(b)
        new, _, _, bound, _, _ = adamw64.step(b, grad, zero, zero, 1, 2e-4, (0.9, 0.95), 1e-8, 0.01, norm, 0.5)
        assert ((m.double() - new).abs() <= bound).all(), i
        assert torch.equal(p, m.to(BF16))


def test_captured_steps_are_the_eager_ones(example):
    """The whole step in a graph, replayed, beside the same steps run eagerly."""
    a, b = (example.NextToken(128, 256, 1000, 2, seed=5) for _ in range(2))
    X, t = _inputs(300, 128, 1000, seed=6)
    for m in (a, b):
        m.step(X, t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, norm = a.step(X, t)
    for k in range(3):
        Y, u = _inputs(300, 128, 1000, seed=7 + k)
        X.copy_(Y)
        t.copy_(u)
        graph.replay()
        want, want_norm = b.step(X, t)
        assert torch.equal(loss, want) and torch.equal(norm, want_norm)
    assert int(a.optimizer.steps) == int(b.optimizer.steps) == 4
    for p, q in zip([*a.params, *a.optimizer.masters], [*b.params, *b.optimizer.masters]):
        assert torch.equal(p, q)
