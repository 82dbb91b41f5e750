"""The plain float64 cross entropy that the kernels are compared with: its gradients against differences, its values against
torch's own."""
import pytest
import torch

import cross_entropy64 as plain


@pytest.mark.parametrize("mean", [True, False])
@pytest.mark.parametrize("weighted", [True, False])
def test_gradients_are_the_losses_differences(mean, weighted):
    gen = torch.Generator().manual_seed(3)
    M, K, V, vocab = 5, 4, 11, 9
    X = torch.randn((M, K), generator=gen, dtype=torch.float64)
    W = torch.randn((K, V), generator=gen, dtype=torch.float64)
    t = torch.tensor([0, 8, -100, 4, 4])
    w = torch.rand((M,), generator=gen, dtype=torch.float64) if weighted else None

    def total(X, W):
        return plain.gradients(X, W, t, vocab, -100, w, mean, 3.0)[0] * 3.0

    _, _, dX, dW, _, _ = plain.gradients(X, W, t, vocab, -100, w, mean, 3.0)
    h = 1e-6
    for which, grad in ((0, dX), (1, dW)):
        for i in range(grad.shape[0]):
            for j in range(grad.shape[1]):
                a, b = [X.clone(), W.clone()], [X.clone(), W.clone()]
                a[which][i, j] += h
                b[which][i, j] -= h
                assert abs((total(*a) - total(*b)) / (2 * h) - grad[i, j]) < 1e-8


def test_values_are_torchs():
    gen = torch.Generator().manual_seed(4)
    X, W = torch.randn((7, 6), generator=gen).double(), torch.randn((6, 12), generator=gen).double()
    t = torch.tensor([1, -100, 3, 9, 0, -100, 9])
    loss, lse, logits, _ = plain.forward(X, W, t, 10, -100)
    want = torch.nn.functional.cross_entropy(X @ W[:, :10], t, reduction="none")
    assert torch.allclose(loss, want, atol=1e-14) and torch.allclose(lse, torch.logsumexp(X @ W[:, :10], 1), atol=1e-14)
