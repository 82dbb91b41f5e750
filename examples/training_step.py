"""One whole training step on virtual ranks of one GPU: a gated block, the loss of a vocabulary-split output layer, the
gradients of both, and AdamW with clipping.

    h    = X + glu(X)                       gated feed-forward block with its residual
    loss = cross entropy of h [W_0 .. W_P-1]  the logits are never stored

Weights are bf16 with float32 copies that AdamW updates, moments are held in 8 bits; the gradients' norm stays on the GPU
and clips them within the update. Run: python examples/training_step.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import resharding_tensor_parallelism_gb300 as rtp

BF16, F32 = torch.bfloat16, torch.float32


class NextToken:
    """A gated block and an output layer over a vocabulary, one list entry per rank; the vocabulary's last columns may be
    padding (each rank has a multiple of 8)."""

    def __init__(self, width, hidden, vocab, ranks, seed=0, lr=2e-4, states=8):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        D, F, P = width, hidden, ranks
        V = (vocab + 8 * P - 1) // (8 * P) * 8 * P

        def shards(rows, cols, std):
            return [(torch.randn((rows, cols), generator=gen, device="cuda") * std).to(BF16) for _ in range(P)]

        self.ranks, self.vocab = P, vocab
        self.Ag, self.Au, self.B = shards(D, F // P, D ** -0.5), shards(D, F // P, D ** -0.5), shards(F // P, D, F ** -0.5)
        self.W = shards(D, V // P, D ** -0.5)
        self.params = [*self.Ag, *self.Au, *self.B, *self.W]
        self.grads = [torch.zeros(p.shape, dtype=F32, device="cuda") for p in self.params]
        self.norms = rtp.GradGroup(self.grads)
        self.optimizer = rtp.AdamWGroup(self.params, lr=lr, betas=(0.9, 0.95), weight_decay=0.01, masters=True, states=states,
                                        seed=seed)

    def backward(self, X, targets):
        """Gradients of the mean loss over the rows whose target is not -100. Returns the loss, on the GPU."""
        P, g = self.ranks, self.grads
        h, Y, Hg, Hu = rtp.tp_glu_train_forward(X, self.Ag, self.Au, self.B, residual=X)
        loss, _, dh, _ = rtp.tp_cross_entropy_train(h, self.W, targets, vocab=self.vocab, dW=g[3 * P:])
        rtp.tp_glu_backward(X, self.Ag, self.Au, self.B, Hg, Hu, Y, dh, dAg=g[:P], dAu=g[P:2 * P], dB=g[2 * P:3 * P])
        return loss

    def step(self, X, targets, max_norm=1.0):
        """One training step. Returns (loss, gradient norm), both on the GPU."""
        loss = self.backward(X, targets)
        norm = self.norms.norm()
        self.optimizer.step(self.grads, norm=norm, max_norm=max_norm)
        return loss, norm

    def log_probs(self, X, targets):
        """Log probabilities of the targets, any number of rows (one token at a time while decoding)."""
        h = rtp.tp_glu(X, self.Ag, self.Au, self.B, residual=X)
        return -rtp.tp_cross_entropy(h, self.W, targets, vocab=self.vocab)[0]


def main(width=512, hidden=2048, vocab=8003, ranks=4, rows=1024, steps=20):
    model = NextToken(width, hidden, vocab, ranks)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    X = torch.randn((rows, width), generator=gen, device="cuda").to(BF16)
    targets = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    targets[:rows // 8] = -100  # a prompt that is not learned
    losses = []
    for k in range(steps):
        loss, norm = model.step(X, targets)
        losses.append(float(loss))
        if k % 5 == 0 or k == steps - 1:
            print("step %2d: loss %.4f, gradient norm %.4f" % (k, losses[-1], float(norm)))
    print("log probability of one row's target: %.3f" % float(model.log_probs(X[-1:].contiguous(), targets[-1:])))
    assert rtp.device_error() == 0
    return losses


if __name__ == "__main__":
    main()
