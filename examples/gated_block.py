"""A gated tensor-parallel block on virtual ranks of one GPU: trained for a few steps, then used to decode tokens.

    h   = X Wi + bi                     column-parallel linear layer, gathered to the full width
    out = h + glu(h)                    gated feed-forward block with its residual
    Z   = sum_i out_i Wo_i + bo + X     row-parallel linear layer with the input as residual

One training step is the forward pass, the backward passes of the three layers, clipping of every rank's gradients by
their global norm, and a plain gradient step. Run: python examples/gated_block.py
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import resharding_tensor_parallelism_gb300 as rtp

BF16, F32 = torch.bfloat16, torch.float32


class GatedBlock:
    """Weights and gradient buffers of the block, one list entry per rank; biases of the row-parallel layer are whole."""

    def __init__(self, width, hidden, ranks, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def shards(rows, cols, n=ranks):
            return [(torch.randn((rows, cols), generator=gen, device="cuda") / (rows * (n if rows < width else 1)) ** 0.5)
                    .to(BF16) for _ in range(n)]

        D, F, P = width, hidden, ranks
        self.ranks, self.width = P, D
        self.Wi, self.Wo = shards(D, D // P), shards(D // P, D)
        self.Ag, self.Au, self.B = shards(D, F // P), shards(D, F // P), shards(F // P, D)
        self.bi = [torch.zeros(D // P, dtype=BF16, device="cuda") for _ in range(P)]
        self.bo = torch.zeros(D, dtype=BF16, device="cuda")
        self.params = [*self.Wi, *self.Ag, *self.Au, *self.B, *self.Wo, *self.bi, self.bo]
        # weight gradients are float32, as a program that adds up micro-batches keeps them
        self.grads = [torch.zeros(p.shape, dtype=F32, device="cuda") for p in self.params]
        self.group = rtp.GradGroup(self.grads)
        self.split = rtp.spec_nd_sbp((P,), (("S", 1),))
        self.whole = rtp.spec_nd_sbp((P,), ("B",))

    def _gather(self, pieces, rows):
        """Column pieces [rows, width/P] to the whole [rows, width] (an all-gather: every rank gets the same)."""
        return rtp.reshard(pieces, (rows, self.width), self.split, self.whole)[0]

    def _scatter(self, whole):
        return rtp.shard(whole, self.split)

    def forward(self, X):
        """Inference, any number of rows (one token at a time while decoding)."""
        h = self._gather(rtp.tp_linear(X, self.Wi, bias=self.bi), X.shape[0])
        out = rtp.tp_glu(h, self.Ag, self.Au, self.B, residual=h)
        return rtp.tp_linear(self._scatter(out), self.Wo, split="row", bias=self.bo, residual=X)[0]

    def step(self, X, target, lr=0.2, max_norm=1.0):
        """One training step on 0.5 mean (Z - target)^2. Returns (loss, gradient norm), both on the GPU."""
        M, P = X.shape[0], self.ranks
        h = self._gather(rtp.tp_linear(X, self.Wi, bias=self.bi), M)
        out, Y, Hg, Hu = rtp.tp_glu_train_forward(h, self.Ag, self.Au, self.B, residual=h)
        out_p = self._scatter(out)
        Z = rtp.tp_linear(out_p, self.Wo, split="row", bias=self.bo, residual=X)[0]
        diff = Z.float() - target.float()
        loss = 0.5 * diff.square().mean()
        dZ = (diff / diff.numel()).to(BF16)

        g = self.grads
        gWi, gAg, gAu, gB, gWo = (g[i * P:(i + 1) * P] for i in range(5))
        gbi, gbo = g[5 * P:6 * P], g[6 * P:]
        d_out_p, _, _ = rtp.tp_linear_backward(out_p, self.Wo, dZ, split="row", dW=gWo, db=gbo)
        d_out = self._gather(d_out_p, M)
        dh, _, _, _ = rtp.tp_glu_backward(h, self.Ag, self.Au, self.B, Hg, Hu, Y, d_out, dAg=gAg, dAu=gAu, dB=gB)
        dh = dh + d_out  # the residual's gradient is d_out itself
        rtp.tp_linear_backward(X, self.Wi, self._scatter(dh), dW=gWi, db=gbi)

        norm, _ = self.group.clip(max_norm)
        for p, grad in zip(self.params, g):
            p.copy_(p.float() - lr * grad)
        return loss, norm


def main(width=1024, hidden=4096, ranks=4, rows=512, steps=20, decode=8):
    block = GatedBlock(width, hidden, ranks)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    X = torch.randn((rows, width), generator=gen, device="cuda").to(BF16)
    target = torch.randn((rows, width), generator=gen, device="cuda").to(BF16)
    losses = []
    for k in range(steps):
        loss, norm = block.step(X, target)
        losses.append(float(loss))
        if k % 5 == 0 or k == steps - 1:
            print("step %2d: loss %.4f, gradient norm %.4f" % (k, losses[-1], float(norm)))
    token = X[:1].contiguous()
    for _ in range(decode):  # each output row is the next input
        token = block.forward(token)
        token = (token / token.float().square().mean().sqrt()).to(BF16)
    print("decoded %d tokens, last one's first values: %s" % (decode, [round(float(v), 3) for v in token[0, :4]]))
    assert rtp.device_error() == 0
    return losses


if __name__ == "__main__":
    main()
