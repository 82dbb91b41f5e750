"""Plain float64 form of the vocabulary-split cross entropy and its gradients, with the bounds that its kernels are held
to. Runs where its tensors are."""
import torch

EPS = 2.0 ** -24  # half a step of float32
BF16 = 2.0 ** -8  # and of bf16, relative


def forward(X, W, targets, vocab, ignore):
    """(loss, lse, logits [M, vocab], counted rows) of one whole W [K, V], everything float64."""
    logits = X.double() @ W.double()[:, :vocab]
    lse = torch.logsumexp(logits, 1)
    counted = targets != ignore
    at = targets.long().clamp(0, vocab - 1)
    loss = lse - logits.gather(1, at[:, None])[:, 0]
    loss[counted & ((targets < 0) | (targets >= vocab))] = float("nan")
    loss[~counted] = 0.0
    return loss, lse, logits, counted


def logit_error(X, W, vocab):
    """How far a float32 logit of the bf16 operands may be off, per row (the largest over its columns)."""
    return 1.2 * X.shape[1] * EPS * (X.double().abs() @ W.double()[:, :vocab].abs()).amax(1)


def lse_bound(X, W, vocab, lse, logits):
    """Of float32 statistics: the logits' error; three roundings of a logit times log2(e); sums over at most 128 terms in a
    row of additions (2^-17), of exponentials within 2^-21; and the last roundings."""
    return logit_error(X, W, vocab) + 4 * EPS * logits.abs().amax(1) + 2.0 ** -17 + 2.0 ** -20 + 4 * EPS * lse.abs()


def gradients(X, W, targets, vocab, ignore, weights=None, mean=True, scale=1.0):
    """(total, loss, dX, dW, bound of dX, bound of dW), the bounds for float32 outputs: add |value| * 2^-8 for bf16 ones."""
    loss, lse, logits, counted = forward(X, W, targets, vocab, ignore)
    w = torch.ones_like(loss) if weights is None else weights.double()
    w = torch.where(counted, w, torch.zeros_like(w))
    total = torch.where(w != 0, w * loss, torch.zeros_like(loss)).sum()
    denom = w.sum() if mean else torch.ones_like(total)
    total = total / denom if denom != 0 else torch.zeros_like(total)
    g = scale * w / denom if denom != 0 else torch.zeros_like(w)
    p = (logits - lse[:, None]).exp() * g[:, None]
    d = p.clone()
    rows = torch.nonzero(counted & (targets >= 0) & (targets < vocab))[:, 0]
    d[rows, targets.long()[rows]] -= g[rows]
    # Both products read d's exponentials (at the target: less the row's sum) rounded to bf16, half a step of d itself; the
    # row's factor takes the target's error back, which gives its half step to the row's others. dW reads rows of X that
    # were multiplied by the factor and rounded, half a step more of every term. The exponentials and the factor are off
    # by the row's error (each once).
    row = p.abs() * lse_bound(X, W, vocab, lse, logits)[:, None] * 2
    others = d.abs().clone()
    others[rows, targets.long()[rows]] = 0
    ex = 2 * BF16 * others * 1.02 + 8 * EPS * d.abs() + row
    ew = ex + BF16 * d.abs() * 1.02
    pad = W.shape[1] - vocab
    d, ex, ew = (torch.nn.functional.pad(t, (0, pad)) for t in (d, ex, ew))
    Xd, Wd = X.double(), W.double()
    dX, dW = d @ Wd.t(), Xd.t() @ d
    bx = ex @ Wd.abs().t() + 1.2 * W.shape[1] * EPS * (d.abs() @ Wd.abs().t())
    bw = Xd.abs().t() @ ew + 1.2 * X.shape[0] * EPS * (Xd.abs().t() @ d.abs())
    return total, loss, dX, dW, bx, bw
