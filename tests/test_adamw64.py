"""The plain float64 AdamW step and 8-bit moments that the kernels are compared with, on the CPU."""
import torch

import adamw64 as plain


def test_step_is_torchs():
    gen = torch.Generator().manual_seed(0)
    p = torch.randn(50, generator=gen, dtype=torch.float64)
    q = torch.nn.Parameter(p.clone())
    opt = torch.optim.AdamW([q], lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    m = v = torch.zeros_like(p)
    for t in range(1, 6):
        g = torch.randn(50, generator=gen, dtype=torch.float64)
        q.grad = g.clone()
        opt.step()
        p, m, v, _, _, _ = plain.step(p, g, m, v, t, 1e-2, (0.8, 0.95), 1e-6, 0.1)
    assert torch.allclose(p, q.detach(), atol=1e-14)


def test_every_code_stands_for_itself():
    """Values that a code stands for are kept, whatever the random number."""
    for signed in (True, False):
        top = 7 if signed else 15
        codes = torch.arange(256)
        size = codes % 128 if signed else codes
        biggest = top + (7 if signed else 15)  # of the exponents: larger ones are only reached by rounding up
        codes = codes[size // 8 <= biggest]
        codes = torch.cat([codes, torch.full((-codes.numel() % 128,), biggest * 8)])
        tops = torch.full((codes.numel() // 128,), 127 + top)
        lead = codes.view(-1, 128)
        lead[:, 0] = biggest * 8  # each block has its largest exponent
        x = plain.values(lead.reshape(-1), tops, signed)
        for u in (0.0, 0.5, 0.999):
            code, e, _ = plain.quantise(x, torch.full_like(x, u), signed)
            assert torch.equal(e, tops)
            assert torch.equal(plain.values(code, e, signed), x)


def test_rounding_keeps_the_mean():
    gen = torch.Generator().manual_seed(1)
    x = torch.rand(128, generator=gen, dtype=torch.float64) + 0.01
    x[0] = 1.0
    u = (torch.arange(1000, dtype=torch.float64) + 0.5) / 1000
    for signed in (True, False):
        got = torch.stack([plain.values(*plain.quantise(x, torch.full_like(x, float(v)), signed)[:2], signed) for v in u])
        assert ((got.mean(0) - x).abs() <= x * 2.0 ** -3 / 1000).all()


def test_nothing_positive_becomes_zero():
    x = torch.full((128,), 1e-30, dtype=torch.float64)
    x[0] = 1.0
    code, e, _ = plain.quantise(x, torch.zeros_like(x), False)
    assert (code > 0).all() and (plain.values(code, e, False) > 0).all()
