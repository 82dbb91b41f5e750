"""GPU parity of the gated feed-forward block and its backward pass against float64, with every output in a guarded
buffer. Bounds: plain64.py. Each product is checked against the bf16 operands that it read (Y, dHg and dHu are outputs
too, and are checked on their own), so the bounds stay those of one product and one rounding."""
import pytest
import torch

import plain64 as p64
from gpu_util import Guarded

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
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


def _normal(shape, std=1.0, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)


def _case(P, M, K, F, N, seed):
    Fp = F // P
    X = _normal((M, K), seed=seed)
    Ag = [_normal((K, Fp), 1.5 / K ** 0.5, seed + 1 + i) for i in range(P)]
    Au = [_normal((K, Fp), 1.0 / K ** 0.5, seed + 10 + i) for i in range(P)]
    B = [_normal((Fp, N), 1.0 / F ** 0.5, seed + 20 + i) for i in range(P)]
    return X, Ag, Au, B, _normal((M, N), seed=seed + 30)


def _check_mid(what, act, X, Ag, Au, Y, Hg=None, Hu=None, rows=slice(None)):
    for i in range(len(Ag)):
        (hg, eg), (hu, eu) = p64.product(X[rows], Ag[i]), p64.product(X[rows], Au[i])
        if Hg is not None:
            p64.check(what + " Hg", Hg[i][rows], hg, eg, p64.BF16_REL)
            p64.check(what + " Hu", Hu[i][rows], hu, eu, p64.BF16_REL)
        a = p64.act(act, hg)
        ea = p64.LIP * eg + p64.act_eval_bound(a, hg)
        p64.check(what + " Y", Y[i][rows], a * hu, ea * (hu.abs() + eu) + a.abs() * eu, p64.BF16_REL)


def _check_z(what, Y, B, R, Z, rows=slice(None)):
    z, e = p64.product(torch.cat([y[rows] for y in Y], 1), torch.cat(B, 0))
    if R is not None:
        z = z + R[rows].double()
        e = e + 2.0 ** -23 * (z.abs() + e)
    p64.check(what + " Z", Z[rows], z, e, p64.rel_of(Z.dtype))


def _forward(P, M, K, F, N, act, residual=True, out_dtype=BF16, train=False, seed=0):
    X, Ag, Au, B, R = _case(P, M, K, F, N, seed)
    R = R if residual else None
    g = Guarded()
    Y = g.many([(M, F // P)] * P, BF16, "Y")
    Z = g.empty((M, N), out_dtype, "Z")
    what = "glu P=%d M=%d K=%d F=%d N=%d %s" % (P, M, K, F, N, act)
    Hg = Hu = None
    if train:
        Hg, Hu = (g.many([(M, F // P)] * P, BF16, n) for n in ("Hg", "Hu"))
        rtp.tp_glu_train_forward(X, Ag, Au, B, act=act, residual=R, Y=Y, Hg=Hg, Hu=Hu, Z=Z)
    else:
        rtp.tp_glu(X, Ag, Au, B, act=act, residual=R, Y=Y, Z=Z)
    g.check(what)
    _check_mid(what, act, X, Ag, Au, Y, Hg, Hu)
    _check_z(what, Y, B, R, Z)
    return Z


@pytest.mark.parametrize("M", [1, 2, 4, 16, 17, 37, 64, 100, 128, 129, 255, 256, 257, 290, 600])
def test_rows_from_one_to_many(M):
    _forward(2, M, 200, 2 * 328, 264, "silu", train=M % 2 == 0, seed=M)


@pytest.mark.parametrize("P,M,K,F,N", [
    (1, 1, 8, 8, 8), (8, 3, 64, 64, 8), (3, 19, 72, 3 * 136, 88), (8, 1, 4096, 8 * 520, 1032), (1, 257, 8, 8, 8),
    (3, 300, 136, 3 * 72, 520), (8, 520, 264, 8 * 40, 264), (5, 1021, 520, 5 * 136, 136), (2, 7, 2056, 5648, 2056),
    (4, 130, 64, 4 * 1000, 64)])
@pytest.mark.parametrize("train", [False, True])
def test_ragged_sizes(P, M, K, F, N, train):
    _forward(P, M, K, F, N, "gelu_tanh", residual=M % 2 == 1, train=train, seed=K)


@pytest.mark.parametrize("P,K,F,N", [(1, 2048, 3192, 264), (5, 2056, 5 * 520, 6152), (2, 64, 2 * 1032, 6392)])
@pytest.mark.parametrize("over", [1, 64])
@pytest.mark.parametrize("train", [False, True])
def test_rows_left_over_by_the_last_whole_tile(P, K, F, N, over, train):
    """25 column tiles in the first product, the second, or both: up to 64 rows over go to the few-row kernel."""
    _forward(P, 768 + over, K, F, N, "silu", train=train, seed=over)


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "silu", "relu"])
@pytest.mark.parametrize("M", [23, 270])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
def test_activations_and_types(act, M, out_dtype):
    _forward(2, M, 136, 2 * 200, 72, act, True, out_dtype, True, seed=3)


def test_full_size():
    """The MLP configuration, gated: sampled rows, and the same bits from a second run."""
    P, M, K, F, N = 8, 8192, 4096, 16384, 4096
    X, Ag, Au, B, R = _case(P, M, K, F, N, 5)
    rows = [0, 1, 127, 128, 255, 256, 4095, 8191]
    Z, Y, Hg, Hu = rtp.tp_glu_train_forward(X, Ag, Au, B, residual=R)
    _check_mid("full size", "silu", X, Ag, Au, Y, Hg, Hu, rows)
    _check_z("full size", Y, B, R, Z, rows)
    assert torch.equal(Z, rtp.tp_glu(X, Ag, Au, B, residual=R))
    one = X[:1].contiguous()
    first = rtp.tp_glu(one, Ag, Au, B)
    for _ in range(20):  # back to back: each call's weights are fetched while the one before it ends
        assert torch.equal(first, rtp.tp_glu(one, Ag, Au, B))


def test_weights_written_just_before_the_call():
    """The second product fetches its weights early; a kernel that writes them right before the call is waited for."""
    P, M, K, F, N = 2, 3, 256, 2 * 2048, 2048
    X, Ag, Au, B, R = _case(P, M, K, F, N, 6)
    want = rtp.tp_glu(X, Ag, Au, B, residual=R)
    for _ in range(30):
        B2 = [torch.zeros_like(b) for b in B]
        big = torch.randn(4096, 4096, device="cuda")
        big = big @ big  # keeps the GPU busy while the copies and the call are queued
        for b2, b in zip(B2, B):
            b2.copy_(b)
        assert torch.equal(rtp.tp_glu(X, Ag, Au, B2, residual=R), want)


def test_no_rows():
    Ag, Au, B = ([torch.ones(s, dtype=BF16, device="cuda")] * 2 for s in ((16, 24), (16, 24), (24, 8)))
    X = torch.empty((0, 16), dtype=BF16, device="cuda")
    Z, Y, Hg, Hu = rtp.tp_glu_train_forward(X, Ag, Au, B)
    assert Z.shape == (0, 8) and Y[1].shape == (0, 24)
    dX, dAg, dAu, dB = rtp.tp_glu_backward(X, Ag, Au, B, Hg, Hu, Y, torch.empty((0, 8), dtype=BF16, device="cuda"))
    assert dX.shape == (0, 16) and all(not bool(t.any()) for t in dAg + dAu + dB)


def test_special_values_stay_in_their_rows():
    for M in (40, 300):
        X, Ag, Au, B, R = _case(2, M, 136, 2 * 72, 264, 8)
        clean = rtp.tp_glu(X, Ag, Au, B, residual=R)
        X[3, 7], X[11, 0] = float("nan"), float("inf")
        got = rtp.tp_glu(X, Ag, Au, B, residual=R)
        rows = torch.ones(M, dtype=torch.bool, device="cuda")
        rows[[3, 11]] = False
        assert torch.equal(got[rows], clean[rows]) and bool(got[3].isnan().all())


def test_another_stream_and_graph():
    for M in (1, 300):
        X, Ag, Au, B, R = _case(4, M, 256, 4 * 264, 136, 11)
        want = rtp.tp_glu(X, Ag, Au, B, residual=R)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = [rtp.tp_glu(X, Ag, Au, B, residual=R, stream=side) for _ in range(8)]
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(t, want) for t in got)
        Y, Z = [torch.empty((M, 264), dtype=BF16, device="cuda") for _ in range(4)], torch.empty_like(want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rtp.tp_glu(X, Ag, Au, B, residual=R, Y=Y, Z=Z)
        X.mul_(2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Z, rtp.tp_glu(X, Ag, Au, B, residual=R)) and not torch.equal(Z, want)


# ---- backward ----------------------------------------------------------------------------------------------------


def _backward(P, M, K, F, N, act, dx_dtype=BF16, dw_dtype=BF16, seed=0, sample=None):
    X, Ag, Au, B, _ = _case(P, M, K, F, N, seed)
    Fp = F // P
    Hg = [_normal((M, Fp), 1.5, seed + 40 + i) for i in range(P)]
    Hu = [_normal((M, Fp), 1.0, seed + 50 + i) for i in range(P)]
    Y = [_normal((M, Fp), 0.7, seed + 60 + i) for i in range(P)]
    dZ = _normal((M, N), 0.5, seed + 70)
    g = Guarded()
    dHg, dHu = g.many([(M, Fp)] * P, BF16, "dHg"), g.many([(M, Fp)] * P, BF16, "dHu")
    dX = g.empty((M, K), dx_dtype, "dX")
    dAg, dAu = g.many([(K, Fp)] * P, dw_dtype, "dAg"), g.many([(K, Fp)] * P, dw_dtype, "dAu")
    dB = g.many([(Fp, N)] * P, dw_dtype, "dB")
    rtp.tp_glu_backward(X, Ag, Au, B, Hg, Hu, Y, dZ, act=act, dHg=dHg, dHu=dHu, dX=dX, dAg=dAg, dAu=dAu, dB=dB)
    what = "glu backward P=%d M=%d K=%d F=%d N=%d %s" % (P, M, K, F, N, act)
    g.check(what)
    for i in range(P):
        dY, e = p64.product(dZ, B[i].T)
        hg, hu = Hg[i].double(), Hu[i].double()
        a, d = p64.act(act, hg), p64.act_grad(act, hg)
        ea, ed = p64.act_eval_bound(a, hg), 2.0 ** -17  # the slope is at most 1.13
        p64.check(what + " dHg", dHg[i], dY * hu * d, e * hu.abs() * d.abs() + (dY.abs() + e) * hu.abs() * ed, p64.BF16_REL)
        p64.check(what + " dHu", dHu[i], dY * a, e * a.abs() + (dY.abs() + e) * ea, p64.BF16_REL)
        p64.check(what + " dAg", dAg[i], *p64.product(X.T, dHg[i]), p64.rel_of(dw_dtype))
        p64.check(what + " dAu", dAu[i], *p64.product(X.T, dHu[i]), p64.rel_of(dw_dtype))
        p64.check(what + " dB", dB[i], *p64.product(Y[i].T, dZ), p64.rel_of(dw_dtype))
    p64.check(what + " dX", dX, *p64.product(torch.cat(dHg + dHu, 1), torch.cat(Ag + Au, 1).T), p64.rel_of(dx_dtype))


@pytest.mark.parametrize("P,M,K,F,N", [(1, 1, 8, 8, 8), (2, 5, 72, 2 * 136, 88), (3, 257, 136, 3 * 72, 520),
                                       (8, 300, 264, 8 * 40, 72), (8, 129, 64, 8 * 264, 64), (1, 520, 520, 1000, 136)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward(P, M, K, F, N, act):
    _backward(P, M, K, F, N, act, seed=M)


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "silu", "relu"])
@pytest.mark.parametrize("dx,dw", [(F32, F32), (BF16, F32), (F32, BF16)])
def test_backward_types(act, dx, dw):
    _backward(2, 290, 136, 2 * 200, 72, act, dx, dw, seed=2)


def test_gradients_against_differences():
    """Directional derivatives of sum(dZ * Z) along the gradients' signs, by central differences of the float32
    forward. The steps move a pre-activation by at most about 0.1, as in the linear layer's test (truncation below 1e-2
    of the derivative); Y's rounding to bf16, at random over F x M values, and the kept values' rounding stay below
    that: 2e-2 of the derivative in all, 4e-2 for B, whose differences hold the rounding of B's own steps only."""
    P, M, K, F, N, act = 2, 64, 128, 2 * 128, 256, "silu"
    X, Ag, Au, B, R = _case(P, M, K, F, N, 90)
    dZ = _normal((M, N), 1.0, 91)
    _, Y, Hg, Hu = rtp.tp_glu_train_forward(X, Ag, Au, B, act=act, residual=R)
    dX, dAg, dAu, dB = rtp.tp_glu_backward(X, Ag, Au, B, Hg, Hu, Y, dZ, act=act, dx_dtype=F32, dw_dtype=F32)

    def loss(a):
        Z = rtp.tp_glu(a["X"][0], a["Ag"], a["Au"], a["B"], act=act, residual=R, out_dtype=F32)
        return float((Z.double() * dZ.double()).sum())

    base = {"X": [X], "Ag": Ag, "Au": Au, "B": B}
    for which, grads, size in (("X", [dX], 2.0 ** -4 / K ** 0.5), ("Ag", dAg, 2.0 ** -4 / K), ("Au", dAu, 2.0 ** -4 / K),
                               ("B", dB, 2.0 ** -4 / F)):
        plus = [(t.float() + size * g.sign()).to(BF16) for t, g in zip(base[which], grads)]
        minus = [(t.float() - size * g.sign()).to(BF16) for t, g in zip(base[which], grads)]
        along = sum(float(((p.double() - m.double()) * g.double()).sum()) for p, m, g in zip(plus, minus, grads))
        diff = loss({**base, which: plus}) - loss({**base, which: minus})
        assert abs(diff - along) <= (4e-2 if which == "B" else 2e-2) * abs(along), (which, diff, along)
