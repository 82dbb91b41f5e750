"""GPU parity of the products whose tiles are shared by several SM pairs (each pair multiplies one part of the K range),
in every epilogue that they have, against float64. The launches' forms are read back, so that a case that is meant for
a form is known to have run in it. Bounds: plain64.py."""
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


def _forms(call):
    """The call's result, and the forms of its launches: those that ran, by name, with their number."""
    rtp.product_launches()
    got = call()
    return got, {k: n for k, n in rtp.product_launches().items() if n}


def _linear(P, M, K, N, act="none", out_dtype=BF16, keep_h=False, bias=True, residual=True, row=True, seed=0):
    """Runs and checks one layer; returns the forms of its launches and its outputs."""
    Kp, Np, outs = (K // P, N, 1) if row else (K, N // P, P)
    X = [_normal((M, Kp), seed=seed + i) for i in range(P if row else 1)]
    W = [_normal((Kp, Np), 1.5 / K ** 0.5, seed + 20 + i) for i in range(P)]
    b = [_normal((Np,), 0.5, seed + 40 + i) for i in range(outs)] if bias else None
    R = [_normal((M, Np), seed=seed + 60 + i) for i in range(outs)] if residual else None
    g = Guarded()
    out = g.many([(M, Np)] * outs, out_dtype, "out")
    H = g.many([(M, Np)] * outs, BF16, "H") if keep_h else None
    _, forms = _forms(lambda: rtp.tp_linear(X if row else X[0], W, split="row" if row else "column", bias=b, act=act,
                                            residual=R, H=H, out=out))
    what = "P=%d M=%d K=%d N=%d %s %s" % (P, M, K, N, act, forms)
    g.check(what)
    for i in range(outs):
        h, e = p64.product(torch.cat(X, 1), torch.cat(W, 0)) if row else p64.product(X[0], W[i])
        if bias:
            h = h + b[i].double()
            e = e + 2.0 ** -23 * (h.abs() + e)
        if keep_h:
            p64.check(what + " H", H[i], h, e, p64.BF16_REL)
        a = p64.act(act, h)
        err = p64.LIP * e + p64.act_eval_bound(a, h) if act != "none" else e
        if residual:
            a = a + R[i].double()
            err = err + 2.0 ** -23 * (a.abs() + err)
        p64.check(what, out[i], a, err, p64.rel_of(out_dtype))
    return forms, out


# ---- a device without room for wide clusters ------------------------------------------------------------------------

def test_clusters_that_do_not_fit_are_not_needed():
    """A size of cluster that finds no room is not used, and is no error."""
    assert _linear(1, 256, 4096, 264)[0] == {4: 1}
    for ctas, form in ((8, 3), (6, 2), (4, "whole"), (8, 3)):
        rtp.test_hook(rtp.HOOK_NO_CLUSTERS, ctas)
        assert _linear(1, 256, 4096, 264)[0] == {form: 1}, ctas
    assert _linear(1, 256, 4096, 264)[0] == {4: 1}  # the hook is for one product
    rtp.test_hook(rtp.HOOK_NO_CLUSTERS, 4)
    assert _linear(1, 5, 4096, 264)[0] == {"few": 1}
    rtp.test_hook(rtp.HOOK_NONE)
    assert _linear(1, 256, 4096, 264)[0] == {4: 1}


# ---- tiles shared by two, three and four pairs ------------------------------------------------------------------------
# 32 or more K blocks of 64 and a few tiles: four pairs share a tile, or, with no room for clusters of 8 or 6 CTAs, three
# or two.

PARTS = {4: None, 3: 8, 2: 6}


def _only(parts):
    if PARTS[parts]:
        rtp.test_hook(rtp.HOOK_NO_CLUSTERS, PARTS[parts])


@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "silu", "relu"])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("keep_h", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_layer_in_parts(parts, act, out_dtype, keep_h, residual):
    _only(parts)
    assert _linear(1, 300, 2056, 328, act, out_dtype, keep_h, bias=act != "relu", residual=residual, seed=parts)[0] == {parts: 1}


@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("P,M,K,N,row", [
    (1, 129, 4104, 8, True), (1, 256, 2048, 256, True), (1, 257, 2112, 72, True), (3, 300, 3 * 712, 200, True),
    (8, 200, 8 * 264, 1000, True), (5, 513, 5 * 520, 40, True), (2, 140, 2056, 2 * 168, False), (4, 290, 3080, 4 * 40, False)])
def test_ragged_layers_in_parts(parts, P, M, K, N, row):
    _only(parts)
    forms, out = _linear(P, M, K, N, "silu", keep_h=M % 2 == 0, row=row, seed=K)
    assert forms == {parts: 1}
    for _ in range(5):  # and the same bits from run to run
        _only(parts)
        again = _linear(P, M, K, N, "silu", keep_h=M % 2 == 0, row=row, seed=K)[1]
        assert all(torch.equal(a, b) for a, b in zip(out, again))


def _glu_case(P, M, K, F, N, seed):
    Fp = F // P
    X = _normal((M, K), seed=seed)
    Ag = [_normal((K, Fp), 1.5 / K ** 0.5, seed + 1 + i) for i in range(P)]
    Au = [_normal((K, Fp), 1.0 / K ** 0.5, seed + 10 + i) for i in range(P)]
    B = [_normal((Fp, N), 1.0 / F ** 0.5, seed + 20 + i) for i in range(P)]
    return X, Ag, Au, B


@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("train", [False, True])
@pytest.mark.parametrize("P,M,K,F,N,act", [
    (2, 300, 2056, 2 * 200, 72, "silu"), (2, 257, 2048, 2 * 136, 72, "gelu"), (1, 129, 4104, 8, 72, "gelu_tanh"),
    (1, 256, 2112, 256, 72, "relu"), (3, 200, 3080, 3 * 72, 72, "none"), (1, 513, 2056, 328, 264, "silu")])
def test_gated_block_in_parts(parts, train, P, M, K, F, N, act):
    """The product of both projections, in parts; the second product has few K blocks."""
    X, Ag, Au, B = _glu_case(P, M, K, F, N, 7)
    R, g = _normal((M, N), seed=5), Guarded()
    Y, Z = g.many([(M, F // P)] * P, BF16, "Y"), g.empty((M, N), BF16, "Z")
    Hg = Hu = None
    _only(parts)
    if train:
        Hg, Hu = (g.many([(M, F // P)] * P, BF16, n) for n in ("Hg", "Hu"))
        _, forms = _forms(lambda: rtp.tp_glu_train_forward(X, Ag, Au, B, act=act, residual=R, Y=Y, Hg=Hg, Hu=Hu, Z=Z))
    else:
        _, forms = _forms(lambda: rtp.tp_glu(X, Ag, Au, B, act=act, residual=R, Y=Y, Z=Z))
    assert forms == {parts: 1, "whole": 1}
    what = "glu P=%d M=%d K=%d F=%d %s in %d" % (P, M, K, F, act, parts)
    g.check(what)
    for i in range(P):
        (hg, eg), (hu, eu) = p64.product(X, Ag[i]), p64.product(X, Au[i])
        if train:
            p64.check(what + " Hg", Hg[i], hg, eg, p64.BF16_REL)
            p64.check(what + " Hu", Hu[i], hu, eu, p64.BF16_REL)
        a = p64.act(act, hg)
        ea = p64.LIP * eg + p64.act_eval_bound(a, hg)
        p64.check(what + " Y", Y[i], a * hu, ea * (hu.abs() + eu) + a.abs() * eu, p64.BF16_REL)
    z, e = p64.product(torch.cat(Y, 1), torch.cat(B, 0))
    z = z + R.double()
    p64.check(what + " Z", Z, z, e + 2.0 ** -23 * (z.abs() + e), p64.BF16_REL)


@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("P,M,K,F,N,act", [
    (2, 300, 72, 2 * 200, 2056, "silu"), (1, 257, 72, 328, 2048, "gelu"), (1, 129, 72, 8, 4104, "gelu_tanh"),
    (1, 256, 72, 256, 2112, "relu"), (3, 200, 72, 3 * 72, 3080, "none")])
def test_gated_block_backward_in_parts(parts, P, M, K, F, N, act):
    """The product with both gradients in its epilogue, in parts; the other products have few K blocks."""
    X, Ag, Au, B = _glu_case(P, M, K, F, N, 9)
    Fp = F // P
    Hg = [_normal((M, Fp), 1.5, 40 + i) for i in range(P)]
    Hu = [_normal((M, Fp), 1.0, 50 + i) for i in range(P)]
    Y = [_normal((M, Fp), 0.7, 60 + i) for i in range(P)]
    dZ, g = _normal((M, N), 0.5, 70), Guarded()
    dHg, dHu = g.many([(M, Fp)] * P, BF16, "dHg"), g.many([(M, Fp)] * P, BF16, "dHu")
    _only(parts)
    (dX, dAg, dAu, dB), forms = _forms(lambda: rtp.tp_glu_backward(X, Ag, Au, B, Hg, Hu, Y, dZ, act=act, dHg=dHg, dHu=dHu))
    assert forms == {parts: 1, "whole": 3}
    what = "glu backward P=%d M=%d F=%d N=%d %s in %d" % (P, M, F, N, act, parts)
    g.check(what)
    for i in range(P):
        dY, e = p64.product(dZ, B[i].T)
        hg, hu = Hg[i].double(), Hu[i].double()
        a, d = p64.act(act, hg), p64.act_grad(act, hg)
        ea, ed = p64.act_eval_bound(a, hg), 2.0 ** -17  # the slope is at most 1.13
        p64.check(what + " dHg", dHg[i], dY * hu * d, e * hu.abs() * d.abs() + (dY.abs() + e) * hu.abs() * ed, p64.BF16_REL)
        p64.check(what + " dHu", dHu[i], dY * a, e * a.abs() + (dY.abs() + e) * ea, p64.BF16_REL)
        p64.check(what + " dAg", dAg[i], *p64.product(X.T, dHg[i]), p64.BF16_REL)
        p64.check(what + " dAu", dAu[i], *p64.product(X.T, dHu[i]), p64.BF16_REL)
        p64.check(what + " dB", dB[i], *p64.product(Y[i].T, dZ), p64.BF16_REL)
    p64.check(what + " dX", dX, *p64.product(torch.cat(dHg + dHu, 1), torch.cat(Ag + Au, 1).T), p64.BF16_REL)


def _addresses(ts):
    return rtp._ptrs([t.data_ptr() for t in ts])


@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("P,M,K,N", [(1, 300, 264, 2056), (3, 129, 72, 3 * 712), (4, 513, 40, 4 * 520)])
def test_input_gradient_in_parts(parts, dtype, P, M, K, N):
    """dX = sum_i dOut_i W_i^T: the second operand transposed, the ranks summed."""
    X, W = _normal((M, K), seed=1), [_normal((K, N // P), 1.0 / N ** 0.5, 2 + i) for i in range(P)]
    dO, g = [_normal((M, N // P), 0.3, 20 + i) for i in range(P)], Guarded()
    dX = [g.empty((M, K), dtype, "dX")]
    _only(parts)
    rc, forms = _forms(lambda: rtp.lib().rtp_tp_linear_backward(
        0, P, M, K, N, _addresses([X]), _addresses(W), None, _addresses(dO), 0, None, rtp._dtype_code(dX[0]), _addresses(dX),
        rtp.BF16, None, None, rtp._stream_ptr(None)))
    assert rc == 0 and forms == {parts: 1}
    g.check("dX in parts")
    p64.check("dX in %d" % parts, dX[0], *p64.product(torch.cat(dO, 1), torch.cat(W, 1).T), p64.rel_of(dtype))


@pytest.mark.parametrize("parts", PARTS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("P,M,K,N", [(1, 2056, 264, 328), (3, 2049, 72, 3 * 40), (2, 4099, 520, 2 * 8)])
def test_weight_gradient_in_parts(parts, dtype, P, M, K, N):
    """dW_i = X^T dOut_i: the first operand transposed, and a K range (the rows) that ends anywhere."""
    X, W = _normal((M, K), seed=3), [_normal((K, N // P), 1.0, 4 + i) for i in range(P)]
    dO, g = [_normal((M, N // P), 0.3, 20 + i) for i in range(P)], Guarded()
    dW = g.many([(K, N // P)] * P, dtype, "dW")
    _only(parts)
    rc, forms = _forms(lambda: rtp.lib().rtp_tp_linear_backward(
        0, P, M, K, N, _addresses([X]), _addresses(W), None, _addresses(dO), 0, None, rtp.BF16, None, rtp._dtype_code(dW[0]),
        _addresses(dW), None, rtp._stream_ptr(None)))
    assert rc == 0 and forms == {parts: 1}
    g.check("dW in parts")
    for i in range(P):
        p64.check("dW in %d" % parts, dW[i], *p64.product(X.T, dO[i]), p64.rel_of(dtype))


def test_special_values_stay_in_their_rows_in_parts():
    """Infinities and NaN in one row reach that row alone, whichever part's K range holds them."""
    for k in (0, 700, 1500, 2055):
        X, W, R = _normal((300, 2056), seed=1), [_normal((2056, 264), 0.02, 2)], [_normal((300, 264), seed=3)]
        clean = rtp.tp_linear(X, W, act="silu", residual=R)[0]
        X[3, k], X[290, k] = float("nan"), float("inf")
        got, forms = _forms(lambda: rtp.tp_linear(X, W, act="silu", residual=R)[0])
        rows = torch.ones(300, dtype=torch.bool, device="cuda")
        rows[[3, 290]] = False
        assert forms == {4: 1} and torch.equal(got[rows], clean[rows])
        assert bool(got[3].isnan().all()) and not bool(got[290].isfinite().all())
