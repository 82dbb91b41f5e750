"""What the linear layer, the gated block and the gradient norm refuse on the host, before anything is launched, through
the C ABI with fake device pointers that are never touched. No GPU needed."""
import ctypes

import pytest
import torch

import resharding_tensor_parallelism_gb300 as rtp
from resharding_tensor_parallelism_gb300 import _build

EINVAL, ESHAPE, EUNSUPPORTED = -1, -2, -3


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def _p(n, base=0x100000):
    return rtp._ptrs([base + 0x1000 * i for i in range(n)])


def _linear(split=0, P=2, M=4, K=16, N=32, X=0, W=0, bias=None, residual=None, act=3, dtype=1, H=None, out=0):
    X, W, out = (_p(8, 0x100000 * (i + 1)) if v == 0 else v for i, v in enumerate((X, W, out)))
    return rtp.lib().rtp_tp_linear(split, P, M, K, N, X, W, bias, residual, act, dtype, H, out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(split=2), EINVAL), (dict(P=0), EUNSUPPORTED), (dict(P=9), EUNSUPPORTED), (dict(act=5), EINVAL),
    (dict(act=-1), EINVAL), (dict(dtype=2), EINVAL), (dict(M=-1), ESHAPE), (dict(M=1 << 31), ESHAPE), (dict(K=0), ESHAPE),
    (dict(N=33), ESHAPE), (dict(N=24), ESHAPE), (dict(K=12), ESHAPE), (dict(split=1, K=17), ESHAPE),
    (dict(split=1, K=24), ESHAPE), (dict(split=1, N=12), ESHAPE), (dict(X=None), EINVAL), (dict(W=None), EINVAL),
    (dict(out=None), EINVAL), (dict(W=rtp._ptrs([4096, 0])), EINVAL), (dict(W=rtp._ptrs([4096, 8200])), EINVAL),
    (dict(X=rtp._ptrs([4098])), EINVAL), (dict(out=rtp._ptrs([4096, 0])), EINVAL),
    (dict(bias=rtp._ptrs([4096, 0])), EINVAL), (dict(bias=rtp._ptrs([4096, 4100])), EINVAL),
    (dict(residual=rtp._ptrs([0, 4096])), EINVAL), (dict(H=rtp._ptrs([4096, 8194])), EINVAL)])
def test_linear(kw, status):
    assert _linear(**kw) == status and "rtp_tp_linear" in rtp.last_error()


def test_linear_without_rows():
    assert _linear(M=0, X=None, out=None) == 0


def _linear_backward(split=0, P=2, M=4, K=16, N=32, H=0, dOut=0, act=3, dH=0, dx=1, dX=0, dw=1, dW=0, db=0):
    H, dOut, dH, dX, dW, db = (_p(8, 0x100000 * (i + 5)) if v == 0 else v for i, v in enumerate((H, dOut, dH, dX, dW, db)))
    return rtp.lib().rtp_tp_linear_backward(split, P, M, K, N, _p(8), _p(8, 0x200000), H, dOut, act, dH, dx, dX, dw, dW, db,
                                            None)


@pytest.mark.parametrize("kw,status", [
    (dict(split=-1), EINVAL), (dict(P=9), EUNSUPPORTED), (dict(act=9), EINVAL), (dict(dx=7), EINVAL), (dict(dw=-1), EINVAL),
    (dict(N=40), ESHAPE), (dict(H=None), EINVAL), (dict(dH=None), EINVAL), (dict(dOut=None), EINVAL),
    (dict(dX=rtp._ptrs([0])), EINVAL), (dict(dW=rtp._ptrs([4096, 0])), EINVAL), (dict(db=rtp._ptrs([4096, 4098])), EINVAL)])
def test_linear_backward(kw, status):
    assert _linear_backward(**kw) == status and "rtp_tp_linear_backward" in rtp.last_error()


def _glu(P=2, M=4, K=16, F=32, N=24, X=4096, Ag=0, Au=0, B=0, R=None, act=3, Y=0, dtype=1, Z=8192, train=False, Hg=0, Hu=0):
    Ag, Au, B, Y, Hg, Hu = (_p(8, 0x100000 * (i + 1)) if v == 0 else v for i, v in enumerate((Ag, Au, B, Y, Hg, Hu)))
    if train:
        return rtp.lib().rtp_tp_glu_train_forward(P, M, K, F, N, X, Ag, Au, B, R, act, Y, Hg, Hu, dtype, Z, None)
    return rtp.lib().rtp_tp_glu(P, M, K, F, N, X, Ag, Au, B, R, act, Y, dtype, Z, None)


@pytest.mark.parametrize("kw,status", [
    (dict(P=0), EUNSUPPORTED), (dict(P=9), EUNSUPPORTED), (dict(F=33), ESHAPE), (dict(F=24), ESHAPE), (dict(F=0), ESHAPE),
    (dict(K=20), ESHAPE), (dict(N=20), ESHAPE), (dict(M=-2), ESHAPE), (dict(act=17), EINVAL), (dict(dtype=5), EINVAL),
    (dict(X=None), EINVAL), (dict(Z=None), EINVAL), (dict(Z=8194), EINVAL), (dict(R=4100), EINVAL), (dict(Ag=None), EINVAL),
    (dict(Au=rtp._ptrs([0, 4096])), EINVAL), (dict(B=rtp._ptrs([4096, 4104])), EINVAL), (dict(Y=None), EINVAL),
    (dict(train=True, Hg=None), EINVAL), (dict(train=True, Hu=rtp._ptrs([4096, 0])), EINVAL)])
def test_glu(kw, status):
    assert _glu(**kw) == status and "rtp_tp_glu" in rtp.last_error()


def test_glu_without_rows():
    assert _glu(M=0, X=None, Y=None, Z=None) == 0
    assert _glu(M=0, X=None, Y=None, Z=None, train=True, Hg=None, Hu=None) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(P=9), EUNSUPPORTED), (dict(dx=3), EINVAL), (dict(dw=3), EINVAL), (dict(Hg=None), EINVAL), (dict(Y=None), EINVAL),
    (dict(dZ=None), EINVAL), (dict(dHu=None), EINVAL), (dict(dAu=None), EINVAL), (dict(dX=8194), EINVAL),
    (dict(dB=rtp._ptrs([4096, 0])), EINVAL), (dict(F=40), ESHAPE)])
def test_glu_backward(kw, status):
    a = dict(P=2, F=32, Hg=_p(8), Hu=_p(8), Y=_p(8), dZ=4096, dHg=_p(8), dHu=_p(8), dx=1, dX=8192, dw=1, dAg=_p(8), dAu=_p(8),
             dB=_p(8))
    a.update(kw)
    rc = rtp.lib().rtp_tp_glu_backward(a["P"], 4, 16, a["F"], 24, 4096, _p(8), _p(8), _p(8), a["Hg"], a["Hu"], a["Y"], a["dZ"],
                                       3, a["dHg"], a["dHu"], a["dx"], a["dX"], a["dw"], a["dAg"], a["dAu"], a["dB"], None)
    assert rc == status and "rtp_tp_glu_backward" in rtp.last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), EINVAL), (dict(dtypes=[0, 2]), EINVAL), (dict(numels=[4, -1]), ESHAPE), (dict(grads=[4096, 0]), EINVAL),
    (dict(grads=[4096, 8193]), EINVAL), (dict(ws=None), EINVAL), (dict(ws=4100), EINVAL), (dict(norm=None), EINVAL),
    (dict(max_norm=-1.0), EINVAL), (dict(max_norm=float("nan")), EINVAL), (dict(grads=[4096, 4100]), EINVAL),
    (dict(out=[16384, 16388]), EINVAL), (dict(out=[8192, 20480]), EINVAL), (dict(out=[16384, 0]), EINVAL)])
def test_clip(kw, status):
    a = dict(n=2, dtypes=[0, 1], numels=[4, 4], grads=[4096, 8192], ws=0x10000, norm=0x20000, max_norm=1.0, out=None)
    a.update(kw)
    rc = rtp.lib().rtp_clip_grad_norm(a["n"], rtp._i32(a["dtypes"]), rtp._i64(a["numels"]), rtp._ptrs(a["grads"]), None,
                                      a["max_norm"], rtp._ptrs(a["out"]) if a["out"] else None, a["ws"], a["norm"], None)
    assert rc == status and "rtp_clip_grad_norm" in rtp.last_error()


def test_workspace_size():
    sizes = [rtp.lib().rtp_grad_workspace_bytes(n) for n in (-1, 0, 1, 64, 65, 513, 100000)]
    assert sizes[0] == 0 and all(b >= a for a, b in zip(sizes[1:], sizes[2:])) and all(s % 8 == 0 for s in sizes)


def test_binding_checks_before_any_launch():
    """Wrong activations, splits, shapes and host tensors raise RtpError in Python."""
    b = torch.bfloat16
    X, W = torch.zeros((4, 16), dtype=b), [torch.zeros((16, 8), dtype=b)] * 2
    for call in (lambda: rtp.tp_linear(X, W, act="swish"), lambda: rtp.tp_linear(X, W, split="rows"),
                 lambda: rtp.tp_linear(X, []), lambda: rtp.tp_linear(X, W),
                 lambda: rtp.tp_linear(X[0], W), lambda: rtp.tp_glu(X, W, W[:1], W), lambda: rtp.tp_glu(X, W, W, W),
                 lambda: rtp.GradGroup([torch.zeros(4)])):
        with pytest.raises(rtp.RtpError):
            call()
