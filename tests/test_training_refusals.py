"""What the cross entropy and the AdamW step refuse on the host, before anything is launched, through the C ABI with fake
device pointers that are never touched. No GPU needed."""
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


COMMON = [
    (dict(P=0), EUNSUPPORTED), (dict(P=9), EUNSUPPORTED), (dict(M=-1), ESHAPE), (dict(M=1 << 31), ESHAPE), (dict(K=0), ESHAPE),
    (dict(K=12), ESHAPE), (dict(V=33), ESHAPE), (dict(V=24), ESHAPE), (dict(V=0), ESHAPE), (dict(vocab=0), ESHAPE),
    (dict(vocab=33), ESHAPE), (dict(M=1 << 24, V=1 << 30), ESHAPE),
    (dict(K=1 << 24, V=1 << 30), ESHAPE), (dict(X=None), EINVAL), (dict(X=4104), EINVAL), (dict(W=None), EINVAL),
    (dict(W=rtp._ptrs([4096, 0])), EINVAL), (dict(W=rtp._ptrs([4096, 8200])), EINVAL), (dict(wide=2), EINVAL),
    (dict(targets=None), EINVAL), (dict(targets=4100), EINVAL), (dict(targets=4098, wide=0), EINVAL), (dict(ws=None), EINVAL),
    (dict(ws=0x10010), EINVAL), (dict(bytes=16), EINVAL), (dict(loss=None), EINVAL), (dict(loss=4097), EINVAL)]


def _loss(P=2, M=4, K=16, V=32, vocab=30, X=4096, W=0, wide=1, targets=8192, ws=0x10000, bytes=1 << 30, loss=0x20000,
          lse=None):
    W = _p(8) if W == 0 else W
    return rtp.lib().rtp_tp_cross_entropy(P, M, K, V, vocab, X, W, wide, targets, -100, ws, bytes, loss, lse, None)


@pytest.mark.parametrize("kw,status", COMMON + [(dict(lse=4099), EINVAL)])
def test_cross_entropy(kw, status):
    assert _loss(**kw) == status and "rtp_tp_cross_entropy" in rtp.last_error()


def test_cross_entropy_without_rows():
    assert _loss(M=0, X=None, targets=None, loss=None) == 0


def _train(P=2, M=4, K=16, V=32, vocab=30, X=4096, W=0, wide=1, targets=8192, weights=None, mean=1, piece=0, ws=0x10000,
           bytes=1 << 30, total=0x30000, loss=0x20000, dx=1, dX=0x40000, dw=1, dW=0, accumulate=0):
    W, dW = (_p(8, 0x100000 * (i + 1)) if v == 0 else v for i, v in enumerate((W, dW)))
    return rtp.lib().rtp_tp_cross_entropy_train(P, M, K, V, vocab, X, W, wide, targets, -100, weights, mean, 1.0, piece, ws,
                                                bytes, total, loss, dx, dX, dw, dW, accumulate, None)


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(weights=4098), EINVAL), (dict(mean=2), EINVAL), (dict(piece=-1), EINVAL), (dict(total=None), EINVAL),
    (dict(total=4098), EINVAL), (dict(dx=2), EINVAL), (dict(dw=7), EINVAL), (dict(dX=4104), EINVAL),
    (dict(dW=rtp._ptrs([4096, 0])), EINVAL), (dict(dW=rtp._ptrs([4096, 4104])), EINVAL), (dict(accumulate=1), EINVAL),
    (dict(accumulate=2, dw=0), EINVAL), (dict(accumulate=1, dw=0, dW=None), EINVAL)])
def test_cross_entropy_train(kw, status):
    assert _train(**kw) == status and "rtp_tp_cross_entropy_train" in rtp.last_error()


def test_workspace():
    n = ctypes.c_int64()
    size = lambda *a: (rtp.lib().rtp_tp_cross_entropy_workspace(*a, ctypes.byref(n)), n.value)[1]
    # statistics of 2 x 2 tiles and a logit for each of 300 rows
    assert size(2, 300, 64, 1024, 0, 0, 1) >= 300 * (4 * 8 + 4)
    # exponentials, and float32 sums of dW where a bf16 dW comes in pieces
    one, pieces, kept = size(2, 600, 64, 1024, 0, 1, 1), size(2, 600, 64, 1024, 256, 1, 1), size(2, 600, 64, 1024, 256, 1, 0)
    assert one >= 600 * 1024 * 2 and pieces - kept == 64 * 1024 * 4 and kept < one
    assert size(2, 0, 64, 1024, 0, 1, 1) > 0
    lib = rtp.lib()
    assert lib.rtp_tp_cross_entropy_workspace(2, 300, 64, 1000, 0, 0, 1, ctypes.byref(n)) == ESHAPE
    assert lib.rtp_tp_cross_entropy_workspace(2, 300, 64, 1024, 0, 0, 1, None) == EINVAL
    _train(bytes=0)
    need = int(rtp.last_error().split("bytes, ")[1].split()[0])
    assert need == size(2, 4, 16, 32, 0, 1, 1)


def _adamw(n=2, dtypes=(0, 1), grads=(0, 1), numel=(4, 4), param=(0x1000, 0x2000), grad=(0x3000, 0x4000), master=(None, 0x5000),
           m=(0x6000, 0x7000), v=(0x8000, 0x9000), scales=(0xA000, 0xB000), decay=0.1, bits=32, lr=0.1, lr_at=None, eps=1e-8,
           norm=None, max_norm=1.0, clock=0x10000, tensors=True):
    t = (rtp.AdamWTensor * 2)()
    for i in range(2):
        t[i].numel, t[i].param, t[i].grad, t[i].master = numel[i], param[i], grad[i], master[i]
        t[i].exp_avg, t[i].exp_avg_sq, t[i].scales = m[i], v[i], scales[i]
        t[i].param_dtype, t[i].grad_dtype, t[i].weight_decay = dtypes[i], grads[i], decay
    return rtp.lib().rtp_adamw_step(n, t if tensors else None, bits, lr, lr_at, eps, norm, max_norm, 0, clock, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), EINVAL), (dict(tensors=False), EINVAL), (dict(bits=16), EINVAL), (dict(clock=None), EINVAL),
    (dict(clock=0x10008), EINVAL), (dict(lr_at=0x10002), EINVAL), (dict(norm=0x10002), EINVAL), (dict(lr=-1.0), EINVAL),
    (dict(lr=float("nan")), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL),
    (dict(norm=0x20000, max_norm=-1.0), EINVAL), (dict(norm=0x20000, max_norm=float("nan")), EINVAL),
    (dict(dtypes=(0, 2)), EINVAL), (dict(grads=(3, 0)), EINVAL), (dict(numel=(4, -1)), ESHAPE), (dict(numel=(1 << 42, 4)), ESHAPE),
    (dict(decay=-0.1), EINVAL), (dict(decay=float("nan")), EINVAL), (dict(param=(0, 0x2000)), EINVAL),
    (dict(grad=(0x3000, 0)), EINVAL), (dict(m=(0, 0x7000)), EINVAL), (dict(v=(0x8000, 0)), EINVAL),
    (dict(bits=8, scales=(0, 0xB000)), EINVAL), (dict(bits=8, scales=(0xA001, 0xB000)), EINVAL),
    (dict(master=(0x5000, None)), EINVAL), (dict(param=(0x1002, 0x2000)), EINVAL), (dict(param=(0x1000, 0x2001)), EINVAL),
    (dict(grad=(0x3001, 0x4000)), EINVAL), (dict(m=(0x6002, 0x7000)), EINVAL), (dict(master=(None, 0x5002)), EINVAL),
    (dict(param=(0x1000, 0x1008)), EINVAL), (dict(master=(None, 0x1004)), EINVAL)])
def test_adamw(kw, status):
    assert _adamw(**kw) == status and "rtp_adamw_step" in rtp.last_error()


@pytest.mark.parametrize("args", [(None, 0, 0.9, 0.9), (0x1008, 0, 0.9, 0.9), (0x1000, -1, 0.9, 0.9), (0x1000, 0, 1.0, 0.9),
                                  (0x1000, 0, 0.9, -0.1), (0x1000, 0, float("nan"), 0.9)])
def test_clock(args):
    assert rtp.lib().rtp_adamw_clock(*args, None) == EINVAL and "rtp_adamw_clock" in rtp.last_error()


@pytest.mark.parametrize("kw,status", [(dict(blocks=-1), ESHAPE), (dict(dtype=2), EINVAL), (dict(m8=None), EINVAL),
                                       (dict(v8=0x2004), EINVAL), (dict(scales=0x3001), EINVAL), (dict(m=0x4008), EINVAL),
                                       (dict(v=None), EINVAL)])
def test_values(kw, status):
    a = dict(blocks=2, m8=0x1000, v8=0x2000, scales=0x3000, dtype=1, m=0x4000, v=0x5000)
    a.update(kw)
    rc = rtp.lib().rtp_adamw_values(a["blocks"], a["m8"], a["v8"], a["scales"], a["dtype"], a["m"], a["v"], None)
    assert rc == status and "rtp_adamw_values" in rtp.last_error()


def test_binding_checks_before_any_launch():
    b = torch.bfloat16
    X, W, t = torch.zeros((4, 16), dtype=b), [torch.zeros((16, 8), dtype=b)] * 2, torch.zeros(4, dtype=torch.int64)
    for call in (lambda: rtp.tp_cross_entropy(X, W, t), lambda: rtp.tp_cross_entropy(X, [], t),
                 lambda: rtp.tp_cross_entropy(X[0], W, t), lambda: rtp.tp_cross_entropy_train(X, W, t),
                 lambda: rtp.tp_cross_entropy_train(X, W, t, reduction="none"),
                 lambda: rtp.tp_cross_entropy_train(X, W, t, accumulate=True),
                 lambda: rtp.AdamWGroup([torch.zeros(4)])):
        with pytest.raises(rtp.RtpError):
            call()


@pytest.mark.parametrize("M", [1, 600, 70000])
def test_workspace_of_a_piece_of_more_rows_than_there_are(M):
    n = ctypes.c_int64()
    size = lambda piece, dw: (rtp.lib().rtp_tp_cross_entropy_workspace(2, M, 64, 1024, piece, 1, dw, ctypes.byref(n)), n.value)
    for dw in (0, 1):
        want = size(M, dw)
        assert want[0] == 0
        for piece in (M + 1, 1 << 31, (1 << 63) - 300, (1 << 63) - 1):
            assert size(piece, dw) == want, piece


def test_noise_below_zero():
    t = (rtp.AdamWTensor * 1)()
    t[0].numel, t[0].param, t[0].grad, t[0].exp_avg, t[0].exp_avg_sq = 4, 0x1000, 0x2000, 0x3000, 0x4000
    t[0].noise = -1
    assert rtp.lib().rtp_adamw_step(1, t, 32, 0.1, None, 1e-8, None, 1.0, 0, 0x10000, None) == EINVAL
    assert "noise" in rtp.last_error()
