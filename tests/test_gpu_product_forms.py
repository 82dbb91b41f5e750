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
