"""GPU parity of the tensor-parallel linear layer (bias, activation and residual in the product's epilogue) and of its
backward pass against float64, with every output in a guarded buffer. Bounds: plain64.py."""
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


def _case(split, P, M, K, N, bias, residual, seed):
    row = split == "row"
    Kp, Np, outs = (K // P, N, 1) if row else (K, N // P, P)
    X = [_normal((M, Kp), seed=seed + i) for i in range(P if row else 1)]
    W = [_normal((Kp, Np), 1.5 / K ** 0.5, seed=seed + 20 + i) for i in range(P)]
    b = [_normal((Np,), 0.5, seed=seed + 40 + i) for i in range(outs)] if bias else None
    R = [_normal((M, Np), seed=seed + 60 + i) for i in range(outs)] if residual else None
    return X, W, b, R, outs, Np


def _pre(split, X, W, b):
    """Float64 pre-activations and their float32 accumulation bounds, per output buffer."""
    if split == "row":
        h, e = p64.product(torch.cat(X, 1), torch.cat(W, 0))
        hs = [(h, e)]
    else:
        hs = [p64.product(X[0], w) for w in W]
    out = []
    for i, (h, e) in enumerate(hs):
        if b is not None:
            h = h + b[i].double()
            e = e + 2.0 ** -23 * (h.abs() + e)
        out.append((h, e))
    return out


def _run_and_check(split, P, M, K, N, act, bias, residual, out_dtype=BF16, keep_h=False, seed=0):
    X, W, b, R, outs, Np = _case(split, P, M, K, N, bias, residual, seed)
    g = Guarded()
    out = g.many([(M, Np)] * outs, out_dtype, "out")
    H = g.many([(M, Np)] * outs, BF16, "H") if keep_h else None
    rtp.tp_linear(X if split == "row" else X[0], W, split=split, bias=b, act=act, residual=R, H=H, out=out)
    what = "%s P=%d M=%d K=%d N=%d %s" % (split, P, M, K, N, act)
    g.check(what)
    for i, (h, e) in enumerate(_pre(split, X, W, b)):
        if keep_h:
            p64.check(what + " H", H[i], h, e, p64.BF16_REL)
        a = p64.act(act, h)
        err = p64.LIP * e + p64.act_eval_bound(a, h) if act != "none" else e
        if residual:
            a = a + R[i].double()
            err = err + 2.0 ** -23 * (a.abs() + err)
        p64.check(what, out[i], a, err, p64.rel_of(out_dtype))


@pytest.mark.parametrize("split", ["column", "row"])
@pytest.mark.parametrize("M", [1, 2, 5, 16, 17, 33, 100, 128, 129, 200, 256, 257, 300, 777])
def test_rows_from_one_to_many(split, M):
    _run_and_check(split, 2, M, 336, 272, "silu", True, True, seed=M)


@pytest.mark.parametrize("split,P,M,K,N", [
    ("column", 1, 3, 8, 8), ("row", 1, 3, 8, 8), ("column", 8, 1, 64, 64), ("row", 8, 1, 64, 8),
    ("column", 3, 19, 72, 24 * 11), ("row", 3, 19, 24 * 11, 72), ("row", 8, 7, 8 * 1000, 136),
    ("column", 4, 9, 2056, 4 * 520), ("row", 1, 4, 4096, 128), ("column", 1, 260, 8, 8), ("row", 8, 513, 64, 8),
    ("column", 3, 300, 136, 3 * 264), ("row", 5, 513, 5 * 72, 520), ("column", 8, 1030, 200, 8 * 40),
    ("row", 1, 256, 16384, 264)])
def test_ragged_sizes(split, P, M, K, N):
    _run_and_check(split, P, M, K, N, "none", True, True, seed=K)


@pytest.mark.parametrize("split,P,K,N", [("column", 5, 2048, 5 * 1048), ("column", 1, 2056, 6392), ("row", 2, 2 * 1032, 6152)])
@pytest.mark.parametrize("over", [1, 17, 64, 65])
@pytest.mark.parametrize("out_dtype", [BF16, F32])
def test_rows_left_over_by_the_last_whole_tile(split, P, K, N, over, out_dtype):
    """25 column tiles and a little over 768 rows: up to 64 rows over go to the few-row kernel."""
    _run_and_check(split, P, 768 + over, K, N, "gelu", True, True, out_dtype, keep_h=split == "column", seed=over)


def test_rows_left_over_read_weights_written_just_before():
    X, W, b, R, outs, Np = _case("column", 1, 777, 2048, 6400, True, True, 5)
    want = rtp.tp_linear(X[0], W, bias=b, residual=R)[0].clone()
    late = torch.zeros_like(W[0])
    for _ in range(20):
        late.zero_()
        late.copy_(W[0])
        got = rtp.tp_linear(X[0], [late], bias=b, residual=R)[0]
        assert torch.equal(got, want)


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "silu", "relu"])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("M", [21, 290])
def test_epilogues(act, bias, residual, M):
    for dtype in (BF16, F32):
        for keep_h in (False, True):
            _run_and_check("column", 2, M, 136, 400, act, bias, residual, dtype, keep_h, seed=7)
    _run_and_check("row", 2, M, 272, 200, act, bias, residual, F32, True, seed=8)


def test_full_size_and_run_to_run_bits():
    """The MLP configuration's row-parallel projection, sampled rows; a second run gives the same bits."""
    P, M, K, N = 8, 8192, 16384, 4096
    X, W, b, R, _, _ = _case("row", P, M, K, N, True, True, 3)
    out = rtp.tp_linear(X, W, split="row", bias=b, residual=R)[0]
    rows = [0, 1, 127, 128, 255, 256, 4095, 8191]
    (h, e), = _pre("row", [x[rows] for x in X], W, b)
    a = h + R[0][rows].double()
    p64.check("full size", out[rows], a, e + 2.0 ** -23 * (a.abs() + e), p64.BF16_REL)
    assert torch.equal(out, rtp.tp_linear(X, W, split="row", bias=b, residual=R)[0])
    few = [x[:5].contiguous() for x in X]
    first = rtp.tp_linear(few, W, split="row")[0]
    for _ in range(20):
        assert torch.equal(first, rtp.tp_linear(few, W, split="row")[0])


def test_refusals_on_the_gpu():
    """Calls that a decoding loop makes refuse wrong buffers with the message of the checked path."""
    X, W, b, R, _, _ = _case("row", 2, 5, 64, 72, True, True, 2)
    good = rtp.tp_linear(X, W, split="row", bias=b, residual=R)
    for kw, status in ((dict(bias=[b[0][:64]]), -2), (dict(bias=[b[0].float()]), -2), (dict(residual=[R[0].t()]), -2),
                       (dict(residual=[R[0].cpu()]), -1), (dict(act="swish"), -1), (dict(split="rows"), -1),
                       (dict(bias=b * 2), -1)):
        with pytest.raises(rtp.RtpError) as e:
            rtp.tp_linear(X, W, **{**dict(split="row", bias=b, residual=R), **kw})
        assert e.value.status == status, kw
    for X2, W2, status in ((X[:1], W, -1), ([x[:, :8].contiguous() for x in X], W, -2), (X, [w.float() for w in W], -2),
                           ([X[0], X[1].t().contiguous().t()], W, -1), ([x.cpu() for x in X], W, -1)):
        with pytest.raises(rtp.RtpError) as e:
            rtp.tp_linear(X2, W2, split="row")
        assert e.value.status == status
    with pytest.raises(rtp.RtpError) as e:  # refused by the library itself
        rtp.tp_linear([x[:, :12].contiguous() for x in X], [w[:12].contiguous() for w in W], split="row")
    assert e.value.status == -2 and "multiples of 8" in str(e.value)
    with pytest.raises(rtp.RtpError):
        rtp.tp_glu(X[0], [W[0]] * 2, [W[0]], [W[0]] * 2)
    assert torch.equal(rtp.tp_linear(X, W, split="row", bias=b[0], residual=R[0])[0], good[0])
    assert torch.equal(rtp.tp_linear(tuple(X), tuple(W), split="row", bias=b, residual=R)[0], good[0])


def test_outputs_past_two_to_the_31_elements():
    """Row offsets past 2^31 elements: the last rows of a 262,147 x 8,200 output, and of its gradient's input."""
    M, K, N = 262147, 64, 8200
    X, W = _normal((M, K), seed=1), [_normal((K, N), 0.2, seed=2)]
    b, R = [_normal((N,), 0.5, seed=3)], [torch.zeros((M, N), dtype=BF16, device="cuda")]
    R[0][-5:] = 1.5
    out = rtp.tp_linear(X, W, bias=b, residual=R, act="relu")[0]
    rows = [0, 1, 261888, M - 257, M - 6, M - 5, M - 1]
    (h, e), = _pre("column", [X[rows]], W, b)
    a = p64.act("relu", h) + R[0][rows].double()
    p64.check("long output", out[rows], a, e + p64.act_eval_bound(a, h) + 2.0 ** -23 * a.abs(), p64.BF16_REL)
    _, dW, db = rtp.tp_linear_backward(X, W, [out], H=[out], act="relu")
    d = (out.float() * (out > 0)).to(BF16)
    cols = [0, 63, 64, 8199]
    ref, e = p64.product(X.T, d[:, cols])
    p64.check("long dW", dW[0][:, cols], ref, e, p64.BF16_REL)
    p64.check("long db", db[0][cols], d[:, cols].double().sum(0), p64.acc_bound(M, d[:, cols].double().abs().sum(0)),
              2.0 ** -23)


def test_two_threads_on_their_own_streams():
    """Concurrent calls keep their launch arguments and results apart."""
    import threading

    cases = [_case("row", 4, m, 512, 264, True, True, 100 + m) for m in (3, 300)]
    want = [rtp.tp_linear(X, W, split="row", bias=b, residual=R)[0] for X, W, b, R, _, _ in cases]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        X, W, b, R, _, _ = cases[i]
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(200):
                if not torch.equal(rtp.tp_linear(X, W, split="row", bias=b, residual=R)[0], want[i]):
                    bad.append(i)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_no_rows():
    W = [torch.ones((16, 8), dtype=BF16, device="cuda")] * 2
    out = rtp.tp_linear(torch.empty((0, 16), dtype=BF16, device="cuda"), W, act="silu", keep_h=True)
    assert [tuple(t.shape) for ts in out for t in ts] == [(0, 8)] * 4
    dX, dW, db = rtp.tp_linear_backward(torch.empty((0, 16), dtype=BF16, device="cuda"), W,
                                        [torch.empty((0, 8), dtype=BF16, device="cuda")] * 2)
    assert dX[0].shape == (0, 16) and all(not bool(t.any()) for t in dW + db)


def test_special_values_stay_in_their_rows():
    """Infinities and NaN in one row of X, or of the residual, reach that row alone (both kernels)."""
    for M in (40, 300):
        X, W, _, R, _, _ = _case("column", 1, M, 136, 264, False, True, 5)
        clean = rtp.tp_linear(X[0], W, act="silu", residual=R)[0]
        X[0][3, 7], X[0][11, 0], R[0][20, 5] = float("nan"), float("inf"), float("-inf")
        got = rtp.tp_linear(X[0], W, act="silu", residual=R)[0]
        rows = torch.ones(M, dtype=torch.bool, device="cuda")
        rows[[3, 11, 20]] = False
        assert torch.equal(got[rows], clean[rows])
        assert bool(got[3].isnan().all()) and not bool(got[11].isfinite().all())
        assert float(got[20, 5]) == float("-inf")
        keep = torch.arange(264, device="cuda") != 5
        assert torch.equal(got[20][keep], clean[20][keep])


def test_another_stream_and_graph():
    """A call on a stream of its own, and captured in a graph and replayed with new inputs, gives the same bits."""
    for M in (6, 300):
        X, W, b, R, _, _ = _case("row", 4, M, 512, 264, True, True, 9)
        want = rtp.tp_linear(X, W, split="row", bias=b, act="gelu", residual=R)[0]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = rtp.tp_linear(X, W, split="row", bias=b, act="gelu", residual=R, stream=side)[0]
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)
        out = [torch.empty_like(want)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rtp.tp_linear(X, W, split="row", bias=b, act="gelu", residual=R, out=out)
        for x in X:
            x.mul_(2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], rtp.tp_linear(X, W, split="row", bias=b, act="gelu", residual=R)[0])
        assert not torch.equal(out[0], want)


# ---- backward ----------------------------------------------------------------------------------------------------


def _backward_check(split, P, M, K, N, act, dx_dtype=BF16, dw_dtype=BF16, seed=0):
    row = split == "row"
    X, W, _, _, outs, Np = _case(split, P, M, K, N, False, False, seed)
    Kp, ins = W[0].shape[0], len(X)
    H = [_normal((M, Np), 1.5, seed + 80 + i) for i in range(outs)] if act != "none" else None
    dO = [_normal((M, Np), 0.3, seed + 90 + i) for i in range(outs)]
    g = Guarded()
    dH = g.many([(M, Np)] * outs, BF16, "dH") if act != "none" else None
    dX = g.many([(M, Kp)] * ins, dx_dtype, "dX")
    dW = g.many([(Kp, Np)] * P, dw_dtype, "dW")
    db = g.many([(Np,)] * outs, F32, "db")
    rtp.tp_linear_backward(X if row else X[0], W, dO, split=split, H=H, act=act, dH=dH, dX=dX, dW=dW, db=db)
    what = "backward %s P=%d M=%d K=%d N=%d %s" % (split, P, M, K, N, act)
    g.check(what)
    d = []
    for i in range(outs):
        ref = dO[i].double()
        err = torch.zeros_like(ref)
        if act != "none":
            slope = p64.act_grad(act, H[i].double())
            ref = ref * slope
            err = 2.0 ** -17 * dO[i].double().abs()  # the slope, at most 1.13, evaluated to 2^-18 of max(slope, 1/2)
            p64.check(what + " dH", dH[i], ref, err, p64.BF16_REL)
        p64.check(what + " db", db[i], ref.sum(0), err.sum(0) + p64.acc_bound(M, ref.abs().sum(0)), 2.0 ** -23)
        d.append(dH[i] if act != "none" else dO[i])
    # the products, of the dH that the kernel rounded
    if row:
        for i in range(P):
            p64.check(what + " dX", dX[i], *p64.product(d[0], W[i].T), p64.rel_of(dx_dtype))
    else:
        p64.check(what + " dX", dX[0], *p64.product(torch.cat(d, 1), torch.cat(W, 1).T), p64.rel_of(dx_dtype))
    for i in range(P):
        p64.check(what + " dW", dW[i], *p64.product(X[i if row else 0].T, d[0 if row else i]), p64.rel_of(dw_dtype))


@pytest.mark.parametrize("split,P,M,K,N", [
    ("column", 1, 1, 8, 8), ("row", 2, 1, 16, 8), ("column", 2, 5, 72, 144), ("row", 2, 33, 144, 72),
    ("column", 3, 257, 136, 3 * 88), ("row", 3, 300, 3 * 88, 136), ("column", 8, 520, 264, 8 * 72),
    ("row", 8, 129, 8 * 72, 264)])
@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_backward(split, P, M, K, N, act):
    _backward_check(split, P, M, K, N, act, seed=M)


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "silu", "relu"])
@pytest.mark.parametrize("dx,dw", [(F32, F32), (BF16, F32), (F32, BF16)])
def test_backward_types(act, dx, dw):
    _backward_check("column", 2, 290, 136, 272, act, dx, dw, seed=1)


def test_gradients_against_differences():
    """Directional derivatives of sum(dOut * forward) by central differences of the float32 forward. A step
    along the gradient's signs moves a pre-activation by at most about 0.1 (K steps of 2^-4 / sqrt(K) times weights of
    about 1 / sqrt(K), or of 2^-4 / K times inputs of about 1, or one of 2^-4), so the truncation error is about
    0.1^2 / 6 of the third derivative's size, below 1e-2 of the derivative; dH's rounding to bf16 adds at most 2^-8."""
    P, M, K, N, act = 2, 64, 128, 256, "silu"
    X, W, b, _, outs, Np = _case("column", P, M, K, N, True, False, 30)
    dO = [_normal((M, Np), 1.0, 95 + i) for i in range(P)]
    _, H = rtp.tp_linear(X[0], W, bias=b, act=act, keep_h=True)
    dX, dW, db = rtp.tp_linear_backward(X[0], W, dO, H=H, act=act, dx_dtype=F32, dw_dtype=F32)

    def loss(Xs, Ws, bs):
        out = rtp.tp_linear(Xs, Ws, bias=bs, act=act, out_dtype=F32)
        return sum(float((o.double() * d.double()).sum()) for o, d in zip(out, dO))

    # directions along the gradients themselves: large derivatives, exact bf16 steps
    for which in ("X", "W", "b"):
        grads = {"X": dX, "W": dW, "b": db}[which]
        base = {"X": X, "W": W, "b": b}[which]
        size = {"X": 2.0 ** -4 / K ** 0.5, "W": 2.0 ** -4 / K, "b": 2.0 ** -4}[which]
        plus = [(t.float() + size * g.sign()).to(BF16) for t, g in zip(base, grads)]
        minus = [(t.float() - size * g.sign()).to(BF16) for t, g in zip(base, grads)]
        along = sum(float(((p.double() - m.double()) * g.double()).sum()) for p, m, g in zip(plus, minus, grads))
        args = {"X": X, "W": W, "b": b}
        hi, lo = dict(args, **{which: plus}), dict(args, **{which: minus})
        diff = loss(hi["X"][0], hi["W"], hi["b"]) - loss(lo["X"][0], lo["W"], lo["b"])
        assert abs(diff - along) <= 2e-2 * abs(along), (which, diff, along)
