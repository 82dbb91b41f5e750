"""Vocabulary-split cross entropy and its gradients against float64."""
import pytest
import torch

import cross_entropy64 as plain
import resharding_tensor_parallelism_gb300 as rtp
from gpu_util import Guarded

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
IGNORE = -100
# M, K, V, P, vocab: one token and few (the few-row kernel, up to 128), the border to the pair kernel, row tiles of 256 and
# one more; vocabularies inside a tile, of odd widths, with padding inside a tile, over a whole rank, and of one word
SIZES = [(1, 8, 8, 1, 8), (1, 520, 4096, 2, 4096), (3, 64, 264, 3, 264), (37, 512, 2048, 8, 2041), (127, 136, 1000, 1, 1000),
         (128, 72, 1048, 1, 1), (129, 72, 1048, 1, 1), (129, 264, 528, 2, 300), (255, 8, 24, 3, 24), (256, 128, 512, 2, 512),
         (257, 200, 2064, 2, 2063), (300, 64, 768, 3, 250), (777, 328, 1256, 1, 1255), (512, 1024, 1024, 4, 1024)]


def _inputs(M, K, V, P, vocab, seed=0, ignored=0.2, dtype=torch.int64, spread=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    X = (torch.randn((M, K), generator=gen, device="cuda") * spread).to(BF16)
    W = (torch.randn((K, V), generator=gen, device="cuda") / K ** 0.5).to(BF16)
    t = torch.randint(0, vocab, (M,), generator=gen, device="cuda")
    t[torch.rand((M,), generator=gen, device="cuda") < ignored] = IGNORE
    t[-1] = vocab - 1
    return X, W, [w.contiguous() for w in W.chunk(P, 1)], t.to(dtype)


def _near(got, want, bound, what):
    got, want = got.double(), want.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    bad = (got - want).abs() > bound
    assert not bad.any(), "%s: %d outside the bound, worst %.3g of it" % (
        what, int(bad.sum()), float(((got - want).abs() / bound).nan_to_num(0).max()))


def _check_forward(X, W, t, vocab, loss, lse):
    want, want_lse, logits, _ = plain.forward(X, W, t, vocab, IGNORE)
    bound = plain.lse_bound(X, W, vocab, want_lse, logits)
    _near(lse, want_lse, bound, "lse")
    _near(loss, want, bound + plain.logit_error(X, W, vocab) + 2 * plain.EPS * want_lse.abs(), "loss")


@pytest.mark.parametrize("dtype", [torch.int64, torch.int32])
@pytest.mark.parametrize("M,K,V,P,vocab", SIZES)
def test_forward(M, K, V, P, vocab, dtype):
    X, W, shards, t = _inputs(M, K, V, P, vocab, dtype=dtype)
    out = Guarded()
    loss, lse = out.empty((M,), F32, "loss"), out.empty((M,), F32, "lse")
    got = rtp.tp_cross_entropy(X, shards, t, vocab=vocab, ignore_index=IGNORE, loss=loss, lse=lse)
    assert got[0] is loss and got[1] is lse
    out.check("forward")
    _check_forward(X, W, t, vocab, loss, lse)
    assert rtp.device_error() == 0


def _check_train(X, W, t, vocab, got, weights=None, mean=True, scale=1.0, before=None):
    total, loss, dX, dW = got
    want_total, want, want_x, want_w, bx, bw = plain.gradients(X, W, t, vocab, IGNORE, weights, mean, scale)
    _, lse, logits, _ = plain.forward(X, W, t, vocab, IGNORE)
    bound = plain.lse_bound(X, W, vocab, lse, logits) + plain.logit_error(X, W, vocab) + 2 * plain.EPS * lse.abs()
    _near(loss, want, bound, "loss")
    w = torch.ones_like(want) if weights is None else weights.double()
    w = w * (t != IGNORE)
    most = (w.abs() * bound).sum() / (w.sum().abs() if mean and w.sum() != 0 else 1.0)
    _near(total, want_total, most + 2 * plain.EPS * want_total.abs(), "total")
    half = {BF16: plain.BF16, F32: 2 * plain.EPS}
    tiny = 1e-37  # subnormals count as zero in places
    _near(dX, want_x, bx * 1.01 + half[dX.dtype] * want_x.abs() + tiny, "dX")
    dW = torch.cat(dW, 1)
    if before is not None:
        want_w = want_w + before.double()
        bw = bw + 8 * plain.EPS * (before.double().abs() + want_w.abs())
    _near(dW, want_w, bw * 1.01 + half[dW.dtype] * want_w.abs() + tiny, "dW")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,K,V,P,vocab", SIZES)
def test_train(M, K, V, P, vocab, dtype):
    X, W, shards, t = _inputs(M, K, V, P, vocab, seed=1)
    out = Guarded()
    dX, dW = out.empty((M, K), dtype, "dX"), out.many([(K, V // P)] * P, dtype, "dW")
    loss = out.empty((M,), F32, "loss")
    got = rtp.tp_cross_entropy_train(X, shards, t, vocab=vocab, ignore_index=IGNORE, dX=dX, dW=dW, loss=loss)
    out.check("train")
    _check_train(X, W, t, vocab, got)
    assert rtp.device_error() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,K,V,P", [(256, 512, 8192, 2), (5, 64, 16384, 1), (300, 264, 24600, 3), (130, 520, 12352, 1),
                                     (257, 72, 8 * 1032, 8), (600, 136, 16392, 1)])
def test_narrow_models(M, K, V, P, dtype):
    """Few tiles of dX, whose columns are summed in slices: even and ragged ones, on one to eight ranks."""
    X, W, shards, t = _inputs(M, K, V, P, V - 3, seed=14)
    out = Guarded()
    dX, dW = out.empty((M, K), dtype, "dX"), out.many([(K, V // P)] * P, dtype, "dW")
    got = rtp.tp_cross_entropy_train(X, shards, t, vocab=V - 3, ignore_index=IGNORE, dX=dX, dW=dW)
    out.check("train")
    _check_train(X, W, t, V - 3, got)
    _check_train(X, W, t, V - 3, rtp.tp_cross_entropy_train(X, shards, t, vocab=V - 3, ignore_index=IGNORE, dx_dtype=dtype,
                                                            dw_dtype=dtype, piece_rows=256))


@pytest.mark.parametrize("reduction", ["mean", "sum"])
@pytest.mark.parametrize("M,K,V,P,vocab", [(5, 64, 264, 3, 260), (333, 128, 1040, 2, 1040)])
def test_weights_and_scale(M, K, V, P, vocab, reduction):
    X, W, shards, t = _inputs(M, K, V, P, vocab, seed=2)
    w = torch.rand((M,), device="cuda") * 2
    w[::3] = 0.0
    w[1] = -0.5
    got = rtp.tp_cross_entropy_train(X, shards, t, weights=w, vocab=vocab, ignore_index=IGNORE, reduction=reduction,
                                     scale=128.0)
    _check_train(X, W, t, vocab, got, w, reduction == "mean", 128.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,piece,P", [(600, 256, 2), (600, 300, 3), (700, 256, 1), (1025, 512, 2)])
def test_pieces_of_rows(M, piece, P, dtype):
    """The last piece of 600 rows has 88 of them (few rows), of 700 188, of 1025 one."""
    X, W, shards, t = _inputs(M, 136, 264 * P, P, 264 * P - 3, seed=3)
    w = torch.rand((M,), device="cuda")
    got = rtp.tp_cross_entropy_train(X, shards, t, weights=w, vocab=264 * P - 3, ignore_index=IGNORE, piece_rows=piece,
                                     dw_dtype=dtype)
    _check_train(X, W, t, 264 * P - 3, got, w)


def test_pieces_by_default():
    """2048 rows a piece for a narrow model with a vocabulary of which they take 1 GiB."""
    X, W, shards, t = _inputs(2304, 64, 262144, 2, 262144, seed=4)
    _check_train(X, W, t, 262144, rtp.tp_cross_entropy_train(X, shards, t, ignore_index=IGNORE))


@pytest.mark.parametrize("M,piece", [(100, 0), (300, 0), (600, 256)])
def test_accumulated_weight_gradients(M, piece):
    X, W, shards, t = _inputs(M, 136, 528, 2, 520, seed=5)
    dW = [torch.randn((136, 264), device="cuda") * 1e-3 for _ in range(2)]
    before = torch.cat(dW, 1)
    got = rtp.tp_cross_entropy_train(X, shards, t, vocab=520, ignore_index=IGNORE, dW=dW, accumulate=True, piece_rows=piece)
    assert got[3] is dW
    _check_train(X, W, t, 520, got, before=before)


@pytest.mark.parametrize("M", [4, 300])
def test_nothing_to_learn_from(M):
    X, W, shards, t = _inputs(M, 64, 512, 2, 512)
    t.fill_(IGNORE)
    X[1] = float("nan")
    total, loss, dX, dW = rtp.tp_cross_entropy_train(X, shards, t, ignore_index=IGNORE)
    assert float(total) == 0 and not loss.any() and not dX.any()
    assert not any(d.any() for d in dW)


@pytest.mark.parametrize("M", [4, 300])
def test_rows_without_a_part_hold_anything(M):
    """Infinities and NaN in rows that are ignored or of weight 0 leave the other rows alone."""
    X, W, shards, t = _inputs(M, 64, 512, 2, 512, ignored=0.0)
    t[0] = IGNORE
    w = torch.ones((M,), device="cuda")
    w[2] = 0.0
    want = rtp.tp_cross_entropy_train(X, shards, t, weights=w, ignore_index=IGNORE)
    Y = X.clone()
    Y[0], Y[2] = float("nan"), float("inf")
    total, loss, dX, dW = rtp.tp_cross_entropy_train(Y, shards, t, weights=w, ignore_index=IGNORE)
    assert torch.equal(total, want[0]) and not dX[0].any() and not dX[2].any() and float(loss[0]) == 0
    assert all(torch.equal(a, b) for a, b in zip(dW, want[3]))
    keep = [i for i in range(M) if i not in (0, 2)]
    assert torch.equal(loss[keep], want[1][keep]) and torch.equal(dX[keep], want[2][keep])


@pytest.mark.parametrize("M", [4, 300])
def test_targets_outside_the_vocabulary_show(M):
    X, W, shards, t = _inputs(M, 64, 512, 2, 500, ignored=0.0)
    for bad in (500, 511, 512, -1, 1 << 40):
        u = t.clone()
        u[1] = bad
        loss, lse = rtp.tp_cross_entropy(X, shards, u, vocab=500, ignore_index=IGNORE)
        assert torch.isnan(loss[1]) and not torch.isnan(lse).any() and int(torch.isnan(loss).sum()) == 1
        total, loss, dX, _ = rtp.tp_cross_entropy_train(X, shards, u, vocab=500, ignore_index=IGNORE)
        assert torch.isnan(total) and torch.isnan(dX[1]).all() and not torch.isnan(dX[[0, 2, 3]]).any()


@pytest.mark.parametrize("M", [3, 260])
@pytest.mark.parametrize("how", ["all", "some rows", "one rank", "all low", "one rank low"])
def test_far_logits(M, how):
    """Logits of some thousands: far beyond what an exponential holds, in tiles that differ by more than that; in some rows
    only, in one rank's tiles only, and far below zero, beside ordinary ones or not."""
    X, W, shards, t = _inputs(M, 64, 1024, 2, 1020, spread=1000.0 if how == "all" else 1.0, seed=7)
    if how == "some rows":
        X[::3] *= 300
    if how == "one rank":
        W[:, 600:] *= 200
    if how.endswith("low"):
        X[:, 0] = 16.0
        W[0, 512 if how.startswith("one") else 0:] = -20.0
    shards = [w.contiguous() for w in W.chunk(2, 1)]
    loss, lse = rtp.tp_cross_entropy(X, shards, t, vocab=1020, ignore_index=IGNORE)
    _check_forward(X, W, t, 1020, loss, lse)
    _check_train(X, W, t, 1020, rtp.tp_cross_entropy_train(X, shards, t, vocab=1020, ignore_index=IGNORE))


@pytest.mark.parametrize("M", [4, 300])
def test_infinite_and_nan_logits_stay_in_their_row(M):
    X, W, shards, t = _inputs(M, 64, 512, 2, 512, ignored=0.0)
    X[1] = float("nan")
    X[2, 0] = float("inf")
    loss, lse = rtp.tp_cross_entropy(X, shards, t, ignore_index=IGNORE)
    assert torch.isnan(loss[1]) and torch.isnan(lse[1]) and not torch.isfinite(loss[2])
    keep = [i for i in range(M) if i not in (1, 2)]
    _check_forward(X[keep], W, t[keep], 512, loss[keep], lse[keep])


@pytest.mark.parametrize("M", [7, 300])
def test_runs_are_alike_and_rows_do_not_meet(M):
    X, W, shards, t = _inputs(M, 200, 1040, 2, 1040, seed=8)
    a, b = (rtp.tp_cross_entropy_train(X, shards, t, ignore_index=IGNORE) for _ in range(2))
    assert all(torch.equal(x, y) for x, y in zip([*a[:3], *a[3]], [*b[:3], *b[3]]))
    half = rtp.tp_cross_entropy(X, shards, t, ignore_index=IGNORE)[0]
    assert torch.equal(rtp.tp_cross_entropy(X, shards, t, ignore_index=IGNORE)[0], half)


def test_without_rows():
    X, W, shards, t = _inputs(2, 64, 512, 2, 512)
    loss, lse = rtp.tp_cross_entropy(X[:0], shards, t[:0])
    assert loss.shape == (0,) and lse.shape == (0,)
    total, loss, dX, dW = rtp.tp_cross_entropy_train(X[:0], shards, t[:0])
    assert float(total) == 0 and dX.shape == (0, 64) and not any(d.any() for d in dW)
    kept = [torch.ones((64, 256), device="cuda") for _ in range(2)]
    rtp.tp_cross_entropy_train(X[:0], shards, t[:0], dW=kept, accumulate=True)
    assert all(bool((d == 1).all()) for d in kept)


def test_other_streams():
    X, W, shards, t = _inputs(300, 200, 1040, 2, 1040, seed=9)
    want = rtp.tp_cross_entropy_train(X, shards, t, ignore_index=IGNORE)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = rtp.tp_cross_entropy_train(X, shards, t, ignore_index=IGNORE, stream=s)
    alone = rtp.tp_cross_entropy(X, shards, t, ignore_index=IGNORE, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip([*got[:3], *got[3]], [*want[:3], *want[3]]))
    _check_forward(X, W, t, 1040, *alone)


@pytest.mark.parametrize("M", [5, 300])
def test_captured_calls_read_what_is_there_when_replayed(M):
    """Two graphs of one stream, replayed in turn with other inputs."""
    X, W, shards, t = _inputs(M, 136, 528, 2, 520, seed=10)
    rtp.tp_cross_entropy_train(X, shards, t, vocab=520, ignore_index=IGNORE)
    rtp.tp_cross_entropy(X, shards, t, vocab=520, ignore_index=IGNORE)
    torch.cuda.synchronize()
    graphs, got = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    with torch.cuda.graph(graphs[0]):
        got.append(rtp.tp_cross_entropy_train(X, shards, t, vocab=520, ignore_index=IGNORE))
    with torch.cuda.graph(graphs[1]):
        got.append(rtp.tp_cross_entropy(X, shards, t, vocab=520, ignore_index=IGNORE))
    for seed in (11, 12):
        Y, V, _, u = _inputs(M, 136, 528, 2, 520, seed=seed)
        X.copy_(Y)
        t.copy_(u)
        for s, v in zip(shards, V.chunk(2, 1)):
            s.copy_(v)
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        _check_train(Y, V, u, 520, got[0])
        _check_forward(Y, V, u, 520, *got[1])


def test_more_exponentials_than_31_bits_count():
    """17000 rows of 131072 columns in one piece (2.2 G exponentials on one rank): the last rows against float64."""
    M, K, V = 17000, 64, 131072
    X, W, shards, t = _inputs(M, K, V, 1, V, ignored=0.0, seed=13)
    t[-1] = IGNORE
    w = torch.zeros((M,), device="cuda")
    w[-4:] = torch.tensor([1.0, 2.0, 0.5, 1.0], device="cuda")
    got = rtp.tp_cross_entropy_train(X, shards, t, weights=w, ignore_index=IGNORE, piece_rows=M)
    total, loss, dX, dW = got
    assert not dX[:-4].any()
    _check_train(X[-4:], W, t[-4:], V, (total, loss[-4:], dX[-4:], dW), w[-4:])
    first = plain.forward(X[:4], W, t[:4], V, IGNORE)
    _near(loss[:4], first[0], plain.lse_bound(X[:4], W, V, first[1], first[2]) * 2, "first rows")


def _c_train(X, shards, t, V, dX, dW, dw_dtype=rtp.BF16, piece=0):
    """rtp_tp_cross_entropy_train through the C ABI, dX or dW may be None. Returns (total, loss)."""
    M, K = X.shape
    P = len(shards)
    ws, n = rtp._loss_workspace(P, M, K, V, piece, 1, dw_dtype, 0, None)
    total, loss = torch.full((), 7.0, device="cuda"), torch.full((M,), 7.0, device="cuda")
    rtp._check(rtp.lib().rtp_tp_cross_entropy_train(
        P, M, K, V, V, X.data_ptr(), rtp._ptrs([w.data_ptr() for w in shards]), 1, t.data_ptr(), IGNORE, None, 1, 1.0, piece,
        ws.data_ptr(), n, total.data_ptr(), loss.data_ptr(), rtp.BF16, None if dX is None else dX.data_ptr(), dw_dtype,
        None if dW is None else rtp._ptrs([d.data_ptr() for d in dW]), 0, rtp._stream_ptr(None)))
    return total, loss


@pytest.mark.parametrize("M,piece", [(5, 0), (300, 0), (600, 256)])
def test_gradients_that_are_not_wanted(M, piece):
    X, W, shards, t = _inputs(M, 136, 1040, 2, 1040, seed=15)
    want = rtp.tp_cross_entropy_train(X, shards, t, ignore_index=IGNORE, piece_rows=piece)
    dX, dW = torch.empty_like(X), [torch.empty_like(w) for w in shards]
    for x, w in ((dX, None), (None, dW), (None, None)):
        total, loss = _c_train(X, shards, t, 1040, x, w, piece=piece)
        assert torch.equal(total, want[0]) and torch.equal(loss, want[1])
    assert torch.equal(dX, want[2]) and all(torch.equal(a, b) for a, b in zip(dW, want[3]))
    alone = torch.empty((M,), device="cuda")
    ws, n = rtp._loss_workspace(2, M, 136, 1040, 0, 0, rtp.F32, 0, None)
    rtp._check(rtp.lib().rtp_tp_cross_entropy(2, M, 136, 1040, 1040, X.data_ptr(), rtp._ptrs([w.data_ptr() for w in shards]), 1,
                                              t.data_ptr(), IGNORE, ws.data_ptr(), n, alone.data_ptr(), None,
                                              rtp._stream_ptr(None)))
    assert torch.equal(alone, rtp.tp_cross_entropy(X, shards, t, ignore_index=IGNORE)[0])


def test_two_calls_at_once():
    """Calls on two streams beside each other, each with its own workspace, again and again."""
    sizes = [(300, 136, 4112, 2), (60, 520, 8208, 1)]
    sets = [_inputs(M, K, V, P, V, seed=16 + i) for i, (M, K, V, P) in enumerate(sizes)]
    want = [rtp.tp_cross_entropy_train(X, s, t, ignore_index=IGNORE) for X, _, s, t in sets]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(8):
        for s, (X, _, shards, t) in zip(streams, sets):
            with torch.cuda.stream(s):
                got.append(rtp.tp_cross_entropy_train(X, shards, t, ignore_index=IGNORE))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        w = want[i % 2]
        assert all(torch.equal(a, b) for a, b in zip([*g[:3], *g[3]], [*w[:3], *w[3]]))


def test_an_ignored_index_inside_the_vocabulary():
    X, W, shards, t = _inputs(300, 64, 512, 2, 512, ignored=0.0, seed=18)
    u = torch.where(t < 100, IGNORE, t)
    t[t < 100] = 7
    want = rtp.tp_cross_entropy_train(X, shards, u, ignore_index=IGNORE)
    got = rtp.tp_cross_entropy_train(X, shards, t, ignore_index=7)
    assert all(torch.equal(a, b) for a, b in zip([*got[:3], *got[3]], [*want[:3], *want[3]]))


def test_refusals_of_the_binding():
    X, W, shards, t = _inputs(6, 64, 512, 2, 512)
    call, train = rtp.tp_cross_entropy, rtp.tp_cross_entropy_train
    wide = torch.zeros((6, 128), dtype=BF16, device="cuda")
    for bad in (lambda: call(wide[:, ::2], shards, t), lambda: call(X, shards, t[:5]), lambda: call(X, shards, t.float()),
                lambda: call(X, shards, t.cpu()), lambda: call(X, shards, t[:, None]), lambda: call(X.float(), shards, t),
                lambda: call(X, [shards[0], shards[1][:, :8]], t), lambda: call(X, shards, t, vocab=0),
                lambda: call(X, shards, t, vocab=513), lambda: call(X, [w[:, :252].contiguous() for w in shards], t),
                lambda: train(X, shards, t, weights=torch.ones(6, dtype=torch.float64, device="cuda")),
                lambda: train(X, shards, t, weights=torch.ones(5, device="cuda")), lambda: train(X, shards, t, reduction="none"),
                lambda: train(X, shards, t, accumulate=True, dW=[torch.zeros_like(w) for w in shards]),
                lambda: train(X, shards, t, piece_rows=-1), lambda: train(X, shards, t, dX=wide),
                lambda: train(X, shards, t, loss=torch.zeros(6, dtype=BF16, device="cuda"))):
        with pytest.raises(rtp.RtpError):
            bad()
    with pytest.raises(TypeError):
        train(X, shards, t, dw_dtype=torch.float16)


@pytest.mark.parametrize("reduction", ["mean", "sum"])
@pytest.mark.parametrize("M,piece", [(4, 0), (300, 0), (600, 256)])
def test_weights_of_ignored_rows_hold_anything(M, piece, reduction):
    """NaN, infinite and huge weights in ignored rows (a quotient over padded rows is 0 / 0) change nothing."""
    X, W, shards, t = _inputs(M, 64, 512, 2, 512, ignored=0.0, seed=19)
    w = torch.rand((M,), device="cuda") + 0.5
    bad = [0, 2, M - 2][:M - 1]
    t[bad] = IGNORE
    w[bad] = 1.0
    call = lambda: rtp.tp_cross_entropy_train(X, shards, t, weights=w, ignore_index=IGNORE, reduction=reduction, piece_rows=piece)
    want = call()
    assert torch.isfinite(want[0])
    for value in (float("nan"), float("inf"), -float("inf"), 3e38):
        w[bad] = value
        got = call()
        assert all(torch.equal(a, b) for a, b in zip([*got[:3], *got[3]], [*want[:3], *want[3]])), value


# padding inside a tile, from the middle of a rank on, over whole ranks, with dX in slices of the vocabulary, in pieces
@pytest.mark.parametrize("M,K,V,P,vocab,piece", [
    (3, 64, 512, 2, 509, 0), (100, 64, 768, 3, 300, 0), (300, 64, 512, 2, 500, 0), (300, 136, 2064, 2, 1000, 0),
    (257, 200, 2048, 8, 257, 0), (129, 72, 1048, 1, 1, 0), (256, 512, 8192, 2, 8131, 0), (256, 512, 8192, 2, 4000, 0),
    (300, 264, 24600, 3, 9001, 0), (600, 136, 1056, 2, 1001, 256)])
def test_padding_columns_hold_anything(M, K, V, P, vocab, piece):
    """Columns of the weights from `vocab` on take no part: not NaN, not infinities, nor the largest values."""
    X, W, _, t = _inputs(M, K, V, P, vocab, seed=20)
    call = lambda: rtp.tp_cross_entropy_train(X, [w.contiguous() for w in W.chunk(P, 1)], t, vocab=vocab, ignore_index=IGNORE,
                                              piece_rows=piece)
    W[:, vocab:] = 0.0
    want = call()
    _check_train(X, W, t, vocab, want)
    for value in (float("nan"), float("inf"), -3.38e38):
        W[:, vocab:] = value
        got = call()
        assert all(torch.equal(a, b) for a, b in zip([*got[:3], *got[3]], [*want[:3], *want[3]])), value
        loss, lse = rtp.tp_cross_entropy(X, [w.contiguous() for w in W.chunk(P, 1)], t, vocab=vocab, ignore_index=IGNORE)
        assert torch.isfinite(loss).all() and torch.isfinite(lse).all()
    assert rtp.device_error() == 0


@pytest.mark.parametrize("M", [5, 600])
def test_a_piece_of_more_rows_than_there_are(M):
    X, W, shards, t = _inputs(M, 64, 512, 2, 512, seed=23)
    want = rtp.tp_cross_entropy_train(X, shards, t, ignore_index=IGNORE, piece_rows=M)
    for piece in (1 << 31, (1 << 63) - 1):
        got = rtp.tp_cross_entropy_train(X, shards, t, ignore_index=IGNORE, piece_rows=piece)
        assert all(torch.equal(a, b) for a, b in zip([*got[:3], *got[3]], [*want[:3], *want[3]]))


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("M,K,V,P,piece", [(7, 200, 1040, 2, 0), (300, 200, 1040, 2, 0), (256, 512, 8192, 2, 0),
                                           (600, 136, 1056, 2, 256)])
def test_rows_do_not_meet(M, K, V, P, piece, far):
    """Other rows, of ordinary logits or of some hundreds, leave a row's loss and gradient as they are, bit for bit."""
    X, W, shards, t = _inputs(M, K, V, P, V, seed=21)
    Y, _, _, u = _inputs(M, K, V, P, V, seed=22, spread=100.0 if far else 1.0)
    keep = torch.rand((M,), device="cuda") < 0.5
    keep[0], keep[M // 2] = True, False
    Y[keep], u[keep] = X[keep], t[keep]
    assert not torch.equal(X, Y)
    train = lambda x, y: rtp.tp_cross_entropy_train(x, shards, y, ignore_index=IGNORE, reduction="sum", piece_rows=piece)
    for a, b in zip(train(X, t)[1:3], train(Y, u)[1:3]):
        assert torch.equal(a[keep], b[keep]) and not torch.equal(a, b)
    for a, b in zip(*(rtp.tp_cross_entropy(x, shards, y, ignore_index=IGNORE) for x, y in ((X, t), (Y, u)))):
        assert torch.equal(a[keep], b[keep]) and not torch.equal(a, b)


@pytest.mark.parametrize("P", [1, 3])
def test_far_rows_in_many_tiles(P):
    """Several tiles for every pair of SMs, some of whose rows are gone through once more relative to their largest logit."""
    M, V = 1300, 24 * 1016
    X, W, _, t = _inputs(M, 64, V, P, V - 5, seed=24)
    X[5::7] *= 200
    W[:, 3000:9000] *= 4
    shards = [w.contiguous() for w in W.chunk(P, 1)]
    loss, lse = rtp.tp_cross_entropy(X, shards, t, vocab=V - 5, ignore_index=IGNORE)
    _check_forward(X, W, t, V - 5, loss, lse)
    _check_train(X, W, t, V - 5, rtp.tp_cross_entropy_train(X, shards, t, vocab=V - 5, ignore_index=IGNORE))
