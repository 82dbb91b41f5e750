"""GPU tests of the global gradient norm and of clipping against float64.

Bounds: the norm's sums are float32 over at most 64 squares and float64 beyond, so the norm is within 2^-17 of the exact
one (64 roundings of 2^-24 and the final one); a clipped value is within that plus the roundings of the quotient and the
product (2^-22) of its exact value, and one rounding to its type."""
import math

import pytest
import torch

from gpu_util import GUARD_BYTES, Guarded

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
NORM_REL = 2.0 ** -17
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


def _grads(sizes, dtypes=(BF16, F32), std=1e-2, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * std).to(dtypes[i % len(dtypes)]) for i, n in enumerate(sizes)]


def _exact(grads, counted=None):
    return math.sqrt(sum(float((t.double() ** 2).sum()) for i, t in enumerate(grads) if counted is None or counted[i]))


def _check(grads, max_norm, counted=None, norm_rel=NORM_REL):
    want = _exact(grads, counted)
    assert abs(float(rtp.grad_norm(grads, counted=counted)) - want) <= norm_rel * want
    g = Guarded()
    out = [g.empty(tuple(t.shape), t.dtype, "out[%d]" % i) for i, t in enumerate(grads)]
    before = [t.clone() for t in grads]
    norm, got = rtp.clip_grad_norm(grads, max_norm, counted=counted, out=out)
    g.check("clip")
    assert abs(float(norm) - want) <= norm_rel * want
    c = min(1.0, max_norm / (want + 1e-6))
    for t, b, o in zip(grads, before, got):
        assert torch.equal(t, b)  # the gradients themselves stay
        ref = b.double() * c
        rel = norm_rel + 2.0 ** -22 + (2.0 ** -8 if t.dtype is BF16 else 2.0 ** -23)
        assert bool(((o.double() - ref).abs() <= rel * ref.abs() + 1e-37).all())
    norm2, same = rtp.clip_grad_norm(grads, max_norm, counted=counted)  # in place: the same bits
    assert torch.equal(norm2, norm) and all(torch.equal(a, b) for a, b in zip(same, got)) and same[0] is grads[0]


@pytest.mark.parametrize("sizes", [[1], [7], [8], [9], [1000], [1, 2, 3, 0, 4, 5, 6, 7, 8, 9], [4096 * 8 + 3], [16383, 1, 16385],
                                   [1 << 20, 5, 12345], list(range(1, 64)), list(range(1, 66)), [3] * 513, [777] * 1500])
@pytest.mark.parametrize("dtypes", [(BF16,), (F32,), (BF16, F32)])
def test_sizes(sizes, dtypes):
    _check(_grads(sizes, dtypes), 0.05, seed_counted(sizes))


def seed_counted(sizes):
    return None if len(sizes) < 3 else [i % 3 != 2 for i in range(len(sizes))]


@pytest.mark.parametrize("max_norm", [0.0, 1e-3, 1.0, 1e9, float("inf")])
def test_limits(max_norm):
    _check(_grads([5000, 333, 70001]), max_norm)


def test_large():
    """Past 2^31 bytes in one tensor, and offsets past 2^31 elements."""
    _check(_grads([(1 << 31) + 12345, 99], (BF16,)), 1.0)


def test_unaligned_views():
    """Tensors that start at any element, read and written without vectors."""
    base = _grads([40000, 40000], (BF16, F32), seed=4)
    for lo in (1, 2, 3, 4, 7):
        views = [b[lo:lo + 9999] for b in base] + [base[0][20000 + lo:30000]]
        want = _exact(views)
        norm, out = rtp.clip_grad_norm(views, 0.1, out=[torch.empty_like(v) for v in views])
        assert abs(float(norm) - want) <= NORM_REL * want
        raw = torch.full((2 * 9999 + 64 + 2 * GUARD_BYTES,), 0x5A, dtype=torch.uint8, device="cuda")
        dst = raw[GUARD_BYTES + 2:GUARD_BYTES + 2 + 2 * 9999].view(BF16)  # 2 bytes off
        rtp.clip_grad_norm(views[:1], 1e9, out=[dst])
        assert torch.equal(dst, views[0])
        assert bool((raw[:GUARD_BYTES + 2] == 0x5A).all()) and bool((raw[GUARD_BYTES + 2 + 2 * 9999:] == 0x5A).all())


@pytest.mark.parametrize("value", [1e-30, 3e-25, 1e-12, 1.0, 1e15, 1e25, 1e36])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_squares_outside_float32(value, dtype):
    t = torch.full((5000,), value, dtype=dtype, device="cuda")
    t[::2] = 0
    z = torch.zeros(3000, dtype=dtype, device="cuda")
    want = _exact([t, z])
    assert abs(float(rtp.grad_norm([t, z])) - want) <= NORM_REL * want


def test_zero_nan_and_infinity():
    assert float(rtp.grad_norm([])) == 0.0
    norm, got = rtp.clip_grad_norm([], 1.0)
    assert float(norm) == 0.0 and got == []
    zeros = [torch.zeros(1000, device="cuda"), torch.full((10,), -0.0, dtype=BF16, device="cuda"), torch.empty(0, device="cuda")]
    norm, got = rtp.clip_grad_norm(zeros, 1.0)
    assert float(norm) == 0.0 and not bool(got[0].any())
    for bad in (float("nan"), float("inf"), float("-inf")):
        a, b = _grads([3000, 70000])
        b[69999] = bad
        norm, out = rtp.clip_grad_norm([a, b], 1.0, out=[torch.empty_like(a), torch.empty_like(b)])
        if math.isnan(bad):
            assert math.isnan(float(norm)) and all(bool(o.isnan().all()) for o in out)
        else:  # c = max_norm / inf = 0: finite values become 0, the infinite one 0 * inf
            assert float(norm) == math.inf and not bool(out[0].any()) and math.isnan(float(out[1][-1]))
        # a tensor that does not count does not reach the norm
        assert abs(float(rtp.grad_norm([a, b], counted=[True, False])) - _exact([a])) <= NORM_REL * _exact([a])


def test_rank_pieces_of_a_layout():
    """The norm of a sharded gradient is the logical tensor's: replicas count once, uneven pieces whole."""
    full = _grads([13 * 22], (F32,))[0].view(13, 22)
    want = _exact([full])
    for mesh, entries in (((3,), (("S", 0),)), ((2, 2), ("B", ("S", 1))), ((2, 2), (("S", 0), ("S", 1))), ((4,), ("B",)),
                          ((2, 3), (("S", 1), "B"))):
        spec = rtp.spec_nd_sbp(mesh, entries)
        pieces = rtp.shard(full, spec)
        flags = rtp.counted_pieces(spec)
        assert abs(float(rtp.grad_norm(pieces, counted=flags)) - want) <= NORM_REL * want
    with pytest.raises(rtp.RtpError):
        rtp.counted_pieces(rtp.spec_nd_sbp((2,), ("P",)))


def test_group_reads_new_values_streams_and_graph():
    grads = _grads([5000, 70000, 33])
    group = rtp.GradGroup(grads)
    first = group.norm()
    for t in grads:
        t.mul_(4)
    assert torch.equal(group.norm(), 4 * first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = group.norm(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(on_side, 4 * first)
    out = [torch.empty_like(t) for t in grads]
    group.clip(0.5, out=out)
    want = [t.clone() for t in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm, _ = group.clip(0.5, out=out)
    for t in out:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, 4 * first) and all(torch.equal(a, b) for a, b in zip(out, want))


def test_refusals():
    a, b = _grads([100, 100], (F32,))
    for call, status in ((lambda: rtp.clip_grad_norm([a, a], 1.0), -1),                       # in place, listed twice
                         (lambda: rtp.clip_grad_norm([a, a[10:]], 1.0), -1),                  # in place, overlapping
                         (lambda: rtp.clip_grad_norm([a, b], 1.0, out=[b, torch.empty_like(b)]), -1),
                         (lambda: rtp.clip_grad_norm([a], -1.0), -1), (lambda: rtp.clip_grad_norm([a], float("nan")), -1),
                         (lambda: rtp.clip_grad_norm([a, b], 1.0, out=[torch.empty_like(a)]), -1),
                         (lambda: rtp.clip_grad_norm([a], 1.0, out=[torch.empty(99, device="cuda")]), -2),
                         (lambda: rtp.clip_grad_norm([a], 1.0, out=[torch.empty(100, dtype=BF16, device="cuda")]), -2),
                         (lambda: rtp.grad_norm([a.view(10, 10).t()]), -1), (lambda: rtp.grad_norm([a.cpu()]), -1),
                         (lambda: rtp.grad_norm([a, b.cpu()]), -1), (lambda: rtp.grad_norm([a], counted=[True, True]), -1)):
        with pytest.raises(rtp.RtpError) as e:
            call()
        assert e.value.status == status
    with pytest.raises(TypeError):
        rtp.grad_norm([a.double()])
    assert float(rtp.grad_norm([a, a])) > 0  # reading a tensor twice is allowed
    norm, out = rtp.clip_grad_norm([a, b], 1e9, out=[a, torch.empty_like(b)])  # an output may be its own input
    assert torch.equal(out[1], b)
