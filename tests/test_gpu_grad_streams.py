"""GPU tests of the gradient norm and of clipping on a stream that is not the current one: the workspace is zeroed before
the kernels that count in it, and its memory is not handed out again while they may still run."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
NORM_REL = 2.0 ** -17  # 64 roundings of 2^-24 and the final one
CLIP_REL = NORM_REL + 2.0 ** -22 + 2.0 ** -8  # and the quotient's and the product's, and one to bf16
CYCLES = 100_000_000  # about 50 ms of one busy thread
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


def _grads(sizes=(5000, 70000, 33), seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * 1e-2).to((BF16, F32)[i % 2]) for i, n in enumerate(sizes)]


def _exact(grads):
    return math.sqrt(sum(float((t.double() ** 2).sum()) for t in grads))


def _garbage():
    """Blocks of every small size in the current stream's pool, filled with ones."""
    blocks = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in (512, 1024, 4096, 5632, 6144, 10752, 16384)
              for _ in range(20)]
    del blocks


def _ready_stream():
    """A stream that has waited for all that the current one has been given, and the current one made busy."""
    torch.cuda.synchronize()
    _garbage()
    torch.cuda.synchronize()
    torch.cuda._sleep(CYCLES)
    return torch.cuda.Stream()


def _same(norm, got, want, before, max_norm):
    assert abs(float(norm) - want) <= NORM_REL * want
    c = min(1.0, max_norm / (want + 1e-6))
    for t, b in zip(got, before):
        ref = b.double() * c
        assert bool(((t.double() - ref).abs() <= CLIP_REL * ref.abs() + 1e-37).all())


@pytest.mark.parametrize("as_int", [False, True])
def test_one_call_forms_beside_a_busy_current_stream(as_int):
    """Nothing of the call may be queued on the busy current stream: it would come too late for the kernels."""
    grads = _grads()
    before, want = [t.clone() for t in grads], _exact(grads)
    side = _ready_stream()
    arg = side.cuda_stream if as_int else side
    norm = rtp.grad_norm(grads, stream=arg)
    norm2, got = rtp.clip_grad_norm(grads, 0.05, stream=arg)
    side.synchronize()
    with torch.cuda.stream(side):
        assert abs(float(norm) - want) <= NORM_REL * want
        _same(norm2, got, want, before, 0.05)
    torch.cuda.synchronize()


def test_one_call_forms_whose_kernels_run_late():
    """The workspace outlives the call on the stream that uses it: what the current stream allocates right after the
    call, and fills, is other memory."""
    for clip in (False, True):
        grads = _grads(seed=1)
        before, want = [t.clone() for t in grads], _exact(grads)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            torch.cuda._sleep(CYCLES)
        if clip:
            norm, got = rtp.clip_grad_norm(grads, 0.05, stream=side)
        else:
            norm, got = rtp.grad_norm(grads, stream=side), []
        filled = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in (512, 5136, 5632, 6144) for _ in range(50)]
        side.synchronize()
        with torch.cuda.stream(side):
            _same(norm, got, want, before, 0.05)
        torch.cuda.synchronize()
        del filled


def _call(group, how, side):
    """norm, or clip in place, on `side`: by the argument, or as the current stream."""
    if how.endswith("current"):
        with torch.cuda.stream(side):
            return (group.norm(), []) if how.startswith("norm") else group.clip(0.05)
    return (group.norm(stream=side), []) if how.startswith("norm") else group.clip(0.05, stream=side)


HOW = ["norm by argument", "norm, current", "clip by argument", "clip, current"]


@pytest.mark.parametrize("how", HOW)
def test_kept_group_built_on_a_busy_stream_and_used_on_another(how):
    grads = _grads(seed=2)
    before, want = [t.clone() for t in grads], _exact(grads)
    side = _ready_stream()
    group = rtp.GradGroup(grads)
    norm, got = _call(group, how, side)
    side.synchronize()
    with torch.cuda.stream(side):
        _same(norm, got, want, before, 0.05)
    torch.cuda.synchronize()


@pytest.mark.parametrize("how", HOW)
def test_kept_group_dropped_while_another_stream_uses_it(how):
    grads = _grads(seed=3)
    before, want = [t.clone() for t in grads], _exact(grads)
    group = rtp.GradGroup(grads)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
    norm, got = _call(group, how, side)
    del group
    filled = [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for n in (512, 5136, 5632, 6144) for _ in range(50)]
    side.synchronize()
    with torch.cuda.stream(side):
        _same(norm, got, want, before, 0.05)
    torch.cuda.synchronize()
    del filled


def test_kept_group_first_used_in_a_capture():
    grads = _grads(seed=4)
    before, want = [t.clone() for t in grads], _exact(grads)
    out = [torch.empty_like(t) for t in grads]
    group = rtp.GradGroup(grads)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm, _ = group.clip(0.05, out=out)
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        _same(norm, out, want, before, 0.05)
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        rtp.GradGroup(grads).norm()  # built and used within one capture
