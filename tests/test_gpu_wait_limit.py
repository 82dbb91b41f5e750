"""The limit of the few-row kernel's waits covers its own progress. As a programmatic dependent its blocks can be resident
while the kernel before them still runs, however long that takes."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
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


@pytest.mark.parametrize("K,N", [(4096, 264), (256, 2048)])
def test_a_long_kernel_before_it_is_not_its_own_time(K, N):
    """A kernel of 200 ms that lets its dependents begin at once, before a product whose waits give up after 20 ms: the
    product is right (one that gave up leaves partial sums), and only the long kernel's own wait is reported."""
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    X = torch.randn((5, K), generator=g, device="cuda").to(BF16)
    W = [(torch.randn((K, N), generator=g, device="cuda") / K ** 0.5).to(BF16)]
    want = rtp.tp_linear(X, W, act="silu")[0]
    out = [torch.empty_like(want)]
    flags = rtp.wait_selftest(1_000_000)
    torch.cuda.synchronize()
    assert rtp.device_error() == 5
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    out[0].zero_()
    e0.record()
    rtp.wait_selftest(200_000_000, out=flags)
    rtp.test_hook(rtp.HOOK_WAIT_LIMIT, 20_000_000)
    rtp.tp_linear(X, W, act="silu", out=out)
    e1.record()
    torch.cuda.synchronize()
    assert rtp.device_error() == 5
    assert rtp.device_error() == 0
    assert 190 < e0.elapsed_time(e1) < 2000
    assert torch.equal(out[0], want)
