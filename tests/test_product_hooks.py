"""The test hook and the launch counts of the products, on the host."""
import resharding_tensor_parallelism_gb300 as rtp
from resharding_tensor_parallelism_gb300 import _build


def test_hooks_and_counts():
    _build.build()
    assert rtp.lib().rtp_test_hook(rtp.HOOK_NO_CLUSTERS, 4) == 0
    assert rtp.lib().rtp_test_hook(rtp.HOOK_WAIT_LIMIT, 1_000_000) == 0
    for hook, arg in ((-1, 0), (rtp.HOOK_WAIT_LIMIT + 1, 0), (rtp.HOOK_WAIT_LIMIT, 999_999), (rtp.HOOK_WAIT_LIMIT, 4_000_000_001)):
        assert rtp.lib().rtp_test_hook(hook, arg) == -1
    rtp.test_hook(rtp.HOOK_NONE)
    rtp.product_launches()  # what this thread launched before
    assert rtp.product_launches() == {"few": 0, "whole": 0, 2: 0, 3: 0, 4: 0}
    assert rtp.lib().rtp_product_launches(None) == -1 and "rtp_product_launches" in rtp.last_error()
