"""The bench line's DRAM traffic figures are those of the kernels' present sources. No GPU needed."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


@pytest.mark.parametrize("kernel,workload", [("tp_gemm_kernel", "mlp"), ("tp_gemm_kernel", "mlp_backward"), ("boxing_kernel", "sweep")])
def test_traffic_is_of_the_present_source(kernel, workload):
    import bench

    assert bench._traffic(kernel, workload), "taken at another source of %s: capture it again" % kernel
