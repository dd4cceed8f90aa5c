"""The bench line's DRAM traffic comes from captures of the kernels as they are:
each record's hash is that of the sources its kernel is compiled from. (A
declaration that other kernels need, put into a header of these, drops the
figures without a word.)
"""
import pytest

import bench


@pytest.mark.parametrize("kernel", sorted(bench.KERNEL_SOURCES))
def test_captured_traffic_is_of_the_current_sources(kernel):
    assert bench.ncu_traffic(kernel) is not None
