"""Refusals of the model's operators where a call would leave something unwritten, on the CPU."""
import pytest

import ring_all_reduce_virtual_amd as vrc
from ring_all_reduce_virtual_amd import ops
from tests.test_model_cpu import A, B, INVALID, R, T, W, arr, norm

L = ops.ops_lib()


@pytest.mark.parametrize("join", [0, 1, 2])
def test_rows_without_values_have_no_statistics(join):
    """Nothing would write mean and rstd of a row of width 0; without them, or without rows, the call has nothing to do."""
    def f(rows, mean=None, rstd=None, center=1):
        return L.vrc_layer_norm(norm(rows=rows, width=0, join=join, center=center), arr(A), None, W, None, arr(B), None, mean, rstd, 4, None)

    assert f(8, rstd=arr(R)) == f(8, mean=arr(T)) == f(8, mean=arr(T), rstd=arr(R)) == f(8, rstd=arr(R), center=0) == INVALID
    assert f(8) == f(0, mean=arr(T), rstd=arr(R)) == f(0) == vrc.VRC_OK
