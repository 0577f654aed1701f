"""The model's operators on the CPU: refusals where a call would leave something unwritten, and the
libraries' build where there is no torch."""
import importlib.util
import os

import pytest

import ring_all_reduce_virtual_amd as vrc
from ring_all_reduce_virtual_amd import build, ops
from tests.test_model_cpu import A, B, INVALID, R, T, W, arr, norm

L = ops.ops_lib()


@pytest.mark.parametrize("join", [0, 1, 2])
def test_rows_without_values_have_no_statistics(join):
    """Nothing would write mean and rstd of a row of width 0; without them, or without rows, the call has nothing to do."""
    def f(rows, mean=None, rstd=None, center=1):
        return L.vrc_layer_norm(norm(rows=rows, width=0, join=join, center=center), arr(A), None, W, None, arr(B), None, mean, rstd, 4, None)

    assert f(8, rstd=arr(R)) == f(8, mean=arr(T)) == f(8, mean=arr(T), rstd=arr(R)) == f(8, rstd=arr(R), center=0) == INVALID
    assert f(8) == f(0, mean=arr(T), rstd=arr(R)) == f(0) == vrc.VRC_OK


def test_libraries_build_without_torch(monkeypatch):
    """The binding is against torch's headers; the libraries and their C ABI need none."""
    before = os.stat(build.BINDING_LIB).st_mtime_ns
    monkeypatch.setattr(importlib.util, "find_spec", lambda name: None)
    monkeypatch.setattr(build.subprocess, "run", lambda *a, **k: pytest.fail("nothing is compiled"))
    assert build.build_binding() is None
    assert os.stat(build.BINDING_LIB).st_mtime_ns == before
