"""Calls that the operators' C functions refuse before any GPU work (the addresses are
stand-ins)."""
import ctypes as C

import ring_all_reduce_virtual_amd as vrc
from ring_all_reduce_virtual_amd import ops

L = ops.ops_lib()
A, B, R = 0x10000000, 0x50000000, 0x90000000  # far apart


def arr(base, n, stride=1 << 20):
    return vrc._ptr_array([base + r * stride for r in range(n)])


def test_a_mask_offset_inside_an_output():
    """The offset is read by every workgroup while others already write: in an output
    it would change under the call."""
    def drop(at):
        return C.byref(ops.Dropout(0.5, 1, 2, at))

    count, last = 1000, 3 << 20  # bf16: 2000 bytes a rank; the fourth rank's output
    for at in (B, B + 1992, B + last, B + last + 1992):
        assert L.vrc_allreduce_dropout(arr(A, 4), None, arr(B, 4), 4, count, vrc.VRC_BF16, drop(at), None) == vrc.VRC_ERR_ALIAS
        assert L.vrc_allreduce_dropout(arr(A, 4), arr(R, 4), arr(B, 4), 4, count, vrc.VRC_BF16, drop(at), None) == vrc.VRC_ERR_ALIAS
        assert L.vrc_all_gather_dropout(arr(A, 4), arr(B, 4), 4, count, 1, vrc.VRC_BF16, drop(at), None) == vrc.VRC_ERR_ALIAS
    for at in (B, B + last + 496):  # 500 bytes a rank, the last 8 of which start at 492
        assert L.vrc_reduce_scatter_dropout(arr(A, 4), None, arr(B, 4), 4, count, 1, vrc.VRC_BF16, drop(at), None) == vrc.VRC_ERR_ALIAS
        assert L.vrc_reduce_scatter_dropout(arr(A, 4), arr(R, 4), arr(B, 4), 4, count, 1, vrc.VRC_BF16, drop(at), None) == vrc.VRC_ERR_ALIAS
    # in place: the offset in what is input and output at once
    assert L.vrc_allreduce_dropout(arr(A, 4), None, arr(A, 4), 4, count, vrc.VRC_BF16, drop(A + 8), None) == vrc.VRC_ERR_ALIAS
