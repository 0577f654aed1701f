"""Outputs that an operator allocates: a storage of its own for each rank's."""
import io

import pytest
import torch

from ring_all_reduce_virtual_amd import ops

SHAPES = [(1024,), (64, 4, 8), (8,), (3,), (2, 4096), (1 << 20,), (1 << 21,)]


@pytest.mark.parametrize("shape", SHAPES)
def test_one_output_can_grow(shape):
    """A call that resizes its `out` may be given one rank's output: it does not reach
    into another rank's."""
    ys = ops._allocate([shape] * 3, torch.float32, torch.device("cpu"))
    for r, y in enumerate(ys):
        y.fill_(r)
    wide = (shape[0] * 2,) + shape[1:]
    ys[0].resize_(wide).fill_(7)
    assert (ys[1] == 1).all() and (ys[2] == 2).all()
    torch.add(torch.ones(wide), 1, out=ys[1].resize_(0))
    assert (ys[1] == 2).all() and (ys[2] == 2).all() and (ys[0] == 7).all()


@pytest.mark.parametrize("shape", SHAPES)
def test_one_output_holds_its_own_memory(shape):
    """Keeping or saving one rank's output keeps or writes no other's."""
    ys = ops._allocate([shape] * 4, torch.bfloat16, torch.device("cpu"))
    assert all(y.untyped_storage().nbytes() == y.nbytes and y.storage_offset() == 0 for y in ys)
    assert len({y.untyped_storage().data_ptr() for y in ys}) == 4
    with io.BytesIO() as f:
        torch.save(ys[1], f)
        assert f.tell() < ys[1].nbytes + 4096


def test_uneven_outputs():
    ys = ops._allocate([(5,), (5,), (7,)], torch.float16, torch.device("cpu"))
    assert [y.shape for y in ys] == [(5,), (5,), (7,)]
    assert all(y.untyped_storage().nbytes() == y.nbytes for y in ys)
