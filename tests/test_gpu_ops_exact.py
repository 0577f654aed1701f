"""The dropout collectives' stated arithmetic, bit for bit: the ranks' values folded in
rank order in fp32, the product with the scale rounded to fp32, the residual added in
fp32, and one rounding to the storage type; signed zeros included."""
import numpy as np
import pytest
import torch

import workloads
from tests import ops_reference as ref
from tests.test_gpu_ops import DEV, DT, chunk, say, vrc  # noqa: F401  (vrc: the fixture)

pytestmark = pytest.mark.gpu


def inputs(n, shape, dtype, seed, sigma=1.0):
    """Random values, with signed zeros in the same places of every rank."""
    xs = workloads.random_ranks(n, shape, dtype, seed=seed, device=DEV, sigma=sigma)
    for x in xs:
        x.view(-1)[3::16] = -0.0
        x.view(-1)[5::16] = 0.0
    return xs


def f32(t):
    return t.float().cpu().numpy()


def dropped(parts, p, seed, offset):
    """fp32 values of drop(fold of parts), parts flat and in fp32."""
    y = parts[0]
    for x in parts[1:]:
        y = y + x
    scale = np.float32(1.0 / (1.0 - p)) if p < 1 else np.float32(0)
    return np.where(ref.keep(0, y.size, p, seed, offset).reshape(y.shape), y * scale, np.float32(0))


def same_bits(got, want32, dtype, what):
    want = torch.from_numpy(np.ascontiguousarray(want32, dtype=np.float32)).to(DT[dtype])
    bits = torch.int32 if dtype == "fp32" else torch.int16
    a, b = got.cpu().reshape(-1).view(bits), want.reshape(-1).view(bits)
    bad = (a != b).nonzero()
    assert not len(bad), (what, len(bad), got.cpu().reshape(-1)[bad[:3, 0]], want.reshape(-1)[bad[:3, 0]])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n", [1, 3, 8])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_allreduce_dropout_bits(vrc, n, dtype, p):  # noqa: F811
    count = 100003  # heads and tails beside the vectors
    xs, rs = inputs(n, count, dtype, 1), inputs(n, count, dtype, 2, sigma=4.0)
    y = dropped([f32(x) for x in xs], p, 5, 6)
    assert (np.signbit(y) & (y == 0)).any()
    for r, got in enumerate(vrc.vrc_allreduce_dropout(xs, p, 5, 6)):
        same_bits(got, y, dtype, f"rank {r}")
    for r, got in enumerate(vrc.vrc_allreduce_dropout(xs, p, 5, 6, residual=rs)):
        same_bits(got, y + f32(rs[r]), dtype, f"rank {r} with its residual")
    for r, got in enumerate(vrc.vrc_allreduce_dropout(xs, p, 5, 6, residual=rs[0])):
        same_bits(got, y + f32(rs[0]), dtype, f"rank {r} with the shared residual")


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n,outer,width", [(1, 7, 501), (3, 1, 100003), (3, 4001, 7), (8, 501, 40), (3, 301, 301), (8, 64, 512)])
def test_scattered_and_gathered_bits(vrc, n, outer, width, dtype):  # noqa: F811
    say(f"bits n={n} [{outer}, {width}] {dtype}")
    dim = 1 if outer > 1 else 0
    shape = (outer, width * n) if outer > 1 else (width,)
    xs = inputs(n, shape, dtype, 3)
    y = dropped([f32(x) for x in xs], 0.3, 7, 8)
    spans = [chunk(shape[-1], n, c) for c in range(n)]
    parts = [y[..., lo:hi] for lo, hi in spans]
    rs = [inputs(1, q.shape, dtype, 20 + c, sigma=4.0)[0] for c, q in enumerate(parts)]
    for c, got in enumerate(vrc.vrc_reduce_scatter_dropout(xs, 0.3, 7, 8, dim=dim)):
        same_bits(got, parts[c], dtype, f"chunk {c}")
    for c, got in enumerate(vrc.vrc_reduce_scatter_dropout(xs, 0.3, 7, 8, dim=dim, residual=rs)):
        same_bits(got, parts[c] + f32(rs[c]), dtype, f"chunk {c} with its residual")
    full = dropped([np.concatenate([f32(r) for r in rs], axis=-1)], 0.3, 7, 8)
    for r, got in enumerate(vrc.vrc_all_gather_dropout(rs, 0.3, 7, 8, dim=dim)):
        same_bits(got, full, dtype, f"gather, rank {r}")
