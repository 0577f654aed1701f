"""Dropout in the reduce-scatter and the all-gather over many narrow rows: each
rank's part of a row is a few elements, less than a vector or little more."""
import numpy as np
import pytest
import torch

import workloads
from tests import ops_reference as ref
from tests.test_gpu_ops import DEV, DT, close, f64, say, vrc  # noqa: F401  (vrc: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n,outer,width", [(16, 16384, 1), (5, 16385, 3), (3, 20011, 7), (8, 16384, 8), (2, 30001, 15),
                                           (3, 5003, 23), (2, 5003, 33), (2, 2001, 63), (2, 2001, 64), (3, 1001, 67)])
def test_narrow_rows(vrc, n, outer, width, dtype):  # noqa: F811
    say(f"narrow rows n={n} {dtype} [{outer}, {n} x {width}]")
    xs = workloads.random_ranks(n, (outer, width * n), dtype, seed=width, device=DEV)
    rs = workloads.random_ranks(n, (outer, width), dtype, seed=100 + width, device=DEV)
    y, tol = ref.dropped_sum([f64(x) for x in xs], 0.4, 31, 32)
    y, tol = y.reshape(outer, n, width), tol.reshape(outer, n, width)
    plain = vrc.vrc_reduce_scatter_dropout(xs, 0.4, 31, 32, dim=1)
    added = vrc.vrc_reduce_scatter_dropout(xs, 0.4, 31, 32, residual=rs, dim=1)
    for c in range(n):
        want, t = y[:, c], tol[:, c]
        close(plain[c], want, t + ref.rounding(np.abs(want) + t, dtype), f"chunk {c}")
        r = f64(rs[c])
        t = t + (np.abs(want) + t + np.abs(r)) * 2.0**-24
        close(added[c], want + r, t + ref.rounding(np.abs(want + r) + t, dtype), f"chunk {c} with its residual")
    y, tol = ref.dropped_sum([np.concatenate([f64(r) for r in rs], axis=1)], 0.4, 31, 32)
    got = vrc.vrc_all_gather_dropout(rs, 0.4, 31, 32, dim=1)
    close(got[0], y, tol + ref.rounding(np.abs(y) + tol, dtype), "gather")
    assert all(torch.equal(got[0], g) for g in got)
    again = vrc.vrc_reduce_scatter_dropout(xs, 0.4, 31, 32, residual=rs, dim=1, recv=rs)
    assert all(torch.equal(a, b) for a, b in zip(again, added))


def replay_us(call, calls=4):
    """The least time of one of `calls` calls captured together."""
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(calls):
            call()
    best = float("inf")
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3 / calls)
    return best


@pytest.mark.parametrize("width", [1, 3, 8, 17])
def test_narrow_rows_use_the_whole_card(vrc, width):  # noqa: F811
    """The same elements in wide rows are one stream; narrow rows take a few times as
    long.  On one workgroup they took a thousand times."""
    n, outer = 8, 16384
    times = {}
    for rows, w in ((outer, width), (outer // 1024, width * 1024)):
        xs = workloads.random_ranks(n, (rows, w * n), "fp16", seed=1, device=DEV)
        rs = workloads.random_ranks(n, (rows, w), "fp16", seed=2, device=DEV)
        full, part = [torch.empty_like(x) for x in xs], [torch.empty_like(r) for r in rs]
        times[rows] = (replay_us(lambda: vrc.vrc_reduce_scatter_dropout(xs, 0.3, 1, 2, residual=rs, dim=1, recv=part)),
                       replay_us(lambda: vrc.vrc_all_gather_dropout(rs, 0.3, 1, 2, dim=1, recv=full)))
    say(f"width {width}: {times}")
    for narrow, wide in zip(times[outer], times[outer // 1024]):
        assert narrow < 6 * wide + 10


def test_narrow_rows_past_32_bits(vrc):  # noqa: F811
    n, outer, width = 2, (1 << 29) + 3, 4
    total = outer * n * width
    x = torch.ones(outer, n * width, dtype=torch.float16, device=DEV)
    parts = vrc.vrc_reduce_scatter_dropout([x, x], 0.25, 77, 5, dim=1)
    whole = vrc.vrc_all_gather_dropout(parts, 0.25, 77, 5, dim=1)
    for row in (0, (1 << 28) - 2, (1 << 29) - 2, outer - 4):
        k = ref.keep(row * n * width, 4 * n * width, 0.25, 77, 5).reshape(4, n, width)
        for c in range(n):
            assert ((parts[c][row:row + 4] != 0).cpu().numpy() == k[:, c]).all(), (row, c)
        for w in whole:
            assert ((w[row:row + 4] != 0).cpu().numpy() == k.reshape(4, -1)).all(), row
    assert total > 1 << 32
