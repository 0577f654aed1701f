"""The tensor-parallel layer's operators on the GPU against 64-bit references
(tests/ops_reference.py).

Tolerances count roundings: an fp32 fold of N values and its scaling are off by at
most N + 1 half steps of the sum of magnitudes, the residual's addition by half a
step, the result's rounding by half a step of its type.  Quantisation and decoding
are exact and compared bit for bit.  A product of two 4-bit codes is exact; an fp32
sum of K of them is off by at most K half steps of the sum of magnitudes."""
import numpy as np
import pytest
import torch

import workloads
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def vrc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ring_all_reduce_virtual_amd as m
    return m


def say(msg):
    print(msg, flush=True)


def f64(t):
    return t.detach().double().cpu().numpy()


def chunk(count, n, c):
    base = count // n
    return c * base, (count if c == n - 1 else (c + 1) * base)


def close(got, want, tol, what, over=None):
    """`over`: where the result may have rounded to infinity (of the value's sign)."""
    got = f64(got).reshape(-1)
    want, tol = np.asarray(want).reshape(-1), np.asarray(tol).reshape(-1)
    assert got.shape == want.shape, what
    nan = np.isnan(want)
    assert (np.isnan(got) == nan).all(), what
    with np.errstate(invalid="ignore"):
        bad = ~nan & ~(got == want) & ~(np.abs(got - want) <= tol)
        if over is not None:
            bad &= ~(np.isinf(got) & (np.sign(got) == np.sign(want)) & over.reshape(-1))
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4], np.nonzero(bad)[0][:4])


def check_dropped(got, xs, res, p, seed, offset, dtype, what, first=0):
    y, tol = ref.dropped_sum([f64(x) for x in xs], p, seed, offset, first)
    if res is not None:
        r = f64(res).reshape(-1)
        tol = tol + (np.abs(y) + tol + np.abs(r)) * 2.0**-24
        y = y + r
    close(got, y, tol + ref.rounding(np.abs(y) + tol, dtype), what)


# ---------------------------------------------------------------------------
# Dropout in the all-reduce
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n", [1, 2, 3, 5, 8, 13, 16])
@pytest.mark.parametrize("residual", ["none", "shared", "each"])
def test_allreduce_dropout(vrc, n, dtype, residual):
    for count in (1, 3, 5, 64, 511, 4096, 100003):
        say(f"allreduce_dropout n={n} {dtype} {residual} count={count}")
        xs = workloads.random_ranks(n, count, dtype, seed=10 + count, device=DEV)
        rs = workloads.random_ranks(n, count, dtype, seed=900 + count, device=DEV, sigma=4.0)
        res = {"none": None, "shared": rs[0], "each": rs}[residual]
        seed, offset, p = 0x1234567890ABCDEF ^ count, (1 << 40) + count, 0.3
        ys = vrc.vrc_allreduce_dropout(xs, p, seed, offset, residual=res)
        for r in range(n):
            check_dropped(ys[r], xs, None if res is None else rs[0 if residual == "shared" else r], p, seed, offset, dtype,
                          f"rank {r}")


@pytest.mark.parametrize("dtype", DT)
def test_allreduce_dropout_operands_on_any_element(vrc, dtype):
    n, count = 4, 5003
    for shift in ((0, 1, 2, 3), (5, 5, 5, 5), (1, 0, 7, 4)):
        say(f"offsets {shift} {dtype}")

        def views(seed):
            base = workloads.random_ranks(n, count + 16, dtype, seed=seed, device=DEV)
            return [b[s:s + count] for b, s in zip(base, shift)]

        xs, rs, out = views(1), views(2), views(3)
        guard = [o._base.clone() for o in out]
        vrc.vrc_allreduce_dropout(xs, 0.5, 7, 8, residual=rs, recv=out)
        for r in range(n):
            check_dropped(out[r], xs, rs[r], 0.5, 7, 8, dtype, f"rank {r}")
            g = guard[r]
            g[shift[r]:shift[r] + count] = out[r]
            assert torch.equal(g.view(torch.uint8), out[r]._base.view(torch.uint8)), "written outside"


@pytest.mark.parametrize("n", [1, 3, 8])
def test_allreduce_dropout_in_place(vrc, n):
    count = 70001
    for where in ("send", "residual"):
        xs = workloads.random_ranks(n, count, "bf16", seed=3, device=DEV)
        rs = workloads.random_ranks(n, count, "bf16", seed=4, device=DEV)
        want = [w.clone() for w in vrc.vrc_allreduce_dropout(xs, 0.2, 1, 2, residual=rs)]
        got = vrc.vrc_allreduce_dropout(xs, 0.2, 1, 2, residual=rs, recv=xs if where == "send" else rs)
        for r in range(n):
            assert torch.equal(got[r], want[r]), (where, r)


def test_allreduce_dropout_extreme_probabilities_and_values(vrc):
    n, count = 3, 1000
    xs = workloads.random_ranks(n, count, "fp16", seed=5, device=DEV)
    rs = workloads.random_ranks(n, count, "fp16", seed=6, device=DEV)
    plain = vrc.vrc_allreduce(xs, mode="fused")
    for got, want in zip(vrc.vrc_allreduce_dropout(xs, 0.0, 1, 2), plain):
        assert torch.equal(got, want)
    for got, want in zip(vrc.vrc_allreduce_dropout(xs, 1.0, 1, 2, residual=rs), rs):
        assert torch.equal(got, want)
    assert not any(y.any() for y in vrc.vrc_allreduce_dropout(xs, 1.0, 1, 2))
    # the smallest threshold, and a probability that rounds to dropping everything
    check_dropped(vrc.vrc_allreduce_dropout(xs, 2.0**-32, 1, 2)[0], xs, None, 2.0**-32, 1, 2, "fp16", "2^-32")
    assert not any(y.any() for y in vrc.vrc_allreduce_dropout(xs, 1.0 - 2.0**-34, 1, 2))
    # what is dropped is zero whatever it was; what is kept passes infinities and NaN on
    xs[0][0::3], xs[1][1::3], xs[2][2::3] = float("inf"), float("nan"), -float("inf")
    keep = torch.from_numpy(ref.keep(0, count, 0.5, 9, 10)).to(DEV)
    y = vrc.vrc_allreduce_dropout(xs, 0.5, 9, 10)[0]
    assert not y[~keep].any() and not torch.isfinite(y[keep]).any()
    assert torch.equal(torch.isnan(y[keep]), (torch.arange(count, device=DEV) % 3 == 1)[keep])
    # fp32 sums of fp16 values pass 65504 and come back
    big = [torch.full((64,), v, dtype=torch.float16, device=DEV) for v in (60000.0, 60000.0, -60000.0)]
    assert (vrc.vrc_allreduce_dropout(big, 0.0, 0)[0] == 60000.0).all()
    assert vrc.vrc_allreduce_dropout([x[:0] for x in xs], 0.5, 1)[0].numel() == 0


def test_dropout_fraction_and_independence(vrc):
    x = [torch.ones(1 << 22, device=DEV)]
    for p in (0.1, 0.5, 0.9):
        a = vrc.vrc_allreduce_dropout(x, p, 42, 0)[0] != 0
        b = vrc.vrc_allreduce_dropout(x, p, 42, 1)[0] != 0
        c = vrc.vrc_allreduce_dropout(x, p, 43, 0)[0] != 0
        sd = (p * (1 - p) / x[0].numel()) ** 0.5
        for m in (a, b, c):
            assert abs(m.double().mean().item() - (1 - p)) < 6 * sd
        for m, k in ((a, b), (a, c), (a[:-1], a[1:])):
            both, q = (m & k).double().mean().item(), (1 - p) ** 2
            assert abs(both - q) < 6 * (q * (1 - q) / m.numel()) ** 0.5


def test_allreduce_dropout_past_32_bits(vrc):
    count = (1 << 32) + 37
    x = torch.ones(count, dtype=torch.bfloat16, device=DEV)
    y = vrc.vrc_allreduce_dropout([x], 0.25, 77, 5, recv=[x])[0]
    for first in (0, (1 << 31) - 20, (1 << 32) - 20, count - 40):
        k = ref.keep(first, 40, 0.25, 77, 5)[:min(40, count - first)]
        assert ((y[first:first + 40] != 0).cpu().numpy() == k).all(), first


# ---------------------------------------------------------------------------
# Reduce-scatter and all-gather
# ---------------------------------------------------------------------------
SPLITS = [(1, 1), (1, 5), (1, 16), (1, 1003), (1, 65536), (1, 100001), (2, 1), (3, 7), (13, 512), (64, 33), (1000, 9),
          (7, 2048)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n", [1, 2, 3, 8, 16])
def test_reduce_scatter_dropout(vrc, n, dtype):
    for outer, width in SPLITS:
        w = width if outer == 1 else width * n
        say(f"reduce_scatter_dropout n={n} {dtype} [{outer}, {w}]")
        xs = workloads.random_ranks(n, (outer, w), dtype, seed=outer + w, device=DEV)
        y, tol = ref.dropped_sum([f64(x) for x in xs], 0.4, 11, 12)
        y, tol = y.reshape(outer, w), tol.reshape(outer, w)
        spans = [chunk(w, n, c) for c in range(n)]
        rs = [torch.randn(outer, hi - lo, device=DEV).to(DT[dtype]) for lo, hi in spans]
        for res in (None, rs):
            got = vrc.vrc_reduce_scatter_dropout(xs, 0.4, 11, 12, residual=res, dim=1 if outer > 1 else 0)
            for c, (lo, hi) in enumerate(spans):
                want, t = y[:, lo:hi], tol[:, lo:hi]
                if res is not None:
                    r = f64(rs[c])
                    t = t + (np.abs(want) + t + np.abs(r)) * 2.0**-24
                    want = want + r
                close(got[c], want, t + ref.rounding(np.abs(want) + t, dtype), f"chunk {c}")
        for a, b in zip(vrc.vrc_reduce_scatter_dropout(xs, 0.4, 11, 12, residual=rs, dim=1 if outer > 1 else 0, recv=rs), got):
            assert torch.equal(a.reshape(-1), b.reshape(-1))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n", [1, 2, 3, 8, 16])
def test_all_gather_dropout(vrc, n, dtype):
    for outer, width in SPLITS:
        say(f"all_gather_dropout n={n} {dtype} [{outer}, {width}]")
        xs = workloads.random_ranks(n, (outer, width), dtype, seed=outer + width, device=DEV)
        full = np.concatenate([f64(x) for x in xs], axis=1)
        y, tol = ref.dropped_sum([full], 0.4, 13, 14)
        got = vrc.vrc_all_gather_dropout(xs, 0.4, 13, 14, dim=1)
        for r in range(n):
            assert got[r].shape == full.shape
            close(got[r], y, tol + ref.rounding(np.abs(y) + tol, dtype), f"rank {r}")


def test_uneven_chunks_and_views(vrc):
    n, count = 5, 1003
    for dtype in DT:
        xs = [b[1:1 + count] for b in workloads.random_ranks(n, count + 8, dtype, seed=8, device=DEV)]
        out = [torch.zeros(chunk(count, n, c)[1] - chunk(count, n, c)[0] + 9, dtype=DT[dtype], device=DEV) for c in range(n)]
        views = [o[c % 4:c % 4 + o.numel() - 9] for c, o in enumerate(out)]
        vrc.vrc_reduce_scatter_dropout(xs, 0.3, 1, 2, recv=views)
        y, tol = ref.dropped_sum([f64(x) for x in xs], 0.3, 1, 2)
        for c in range(n):
            lo, hi = chunk(count, n, c)
            close(views[c], y[lo:hi], tol[lo:hi] + ref.rounding(np.abs(y[lo:hi]) + tol[lo:hi], dtype), f"chunk {c}")
            views[c].zero_()
            assert not out[c].any(), "written outside"
        chunks = [xs[0][slice(*chunk(count, n, c))] for c in range(n)]
        y, tol = ref.dropped_sum([f64(xs[0])], 0.3, 1, 2)
        for g in vrc.vrc_all_gather_dropout(chunks, 0.3, 1, 2):
            close(g, y, tol + ref.rounding(np.abs(y) + tol, dtype), "gather")
    with pytest.raises(ValueError):
        vrc.vrc_all_gather_dropout([xs[0][:10], xs[0][10:30], xs[0][30:60]], 0.3, 1)
    with pytest.raises(ValueError):
        vrc.vrc_all_gather_dropout([xs[0][:10], xs[0][10:19]], 0.3, 1)


@pytest.mark.parametrize("outer,width", [(1, 4003), (6, 56)])
def test_dropout_gradients(vrc, outer, width):
    """The documented gradients against the formulas' and against differences: a loss
    <y, dy> of fp32 outputs is linear in every input, so a difference of any size gives
    its slope up to the two evaluations' roundings."""
    n, p, seed, offset = 4, 0.35, 21, 22
    flat = outer == 1
    dim = 0 if flat else 1
    xs = workloads.random_ranks(n, (outer, width), "fp32", seed=30, device=DEV)
    keep = ref.keep(0, outer * width, p, seed, offset).reshape(outer, width) / (1 - p)

    ar_dy = workloads.random_ranks(n, (outer, width), "fp32", seed=31, device=DEV)
    grads = vrc.vrc_allreduce_dropout(ar_dy, p, seed, offset)
    want = keep * sum(f64(d) for d in ar_dy)
    mag = keep * sum(np.abs(f64(d)) for d in ar_dy)
    for g in grads:
        close(g, want, mag * (n + 2) * 2.0**-24, "all-reduce's gradient")

    spans = [chunk(width, n, c) for c in range(n)]
    rs_dy = [torch.randn((hi - lo,) if flat else (outer, hi - lo), device=DEV) for lo, hi in spans]
    full = np.concatenate([f64(d).reshape(outer, -1) for d in rs_dy], axis=1)
    rs_grads = vrc.vrc_all_gather_dropout(rs_dy, p, seed, offset, dim=dim)
    for g in rs_grads:
        close(g, keep * full, np.abs(keep * full) * 2 * 2.0**-24, "reduce-scatter's gradient")

    step = torch.randn(outer, width, device=DEV)
    for q in (0, n - 1):
        moved = [x + step if r == q else x for r, x in enumerate(xs)]
        h = f64(moved[q]) - f64(xs[q])
        for f, dys, grad in (
                (lambda v: vrc.vrc_allreduce_dropout(v, p, seed, offset), ar_dy, grads[q]),
                (lambda v: vrc.vrc_reduce_scatter_dropout(v, p, seed, offset, dim=dim), rs_dy, rs_grads[q])):
            a, b = f(xs), f(moved)
            slope = sum(((f64(v) - f64(u)) * f64(d)).sum() for u, v, d in zip(a, b, dys))
            bound = sum(((np.abs(f64(u)) + np.abs(f64(v))) * np.abs(f64(d))).sum() for u, v, d in zip(a, b, dys)) * 4 * (n + 2) * 2.0**-24
            assert abs(slope - (f64(grad).reshape(outer, width) * h).sum()) <= bound
    # the all-gather's own gradient is the reduce-scatter
    full_dy = workloads.random_ranks(n, (outer, width), "fp32", seed=33, device=DEV)
    back = vrc.vrc_reduce_scatter_dropout(full_dy, p, seed, offset, dim=dim)
    lhs = sum((keep * full * f64(d)).sum() for d in full_dy)
    rhs = sum((f64(g).reshape(-1) * f64(d).reshape(-1)).sum() for g, d in zip(back, rs_dy))
    assert abs(lhs - rhs) <= sum(np.abs(keep * full * f64(d)).sum() for d in full_dy) * (n + 4) * 2.0**-24


# ---------------------------------------------------------------------------
# Microscaled blocks
# ---------------------------------------------------------------------------
def check_quantised(codes, scales, x, what):
    wc, ws = ref.quantise(x)
    assert (scales.cpu().numpy().reshape(ws.shape) == ws).all(), what
    got = ref.unpack(codes.cpu().numpy().reshape(ws.shape[0], -1))
    assert (got == wc).all(), (what, np.argwhere(got != wc)[:4])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("shape", [(1, 1), (1, 31), (1, 32), (3, 33), (5, 8), (33, 1), (64, 64), (257, 100), (2, 1000),
                                   (1000, 3), (300, 256), (31, 2049)])
def test_quantise_both_axes(vrc, dtype, shape):
    n = 3
    xs = []
    for r in range(n):
        x = torch.randn(shape, device=DEV) * torch.exp2(torch.randint(-12, 8, (shape[0], 1), device=DEV).float())
        x[torch.rand(shape, device=DEV) < 0.05] = 0
        xs.append(x.to(DT[dtype]))
    codes, scales = vrc.vrc_mx4_quantize(xs)
    tcodes, tscales = vrc.vrc_mx4_quantize(xs, dim=0)
    assert codes[0].shape == (shape[0], 16 * vrc.mx4_blocks(shape[1]))
    for r in range(n):
        check_quantised(codes[r], scales[r], f64(xs[r]), f"rank {r}")
        check_quantised(tcodes[r], tscales[r], f64(xs[r]).T, f"rank {r} transposed")
        y = vrc.vrc_mx4_dequantize(codes, scales, shape[1], dtype=DT[dtype])[r]
        want = torch.from_numpy(ref.decode(codes[r].cpu().numpy(), scales[r].cpu().numpy())[:, :shape[1]])
        assert torch.equal(y.cpu(), want.to(torch.float32).to(DT[dtype]))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("shape", [(256, 131), (500, 70), (225, 1), (1024, 260)])
def test_quantise_down_columns_in_whole_lines(vrc, dtype, shape):
    """Eight blocks of a column fill a memory line; codes on a line and 16 bytes off it."""
    xs = workloads.random_ranks(2, shape, dtype, seed=90, device=DEV)
    kb = -(-shape[0] // 32)
    room = [torch.full((shape[1] * kb * 16 + 32,), 0xA5, dtype=torch.uint8, device=DEV) for _ in xs]
    off = [t[16:-16].view(shape[1], kb * 16) for t in room]
    on_line = vrc.vrc_mx4_quantize(xs, dim=0)
    moved = vrc.vrc_mx4_quantize(xs, dim=0, codes=off)
    for x, c, s, c2, s2, t in zip(xs, *on_line, *moved, room):
        codes, scales = ref.quantise(f64(x).T)
        assert (ref.unpack(c.cpu().numpy()) == codes).all() and (s.cpu().numpy() == scales).all()
        assert torch.equal(c, c2) and torch.equal(s, s2)
        assert (t[:16] == 0xA5).all() and (t[-16:] == 0xA5).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_quantise_every_16_bit_value(vrc, dtype):
    """Each finite value beside block maxima of every exponent from its own upwards."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(DT[dtype])
    v = bits[torch.isfinite(bits)].double()
    rows = []
    for up in (0, 1, 2, 3, 5, 9):
        top = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0**-133))) + up)
        blk = torch.zeros(v.numel(), 32, dtype=torch.float64)
        blk[:, 7], blk[:, 20] = v, torch.where(v == 0, torch.zeros(()), top)
        rows.append(blk[torch.isfinite(blk.to(DT[dtype])).all(1)])
    x = torch.cat(rows).to(DT[dtype])
    codes, scales = vrc.vrc_mx4_quantize([x.to(DEV)])
    check_quantised(codes[0], scales[0], x.double().numpy(), dtype)
    tcodes, tscales = vrc.vrc_mx4_quantize([x[:4000].t().contiguous().to(DEV)], dim=0)
    check_quantised(tcodes[0], tscales[0], x[:4000].double().numpy(), dtype)


@pytest.mark.parametrize("dtype", DT)
def test_quantise_special_blocks(vrc, dtype):
    """Subnormals, signed zeros, the largest values, infinities and NaN."""
    t = DT[dtype]
    info = torch.finfo(t)
    x = torch.zeros(12, 64, dtype=t)
    x[0, 5] = info.smallest_normal / 2
    x[1, 6] = info.tiny * 2.0**-3
    x[2, :] = -0.0
    x[3, 1], x[3, 2] = info.max, -info.max / 4
    x[4, 3] = float("inf")
    x[5, 40] = -float("inf")
    x[6, 0] = float("nan")
    x[7, 63], x[7, 31] = float("nan"), 1.0
    x[8, :] = torch.linspace(-7, 7, 64).to(t)
    x[9, 0], x[9, 1] = 1.0, info.tiny
    x[10, 33] = 6.0 * info.tiny
    x[11, :] = info.smallest_normal
    codes, scales = vrc.vrc_mx4_quantize([x.to(DEV)])
    check_quantised(codes[0], scales[0], x.double().numpy(), dtype)
    tc, ts = vrc.vrc_mx4_quantize([x.t().contiguous().to(DEV)], dim=0)
    assert torch.equal(tc[0], codes[0]) and torch.equal(ts[0], scales[0])
    y = vrc.vrc_mx4_dequantize(codes, scales, dtype=t)[0].double().cpu()
    assert torch.isnan(y[4, :32]).all() and not torch.isnan(y[4, 32:]).any() and torch.isnan(y[7]).sum() == 32


def test_decode_every_code_and_scale(vrc):
    packed = ((torch.arange(32) % 16).view(16, 2) * torch.tensor([1, 16])).sum(1).to(torch.uint8).expand(256, 16).contiguous()
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1)
    want = torch.from_numpy(ref.decode(packed.numpy(), scales.numpy()))
    for t in DT.values():
        y = vrc.vrc_mx4_dequantize([packed.to(DEV)], [scales.to(DEV)], dtype=t)[0].cpu()
        w = want.to(torch.float32).to(t)  # fp32 holds every value but 2^127 * 2, 3, 4, 6, which overflow
        assert torch.equal(torch.isnan(y), torch.isnan(w)) and torch.equal(y[:255], w[:255])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n", [1, 2, 3, 8, 16])
def test_mx4_all_gather(vrc, n, dtype):
    for rows, cols in ((1, 1), (3, 32), (5, 40), (130, 96), (64, 1000), (1, 4096)):
        say(f"mx4_all_gather n={n} {dtype} [{rows}, {cols}]")
        xs = workloads.random_ranks(n, (rows, cols), dtype, seed=rows + cols, device=DEV)
        codes, scales = vrc.vrc_mx4_quantize(xs)
        own = [torch.from_numpy(ref.decode(c.cpu().numpy(), s.cpu().numpy())[:, :cols]).float().to(DT[dtype]) for c, s in zip(codes, scales)]
        for dim in (0, -1):
            got = vrc.vrc_mx4_all_gather(codes, scales, cols, dim=dim, dtype=DT[dtype])
            want = torch.cat(own, dim)
            for r in range(n):
                assert torch.equal(got[r].cpu(), want), (dim, r)


def test_mx4_all_gather_keeps_leading_dimensions_and_views(vrc):
    xs = workloads.random_ranks(4, (1, 5, 48, 72), "fp16", seed=9, device=DEV)
    codes, scales = vrc.vrc_mx4_quantize(xs)
    assert codes[0].shape == (1, 5, 48, 48) and scales[0].shape == (1, 5, 48, 3)
    own = vrc.vrc_mx4_dequantize(codes, scales, 72, dtype=torch.float16)
    assert own[0].shape == xs[0].shape
    assert torch.equal(vrc.vrc_mx4_all_gather(codes, scales, 72, dim=-1, dtype=torch.float16)[1], torch.cat(own, -1))
    out = [torch.zeros(4 * 5 * 48 * 72 + 8, dtype=torch.float16, device=DEV) for _ in range(4)]
    views = [o[r:r + 4 * 5 * 48 * 72] for r, o in enumerate(out)]
    vrc.vrc_mx4_all_gather(codes, scales, 72, dim=0, dtype=torch.float16, recv=[v.view(4, 5, 48, 72) for v in views])
    for r, v in enumerate(views):
        assert torch.equal(v.view(4, 5, 48, 72), torch.cat(own, 0))
        v.zero_()
        assert not out[r].any()
    # values read at an odd element: the quantiser's input need not sit on a vector's boundary
    flat = workloads.random_ranks(1, 64 * 33 + 8, "bf16", seed=3, device=DEV)[0]
    for off in (1, 2, 5):
        x = flat[off:off + 64 * 33].view(33, 64)
        a, b = vrc.vrc_mx4_quantize([x]), vrc.vrc_mx4_quantize([x.clone()])
        ta, tb = vrc.vrc_mx4_quantize([x], dim=0), vrc.vrc_mx4_quantize([x.clone()], dim=0)
        for u, v in zip(a + ta, b + tb):
            assert torch.equal(u[0], v[0])


def random_mx4(rows, k, seed, spread=4):
    """Random codes and scales, zero past column k."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    kb = -(-k // 32)
    c = torch.randint(0, 16, (rows, kb * 32), generator=g, device=DEV, dtype=torch.uint8)
    c[:, k:] = 0
    s = torch.randint(127 - spread, 128 + spread, (rows, kb), generator=g, device=DEV, dtype=torch.uint8)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous(), s


def product(ac, as_, bc, bs):
    """(sum over ranks, sum of magnitudes) of the decoded products, in 64 bits."""
    y = mag = 0
    for w, x, u, v in zip(ac, as_, bc, bs):
        a = ref.decode(w.cpu().numpy(), x.cpu().numpy())
        b = ref.decode(u.cpu().numpy(), v.cpu().numpy())
        y, mag = y + a @ b.T, mag + np.abs(a) @ np.abs(b).T
    return y, mag


def check_product(got, y, mag, k, dtype, what):
    tol = mag * k * 2.0**-24
    # rounding to nearest even overflows from the largest value and half its step on:
    # 65504 + 16 in fp16, which sums of these codes reach
    over = np.abs(y) + tol >= 65520.0 if dtype == "fp16" else None
    close(got, y, tol + ref.rounding(np.abs(y) + tol, dtype), what, over)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("m,nc,k", [(1, 1, 1), (1, 16, 32), (2, 40, 64), (3, 100, 2048), (16, 16, 96), (17, 33, 200), (31, 257, 500),
                                    (64, 64, 128), (65, 63, 1000), (100, 300, 333), (128, 130, 4100), (257, 255, 160), (300, 520, 1024),
                                    (500, 1, 2048), (1000, 20, 96), (300, 64, 70), (200, 3, 64), (3, 200, 64), (400, 1, 20), (80, 1100, 1536),
                                    (3000, 2, 300), (20, 700, 512), (700, 24, 90), (1, 9000, 96), (30, 9000, 96), (2, 3, 40)])
def test_mx4_matmul(vrc, dtype, m, nc, k):
    for n in (1, 3):
        say(f"mx4_matmul {dtype} n={n} m={m} n={nc} k={k}")
        a = [random_mx4(m, k, 10 + r) for r in range(n)]
        b = [random_mx4(nc, k, 50 + r) for r in range(n)]
        ops = [list(t) for t in zip(*a)] + [list(t) for t in zip(*b)]
        y, mag = product(*ops)
        for got in vrc.vrc_mx4_matmul(*ops, dtype=DT[dtype]):
            check_product(got, y, mag, n * k, dtype, "sum")
        for r, got in enumerate(vrc.vrc_mx4_matmul(*ops, dtype=DT[dtype], join="each")):
            check_product(got, *product(*[[t[r]] for t in ops]), k, dtype, f"each {r}")


@pytest.mark.parametrize("n", [2, 8, 16])
def test_mx4_matmul_many_ranks(vrc, n):
    for m, nc, k in ((1, 500, 512), (5, 96, 64), (40, 200, 96), (200, 200, 40)):
        say(f"mx4_matmul n={n} m={m} n={nc} k={k}")
        a, b = [random_mx4(m, k, r) for r in range(n)], [random_mx4(nc, k, 90 + r) for r in range(n)]
        ops = [list(t) for t in zip(*a)] + [list(t) for t in zip(*b)]
        y, mag = product(*ops)
        out = [torch.full((m * nc + 7,), 3.0, device=DEV) for _ in range(n)]
        views = [o[r % 4:r % 4 + m * nc].view(m, nc) for r, o in enumerate(out)]
        vrc.vrc_mx4_matmul(*ops, dtype=torch.float32, recv=views)
        for r in range(n):
            check_product(views[r], y, mag, n * k, "fp32", f"rank {r}")
            views[r].fill_(3.0)
            assert (out[r] == 3.0).all(), "written outside"


@pytest.mark.parametrize("join,n,m,nc,k", [("sum", 1, 4001, 4100, 200), ("sum", 2, 4096, 4096, 96), ("each", 4, 2050, 1999, 300),
                                           ("sum", 3, 4001, 4100, 512), ("sum", 1, 4090, 3900, 2560), ("sum", 2, 4096, 4096, 1024),
                                           ("each", 4, 2050, 1999, 2048), ("each", 5, 2000, 2048, 1536),
                                           ("sum", 1, 4001, 4100, 20), ("sum", 3, 3700, 4100, 520), ("each", 6, 2050, 1999, 777)])
def test_mx4_matmul_large_tiles(vrc, join, n, m, nc, k):
    """Enough work for the largest tiles, ragged and whole."""
    a, b = [random_mx4(m, k, r) for r in range(n)], [random_mx4(nc, k, 90 + r) for r in range(n)]
    ops = [list(t) for t in zip(*a)] + [list(t) for t in zip(*b)]
    for dtype in ("fp32", "bf16"):
        say(f"mx4_matmul {join} n={n} m={m} n={nc} k={k} {dtype}")
        got = vrc.vrc_mx4_matmul(*ops, dtype=DT[dtype], join=join)
        for r in range(n):
            y, mag = product(*[[t[r]] for t in ops]) if join == "each" else product(*ops)
            check_product(got[r], y, mag, k * (n if join == "sum" else 1), dtype, f"rank {r}")
            if join == "sum":
                assert all(torch.equal(got[0], g) for g in got)
                break


def test_mx4_matmul_special_scales(vrc):
    """A NaN scale reaches its row's or column's results and no others; scales far from
    one another meet in fp32's range; kblocks = 0 gives zeros."""
    for m, nc, k in ((1, 40, 96), (33, 70, 224), (130, 260, 512)):
        (ac, as_), (bc, bs) = random_mx4(m, k, 1), random_mx4(nc, k, 2)
        clean = vrc.vrc_mx4_matmul([ac], [as_], [bc], [bs], dtype=torch.float32)[0].clone()
        as_[m - 1, 1], bs[7, 2] = 255, 255
        y = vrc.vrc_mx4_matmul([ac], [as_], [bc], [bs], dtype=torch.float32)[0]
        bad = torch.zeros(m, nc, dtype=torch.bool, device=DEV)
        bad[m - 1, :], bad[:, 7] = True, True
        assert torch.equal(torch.isnan(y), bad) and torch.equal(y[~bad], clean[~bad])
        (ac, as_), (bc, bs) = random_mx4(m, k, 1, spread=2), random_mx4(nc, k, 2, spread=2)
        for sa, sb in ((100, -100), (-110, 110), (60, 50), (-70, -40)):
            a2, b2 = (as_.int() + sa).to(torch.uint8), (bs.int() + sb).to(torch.uint8)
            y, mag = product([ac], [a2], [bc], [b2])
            check_product(vrc.vrc_mx4_matmul([ac], [a2], [bc], [b2], dtype=torch.float32)[0], y, mag, k, "fp32", f"{sa} {sb}")
    # a NaN scale in the largest tiles, ragged and whole
    for k in (520, 1024):
        (ac, as_), (bc, bs) = random_mx4(3801, k, 1), random_mx4(3900, k, 2)
        clean = vrc.vrc_mx4_matmul([ac], [as_], [bc], [bs], dtype=torch.float32)[0].clone()
        as_[3800, 1], bs[7, 5] = 255, 255
        y = vrc.vrc_mx4_matmul([ac], [as_], [bc], [bs], dtype=torch.float32)[0]
        bad = torch.zeros_like(y, dtype=torch.bool)
        bad[3800, :], bad[:, 7] = True, True
        assert torch.equal(torch.isnan(y), bad) and torch.equal(y[~bad], clean[~bad])
    # the ends of the scales' range: sums of these are whole multiples of their smallest
    # product and below 2^24 of them, so fp32 holds them exactly while they are in its range
    for m, nc, k in ((1, 40, 96), (70, 130, 512), (300, 300, 90)):
        (ac, _), (bc, _) = random_mx4(m, k, 8), random_mx4(nc, k, 9)
        for ea, eb in ((252, 2), (2, 252), (0, 252), (254, 0), (0, 127), (64, 60), (0, 110), (0, 0)):
            sa = torch.full((m, -(-k // 32)), ea, dtype=torch.uint8, device=DEV)
            sb = torch.full((nc, -(-k // 32)), eb, dtype=torch.uint8, device=DEV)
            y, _ = product([ac], [sa], [bc], [sb])
            got = f64(vrc.vrc_mx4_matmul([ac], [sa], [bc], [sb], dtype=torch.float32)[0])
            assert (got == y.astype(np.float32)).all(), (ea, eb)
    none = torch.empty(5, 0, dtype=torch.uint8, device=DEV)
    assert not vrc.vrc_mx4_matmul([none], [none], [none[:3]], [none[:3]])[0].any()


def test_mx4_past_32_bits(vrc):
    """Codes, values and outputs beyond 2^32 bytes and elements."""
    rows, kb = (1 << 17) + 3, 1 << 11  # 4.3e9 bytes of codes
    codes = torch.zeros(rows, kb * 16, dtype=torch.uint8, device=DEV)
    scales = torch.full((rows, kb), 127, dtype=torch.uint8, device=DEV)
    b, bs = random_mx4(8, kb * 32, 4)
    some = [0, 1, (1 << 17) - 1, rows - 1]
    a_rows, s_rows = random_mx4(len(some), kb * 32, 5)
    codes[some], scales[some] = a_rows, s_rows
    y, mag = product([a_rows], [s_rows], [b], [bs])
    for got in (vrc.vrc_mx4_matmul([codes], [scales], [b], [bs], dtype=torch.float32)[0][some],
                vrc.vrc_mx4_matmul([b], [bs], [codes], [scales], dtype=torch.float32)[0].t()[some]):
        check_product(got, y, mag, kb * 32, "fp32", "product")
    x = vrc.vrc_mx4_dequantize([codes], [scales], dtype=torch.bfloat16)[0]
    for i, r in enumerate(some):
        assert torch.equal(x[r].double().cpu(), torch.from_numpy(ref.decode(a_rows[i:i + 1].cpu().numpy(), s_rows[i:i + 1].cpu().numpy())[0]))
    again, again_s = vrc.vrc_mx4_quantize([x])
    back = vrc.vrc_mx4_dequantize(again, again_s, dtype=torch.bfloat16)[0]
    assert torch.equal(back[some], vrc.vrc_mx4_dequantize(*vrc.vrc_mx4_quantize([x[some]]), dtype=torch.bfloat16)[0])
    del again, again_s, back
    tcodes, tscales = vrc.vrc_mx4_quantize([x], dim=0)
    last = rows - 3  # the last block's three rows
    want, want_s = ref.quantise(f64(x[last:]).T[-64:])
    assert (ref.unpack(tcodes[0][-64:, -16:].cpu().numpy()) == want).all() and (tscales[0][-64:, -1:].cpu().numpy() == want_s).all()


def test_mx4_more_workgroups_than_a_grid_axis_holds(vrc):
    """2^32 work items along one axis of a grid: thin matrices reach them first."""
    rows = (1 << 32) + 300
    x = torch.empty(rows, dtype=torch.bfloat16, device=DEV)
    x[: 1 << 31].normal_()
    x[1 << 31:].normal_()
    down = vrc.vrc_mx4_quantize([x.view(rows, 1)], dim=0)
    along = vrc.vrc_mx4_quantize([x.view(1, rows)])
    assert torch.equal(down[0][0].view(-1), along[0][0].view(-1))
    assert torch.equal(down[1][0].view(-1), along[1][0].view(-1))
    del x, down, along
    # one row by 2^27 + 5: a period of B's rows is one of the product
    period, rows = 1 << 20, (1 << 27) + 5
    (ac, as_), (bc, bs) = random_mx4(1, 32, 41), random_mx4(period, 32, 42)
    times = -(-rows // period)
    wide = [t.repeat(times, 1)[:rows].contiguous() for t in (bc, bs)]
    y = torch.full((1, rows), -1.0, dtype=torch.float32, device=DEV)
    vrc.vrc_mx4_matmul([ac], [as_], [wide[0]], [wide[1]], recv=[y], dtype=torch.float32)
    one = vrc.vrc_mx4_matmul([ac], [as_], [bc], [bs], dtype=torch.float32)[0]
    assert torch.equal(y, one.repeat(1, times)[:, :rows])
    yt = torch.full((rows, 1), -1.0, dtype=torch.float32, device=DEV)
    vrc.vrc_mx4_matmul([wide[0]], [wide[1]], [ac], [as_], recv=[yt], dtype=torch.float32)
    assert torch.equal(yt.view(-1), y.view(-1))
    del wide, y, yt
    # nothing to contract: zeros, however many of them
    none = [torch.empty(70000, k, dtype=torch.uint8, device=DEV) for k in (0, 0)]
    z = torch.full((70000, 70000), -1.0, dtype=torch.bfloat16, device=DEV)
    vrc.vrc_mx4_matmul([none[0]], [none[1]], [none[0]], [none[1]], recv=[z])
    assert not z.view(torch.int16).any()


# ---------------------------------------------------------------------------
# As they are used
# ---------------------------------------------------------------------------
def layer(vrc, xs, ws, res, p, seed, dys, buf=None, offset=0):
    """One row-parallel layer in four bits with dropout and a residual, forward and
    backward (straight through the quantiser): y, dx and dw of every rank."""
    n = len(xs)
    xq, wq = vrc.vrc_mx4_quantize(xs), vrc.vrc_mx4_quantize(ws)
    parts = vrc.vrc_mx4_matmul(*xq, *wq, dtype=torch.float32, join="each")
    y = vrc.vrc_reduce_scatter_dropout(parts, p, seed, offset, residual=res, dim=1)
    g = vrc.vrc_all_gather_dropout(dys, p, seed, offset, dim=1)
    gq, gt = vrc.vrc_mx4_quantize(g), vrc.vrc_mx4_quantize(g, dim=0)
    wt, xt = vrc.vrc_mx4_quantize(ws, dim=0), vrc.vrc_mx4_quantize(xs, dim=0)
    dx = vrc.vrc_mx4_matmul(*gq, *wt, dtype=torch.float32, join="each")
    dw = vrc.vrc_mx4_matmul(*gt, *xt, dtype=torch.float32, join="each")
    return list(y) + list(dx) + list(dw)


def layer_inputs(n=4, tokens=96, k=160, out=64):
    xs = workloads.random_ranks(n, (tokens, k), "bf16", seed=70, device=DEV)
    ws = workloads.random_ranks(n, (out, k), "bf16", seed=71, device=DEV, sigma=0.1)
    res = workloads.random_ranks(n, (tokens, out // n), "fp32", seed=72, device=DEV)
    dys = workloads.random_ranks(n, (tokens, out // n), "fp32", seed=73, device=DEV)
    return xs, ws, res, dys


def test_row_parallel_layer_forward_and_backward(vrc):
    n, p, seed = 4, 0.2, 99
    xs, ws, res, dys = layer_inputs()
    got = layer(vrc, xs, ws, res, p, seed, dys)

    def q(t, axis=0):
        v = f64(t).T if axis else f64(t)
        c, s = ref.quantise(v)
        return ref.decode(ref.pack(c), s)[:, :v.shape[1]]

    full = sum(q(x) @ q(w).T for x, w in zip(xs, ws))
    mag = sum(np.abs(q(x)) @ np.abs(q(w)).T for x, w in zip(xs, ws))
    keep = ref.keep(0, full.size, p, seed, 0).reshape(full.shape) / (1 - p)
    w = full.shape[1] // n
    for c in range(n):
        cols = slice(c * w, (c + 1) * w)
        r = f64(res[c])
        want = r + (keep * full)[:, cols]
        tol = (keep * mag)[:, cols] * (160 * n + n + 2) * 2.0**-24 + (np.abs(r) + np.abs(want)) * 2.0**-23
        close(got[c], want, tol, f"y {c}")
    # the gradient that reaches the products is fp32: quantise the same rounded values
    scale = np.float32(1 / (1 - p))
    g32 = np.concatenate([d.cpu().numpy() for d in dys], axis=1) * scale * (keep > 0)
    g = torch.from_numpy(g32.astype(np.float32))
    for r in range(n):
        for name, a, b, k, out in (("dx", q(g), q(ws[r], 1), 64, got[n + r]), ("dw", q(g, 1), q(xs[r], 1), 96, got[2 * n + r])):
            tol = np.abs(a) @ np.abs(b).T * k * 2.0**-24
            close(out, a @ b.T, tol + np.abs(a @ b.T) * 2.0**-24, f"{name} {r}")


def test_captured_layer_replays_with_new_masks(vrc):
    """The whole layer in a graph, its mask's offset in device memory: every replay
    equals the eager result of that offset, with eager work between the replays."""
    n, p, seed = 4, 0.5, 5
    xs, ws, res, dys = layer_inputs()
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        layer(vrc, xs, ws, res, p, seed, dys, offset=step)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = layer(vrc, xs, ws, res, p, seed, dys, offset=step)
    graph2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph2):
        outs2 = layer(vrc, xs, ws, res, p, seed + 1, dys, offset=step)
    for k in (0, 1, 2, (1 << 40) + 3, -1):
        step.fill_(k)
        xs[0].mul_(1.01)
        graph.replay()
        graph2.replay()
        for s, o in ((seed, outs), (seed + 1, outs2)):
            want = layer(vrc, xs, ws, res, p, s, dys, offset=k % (1 << 64))
            torch.cuda.synchronize()
            for u, v in zip(o, want):
                assert torch.equal(u, v), k


def test_streams_and_repeats(vrc):
    """Calls on two streams at once, on a stream that is not the current one, and again:
    the same bits each time."""
    xs, ws, res, dys = layer_inputs(tokens=300)
    want = layer(vrc, xs, ws, res, 0.1, 1, dys)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(layer(vrc, xs, ws, res, 0.1, 1, dys))
    torch.cuda.synchronize()
    for g in got:
        for u, v in zip(g, want):
            assert torch.equal(u, v)
    s = streams[0]
    q = vrc.vrc_mx4_quantize(xs, stream=s)
    y = vrc.vrc_mx4_matmul(*q, *vrc.vrc_mx4_quantize(ws, stream=s), join="each", stream=s)
    z = vrc.vrc_allreduce_dropout(y, 0.3, 4, 5, stream=s)
    s.synchronize()
    want = vrc.vrc_allreduce_dropout(vrc.vrc_mx4_matmul(*vrc.vrc_mx4_quantize(xs), *vrc.vrc_mx4_quantize(ws), join="each"), 0.3, 4, 5)
    torch.cuda.synchronize()
    for u, v in zip(z, want):
        assert torch.equal(u, v)


def test_binding_refusals_on_the_device(vrc):
    x = [torch.zeros(8, 64, dtype=torch.float16, device=DEV) for _ in range(2)]
    codes, scales = vrc.vrc_mx4_quantize(x)
    y = [torch.empty_like(t) for t in x]
    bad = [
        lambda: vrc.vrc_allreduce_dropout([x[0], x[1][:4]], 0.1, 1),
        lambda: vrc.vrc_allreduce_dropout([t.t() for t in x], 0.1, 1),
        lambda: vrc.vrc_allreduce_dropout(x, 0.1, 1, residual=[x[0]]),
        lambda: vrc.vrc_allreduce_dropout(x, 0.1, 1, residual=x[0].float()),
        lambda: vrc.vrc_allreduce_dropout(x, 0.1, 1, residual=x[0].cpu()),
        lambda: vrc.vrc_allreduce_dropout(x, 0.1, 1, recv=y[:1]),
        lambda: vrc.vrc_allreduce_dropout(x, 0.1, 1, recv=[t.float() for t in y]),
        lambda: vrc.vrc_allreduce_dropout(x, 0.1, 1, torch.zeros(1, dtype=torch.int64)),
        lambda: vrc.vrc_reduce_scatter_dropout([t[:, :63].contiguous() for t in x], 0.1, 1, dim=1),
        lambda: vrc.vrc_reduce_scatter_dropout(x, 0.1, 1, residual=x),
        lambda: vrc.vrc_mx4_quantize(x, dim=1, codes=codes, scales=codes),
        lambda: vrc.vrc_mx4_quantize([t.view(2, 4, 64) for t in x], dim=0),
        lambda: vrc.vrc_mx4_dequantize(codes, scales[:1]),
        lambda: vrc.vrc_mx4_dequantize(codes, scales, 65),
        lambda: vrc.vrc_mx4_dequantize(codes, scales, 32),
        lambda: vrc.vrc_mx4_dequantize(scales, scales),
        lambda: vrc.vrc_mx4_all_gather([c.view(2, 4, 32) for c in codes], [s.view(2, 4, 2) for s in scales], dim=1),
        lambda: vrc.vrc_mx4_matmul(codes, scales, codes[:1], scales[:1]),
        lambda: vrc.vrc_mx4_matmul(codes, scales, [c[:, :16].contiguous() for c in codes], [s[:, :1].contiguous() for s in scales]),
    ]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            say(f"not refused: {k}")
    for call in (lambda: vrc.vrc_allreduce_dropout([t.int() for t in x], 0.1, 1), lambda: vrc.vrc_mx4_quantize(codes),
                 lambda: vrc.vrc_mx4_dequantize(x, x)):
        with pytest.raises(TypeError):
            call()
    for p in (-1.0, 2.0, float("nan")):
        with pytest.raises(vrc.VrcError):
            vrc.vrc_allreduce_dropout(x, p, 1)
    with pytest.raises(vrc.VrcError):
        vrc.vrc_allreduce_dropout(x, 0.1, 1, residual=x[0], recv=[x[0], y[1]])
