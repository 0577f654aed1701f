"""The model's operators as programs use them: in place, guarded buffers, masked and bad
values, pieces of a vocabulary, past 32 bits, streams, graphs, and run together.
Tolerances are those of tests/model_reference.py."""
import pytest
import torch

from tests import model_reference as ref
from tests.test_gpu_model import (DEV, DT, IGNORE, JOINS, check_entropy, check_entropy_grad, close, entropy_inputs, gen, listed,
                                  norm_inputs, say, shared, vrc)  # noqa: F401  (vrc: the fixture)

pytestmark = pytest.mark.gpu


def equal(a, b):
    """The same bits, NaN included."""
    view = {4: torch.int32, 2: torch.int16}[a.element_size()]
    return a.shape == b.shape and a.dtype == b.dtype and torch.equal(a.contiguous().view(view), b.contiguous().view(view))


def flat(out):
    """Every tensor of a call's answer, in order."""
    if isinstance(out, torch.Tensor):
        return [out]
    return [] if out is None else [t for x in out for t in flat(x)]


def same(a, b, what=""):
    a, b = flat(a), flat(b)
    assert len(a) == len(b) and all(equal(x, y) for x, y in zip(a, b)), what


class Guarded:
    """Tensors inside allocations whose other elements must stay as they are."""

    def __init__(self):
        self.all = []

    def new(self, shape, dtype, before=5, after=67):
        count = 1
        for k in shape:
            count *= k
        whole = torch.full((before + count + after,), 7.0, dtype=dtype, device=DEV)
        self.all.append((whole, before, count))
        return whole[before:before + count].view(shape)

    def check(self):
        for whole, before, count in self.all:
            assert (whole[:before] == 7).all() and (whole[before + count:] == 7).all()


# ---------------------------------------------------------------------------
# Buffers
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("width", [24, 1001, 16392, 33000])
def test_layer_norm_in_place(vrc, dtype, width):
    for join in ("each", "sum"):
        x, res, w, b = norm_inputs(join, 3, 5, width, DT[dtype], 11)
        y, h, mean, rstd = vrc.vrc_layer_norm(x, w, b, residual=shared(res, join), join=join)
        x2, res2 = [t.clone() for t in x], [t.clone() for t in res]
        y2, h2, mean2, rstd2 = vrc.vrc_layer_norm(x2, w, b, residual=shared(res2, join), join=join, recv=x2, sum=shared(res2, join))
        assert y2 is x2 and (h2 is res2 or h2 is res2[0])
        same([y, h, mean, rstd], [y2, h2, mean2, rstd2], (join, width))
        dx, dw, db = vrc.vrc_layer_norm_grad(x, h, w, mean, rstd, dh=shared(res, join), join=join)
        x3 = [t.clone() for t in x]
        dx3, dw3, db3 = vrc.vrc_layer_norm_grad(x3, h, w, mean, rstd, dh=shared(res, join), join=join, recv=x3)
        assert dx3 is x3
        same([dx, dw, db], [dx3, dw3, db3], (join, width))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("join", JOINS)
def test_layer_norm_writes_nothing_else(vrc, dtype, join):
    for rows, width in ((1, 3), (7, 1053), (3, 20001), (530, 130)):
        x, res, w, b = norm_inputs(join, 3, rows, width, DT[dtype], 12)
        want = vrc.vrc_layer_norm(x, w, b, residual=shared(res, join), join=join)
        g = Guarded()
        recv = [g.new(t.shape, t.dtype) for t in want[0]]
        into = [g.new(t.shape, t.dtype) for t in listed(want[1])]
        same(want, vrc.vrc_layer_norm(x, w, b, residual=shared(res, join), join=join, recv=recv, sum=shared(into, join)))
        _, h, mean, rstd = want
        grads = vrc.vrc_layer_norm_grad(x, h, w, mean, rstd, join=join)
        dx = [g.new(t.shape, t.dtype) for t in grads[0]]
        same(grads, vrc.vrc_layer_norm_grad(x, h, w, mean, rstd, join=join, recv=dx))
        torch.cuda.synchronize()
        g.check()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("tokens,vocab,width", [(1, [3], 5), (20, [70, 0, 300], 129), (40, [130], 72), (100, [257, 1], 200), (300, [500, 13], 1053)])
def test_cross_entropy_grad_writes_nothing_else(vrc, dtype, tokens, vocab, width):
    hidden, weight, target = entropy_inputs(tokens, vocab, width, DT[dtype], 13)
    loss, lse = vrc.vrc_cross_entropy(hidden, weight, target)
    dloss = torch.ones_like(loss)
    want = vrc.vrc_cross_entropy_grad(hidden, weight, target, lse, dloss)
    g = Guarded()
    recv = (g.new(hidden.shape, hidden.dtype), [g.new(w.shape, w.dtype) for w in weight])
    got = vrc.vrc_cross_entropy_grad(hidden, weight, target, lse, dloss, recv=recv)
    assert got[0] is recv[0] and got[1] is recv[1]
    same(want, got)
    torch.cuda.synchronize()
    g.check()


def test_empty_calls(vrc):
    f = gen(1)
    w = f(16)
    for join in JOINS:
        y, h, mean, rstd = vrc.vrc_layer_norm([f(0, 16)] * 2, w, join=join)
        assert all(t.shape == (0, 16) for t in y)
        dx, dw, db = vrc.vrc_layer_norm_grad([f(0, 16)] * 2, h, w, mean, rstd, join=join)
        assert not dw.any() and not db.any() and dw.shape == (16,)
    loss, lse = vrc.vrc_cross_entropy(f(0, 16), [f(5, 16)], torch.zeros(0, dtype=torch.int64, device=DEV))
    assert loss.shape == lse.shape == (0,)
    for dtype in DT.values():
        dh, dw = vrc.vrc_cross_entropy_grad(f(0, 16).to(dtype), [f(5, 16).to(dtype), f(300, 16).to(dtype)],
                                            torch.zeros(0, dtype=torch.int64, device=DEV), lse, loss)
        assert dh.shape == (0, 16) and not any(t.any() for t in dw)
    t = torch.zeros(3, dtype=torch.int64, device=DEV)
    loss, lse = vrc.vrc_cross_entropy(f(3, 16), [f(0, 16)] * 2, t)
    assert (lse == float("-inf")).all() and torch.isnan(loss).all()
    dh, dw = vrc.vrc_cross_entropy_grad(f(3, 16), [f(0, 16)] * 2, t, lse, torch.ones(3, device=DEV))
    assert not dh.any() and all(d.shape == (0, 16) for d in dw)


def test_one_row_and_one_token_without_leading_dimensions(vrc):
    f = gen(2)
    x, w, b = f(100), f(100), f(100)
    y, h, mean, rstd = vrc.vrc_layer_norm([x, x], w, b, join="sum")
    assert y[0].shape == h.shape == (100,) and mean.shape == rstd.shape == ()
    want = ref.layer_norm([x, x], None, w, b, 1e-5, True)
    close(y[1], want[0], "y")
    dx, dw, db = vrc.vrc_layer_norm_grad([x, x], h, w, mean, rstd, join="sum")
    assert dx[0].shape == dw.shape == db.shape == (100,)
    t = torch.tensor(3, device=DEV)
    loss, lse = vrc.vrc_cross_entropy(x, [f(7, 100)], t)
    assert loss.shape == lse.shape == ()
    dh, _ = vrc.vrc_cross_entropy_grad(x, [f(7, 100)], t, lse, torch.ones_like(loss))
    assert dh.shape == (100,)
    loss3, lse3 = vrc.vrc_cross_entropy(f(2, 3, 100), [f(7, 100)], torch.zeros(2, 3, dtype=torch.int64, device=DEV))
    assert loss3.shape == lse3.shape == (2, 3)


def test_rows_that_y_overwrites_are_not_returned_as_h(vrc):
    """Without a residual each rank's rows are h; in place they are gone."""
    x, _, w, b = norm_inputs("each", 2, 4, 64, torch.float32, 14)
    want = vrc.vrc_layer_norm(x, w, b)
    assert want[1] is x
    rows = [t.clone() for t in x]
    y, h, mean, rstd = vrc.vrc_layer_norm(rows, w, b, recv=rows)
    assert y is rows and h is None
    same([want[0], want[2], want[3]], [y, mean, rstd])
    assert vrc.vrc_layer_norm(x, w, b, recv=[torch.empty_like(t) for t in x])[1] is x


# ---------------------------------------------------------------------------
# Values
# ---------------------------------------------------------------------------
def test_layer_norm_far_from_zero(vrc):
    """The variance of rows whose mean is 10^4 times their spread: by sums of squares fp32
    would lose all of it."""
    x, _, w, b = norm_inputs("each", 1, 9, 4096, torch.float32, 21)
    x = [t + 1e4 for t in x]
    y, _, mean, rstd = vrc.vrc_layer_norm(x, w, b)
    ry, _, rm, rr = ref.layer_norm(x, None, w, b, 1e-5, True)
    close(y[0], ry, "y")
    close(mean[0], rm, "mean")
    close(rstd[0], rr, "rstd")
    assert ((rstd[0].double() - rr[0]).abs() < 1e-2 * rr[0]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("join,n", [("each", 2), ("sum", 2)])
@pytest.mark.parametrize("width", [2, 4, 64])
def test_layer_norm_grad_of_constant_rows_far_from_zero(vrc, width, join, n, dtype):
    """h = 2^100 everywhere and rstd = 2^33: what lanes without a value compute in place of x,
    (0 - mean) rstd, would be infinite, and NaN times their gradient of zero."""
    f = gen(22)
    x = [torch.full((3, width), 2.0**(100 if join == "each" else 99), dtype=dtype, device=DEV) for _ in range(n)]
    w, dy = f(width).to(dtype), [f(3, width).to(dtype) for _ in range(n)]
    y, h, mean, rstd = vrc.vrc_layer_norm(x, w, eps=2.0**-66, join=join)
    assert all((t == 0).all() for t in y)
    dx, dw, db = vrc.vrc_layer_norm_grad(dy, h, w, mean, rstd, join=join)
    db_want, db_bound = 0, 0
    for p, (hp, m, r) in enumerate(zip(listed(h), listed(mean), listed(rstd))):
        assert (hp == 2.0**100).all() and (m == 2.0**100).all() and (r == 2.0**33).all()
        rx, _, rb = ref.layer_norm_grad(dy if join == "sum" else [dy[p]], hp, w, m, r, None)
        for q in range(n) if join == "sum" else [p]:
            close(dx[q], rx, "dx")
        db_want, db_bound = db_want + rb[0], db_bound + rb[1]
    assert (dw == 0).all()
    close(db, (db_want, db_bound), "dbias")


@pytest.mark.parametrize("dtype", DT)
def test_layer_norm_bad_rows_stay_alone(vrc, dtype):
    for width in (40, 1053, 9000, 40000):
        for center in (True, False):
            x, res, w, b = norm_inputs("sum", 2, 6, width, DT[dtype], 22)
            good = vrc.vrc_layer_norm(x, w, b, residual=res[0], join="sum", center=center)
            x[1][1, width - 1] = float("inf")
            x[0][3, 0] = float("nan")
            y, h, mean, rstd = vrc.vrc_layer_norm(x, w, b, residual=res[0], join="sum", center=center)
            keep = [0, 2, 4, 5]
            same([y[0][keep], y[1][keep], h[keep], rstd[keep]], [good[0][0][keep], good[0][1][keep], good[1][keep], good[3][keep]])
            assert torch.isnan(y[0][3]).all() and torch.isnan(y[0][1]).any() and h[1, width - 1] == float("inf")
            dx, dw, _ = vrc.vrc_layer_norm_grad(x, h, w, mean, rstd, join="sum")
            clean = vrc.vrc_layer_norm_grad(x, good[1], w, good[2], good[3], join="sum")
            same(dx[0][keep], clean[0][0][keep])
            assert torch.isnan(dx[0][3]).all() and torch.isnan(dw).any()
    constant = [torch.full((2, 64), 3.0, dtype=DT[dtype], device=DEV)]
    w = torch.ones(64, dtype=DT[dtype], device=DEV)
    assert not vrc.vrc_layer_norm(constant, w)[0][0].any()
    assert torch.isnan(vrc.vrc_layer_norm(constant, w, eps=0.0)[0][0]).all()  # 0 / 0


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("tokens", [20, 100, 300])
def test_masked_tokens_reach_nothing(vrc, dtype, tokens):
    """What tokens without gradient hold: infinities, NaN, any lse."""
    hidden, weight, target = entropy_inputs(tokens, [300, 77], 192, DT[dtype], 31, ignored=0.4)
    loss, lse = vrc.vrc_cross_entropy(hidden, weight, target)
    dloss = torch.rand(tokens, device=DEV) + 0.1
    dloss[::7] = 0  # weighted with zero
    gone = (target == IGNORE) | (dloss == 0)
    want = vrc.vrc_cross_entropy_grad(hidden, weight, target, lse, dloss)
    bad, bad_lse = hidden.clone(), lse.clone()
    bad[gone] = float("nan")
    bad[gone, 1] = float("inf")
    bad_lse[gone] = float("nan")
    bad_lse[torch.nonzero(gone)[0]] = float("-inf")
    got = vrc.vrc_cross_entropy_grad(bad, weight, target, bad_lse, dloss)
    same(want, got)
    assert not got[0][gone].any()
    loss2, lse2 = vrc.vrc_cross_entropy(bad, weight, target)
    kept = target != IGNORE
    assert (loss2[~kept] == 0).all()
    same(loss2[~gone], loss[~gone])
    # dloss of an ignored token does not count
    dloss2 = torch.where(kept, dloss, torch.full_like(dloss, float("nan")))
    same(want, vrc.vrc_cross_entropy_grad(bad, weight, target, bad_lse, dloss2))
    # none left
    dh, dw = vrc.vrc_cross_entropy_grad(bad, weight, torch.full_like(target, IGNORE), bad_lse, dloss2)
    assert not dh.any() and not any(t.any() for t in dw)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("tokens", [5, 70, 200])
def test_targets_outside_the_vocabulary(vrc, dtype, tokens):
    hidden, weight, target = entropy_inputs(tokens, [130, 60], 64, DT[dtype], 32, ignored=0.0)
    loss, lse = vrc.vrc_cross_entropy(hidden, weight, target, ignore_index=0)
    assert (loss[target == 0] == 0).all()  # one within it may be the ignored one
    bad = target.clone()
    bad[0], bad[1], bad[2] = 190, -1, 1 << 40
    loss2, lse2 = vrc.vrc_cross_entropy(hidden, weight, bad, ignore_index=0)
    same([loss2[3:], lse2], [loss[3:], lse])
    assert torch.isnan(loss2[:3]).all()
    dloss = torch.ones_like(loss)
    want, _ = vrc.vrc_cross_entropy_grad(hidden, weight, target, lse, dloss, ignore_index=0)
    dh, dw = vrc.vrc_cross_entropy_grad(hidden, weight, bad, lse, dloss, ignore_index=0)
    same(dh[3:], want[3:])
    assert torch.isnan(dh[:3]).all() and all(torch.isnan(t).all() for t in dw)


def test_infinite_logits(vrc):
    """As torch's logsumexp has them: a row with +infinity is infinite, one with -infinity
    goes on without that element, NaN stays NaN."""
    hidden = torch.zeros(40, 8, device=DEV)
    hidden[:, 0] = 1.0
    weight = [torch.zeros(300, 8, device=DEV), torch.zeros(5, 8, device=DEV)]
    weight[0][:, 0] = torch.linspace(-3, 3, 300, device=DEV)
    hidden[1, 1], hidden[2, 2], hidden[3, 3], hidden[4, 0] = 1e30, 1e30, float("nan"), -2000.0
    weight[0][7, 1], weight[1][2, 1] = 1e30, -1e30   # token 1: +inf and -inf logits
    weight[0][150, 2] = -1e30                        # token 2: one -inf
    target = torch.full((40,), 9, dtype=torch.int64, device=DEV)
    target[2] = 150
    loss, lse = vrc.vrc_cross_entropy(hidden, weight, target)
    z = hidden @ torch.cat(weight).t()
    want = torch.logsumexp(z, 1)
    assert lse[1] == float("inf") and loss[1] == float("inf") and loss[2] == float("inf") and torch.isnan(lse[3])
    fine = [i for i in range(40) if i not in (1, 3)]
    assert torch.allclose(lse[fine], want[fine], rtol=1e-5)
    every = [torch.full((3, 8), float("-inf"), device=DEV)]
    assert (vrc.vrc_cross_entropy(torch.ones(2, 8, device=DEV), every)[1] == float("-inf")).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1.0, 60000.0])
def test_gradients_of_any_scale(vrc, dtype, scale):
    """The gradients of the logits are held in units of the largest, so that their scale
    does not matter (that of the results' type does)."""
    if dtype == "bf16" or scale >= 1.0:
        check_entropy_grad(vrc, 200, [300, 40], 64, DT[dtype], scale=scale)
        check_entropy_grad(vrc, 30, [300, 40], 64, DT[dtype], scale=scale)
    else:
        check_entropy_grad(vrc, 200, [300, 40], 64, DT[dtype], scale=scale, weighted=False)


# ---------------------------------------------------------------------------
# Sizes
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", DT)
def test_pieces_of_the_vocabulary(vrc, dtype):
    """More columns than one piece of the logits' gradients holds, cut inside a rank."""
    check_entropy_grad(vrc, 8192, [9000, 1, 5003], 40, DT[dtype])
    check_entropy_grad(vrc, 8192, [4097, 4500], 33, DT[dtype], weighted=False)


@pytest.mark.parametrize("dtype", DT)
def test_more_tokens_than_one_pass(vrc, dtype):
    check_entropy(vrc, 16384 + 300, [700, 55], 24, DT[dtype])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("tokens,vocab,width", [(1, [20000], 512), (40, [9001, 9000], 256), (200, [5000], 1024), (300, [2000, 2100], 777), (1500, [1500], 640)])
def test_larger_products(vrc, dtype, tokens, vocab, width):
    say(f"{dtype} {tokens} {vocab} {width}")
    check_entropy(vrc, tokens, vocab, width, DT[dtype])
    check_entropy_grad(vrc, tokens, vocab, width, DT[dtype])


@pytest.mark.parametrize("tokens,vocab,width", [(65, [33, 1, 95], 36), (129, [31] * 16, 52), (315, [274] * 6 + [271], 180),
                                                (513, [4100], 200), (640, [4096], 128), (1024, [2048], 33), (257, [120, 5, 129], 1030)])
def test_fp32_products_of_each_tile(vrc, tokens, vocab, width):
    """Few and many tiles for the CUs, of every side, with ends in each."""
    say(f"{tokens} {vocab} {width}")
    check_entropy(vrc, tokens, vocab, width, torch.float32)
    check_entropy_grad(vrc, tokens, vocab, width, torch.float32)


def test_layer_norm_past_32_bits(vrc):
    rows, width = (1 << 20) + 3, 4104  # 8.6 GB a tensor
    x = [torch.empty(rows, width, dtype=torch.bfloat16, device=DEV).normal_()]
    w = torch.ones(width, dtype=torch.bfloat16, device=DEV)
    y, h, mean, rstd = vrc.vrc_layer_norm(x, w)
    pick = [0, 1, 523264, 523265, rows - 2, rows - 1]
    ry, _, rm, rr = ref.layer_norm([x[0][pick]], None, w, None, 1e-5, True)
    close(y[0][pick], ry, "y")
    close(mean[0][pick], rm, "mean")
    dx, dw, db = vrc.vrc_layer_norm_grad(x, x, w, mean, rstd, recv=y)
    (d, e), _, _ = ref.layer_norm_grad([x[0][pick]], x[0][pick], w, mean[0][pick], rstd[0][pick], None)
    close(dx[0][pick], (d, e), "dx")


def test_cross_entropy_past_32_bits(vrc):
    vocab, width, tokens = 140001, 16384, 3  # 4.6 GB of weights
    hidden, weight, target = entropy_inputs(tokens, [5, vocab], width, torch.bfloat16, 41, ignored=0.0)
    target[0] = vocab + 4
    loss, lse = vrc.vrc_cross_entropy(hidden, weight, target)
    dh, dw = vrc.vrc_cross_entropy_grad(hidden, weight, target, lse, torch.ones_like(loss))
    z = torch.cat([hidden.float() @ w[i:i + 20000].float().t() for w in weight for i in range(0, w.shape[0], 20000)], 1).double()
    assert torch.allclose(lse.double(), torch.logsumexp(z, 1), rtol=1e-5)
    assert torch.allclose(loss.double(), torch.logsumexp(z, 1) - z.gather(1, target[:, None])[:, 0], rtol=1e-5, atol=1e-4)
    pick = torch.tensor([0, 1, 131072, 131073, vocab - 2, vocab - 1], device=DEV)
    g = (z - lse.double()[:, None]).exp()
    g[torch.arange(tokens, device=DEV), target] -= 1
    want = g[:, 5 + pick].t() @ hidden.double()
    # fp32 logits of 16384 products (2^-10 of their largest), the rounding to bf16, and near p = 1 the difference from it
    assert ((dw[1][pick].double() - want).abs() <= 2.0**-7 * want.abs() + 2.0**-9 * want.abs().amax(1, keepdim=True)).all()


# ---------------------------------------------------------------------------
# Streams, graphs, the same call again
# ---------------------------------------------------------------------------
def passes(vrc, d):
    """One pass of everything over the inputs of `inputs`."""
    out = []
    for join in JOINS:
        y, h, mean, rstd = vrc.vrc_layer_norm(d["x"], d["w"], d["b"], residual=shared(d["res"][join], join), join=join)
        out += [y, h, mean, rstd, vrc.vrc_layer_norm_grad(d["x"], h, d["w"], mean, rstd, join=join)]
    for hidden, target in ((d["few"], d["target"][:20]), (d["many"], d["target"])):
        loss, lse = vrc.vrc_cross_entropy(hidden, d["weight"], target)
        out += [loss, lse, vrc.vrc_cross_entropy_grad(hidden, d["weight"], target, lse, d["dloss"][:hidden.shape[0]], dlse=loss)]
    return out


def inputs(seed, dtype=torch.bfloat16):
    f = gen(seed)
    d = {"x": [f(50, 264).to(dtype) for _ in range(3)], "w": f(264), "b": f(264), "res": {}}
    for join in JOINS:
        rows = [50] if join == "sum" else [50] * 3 if join == "each" else [16, 16, 18]
        d["res"][join] = [f(r, 264).to(dtype) for r in rows]
    d["many"], d["weight"], d["target"] = entropy_inputs(300, [1000, 0, 333], 192, dtype, seed + 1)
    d["few"], d["dloss"] = d["many"][:20].clone(), f(300)
    return d


def test_equal_calls_give_equal_bits(vrc):
    d = inputs(51)
    first = passes(vrc, d)
    for _ in range(4):
        junk = [torch.full((1 << 22,), float("nan"), device=DEV) for _ in range(3)]  # what workspaces may find
        del junk
        same(first, passes(vrc, d))


def test_streams(vrc):
    """Calls on two streams at once, each on data that it makes itself; and a stream given by name."""
    da, db = inputs(61), inputs(62, torch.float16)
    want = [passes(vrc, da), passes(vrc, db)]
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    got = [None, None]
    for _ in range(5):
        for i, (s, d) in enumerate(((sa, da), (sb, db))):
            with torch.cuda.stream(s):
                got[i] = passes(vrc, d)
    torch.cuda.synchronize()
    same(want, got)
    y = vrc.vrc_layer_norm(da["x"], da["w"], da["b"], join="sum", stream=sa)
    g = vrc.vrc_layer_norm_grad(da["x"], y[1], da["w"], y[2], y[3], join="sum", stream=sa)
    l = vrc.vrc_cross_entropy(da["few"], da["weight"], da["target"][:20], stream=sa)
    e = vrc.vrc_cross_entropy_grad(da["few"], da["weight"], da["target"][:20], l[1], da["dloss"][:20], stream=sa)
    sa.synchronize()
    y2 = vrc.vrc_layer_norm(da["x"], da["w"], da["b"], join="sum")
    l2 = vrc.vrc_cross_entropy(da["few"], da["weight"], da["target"][:20])
    same([y, g, l, e], [y2, vrc.vrc_layer_norm_grad(da["x"], y2[1], da["w"], y2[2], y2[3], join="sum"), l2,
                        vrc.vrc_cross_entropy_grad(da["few"], da["weight"], da["target"][:20], l2[1], da["dloss"][:20])])


def test_captured_and_replayed(vrc):
    """Two graphs, each with workspaces of its own, replayed on new inputs between eager calls."""
    static = [inputs(71), inputs(72)]
    for d in static:
        passes(vrc, d)
    torch.cuda.synchronize()
    graphs = []
    for d in static:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = passes(vrc, d)
        graphs.append((g, out, d))

    def copy(into, of):
        for a, b in zip(into, of):
            a.copy_(b)

    for turn in range(4):
        for k, (g, out, d) in enumerate(graphs):
            new = inputs(80 + 2 * turn + k)
            copy(d["x"] + [d["w"], d["b"], d["many"], d["few"], d["dloss"], d["target"]] + d["weight"],
                 new["x"] + [new["w"], new["b"], new["many"], new["few"], new["dloss"], new["target"]] + new["weight"])
            for join in JOINS:
                copy(d["res"][join], new["res"][join])
            g.replay()
            want = passes(vrc, new)
            torch.cuda.synchronize()
            same(want, out, (turn, k))
    for g, _, _ in graphs:  # one after the other, nothing between
        g.replay()
    torch.cuda.synchronize()
    for _, out, d in graphs:
        same(passes(vrc, d), out)


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("join", ["sum", "scatter"])
def test_the_end_of_a_model(vrc, join):
    """The last layer's sum over four ranks, its norm, the loss of a split vocabulary, and back
    to the layer's inputs and every weight, in fp32 against autograd in 64 bits.  Each operator's
    bound is checked elsewhere; here the errors of six calls on values of the order of 1 add up,
    each at most some hundred half steps of fp32 of the largest value: 2^-13 of it is a bound."""
    f = gen(91)
    n, tokens, width, vocab = 4, 90, 136, [200, 177, 60, 1]
    x, res = [f(tokens, width) for _ in range(n)], f(tokens, width) * 2
    w, b = f(width) * 0.2 + 1, f(width) * 0.1
    weight = [f(v, width) * 0.15 for v in vocab]
    target = torch.randint(0, sum(vocab), (tokens,), device=DEV)
    target[::5] = IGNORE
    kept = (target != IGNORE).sum()
    spans = ref.spans(tokens, n)
    parts = res if join == "sum" else [res[a:c].contiguous() for a, c in spans]
    y, h, mean, rstd = vrc.vrc_layer_norm(x, w, b, residual=parts, join=join)
    hidden = y[0] if join == "sum" else vrc.vrc_all_gather(y)[0] if tokens % n == 0 else torch.cat(y)
    loss, lse = vrc.vrc_cross_entropy(hidden, weight, target)
    dloss = torch.full_like(loss, 1.0) / kept
    dlse = 2e-2 * lse * (target != IGNORE) / kept  # of a penalty of 1e-2 lse^2
    dhidden, dweight = vrc.vrc_cross_entropy_grad(hidden, weight, target, lse, dloss, dlse=dlse)
    share = [dhidden * (0.5 if r == 0 else 0.5 / (n - 1)) for r in range(n)]  # column-parallel: each rank has a part of it
    dx, dw, db = vrc.vrc_layer_norm_grad(share, h, w, mean, rstd, join=join)
    dx = dx[0] if join == "sum" else torch.cat(dx)

    leaves = [t.double().requires_grad_() for t in (*x, res, w, b, *weight)]
    xs, r64, w64, b64, ws = leaves[:n], leaves[n], leaves[n + 1], leaves[n + 2], leaves[n + 3:]
    y64 = torch.nn.functional.layer_norm(sum(xs) + r64, (width,), w64, b64, 1e-5)
    z = y64 @ torch.cat(ws).t()
    lse64 = torch.logsumexp(z, 1)
    total = (torch.nn.functional.cross_entropy(z, target, ignore_index=IGNORE)
             + 1e-2 * (lse64.square() * (target != IGNORE)).sum() / kept)
    total.backward()
    mine = (loss.sum() + 1e-2 * (lse.square() * (target != IGNORE)).sum()) / kept
    assert abs(float(mine) - float(total.detach())) < 2.0**-13 * abs(float(total.detach()))
    for got, want, what in [(dx, xs[0].grad, "x"), (dx, xs[3].grad, "x3"), (dx, r64.grad, "residual"), (dw, w64.grad, "weight"),
                            (db, b64.grad, "bias")] + [(g, t.grad, "vocabulary") for g, t in zip(dweight, ws)]:
        assert float((got.double() - want).abs().max()) < 2.0**-13 * float(want.abs().max()), what


def test_binding_refusals_on_the_device(vrc):
    f = gen(99)
    x, w, s = [f(4, 64) for _ in range(2)], f(64), f(4)
    h, ws, t = f(4, 64), [f(9, 64)], torch.zeros(4, dtype=torch.int64, device=DEV)
    ints = [torch.zeros(4, 64, dtype=torch.int32, device=DEV)] * 2
    for call in (lambda: vrc.vrc_layer_norm(ints, w), lambda: vrc.vrc_layer_norm([v.double() for v in x], w.double()),
                 lambda: vrc.vrc_layer_norm(x, w.half()), lambda: vrc.vrc_cross_entropy(h.double(), [v.double() for v in ws], t)):
        with pytest.raises(TypeError):
            call()
    for call in (
            lambda: vrc.vrc_layer_norm([x[0], x[1].half()], w), lambda: vrc.vrc_layer_norm([x[0], x[1][:2]], w),
            lambda: vrc.vrc_layer_norm([v.t() for v in x], f(4)), lambda: vrc.vrc_layer_norm(x, w[:63]), lambda: vrc.vrc_layer_norm(x, w.cpu()),
            lambda: vrc.vrc_layer_norm(x, w, bias=w.half()), lambda: vrc.vrc_layer_norm(x, w, residual=x[0]),
            lambda: vrc.vrc_layer_norm(x, w, residual=x, join="sum"), lambda: vrc.vrc_layer_norm(x, w, residual=x, join="scatter"),
            lambda: vrc.vrc_layer_norm(x, w, recv=x[:1]), lambda: vrc.vrc_layer_norm(x, w, sum=x), lambda: vrc.vrc_layer_norm([f(())], w),
            lambda: vrc.vrc_layer_norm(x, w, residual=[x[0]]), lambda: vrc.vrc_layer_norm(x, w, join="sum", sum=[x[0]]),
            lambda: vrc.vrc_layer_norm_grad(x, x, w, s, [s, s]), lambda: vrc.vrc_layer_norm_grad(x, x, w, None, s),
            lambda: vrc.vrc_layer_norm_grad(x, x, w, None, [s, s.half()]), lambda: vrc.vrc_layer_norm_grad(x, x, w, None, [s, s[:3]]),
            lambda: vrc.vrc_layer_norm_grad(x, x, w, None, [s, s], dh=x[0]), lambda: vrc.vrc_layer_norm_grad(x, x, w, None, [s, s], recv=[x[0]]),
            lambda: vrc.vrc_cross_entropy(h, ws, t.int()), lambda: vrc.vrc_cross_entropy(h, ws, t[:3]), lambda: vrc.vrc_cross_entropy(h, ws, t.cpu()),
            lambda: vrc.vrc_cross_entropy(h, [f(9, 65)], t), lambda: vrc.vrc_cross_entropy(h, [f(9, 64).half()], t),
            lambda: vrc.vrc_cross_entropy(h, [f(64, 9).t()], t), lambda: vrc.vrc_cross_entropy(h.t(), [f(9, 4)], t), lambda: vrc.vrc_cross_entropy(h, ws * 17, t),
            lambda: vrc.vrc_cross_entropy(h, ws, t, ignore_index=1 << 63), lambda: vrc.vrc_cross_entropy(f(4, 0), [f(9, 0)], t),
            lambda: vrc.vrc_cross_entropy_grad(h, ws, t, s.half(), s), lambda: vrc.vrc_cross_entropy_grad(h, ws, t, s, s[:3]),
            lambda: vrc.vrc_cross_entropy_grad(h, ws, t, s, s.sum().expand(4)), lambda: vrc.vrc_cross_entropy_grad(h, ws, t, s, s, recv=(h[:3], ws)),
            lambda: vrc.vrc_cross_entropy_grad(h, ws, t, s, s, recv=(f(4, 64), f(9, 64)))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(vrc.VrcError):  # the C functions' own: an output over an input
        vrc.vrc_cross_entropy_grad(h, ws, t, s, s, recv=(h, [f(9, 64)]))
    with pytest.raises(vrc.VrcError):
        vrc.vrc_layer_norm(x, w, recv=[x[1], x[0]])
    with pytest.raises(vrc.VrcError):
        vrc.vrc_layer_norm(x, w, eps=-1.0)
