"""The model's operators where their rules meet: tokens without weight whose targets are
invalid, rows without values, shapes that hold as many elements, weights far apart, the
precision of few tokens, and tensors too large for the caches or for 32-bit offsets.
Tolerances are those of tests/model_reference.py."""
import threading

import pytest
import torch

from tests import model_reference as ref
from tests.test_gpu_model import (DEV, DT, IGNORE, check_entropy, check_entropy_grad, check_norm, check_norm_grad, close,
                                  entropy_inputs, gen, say, vrc)  # noqa: F401  (vrc: the fixture)
from tests.test_gpu_model_use import inputs, passes, same

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# Targets outside the vocabulary
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("tokens", [5, 32, 70, 128, 200])
def test_invalid_targets_without_weight_reach_nothing(vrc, dtype, tokens):
    """A token whose dloss and dlse are 0 has no gradient, whatever its target, hidden state and
    lse are: the bits are those of the same tokens ignored."""
    say(f"{dtype} {tokens}")
    torch.manual_seed(9)
    hidden, weight, target = entropy_inputs(tokens, [130, 0, 60], 72, DT[dtype], 33, ignored=0.1)
    _, lse = vrc.vrc_cross_entropy(hidden, weight, target)
    dloss = torch.rand(tokens, device=DEV) + 0.1
    gone = torch.arange(tokens, device=DEV) % 4 == 1
    dloss[gone] = 0.0
    dloss[1] = -0.0
    stray = torch.tensor([-1, 190, 1 << 40, -(1 << 63), 1 << 31], device=DEV)
    bad_target = torch.where(gone, stray[torch.arange(tokens, device=DEV) % 5], target)
    bad_hidden, bad_lse = hidden.clone(), lse.clone()
    bad_hidden[gone] = float("nan")
    bad_lse[gone] = float("inf")
    dlse = torch.rand(tokens, device=DEV) * ~gone
    for second in (None, torch.zeros_like(dloss), dlse):
        want = vrc.vrc_cross_entropy_grad(hidden, weight, torch.where(gone, torch.full_like(target, IGNORE), target), lse, dloss, dlse=second)
        got = vrc.vrc_cross_entropy_grad(bad_hidden, weight, bad_target, bad_lse, dloss, dlse=second)
        same(want, got, "as ignored")
        assert not got[0][gone].any() and all(torch.isfinite(t).all() for t in got[1])
    # one with any weight: NaN in all of its gradients, and the others' as before
    for first, second in ((1.0, 0.0), (0.0, 1.0), (1.0, -1.0)):
        one, two = dloss.clone(), torch.zeros_like(dloss)
        one[1], two[1] = first, second
        dh, dw = vrc.vrc_cross_entropy_grad(hidden, weight, bad_target, lse, one, dlse=two)
        assert torch.isnan(dh[1]).all() and all(torch.isnan(t).all() for t in dw)
        rest = torch.arange(tokens, device=DEV) != 1
        assert torch.isfinite(dh[rest]).all() and not dh[gone & rest].any()


# ---------------------------------------------------------------------------
# Sizes and shapes
# ---------------------------------------------------------------------------
def test_rows_without_values_are_refused(vrc):
    """They have no mean and rstd to return."""
    w = torch.ones(0, device=DEV)
    for join in ("each", "sum", "scatter"):
        for center in (True, False):
            with pytest.raises(vrc.VrcError):
                vrc.vrc_layer_norm([torch.ones(3, 0, device=DEV)] * 2, w, join=join, center=center)
        y, h, mean, rstd = vrc.vrc_layer_norm([torch.ones(0, 0, device=DEV)] * 2, w, join=join)  # no rows either
        assert all(t.shape == (0, 0) for t in y)


def test_shapes_of_as_many_elements_are_refused(vrc):
    """What is read or written row by row has the documented shape, not only its number of elements."""
    f = gen(98)
    x, w, b = [f(6, 4) for _ in range(2)], f(4), f(4)
    y, h, mean, rstd = vrc.vrc_layer_norm(x, w, b, join="sum")
    turned, wide = f(4, 6), f(3, 8)
    for call in (
            lambda: vrc.vrc_layer_norm(x, f(2, 2)), lambda: vrc.vrc_layer_norm(x, w, f(1, 4)), lambda: vrc.vrc_layer_norm(x, w, residual=[x[0], turned]),
            lambda: vrc.vrc_layer_norm(x, w, residual=wide, join="sum"), lambda: vrc.vrc_layer_norm(x, w, recv=[turned, f(6, 4)]),
            lambda: vrc.vrc_layer_norm(x, w, join="sum", sum=turned), lambda: vrc.vrc_layer_norm(x, w, join="sum", sum=f(24)),
            lambda: vrc.vrc_layer_norm(x, w, residual=[f(4, 3), f(3, 4)], join="scatter"),
            lambda: vrc.vrc_layer_norm_grad(x, turned, w, mean, rstd, join="sum"), lambda: vrc.vrc_layer_norm_grad(x, h, f(4, 1), mean, rstd, join="sum"),
            lambda: vrc.vrc_layer_norm_grad(x, h, w, mean.view(2, 3), rstd, join="sum"), lambda: vrc.vrc_layer_norm_grad(x, h, w, mean, rstd.view(6, 1), join="sum"),
            lambda: vrc.vrc_layer_norm_grad(x, h, w, mean, rstd, dh=wide, join="sum"), lambda: vrc.vrc_layer_norm_grad(x, h, w, mean, rstd, join="sum", recv=[f(6, 4), turned])):
        with pytest.raises(ValueError):
            call()
    hidden, weight, target = f(2, 3, 8), [f(5, 8), f(4, 8)], torch.zeros(2, 3, dtype=torch.int64, device=DEV)
    loss, lse = vrc.vrc_cross_entropy(hidden, weight, target)
    for call in (
            lambda: vrc.vrc_cross_entropy_grad(hidden, weight, target, lse.view(6), loss), lambda: vrc.vrc_cross_entropy_grad(hidden, weight, target, lse, loss.view(3, 2)),
            lambda: vrc.vrc_cross_entropy_grad(hidden, weight, target, lse, loss, dlse=loss.view(6)),
            lambda: vrc.vrc_cross_entropy_grad(hidden, weight, target, lse, loss, recv=(f(6, 8), None)),
            lambda: vrc.vrc_cross_entropy_grad(hidden, weight, target, lse, loss, recv=(None, [f(8, 5), f(4, 8)]))):
        with pytest.raises(ValueError):
            call()
    dh, dw = vrc.vrc_cross_entropy_grad(hidden, weight, target, lse, loss, dlse=loss)
    assert dh.shape == (2, 3, 8) and [t.shape for t in dw] == [(5, 8), (4, 8)]


# ---------------------------------------------------------------------------
# The gradients of the logits, G, between the products
# ---------------------------------------------------------------------------
def grad_inputs(tokens, dtype, seed):
    hidden, weight, target = entropy_inputs(tokens, [700, 0, 333], 192, dtype, seed, ignored=0.1)
    target[0] = 699
    z, _ = ref.logits(hidden, weight)
    return hidden, weight, target, z, torch.logsumexp(z, 1).float()


def logit_grads(z, target, lse, dloss):
    """G in 64 bits, and the largest |a| or |b|, in whose units it is held."""
    b = torch.where(target != IGNORE, dloss, torch.zeros_like(dloss)).double()
    g = (z - lse.double()[:, None]).exp() * b[:, None]
    rows = torch.nonzero(target != IGNORE)[:, 0]
    g[rows, target[rows]] -= b[rows]
    return g, float(b.abs().max())


def bounds(hidden, weight, target, lse, dloss, of_g):
    """((dhidden, bound), [(dweight, bound)]) where G is off by at most `of_g` (element by element) from its rounding."""
    (dh, edh), dw = ref.cross_entropy_grad(hidden, weight, target, lse, dloss, None, IGNORE, torch.float32)
    w, h = torch.cat(weight).double().abs(), hidden.double().abs()
    more = (of_g.t() @ h).split([x.shape[0] for x in weight])
    return (dh, edh + of_g @ w), [(d, e + m) for (d, e), m in zip(dw, more)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("tokens", [1, 7, 32, 33, 64, 128])
def test_few_tokens_hold_two_values_of_each(vrc, dtype, tokens):
    """Up to 128 tokens of 16-bit types G is its rounding and the rounding of what that left: off by at most
    half a step of half a step of the type (and fp16's subnormals, in units of 2^-14 of the largest)."""
    dtype = DT[dtype]
    hidden, weight, target, z, lse = grad_inputs(tokens, dtype, 35)
    f = gen(36)
    dloss = f(tokens) + 0.3
    g, most = logit_grads(z, target, lse, dloss)
    half = ref.EPS_HALF[dtype]
    least = 2.0**-25 * 2.0**-14 * most if dtype is torch.float16 else 0.0
    want_h, want_w = bounds(hidden, weight, target, lse, dloss, g.abs() * half * half + least * (g != 0))
    dh, dw = vrc.vrc_cross_entropy_grad(hidden, weight, target, lse, dloss)
    close(dh, want_h, (tokens, "dhidden"))
    for got, want in zip(dw, want_w):
        close(got, want, (tokens, "dweight"))
    # one value of each would not pass: the bound tells the two apart
    unit = most * (2.0**-14 if dtype is torch.float16 else 1.0)
    once = ((g / unit).to(dtype).double() * unit).t() @ torch.where(dloss[:, None] != 0, hidden.double(), 0.0)
    with pytest.raises(AssertionError):
        close(once[:700].to(dtype), want_w[0], "once")


@pytest.mark.parametrize("tokens", [40, 200])
def test_weights_far_apart_in_fp16(vrc, tokens):
    """One unit holds all tokens' G: elements from 2^-28 of the largest weight on keep all bits of fp16, smaller ones
    are rounded to multiples of 2^-38 of it."""
    hidden, weight, target, z, lse = grad_inputs(tokens, torch.float16, 37)
    dloss = 1024.0 * 2.0 ** -(torch.arange(tokens, device=DEV) % 31).float()
    g, most = logit_grads(z, target, lse, dloss)
    assert most == 1024.0
    of_g = torch.where(g.abs() >= 2.0**-28 * most, g.abs() * 2.0**-11, torch.full_like(g, 2.0**-39 * most)) * (g != 0)
    want_h, want_w = bounds(hidden, weight, target, lse, dloss, of_g)
    dh, dw = vrc.vrc_cross_entropy_grad(hidden, weight, target, lse, dloss)
    close(dh, want_h, (tokens, "dhidden"))
    for got, want in zip(dw, want_w):
        close(got, want, (tokens, "dweight"))


# ---------------------------------------------------------------------------
# Large tensors
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("join,n,vectors", [("sum", 2, 60.3), ("scatter", 3, 128), ("sum", 3, 250.2), ("scatter", 2, 512), ("sum", 4, 1000.7), ("scatter", 3, 2048),
                                            ("sum", 16, 2040.2)])
def test_rows_that_pass_by_the_caches(vrc, join, n, vectors, dtype):
    """256 MiB and more, of several sources, for each kind of row: narrow and wide, with and without elements behind
    the last vector, many rows and few."""
    dtype = DT[dtype]
    size = torch.finfo(dtype).bits // 8
    width = int(vectors * (16 // size))
    rows = -(-(256 << 20) // (width * n * size)) + 1
    say(f"{join} {n} {dtype} {rows} x {width}")
    check_norm(vrc, join, n, rows, width, dtype, residual=n == 3)
    torch.cuda.empty_cache()
    check_norm_grad(vrc, join, n, rows, width, dtype, residual=n == 3)
    torch.cuda.empty_cache()


def test_layer_norm_weights_past_32_bits(vrc):
    """All gradients of 8.6 GB of rows of which twelve, around the places where 32-bit offsets end, have any."""
    rows, width = (1 << 20) + 3, 4104
    torch.manual_seed(8)
    x = torch.empty(rows, width, dtype=torch.bfloat16, device=DEV).normal_()
    w = gen(5)(width).bfloat16()
    _, _, mean, rstd = vrc.vrc_layer_norm([x], w)
    pick = torch.tensor([0, 1, 261632, 261633, 523263, 523264, 523265, 523266, 784896, 784897, rows - 2, rows - 1], device=DEV)
    dy = torch.zeros_like(x)
    dy[pick] = gen(6)(12, width).bfloat16()
    dx, dw, db = vrc.vrc_layer_norm_grad([dy], [x], w, mean, rstd)
    rx, rw, rb = ref.layer_norm_grad([dy[pick]], x[pick], w, mean[0][pick], rstd[0][pick], None)
    close(dw, rw, "dweight")
    close(db, rb, "dbias")
    close(dx[0][pick], rx, "dx")
    dx[0][pick] = 0
    assert not dx[0].any()


def test_cross_entropy_gradients_past_32_bits(vrc):
    """Both gradients of 4.6 GB of weights, whole.  The hidden states have 16 values, so that a logit's bound
    counts as many products; some rows, on both sides of 4 GiB, have an eighth of the probability."""
    tokens, width, vocab = 3, 16384, 140001
    torch.manual_seed(7)
    f = gen(7)
    cols = torch.randperm(width, device=DEV)[:16]
    hidden = torch.zeros(tokens, width, device=DEV)
    hidden[:, cols] = f(tokens, 16) / 8  # logits of about half around 0
    hidden[:, cols[0]] = 1.0
    hidden = hidden.bfloat16()
    weight = [f(5, width).bfloat16(), torch.empty(vocab, width, dtype=torch.bfloat16, device=DEV).normal_()]
    likely = torch.tensor([0, 65536, 131071, 131072, 131073, vocab - 2, vocab - 1], device=DEV)
    weight[1][likely[:, None], cols] = 0.0
    weight[1][likely, cols[0]] = 12.0  # the logit of each likely row
    target = torch.tensor([vocab + 4, 5 + 131072, 3], device=DEV)

    def chunks():
        at = 0
        for r, w in enumerate(weight):
            for i in range(0, w.shape[0], 10000):
                yield at, r, i, w[i:i + 10000].double()
                at += min(10000, w.shape[0] - i)

    h = hidden.double()
    z = torch.cat([h @ c.t() for _, _, _, c in chunks()], 1)
    ez = torch.cat([17 * ref.U * (h.abs() @ c.abs().t()) for _, _, _, c in chunks()], 1)
    lse, dloss = torch.logsumexp(z, 1).float(), f(tokens)
    dh, dw = vrc.vrc_cross_entropy_grad(hidden, weight, target, lse, dloss)
    off = z - lse.double()[:, None]
    p = off.exp() * dloss.double()[:, None]
    g = p.clone()
    g[torch.arange(tokens, device=DEV), target] -= dloss.double()
    eg = p.abs() * (ez + 4 * ref.U * (1 + off.abs()) + 2 * ref.U) + 4 * ref.U * (p.abs() + g.abs()) + g.abs() * 2.0**-16
    want, bound, size = torch.zeros_like(h), torch.zeros_like(h), torch.zeros_like(h)
    for at, r, i, c in chunks():
        a, b = at, at + c.shape[0]
        want += g[:, a:b] @ c
        bound += eg[:, a:b] @ c.abs()
        size += g[:, a:b].abs() @ c.abs()
        close(dw[r][i:i + 10000], (g[:, a:b].t() @ h, eg[:, a:b].t() @ h.abs() + (tokens + 4) * ref.U * (g[:, a:b].abs().t() @ h.abs())), ("dweight", r, i))
    bound += (vocab + 160) * ref.U * size
    # a likely row's part (its G times a mean absolute value of 0.8) is well above what the sums' order may change
    assert (4 * bound.mean(1) < 0.8 * g[:, 5 + likely].abs().min(1).values).all()
    close(dh, (want, bound), "dhidden")


# ---------------------------------------------------------------------------
# The largest sizes, and calls at once
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", DT)
def test_norms_of_more_rows_than_one_turn_has(vrc, dtype):
    """Five million rows, which the largest grid takes in two turns."""
    for width in (3, 16):
        check_norm(vrc, "each", 1, (5 << 20) + 3, width, DT[dtype])
        check_norm_grad(vrc, "each", 1, (5 << 20) + 3, width, DT[dtype])
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_norms_of_the_widest_rows(vrc, dtype):
    check_norm(vrc, "sum", 2, 1, (1 << 26) - 1, DT[dtype])
    check_norm_grad(vrc, "sum", 2, 1, (1 << 26) - 1, DT[dtype])
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("tokens,width", [(3, (1 << 20) - 1), (40, (1 << 20) - 64), (200, (1 << 20) - 1)])
def test_cross_entropy_of_the_widest_rows(vrc, dtype, tokens, width):
    say(f"{dtype} {tokens} x {width}")
    check_entropy(vrc, tokens, [5, 0, 150], width, DT[dtype])
    check_entropy_grad(vrc, tokens, [5, 0, 150], width, DT[dtype])
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("tokens", [2, 100, 130])
def test_cross_entropy_of_the_largest_vocabulary(vrc, dtype, tokens):
    vocab = [(1 << 23) - 301, 300] if tokens < 10 else [1 << 20, 300]
    say(f"{dtype} {tokens} of {sum(vocab)}")
    check_entropy(vrc, tokens, vocab, 8, DT[dtype])
    check_entropy_grad(vrc, tokens, vocab, 8, DT[dtype])
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", DT)
def test_cross_entropy_of_the_most_tokens(vrc, dtype):
    say(dtype)
    check_entropy(vrc, (1 << 24) - 1, [2, 1], 1, DT[dtype])
    check_entropy_grad(vrc, (1 << 24) - 1, [2, 1], 1, DT[dtype], weighted=False, scale=1024.0)
    torch.cuda.empty_cache()


def test_calls_of_several_threads_at_once(vrc):
    """Each thread on a stream and on data of its own; host code runs without the interpreter's lock."""
    data = [inputs(110 + i, [torch.bfloat16, torch.float16, torch.float32][i % 3]) for i in range(4)]
    want = [passes(vrc, d) for d in data]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got[i] = passes(vrc, data[i])
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    same(want, got)
