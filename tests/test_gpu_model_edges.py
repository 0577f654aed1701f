"""The model's operators where their rules meet: tokens without weight whose targets are
invalid, rows without values, shapes that hold as many elements, weights far apart, the
precision of few tokens, and tensors too large for the caches or for 32-bit offsets.
Tolerances are those of tests/model_reference.py."""
import pytest
import torch

from tests import model_reference as ref
from tests.test_gpu_model import (DEV, DT, IGNORE, check_norm, check_norm_grad, close, entropy_inputs, gen, say,  # noqa: F401
                                  vrc)  # (vrc: the fixture)
from tests.test_gpu_model_use import same

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
