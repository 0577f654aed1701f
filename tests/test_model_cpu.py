"""The model's operators on the CPU: symbols, refusals before any GPU call, workspace
sizes, the binding's checks, and the references' own pins (by differences and by hand)."""
import ctypes as C
import os
import re
import subprocess

import pytest
import torch

import ring_all_reduce_virtual_amd as vrc
from ring_all_reduce_virtual_amd import model, ops
from tests import model_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "include", "vrc_model.h")).read()
L = ops.ops_lib()
K = 1 << 28
A, B, R, S, T, W = 1 * K, 3 * K, 5 * K, 7 * K, 9 * K, 11 * K  # stand-in addresses, far apart
INVALID, UNSUPPORTED, ALIAS = vrc.VRC_ERR_INVALID_ARG, vrc.VRC_ERR_UNSUPPORTED, vrc.VRC_ERR_ALIAS


def arr(base, n=4, stride=1 << 20):
    return vrc._ptr_array([base + r * stride for r in range(n)])


def test_every_declared_symbol_is_exported_and_bound():
    text = re.sub(r"/\*.*?\*/", "", HEADER, flags=re.S)
    names = sorted(set(re.findall(r"\b(vrc_[a-z_0-9]+)\s*\(", text)))
    assert len(names) == 7
    for n in names:
        assert hasattr(L, n), n
        if not n.endswith("_workspace"):
            assert n in vrc.__all__ and callable(getattr(vrc, n))


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "vrc_model.h"\nint main(void) { vrc_layer_norm_t n = {1, 2, VRC_FP32, VRC_FP32, VRC_NORM_SUM, 1, 1e-5};\n'
                   ' vrc_cross_entropy_t e = {1, 2, 0, VRC_BF16, -100}; size_t b; return vrc_layer_norm_grad_workspace(&n, 1, &b) + (int)e.tokens; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-c", "-o",
                    str(tmp_path / "t.o"), str(src)], check=True)


def norm(rows=8, width=64, dt=vrc.VRC_BF16, wdt=None, join=0, center=1, eps=1e-5):
    return C.byref(model.LayerNorm(rows, width, dt, dt if wdt is None else wdt, join, center, eps))


def test_layer_norm_refusals():
    def f(d=norm(), x=arr(A), res=None, w=W, b=None, y=arr(B), h=None, mean=None, rstd=None, n=4):
        return L.vrc_layer_norm(d, x, res, w, b, y, h, mean, rstd, n, None)

    assert f(n=0) == f(n=17) == f(d=None) == f(x=None) == f(y=None) == f(w=None) == INVALID
    assert f(x=vrc._ptr_array([A, None, A, A])) == f(y=vrc._ptr_array([B, None, R, R])) == INVALID
    assert f(d=norm(eps=-1.0)) == f(d=norm(eps=float("nan"))) == f(d=norm(eps=float("inf"))) == INVALID
    assert f(d=norm(width=1 << 26)) == f(d=norm(rows=1 << 57)) == f(d=norm(rows=1 << 40, width=1 << 20)) == INVALID
    assert f(d=norm(dt=vrc.VRC_INT32)) == f(d=norm(dt=9)) == f(d=norm(wdt=vrc.VRC_FP16)) == UNSUPPORTED
    assert f(d=norm(join=3)) == f(d=norm(join=-1)) == UNSUPPORTED
    assert f(d=norm(center=0), mean=arr(R)) == INVALID                       # RMS norm has no mean
    assert f(d=norm(rows=0), x=None, y=None, w=None) == f(d=norm(width=0), x=None) == vrc.VRC_OK
    # overlaps: recv[r] may be send[r] itself, but another rank's, a shifted or a scattered one is not
    assert f(y=arr(A + 2)) == f(y=vrc._ptr_array([A + (1 << 20), B, R, S])) == ALIAS
    assert f(d=norm(join=2), y=arr(A)) == f(y=vrc._ptr_array([B, B, R, S])) == f(y=vrc._ptr_array([W, B, R, S])) == ALIAS
    assert f(res=arr(R), h=vrc._ptr_array([R + (1 << 20), S, T, W + (1 << 20)])) == f(h=arr(A)) == f(h=arr(B)) == ALIAS
    assert f(res=arr(R), y=arr(R)) == f(rstd=arr(B)) == f(mean=arr(A + 100)) == f(rstd=arr(R), mean=arr(R)) == ALIAS
    assert f(b=B + 100) == ALIAS
    # the parts: four for the scatter, one for the sum; a part without rows may be null
    assert f(d=norm(join=1), res=vrc._ptr_array([None])) == f(res=vrc._ptr_array([R, None, R, R])) == INVALID
    assert f(d=norm(rows=3, join=2), y=vrc._ptr_array([None, None, None, A])) == ALIAS  # three parts are empty


def test_layer_norm_grad_refusals():
    big = 1 << 20

    def f(d=norm(), dy=arr(A), h=arr(R), mean=arr(S), rstd=arr(T), w=W, res=None, y=arr(B), dw=W + big, db=W + 2 * big, n=4,
          ws=W + 4 * big, size=64 * big):
        return L.vrc_layer_norm_grad(d, dy, h, mean, rstd, w, res, y, dw, db, n, ws, size, None)

    assert f(n=0) == f(n=17) == f(d=None) == f(dy=None) == f(h=None) == f(rstd=None) == f(w=None) == f(y=None) == f(dw=None) == INVALID
    assert f(mean=None) == f(d=norm(center=0)) == INVALID                   # mean where centred, and only there
    need = C.c_size_t()
    assert L.vrc_layer_norm_grad_workspace(norm(), 4, C.byref(need)) == vrc.VRC_OK and need.value == 4 * 8 * 2 * 64 * 4
    assert f(size=need.value - 1) == f(ws=None) == f(ws=W + 4 * big + 8) == INVALID
    assert f(d=norm(dt=vrc.VRC_INT32)) == f(d=norm(join=5)) == UNSUPPORTED
    assert f(dw=B) == f(db=A) == f(ws=R) == f(dw=W) == f(db=W + big) == f(y=arr(R)) == f(y=arr(A + 2)) == ALIAS
    assert f(d=norm(join=2), y=arr(A)) == f(res=arr(S + 64), y=arr(S + 64)) == ALIAS
    for d in (norm(rows=1 << 30, width=64, join=1), norm(rows=1 << 30, width=64)):
        assert L.vrc_layer_norm_grad_workspace(d, 16, C.byref(need)) == vrc.VRC_OK
        assert 0 < need.value <= 512 * 2 * 64 * 4                           # bounded, however many rows
    assert L.vrc_layer_norm_grad_workspace(norm(), 4, None) == L.vrc_layer_norm_grad_workspace(None, 4, C.byref(need)) == INVALID


def ce(tokens=8, width=64, vocab=(100, 50), dt=vrc.VRC_BF16, ignore=-100):
    sizes = (C.c_size_t * max(1, len(vocab)))(*vocab)
    d = model.CrossEntropy(tokens, width, sizes, dt, ignore)
    d.keep = sizes
    return d


def entropy_space(d, n, grad, hidden=A, weight=None, dhidden=1):
    need = C.c_size_t()
    weight = arr(B, n) if weight is None else weight
    st = (L.vrc_cross_entropy_grad_workspace(C.byref(d), hidden, weight, dhidden, n, C.byref(need)) if grad
          else L.vrc_cross_entropy_workspace(C.byref(d), hidden, weight, n, C.byref(need)))
    assert st == vrc.VRC_OK
    return need.value


def test_cross_entropy_refusals():
    def f(d=None, h=A, w=arr(B, 2), t=R, loss=S, lse=T, n=2, ws=W, size=1 << 28):
        return L.vrc_cross_entropy(C.byref(ce() if d is None else d), h, w, t, loss, lse, n, ws, size, None)

    assert f(n=0) == f(n=17) == f(h=None) == f(w=None) == f(t=None) == f(lse=None) == f(w=vrc._ptr_array([B, None])) == INVALID
    assert L.vrc_cross_entropy(None, A, arr(B, 2), R, S, T, 2, W, 1 << 28, None) == INVALID
    assert f(d=ce(width=0)) == f(d=ce(width=1 << 20)) == f(d=ce(tokens=1 << 24)) == INVALID
    assert f(d=ce(vocab=(1 << 23, 1))) == f(d=ce(vocab=(1 << 22, 1 << 22))) == INVALID
    assert f(d=ce(width=1 << 19, vocab=(1 << 18, 0))) == f(d=ce(width=1 << 19, tokens=1 << 18)) == INVALID
    assert f(d=ce(dt=vrc.VRC_INT32)) == f(d=ce(dt=7)) == UNSUPPORTED
    assert f(t=R + 4) == f(lse=T + 2) == f(ws=W + 8) == f(ws=None) == f(size=entropy_space(ce(), 2, False) - 1) == INVALID
    assert f(lse=A) == f(loss=B + 64) == f(loss=T) == f(ws=R) == f(ws=S) == f(lse=R) == ALIAS
    assert f(d=ce(tokens=0), h=None, lse=None) == vrc.VRC_OK


def test_cross_entropy_grad_refusals():
    def f(d=None, h=A, w=arr(B, 2), t=R, lse=R + 4096, dloss=R + 8192, dlse=None, dh=S, dw=arr(T, 2), n=2, ws=W, size=1 << 28):
        return L.vrc_cross_entropy_grad(C.byref(ce() if d is None else d), h, w, t, lse, dloss, dlse, dh, dw, n, ws, size, None)

    assert f(n=0) == f(h=None) == f(w=None) == f(t=None) == f(lse=None) == f(dloss=None) == f(dw=vrc._ptr_array([T, None])) == INVALID
    assert f(t=R + 4) == f(dlse=R + 12290) == f(ws=None) == f(size=entropy_space(ce(), 2, True) - 1) == INVALID
    assert f(d=ce(dt=vrc.VRC_INT32)) == UNSUPPORTED
    assert f(dh=A) == f(dw=arr(B, 2)) == f(dh=T) == f(ws=B) == f(dh=R) == f(dw=vrc._ptr_array([T, T])) == ALIAS
    assert f(dh=None, dw=None, ws=None, size=0) == vrc.VRC_OK                # nothing is asked for


@pytest.mark.parametrize("dt", [vrc.VRC_FP32, vrc.VRC_FP16, vrc.VRC_BF16])
def test_workspace_sizes(dt):
    """Bounded however large the vocabulary and however many tokens: no logits are kept."""
    esz = 4 if dt == vrc.VRC_FP32 else 2
    for tokens, width, vocab in ((1, 1, (1,)), (7, 4096, (4096,) * 8), (4096, 4096, (8192,) * 8), (8192, 1000, (300000,)),
                                 (131072, 4096, (16384,) * 8), (3, 8192, (1 << 20,)), (5000, 1053, (50003,))):
        d = ce(tokens, width, vocab, dt)
        n, total, wide = len(vocab), sum(vocab), -(-width // 64) * 64
        loss, grad = entropy_space(d, n, False), entropy_space(d, n, True)
        packed = min(total + 256 * n, max(256, (1 << 30) // (wide * esz))) * wide * esz if width * esz % 16 else 0
        stats = (total // 64 + 4 * n + 4) * min(tokens, 16384) * 8
        assert loss <= stats + tokens * wide * esz + packed + (1 << 20)
        rows = max(128, -(-tokens // 64) * 64)
        sums = max(512 * 128 * 128 * 4, 2 * rows * wide * 4) * 3
        assert grad <= max(1 << 27, rows * 4352 * esz) + rows * (wide * esz + 16) + sums + packed + wide * 128 * esz + (4 << 20)
        if tokens * total * esz > 1 << 31:
            assert grad < tokens * total * esz                               # less than the logits
    assert entropy_space(ce(vocab=(0, 0), dt=dt), 2, True) == 0
    assert entropy_space(ce(4096, 4096, (8192,) * 8, dt), 8, True, dhidden=0) < entropy_space(ce(4096, 4096, (8192,) * 8, dt), 8, True)
    # rows or addresses off the 16-byte grid are packed first
    odd = ce(64, 72, (1000, 1000), dt)
    assert entropy_space(odd, 2, False, weight=arr(B + esz, 2)) > entropy_space(odd, 2, False)


def test_binding_refuses_cpu_tensors_and_bad_arguments():
    x, w = [torch.zeros(4, 64, dtype=torch.bfloat16)] * 2, torch.zeros(64, dtype=torch.bfloat16)
    h, ws, t, s = torch.zeros(4, 64), [torch.zeros(9, 64)], torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    for call in (lambda: vrc.vrc_layer_norm(x, w), lambda: vrc.vrc_layer_norm([], w), lambda: vrc.vrc_layer_norm(x * 9, w),
                 lambda: vrc.vrc_layer_norm(x[0], w), lambda: vrc.vrc_layer_norm([1, 2], w), lambda: vrc.vrc_layer_norm(x, w, join="mean"),
                 lambda: vrc.vrc_layer_norm_grad(x, x, w, None, [s] * 2), lambda: vrc.vrc_layer_norm_grad(x, x, w, None, [s] * 2, join=1),
                 lambda: vrc.vrc_cross_entropy(h, ws, t), lambda: vrc.vrc_cross_entropy(h, ws[0], t), lambda: vrc.vrc_cross_entropy(h, [], t),
                 lambda: vrc.vrc_cross_entropy_grad(h, ws, t, s, s), lambda: vrc.vrc_cross_entropy_grad(h, ws, None, s, s)):
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------------------
# The references
# ---------------------------------------------------------------------------
def slope(f, x, d, step=1e-5):
    """The derivative of the scalar f at x along d, by central differences: the error is
    of the order of step^2 and of 2^-53 |f| / step."""
    return (f(x + step * d) - f(x - step * d)) / (2 * step)


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("join", ["each", "sum", "scatter"])
def test_layer_norm_reference_by_differences(join, center):
    g = torch.Generator().manual_seed(3)
    n, rows, width, eps = 3, 5, 7, 1e-2
    x = [torch.randn(rows, width, generator=g, dtype=torch.float64) for _ in range(n)]
    w, b = (torch.randn(width, generator=g, dtype=torch.float64) for _ in range(2))
    parts = ref.parts_of(x, join)
    dys = [torch.randn(p[0].shape, generator=g, dtype=torch.float64) for p in parts]

    def loss(x, w, b):
        return sum(float((ref.layer_norm(p, None, w, b, eps, center)[0][0] * dy).sum()) for p, dy in zip(ref.parts_of(x, join), dys))

    dw = db = 0.0
    dx = []
    for p, dy in zip(parts, dys):
        _, (h, _), (mean, _), (rstd, _) = ref.layer_norm(p, None, w, b, eps, center)
        (d, _), (tw, _), (tb, _) = ref.layer_norm_grad([dy], h, w, mean if center else None, rstd, None)
        dx.append(d)
        dw, db = dw + tw, db + tb
    full = dx if join == "each" else [torch.cat(dx)] * n  # every send's
    for r in range(n):
        v = torch.randn(rows, width, generator=g, dtype=torch.float64)
        got = slope(lambda t: loss(x[:r] + [t] + x[r + 1:], w, b), x[r], v)
        assert abs(got - float((full[r] * v).sum())) < 1e-7 * (1 + abs(got))
    v = torch.randn(width, generator=g, dtype=torch.float64)
    assert abs(slope(lambda t: loss(x, t, b), w, v) - float((dw * v).sum())) < 1e-7
    assert abs(slope(lambda t: loss(x, w, t), b, v) - float((db * v).sum())) < 1e-7


def test_cross_entropy_reference_by_differences_and_by_hand():
    g = torch.Generator().manual_seed(5)
    hidden = torch.randn(6, 4, generator=g, dtype=torch.float64)
    weight = [torch.randn(v, 4, generator=g, dtype=torch.float64) for v in (3, 5, 1)]
    target = torch.tensor([0, 8, -100, 4, 2, -100])
    dloss, dlse = (torch.randn(6, generator=g, dtype=torch.float64) for _ in range(2))
    dlse[2] = 0.0

    def loss(hidden, weight):
        (l, _), (s, _) = ref.cross_entropy(hidden, weight, target, -100)
        return float((l * dloss + s * dlse).sum())

    lse = torch.logsumexp(ref.logits(hidden, weight)[0], 1)
    (dh, _), dw = ref.cross_entropy_grad(hidden, weight, target, lse, dloss, dlse, -100, torch.float32)
    assert not dh[2].any()  # ignored, and no gradient by lse
    v = torch.randn(6, 4, generator=g, dtype=torch.float64)
    assert abs(slope(lambda t: loss(t, weight), hidden, v) - float((dh * v).sum())) < 1e-7
    for r in range(3):
        v = torch.randn(weight[r].shape, generator=g, dtype=torch.float64)
        got = slope(lambda t: loss(hidden, weight[:r] + [t] + weight[r + 1:]), weight[r], v)
        assert abs(got - float((dw[r][0] * v).sum())) < 1e-7
    # by hand: logits 0, log 3 -> lse log 4, loss of the second log(4 / 3)
    h, w = torch.tensor([[1.0]]), [torch.tensor([[0.0]]), torch.tensor([[3.0]]).log()]
    (l, _), (s, _) = ref.cross_entropy(h, w, torch.tensor([1]), -100)
    assert abs(float(s) - torch.log(torch.tensor(4.0)).item()) < 1e-6
    assert abs(float(l) - torch.log(torch.tensor(4.0 / 3.0)).item()) < 1e-6
    assert torch.isnan(ref.cross_entropy(h, w, torch.tensor([2]), -100)[0][0]).all()
