"""The model's operators on the GPU against 64-bit references (tests/model_reference.py,
which derives the tolerances: every rounding of the evaluation counted)."""
import pytest
import torch

from tests import model_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
IGNORE = -100


@pytest.fixture(scope="module")
def vrc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import ring_all_reduce_virtual_amd as m
    return m


def say(msg):
    print(msg, flush=True)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return lambda *shape: torch.randn(*shape, generator=g, device=DEV)


def off_grid(x, by=1):
    """The same values, `by` elements past an allocation's start."""
    flat = torch.empty(x.numel() + by, dtype=x.dtype, device=x.device)
    flat[by:] = x.reshape(-1)
    return flat[by:].view(x.shape)


def close(got, want, what, dtype=None):
    """`want`: (value, bound before the rounding to got's type)."""
    y, tol = want
    y = y.reshape(got.shape)
    tol = ref.rounded(y, tol.reshape(got.shape), got.dtype)
    g = got.double()
    assert (torch.isnan(g) == torch.isnan(y)).all(), what
    bad = ~torch.isnan(y) & ~(g == y) & ~((g - y).abs() <= tol)
    if bool(bad.any()):
        i = torch.nonzero(bad)[:4]
        raise AssertionError((what, int(bad.sum()), bad.numel(), i.tolist(), g[bad][:4].tolist(), y[bad][:4].tolist(), tol[bad][:4].tolist()))


# ---------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------
def norm_inputs(join, n, rows, width, dtype, seed, residual=True, bias=True, wide=False, shift=0):
    f = gen(seed)
    put = (lambda x: off_grid(x, shift)) if shift else (lambda x: x)
    wd = torch.float32 if wide else dtype
    x = [put(f(rows, width).to(dtype)) for _ in range(n)]
    part_rows = [rows] if join == "sum" else [rows] * n if join == "each" else [b - a for a, b in ref.spans(rows, n)]
    res = [put((f(r, width) * 3 + 0.7).to(dtype)) for r in part_rows] if residual else None
    w = put((f(width) * 0.3 + 1).to(wd))
    b = put((f(width) * 0.2).to(wd)) if bias else None
    return x, res, w, b


def shared(ts, join):
    return ts[0] if ts is not None and join == "sum" else ts


def listed(ts):
    return ts if isinstance(ts, (list, tuple)) else [ts]


def check_norm(vrc, join, n, rows, width, dtype, seed=1, center=True, eps=1e-5, **kw):
    x, res, w, b = norm_inputs(join, n, rows, width, dtype, seed, **kw)
    y, h, mean, rstd = vrc.vrc_layer_norm(x, w, b, eps, residual=shared(res, join), join=join, center=center)
    parts = ref.parts_of(x, join)
    assert len(y) == n
    for p, xs in enumerate(parts):
        ry, rh, rm, rr = ref.layer_norm(xs, None if res is None else res[p], w, b, eps, center)
        what = (join, n, rows, width, str(dtype), p)
        for q in (range(n) if join == "sum" else [p]):
            close(y[q], ry, what + ("y", q))
        if res is None and join == "each":
            assert h is x
        else:
            close(listed(h)[p], rh, what + ("h",))
        close(listed(rstd)[p], rr, what + ("rstd",))
        if center:
            close(listed(mean)[p], rm, what + ("mean",))
        else:
            assert mean is None


def check_norm_grad(vrc, join, n, rows, width, dtype, seed=2, center=True, bias=True, wide=False, residual=True, shift=0, eps=1e-5):
    dy, dh, w, _ = norm_inputs(join, n, rows, width, dtype, seed, residual=residual, bias=False, wide=wide, shift=shift)
    f = gen(seed + 100)
    put = (lambda x: off_grid(x, shift)) if shift else (lambda x: x)
    h, mean, rstd = [], [], []
    for xs in ref.parts_of(dy, join):
        v = (f(*xs[0].shape) * 3 + 0.5).to(dtype)
        m = v.double().mean(-1) if center else torch.zeros_like(v[:, 0]).double()
        h.append(put(v))
        mean.append(put(m.float()))
        rstd.append(put(((v.double() - m.unsqueeze(-1)).square().mean(-1) + eps).rsqrt().float()))
    dx, dw, db = vrc.vrc_layer_norm_grad(dy, shared(h, join), w, shared(mean, join) if center else None, shared(rstd, join),
                                         dh=shared(dh, join), join=join, bias=bias)
    tw = tb = 0.0
    ew = eb = 0.0
    for p, xs in enumerate(ref.parts_of(dy, join)):
        rx, rw, rb = ref.layer_norm_grad(xs, h[p], w, mean[p] if center else None, rstd[p], None if dh is None else dh[p])
        for q in (range(n) if join == "sum" else [p]):
            close(dx[q], rx, (join, n, rows, width, str(dtype), p, "dx", q))
        tw, ew, tb, eb = tw + rw[0], ew + rw[1], tb + rb[0], eb + rb[1]
    close(dw, (tw, ew), (join, n, rows, width, str(dtype), "dweight"))
    if bias:
        close(db, (tb, eb), (join, n, rows, width, str(dtype), "dbias"))
    else:
        assert db is None


JOINS = ["each", "sum", "scatter"]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("join", JOINS)
@pytest.mark.parametrize("n,rows,width", [(1, 1, 1), (2, 1, 5), (3, 7, 8), (8, 1, 4096), (5, 13, 1053), (16, 9, 130), (4, 70, 512)])
def test_layer_norm(vrc, join, dtype, n, rows, width):
    say(f"layer_norm {join} {dtype} {n} {rows} {width}")
    check_norm(vrc, join, n, rows, width, DT[dtype])
    check_norm(vrc, join, n, rows, width, DT[dtype], center=False, residual=False, bias=False, wide=True)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("width", [3, 64, 250, 513, 1000, 1025, 2048, 2050, 4095, 4100, 8192, 8200, 16384, 16390, 40001])
@pytest.mark.parametrize("rows", [3, 600])
def test_layer_norm_every_row_shape(vrc, dtype, width, rows):
    """Rows in one wave, in workgroups of each size and past a workgroup's registers,
    few and many of them, with and without elements behind the last vector."""
    if rows > 3 and width > 9000:
        rows = 515
    say(f"layer_norm rows {dtype} {rows} {width}")
    check_norm(vrc, "each", 1, rows, width, DT[dtype], residual=True)
    check_norm(vrc, "sum", 2, rows, width, DT[dtype], residual=False, bias=False, wide=True, center=False)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("join", JOINS)
@pytest.mark.parametrize("n,rows,width", [(1, 1, 1), (2, 1, 5), (3, 7, 8), (8, 1, 4096), (5, 13, 1053), (16, 40, 130), (4, 70, 512)])
def test_layer_norm_grad(vrc, join, dtype, n, rows, width):
    say(f"layer_norm_grad {join} {dtype} {n} {rows} {width}")
    check_norm_grad(vrc, join, n, rows, width, DT[dtype])
    check_norm_grad(vrc, join, n, rows, width, DT[dtype], center=False, bias=False, wide=True, residual=False)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("width", [3, 64, 250, 513, 1025, 2050, 4100, 8200, 16384, 16390, 20001])
@pytest.mark.parametrize("rows", [3, 1100])
def test_layer_norm_grad_every_row_shape(vrc, dtype, width, rows):
    say(f"layer_norm_grad rows {dtype} {rows} {width}")
    check_norm_grad(vrc, "each", 1, rows, width, DT[dtype])
    check_norm_grad(vrc, "sum", 2, min(rows, 30), width, DT[dtype], center=False, bias=False, wide=True)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("shift", [1, 3])
def test_layer_norm_operands_on_any_element(vrc, dtype, shift):
    for width in (1000, 1001):
        check_norm(vrc, "scatter", 3, 11, width, DT[dtype], shift=shift)
        check_norm_grad(vrc, "scatter", 3, 11, width, DT[dtype], shift=shift)
        check_norm(vrc, "sum", 2, 11, width, DT[dtype], shift=shift, wide=True)
        check_norm_grad(vrc, "sum", 2, 11, width, DT[dtype], shift=shift, wide=True)


# ---------------------------------------------------------------------------
# Cross entropy
# ---------------------------------------------------------------------------
def entropy_inputs(tokens, vocab, width, dtype, seed, ignored=0.2, shift=0):
    f = gen(seed)
    put = (lambda x: off_grid(x, shift)) if shift else (lambda x: x)
    hidden = put(f(tokens, width).to(dtype))
    weight = [put((f(v, width) * (2.0 / width**0.5)).to(dtype)) for v in vocab]
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + 7)
    target = torch.randint(0, max(1, sum(vocab)), (tokens,), generator=g, device=DEV)
    gone = torch.rand(tokens, generator=g, device=DEV) < ignored
    return hidden, weight, torch.where(gone, torch.full_like(target, IGNORE), target)


def check_entropy(vrc, tokens, vocab, width, dtype, seed=3, shift=0):
    hidden, weight, target = entropy_inputs(tokens, vocab, width, dtype, seed, shift=shift)
    loss, lse = vrc.vrc_cross_entropy(hidden, weight, target, ignore_index=IGNORE)
    rl, rs = ref.cross_entropy(hidden, weight, target, IGNORE)
    what = (tokens, vocab, width, str(dtype))
    close(lse, rs, what + ("lse",))
    close(loss, rl, what + ("loss",))
    none, again = vrc.vrc_cross_entropy(hidden, weight)
    assert none is None and torch.equal(again, lse)


def check_entropy_grad(vrc, tokens, vocab, width, dtype, seed=4, shift=0, weighted=True, scale=1.0):
    hidden, weight, target = entropy_inputs(tokens, vocab, width, dtype, seed, shift=shift)
    z, _ = ref.logits(hidden, weight)
    lse = torch.logsumexp(z, 1).float()
    f = gen(seed + 9)
    dloss = (f(tokens) * scale / tokens) if weighted else torch.full((tokens,), scale / tokens, device=DEV)
    dlse = f(tokens) * 0.1 * scale / tokens if weighted else None
    rh, rw = ref.cross_entropy_grad(hidden, weight, target, lse, dloss, dlse, IGNORE, dtype)
    dh, dw = vrc.vrc_cross_entropy_grad(hidden, weight, target, lse, dloss, dlse=dlse, ignore_index=IGNORE)
    what = (tokens, vocab, width, str(dtype))
    close(dh, rh, what + ("dhidden",))
    for r, (g, want) in enumerate(zip(dw, rw)):
        close(g, want, what + ("dweight", r))
    only, none = vrc.vrc_cross_entropy_grad(hidden, weight, target, lse, dloss, dlse=dlse, ignore_index=IGNORE, need_weight=False)
    assert none is None and torch.equal(only, dh)
    none, only = vrc.vrc_cross_entropy_grad(hidden, weight, target, lse, dloss, dlse=dlse, ignore_index=IGNORE, need_hidden=False)
    assert none is None and all(torch.equal(a, b) for a, b in zip(only, dw))


SIZES = [(1, [1], 1), (1, [5, 0, 3], 8), (2, [64], 64), (3, [100, 41], 40), (17, [257, 1, 300], 128), (32, [129], 200),
         (33, [300, 500], 64), (64, [1000], 129), (65, [130, 7], 256), (128, [513], 96), (129, [300, 301, 302], 100),
         (257, [700, 255], 192), (300, [256] * 16, 72), (600, [1025], 33)]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("tokens,vocab,width", SIZES)
def test_cross_entropy(vrc, dtype, tokens, vocab, width):
    say(f"cross_entropy {dtype} {tokens} {vocab} {width}")
    check_entropy(vrc, tokens, vocab, width, DT[dtype])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("tokens,vocab,width", SIZES)
def test_cross_entropy_grad(vrc, dtype, tokens, vocab, width):
    say(f"cross_entropy_grad {dtype} {tokens} {vocab} {width}")
    check_entropy_grad(vrc, tokens, vocab, width, DT[dtype])


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("width", [64, 65])
def test_cross_entropy_operands_on_any_element(vrc, dtype, width):
    for shift in (1, 8):
        check_entropy(vrc, 20, [70, 33], width, DT[dtype], shift=shift)
        check_entropy_grad(vrc, 20, [70, 33], width, DT[dtype], shift=shift)
