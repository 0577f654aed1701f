"""Python binding of include/vrc_model.h: a tensor-parallel model's operators
around its layers (``libvrc_ops.so``): layer norm in the collective before it,
the cross entropy over a vocabulary split over the ranks, and their gradients.

Conventions are those of ``ops``: one tensor per rank, HIP kernels on the current
(or the given) stream, nothing recorded by autograd.  Workspaces come from torch's
allocator for the stream that the call runs on."""
from __future__ import annotations

import ctypes as C
from math import prod as _prod

from . import MAX_RANKS, _check_ranks, _torch
from .ops import _allocate, _chunk_sizes, _done, _float_code, _on, _ops, _outputs, _pointers

NORM_JOINS = {"each": 0, "sum": 1, "scatter": 2}


class LayerNorm(C.Structure):
    """vrc_layer_norm_t of include/vrc_model.h."""
    _fields_ = [("rows", C.c_size_t), ("width", C.c_size_t), ("dtype", C.c_int), ("wdtype", C.c_int), ("join", C.c_int),
                ("center", C.c_int), ("eps", C.c_double)]


class CrossEntropy(C.Structure):
    """vrc_cross_entropy_t of include/vrc_model.h."""
    _fields_ = [("tokens", C.c_size_t), ("width", C.c_size_t), ("vocab", C.POINTER(C.c_size_t)), ("dtype", C.c_int),
                ("ignore_index", C.c_longlong)]


def _bind():
    vp, sz, i = C.c_void_p, C.c_size_t, C.c_int
    ptrs, norm, ce, size = C.POINTER(C.c_void_p), C.POINTER(LayerNorm), C.POINTER(CrossEntropy), C.POINTER(C.c_size_t)
    for name, args in (
            ("vrc_layer_norm", [norm, ptrs, ptrs, vp, vp, ptrs, ptrs, ptrs, ptrs, i, vp]),
            ("vrc_layer_norm_grad", [norm, ptrs, ptrs, ptrs, ptrs, vp, ptrs, ptrs, vp, vp, i, vp, sz, vp]),
            ("vrc_layer_norm_grad_workspace", [norm, i, size]),
            ("vrc_cross_entropy", [ce, vp, ptrs, vp, vp, vp, i, vp, sz, vp]),
            ("vrc_cross_entropy_workspace", [ce, vp, ptrs, i, size]),
            ("vrc_cross_entropy_grad", [ce, vp, ptrs, vp, vp, vp, vp, vp, ptrs, i, vp, sz, vp]),
            ("vrc_cross_entropy_grad_workspace", [ce, vp, ptrs, i, i, size])):
        f = getattr(_ops, name)
        f.argtypes, f.restype = args, i


_bind()


def _on_stream(stream, make):
    """What `make` allocates, of the pool of the stream that the call runs on."""
    if stream is None:
        return make()
    with _torch().cuda.stream(stream):
        return make()


def _same(t, shape, dtype, at, where, what):
    """Check one contiguous tensor of a shape (its number of elements), type and device."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{where}: {what} must be a tensor")
    if t.dtype is not dtype or t.numel() != _prod(shape) or t.get_device() != at or not t.is_contiguous():
        raise ValueError(f"{where}: {what} must be contiguous {tuple(shape)} {dtype} on the inputs' device")
    return t


def _parts(ts, shapes, dtype, at, where, what, one):
    """A list of one tensor per part; a single tensor where all ranks share it."""
    torch = _torch()
    if one:
        return [_same(ts, shapes[0], dtype, at, where, what)]
    if isinstance(ts, torch.Tensor) or not isinstance(ts, (list, tuple)) or len(ts) != len(shapes):
        raise ValueError(f"{where}: {what} must be one tensor per rank")
    for t, s in zip(ts, shapes):
        _same(t, s, dtype, at, where, what)
    return ts


def _norm_shapes(send, join, where):
    """(shape of every send, rows, width, shapes of the parts, shapes of the outputs)."""
    shape = tuple(send[0].shape)
    if not shape:
        raise ValueError("tensors need at least one dimension")
    rows, width, n = _prod(shape[:-1]), shape[-1], len(send)
    if join == "scatter":
        parts = [(k, width) for k in _chunk_sizes(rows, n)]
        return shape, rows, width, parts, parts
    return shape, rows, width, [shape] * (1 if join == "sum" else n), [shape] * n


def _norm_weight(weight, width, dtype, at, where):
    torch = _torch()
    if not isinstance(weight, torch.Tensor) or weight.dtype not in (dtype, torch.float32):
        raise TypeError(f"{where}: weight must be a tensor of the rows' dtype or float32")
    return _same(weight, (width,), weight.dtype, at, where, "weight")


def _join(join):
    if join not in NORM_JOINS:
        raise ValueError(f"join must be one of {sorted(NORM_JOINS)}")
    return NORM_JOINS[join]


def vrc_layer_norm(send, weight, bias=None, eps=1e-5, residual=None, join="each", center=True, recv=None, sum=None,
                   stream=None):
    """(y, h, mean, rstd): layer norm over the last dimension (``center=False``: RMS
    norm), y = (h - mean) rstd weight + bias, of the rows that ``join`` names:

    * ``"each"``: rank r's own, h[r] = send[r] + residual[r]; y, h, mean and rstd are
      lists of one tensor per rank;
    * ``"sum"``: the all-reduced rows, h = sum over ranks of send[r] + residual (one
      tensor); y is one tensor per rank, h, mean and rstd are single tensors;
    * ``"scatter"``: rank c's rows of that sum (equal runs of the rows, the last rank with
      the remainder) + residual[c]; lists of one [rows of c, width] tensor per rank.

    ``weight`` and ``bias`` are of the rows' dtype or float32.  h is rounded from the
    fp32 values that y is computed from (without anything added, ``"each"`` returns
    ``send`` itself); mean and rstd are float32, one per row, mean None where not
    centred.  ``recv=send`` (not for ``"scatter"``) and ``sum=residual``, where h goes,
    run in place.  Gradient: ``vrc_layer_norm_grad``."""
    where = "vrc_layer_norm"
    torch = _torch()
    code = _join(join)
    dev = _check_ranks(send, where)
    x0, n, one = send[0], len(send), join == "sum"
    dtype, at = x0.dtype, x0.get_device()
    dt = _float_code(dtype, where)
    shape, rows, width, parts, outs = _norm_shapes(send, join, where)
    _norm_weight(weight, width, dtype, at, where)
    if bias is not None:
        _same(bias, (width,), weight.dtype, at, where, "bias")
    res = None if residual is None else _pointers(_parts(residual, parts, dtype, at, where, "residual", one))
    d = LayerNorm(rows, width, dt, _float_code(weight.dtype, where), code, bool(center), eps)
    st = _on(stream, dev, where)
    added = residual is not None or join != "each"
    if sum is not None and not added:
        raise ValueError(f"{where}: without a residual each rank's rows are their own sum")
    y = _outputs(recv, outs, x0, where, stream)
    h = send
    if sum is not None:
        h = _parts(sum, parts, dtype, at, where, "sum", one)
    elif added:
        h = _on_stream(stream, lambda: _allocate(parts, dtype, x0.device))
    lines = [s[:-1] for s in parts]
    count = len(lines) * (2 if center else 1)
    stats = _on_stream(stream, lambda: _allocate((lines * 2)[:count], torch.float32, x0.device))
    rstd, mean = stats[:len(lines)], stats[len(lines):]
    _done(_ops.vrc_layer_norm(C.byref(d), _pointers(send), res, weight.data_ptr(), None if bias is None else bias.data_ptr(),
                              _pointers(y), _pointers(h) if added else None, _pointers(mean) if center else None,
                              _pointers(rstd), n, st or None), where)
    if one:
        return y, h[0], mean[0] if center else None, rstd[0]
    return y, h, mean if center else None, rstd


def vrc_layer_norm_grad(dy, h, weight, mean, rstd, dh=None, join="each", bias=True, recv=None, stream=None):
    """(dx, dweight, dbias): the gradients of ``vrc_layer_norm`` with the same ``join``,
    from those of its outputs y and the h, mean (None: RMS norm) and rstd it returned.

    ``dy``: one tensor per rank: of rank r's own rows (``"each"``), or each rank's part
    of the gradient of all rows, which are summed (``"sum"``, ``"scatter"``).
    ``dh``: None, or what reaches h by the residual stream and is added to dx: one
    tensor per rank, a single tensor for ``"sum"``.
    dx: one tensor per rank: the gradient of rank r's send and residual (``"each"``); that
    of every send and of the residual (``"sum"``); that of residual c, and by
    ``vrc_all_gather`` of every send (``"scatter"``).  dweight and dbias (None where
    ``bias`` is false) are single tensors of the weight's dtype, summed over all rows of
    all ranks, in a fixed order.  ``recv=dy`` (not for ``"scatter"``) runs in place."""
    where = "vrc_layer_norm_grad"
    torch = _torch()
    code = _join(join)
    dev = _check_ranks(dy, where)
    x0, n, one = dy[0], len(dy), join == "sum"
    dtype, at = x0.dtype, x0.get_device()
    dt = _float_code(dtype, where)
    shape, rows, width, parts, outs = _norm_shapes(dy, join, where)
    _norm_weight(weight, width, dtype, at, where)
    h = _parts(h, parts, dtype, at, where, "h", one)
    lines = [s[:-1] for s in parts]
    mean_ = None if mean is None else _parts(mean, lines, torch.float32, at, where, "mean", one)
    rstd = _parts(rstd, lines, torch.float32, at, where, "rstd", one)
    res = None if dh is None else _pointers(_parts(dh, parts, dtype, at, where, "dh", one))
    d = LayerNorm(rows, width, dt, _float_code(weight.dtype, where), code, mean is not None, 0.0)
    st = _on(stream, dev, where)
    size = C.c_size_t()
    _done(_ops.vrc_layer_norm_grad_workspace(C.byref(d), n, C.byref(size)), where)
    dx = _outputs(recv, outs, x0, where, stream)

    def make():
        grads = _allocate([(width,)] * (2 if bias else 1), weight.dtype, x0.device)
        return grads, torch.empty(size.value, dtype=torch.uint8, device=x0.device)

    grads, space = _on_stream(stream, make)
    _done(_ops.vrc_layer_norm_grad(C.byref(d), _pointers(dy), _pointers(h), None if mean_ is None else _pointers(mean_),
                                   _pointers(rstd), weight.data_ptr(), res, _pointers(dx), grads[0].data_ptr(),
                                   grads[1].data_ptr() if bias else None, n, space.data_ptr() or None, size.value,
                                   st or None), where)
    return dx, grads[0], grads[1] if bias else None


def _entropy(hidden, weight, target, ignore_index, where):
    """The checked call: (description, device index, pointers of the weights, tokens)."""
    torch = _torch()
    if not isinstance(weight, (list, tuple)) or not 1 <= len(weight) <= MAX_RANKS:
        raise ValueError(f"{where}: weight must be one tensor per rank, {MAX_RANKS} at most")
    dev = _check_ranks([hidden], where)
    if hidden.dim() == 0 or hidden.shape[-1] == 0:
        raise ValueError(f"{where}: hidden must be [..., width]")
    width, at, dtype = hidden.shape[-1], hidden.get_device(), hidden.dtype
    dt = _float_code(dtype, where)
    for r, w in enumerate(weight):
        if not isinstance(w, torch.Tensor) or w.dim() != 2 or w.shape[1] != width:
            raise ValueError(f"{where}: weight {r} must be [vocabulary of the rank, {width}]")
        if w.dtype is not dtype or w.get_device() != at or not w.is_contiguous():
            raise ValueError(f"{where}: weight {r} must be contiguous {dtype} on {hidden.device}")
    lead = tuple(hidden.shape[:-1])
    if target is not None:
        if not isinstance(target, torch.Tensor) or target.dtype is not torch.int64 or tuple(target.shape) != lead:
            raise ValueError(f"{where}: target must be int64 {lead}")
        if target.get_device() != at or not target.is_contiguous():
            raise ValueError(f"{where}: target must be contiguous on {hidden.device}")
    if not -(1 << 63) <= ignore_index < 1 << 63:
        raise ValueError(f"{where}: ignore_index must be a signed 64-bit number")
    vocab = (C.c_size_t * len(weight))(*[w.shape[0] for w in weight])
    return CrossEntropy(_prod(lead), width, vocab, dt, ignore_index), dev, lead


def _space(query, where, device):
    size = C.c_size_t()
    _done(query(C.byref(size)), where)
    return _torch().empty(size.value, dtype=_torch().uint8, device=device)


def vrc_cross_entropy(hidden, weight, target=None, ignore_index=-100, stream=None):
    """(loss, lse), float32 of hidden's leading shape: the cross entropy of the logits
    z = hidden W^T, W being the concatenation of the ranks' ``weight[r]`` ([rows of the
    vocabulary that rank r holds, width]; any numbers of rows), without keeping them:
    lse = log sum exp z, loss = lse - z[target].

    ``hidden`` [..., width] is shared by all ranks; ``target`` int64 of its leading
    shape, or None for lse alone (loss is None then).  A token whose target is
    ``ignore_index`` has loss 0, one whose target is otherwise outside the vocabulary NaN.
    Gradient: ``vrc_cross_entropy_grad``."""
    where = "vrc_cross_entropy"
    torch = _torch()
    d, dev, lead = _entropy(hidden, weight, target, ignore_index, where)
    st = _on(stream, dev, where)
    ptrs, n = _pointers(weight), len(weight)

    def make():
        out = _allocate([lead] * (1 if target is None else 2), torch.float32, hidden.device)
        return out, _space(lambda size: _ops.vrc_cross_entropy_workspace(C.byref(d), hidden.data_ptr(), ptrs, n, size), where,
                           hidden.device)

    out, space = _on_stream(stream, make)
    loss = None if target is None else out[1]
    _done(_ops.vrc_cross_entropy(C.byref(d), hidden.data_ptr(), ptrs, None if target is None else target.data_ptr(),
                                 None if loss is None else loss.data_ptr(), out[0].data_ptr(), n, space.data_ptr() or None,
                                 space.numel(), st or None), where)
    return loss, out[0]


def vrc_cross_entropy_grad(hidden, weight, target, lse, dloss, dlse=None, ignore_index=-100, need_hidden=True,
                           need_weight=True, recv=None, stream=None):
    """(dhidden, dweight): the gradients of ``vrc_cross_entropy`` from those of its loss
    and (``dlse``, or None) of its lse: float32 of hidden's leading shape, contiguous.

    dhidden, like hidden, is summed over the ranks; dweight is one tensor per rank.
    ``need_hidden=False`` and ``need_weight=False`` (a frozen projection) leave one
    out, as None.  Tokens whose dloss (or target: ``ignore_index``) and dlse leave
    nothing get zeros and add nothing to dweight, whatever their hidden states hold.
    ``recv``: (dhidden, list of dweight) to write to."""
    where = "vrc_cross_entropy_grad"
    torch = _torch()
    if target is None:
        raise ValueError(f"{where}: target is missing")
    d, dev, lead = _entropy(hidden, weight, target, ignore_index, where)
    at, n = hidden.get_device(), len(weight)
    for t, what in ((lse, "lse"), (dloss, "dloss")) + (() if dlse is None else ((dlse, "dlse"),)):
        _same(t, lead, torch.float32, at, where, what)
    st = _on(stream, dev, where)
    out_h, out_w = (None, None) if recv is None else recv
    dh = _outputs(None if out_h is None else [out_h], [tuple(hidden.shape)], hidden, where, stream)[0] if need_hidden else None
    dw = _outputs(out_w, [tuple(w.shape) for w in weight], hidden, where, stream) if need_weight else None
    ptrs = _pointers(weight)
    space = _on_stream(stream, lambda: _space(
        lambda size: _ops.vrc_cross_entropy_grad_workspace(C.byref(d), hidden.data_ptr(), ptrs, need_hidden, n, size), where,
        hidden.device))
    _done(_ops.vrc_cross_entropy_grad(C.byref(d), hidden.data_ptr(), ptrs, target.data_ptr(), lse.data_ptr(), dloss.data_ptr(),
                                      None if dlse is None else dlse.data_ptr(), None if dh is None else dh.data_ptr(),
                                      None if dw is None else _pointers(dw), n, space.data_ptr() or None, space.numel(),
                                      st or None), where)
    return dh, dw


__all__ = ["vrc_layer_norm", "vrc_layer_norm_grad", "vrc_cross_entropy", "vrc_cross_entropy_grad", "LayerNorm",
           "CrossEntropy", "NORM_JOINS"]
