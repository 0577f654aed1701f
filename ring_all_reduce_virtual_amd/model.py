"""Python binding of include/vrc_model.h: a tensor-parallel model's operators
around its layers (``libvrc_ops.so``): layer norm in the collective before it,
the cross entropy over a vocabulary split over the ranks, and their gradients.

Conventions are those of ``ops``: one tensor per rank, HIP kernels on the current
(or the given) stream, nothing recorded by autograd.  Workspaces come from torch's
allocator for the stream that the call runs on.  The functions here document the
calls; a compiled module (``_vrc_model.so``, csrc_ops/vrc_model_binding.cpp) checks
the tensors, allocates and calls the library."""
from __future__ import annotations

import ctypes as C
import importlib.machinery
import importlib.util
import os
import threading

from . import PKG, VRC_OK, VrcError, _stream, _torch
from .ops import OPS_VERSION, _on, _ops

NORM_JOINS = {"each": 0, "sum": 1, "scatter": 2}
MODEL_BINDING_PATH = os.path.join(PKG, "_vrc_model.so")


class LayerNorm(C.Structure):
    """vrc_layer_norm_t of include/vrc_model.h."""
    _fields_ = [("rows", C.c_size_t), ("width", C.c_size_t), ("dtype", C.c_int), ("wdtype", C.c_int), ("join", C.c_int),
                ("center", C.c_int), ("eps", C.c_double)]


class CrossEntropy(C.Structure):
    """vrc_cross_entropy_t of include/vrc_model.h."""
    _fields_ = [("tokens", C.c_size_t), ("width", C.c_size_t), ("vocab", C.POINTER(C.c_size_t)), ("dtype", C.c_int),
                ("ignore_index", C.c_longlong)]


def _bind():
    """The C ABI, for those that call it without torch."""
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


def _failed(status: int, where: str):
    if status != VRC_OK:
        raise VrcError(status, where, _ops.vrc_ops_last_hip_error())


_module = None
_loading = threading.Lock()


def _native():
    """The compiled module, loaded by the first call (it needs torch, as the tensors do)."""
    return _module or _load()


def _load():
    global _module
    with _loading:
        if _module is not None:
            return _module
        torch = _torch()
        if not os.path.exists(MODEL_BINDING_PATH):
            raise ImportError(f"{MODEL_BINDING_PATH} is missing: build the HIP libraries first "
                              "(python ring_all_reduce_virtual_amd/build.py, or __graft_entry__.build())")
        loader = importlib.machinery.ExtensionFileLoader("_vrc_model", MODEL_BINDING_PATH)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_vrc_model", loader))
        loader.exec_module(module)
        version = module.init(lambda device: _stream(None, device), _failed, torch.cuda.OutOfMemoryError)
        if version != OPS_VERSION:
            raise ImportError(f"{MODEL_BINDING_PATH} reports version {version}, this binding needs {OPS_VERSION}: rebuild it")
        _module = module
        return module


def _run(call, where, first, stream, args):
    """The call on the current stream of the tensors' device, or, with what it allocates, on `stream`."""
    if stream is None:
        return call(*args, None)
    first = first[0] if isinstance(first, (list, tuple)) and first else first
    torch = _torch()
    if not isinstance(first, torch.Tensor) or not first.is_cuda:
        return call(*args, 0)  # which refuses them
    handle = _on(stream, first.get_device(), where)
    with torch.cuda.stream(stream):
        return call(*args, handle)


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
    ``send`` itself, or None where ``recv`` overwrites it); mean and rstd are float32, one per row, mean None where not
    centred; rows need at least one value.  ``recv=send`` (not for ``"scatter"``) and ``sum=residual``, where h goes,
    run in place.  Gradient: ``vrc_layer_norm_grad``."""
    return _run(_native().layer_norm, "vrc_layer_norm", send, stream,
                (send, weight, bias, eps, residual, _join(join), center, recv, sum))


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
    return _run(_native().layer_norm_grad, "vrc_layer_norm_grad", dy, stream,
                (dy, h, weight, mean, rstd, dh, _join(join), bias, recv))


def vrc_cross_entropy(hidden, weight, target=None, ignore_index=-100, stream=None):
    """(loss, lse), float32 of hidden's leading shape: the cross entropy of the logits
    z = hidden W^T, W being the concatenation of the ranks' ``weight[r]`` ([rows of the
    vocabulary that rank r holds, width]; any numbers of rows), without keeping them:
    lse = log sum exp z, loss = lse - z[target].

    ``hidden`` [..., width] is shared by all ranks; ``target`` int64 of its leading
    shape, or None for lse alone (loss is None then).  A token whose target is
    ``ignore_index`` has loss 0, one whose target is otherwise outside the vocabulary NaN.
    Gradient: ``vrc_cross_entropy_grad``."""
    return _run(_native().cross_entropy, "vrc_cross_entropy", hidden, stream, (hidden, weight, target, ignore_index))


def vrc_cross_entropy_grad(hidden, weight, target, lse, dloss, dlse=None, ignore_index=-100, need_hidden=True,
                           need_weight=True, recv=None, stream=None):
    """(dhidden, dweight): the gradients of ``vrc_cross_entropy`` from those of its loss
    and (``dlse``, or None) of its lse: float32 of hidden's leading shape, contiguous.

    dhidden, like hidden, is summed over the ranks; dweight is one tensor per rank.
    ``need_hidden=False`` and ``need_weight=False`` (a frozen projection) leave one
    out, as None.  Tokens whose dloss (or target: ``ignore_index``) and dlse leave
    nothing get zeros and add nothing to dweight, whatever their hidden states and targets
    hold.  Any other token whose target is outside the vocabulary makes its row of dhidden
    and all of dweight NaN.  16-bit types round the gradients of the logits on the way, fp16
    in one range for the whole call: include/vrc_model.h has what that keeps of tokens that
    weigh little.
    ``recv``: (dhidden, list of dweight) to write to."""
    dhidden, dweight = (None, None) if recv is None else recv
    return _run(_native().cross_entropy_grad, "vrc_cross_entropy_grad", hidden, stream,
                (hidden, weight, target, lse, dloss, dlse, ignore_index, need_hidden, need_weight, dhidden, dweight))


__all__ = ["vrc_layer_norm", "vrc_layer_norm_grad", "vrc_cross_entropy", "vrc_cross_entropy_grad", "LayerNorm",
           "CrossEntropy", "NORM_JOINS", "MODEL_BINDING_PATH"]
