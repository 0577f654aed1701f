"""Python binding of include/vrc_ops.h: the tensor-parallel layer's operators
over virtual ranks (``libvrc_ops.so``).

Like the collectives' functions these take one tensor per rank, check shapes
and marshal pointers and the current HIP stream; the computation runs in HIP
kernels.  Where a ``stream`` is given, outputs that the call allocates belong
to that stream's pool.  As with the collectives, autograd records none of the
calls: outputs require no gradients, and each call's docstring names the calls
that compute its gradients."""
from __future__ import annotations

import ctypes as C
import os

from math import prod as _prod

from . import (MAX_RANKS, PKG, VRC_BF16, VRC_FP16, VRC_FP32, VRC_OK, VrcError, _check_ranks, _outer, _stream, _torch,
               reduce_scatter_shape)

OPS_LIB_PATH = os.path.join(PKG, "libvrc_ops.so")
OPS_VERSION = 101  # VRC_OPS_VERSION of include/vrc_ops.h that this binding follows
MX4_BLOCK = 32     # values that share a scale
MX4_ALONG_COLS, MX4_ALONG_ROWS = 0, 1
MX4_JOINS = {"sum": 0, "each": 1}


class Dropout(C.Structure):
    """vrc_dropout_t of include/vrc_ops.h."""
    _fields_ = [("p", C.c_double), ("seed", C.c_ulonglong), ("offset", C.c_ulonglong), ("offset_dev", C.c_void_p)]


def _load():
    if not os.path.exists(OPS_LIB_PATH):
        raise ImportError(
            f"{OPS_LIB_PATH} is missing: build the HIP libraries first "
            "(python ring_all_reduce_virtual_amd/build.py, or __graft_entry__.build())")
    L = C.CDLL(OPS_LIB_PATH)
    vp, sz, i = C.c_void_p, C.c_size_t, C.c_int
    ptrs, drop = C.POINTER(C.c_void_p), C.POINTER(Dropout)
    L.vrc_allreduce_dropout.argtypes = [ptrs, ptrs, ptrs, i, sz, i, drop, vp]
    L.vrc_reduce_scatter_dropout.argtypes = [ptrs, ptrs, ptrs, i, sz, sz, i, drop, vp]
    L.vrc_all_gather_dropout.argtypes = [ptrs, ptrs, i, sz, sz, i, drop, vp]
    L.vrc_mx4_quantize.argtypes = [ptrs, ptrs, ptrs, i, sz, sz, i, i, vp]
    L.vrc_mx4_dequantize.argtypes = [ptrs, ptrs, ptrs, i, sz, sz, i, vp]
    L.vrc_mx4_all_gather.argtypes = [ptrs, ptrs, ptrs, i, sz, sz, i, i, vp]
    L.vrc_mx4_matmul.argtypes = [ptrs, ptrs, ptrs, ptrs, ptrs, i, sz, sz, sz, i, i, vp]
    for f in ("vrc_allreduce_dropout", "vrc_reduce_scatter_dropout", "vrc_all_gather_dropout", "vrc_mx4_quantize",
              "vrc_mx4_dequantize", "vrc_mx4_all_gather", "vrc_mx4_matmul", "vrc_ops_last_hip_error",
              "vrc_ops_version"):
        getattr(L, f).restype = i
    L.vrc_ops_last_hip_error.argtypes = []
    L.vrc_ops_version.argtypes = []
    if L.vrc_ops_version() != OPS_VERSION:
        raise ImportError(f"{OPS_LIB_PATH} reports version {L.vrc_ops_version()}, this binding needs {OPS_VERSION}: "
                          "rebuild the library")
    return L


_ops = _load()


def ops_lib() -> C.CDLL:
    """The loaded libvrc_ops.so."""
    return _ops


def _on(stream, dev: int, where: str) -> int:
    """The HIP stream to enqueue on (see ``_stream``), which must be on the tensors' device."""
    if stream is not None and stream.device_index != dev:
        raise ValueError(f"{where}: the stream is on cuda:{stream.device_index}, the tensors on cuda:{dev}")
    return _stream(stream, dev)


def _done(status: int, where: str):
    if status != VRC_OK:
        raise VrcError(status, where, _ops.vrc_ops_last_hip_error())


_POINTERS = [C.c_void_p * n for n in range(MAX_RANKS + 1)]


def _pointers(tensors):
    return _POINTERS[len(tensors)](*[t.data_ptr() for t in tensors])


def _allocate(shapes, dtype, device):
    """New outputs, each with a storage of its own: parts of one allocation would take
    half the host time (5 us for eight instead of 10), but one that grows in place
    would grow over the others, and keeping or saving one would keep or write them all."""
    torch = _torch()
    first, like = shapes[0], torch.empty_like
    t0 = torch.empty(first, dtype=dtype, device=device)
    return [t0] + [like(t0) if s == first else torch.empty(s, dtype=dtype, device=device) for s in shapes[1:]]


def _outputs(recv, shapes, like, where, stream, dtype=None):
    """`recv` checked against one shape per rank, or new tensors.  Those belong to
    `stream` if one is given: a block of another stream's pool might still be in use
    there."""
    dtype = like.dtype if dtype is None else dtype
    n, device = len(shapes), like.device
    if recv is None:
        if stream is None:
            return _allocate(shapes, dtype, device)
        with _torch().cuda.stream(stream):
            return _allocate(shapes, dtype, device)
    if not isinstance(recv, (list, tuple)) or len(recv) != n:
        raise ValueError(f"{where}: one output per rank")
    at = like.get_device()
    for c, (t, s) in enumerate(zip(recv, shapes)):
        if t.dtype is not dtype or t.numel() != _prod(s) or not t.is_contiguous():
            raise ValueError(f"{where}: output {c} must be contiguous {tuple(s)} {dtype}")
        if t.get_device() != at:
            raise ValueError(f"{where}: outputs must be on the inputs' device {device}")
    return recv


_CODES: dict = {}  # torch dtype -> vrc_dtype_t, filled by the first call


def _float_code(dtype, where) -> int:
    if not _CODES:
        torch = _torch()
        _CODES.update({torch.float32: VRC_FP32, torch.float16: VRC_FP16, torch.bfloat16: VRC_BF16})
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"{where}: unsupported dtype {dtype}")
    return code


def _chunk_sizes(count: int, n: int) -> list:
    """The lengths of vrc_chunk_range's chunks: equal ones, the last with the remainder."""
    return [count // n] * (n - 1) + [count - (n - 1) * (count // n)]


def _dropout(p, seed, offset, device, where) -> Dropout:
    """`offset`: a number, or a one-element int64 CUDA tensor that the kernel
    reads when it runs (for graphs that draw a new mask at every replay)."""
    torch = _torch()
    if not 0 <= seed < 1 << 64:
        raise ValueError(f"{where}: seed must be an unsigned 64-bit number")
    if isinstance(offset, torch.Tensor):
        if offset.dtype != torch.int64 or offset.numel() != 1 or offset.device != device:
            raise ValueError(f"{where}: a tensor offset must be one int64 on {device}")
        return Dropout(p, seed, 0, offset.data_ptr())
    if not 0 <= offset < 1 << 64:
        raise ValueError(f"{where}: offset must be an unsigned 64-bit number")
    return Dropout(p, seed, offset, None)


def _residuals(residual, shapes, like, where):
    if not isinstance(residual, (list, tuple)) or len(residual) != len(shapes):
        raise ValueError(f"{where}: one residual per rank")
    dtype, at = like.dtype, like.get_device()
    for c, (t, s) in enumerate(zip(residual, shapes)):
        if t.numel() != _prod(s) or t.dtype is not dtype or t.get_device() != at or not t.is_contiguous():
            raise ValueError(f"{where}: residual {c} must be contiguous {tuple(s)} {like.dtype} on {like.device}")
    return residual


def vrc_allreduce_dropout(send, p, seed, offset=0, residual=None, recv=None, stream=None):
    """recv[r] = residual[r] + dropout(sum over ranks of send[r]), every rank.

    ``residual``: None, one tensor per rank, or a single tensor for all ranks.
    ``recv=send`` and ``recv=residual`` (a list) run in place.  The mask is a
    function of (p, seed, offset) and the element's index.

    Gradient: of every send, this call over the outputs' gradients with the same
    (p, seed, offset) and no residual; of a residual, its output's gradient (of a
    single one, their all-reduce)."""
    where = "vrc_allreduce_dropout"
    torch = _torch()
    dev = _check_ranks(send, where)
    code = _float_code(send[0].dtype, where)
    n = len(send)
    shape = tuple(send[0].shape)
    shapes = [shape] * n
    res = None
    if isinstance(residual, torch.Tensor):
        _residuals([residual], [shape], send[0], where)
        res = _POINTERS[n](*[residual.data_ptr()] * n)
    elif residual is not None:
        res = _pointers(_residuals(residual, shapes, send[0], where))
    drop = _dropout(p, seed, offset, send[0].device, where)
    st = _on(stream, dev, where)
    recv = _outputs(recv, shapes, send[0], where, stream)
    _done(_ops.vrc_allreduce_dropout(_pointers(send), res, _pointers(recv), n, send[0].numel(), code, C.byref(drop),
                                     st or None), where)
    return recv


def vrc_reduce_scatter_dropout(send, p, seed, offset=0, residual=None, dim=0, recv=None, stream=None):
    """recv[c] = residual[c] + chunk c of dropout(sum over ranks of send[r]); the
    chunks are those of ``vrc_reduce_scatter``, the mask that of the unsplit tensor.

    ``residual``: None or one tensor per rank, laid out as recv; ``recv=residual``
    runs in place.  Gradient: of every send, ``vrc_all_gather_dropout`` of the
    outputs' gradients with the same (p, seed, offset)."""
    where = "vrc_reduce_scatter_dropout"
    dev = _check_ranks(send, where)
    code = _float_code(send[0].dtype, where)
    outer, _ = _outer(send[0].shape, dim)
    n, shape = len(send), tuple(send[0].shape)
    shapes = [(k,) for k in _chunk_sizes(_prod(shape), n)] if outer == 1 else reduce_scatter_shape(shape, n, dim)
    if residual is not None:
        _residuals(residual, shapes, send[0], where)
    drop = _dropout(p, seed, offset, send[0].device, where)
    st = _on(stream, dev, where)
    recv = _outputs(recv, shapes, send[0], where, stream)
    if send[0].numel() == 0:
        return recv
    _done(_ops.vrc_reduce_scatter_dropout(_pointers(send), None if residual is None else _pointers(residual),
                                          _pointers(recv), n, send[0].numel(), outer, code, C.byref(drop),
                                          st or None), where)
    return recv


def vrc_all_gather_dropout(send, p, seed, offset=0, dim=0, recv=None, stream=None):
    """recv[r] = dropout(concatenation of all send tensors along ``dim``), every
    rank; one tensor's elements are numbered as in the concatenation.

    One-dimensional inputs may also be the uneven chunks of a flat tensor (the last
    one takes the remainder), as ``vrc_reduce_scatter_dropout`` returns them.
    Gradient: of each send, its chunk of ``vrc_reduce_scatter_dropout`` of the
    outputs' gradients with the same (p, seed, offset)."""
    where = "vrc_all_gather_dropout"
    n = len(send) if isinstance(send, (list, tuple)) else 0
    if n > 1 and send[0].dim() == 1 and send[-1].dim() == 1 and send[-1].shape != send[0].shape:
        dev = _check_ranks(send[:-1], where)
        _check_ranks(send[-1:], where)
        total = sum(t.numel() for t in send)
        if [t.numel() for t in send] != _chunk_sizes(total, n):
            raise ValueError(f"{where}: uneven inputs must be the chunks of a flat tensor, the last with the remainder")
        if send[-1].dtype != send[0].dtype or send[-1].device != send[0].device:
            raise ValueError(f"{where}: all ranks need the same dtype and device")
        _outer(send[0].shape, dim)
        outer, shape = 1, (total,)
    else:
        dev = _check_ranks(send, where)
        outer, d = _outer(send[0].shape, dim)
        shape = list(send[0].shape)
        shape[d] *= n
        total = _prod(shape)
    code = _float_code(send[0].dtype, where)
    drop = _dropout(p, seed, offset, send[0].device, where)
    st = _on(stream, dev, where)
    recv = _outputs(recv, [tuple(shape)] * n, send[0], where, stream)
    if total == 0:
        return recv
    _done(_ops.vrc_all_gather_dropout(_pointers(send), _pointers(recv), n, total, outer, code, C.byref(drop),
                                      st or None), where)
    return recv


# ---------------------------------------------------------------------------
# Microscaled 4-bit matrices
# ---------------------------------------------------------------------------
def mx4_blocks(cols: int) -> int:
    """Blocks that a row of `cols` values is held in."""
    return -(-cols // MX4_BLOCK)


def vrc_mx4_quantize(x, dim=-1, codes=None, scales=None, stream=None):
    """(codes, scales), one uint8 tensor per rank each: x[r] as blocks of 32 4-bit
    values with one scale.

    ``dim=-1``: blocks along the last dimension; codes are [..., 16 KB] and scales
    [..., KB] with KB = ceil(cols / 32).  ``dim=0`` (matrices only): blocks down the
    columns, stored as the transposed matrix's rows: [cols, 16 KB], KB = ceil(rows / 32)."""
    where = "vrc_mx4_quantize"
    torch = _torch()
    dev = _check_ranks(x, where)
    code = _float_code(x[0].dtype, where)
    shape = tuple(x[0].shape)
    if not shape:
        raise ValueError("tensors need at least one dimension")
    cols = shape[-1]
    rows = _prod(shape[:-1])
    if dim in (-1, len(shape) - 1):
        lead, kb, axis = shape[:-1], mx4_blocks(cols), MX4_ALONG_COLS
    elif dim == 0 and len(shape) == 2 or dim == -2 and len(shape) == 2:
        lead, kb, axis = (cols,), mx4_blocks(rows), MX4_ALONG_ROWS
    else:
        raise ValueError(f"{where}: dim must be the last dimension, or the first of a matrix")
    st = _on(stream, dev, where)
    codes = _outputs(codes, [lead + (kb * 16,)] * len(x), x[0], where, stream, torch.uint8)
    scales = _outputs(scales, [lead + (kb,)] * len(x), x[0], where, stream, torch.uint8)
    _done(_ops.vrc_mx4_quantize(_pointers(x), _pointers(codes), _pointers(scales), len(x), rows, cols, code, axis,
                                st or None), where)
    return codes, scales


def _quantised(codes, scales, where):
    """(leading shape, blocks per row, device index) of one matrix per rank."""
    torch = _torch()
    dev = _check_ranks(codes, where)
    if _check_ranks(scales, where) != dev or len(scales) != len(codes):
        raise ValueError(f"{where}: one scales tensor per codes tensor, on its device")
    if codes[0].dtype is not torch.uint8 or scales[0].dtype is not torch.uint8:
        raise TypeError(f"{where}: codes and scales are uint8")
    lead, kb = tuple(scales[0].shape[:-1]), scales[0].shape[-1] if scales[0].dim() else 0
    if scales[0].dim() == 0 or tuple(codes[0].shape) != lead + (kb * 16,):
        raise ValueError(f"{where}: codes must be [..., 16 KB] beside scales [..., KB]")
    return lead, kb, dev


def _decoded_cols(cols, kb, where) -> int:
    cols = kb * MX4_BLOCK if cols is None else cols
    if mx4_blocks(cols) != kb:
        raise ValueError(f"{where}: rows of {kb} blocks do not hold {cols} values")
    return cols


def vrc_mx4_dequantize(codes, scales, cols=None, dtype=None, recv=None, stream=None):
    """recv[r] = the [..., cols] values of rank r's codes (``cols=None``: whole
    blocks), in ``dtype`` (default bfloat16)."""
    where = "vrc_mx4_dequantize"
    torch = _torch()
    dtype = torch.bfloat16 if dtype is None else dtype
    code = _float_code(dtype, where)
    lead, kb, dev = _quantised(codes, scales, where)
    cols = _decoded_cols(cols, kb, where)
    st = _on(stream, dev, where)
    recv = _outputs(recv, [lead + (cols,)] * len(codes), codes[0], where, stream, dtype)
    _done(_ops.vrc_mx4_dequantize(_pointers(codes), _pointers(scales), _pointers(recv), len(codes), _prod(lead), cols,
                                  code, st or None), where)
    return recv


def vrc_mx4_all_gather(codes, scales, cols=None, dim=0, dtype=None, recv=None, stream=None):
    """recv[r] = the decoded concatenation of all ranks' matrices, for every rank:
    along the first dimension (``dim=0``) or the last (``dim=-1``)."""
    where = "vrc_mx4_all_gather"
    torch = _torch()
    dtype = torch.bfloat16 if dtype is None else dtype
    code = _float_code(dtype, where)
    lead, kb, dev = _quantised(codes, scales, where)
    cols = _decoded_cols(cols, kb, where)
    n, nd = len(codes), len(lead) + 1
    if dim in (-1, nd - 1):
        by_cols, shape = 1, lead + (n * cols,)
    elif dim in (0, -nd):
        by_cols, shape = 0, (n * lead[0],) + lead[1:] + (cols,)
    else:
        raise ValueError(f"{where}: dim must be the first or the last dimension")
    st = _on(stream, dev, where)
    recv = _outputs(recv, [shape] * n, codes[0], where, stream, dtype)
    _done(_ops.vrc_mx4_all_gather(_pointers(codes), _pointers(scales), _pointers(recv), n, _prod(lead), cols, by_cols,
                                  code, st or None), where)
    return recv


def vrc_mx4_matmul(a_codes, a_scales, b_codes, b_scales, recv=None, dtype=None, join="sum", stream=None):
    """Products of quantised matrices A_r [m, k] and B_r [n, k] (``vrc_mx4_quantize``
    along the last dimension): with ``join="sum"`` every recv[r] is the sum over
    ranks q of A_q B_q^T, with ``"each"`` recv[r] = A_r B_r^T.  Sums are held in fp32
    and rounded once to ``dtype`` (default bfloat16).

    A's leading dimensions are kept: recv[r] is [..., n].  Gradients, with G the
    output's: A's is G B, so the product of G and of B quantised with ``dim=0``; B's is
    G^T A, of G and A quantised with ``dim=0``."""
    where = "vrc_mx4_matmul"
    torch = _torch()
    dtype = torch.bfloat16 if dtype is None else dtype
    code = _float_code(dtype, where)
    if join not in MX4_JOINS:
        raise ValueError(f"join must be one of {sorted(MX4_JOINS)}")
    lead, kb, dev = _quantised(a_codes, a_scales, where)
    lead_b, kb_b, dev_b = _quantised(b_codes, b_scales, where)
    if len(lead_b) != 1 or kb_b != kb or dev_b != dev or len(b_codes) != len(a_codes):
        raise ValueError(f"{where}: B must be a matrix per rank with A's blocks, on A's device")
    st = _on(stream, dev, where)
    recv = _outputs(recv, [lead + lead_b] * len(a_codes), a_codes[0], where, stream, dtype)
    _done(_ops.vrc_mx4_matmul(_pointers(a_codes), _pointers(a_scales), _pointers(b_codes), _pointers(b_scales),
                              _pointers(recv), len(a_codes), _prod(lead), lead_b[0], kb, code, MX4_JOINS[join],
                              st or None), where)
    return recv


__all__ = [
    "vrc_allreduce_dropout", "vrc_reduce_scatter_dropout", "vrc_all_gather_dropout", "vrc_mx4_quantize",
    "vrc_mx4_dequantize", "vrc_mx4_all_gather", "vrc_mx4_matmul", "mx4_blocks", "Dropout", "ops_lib", "OPS_LIB_PATH",
    "OPS_VERSION", "MX4_BLOCK", "MX4_ALONG_COLS", "MX4_ALONG_ROWS", "MX4_JOINS",
]
