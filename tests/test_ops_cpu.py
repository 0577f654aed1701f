"""The operators' library on the CPU: symbols, refusals before any GPU call, the
binding's checks, the references' own pins, and the built kernels' resources."""
import ctypes as C
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import ring_all_reduce_virtual_amd as vrc
from ring_all_reduce_virtual_amd import ops
from tests import ops_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "include", "vrc_ops.h")).read()
FAKE = 0x10000000  # stand-in addresses: these calls must fail before any GPU work
L = ops.ops_lib()


def declared():
    text = re.sub(r"/\*.*?\*/", "", HEADER, flags=re.S)
    return sorted(set(re.findall(r"\b(vrc_[a-z_0-9]+)\s*\(", text)))


def test_every_declared_symbol_is_exported_and_bound():
    names = declared()
    assert len(names) == 9
    for n in names:
        assert hasattr(L, n), n
        if not n.startswith("vrc_ops_"):
            assert n in vrc.__all__ and callable(getattr(vrc, n))
    assert L.vrc_ops_version() == ops.OPS_VERSION == int(re.search(r"#define VRC_OPS_VERSION (\d+)", HEADER).group(1))
    assert L.vrc_ops_last_hip_error() == 0


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "vrc_ops.h"\nint main(void) { vrc_dropout_t d = {0.5, 1, 2, 0}; return d.p > 1 || vrc_ops_version() != VRC_OPS_VERSION; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-c", "-o",
                    str(tmp_path / "t.o"), str(src)], check=True)


def arr(base, n, stride=1 << 20):
    return vrc._ptr_array([base + r * stride for r in range(n)])


def drop(p=0.5, seed=1, offset=2, dev=None):
    return C.byref(ops.Dropout(p, seed, offset, dev))


A, B, R = FAKE, FAKE + (1 << 30), FAKE + (2 << 30)  # far apart


def test_dropout_refusals():
    def ar(x=arr(A, 4), res=None, y=arr(B, 4), n=4, count=1000, dt=vrc.VRC_BF16, d=drop()):
        return L.vrc_allreduce_dropout(x, res, y, n, count, dt, d, None)

    assert ar(n=0) == ar(n=17) == ar(count=(1 << 56) + 1) == vrc.VRC_ERR_INVALID_ARG
    assert ar(x=None) == ar(y=None) == ar(x=vrc._ptr_array([A, None, A, A])) == vrc.VRC_ERR_INVALID_ARG
    assert ar(res=vrc._ptr_array([R, R, None, R])) == vrc.VRC_ERR_INVALID_ARG
    assert ar(dt=vrc.VRC_INT32) == ar(dt=9) == ar(dt=-1) == vrc.VRC_ERR_UNSUPPORTED
    for p in (-0.1, 1.0001, float("nan"), float("inf")):
        assert ar(d=drop(p)) == vrc.VRC_ERR_INVALID_ARG
    assert ar(d=None) == ar(d=drop(dev=FAKE + 4)) == vrc.VRC_ERR_INVALID_ARG
    assert ar(count=0, x=None, y=None) == vrc.VRC_OK
    # overlaps: an output inside an input, in a residual, in another output; send[q] as recv[r]
    assert ar(y=arr(A + 2, 4)) == vrc.VRC_ERR_ALIAS
    assert ar(y=vrc._ptr_array([A + (1 << 20), A, B, B + 4096])) == vrc.VRC_ERR_ALIAS
    assert ar(y=vrc._ptr_array([B, B, R, R + 4096])) == vrc.VRC_ERR_ALIAS
    assert ar(res=arr(R, 4), y=arr(R + 1998, 4)) == vrc.VRC_ERR_ALIAS
    shared = vrc._ptr_array([R] * 4)
    assert ar(res=shared, y=vrc._ptr_array([R, B, B + 4096, B + 8192])) == vrc.VRC_ERR_ALIAS

    def rs(x=arr(A, 4), res=None, y=arr(B, 4), n=4, count=1000, outer=1, dt=vrc.VRC_BF16, d=drop()):
        return L.vrc_reduce_scatter_dropout(x, res, y, n, count, outer, dt, d, None)

    assert rs(outer=0) == rs(outer=3) == rs(count=1000, outer=500) == vrc.VRC_ERR_INVALID_ARG
    assert rs(y=arr(A, 4)) == rs(res=arr(R, 4), y=vrc._ptr_array([R + (1 << 20), B, B + 4096, B + 8192])) == vrc.VRC_ERR_ALIAS
    assert rs(d=drop(2.0)) == vrc.VRC_ERR_INVALID_ARG
    assert rs(dt=vrc.VRC_INT32) == vrc.VRC_ERR_UNSUPPORTED
    assert rs(count=0) == vrc.VRC_OK

    def ag(x=arr(A, 4), y=arr(B, 4), n=4, total=1000, outer=1, dt=vrc.VRC_BF16, d=drop()):
        return L.vrc_all_gather_dropout(x, y, n, total, outer, dt, d, None)

    assert ag(outer=0) == ag(outer=500) == ag(x=None) == ag(y=arr(0, 4)) == vrc.VRC_ERR_INVALID_ARG
    assert ag(y=arr(A + 100, 4)) == ag(y=vrc._ptr_array([B, B + 1998, R, R + 4096])) == vrc.VRC_ERR_ALIAS
    assert ag(dt=vrc.VRC_INT32) == vrc.VRC_ERR_UNSUPPORTED


def test_mx4_refusals():
    def q(x=arr(A, 2), c=arr(B, 2), s=arr(R, 2), n=2, rows=8, cols=64, dt=vrc.VRC_FP16, axis=0):
        return L.vrc_mx4_quantize(x, c, s, n, rows, cols, dt, axis, None)

    assert q(n=0) == q(n=17) == q(x=None) == q(c=None) == q(s=None) == vrc.VRC_ERR_INVALID_ARG
    assert q(c=arr(B + 8, 2)) == q(rows=1 << 40, cols=1 << 40) == q(rows=(1 << 56) + 1) == vrc.VRC_ERR_INVALID_ARG
    assert q(dt=vrc.VRC_INT32) == q(axis=2) == q(axis=-1) == vrc.VRC_ERR_UNSUPPORTED
    assert q(c=arr(A, 2)) == q(s=arr(B, 2)) == q(s=arr(A + 1023, 2)) == vrc.VRC_ERR_ALIAS
    assert q(rows=0) == q(cols=0) == vrc.VRC_OK

    def d(c=arr(A, 2), s=arr(B, 2), y=arr(R, 2), n=2, rows=8, cols=64, dt=vrc.VRC_FP16):
        return L.vrc_mx4_dequantize(c, s, y, n, rows, cols, dt, None)

    assert d(n=0) == d(c=None) == d(s=None) == d(y=None) == d(c=arr(A + 1, 2)) == vrc.VRC_ERR_INVALID_ARG
    assert d(dt=vrc.VRC_INT32) == vrc.VRC_ERR_UNSUPPORTED
    assert d(y=arr(A, 2)) == d(y=arr(B, 2)) == vrc.VRC_ERR_ALIAS
    # the gather's outputs are nranks times as long: 2 x 1 MiB apart no longer fit
    assert L.vrc_mx4_all_gather(arr(A, 2), arr(B, 2), arr(R, 2), 2, 8192, 64, 0, vrc.VRC_FP16, None) == vrc.VRC_ERR_ALIAS
    assert L.vrc_mx4_all_gather(None, None, None, 2, 0, 64, 0, vrc.VRC_FP16, None) == vrc.VRC_OK

    def mm(ac=arr(A, 2), as_=arr(A + (1 << 28), 2), bc=arr(B, 2), bs=arr(B + (1 << 28), 2), y=arr(R, 2), n=2, m=8, nc=8,
           kb=4, dt=vrc.VRC_FP16, join=0):
        return L.vrc_mx4_matmul(ac, as_, bc, bs, y, n, m, nc, kb, dt, join, None)

    assert mm(n=0) == mm(n=17) == mm(ac=None) == mm(as_=None) == mm(bc=None) == mm(bs=None) == vrc.VRC_ERR_INVALID_ARG
    assert mm(y=None) == mm(ac=arr(A + 4, 2)) == mm(bc=arr(B + 8, 2)) == vrc.VRC_ERR_INVALID_ARG
    assert mm(m=1 << 31) == mm(nc=1 << 31) == mm(kb=1 << 20) == mm(m=1 << 30, nc=1 << 30) == vrc.VRC_ERR_INVALID_ARG
    assert mm(dt=vrc.VRC_INT32) == mm(join=2) == vrc.VRC_ERR_UNSUPPORTED
    assert mm(y=arr(A, 2)) == mm(y=arr(B + (1 << 28), 2)) == mm(y=vrc._ptr_array([R, R + 64])) == vrc.VRC_ERR_ALIAS
    assert mm(m=0) == mm(nc=0) == vrc.VRC_OK


def test_binding_refuses_cpu_tensors_and_bad_shapes():
    x = [torch.zeros(4, 64, dtype=torch.bfloat16)] * 2
    u = [torch.zeros(4, 32, dtype=torch.uint8)] * 2
    for call in (lambda: vrc.vrc_allreduce_dropout(x, 0.1, 1), lambda: vrc.vrc_reduce_scatter_dropout(x, 0.1, 1),
                 lambda: vrc.vrc_all_gather_dropout(x, 0.1, 1), lambda: vrc.vrc_all_gather_dropout([], 0.1, 1),
                 lambda: vrc.vrc_mx4_quantize(x), lambda: vrc.vrc_mx4_dequantize(u, u), lambda: vrc.vrc_mx4_all_gather(u, u),
                 lambda: vrc.vrc_mx4_matmul(u, u, u, u), lambda: vrc.vrc_mx4_matmul(u, u, u, u, join="mean")):
        with pytest.raises(ValueError):
            call()
    for dtype in (torch.int32, torch.float64):
        with pytest.raises(TypeError):
            vrc.vrc_mx4_dequantize(u, u, dtype=dtype)
    dev = torch.device("cpu")
    for seed, offset in ((-1, 0), (1 << 64, 0), (0, -1), (0, 1 << 64), (0, torch.zeros(2, dtype=torch.int64)),
                         (0, torch.zeros(1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            ops._dropout(0.5, seed, offset, dev, "t")


def test_binding_refuses_a_stream_of_another_device():
    stream = type("Stream", (), {"device_index": 1, "cuda_stream": FAKE})()
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        ops._on(stream, 0, "vrc_mx4_matmul")


@pytest.mark.parametrize("shape", [(1024,), (64, 4, 8), (8,), (3,), (0, 8), (1 << 21,)])
def test_new_outputs_are_tensors_of_their_own(shape):
    """One output may be written in place, also by something that needs gradients,
    while another one is saved for a backward pass."""
    ys = ops._allocate([shape] * 3, torch.float32, torch.device("cpu"))
    w = torch.ones(shape, requires_grad=True)
    assert all(y.shape == shape and y.is_contiguous() and not y._is_view() for y in ys)
    spans = sorted((y.data_ptr(), y.data_ptr() + y.nbytes) for y in ys)
    assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
    for y in ys:
        y.fill_(2)
    loss = (w * ys[1]).sum()
    ys[0].add_(w)
    ys[2].zero_()
    loss.backward()
    assert torch.equal(w.grad, ys[1])


def test_reference_generator_known_answers():
    """The generator's published vectors (Random123's known answers)."""
    assert [hex(w) for w in ref.philox([0], 0, 0)[0]] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]
    ones = (1 << 64) - 1
    assert [hex(w) for w in ref.philox([ones], ones, ones)[0]] == ["0x408f276d", "0x41c83b0e", "0xa20bc7c6", "0x6d5451fd"]
    assert ref.keep(0, 1000, 0.0, 5, 6).all() and not ref.keep(0, 1000, 1.0, 5, 6).any()
    k = ref.keep(0, 1 << 20, 0.3, 5, 6)
    assert abs(k.mean() - 0.7) < 5 * (0.21 / (1 << 20)) ** 0.5
    assert (ref.keep(13, 50, 0.3, 5, 6) == k[13:63]).all()


def test_reference_quantiser_by_hand():
    row = np.zeros((1, 40))
    row[0, :12] = [6.0, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, -0.25, -7.9]
    codes, scales = ref.quantise(row)
    assert scales.tolist() == [[127, 0]]  # 7.9 has exponent 2: X = 0; the second block is all zero
    assert codes[0, :12].tolist() == [7, 0, 1, 2, 2, 4, 4, 6, 6, 7, 8, 15]
    v = ref.decode(ref.pack(codes), scales)
    assert v[0, :12].tolist() == [6.0, 0.0, 0.5, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 0.0, -6.0]
    bad = np.array([[1.0, np.inf] + [0.0] * 30])
    codes, scales = ref.quantise(bad)
    assert scales[0, 0] == 255 and not codes.any() and np.isnan(ref.decode(ref.pack(codes), scales)).all()
    assert ref.quantise(np.full((1, 32), 2.0**-149))[1][0, 0] == 0


def test_kernels_use_no_scratch(tmp_path):
    llvm = "/opt/rocm/llvm/bin/"
    if not all(os.path.exists(llvm + t) for t in ("llvm-objcopy", "clang-offload-bundler", "llvm-readelf")):
        pytest.skip("LLVM tools not available")
    fat = tmp_path / "fat.bin"
    subprocess.run([llvm + "llvm-objcopy", "--dump-section", f".hip_fatbin={fat}", ops.OPS_LIB_PATH,
                    str(tmp_path / "lib.so")], check=True, capture_output=True)
    blob = fat.read_bytes()
    starts = [m.start() for m in re.finditer(b"__CLANG_OFFLOAD_BUNDLE__", blob)] + [len(blob)]
    total = 0
    for i in range(len(starts) - 1):
        part, obj = tmp_path / f"b{i}.bin", tmp_path / f"c{i}.o"
        part.write_bytes(blob[starts[i]:starts[i + 1]])
        subprocess.run([llvm + "clang-offload-bundler", "--unbundle", "--type=o", f"--input={part}",
                        "--targets=hipv4-amdgcn-amd-amdhsa--gfx950", f"--output={obj}"], check=True, capture_output=True)
        if not obj.stat().st_size:
            continue
        notes = subprocess.run([llvm + "llvm-readelf", "--notes", str(obj)], check=True, capture_output=True, text=True).stdout
        for entry in notes.split("\n  - .agpr_count:")[1:]:
            name = re.search(r"\n\s+\.name:\s+(\S+)", entry).group(1)
            total += 1
            assert int(re.search(r"\.private_segment_fixed_size:\s+(\d+)", entry).group(1)) == 0, name
            assert int(re.search(r"\.vgpr_spill_count:\s+(\d+)", entry).group(1)) == 0, name
            assert int(re.search(r"\.group_segment_fixed_size:\s+(\d+)", entry).group(1)) <= 160 * 1024, name
    assert total > 100
