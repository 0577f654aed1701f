"""Plain references of the tensor-parallel layer's operators (include/vrc_ops.h)
in numpy, in 64 bits, from their definitions.  They share no code with the HIP
path."""
from __future__ import annotations

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
EPS_HALF = {"fp32": 2.0**-24, "fp16": 2.0**-11, "bf16": 2.0**-8}   # half a step, relative
TINY_HALF = {"fp32": 2.0**-150, "fp16": 2.0**-25, "bf16": 2.0**-134}  # half a step of the subnormals


def philox(block, offset: int, seed: int) -> np.ndarray:
    """Philox-4x32-10 words [len(block), 4] of the counters (block, offset) under key `seed`."""
    low = np.uint64(0xFFFFFFFF)
    c = np.asarray(block, dtype=np.uint64)
    x = [c & low, c >> np.uint64(32), np.full_like(c, offset & 0xFFFFFFFF), np.full_like(c, offset >> 32)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        p0, p1 = np.uint64(0xD2511F53) * x[0], np.uint64(0xCD9E8D57) * x[2]
        x = [(p1 >> np.uint64(32)) ^ x[1] ^ np.uint64(k0), p1 & low, (p0 >> np.uint64(32)) ^ x[3] ^ np.uint64(k1), p0 & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(x, axis=1)


def keep(first: int, count: int, p: float, seed: int, offset: int) -> np.ndarray:
    """Whether elements first .. first + count - 1 are kept."""
    b0, b1 = first // 4, (first + count + 3) // 4
    w = philox(np.arange(b0, b1, dtype=np.uint64), offset, seed).reshape(-1)[first - 4 * b0:][:count]
    return w >= np.uint64(round(p * 2.0**32))


def dropped_sum(xs, p, seed, offset, first: int = 0):
    """drop(sum of xs) in 64 bits over flat arrays (element `first` onwards), and
    the bound of an fp32 evaluation of it: n - 1 additions and one multiplication by
    a rounded scale, each off by half a step of at most the sum of magnitudes."""
    xs = [np.asarray(x, dtype=np.float64).reshape(-1) for x in xs]
    k = keep(first, xs[0].size, p, seed, offset)
    scale = 0.0 if p == 1.0 else 1.0 / (1.0 - p)
    with np.errstate(invalid="ignore"):
        y = np.where(k, sum(xs[1:], xs[0]) * scale, 0.0)
        mag = np.where(k, sum(np.abs(x) for x in xs) * scale, 0.0)
    return y, mag * (len(xs) + 1) * 2.0**-24


def rounding(y, dtype: str):
    """The bound of one rounding of y to `dtype`."""
    return np.abs(y) * EPS_HALF[dtype] + TINY_HALF[dtype]


def quantise(x):
    """(codes [rows, 32 KB] one a byte, scale bytes [rows, KB]) of a float64 matrix, by
    search for the nearest of the eight magnitudes, ties to the even code."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    kb = -(-cols // 32)
    v = np.zeros((rows, kb * 32))
    v[:, :cols] = x
    v = v.reshape(rows, kb, 32)
    finite = np.isfinite(v).all(2)
    v = np.where(finite[:, :, None], v, 0.0)
    top = np.abs(v).max(2)
    _, e = np.frexp(top)  # top = f * 2^e, 0.5 <= f < 1
    byte = np.where(top == 0, 0, np.clip(e - 1 - 2, -127, 127) + 127)
    q = np.abs(v) / np.exp2(byte.astype(np.float64) - 127)[:, :, None]
    d = np.abs(q[..., None] - MAGNITUDES)
    best = d.min(-1, keepdims=True)
    near = d == best
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    code = code + 8 * np.signbit(v)
    code = np.where(finite[:, :, None], code, 0)
    return code.reshape(rows, kb * 32).astype(np.uint8), np.where(finite, byte, 255).astype(np.uint8)


def pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def unpack(packed):
    return np.stack([packed & 15, packed >> 4], axis=2).reshape(packed.shape[0], -1)


def decode(packed, scales):
    """The values [rows, 32 KB] in 64 bits; a block whose scale byte is 255 is NaN."""
    c = unpack(np.asarray(packed))
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    v = np.where(c >= 8, -1.0, 1.0) * MAGNITUDES[c % 8]
    return v * np.repeat(s, 32, axis=1)
