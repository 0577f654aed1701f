"""4-bit blocks, what tests/test_gpu_ops.py does not reach: the product's 128 x 128
tiles, scales at any address, block maxima of every exponent, and scales at the end of
fp32's range."""
import pytest
import torch

from tests import ops_reference as ref
from tests.test_gpu_ops import DEV, DT, check_product, check_quantised, product, random_mx4, say, vrc  # noqa: F401
from tests.test_gpu_ops_narrow import replay_us

pytestmark = pytest.mark.gpu


def tiles(size, m, nc, products):
    return -(-m // size) * -(-nc // size) * products


# 2 whole tiles of the contraction, an odd number of pairs, and many; ragged: two tiles of
# which the second has one block, and so on
@pytest.mark.parametrize("k", [512, 1536, 4096, 288, 257, 540, 4100])
@pytest.mark.parametrize("join,n,m,nc", [("sum", 1, 2001, 2048), ("sum", 3, 1030, 2500), ("each", 3, 1500, 1450)])
def test_mx4_matmul_middle_tiles(vrc, join, n, m, nc, k):  # noqa: F811
    """Too much for 64 x 64 tiles and too little for 256 x 256."""
    room = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    products = n if join == "each" else 1
    assert tiles(64, m, nc, products) > room >= tiles(128, m, nc, products)
    a, b = [random_mx4(m, k, 7 + r) for r in range(n)], [random_mx4(nc, k, 70 + r) for r in range(n)]
    ops = [list(t) for t in zip(*a)] + [list(t) for t in zip(*b)]
    want = [product(*[[t[r]] for t in ops]) for r in range(n)]
    if join == "sum":
        want = [(sum(y for y, _ in want), sum(mag for _, mag in want))] * n
    for dtype in ("fp32", "bf16"):
        say(f"mx4_matmul {join} n={n} m={m} n={nc} k={k} {dtype}")
        got = vrc.vrc_mx4_matmul(*ops, dtype=DT[dtype], join=join)
        for r in range(n):
            if join == "sum" and r:
                assert torch.equal(got[r], got[0])
                continue
            check_product(got[r], *want[r], k * (n if join == "sum" else 1), dtype, f"rank {r}")


@pytest.mark.parametrize("m,nc,k", [(1, 300, 512), (16, 300, 1024), (30, 9000, 512), (50, 600, 512), (100, 300, 1024), (500, 500, 512),
                                    (2001, 2048, 512), (4001, 4100, 512), (4001, 4100, 1024), (300, 7, 512)])
def test_mx4_matmul_scales_at_any_address(vrc, m, nc, k):  # noqa: F811
    """Whole tiles whose scales are off the kernels' alignment: the aligned call's bits."""
    (ac, as_), (bc, bs) = random_mx4(m, k, 3), random_mx4(nc, k, 4)
    want = vrc.vrc_mx4_matmul([ac], [as_], [bc], [bs], dtype=torch.float32)[0]
    y, mag = product([ac], [as_], [bc], [bs])
    check_product(want, y, mag, k, "fp32", "aligned")

    def moved(s, by):
        room = torch.full((s.numel() + 64,), 0x85, dtype=torch.uint8, device=DEV)
        view = room[by:by + s.numel()].view(s.shape)
        view.copy_(s)
        return view

    for by_a, by_b in ((1, 0), (0, 1), (8, 8), (3, 13)):
        say(f"m={m} n={nc} k={k} scales {by_a} and {by_b} bytes off")
        got = vrc.vrc_mx4_matmul([ac], [moved(as_, by_a)], [bc], [moved(bs, by_b)], dtype=torch.float32)[0]
        assert torch.equal(got, want), (by_a, by_b)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_quantise_every_16_bit_value_under_every_near_maximum(vrc, dtype):  # noqa: F811
    """Each finite value beside a block maximum of its own exponent and up to eight above:
    v / 2^X then lies in every power of two from [4, 8) down to [1/64, 1/32), the tie at
    1/4 and all that rounds up to 1/2 among them.  Along the rows and down the columns."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(DT[dtype])
    v = bits[torch.isfinite(bits)].double()
    own = torch.floor(torch.log2(v.abs().clamp(min=2.0**-133)))
    for up in (0, 1, 2, 3, 4, 5, 6, 7, 8):
        say(f"{dtype} maximum {up} exponents up")
        blk = torch.zeros(v.numel(), 32, dtype=torch.float64)
        blk[:, 7], blk[:, 20] = v, torch.where(v == 0, torch.zeros(()), torch.exp2(own + up))
        x = blk[torch.isfinite(blk.to(DT[dtype])).all(1)].to(DT[dtype])
        codes, scales = vrc.vrc_mx4_quantize([x.to(DEV)])
        check_quantised(codes[0], scales[0], x.double().numpy(), f"{dtype} {up}")
        down, down_scales = vrc.vrc_mx4_quantize([x.t().contiguous().to(DEV)], dim=0)
        assert torch.equal(down[0], codes[0]) and torch.equal(down_scales[0], scales[0]), up


def test_decode_past_fp32(vrc):  # noqa: F811
    """Magnitudes of 2^128 and more, which only scale bytes 253 and 254 reach, are
    infinite in fp32; every other is exact."""
    packed = ((torch.arange(32) % 16).view(16, 2) * torch.tensor([1, 16])).sum(1).to(torch.uint8).view(1, 16)
    for byte, over in ((252, ()), (253, (6, 7)), (254, (4, 5, 6, 7))):
        scales = torch.tensor([[byte]], dtype=torch.uint8)
        want = torch.from_numpy(ref.decode(packed.numpy(), scales.numpy()))[0]
        got = vrc.vrc_mx4_dequantize([packed.to(DEV)], [scales.to(DEV)], dtype=torch.float32)[0][0].double().cpu()
        for i in range(32):
            if i % 8 in over:
                assert torch.isinf(got[i]) and torch.signbit(got[i]) == (i % 16 >= 8), (byte, i)
            else:
                assert got[i] == want[i], (byte, i)


@pytest.mark.parametrize("dim", [0, -1])
def test_gather_in_fp32_takes_its_bytes_time(vrc, dim):  # noqa: F811
    """Twice the bytes of a 16-bit gather, and little more than twice its time; with
    stores of half lines it took nine times as long."""
    n, rows, cols = 8, 20480, 128
    codes, scales = vrc.vrc_mx4_quantize([torch.randn(rows, cols, device=DEV) for _ in range(n)])
    shape = (n * rows, cols) if dim == 0 else (rows, n * cols)
    times = {}
    for dtype in ("bf16", "fp32"):
        out = [torch.empty(shape, dtype=DT[dtype], device=DEV) for _ in range(n)]
        times[dtype] = replay_us(lambda: vrc.vrc_mx4_all_gather(codes, scales, cols, dim=dim, dtype=DT[dtype], recv=out))
    say(f"dim {dim}: {times}")
    assert times["fp32"] < 4 * times["bf16"]
