"""Cases of the tensor-parallel layer's operators, measured on one GPU.

Two families, which meet in the row-parallel half of a tensor-parallel
layer over virtual ranks:

* dropout (with its residual) in the collective that ends the layer: the
  all-reduce, the reduce-scatter of the sequence-parallel form, and the
  masked all-gather that is the reduce-scatter's gradient.  The gradient of
  the all-reduce form is the same call without a residual.  The mask comes
  from a counter-based generator and is never stored;
* microscaled 4-bit floating point: quantisation along rows or columns, the
  gather that decodes every rank's shard, and the product, summed over the
  ranks' parts of the contraction or one product per rank (the gradients).

``own`` says which side runs: the plain torch forms (32-bit arithmetic, one
rounding at the end) or the framework's calls.

Definitions.  Element i of a tensor is dropped when word i mod 4 of
Philox-4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
easy as 1, 2, 3", SC 2011), with counter (i / 4, offset) and key seed, is
below round(p * 2^32); kept ones are scaled by 1 / (1 - p).  A block of 32
values shares the scale 2^X, X = floor(log2 max|v|) - 2 (OCP Microscaling
Formats 1.0), held as the byte X + 127; its values v / 2^X are rounded to
the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code).
"""
import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
ESIZE = {"fp32": 4, "fp16": 2, "bf16": 2}
BLOCK = 32  # values that share a scale
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # One [8, 4096] fp16 activation per rank at the end of a layer: the smallest call, launch latency.
        dict(name="allreduce_dropout_act", op="allreduce_dropout", n=8, outer=8, width=4096, dtype="fp16", p=0.1, residual="shared"),
        # The same sum over a training step's tokens, each rank with its own residual buffer.
        dict(name="allreduce_dropout_tokens", op="allreduce_dropout", n=8, outer=8192, width=4096, dtype="bf16", p=0.1, residual="each"),
        # Sequence parallel: a rank keeps its columns of every token, odd row count, wide and small rows.
        dict(name="reduce_scatter_dropout_act", op="reduce_scatter_dropout", n=8, outer=13, width=4096, dtype="fp16", p=0.25, residual="each"),
        # The flat form over fp32 with a length that nothing divides, and no residual.
        dict(name="reduce_scatter_dropout_flat", op="reduce_scatter_dropout", n=4, outer=1, width=16777213, dtype="fp32", p=0.5, residual="none"),
        # Their gradients: the shards of the output's gradient, masked and gathered to every rank.
        dict(name="all_gather_dropout_tokens", op="all_gather_dropout", n=8, outer=8192, width=512, dtype="bf16", p=0.1),
        dict(name="all_gather_dropout_odd", op="all_gather_dropout", n=3, outer=1001, width=1053, dtype="fp32", p=0.3),
        # The attention heads' slices, gathered over a wire of four bits a value.
        dict(name="mx4_gather_heads", op="mx4_gather", n=8, rows=20480, cols=128, dtype="fp16"),
        # The transposed codes that a backward product needs: blocks along the rows, ragged both ways.
        dict(name="mx4_transpose_weights", op="mx4_transpose", n=2, rows=8200, cols=4100, dtype="bf16"),
        # One token against the weights of a whole group: memory-bound.
        dict(name="mx4_matmul_token", op="mx4_matmul", n=8, m=1, ncols=8192, k=4096, dtype="bf16", join="sum"),
        # A batch of decoded tokens, ragged everywhere, in full precision.
        dict(name="mx4_matmul_batch", op="mx4_matmul", n=4, m=48, ncols=5003, k=1000, dtype="fp32", join="sum"),
        # A prompt or a training step: matrix-core bound.
        dict(name="mx4_matmul_tokens", op="mx4_matmul", n=8, m=4096, ncols=8192, k=4096, dtype="bf16", join="sum"),
        # The weights' gradients: one ragged product for each rank.
        dict(name="mx4_matmul_each", op="mx4_matmul", n=4, m=2056, ncols=1000, k=4100, dtype="fp32", join="each"),
    ]


MOST_BYTES = 1 << 30  # inputs and outputs of one drawn case
MOST_MASKED = 1 << 25  # elements under one mask, as many as the largest listed case has
MOST_FLOPS = 2.0e12   # the largest listed product has 2.2e12


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    while True:
        op = rng.choice(["allreduce_dropout", "reduce_scatter_dropout", "all_gather_dropout", "mx4_gather",
                         "mx4_transpose", "mx4_matmul", "mx4_matmul"])
        n = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8, 8, 12, 16])
        case = dict(op=op, n=n, dtype=rng.choice(["fp32", "fp16", "bf16"]))
        if op in ("allreduce_dropout", "reduce_scatter_dropout", "all_gather_dropout"):
            outer = rng.choice([1, _log(rng, 1, 16384)])
            width = _log(rng, 1, 1 << 24) if outer == 1 else _log(rng, 1, 16384)
            if op == "reduce_scatter_dropout" and outer > 1:
                width = -(-width // n) * n  # the columns split evenly
            if outer * width * (n if op == "all_gather_dropout" else 1) > MOST_MASKED:
                continue
            case.update(outer=outer, width=width, p=rng.choice([0.0, 0.1, 0.5, round(rng.uniform(0.01, 0.95), 3), round(rng.uniform(0.01, 0.95), 3)]))
            if op != "all_gather_dropout":
                case["residual"] = rng.choice(["none", "shared", "each"] if op == "allreduce_dropout" else ["none", "each"])
        elif op in ("mx4_gather", "mx4_transpose"):
            case.update(rows=_log(rng, 1, 32768), cols=_log(rng, 1, 16384))
        else:
            case.update(m=_log(rng, 1, 8192), ncols=_log(rng, 1, 8192), k=_log(rng, 1, 8192),
                        join=rng.choice(["sum", "sum", "each"]))
        w = work(case)
        if w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS:
            return case


def _blocks(k):
    return -(-k // BLOCK)


def _chunk(count, n, c):
    base = count // n
    return c * base, (count if c == n - 1 else (c + 1) * base)


def work(case):
    """Every input read once, every output written once; the generator's and
    the rounding's operations are not counted as floating point."""
    n, e = case["n"], ESIZE[case["dtype"]]
    op = case["op"]
    if op == "allreduce_dropout":
        size = case["outer"] * case["width"]
        res = {"none": 0, "shared": 1, "each": n}[case["residual"]]
        return {"bytes": (2 * n + res) * size * e, "flops": (n + 1) * size}
    if op == "reduce_scatter_dropout":
        size = case["outer"] * case["width"]
        return {"bytes": (n + 1 + (case["residual"] == "each")) * size * e, "flops": (n + 1) * size}
    if op == "all_gather_dropout":
        size = n * case["outer"] * case["width"]
        return {"bytes": (1 + n) * size * e, "flops": size}
    if op in ("mx4_gather", "mx4_transpose"):
        rows, cols = case["rows"], case["cols"]
        values = n * rows * cols
        scales = n * (rows * _blocks(cols) if op == "mx4_gather" else cols * _blocks(rows))
        copies = n if op == "mx4_gather" else 1
        return {"bytes": values * e * (1 + copies) + scales, "flops": 2 * values}
    m, nc, k = case["m"], case["ncols"], case["k"]
    return {"bytes": n * ((m + nc) * _blocks(k) * (BLOCK // 2 + 1) + m * nc * e), "flops": 2.0 * n * m * nc * k}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape, dtype=DTYPES[case["dtype"]], sigma=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * sigma).to(dtype)

    n, op = case["n"], case["op"]
    state = {"case": dict(case), "seed": (seed * 0x9E3779B97F4A7C15 + 12345) % (1 << 64), "offset": seed % (1 << 40)}
    if op in ("allreduce_dropout", "reduce_scatter_dropout", "all_gather_dropout"):
        outer, width = case["outer"], case["width"]
        state["x"] = [normal(outer, width) for _ in range(n)]
        res = case.get("residual", "none")
        if res == "shared":
            state["res"] = normal(outer, width, sigma=4.0)
        elif res == "each" and op == "allreduce_dropout":
            state["res"] = [normal(outer, width, sigma=4.0) for _ in range(n)]
        elif res == "each" and outer > 1:
            state["res"] = [normal(outer, width // n, sigma=4.0) for _ in range(n)]
        elif res == "each":
            spans = [_chunk(width, n, c) for c in range(n)]
            state["res"] = [normal(hi - lo, sigma=4.0) for lo, hi in spans]
    elif op in ("mx4_gather", "mx4_transpose"):
        # activations and gradients: normal values whose rows and columns differ in size, a few of them all zero
        rows, cols = case["rows"], case["cols"]
        state["x"] = []
        for _ in range(n):
            size = torch.exp2(torch.randint(-9, 9, (rows, 1), generator=g, device=DEV).float())
            live = torch.rand(rows, 1, generator=g, device=DEV) > 0.02
            spread = torch.exp2(torch.randint(-4, 5, (1, cols), generator=g, device=DEV).float())
            state["x"].append((torch.randn(rows, cols, generator=g, device=DEV) * size * live * spread).clamp(-6e4, 6e4).to(DTYPES[case["dtype"]]))
    else:
        for name, rows in (("a", case["m"]), ("b", case["ncols"])):
            pairs = [_quantise(normal(rows, case["k"], dtype=torch.float32)) for _ in range(n)]
            state[name + "_codes"] = [_pack(c) for c, _ in pairs]
            state[name + "_scales"] = [s for _, s in pairs]
    return state


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    import ring_all_reduce_virtual_amd as vrc

    case = state["case"]
    op, n = case["op"], case["n"]
    if op == "allreduce_dropout":
        return vrc.vrc_allreduce_dropout(state["x"], case["p"], state["seed"], state["offset"], residual=state.get("res"))
    if op == "reduce_scatter_dropout":
        return vrc.vrc_reduce_scatter_dropout(state["x"], case["p"], state["seed"], state["offset"],
                                              residual=state.get("res"), dim=1 if case["outer"] > 1 else 0)
    if op == "all_gather_dropout":
        return vrc.vrc_all_gather_dropout(state["x"], case["p"], state["seed"], state["offset"], dim=1)
    if op == "mx4_gather":
        codes, scales = vrc.vrc_mx4_quantize(state["x"])
        return {"y": vrc.vrc_mx4_all_gather(codes, scales, case["cols"], dtype=DTYPES[case["dtype"]]), "scales": scales}
    if op == "mx4_transpose":
        codes, scales = vrc.vrc_mx4_quantize(state["x"], dim=0)
        return {"y": vrc.vrc_mx4_dequantize(codes, scales, case["rows"], dtype=DTYPES[case["dtype"]]), "scales": scales}
    return vrc.vrc_mx4_matmul(state["a_codes"], state["a_scales"], state["b_codes"], state["b_scales"],
                              dtype=DTYPES[case["dtype"]], join=case["join"])


def _run_plain(state):
    case = state["case"]
    op, n, dtype = case["op"], case["n"], DTYPES[case["dtype"]]
    if op == "allreduce_dropout":
        y = _drop(_fold(state["x"]), state)
        res = state.get("res")
        if isinstance(res, list):
            return [(y + r.float()).to(dtype) for r in res]
        y = (y if res is None else y + res.float()).to(dtype)
        return [y.clone() for _ in range(n)]
    if op == "reduce_scatter_dropout":
        y = _drop(_fold(state["x"]), state)
        outer, width = y.shape
        if outer > 1:
            parts = [p.contiguous() for p in y.view(outer, n, width // n).unbind(1)]
        else:
            spans = [_chunk(width, n, c) for c in range(n)]
            parts = [y[0, lo:hi] for lo, hi in spans]
        res = state.get("res")
        return [p.to(dtype) for p in parts] if res is None else [(p + r.float()).to(dtype) for p, r in zip(parts, res)]
    if op == "all_gather_dropout":
        y = _drop(torch.cat([x.float() for x in state["x"]], 1), state).to(dtype)
        return [y.clone() for _ in range(n)]
    if op == "mx4_gather":
        pairs = [_quantise(x) for x in state["x"]]
        y = torch.cat([_decode(c, s, case["cols"]) for c, s in pairs], 0).to(dtype)
        return {"y": [y.clone() for _ in range(n)], "scales": [s for _, s in pairs]}
    if op == "mx4_transpose":
        pairs = [_quantise(x.t()) for x in state["x"]]
        return {"y": [_decode(c, s, case["rows"]).to(dtype) for c, s in pairs], "scales": [s for _, s in pairs]}
    a = [_decode(_unpack(c), s, s.shape[1] * BLOCK) for c, s in zip(state["a_codes"], state["a_scales"])]
    b = [_decode(_unpack(c), s, s.shape[1] * BLOCK) for c, s in zip(state["b_codes"], state["b_scales"])]
    if case["join"] == "sum":
        y = torch.mm(torch.cat(a, 1), torch.cat(b, 1).t().contiguous()).to(dtype)
        return [y.clone() for _ in range(n)]
    y = torch.bmm(torch.stack(a), torch.stack(b).transpose(1, 2).contiguous()).to(dtype)
    return [p.clone() for p in y.unbind(0)]


def _fold(xs):
    """x_0 + x_1 + ... in fp32, in rank order."""
    y = xs[0].float()
    for x in xs[1:]:
        y = y + x.float()
    return y


def _mulhilo(a, m):
    """High and low words of the 32 x 32-bit products, held in int64 (the
    product's 64 bits wrap into the sign; the shifted words are masked)."""
    p = a * m
    return (p >> 32) & 0xFFFFFFFF, p & 0xFFFFFFFF


def _words(count, seed, offset, device):
    """Philox-4x32-10 word of each of elements 0 .. count-1."""
    block = torch.arange(-(-count // 4), dtype=torch.int64, device=device)
    c0, c1 = block & 0xFFFFFFFF, block >> 32
    c2 = torch.full_like(block, offset & 0xFFFFFFFF)
    c3 = torch.full_like(block, offset >> 32)
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        h0, l0 = _mulhilo(c0, 0xD2511F53)
        h1, l1 = _mulhilo(c2, 0xCD9E8D57)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return torch.stack((c0, c1, c2, c3), 1).view(-1)[:count]


def _drop(y, state):
    p = state["case"]["p"]
    keep = _words(y.numel(), state["seed"], state["offset"], y.device) >= int(round(p * 4294967296.0))
    scale = float(np.float32(0.0 if p == 1.0 else 1.0 / (1.0 - p)))
    return torch.where(keep.view(y.shape), y * scale, torch.zeros_like(y))


def _quantise(x):
    """Codes [rows, blocks * 32] (one a byte) and scale bytes [rows, blocks]
    of the rows of x, zero-filled to whole blocks."""
    rows, cols = x.shape
    kb = _blocks(cols)
    v = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - cols)).view(rows, kb, BLOCK)
    top = v.abs().amax(2)
    e = torch.frexp(top).exponent.to(torch.int32) - 3
    e = torch.where(top == 0, torch.full_like(e, -127), e.clamp(-127, 127))
    q = torch.ldexp(v, -e.unsqueeze(2))
    a = q.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = code + torch.signbit(q).to(torch.uint8) * 8
    bad = ~torch.isfinite(top)
    code = torch.where(bad.unsqueeze(2), torch.zeros_like(code), code)
    return code.view(rows, kb * BLOCK), torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)


def _pack(codes):
    """Two codes to a byte, the even column in the low half."""
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def _unpack(packed):
    return torch.stack((packed & 15, packed >> 4), 2).view(packed.shape[0], -1)


def _decode(codes, scales, cols):
    """The first `cols` values of each row, in fp32."""
    table = torch.tensor(VALUES + tuple(-v for v in VALUES), device=codes.device)
    rows, kb = scales.shape
    s = torch.ldexp(torch.ones((), device=codes.device), scales.to(torch.int32) - 127)
    s = torch.where(scales == 255, torch.full_like(s, float("nan")), s)
    return (table[codes.long()].view(rows, kb, BLOCK) * s.unsqueeze(2)).view(rows, kb * BLOCK)[:, :cols].contiguous()


# ---------------------------------------------------------------------------
# In 64 bits, from the definitions
# ---------------------------------------------------------------------------
def exact(case, seed):
    state = prepare(case, seed)
    op, n = case["op"], case["n"]
    if "dropout" in op:
        xs = [x.double().cpu().numpy() for x in state["x"]]
        y = np.concatenate(xs, axis=1) if op == "all_gather_dropout" else sum(xs[1:], xs[0])
        keep = _exact_words(y.size, state["seed"], state["offset"]).reshape(y.shape) >= np.uint64(round(case["p"] * 2.0**32))
        y = np.where(keep, y / (1.0 - case["p"]) if case["p"] < 1.0 else 0.0, 0.0)
        res = state.get("res")
        res = [r.double().cpu().numpy() for r in res] if isinstance(res, list) else None if res is None else res.double().cpu().numpy()
        if op == "all_gather_dropout":
            return [y] * n
        if op == "allreduce_dropout":
            return [y + r for r in res] if isinstance(res, list) else [y if res is None else y + res] * n
        outer, width = y.shape
        if outer > 1:
            w = width // n
            parts = [np.ascontiguousarray(y[:, c * w:(c + 1) * w]) for c in range(n)]
        else:
            parts = [y[0, slice(*_chunk(width, n, c))] for c in range(n)]
        return parts if res is None else [p + r for p, r in zip(parts, res)]
    if op in ("mx4_gather", "mx4_transpose"):
        got = [_exact_round(x.double() if op == "mx4_gather" else x.double().t()) for x in state["x"]]
        y = [torch.cat([v for v, _ in got], 0)] * n if op == "mx4_gather" else [v for v, _ in got]
        return {"y": y, "scales": [s for _, s in got]}
    a = [_exact_values(c, s) for c, s in zip(state["a_codes"], state["a_scales"])]
    b = [_exact_values(c, s) for c, s in zip(state["b_codes"], state["b_scales"])]
    each = [x @ y.t() for x, y in zip(a, b)]
    return each if case["join"] == "each" else [sum(each[1:], each[0])] * n


def _exact_words(count, seed, offset):
    """The generator's words from its definition, on the host: a bijection of
    four 32-bit words applied in ten rounds, the key stepped by the two
    constants between rounds."""
    mask = np.uint64(0xFFFFFFFF)
    i = np.arange((count + 3) // 4, dtype=np.uint64)
    x = [i & mask, i >> np.uint64(32), np.full_like(i, offset % 2**32), np.full_like(i, offset // 2**32)]
    for r in range(10):
        key = [np.uint64((seed % 2**32 + r * 0x9E3779B9) % 2**32), np.uint64((seed // 2**32 + r * 0xBB67AE85) % 2**32)]
        p, q = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(q >> np.uint64(32)) ^ x[1] ^ key[0], q & mask, (p >> np.uint64(32)) ^ x[3] ^ key[1], p & mask]
    return np.stack(x, axis=1).reshape(-1)[:count]


def _exact_round(x):
    """Nearest values on each block's grid: of the two neighbours of |v| / 2^X
    among the eight magnitudes the nearer, on a tie the one of even index."""
    rows, cols = x.shape
    kb = -(-cols // BLOCK)
    v = torch.zeros(rows, kb * BLOCK, dtype=torch.float64, device=x.device)
    v[:, :cols] = x
    v = v.view(rows, kb, BLOCK)
    top = v.abs().amax(2)
    e = (torch.floor(torch.log2(top.clamp(min=2.0**-200))) - 2).clamp(-127, 127)
    e = e - (torch.exp2(e + 2) > top).double() * (e > -127)  # log2 may round up to the next whole number
    scale = torch.exp2(e).unsqueeze(2)
    q = (v / scale).abs()
    grid = torch.tensor(VALUES, dtype=torch.float64, device=x.device)
    lo = (torch.bucketize(q, grid, right=True) - 1).clamp(0, 6)
    below, above = q - grid[lo], grid[lo + 1] - q
    up = (above < below) | ((above == below) & (lo % 2 == 1))
    y = torch.sign(v) * grid[lo + up.long()] * scale
    return y.view(rows, kb * BLOCK)[:, :cols].contiguous(), (e + 127).to(torch.uint8)


def _exact_values(packed, scales):
    rows, kb = scales.shape
    b = packed.to(torch.int64)
    c = torch.stack((b % 16, b // 16), 2).view(rows, kb, BLOCK)
    m = c % 8
    # sign, two exponent bits (bias 1), one mantissa bit; exponent 0 is subnormal
    mag = torch.where(m < 2, m * 0.5, (1 + 0.5 * (m % 2)) * torch.exp2((m // 2 - 1).double()))
    v = torch.where(c >= 8, -mag, mag).double() * torch.exp2(scales.double() - 127).unsqueeze(2)
    return v.view(rows, kb * BLOCK)
