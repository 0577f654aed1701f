"""Cases of a tensor-parallel model's normalisation and loss, measured on one GPU.

Two families, which stand before and behind the collectives of a layer:

* layer norm (or, not centred, RMS norm) of each rank's rows, of the sum over
  the ranks with the residual stream (the all-reduce that ends a layer), or of
  each rank's rows of that sum (the reduce-scatter of the sequence-parallel
  form); and its gradient, joined over the ranks in the same three ways, with
  the weight's and the bias's gradients reduced over all rows of all ranks;
* softmax cross entropy of an output projection whose vocabulary is split over
  the ranks, from the hidden states, and its gradient: no logits are kept.

``own`` says which side runs: the plain torch forms (32-bit arithmetic, one
rounding at the end) or the framework's calls.

Definitions.  With h a row of W values, mean = sum h / W (0 if not centred),
rstd = (sum (h - mean)^2 / W + eps)^(-1/2), x = (h - mean) rstd, y = x w + b.
With g = dy w: dh = rstd (g - sum g / W [centred only] - x sum (g x) / W), dw
the sum of dy x over all rows, db that of dy.
With z_v = <hidden, w_v> over the whole vocabulary: lse = log sum exp z and
loss = lse - z_target; with a = dloss + dlse the gradient of z_v is
a exp(z_v - lse) - dloss [v = target].  A token whose target is ignore_index
has loss 0 and takes nothing from dloss; one whose z get no gradient at all
adds nothing to the weights', whatever its hidden state holds.
"""
import torch

own = False

DEV = "cuda"
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
ESIZE = {"fp32": 4, "fp16": 2, "bf16": 2}
EPS = 1e-5
IGNORE = -100


def listed():
    return [
        # One token's row at the end of a layer, summed over the ranks: decoding, where latency counts.
        dict(name="layer_norm_token", op="layer_norm", join="sum", n=8, rows=1, width=4096, dtype="fp16", residual=True, center=True, bias=True, wide=False),
        # The same over a training step's tokens: the all-reduce, the residual stream and the next layer's input.
        dict(name="layer_norm_tokens", op="layer_norm", join="sum", n=8, rows=8192, width=4096, dtype="bf16", residual=True, center=True, bias=True, wide=False),
        # Sequence parallel, RMS norm, fp32, rows that neither the ranks nor vectors divide.
        dict(name="layer_norm_scatter_odd", op="layer_norm", join="scatter", n=3, rows=4003, width=1053, dtype="fp32", residual=True, center=False, bias=False, wide=False),
        # Gradients of a sequence-parallel norm: each rank's own rows, weights in fp32.
        dict(name="layer_norm_grad_tokens", op="layer_norm_grad", join="each", n=8, rows=2048, width=8192, dtype="bf16", residual=True, center=True, bias=True, wide=True),
        # Behind a column-parallel product: the ranks' partial gradients are summed first; ragged rows.
        dict(name="layer_norm_grad_sum", op="layer_norm_grad", join="sum", n=4, rows=2056, width=1000, dtype="fp16", residual=True, center=True, bias=True, wide=False),
        # A few rows: a short prompt's gradients.
        dict(name="layer_norm_grad_few", op="layer_norm_grad", join="scatter", n=8, rows=13, width=4096, dtype="fp16", residual=False, center=False, bias=False, wide=False),
        # The score of one token under a vocabulary held by eight ranks: one pass over the weights.
        dict(name="cross_entropy_token", op="cross_entropy", n=8, tokens=1, vocab=65536, width=4096, dtype="bf16", ignored=0.0),
        # Scores of a short text in full precision, ragged everywhere.
        dict(name="cross_entropy_text", op="cross_entropy", n=4, tokens=48, vocab=20011, width=1000, dtype="fp32", ignored=0.1),
        # A training step's or a long text's loss: matrix-core bound.
        dict(name="cross_entropy_tokens", op="cross_entropy", n=8, tokens=4096, vocab=65536, width=4096, dtype="bf16", ignored=0.1),
        # Its gradients: the logits again, and two products from them.
        dict(name="cross_entropy_grad_tokens", op="cross_entropy_grad", n=8, tokens=4096, vocab=65536, width=4096, dtype="bf16", ignored=0.1, weighted=False),
        # The same of ragged sizes, each token's loss weighted, and a penalty on lse.
        dict(name="cross_entropy_grad_odd", op="cross_entropy_grad", n=5, tokens=1003, vocab=50003, width=1053, dtype="fp16", ignored=0.5, weighted=True),
        # A few tokens of a tuned text: reads and writes of the weights count.
        dict(name="cross_entropy_grad_few", op="cross_entropy_grad", n=8, tokens=7, vocab=32768, width=4096, dtype="bf16", ignored=0.0, weighted=False),
    ]


MOST_BYTES = 3 << 29   # what a drawn case reads and writes
MOST_LOGITS = 1 << 28  # as many as the largest listed case has
MOST_FLOPS = 3.0e12    # the largest listed case has 6.6e12


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    while True:
        n = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 8, 8, 12, 16])
        case = dict(op=rng.choice(["layer_norm", "layer_norm_grad", "cross_entropy", "cross_entropy_grad"]), n=n,
                    dtype=rng.choice(["fp32", "fp16", "bf16", "bf16"]))
        if case["op"].startswith("layer_norm"):
            case.update(join=rng.choice(["each", "sum", "scatter"]), rows=_log(rng, 1, 16384), width=_log(rng, 8, 20000),
                        residual=rng.random() < 0.6, center=rng.random() < 0.6, bias=rng.random() < 0.5, wide=rng.random() < 0.4)
        else:
            case.update(tokens=_log(rng, 1, 8192), vocab=_log(rng, 64, 131072), width=_log(rng, 16, 8192),
                        ignored=rng.choice([0.0, 0.1, 0.5]))
            if rng.random() < 0.5:
                case["width"] = -(-case["width"] // 64) * 64
            if case["op"] == "cross_entropy_grad":
                case["weighted"] = rng.random() < 0.5
            if case["tokens"] * case["vocab"] > MOST_LOGITS or case["vocab"] < n:
                continue
        w = work(case)
        if w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS:
            return case


def _spans(count, n):
    """The ranks' parts of `count` rows: equal ones, the last with the remainder."""
    each = count // n
    return [(c * each, (c + 1) * each if c < n - 1 else count) for c in range(n)]


def work(case):
    """Every input read once, every output written once."""
    n, e, op = case["n"], ESIZE[case["dtype"]], case["op"]
    if op.startswith("layer_norm"):
        rows, width = case["rows"], case["width"]
        total = rows * width * (n if case["join"] == "each" else 1)  # values that are normalised
        ranks = rows * width * n                                    # values of one tensor per rank
        copies = total if case["join"] == "scatter" else ranks      # what goes out, to one rank or to all
        params = width * (4 if case["wide"] else e) * (1 + case["bias"])
        stats = total // width * (8 if case["center"] else 4)
        if op == "layer_norm":
            out = copies + (total if case["residual"] or case["join"] != "each" else 0)
            return {"bytes": (ranks + total * case["residual"] + out) * e + params + stats, "flops": ranks + 8 * total}
        return {"bytes": (ranks + total + total * case["residual"] + copies) * e + 2 * params + stats, "flops": ranks + 14 * total}
    t, v, k = case["tokens"], case["vocab"], case["width"]
    if op == "cross_entropy":
        return {"bytes": (t + v) * k * e + 16 * t, "flops": 2.0 * t * v * k}
    return {"bytes": 2 * (t + v) * k * e + 16 * t, "flops": 6.0 * t * v * k}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, sigma=1.0, mu=0.0, dtype=dtype):
        return (torch.randn(*shape, generator=g, device=DEV) * sigma + mu).to(dtype)

    n, op = case["n"], case["op"]
    state = {"case": dict(case)}
    if op.startswith("layer_norm"):
        rows, width = case["rows"], case["width"]
        own_rows = [rows] * n if case["join"] == "each" else [b - a for a, b in _spans(rows, n)]
        wdtype = torch.float32 if case["wide"] else dtype
        state["weight"] = normal(width, sigma=0.3, mu=1.0, dtype=wdtype)
        if case["bias"]:
            state["bias"] = normal(width, sigma=0.1, dtype=wdtype)
        state["x"] = [normal(rows, width) for _ in range(n)]
        stream = [rows] if case["join"] == "sum" else own_rows
        if op == "layer_norm":
            if case["residual"]:  # the residual stream: larger than a layer's output, off centre
                state["residual"] = [normal(r, width, sigma=4.0, mu=0.5) for r in stream]
            return state
        state["h"] = [normal(r, width, sigma=4.0, mu=0.5) for r in stream]
        state["mean"], state["rstd"] = [], []
        for h in state["h"]:
            h = h.double()
            mean = h.mean(1, keepdim=True) if case["center"] else torch.zeros(h.shape[0], 1, dtype=torch.float64, device=DEV)
            state["mean"].append(mean[:, 0].float())
            state["rstd"].append(((h - mean).square().mean(1) + EPS).rsqrt().float())
        if case["residual"]:
            state["dh"] = [normal(r, width) for r in stream]
        return state
    t, v, k = case["tokens"], case["vocab"], case["width"]
    state["hidden"] = normal(t, k)
    state["weight"] = [normal(b - a, k, sigma=2.0 / k**0.5) for a, b in _spans(v, n)]
    target = torch.randint(0, v, (t,), generator=g, device=DEV)
    state["target"] = torch.where(torch.rand(t, generator=g, device=DEV) < case["ignored"], torch.full_like(target, IGNORE), target)
    if op == "cross_entropy_grad":
        z = state["hidden"].float() @ torch.cat(state["weight"]).float().t()
        state["lse"] = torch.logsumexp(z, 1)
        kept = (state["target"] != IGNORE).float()
        scale = 1024.0 if case["dtype"] == "fp16" else 1.0  # fp16 training scales its loss
        if case["weighted"]:
            state["dloss"] = torch.rand(t, generator=g, device=DEV) * scale / t
            state["dlse"] = 1e-3 * scale * state["lse"] * kept / t  # a penalty on lse^2 over the same tokens
        else:
            state["dloss"] = torch.full((t,), scale / t, device=DEV)  # the mean
    return state


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _one(xs, case):
    """What the framework takes: one tensor for all ranks where they share it."""
    return xs[0] if xs is not None and case["join"] == "sum" else xs


def _all(xs):
    return xs if isinstance(xs, (list, tuple)) else [xs]


def _run_own(state):
    import ring_all_reduce_virtual_amd as vrc

    case = state["case"]
    op = case["op"]
    if op == "layer_norm":
        y, h, mean, rstd = vrc.vrc_layer_norm(state["x"], state["weight"], state.get("bias"), EPS, join=case["join"],
                                              residual=_one(state.get("residual"), case), center=case["center"])
        out = {"y": y, "rstd": _all(rstd)}
        if case["residual"] or case["join"] != "each":
            out["h"] = _all(h)
        if case["center"]:
            out["mean"] = _all(mean)
        return out
    if op == "layer_norm_grad":
        dx, dw, db = vrc.vrc_layer_norm_grad(state["x"], _one(state["h"], case), state["weight"],
                                             _one(state["mean"], case) if case["center"] else None, _one(state["rstd"], case),
                                             dh=_one(state.get("dh"), case), join=case["join"], bias=case["bias"])
        return {"dx": dx, "dweight": dw, "dbias": db} if case["bias"] else {"dx": dx, "dweight": dw}
    if op == "cross_entropy":
        loss, lse = vrc.vrc_cross_entropy(state["hidden"], state["weight"], state["target"], ignore_index=IGNORE)
        return {"loss": loss, "lse": lse}
    dhidden, dweight = vrc.vrc_cross_entropy_grad(state["hidden"], state["weight"], state["target"], state["lse"],
                                                  state["dloss"], dlse=state.get("dlse"), ignore_index=IGNORE)
    return {"dhidden": dhidden, "dweight": dweight}


def _run_plain(state):
    case = state["case"]
    return {"layer_norm": _norm, "layer_norm_grad": _norm_grad, "cross_entropy": _entropy,
            "cross_entropy_grad": _entropy_grad}[case["op"]](state, case)


def _joined(xs, case):
    """The rows that are worked on, in fp32: each rank's, their sum, or each rank's rows of the sum."""
    if case["join"] == "each":
        return [x.float() for x in xs]
    total = torch.stack([x.float() for x in xs]).sum(0)
    return [total] if case["join"] == "sum" else [total[a:b] for a, b in _spans(case["rows"], case["n"])]


def _copies(ys, case):
    return [ys[0].clone() for _ in range(case["n"])] if case["join"] == "sum" else ys


def _norm(state, case):
    dtype = DTYPES[case["dtype"]]
    h = _joined(state["x"], case)
    if case["residual"]:
        h = [a + r.float() for a, r in zip(h, state["residual"])]
    w = state["weight"].float()
    b = state["bias"].float() if case["bias"] else torch.zeros_like(w)
    mean = [a.mean(1) if case["center"] else torch.zeros_like(a[:, 0]) for a in h]
    rstd = [((a - m[:, None]).square().mean(1) + EPS).rsqrt() for a, m in zip(h, mean)]
    y = [((a - m[:, None]) * s[:, None] * w + b).to(dtype) for a, m, s in zip(h, mean, rstd)]
    out = {"y": _copies(y, case), "rstd": rstd}
    if case["residual"] or case["join"] != "each":
        out["h"] = [a.to(dtype) for a in h]
    if case["center"]:
        out["mean"] = mean
    return out


def _norm_grad(state, case):
    dtype, w = DTYPES[case["dtype"]], state["weight"].float()
    dy = _joined(state["x"], case)
    x = [(h.float() - m[:, None]) * s[:, None] for h, m, s in zip(state["h"], state["mean"], state["rstd"])]
    g = [d * w for d in dy]
    c = 1.0 if case["center"] else 0.0
    dx = [s[:, None] * (a - c * a.mean(1, keepdim=True) - b * (a * b).mean(1, keepdim=True)) for s, a, b in zip(state["rstd"], g, x)]
    if case["residual"]:
        dx = [d + r.float() for d, r in zip(dx, state["dh"])]
    out = {"dx": _copies([d.to(dtype) for d in dx], case),
           "dweight": torch.cat([d * b for d, b in zip(dy, x)]).sum(0).to(state["weight"].dtype)}
    if case["bias"]:
        out["dbias"] = torch.cat(dy).sum(0).to(state["weight"].dtype)
    return out


def _entropy(state, case):
    z = state["hidden"].float() @ torch.cat(state["weight"]).float().t()
    top = z.max(1).values
    lse = top + (z - top[:, None]).exp().sum(1).log()
    kept = state["target"] != IGNORE
    picked = z.gather(1, state["target"].clamp(min=0)[:, None])[:, 0]
    return {"loss": torch.where(kept, lse - picked, torch.zeros_like(lse)), "lse": lse}


def _entropy_grad(state, case):
    dtype = DTYPES[case["dtype"]]
    kept = state["target"] != IGNORE
    b = torch.where(kept, state["dloss"], torch.zeros_like(state["dloss"]))
    a = b + state["dlse"] if "dlse" in state else b
    live = (a != 0) | (b != 0)
    h = torch.where(live[:, None], state["hidden"].float(), torch.zeros((), device=DEV))
    w = torch.cat(state["weight"]).float()
    p = (h @ w.t() - state["lse"][:, None]).exp() * a[:, None]
    p = torch.where(live[:, None], p, torch.zeros((), device=DEV))
    p.scatter_add_(1, state["target"].clamp(min=0)[:, None], -b[:, None])
    dw = (p.t() @ h).to(dtype)
    return {"dhidden": (p @ w).to(dtype), "dweight": [dw[lo:hi].clone() for lo, hi in _spans(case["vocab"], case["n"])]}


# ---------------------------------------------------------------------------
# In 64 bits, from the definitions
# ---------------------------------------------------------------------------
def exact(case, seed):
    state = prepare(case, seed)
    return (_exact_norm if case["op"].startswith("layer_norm") else _exact_entropy)(state, case)


def _exact_norm(state, case):
    n, join, width = case["n"], case["join"], case["width"]
    parts = [(0, case["rows"])] if join != "scatter" else _spans(case["rows"], n)
    grads = case["op"] == "layer_norm_grad"
    out = {"dx": [], "dweight": 0.0, "dbias": 0.0} if grads else {"y": [], "h": [], "mean": [], "rstd": []}
    for r in range(1 if join == "sum" else n):
        lo, hi = parts[r if join == "scatter" else 0]
        v = torch.zeros(hi - lo, width, dtype=torch.float64, device=DEV)
        for x in ([state["x"][r]] if join == "each" else state["x"]):
            v += x[lo:hi]
        if not grads:
            if case["residual"]:
                v += state["residual"][r]
            mean = torch.einsum("rw->r", v) / width if case["center"] else torch.zeros_like(v[:, 0])
            off = v - mean.unsqueeze(1)
            rstd = 1.0 / torch.sqrt((off * off).sum(1) / width + EPS)
            y = off * rstd.unsqueeze(1) * state["weight"].double() + (state["bias"].double() if case["bias"] else 0.0)
            for key, value in (("y", y), ("h", v), ("mean", mean), ("rstd", rstd)):
                out[key].append(value)
            continue
        rstd = state["rstd"][r].double().unsqueeze(1)
        x = (state["h"][r].double() - (state["mean"][r].double().unsqueeze(1) if case["center"] else 0.0)) * rstd
        g = v * state["weight"].double()
        along = (g * x).sum(1, keepdim=True) / width
        level = g.sum(1, keepdim=True) / width if case["center"] else 0.0
        out["dx"].append(rstd * (g - level - x * along) + (state["dh"][r].double() if case["residual"] else 0.0))
        out["dweight"] = out["dweight"] + (v * x).sum(0)
        out["dbias"] = out["dbias"] + v.sum(0)
    if join == "sum":
        key = "dx" if grads else "y"
        out[key] = out[key] * n
    if grads and not case["bias"]:
        del out["dbias"]
    if not grads and not case["center"]:
        del out["mean"]
    if not grads and join == "each" and not case["residual"]:
        del out["h"]
    return out


def _exact_entropy(state, case):
    hidden, target = state["hidden"].double(), state["target"]
    t = case["tokens"]
    if case["op"] == "cross_entropy":
        top = torch.full((t,), -float("inf"), dtype=torch.float64, device=DEV)
        total = torch.zeros_like(top)
        picked = torch.zeros_like(top)
        for (lo, hi), w in zip(_spans(case["vocab"], case["n"]), state["weight"]):
            z = hidden @ w.double().t()
            new = torch.maximum(top, z.max(1).values)
            total = total * torch.exp(top - new) + torch.exp(z - new.unsqueeze(1)).sum(1)
            top = new
            here = (target >= lo) & (target < hi)
            picked[here] = z[here, target[here] - lo]
        lse = top + torch.log(total)
        return {"loss": (lse - picked) * (target != IGNORE), "lse": lse}
    count = state["dloss"].double() * (target != IGNORE)
    weight = count + (state["dlse"].double() if "dlse" in state else 0.0)
    hidden = hidden * ((count != 0) | (weight != 0)).unsqueeze(1)
    dhidden, dweight = torch.zeros_like(hidden), []
    for (lo, hi), w in zip(_spans(case["vocab"], case["n"]), state["weight"]):
        w = w.double()
        dz = torch.exp(hidden @ w.t() - state["lse"].double().unsqueeze(1)) * weight.unsqueeze(1)
        here = ((target >= lo) & (target < hi)).nonzero()[:, 0]
        dz[here, target[here] - lo] -= count[here]
        dhidden += dz @ w
        dweight.append(dz.t() @ hidden)
    return {"dhidden": dhidden, "dweight": dweight}
