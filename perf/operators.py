"""Measured cases of the training-step operators that stand next to the collectives.

The reduce-scatter reads bf16 gradients and writes fp32 shards; these operators make the gradients
that are reductions over tokens (layer norm, embedding) and take the shards the collective leaves
(global norm, clipping):

* ``norm``    the L2 norm over a list of gradient tensors, and the sum of squares a data-parallel
              job adds up over its ranks;
* ``clip``    the same norm, and every tensor scaled by min(1, max_norm / (norm + 1e-6));
* ``ln``      layer norm over the last dimension, with the row statistics its gradient needs;
* ``ln_bwd``  its gradients: input, weight and bias;
* ``emb``     scaled embedding lookup (an id outside the table, such as -1 for padding, reads zeros);
* ``emb_bwd`` the table's gradient, every row of it.

``own`` false: the plain forms, elementary torch operations in 32 bits (sums of squares in 64),
rounded once.  ``own`` true: the package's entry points.
"""
import math

import torch

if torch.cuda.is_available():
    DEVICE = torch.device("cuda")
else:
    DEVICE = torch.device("cpu")

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
IDS = {"int32": torch.int32, "int64": torch.int64}
EPS = 1e-5


# ------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------

def listed():
    return [
        # Gradients of a three-parameter toy group before the reduce-scatter: launch latency alone.
        dict(name="norm toy group bf16", op="norm", tensors=3, numel=48, spread=0.8, dtype="bf16"),
        # One mixture-of-experts layer, a tensor per expert projection: hundreds of bf16 gradients of 3 MiB.
        dict(name="norm moe layer bf16", op="norm", tensors=391, numel=1572864, spread=0.0, dtype="bf16"),
        # The four fp32 shards of a toy group after the reduce-scatter.
        dict(name="clip toy shards fp32", op="clip", tensors=4, numel=31, spread=0.0, dtype="fp32", max_norm=0.25),
        # 64 flat shards of a diffusion transformer block, padded rows included: 1.4 GB of fp32 gradients.
        dict(name="clip 64 shards fp32", op="clip", tensors=64, numel=5490400, spread=0.0, dtype="fp32", max_norm=1.0),
        # A single token on its way through a decoder.
        dict(name="ln one token bf16", op="ln", rows=1, cols=4096, dtype="bf16", pdtype="bf16"),
        # A video clip's tokens in a diffusion transformer block.
        dict(name="ln video tokens bf16", op="ln", rows=32760, cols=5120, dtype="bf16", pdtype="bf16"),
        # Training at 8192 tokens a GPU, the widest layer group.
        dict(name="ln_bwd 8k tokens bf16", op="ln_bwd", rows=8192, cols=8192, dtype="bf16", pdtype="bf16"),
        # A short ragged batch in full precision, an odd width: rows start on 4-byte boundaries only.
        dict(name="ln_bwd odd width fp32", op="ln_bwd", rows=1023, cols=1001, dtype="fp32", pdtype="fp32"),
        # A short prompt.
        dict(name="emb short prompt bf16", op="emb", tokens=17, vocab=32000, dim=4096, dtype="bf16", ids="int64",
             pad=0.0, scale=1.0),
        # A packed training batch, inputs scaled by the root of the width.
        dict(name="emb 64k tokens bf16", op="emb", tokens=65536, vocab=131072, dim=4096, dtype="bf16", ids="int64",
             pad=0.02, scale=64.0),
        # The same table's gradient at 8192 tokens a GPU: most of its rows are zeros that have to be written.
        dict(name="emb_bwd 8k tokens bf16", op="emb_bwd", tokens=8192, vocab=131072, dim=4096, dtype="bf16",
             ids="int64", pad=0.02, scale=1.0),
        # More tokens than rows, an odd width and 32-bit ids, in full precision: sums over frequent tokens.
        dict(name="emb_bwd odd width fp32", op="emb_bwd", tokens=50021, vocab=20011, dim=1001, dtype="fp32",
             ids="int32", pad=0.05, scale=31.5),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm; odd ones as often as even ones."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("norm", "clip", "ln", "ln_bwd", "emb", "emb_bwd"))
    dtype = rng.choice(("bf16", "fp32"))
    if op in ("norm", "clip"):
        tensors = _spread(rng, 1, 600)
        numel = _spread(rng, 1, 300_000_000 // tensors)
        case = dict(op=op, tensors=tensors, numel=numel, spread=rng.choice((0.0, 0.5, 0.95)), dtype=dtype)
        if op == "clip":
            case["max_norm"] = rng.choice((0.1, 1.0, 50.0))
        return case
    if op in ("ln", "ln_bwd"):
        cols = _spread(rng, 8, 20000)
        rows = _spread(rng, 1, min(200_000, 32_000_000 // cols))
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, pdtype=rng.choice(("bf16", "fp32")))
    dim = _spread(rng, 1, 8192)
    vocab = _spread(rng, 1, min(200_000, 250_000_000 // dim))
    tokens = _spread(rng, 1, min(65536, 100_000_000 // dim))
    return dict(op=op, tokens=tokens, vocab=vocab, dim=dim, dtype=dtype, ids=rng.choice(("int32", "int64")),
                pad=rng.choice((0.0, 0.1)), scale=rng.choice((1.0, math.sqrt(dim))))


def _numels(case):
    """Elements of each tensor: `numel`, less up to the share `spread` of it, by a fixed pattern."""
    n, spread = case["numel"], case["spread"]
    return [n - int(n * spread * ((i * 0.6180339887498949) % 1.0)) for i in range(case["tensors"])]


def _packed(sizes, dtype):
    """A zeroed buffer and the views of it that hold tensors of these sizes."""
    places = [-(-n // 64) * 64 for n in sizes]
    flat = torch.zeros((sum(places),), dtype=dtype, device=DEVICE)
    return flat, [part[:n] for part, n in zip(flat.split(places), sizes)]


def _size(dtype):
    return 2 if dtype == "bf16" else 4


def work(case):
    op, e = case["op"], _size(case["dtype"])
    if op in ("norm", "clip"):
        n = sum(_numels(case))
        return {"bytes": n * e * (1 if op == "norm" else 2) + 12, "flops": n * (2 if op == "norm" else 3)}
    if op in ("ln", "ln_bwd"):
        rows, cols, p = case["rows"], case["cols"], _size(case["pdtype"])
        if op == "ln":  # x, y, both statistics, weight and bias
            return {"bytes": 2 * rows * cols * e + 8 * rows + 2 * cols * p, "flops": 8 * rows * cols}
        # dy, x, dx, both statistics, weight, and the two parameter gradients
        return {"bytes": 3 * rows * cols * e + 8 * rows + 3 * cols * p, "flops": 14 * rows * cols}
    tokens, vocab, dim = case["tokens"], case["vocab"], case["dim"]
    i = 4 if case["ids"] == "int32" else 8
    if op == "emb":  # ids, the rows of the table that occur (about: ids are drawn with P(k) ~ 1/(k+1)), the output
        s = math.log(vocab + 1)
        rows = sum(-math.expm1(-tokens * (1 - case["pad"]) * math.log1p(1 / (k + 1)) / s) for k in range(vocab))
        return {"bytes": tokens * (i + dim * e) + int(rows) * dim * e, "flops": tokens * dim}
    return {"bytes": tokens * (i + dim * e) + vocab * dim * e, "flops": tokens * dim}


# ------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------

def _normal(shape, dtype, gen, scale=1.0, shift=0.0):
    x = torch.empty(shape, device=DEVICE, dtype=torch.float32).normal_(shift, scale, generator=gen)
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    state = dict(case=case)
    if op in ("norm", "clip"):
        # gradients of a thousandth's size, each tensor with a scale of its own
        sizes = _numels(case)
        flat = _normal((sum(sizes),), torch.float32, gen, 1e-3)
        state["grads"] = [(g * (0.25 + (i % 7) / 4)).to(dtype) for i, g in enumerate(flat.split(sizes))]
        if op == "clip":
            # one buffer for all, each tensor on a boundary of 64 elements, as a sharded optimizer keeps them
            state["flat"], state["outs"] = _packed(sizes, dtype)
        return state
    if op in ("ln", "ln_bwd"):
        rows, cols, pdtype = case["rows"], case["cols"], DTYPES[case["pdtype"]]
        # activations: each row with a mean and a size of its own
        x = _normal((rows, cols), torch.float32, gen)
        x = x * _normal((rows, 1), torch.float32, gen, 0.3, 1.5) + _normal((rows, 1), torch.float32, gen)
        state["x"] = x.to(dtype)
        state["weight"] = _normal((cols,), pdtype, gen, 0.2, 1.0)
        state["bias"] = _normal((cols,), pdtype, gen, 0.1)
        if op == "ln_bwd":
            # the statistics that the forward pass left
            d = state["x"].double()
            mean = d.mean(1)
            state["mean"] = mean.float()
            state["rstd"] = ((d - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
            state["dy"] = _normal((rows, cols), dtype, gen)
        return state
    tokens, vocab, dim = case["tokens"], case["vocab"], case["dim"]
    # tokens of a text: the k-th most frequent about 1/k as often as the first; -1 where a sequence is padded
    u = torch.rand((2, tokens), device=DEVICE, dtype=torch.float64, generator=gen)
    ids = (torch.exp(u[0] * math.log(vocab + 1)) - 1).floor().long().clamp_(0, vocab - 1)
    state["ids"] = ids.masked_fill(u[1] < case["pad"], -1).to(IDS[case["ids"]])
    if op == "emb":
        state["table"] = _normal((vocab, dim), dtype, gen)
    else:
        state["dy"] = _normal((tokens, dim), dtype, gen)
    return state


# ------------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return PLAIN[state["case"]["op"]](state)


def _run_own(state):
    import all_gather_placement_amd as tide

    case = state["case"]
    op = case["op"]
    if op == "norm":
        return tide.grad_norm(state["grads"])
    if op == "clip":
        return tide.clip_grad_norm(state["grads"], case["max_norm"], outs=state["outs"]), state["flat"]
    if op == "ln":
        return tide.layer_norm(state["x"], state["weight"], state["bias"], EPS)
    if op == "ln_bwd":
        return tide.layer_norm_bwd(state["dy"], state["x"], state["weight"], state["mean"], state["rstd"])
    if op == "emb":
        return tide.embedding(state["ids"], state["table"], case["scale"])
    return tide.embedding_bwd(state["ids"], state["dy"], case["vocab"], case["scale"])


def _sum_of_squares(grads):
    return torch.stack([g.float().square().sum(dtype=torch.float64) for g in grads]).sum()


def _plain_norm(state):
    return _sum_of_squares(state["grads"]).sqrt().float()


def _plain_clip(state):
    norm = _sum_of_squares(state["grads"]).sqrt()
    coef = (state["case"]["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    for g, out in zip(state["grads"], state["outs"]):
        out.copy_(g.float() * coef)
    return norm.float(), state["flat"]


def _plain_ln(state):
    x = state["x"].float()
    mean = x.mean(1, keepdim=True)
    rstd = ((x - mean).square().mean(1, keepdim=True) + EPS).rsqrt()
    y = (x - mean) * rstd * state["weight"].float() + state["bias"].float()
    return y.to(state["x"].dtype), mean[:, 0], rstd[:, 0]


def _plain_ln_bwd(state):
    x, dy, w = state["x"].float(), state["dy"].float(), state["weight"].float()
    rstd = state["rstd"][:, None]
    xhat = (x - state["mean"][:, None]) * rstd
    g = dy * w
    dx = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * rstd
    pdtype = state["weight"].dtype
    return dx.to(state["x"].dtype), (dy * xhat).sum(0).to(pdtype), dy.sum(0).to(pdtype)


def _plain_emb(state):
    ids, table = state["ids"].long(), state["table"]
    inside = (ids >= 0) & (ids < table.shape[0])
    rows = table[torch.where(inside, ids, 0)].float() * state["case"]["scale"]
    return torch.where(inside[:, None], rows, 0.0).to(table.dtype)


def _plain_emb_bwd(state):
    ids, dy, vocab = state["ids"].long(), state["dy"], state["case"]["vocab"]
    inside = (ids >= 0) & (ids < vocab)
    rows = torch.where(inside[:, None], dy.float(), 0.0)
    grad = torch.zeros((vocab, dy.shape[1]), device=dy.device, dtype=torch.float32)
    grad.index_add_(0, torch.where(inside, ids, 0), rows)
    return (grad * state["case"]["scale"]).to(dy.dtype)


PLAIN = {"norm": _plain_norm, "clip": _plain_clip, "ln": _plain_ln, "ln_bwd": _plain_ln_bwd,
         "emb": _plain_emb, "emb_bwd": _plain_emb_bwd}


# ------------------------------------------------------------------------------------------------
# The definition in 64 bits
# ------------------------------------------------------------------------------------------------

def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "clip"):
        total = math.fsum(float(torch.dot(d, d)) for d in (g.double().reshape(-1) for g in state["grads"]))
        norm = math.sqrt(total)
        value = torch.tensor(norm, dtype=torch.float64)
        if op == "norm":
            return value
        coef = min(1.0, case["max_norm"] / (norm + 1e-6))
        flat, outs = _packed([g.numel() for g in state["grads"]], torch.float64)
        for g, o in zip(state["grads"], outs):
            o.add_(g.double(), alpha=coef)
        return value, flat
    if op == "ln":
        x = state["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = 1.0 / torch.sqrt(var + EPS)
        y = torch.addcmul(state["bias"].double(), (x - mean.unsqueeze(1)) * rstd.unsqueeze(1), state["weight"].double())
        return y, mean, rstd
    if op == "ln_bwd":
        # the gradient as the Jacobian of (x - mean) * rstd applied to dy * weight, from the given statistics
        rows, cols = state["x"].shape
        rstd = state["rstd"].double().unsqueeze(1)
        xhat = (state["x"].double() - state["mean"].double().unsqueeze(1)) * rstd
        dy = state["dy"].double()
        weight = state["weight"].double()
        ones = torch.ones(rows, dtype=torch.float64, device=dy.device)
        along = (dy * xhat) @ weight / cols
        level = dy @ weight / cols
        dx = torch.addcmul(dy * weight - level.unsqueeze(1), xhat, along.unsqueeze(1), value=-1.0) * rstd
        return dx, ones @ (dy * xhat), ones @ dy
    ids, vocab = state["ids"].long(), case["vocab"]
    keep = torch.nonzero((ids >= 0) & (ids < vocab)).reshape(-1)
    if op == "emb":
        out = torch.zeros((case["tokens"], case["dim"]), dtype=torch.float64, device=ids.device)
        out[keep] = torch.index_select(state["table"], 0, ids[keep]).double().mul_(case["scale"])
        return out
    # rows of equal ids brought together, summed as differences of a running sum
    order = keep[torch.argsort(ids[keep], stable=True)]
    rows, counts = torch.unique_consecutive(ids[order], return_counts=True)
    out = torch.zeros((vocab, case["dim"]), dtype=torch.float64, device=ids.device)
    if rows.numel():
        running = torch.cumsum(state["dy"][order].double(), 0)[torch.cumsum(counts, 0) - 1]
        running[1:] -= running[:-1].clone()
        out[rows] = running * case["scale"]
    return out
