"""Measured cases of the operators that a transformer block's training step passes its tokens through,
beside layer norm and embedding: the experts of a mixture, rotary positions of several axes, dropout.

* ``sort``     (token, choice) pairs brought into the order of their experts: where each pair's row goes,
               what each row comes from, where each expert's rows start (rounded up to ``align``);
* ``dispatch`` the tokens' rows in that order (a row of no token is zeros); backward: their gradient;
* ``combine``  the experts' rows back at their tokens, weighted and summed; backward: the gradients of
               the rows and of the weights;
* ``rotary``   pairs of a head's elements turned by an angle: the token's position along the pair's axis
               times the pair's frequency; backward: turned back;
* ``dropout``  elements dropped by a counter-based generator and the others scaled, added to a residual;
               backward: the same elements of the gradient.  The mask is stored nowhere.

The generator is Philox4x32 with 10 rounds (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3",
2011): element e of a call takes 16 bits, number e mod 8 from the low end, of the 128 that key = seed and
counter = e div 8 give, and is kept where they are at least p * 65536, rounded.

``own`` false: the plain forms, elementary torch operations in 32 bits (angles in 64), rounded once.
``own`` true: the package's entry points.
"""
import math
import random

import numpy as np
import torch

if torch.cuda.is_available():
    DEVICE = torch.device("cuda")
else:
    DEVICE = torch.device("cpu")

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
KINDS = {"int32": torch.int32, "int64": torch.int64, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------

def listed():
    return [
        # A decoding batch at the router of a layer of 128 experts: launch latency alone.
        dict(name="sort 17 tokens", op="sort", tokens=17, choices=8, experts=128, align=1, ids="int64", pad=0.0),
        # A packed training batch at the same router; each expert's rows end on a tile of a grouped product.
        dict(name="sort 64k tokens", op="sort", tokens=65536, choices=8, experts=128, align=128, ids="int64",
             pad=0.02),
        # Training at 8192 tokens a GPU through a layer of 128 experts, eight a token.
        dict(name="dispatch 8k tokens bf16", op="dispatch", backward=False, tokens=8192, choices=8, experts=128,
             align=128, dim=2048, dtype="bf16", pad=0.02),
        # The gradient of a ragged batch in full precision, an odd width: rows start on 4-byte boundaries only.
        dict(name="dispatch_bwd odd width fp32", op="dispatch", backward=True, tokens=4099, choices=3, experts=60,
             align=1, dim=1001, dtype="fp32", pad=0.1),
        # A single token on its way back from eight experts.
        dict(name="combine one token bf16", op="combine", backward=False, tokens=1, choices=8, experts=128, align=1,
             dim=2048, dtype="bf16", wdtype="fp32", pad=0.0),
        # The backward pass of the 8192 tokens: gradients of the experts' rows and of the router's weights.
        dict(name="combine_bwd 8k tokens bf16", op="combine", backward=True, tokens=8192, choices=8, experts=128,
             align=128, dim=2048, dtype="bf16", wdtype="fp32", pad=0.02),
        # The queries of one token far into a text.
        dict(name="rotary one token bf16", op="rotary", backward=False, frames=1, height=1, width=1, start=100000.0,
             step=1.0, heads=32, dim=128, sections="64", pairing="halves", positions="int64", dtype="bf16",
             fused=False),
        # The queries of a video clip in a diffusion transformer block: time, height and width.
        dict(name="rotary video tokens bf16", op="rotary", backward=False, frames=21, height=30, width=52, start=0.0,
             step=1.0, heads=40, dim=128, sections="22,21,21", pairing="neighbours", positions="int32", dtype="bf16",
             fused=False),
        # An image's keys in full precision, a part of each head turned, heads of one buffer with queries and values.
        dict(name="rotary_bwd odd image fp32", op="rotary", backward=True, frames=1, height=37, width=53, start=0.0,
             step=0.75, heads=5, dim=80, sections="17,19", pairing="halves", positions="fp32", dtype="fp32",
             fused=True),
        # One token's vector, the seed on the device as a captured step keeps it.
        dict(name="dropout one token bf16", op="dropout", backward=False, rows=1, cols=4096, p=0.1, offset=0,
             residual=True, device_seed=True, dtype="bf16"),
        # The output of a diffusion transformer block's attention, dropped and added to the residual.
        dict(name="dropout video tokens bf16", op="dropout", backward=False, rows=32760, cols=5120, p=0.1, offset=0,
             residual=True, device_seed=False, dtype="bf16"),
        # A later rank's part of a ragged batch in full precision: its elements are counted from an odd one on.
        dict(name="dropout_bwd odd width fp32", op="dropout", backward=True, rows=1023, cols=1001, p=0.3,
             offset=1023 * 1001, residual=False, device_seed=False, dtype="fp32"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm; odd ones as often as even ones."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("sort", "dispatch", "combine", "rotary", "rotary", "dropout", "dropout"))
    dtype = rng.choice(("bf16", "fp32"))
    if op == "rotary":
        axes = rng.choice((1, 2, 3))
        pairs = _spread(rng, axes, 128)
        cuts = sorted(rng.sample(range(1, pairs), axes - 1))
        sections = [b - a for a, b in zip([0] + cuts, cuts + [pairs])]
        dim = 2 * pairs + rng.choice((0, 0, 0, 8, 2 * pairs, rng.randrange(1, 64)))
        heads = _spread(rng, 1, 64)
        most = min(100_000, 80_000_000 // (heads * dim))
        frames = _spread(rng, 1, 32) if axes == 3 else 1
        height = _spread(rng, 1, 128) if axes >= 2 else 1
        frames, height = min(frames, most), max(1, min(height, most // min(frames, most)))
        return dict(op=op, backward=rng.random() < 0.4, frames=frames, height=height,
                    width=_spread(rng, 1, max(1, most // (frames * height))),
                    start=rng.choice((0.0, 0.0, 4096.0, 1000000.0)), step=rng.choice((1.0, 1.0, 0.75, 2.0)),
                    heads=heads, dim=dim, sections=",".join(map(str, sections)),
                    pairing=rng.choice(("halves", "neighbours")), positions=rng.choice(("int32", "int64", "fp32")),
                    dtype=dtype, fused=rng.random() < 0.3)
    if op == "dropout":
        cols = _spread(rng, 1, 20000)
        backward = rng.random() < 0.4
        return dict(op=op, backward=backward, rows=_spread(rng, 1, 80_000_000 // cols), cols=cols,
                    p=rng.choice((0.0, 0.05, 0.1, 0.3, 0.5)), offset=rng.choice((0, 0, rng.randrange(1 << 40))),
                    residual=not backward and rng.random() < 0.6, device_seed=rng.random() < 0.3, dtype=dtype)
    experts = _spread(rng, 2, 512)
    case = dict(op=op, choices=min(experts, rng.choice((1, 2, 3, 4, 6, 8, 10))), experts=experts,
                align=rng.choice((1, 1, 16, 128)), pad=rng.choice((0.0, 0.1, 0.5)))
    if op == "sort":
        return dict(case, tokens=_spread(rng, 1, 400_000 // case["choices"]), ids=rng.choice(("int32", "int64")))
    dim = _spread(rng, 8, 8192)
    case["experts"] = max(2, min(experts, 100_000_000 // (2 * dim * case["align"])))
    case["choices"] = min(case["choices"], case["experts"])
    most = 100_000_000 // dim - case["experts"] * (case["align"] - 1)
    case.update(tokens=_spread(rng, 1, max(1, min(65536, most // case["choices"]))), dim=dim, dtype=dtype,
                backward=rng.random() < 0.5)
    if op == "combine":
        case["wdtype"] = rng.choice(("bf16", "fp32"))
    return case


def _size(kind):
    return {"bf16": 2, "int64": 8}.get(kind, 4)


def _rows(case):
    """Rows of the sorted buffer: each expert that has any starts on a multiple of `align`."""
    pairs = case["tokens"] * case["choices"]
    return pairs + min(case["experts"], pairs) * (case["align"] - 1)


def _sections(case):
    return tuple(map(int, case["sections"].split(",")))


def _tokens(case):
    return case["frames"] * case["height"] * case["width"]


def _threshold(case):
    return round(case["p"] * 65536)


def work(case):
    op = case["op"]
    if op == "rotary":
        tokens, axes = _tokens(case), len(_sections(case))
        numel, turned = tokens * case["heads"] * case["dim"], tokens * case["heads"] * 2 * sum(_sections(case))
        return {"bytes": 2 * numel * _size(case["dtype"]) + tokens * axes * _size(case["positions"]), "flops": 3 * turned}
    if op == "dropout":
        numel = case["rows"] * case["cols"]
        return {"bytes": numel * _size(case["dtype"]) * (3 if case["residual"] else 2), "flops": 2 * numel}
    pairs, rows = case["tokens"] * case["choices"], _rows(case)
    if op == "sort":
        return {"bytes": pairs * (_size(case["ids"]) + 4) + 4 * rows + 4 * (case["experts"] + 1), "flops": pairs}
    row = case["dim"] * _size(case["dtype"])
    real = int(case["tokens"] * (1 - case["pad"]))  # tokens that have experts, about
    if op == "dispatch":
        if case["backward"]:
            return {"bytes": real * case["choices"] * row + case["tokens"] * row + 4 * pairs,
                    "flops": pairs * case["dim"]}
        return {"bytes": real * row + rows * row + 4 * rows, "flops": rows}
    weights = pairs * (4 + _size(case["wdtype"]))
    if case["backward"]:
        return {"bytes": real * (1 + case["choices"]) * row + rows * row + weights + pairs * _size(case["wdtype"]),
                "flops": 3 * pairs * case["dim"]}
    return {"bytes": real * case["choices"] * row + case["tokens"] * row + weights, "flops": 2 * pairs * case["dim"]}


# ------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------

def _normal(shape, dtype, gen, scale=1.0, shift=0.0):
    x = torch.empty(shape, device=DEVICE, dtype=torch.float32).normal_(shift, scale, generator=gen)
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    op = case["op"]
    state = dict(case=case)
    if op == "rotary":
        sections, dtype = _sections(case), DTYPES[case["dtype"]]
        grid = torch.meshgrid(*(torch.arange(n, device=DEVICE, dtype=torch.float64)
                                for n in (case["frames"], case["height"], case["width"])), indexing="ij")
        # the first axis runs from `start` on in steps of `step`; another batch begins elsewhere
        axes = [g.reshape(-1) for g in grid[3 - len(sections):]]
        axes[0] = case["start"] + seed % 7 + axes[0] * case["step"]
        state["positions"] = torch.stack(axes).to(KINDS[case["positions"]])
        # an axis's frequencies fall from one by a power of 10000
        ramp = [torch.arange(n, device=DEVICE, dtype=torch.float64) / n for n in sections]
        state["freqs"] = torch.cat([torch.exp(-math.log(10000.0) * r) for r in ramp])
        tokens, heads = _tokens(case), case["heads"]
        if case["fused"]:  # queries, keys and values beside each other
            state["x"] = _normal((tokens, 3 * heads, case["dim"]), dtype, gen)[:, heads:2 * heads]
        else:
            state["x"] = _normal((tokens, heads, case["dim"]), dtype, gen)
        return state
    if op == "dropout":
        dtype = DTYPES[case["dtype"]]
        state["x"] = _normal((case["rows"], case["cols"]), dtype, gen)
        state["residual"] = _normal((case["rows"], case["cols"]), dtype, gen, 2.0) if case["residual"] else None
        number = random.Random(seed).getrandbits(63)
        state["seed"] = torch.tensor([number], device=DEVICE) if case["device_seed"] else number
        return state
    # a router's logits: some experts are preferred; the pairs of padded tokens have no expert
    tokens, experts, choices = case["tokens"], case["experts"], case["choices"]
    logits = _normal((tokens, experts), torch.float32, gen) + _normal((experts,), torch.float32, gen, 0.5)
    top, ids = torch.topk(logits, choices, dim=1)
    padded = torch.rand((tokens, 1), device=DEVICE, generator=gen) < case["pad"]
    ids = ids.masked_fill(padded, -1)
    if op == "sort":
        state["ids"] = ids.to(KINDS[case["ids"]])
        return state
    dtype, dim = DTYPES[case["dtype"]], case["dim"]
    state["sort"] = _plain_sort(dict(case=case, ids=ids))
    if op == "combine":
        state["weights"] = torch.softmax(top, dim=1).to(DTYPES[case["wdtype"]])
    if op == "dispatch" and not case["backward"]:
        state["x"] = _normal((tokens, dim), dtype, gen)
    else:
        state["rows"] = _normal((_rows(case), dim), dtype, gen)
    if op == "combine" and case["backward"]:
        state["dy"] = _normal((tokens, dim), dtype, gen)
    return state


# ------------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    if case.get("backward"):
        return PLAIN_BACKWARD[case["op"]](state)
    return PLAIN[case["op"]](state)


def _run_own(state):
    import all_gather_placement_amd as tide

    case = state["case"]
    op, backward = case["op"], case.get("backward")
    if op == "sort":
        return tuple(tide.expert_sort(state["ids"], case["experts"], align=case["align"]))
    if op == "dispatch":
        if backward:
            return tide.expert_dispatch_bwd(state["rows"], state["sort"])
        return tide.expert_dispatch(state["x"], state["sort"])
    if op == "combine":
        if backward:
            return tide.expert_combine_bwd(state["dy"], state["rows"], state["weights"], state["sort"])
        return tide.expert_combine(state["rows"], state["weights"], state["sort"])
    if op == "rotary":
        turn = tide.rotary_bwd if backward else tide.rotary
        return turn(state["x"], state["positions"], state["freqs"], _sections(case), pairing=case["pairing"])
    if backward:
        return tide.dropout_bwd(state["x"], case["p"], state["seed"], offset=case["offset"])
    return tide.dropout(state["x"], case["p"], state["seed"], offset=case["offset"], residual=state["residual"])


def _plain_sort(state):
    """place[t, j]: the row of pair (t, j), -1 if it has no expert; source[r]: its number t * choices + j, -1
    for a row of no pair; offsets[e]: where expert e's rows start."""
    case, ids = state["case"], state["ids"]
    experts, align = case["experts"], case["align"]
    flat = ids.reshape(-1).long()
    inside = (flat >= 0) & (flat < experts)
    key = torch.where(inside, flat, experts)
    counts = torch.zeros(experts + 1, device=flat.device, dtype=torch.int64).scatter_add_(0, key, torch.ones_like(key))
    padded = (counts[:experts] + align - 1) // align * align
    offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    order = torch.argsort(key, stable=True)
    before = counts.cumsum(0) - counts  # pairs of lower experts
    row = offsets[key[order]] + torch.arange(len(flat), device=flat.device) - before[key[order]]
    source = torch.full((_rows(case) + 1,), -1, device=flat.device, dtype=torch.int32)
    place = torch.full_like(flat, -1)
    there = inside[order]
    source[torch.where(there, row, _rows(case))] = torch.where(there, order, -1).int()
    place[order] = torch.where(there, row, -1)
    return place.int().reshape(ids.shape), source[:-1], offsets.int()


def _plain_dispatch(state):
    x, (place, source, _) = state["x"], state["sort"]
    token = torch.where(source >= 0, source, 0).long() // place.shape[1]
    return torch.where((source >= 0)[:, None], x[token], 0.0)


def _plain_dispatch_bwd(state):
    rows, (place, _, _) = state["rows"], state["sort"]
    total = torch.zeros((place.shape[0], rows.shape[1]), device=rows.device, dtype=torch.float32)
    for j in range(place.shape[1]):
        at = place[:, j].long()
        total += torch.where((at >= 0)[:, None], rows[at.clamp(min=0)].float(), 0.0)
    return total.to(rows.dtype)


def _plain_combine(state):
    rows, weights, (place, _, _) = state["rows"], state["weights"].float(), state["sort"]
    total = torch.zeros((place.shape[0], rows.shape[1]), device=rows.device, dtype=torch.float32)
    for j in range(place.shape[1]):
        at = place[:, j].long()
        total += torch.where((at >= 0)[:, None], rows[at.clamp(min=0)].float() * weights[:, j, None], 0.0)
    return total.to(rows.dtype)


def _plain_combine_bwd(state):
    dy, rows, weights, (place, source, _) = state["dy"].float(), state["rows"], state["weights"], state["sort"]
    at = torch.where(source >= 0, source, 0).long()
    drows = dy[at // place.shape[1]] * weights.float().reshape(-1)[at][:, None]
    drows = torch.where((source >= 0)[:, None], drows, 0.0).to(rows.dtype)
    dots = []
    for j in range(place.shape[1]):
        at = place[:, j].long()
        dots.append(torch.where(at >= 0, (rows[at.clamp(min=0)].float() * dy).sum(1), 0.0))
    return drows, torch.stack(dots, 1).to(weights.dtype)


def _plain_rotary(state, sign=1.0):
    case, x = state["case"], state["x"]
    sections = _sections(case)
    pairs = sum(sections)
    axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).to(x.device)
    angle = state["positions"].double()[axis] * state["freqs"][:, None]
    cos, sin = angle.cos().float().T[:, None], angle.sin().float().T[:, None] * sign
    f = x.float()
    out = f.clone()
    if case["pairing"] == "halves":
        first, second = slice(0, pairs), slice(pairs, 2 * pairs)
    else:
        first, second = slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)
    out[..., first] = f[..., first] * cos - f[..., second] * sin
    out[..., second] = f[..., second] * cos + f[..., first] * sin
    return out.to(x.dtype)


def _plain_keep(case, seed, device):
    """Which elements are kept, by number from `offset` on."""
    low = 0xffffffff
    first, numel = case["offset"], case["rows"] * case["cols"]
    block = torch.arange(first >> 3, (first + numel + 7) >> 3, device=device)
    c0, c1, c2, c3 = block & low, block >> 32, torch.zeros_like(block), torch.zeros_like(block)
    k0, k1 = seed & low, (seed >> 32) & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & low) ^ c1 ^ k0, b & low, ((a >> 32) & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    bits = torch.stack([half for c in (c0, c1, c2, c3) for half in (c & 0xffff, c >> 16)], 1).reshape(-1)
    bits = bits[first & 7:(first & 7) + numel]
    return (bits >= _threshold(case)).reshape(case["rows"], case["cols"])


def _plain_dropout(state):
    case, x = state["case"], state["x"]
    scale = 65536 / (65536 - _threshold(case))
    y = torch.where(_plain_keep(case, state["seed"], x.device), x.float() * scale, 0.0)
    if state["residual"] is not None:
        y = y + state["residual"].float()
    return y.to(x.dtype)


PLAIN = {"sort": _plain_sort, "dispatch": _plain_dispatch, "combine": _plain_combine, "rotary": _plain_rotary,
         "dropout": _plain_dropout}
PLAIN_BACKWARD = {"dispatch": _plain_dispatch_bwd, "combine": _plain_combine_bwd,
                  "rotary": lambda state: _plain_rotary(state, -1.0), "dropout": _plain_dropout}


# ------------------------------------------------------------------------------------------------
# The definition in 64 bits
# ------------------------------------------------------------------------------------------------

def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "sort":
        return _exact_sort(state["ids"].cpu().numpy(), case)
    if op == "rotary":
        return _exact_rotary(state)
    if op == "dropout":
        numel = case["rows"] * case["cols"]
        kept = np.empty(numel, dtype=bool)
        for start in range(0, numel, 1 << 24):
            stop = min(numel, start + (1 << 24))
            kept[start:stop] = _exact_bits(int(state["seed"]), case["offset"] + start, stop - start) >= _threshold(case)
        y = state["x"].double() / (1 - _threshold(case) / 65536)
        y.masked_fill_(torch.from_numpy(~kept).to(y.device).reshape(y.shape), 0.0)
        return y if state["residual"] is None else y.add_(state["residual"])
    place, source, _ = state["sort"]
    tokens, choices = place.shape
    if op == "dispatch" and not case["backward"]:
        real = torch.nonzero(source >= 0)[:, 0]
        out = torch.zeros((len(source), case["dim"]), device=DEVICE, dtype=torch.float64)
        return out.index_copy_(0, real, state["x"].double()[torch.div(source[real], choices, rounding_mode="floor").long()])
    # the same as a sum over rows: row r belongs to token source[r] // choices
    real = torch.nonzero(source >= 0)[:, 0]
    pair = source[real].long()
    rows = state["rows"].double()
    weight = state["weights"].double().reshape(-1)[pair] if op == "combine" else torch.ones(len(pair), device=DEVICE).double()
    if op == "combine" and case["backward"]:
        dy = state["dy"].double()[pair // choices]
        dots = torch.zeros(tokens * choices, device=DEVICE, dtype=torch.float64)
        for start in range(0, len(pair), 8192):
            part = slice(start, start + 8192)
            dots[pair[part]] = torch.bmm(rows[real[part]][:, None], dy[part][:, :, None])[:, 0, 0]
        drows = torch.zeros_like(rows).index_copy_(0, real, dy * weight[:, None])
        return drows, dots.reshape(tokens, choices)
    out = torch.zeros((tokens, case["dim"]), device=DEVICE, dtype=torch.float64)
    return out.index_add_(0, pair // choices, rows[real] * weight[:, None])


def _exact_sort(ids, case):
    place = np.full(ids.shape, -1, dtype=np.int32)
    source = np.full(_rows(case), -1, dtype=np.int32)
    offsets = np.zeros(case["experts"] + 1, dtype=np.int32)
    flat = ids.reshape(-1)
    order = np.argsort(flat, kind="stable")
    starts = np.searchsorted(flat[order], np.arange(case["experts"] + 1))
    at = 0
    for e in range(case["experts"]):
        pairs = order[starts[e]:starts[e + 1]]
        rows = np.arange(at, at + len(pairs))
        source[rows] = pairs
        place.reshape(-1)[pairs] = rows
        at += -(-len(pairs) // case["align"]) * case["align"]
        offsets[e + 1] = at
    return tuple(torch.from_numpy(a).to(DEVICE) for a in (place, source, offsets))


def _exact_rotary(state):
    case, x = state["case"], state["x"].double()
    sections = _sections(case)
    pairs, parts = sum(sections), []
    for positions, freqs in zip(state["positions"].double(), state["freqs"].split(sections)):
        parts.append(torch.outer(positions, freqs))
    turn = torch.polar(torch.ones((), device=x.device, dtype=torch.float64), torch.cat(parts, 1))
    if case["backward"]:
        turn = turn.conj()
    head = x[..., :2 * pairs]
    if case["pairing"] == "halves":
        z = torch.complex(head[..., :pairs], head[..., pairs:]) * turn[:, None]
        out = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(head.unflatten(-1, (pairs, 2)).contiguous()) * turn[:, None]
        out = torch.view_as_real(z).flatten(-2)
    return torch.cat([out, x[..., 2 * pairs:]], -1)


def _exact_bits(seed, first, count):
    """The 16 bits of elements first, first + 1, ..., on the host."""
    block = np.arange(first // 8, (first + count + 7) // 8, dtype=np.uint64)
    x = [block % 2 ** 32, block // 2 ** 32, np.zeros_like(block), np.zeros_like(block)]
    for r in range(10):
        keys = [(seed % 2 ** 32 + r * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32]
        first_product, second_product = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [second_product // 2 ** 32 ^ x[1] ^ np.uint64(keys[0]), second_product % 2 ** 32,
             first_product // 2 ** 32 ^ x[3] ^ np.uint64(keys[1]), first_product % 2 ** 32]
    words = np.stack(x, 1).astype("<u4")
    return words.view("<u2").reshape(-1)[first % 8:first % 8 + count]
