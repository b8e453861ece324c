"""Numerics of the block operators (experts, rotary positions, dropout) on the GPU, against their definitions
in 64 bits on the same inputs.

Tolerances are error bounds of the formulas, not measured: U is the unit roundoff of fp32 (2^-24), `uo` that of
the output's type.  A sum of n products, each added by a fused operation, is off by at most n U times the sum
of their magnitudes; rounding the output adds uo times what is rounded.  Whole numbers and truth values are
equal, and so are results that are whole numbers below 2^24.
"""
import math

import numpy as np
import pytest
import torch

import block_oracle as oracle
from all_gather_placement_amd import (dropout, dropout_bwd, expert_combine, expert_combine_bwd, expert_dispatch,
                                      expert_dispatch_bwd, expert_sort, rotary, rotary_bwd, rotary_freqs)
from test_gpu_step import BF16, DTYPES, FP32, U, gen, normal, say, uo, whole, within

pytestmark = pytest.mark.gpu
NAN = float("nan")


def nans(shape, dtype):
    return torch.full(shape, NAN, dtype=dtype, device="cuda")


def framed(rows, cols, dtype, left=3, right=2):
    """A matrix of NaN inside a larger buffer of NaN, and the buffer."""
    buf = nans((rows + 2, cols + left + right), dtype)
    return buf[1:-1, left:left + cols], buf


def untouched(buf, inner):
    """Whether everything beside `inner` is still NaN."""
    return int(buf.isnan().sum()) - int(inner.isnan().sum()) == buf.numel() - inner.numel()


# ------------------------------------------------------------------------------------------------
# Experts: sort
# ------------------------------------------------------------------------------------------------

def make_ids(tokens, choices, experts, kind, seed):
    g = gen(seed)
    if kind == "one":  # all to the last expert
        return torch.full((tokens, choices), experts - 1, device="cuda")
    if kind == "none":
        return torch.where(torch.rand((tokens, choices), device="cuda", generator=g) < 0.5, -1, experts)
    ids = (torch.rand((tokens, choices), device="cuda", generator=g).square() * experts).long().clamp(max=experts - 1)
    if kind == "some":
        drop = torch.rand((tokens, choices), device="cuda", generator=g)
        ids = ids.masked_fill(drop < 0.2, -1).masked_fill(drop > 0.9, experts).masked_fill(drop > 0.99, -(1 << 31))
    return ids


def check_sort(ids, experts, align):
    got = expert_sort(ids, experts, align=align)
    pairs = ids.numel()
    rows = pairs + min(experts, pairs) * (align - 1)
    assert got.source.shape == (rows,) and got.place.shape == ids.shape and got.offsets.shape == (experts + 1,)
    want = oracle.sort(ids.cpu().numpy(), experts, align, rows)
    for name, g, w in zip(got._fields, got, want):
        assert g.dtype == torch.int32 and np.array_equal(g.cpu().numpy(), w), name
    return got


@pytest.mark.parametrize("kind", ["all", "some", "none", "one"])
@pytest.mark.parametrize("tokens,choices,experts", [
    (0, 4, 3), (1, 1, 1), (1, 64, 5), (17, 8, 128), (63, 1, 7), (512, 8, 64), (513, 8, 60), (1365, 3, 129), (4097, 1, 513),
    (3000, 5, 1025), (1500, 10, 2048), (70001, 1, 2), (9001, 8, 1000)])
def test_sort(gpu_available, tokens, choices, experts, kind):
    say("sort", tokens, choices, experts, kind)
    ids = make_ids(tokens, choices, experts, kind, tokens + experts)
    check_sort(ids, experts, 1)
    check_sort(ids.int(), experts, 16 if experts > 500 else 128)


def test_sort_of_many_pairs(gpu_available):
    """More pairs than a workgroup holds in registers."""
    say("sort of 2.6 million pairs")
    ids = make_ids(328_001, 8, 128, "some", 1)
    place, source, offsets = expert_sort(ids, 128, align=16)
    flat = ids.reshape(-1)
    inside = (flat >= 0) & (flat < 128)
    order = torch.argsort(torch.where(inside, flat, 128), stable=True)[:int(inside.sum())]
    counts = torch.bincount(flat[inside], minlength=128)
    want = torch.cat([torch.zeros(1, device="cuda", dtype=torch.int64), ((counts + 15) // 16 * 16).cumsum(0)])
    assert torch.equal(offsets.long(), want)
    within_expert = torch.arange(len(order), device="cuda") - (counts.cumsum(0) - counts)[flat[order]]
    row = want[flat[order]] + within_expert
    assert torch.equal(place.reshape(-1)[order].long(), row) and int((place >= 0).sum()) == len(order)
    assert torch.equal(source[row].long(), order) and int((source >= 0).sum()) == len(order)


def test_sort_ids_of_64_bits(gpu_available):
    """Ids that would be experts if their high bits were lost."""
    ids = torch.tensor([[0, 1 << 32], [(1 << 32) + 1, 1], [-(1 << 32), (1 << 62) + 1]], device="cuda")
    place, source, offsets = expert_sort(ids, 2)
    assert place.tolist() == [[0, -1], [-1, 1], [-1, -1]] and source.tolist() == [0, 3, -1, -1, -1, -1]
    assert offsets.tolist() == [0, 1, 2]


def test_sort_into_more_rows(gpu_available):
    ids = make_ids(40, 4, 9, "some", 2)
    source = torch.full((5000,), 77, dtype=torch.int32, device="cuda")
    got = expert_sort(ids, 9, align=8, source=source[:4000])
    assert bool((source[4000:] == 77).all())
    want = oracle.sort(ids.cpu().numpy(), 9, 8, 4000)
    assert all(np.array_equal(g.cpu().numpy(), w) for g, w in zip(got, want))


# ------------------------------------------------------------------------------------------------
# Experts: rows
# ------------------------------------------------------------------------------------------------

# tokens, choices, experts, align, dim: one vector, parts of one, several waves a row, more choices than are in
# flight at a time, rows on every alignment
ROWS = [(1, 1, 1, 1, 1), (3, 2, 4, 1, 2), (5, 3, 4, 4, 7), (40, 8, 16, 1, 8), (40, 1, 3, 16, 33), (17, 4, 5, 1, 100),
        (9, 64, 70, 1, 129), (300, 5, 7, 16, 250), (64, 8, 128, 128, 512), (33, 10, 20, 1, 1001), (20, 6, 60, 8, 2048),
        (7, 2, 8, 1, 5003), (3, 9, 9, 2, 20000), (1000, 3, 40, 1, 24), (0, 2, 3, 4, 64)]


@pytest.fixture(params=ROWS, ids=lambda r: "x".join(map(str, r)))
def routed(request, gpu_available):
    tokens, choices, experts, align, dim = request.param
    ids = make_ids(tokens, choices, experts, "some", dim)
    if tokens > 2:
        ids[1] = -1  # a token without experts
    sort = expert_sort(ids, experts, align=align)
    return dim, sort, sort.place.long(), sort.source.long()


def by_pair(rows, place):
    """[tokens, choices, dim] in 64 bits, zeros for pairs without a row."""
    got = rows.double()[place.clamp(min=0)] if rows.shape[0] else rows.new_zeros((*place.shape, rows.shape[1])).double()
    return torch.where((place >= 0)[..., None], got, 0.0)


def sorted_rows(dim, source, dtype, seed, make=normal):
    """Rows of the sorted buffer; those of no pair hold NaN, which must not be read."""
    rows = make((len(source), dim), dtype, seed)
    return rows.masked_fill((source < 0)[:, None], NAN)


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_dispatch(routed, dtype):
    dim, sort, place, source = routed
    say("dispatch", tuple(place.shape), dim, dtype)
    x = normal((place.shape[0], dim), dtype, 1)
    want = torch.zeros((len(source), dim), dtype=dtype, device="cuda")
    want[source >= 0] = x[source[source >= 0] // place.shape[1]]
    assert torch.equal(expert_dispatch(x, sort), want)
    out, buf = framed(len(source), dim, dtype)
    xs, _ = framed(place.shape[0], dim, dtype, 5, 4)
    xs.copy_(x)
    assert expert_dispatch(xs, sort, out=out) is out
    assert torch.equal(out, want) and untouched(buf, out)


@pytest.mark.parametrize("weight", [None, BF16, FP32], ids=str)
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_combine(routed, dtype, weight):
    dim, sort, place, source = routed
    say("combine", tuple(place.shape), dim, dtype, weight)
    rows = sorted_rows(dim, source, dtype, 1)
    w = None if weight is None else normal(place.shape, weight, 2).masked_fill(place < 0, NAN)
    parts = by_pair(rows, place)
    if w is not None:
        parts = parts * torch.where(place >= 0, w.double(), 0.0)[..., None]
    want, size = parts.sum(1), parts.abs().sum(1)
    tol = place.shape[1] * U * size
    tol = tol + uo(dtype) * (want.abs() + tol) + 1e-44
    got = expert_dispatch_bwd(rows, sort) if w is None else expert_combine(rows, w, sort)
    within(got, want, tol, "y")
    assert not bool(got[(place < 0).all(1)].any())
    out, buf = framed(place.shape[0], dim, dtype)
    rs, _ = framed(len(source), dim, dtype, 1, 8)
    rs.copy_(rows)
    assert expert_combine(rs, w, sort, out=out) is out
    assert torch.equal(out, got) and untouched(buf, out)


@pytest.mark.parametrize("weight", [BF16, FP32], ids=str)
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_combine_bwd(routed, dtype, weight):
    dim, sort, place, source = routed
    say("combine_bwd", tuple(place.shape), dim, dtype, weight)
    rows, dy = sorted_rows(dim, source, dtype, 1), normal((place.shape[0], dim), dtype, 3)
    w = normal(place.shape, weight, 2).masked_fill(place < 0, NAN)
    drows, dw = expert_combine_bwd(dy, rows, w, sort)
    real = source >= 0
    want = w.double().reshape(-1)[source[real]][:, None] * dy.double()[source[real] // place.shape[1]]
    within(drows[real], want, (uo(dtype) * (1 + U) + U) * want.abs() + 1e-44, "drows")
    assert not bool(drows[~real].any())
    parts = by_pair(rows, place) * dy.double()[:, None]
    want, size = parts.sum(2), parts.abs().sum(2)
    tol = dim * U * size
    within(dw, want, tol + uo(weight) * (want.abs() + tol) + 1e-44, "dweights")
    assert not bool(dw[place < 0].any())
    # other strides, and in place
    out, buf = framed(len(source), dim, dtype)
    ds, _ = framed(place.shape[0], dim, dtype, 7, 0)
    ds.copy_(dy)
    again = expert_combine_bwd(ds, rows, w, sort, drows=out, dweights=torch.empty_like(w))
    assert torch.equal(out, drows) and torch.equal(again[1], dw) and untouched(buf, out)
    rs, buf = framed(len(source), dim, dtype, 1, 1)
    rs.copy_(rows)
    again = expert_combine_bwd(dy, rs, w, sort, drows=rs)
    assert again[0] is rs and torch.equal(rs, drows) and torch.equal(again[1], dw) and untouched(buf, rs)


def test_gradients_of_experts_are_differences(gpu_available):
    """Whole numbers: the operators are linear in each input, and their differences are exact."""
    for dim, choices in ((64, 3), (37, 9), (4104, 2)):
        say("differences of combine", dim, choices)
        sort = expert_sort(make_ids(50, choices, 11, "some", 4), 11, align=4)
        x, dy = whole((50, dim), FP32, 1), whole((50, dim), FP32, 2)
        w, step = whole(sort.place.shape, FP32, 3), whole(sort.place.shape, FP32, 4)
        rows, move = expert_dispatch(x, sort), whole((len(sort.source), dim), FP32, 5)
        drows, dw = expert_combine_bwd(dy, rows, w, sort)
        y = expert_combine(rows, w, sort)
        dot = lambda a, b: float((a.double() * b.double()).sum())
        assert dot(dy, expert_combine(rows + move, w, sort) - y) == dot(drows, move)
        assert dot(dy, expert_combine(rows, w + step, sort) - y) == dot(dw, step)
        dx = expert_dispatch_bwd(drows, sort)
        move = whole((50, dim), FP32, 6)
        assert dot(drows, expert_dispatch(x + move, sort) - rows) == dot(dx, move)
        # a token that names an expert twice
        sort = expert_sort(torch.full((4, choices), 3, device="cuda"), 5)
        assert torch.equal(expert_combine(expert_dispatch(x[:4], sort), None, sort), x[:4] * choices)


@pytest.mark.parametrize("dim", [3, 8, 77])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_dispatch_moves_bits(gpu_available, dtype, dim):
    """Every bit pattern: denormal numbers and what a NaN carries."""
    bits = torch.int16 if dtype == BF16 else torch.int32
    low, high = torch.iinfo(bits).min, torch.iinfo(bits).max
    x = torch.randint(low, high, (900, dim), device="cuda", generator=gen(1)).to(bits)
    sort = expert_sort(make_ids(900, 2, 7, "some", 2), 7)
    rows = expert_dispatch(x.view(dtype), sort).view(bits)
    real = sort.source >= 0
    assert torch.equal(rows[real], x[sort.source[real].long() // 2]) and not bool(rows[~real].any())


@pytest.mark.parametrize("dtype", DTYPES, ids=str)
def test_experts_special_values(gpu_available, dtype):
    sort = expert_sort(torch.tensor([[0, -1], [1, 0], [-1, -1]], device="cuda"), 2, align=4)
    x = normal((3, 70), dtype, 1)
    x[0, 3], x[1, 5], x[1, 69], x[2] = math.inf, NAN, -math.inf, NAN
    rows = expert_dispatch(x, sort)
    assert int(rows.isnan().sum()) == 2 and torch.equal(rows[0], x[0]) and not bool(rows[2:4].any())
    w = torch.tensor([[0.0, NAN], [1.0, 0.5], [NAN, NAN]], device="cuda")
    y = expert_combine(rows, w, sort)
    assert bool(y[0, 3].isnan()) and int(y[0].isnan().sum()) == 1  # 0 * infinity
    assert bool(y[1, 5].isnan()) and float(y[1, 69]) == -math.inf and int(y[1].isnan().sum()) == 1
    assert not bool(y[2].any())
    drows, dw = expert_combine_bwd(torch.ones_like(x), rows, w, sort)
    assert float(dw[0, 0]) == math.inf and bool(dw[1].isnan().all()) and dw[0, 1] == 0 and not bool(dw[2].any())
    assert bool((drows[0] == 0).all()) and bool((drows[4] == 1).all()) and bool((drows[1] == 0.5).all())


def test_numbers_that_no_sort_gives_touch_nothing_outside(gpu_available):
    """Rows and pairs outside the tensors count as none."""
    x, dy = normal((6, 40), FP32, 1), normal((6, 40), FP32, 2)
    place = torch.tensor([[0, 99], [-7, 1 << 30], [5, 2], [-(1 << 31), 3], [4, 12], [1, 1 << 29]], dtype=torch.int32, device="cuda")
    source = torch.tensor([0, 10, 5, 7, 8, 4, 12, 1 << 30, -9, (1 << 31) - 1, -1, -(1 << 31)], dtype=torch.int32, device="cuda")
    sort = (place, source, source)
    out, buf = framed(12, 40, FP32)
    expert_dispatch(x, sort, out=out)
    real = (source >= 0) & (source < 12)
    assert torch.equal(out[real], x[source[real].long() // 2]) and not bool(out[~real].any()) and untouched(buf, out)
    rows = normal((12, 40), FP32, 3)
    w = normal((6, 2), FP32, 4)
    y, buf = framed(6, 40, FP32)
    expert_combine(rows, w, sort, out=y)
    there = (place >= 0) & (place < 12)
    parts = torch.where(there[..., None], rows.double()[place.long().clamp(0, 11)] * w.double()[..., None], 0.0)
    within(y, parts.sum(1), 3 * U * parts.abs().sum(1), "y")
    assert untouched(buf, y)
    drows, buf = framed(12, 40, FP32)
    _, dw = expert_combine_bwd(dy, rows, w, sort, drows=drows)
    assert not bool(dw[~there].any()) and not bool(drows[~real].any()) and untouched(buf, drows)


# ------------------------------------------------------------------------------------------------
# Rotary positions
# ------------------------------------------------------------------------------------------------

# tokens, heads, dim, sections
ROTARY = [(1, 1, 2, (1,)), (1, 32, 128, (64,)), (5, 3, 6, (1, 2)), (70, 4, 64, (8, 12, 12)), (33, 7, 80, (17, 19)),
          (300, 2, 96, (16, 16, 16)), (9, 40, 128, (22, 21, 21)), (129, 1, 256, (128,)), (11, 5, 100, (3, 4, 5, 6)),
          (2, 1, 1024, (125, 387)), (3, 2, 1021, (1,)), (3, 130, 40, (20,)), (1000, 1, 10, (1, 1, 1, 1, 1)), (4, 9, 31, (7, 8)),
          (2, 3, 18, (1, 1, 1, 1, 1, 1, 1, 1)), (50, 3, 576, (32,)), (257, 20, 90, (39,)),
          (100, 33, 59, (21,)), (65, 40, 126, (20, 21, 22))]


def positions_of(tokens, axes, kind, seed):
    if kind == FP32:
        return torch.empty((axes, tokens), device="cuda").uniform_(-300.0, 5000.0, generator=gen(seed))
    high = 100_000 if kind == torch.int32 else 1 << 40
    return torch.randint(-high // 8, high, (axes, tokens), device="cuda", generator=gen(seed)).to(kind)


def rotary_tolerance(size, want, x, positions, freqs, dtype):
    # cos and sin rounded once, and within 2^-35 by their series; two products and a sum; the angle itself is
    # off by 4 roundings of 64 bits; then the output's rounding
    turn = (positions.double().abs().max() * freqs.abs().max()) * 2.0 ** -51 + 2.0 ** -35
    tol = 4 * U * size + float(turn) * 2 * x.double().abs().amax(-1, keepdim=True)
    return tol + uo(dtype) * (want.abs() + tol) + 1e-44


@pytest.mark.parametrize("kind", [torch.int32, torch.int64, FP32], ids=str)
@pytest.mark.parametrize("pairing", ["halves", "neighbours"])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("tokens,heads,dim,sections", ROTARY, ids=lambda v: str(v).replace(" ", ""))
def test_rotary(gpu_available, tokens, heads, dim, sections, dtype, pairing, kind):
    say("rotary", tokens, heads, dim, sections, dtype, pairing, kind)
    x = normal((tokens, heads, dim), dtype, 1)
    positions, freqs = positions_of(tokens, len(sections), kind, 2), rotary_freqs(sections)
    want, size = oracle.rotary(x, positions, freqs, sections, pairing)
    got = rotary(x, positions, freqs, sections, pairing)
    within(got, want, rotary_tolerance(size, want, x, positions, freqs, dtype), "out")
    want, size = oracle.rotary(x, positions, freqs, sections, pairing, inverse=True)
    back = rotary_bwd(x, positions, freqs, sections, pairing)
    within(back, want, rotary_tolerance(size, want, x, positions, freqs, dtype), "gradient")
    assert torch.equal(got[..., 2 * sum(sections):], x[..., 2 * sum(sections):])
    # heads between others of one buffer, heads before tokens, in place
    buf = nans((tokens, heads + 3, dim), dtype)
    buf[:, 2:2 + heads] = x
    assert torch.equal(rotary(buf[:, 2:2 + heads], positions, freqs, sections, pairing), got)
    heads_first = nans((heads, tokens, dim + 1), dtype)[..., :dim].transpose(0, 1)
    assert rotary(x, positions, freqs, sections, pairing, out=heads_first) is heads_first
    assert torch.equal(heads_first, got)
    assert torch.equal(rotary(heads_first.copy_(x), positions, freqs, sections, pairing), got)
    view = buf[:, 2:2 + heads]
    assert rotary(view, positions, freqs, sections, pairing, out=view) is view
    assert torch.equal(view, got) and untouched(buf, view)


def test_rotary_shapes(gpu_available):
    sections = (2, 3)
    freqs = rotary_freqs(sections, base=500.0)
    x = normal((2, 7, 3, 12), FP32, 1)
    positions = torch.randint(0, 50, (2, 2, 7), device="cuda", generator=gen(2))
    want = rotary(x.view(14, 3, 12), positions.view(2, 14), freqs, sections)
    assert torch.equal(rotary(x, positions, freqs, sections), want.view(x.shape))
    one = rotary(x[0, 0], positions[:, 0, 0].contiguous(), freqs, sections)  # a single token without its dimension
    assert torch.equal(one, want[0])
    for empty in (x[:0], x[:, :0], x[:, :, :0]):
        assert rotary(empty, positions[:, :empty.shape[0], :empty.shape[1]].contiguous(), freqs, sections).shape == empty.shape
    shared = x[:, :, :1].reshape(14, 1, 12).expand(14, 5, 12)  # one head read as five
    got = rotary(shared, positions.view(2, 14), freqs, sections)
    assert torch.equal(got, rotary(shared.contiguous(), positions.view(2, 14), freqs, sections))


def test_rotary_freqs(gpu_available):
    want = [100.0 ** -0.0, 100.0 ** -0.5, 1.0, 100.0 ** (-1 / 3), 100.0 ** (-2 / 3)]
    assert torch.allclose(rotary_freqs((2, 3), base=100.0).cpu(), torch.tensor(want, dtype=torch.float64), rtol=1e-15)
    want = [100.0 ** (-i / 5) for i in range(5)]
    assert torch.allclose(rotary_freqs((2, 3), base=100.0, shared=True).cpu(), torch.tensor(want, dtype=torch.float64), rtol=1e-15)


@pytest.mark.parametrize("pairing", ["halves", "neighbours"])
def test_rotary_quarter_turns_are_exact(gpu_available, pairing):
    """At multiples of a quarter turn whole numbers go to whole numbers, and the gradient turns them back.

    An angle of up to 44 quarters is off by 2^-51 of itself, less than 2^-44, so its sine or cosine that should
    be 0 is less than 2^-44, and the other is 1 to fp32.  With |x| <= 1000 that leaves less than 2^-34 beside a
    whole number, which fp32 keeps only where that number is 0.
    """
    x = whole((64, 3, 32), FP32, 1, -1000, 1001)
    positions = torch.arange(-20, 44, device="cuda")[None]
    freqs = torch.full((16,), math.pi / 2, dtype=torch.float64, device="cuda")
    got = rotary(x, positions, freqs, (16,), pairing)
    want, _ = oracle.rotary(x, positions, freqs, (16,), pairing)
    within(got, want.round(), 2.0 ** -34, "turned")
    within(rotary_bwd(got, positions, freqs, (16,), pairing), x.double(), 2.0 ** -33, "turned back")
    # <dy, f(x + d) - f(x)> = <gradient, d>, of 6144 products of numbers up to 1000
    dy, d = whole(x.shape, FP32, 2), whole(x.shape, FP32, 3)
    diff = rotary(x + d, positions, freqs, (16,), pairing) - got
    grad = rotary_bwd(dy, positions, freqs, (16,), pairing)
    assert abs(float((dy.double() * diff.double()).sum()) - float((grad.double() * d.double()).sum())) < 6144 * 2.0 ** -30


def test_rotary_special_values(gpu_available):
    x = normal((4, 2, 8), FP32, 1)
    x[1, 0, 1], x[2, 1, 7] = math.inf, NAN
    positions = torch.tensor([[0.0, 1.0, 0.0, math.inf], [0.0, 2.0, NAN, 1.0]], device="cuda")
    got = rotary(x, positions, rotary_freqs((1, 2)), (1, 2), "neighbours")
    assert torch.equal(got[0], x[0])  # position 0 turns nothing
    assert torch.equal(got[..., 6:].isnan(), x[..., 6:].isnan())
    assert not bool(got[1, 0, :2].isfinite().any()) and bool(got[1, 0, 2:].isfinite().all())
    assert torch.equal(got[2, :, :2], x[2, :, :2]) and bool(got[2, :, 2:6].isnan().all())
    assert bool(got[3, :, :2].isnan().all()) and bool(got[3, :, 2:].isfinite().all())


# ------------------------------------------------------------------------------------------------
# Dropout
# ------------------------------------------------------------------------------------------------

def check_dropout(x, p, seed, offset, residual):
    keep = oracle.keep(x.numel(), p, seed, offset).to("cuda").view(x.shape)
    scaled = torch.where(keep, x.double() * oracle.scale_of(p), 0.0)
    add = 0.0 if residual is None else residual.double()
    want, size = scaled + add, scaled.abs() + (0.0 if residual is None else add.abs())
    got = dropout(x, p, seed, offset=offset, residual=residual)
    tol = 3 * U * size  # the scale's rounding, the product's, the sum's
    within(got, want, tol + uo(x.dtype) * (want.abs() + tol) + 1e-44, "out")
    if residual is None:
        assert not bool(got[~keep].any())
    else:
        assert torch.equal(got[~keep], residual[~keep])
    return got, keep


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", DTYPES, ids=str)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (3, 8), (5, 13), (1, 4096), (40, 33), (2, 2049), (700, 3), (9, 1000)])
def test_dropout(gpu_available, rows, cols, dtype, residual):
    for i, (p, offset) in enumerate(((0.1, 0), (0.5, 3), (0.25, 1 << 35), (1 / 3, 12345678901), (0.0, 1), (1.0, 0), (3e-5, 0))):
        say("dropout", rows, cols, dtype, residual, p, offset)
        seed = (-5, 7, (1 << 64) - 1, 1 << 63, 0x123456789abcdef, 0, 1)[i]
        x, r = normal((rows, cols), dtype, 1), normal((rows, cols), dtype, 2) if residual else None
        got, _ = check_dropout(x, p, seed, offset, r)
        signed = seed - (1 << 64) if seed >= 1 << 63 else seed
        there = torch.tensor([signed], device="cuda")
        assert torch.equal(dropout(x, p, there, offset=offset, residual=r), got)
        assert torch.equal(dropout(x, p, signed, offset=offset, residual=r), got)
        if not residual:
            assert torch.equal(dropout_bwd(x, p, seed, offset=offset), got)
        # other strides, in place of x, in place of the residual
        out, buf = framed(rows, cols, dtype)
        xs, _ = framed(rows, cols, dtype, 1, 6)
        xs.copy_(x)
        assert dropout(xs, p, seed, offset=offset, residual=r, out=out) is out
        assert torch.equal(out, got) and untouched(buf, out)
        xs, buf = framed(rows, cols, dtype, 1, 6)
        xs.copy_(x)
        dropout(xs, p, seed, offset=offset, residual=r, out=xs)
        assert torch.equal(xs, got) and untouched(buf, xs)
        if residual:
            assert dropout(x, p, seed, offset=offset, residual=r, out=r) is r
            assert torch.equal(r, got)


def test_dropout_of_parts_is_that_of_the_whole(gpu_available):
    x = normal((50, 1001), BF16, 1)
    want = dropout(x, 0.3, 99, offset=17)
    for lo, hi in ((0, 1), (1, 20), (20, 50)):
        assert torch.equal(dropout(x[lo:hi], 0.3, 99, offset=17 + lo * 1001), want[lo:hi])
    assert torch.equal(dropout(x.view(5, 10, 1001), 0.3, 99, offset=17), want.view(5, 10, 1001))
    assert torch.equal(dropout(x.reshape(-1), 0.3, 99, offset=17), want.view(-1))
    assert not torch.equal(dropout(x, 0.3, 98, offset=17), want)
    assert dropout(x[:0], 0.3, 1).shape == (0, 1001)


def test_dropout_drops_whatever_an_element_holds(gpu_available):
    x = torch.full((4, 100), NAN, device="cuda")
    x[1], x[2] = math.inf, -math.inf
    keep = oracle.keep(400, 0.5, 3).view(4, 100).to("cuda")
    got = dropout(x, 0.5, 3)
    assert not bool(got[~keep].any()) and torch.equal(got[1][keep[1]], x[1][keep[1]]) and bool(got[3][keep[3]].isnan().all())
    assert not bool(dropout(x, 1.0, 3).any())
    r = normal((4, 100), FP32, 1)
    assert torch.equal(dropout(x, 1.0, 3, residual=r), r)
    assert torch.equal(dropout(r, 0.0, 3), r)


def test_dropout_gradient_is_a_difference(gpu_available):
    """Whole numbers and p = 1/2: doubled or dropped, exactly."""
    x, d, dy = whole((300, 77), FP32, 1), whole((300, 77), FP32, 2), whole((300, 77), FP32, 3)
    r = whole((300, 77), FP32, 4)
    diff = dropout(x + d, 0.5, 11, residual=r) - dropout(x, 0.5, 11, residual=r)
    grad = dropout_bwd(dy, 0.5, 11)
    assert float((dy.double() * diff.double()).sum()) == float((grad.double() * d.double()).sum())


def test_dropout_of_many_elements(gpu_available):
    """Element numbers beyond 32 bits: the ends of a tensor of 2^32 + 40 elements against the same numbers apart."""
    n = (1 << 32) + 40
    x = torch.ones(n, dtype=BF16, device="cuda")
    got = dropout(x, 0.5, 21, out=x)
    for at in (0, (1 << 31) - 20, (1 << 32) - 24, n - 64):
        keep = oracle.keep(64, 0.5, 21, at).to("cuda")
        assert torch.equal(got[at:at + 64] == 2, keep), at
    kept = sum(int((part == 2).sum()) for part in got.split(1 << 30))
    # within six deviations of a half (the generator's words are independent fair bits to any such test)
    assert abs(kept - n / 2) < 6 * 0.5 * math.sqrt(n)


# ------------------------------------------------------------------------------------------------
# Far offsets
# ------------------------------------------------------------------------------------------------

def test_rows_beyond_32_bit_offsets(gpu_available):
    """A sorted buffer of 2.3e9 elements: its last rows, and the first, as those of a small one."""
    say("far rows")
    dim, tokens, take = 16384, 140_000, 40
    ids = torch.zeros((tokens, 1), dtype=torch.int64, device="cuda")
    ids[:take] = 1  # the first tokens' rows come last
    sort = expert_sort(ids, 2)
    assert int(sort.place[0, 0]) == tokens - take
    x = torch.zeros((tokens, dim), dtype=BF16, device="cuda")
    x[:take], x[take:2 * take] = normal((take, dim), BF16, 1), normal((take, dim), BF16, 2)
    rows = expert_dispatch(x, sort)
    assert torch.equal(rows[tokens - take:], x[:take]) and torch.equal(rows[:take], x[take:2 * take])
    w = torch.full((tokens, 1), 2.0, device="cuda")
    y = expert_combine(rows, w, sort)
    assert torch.equal(y[:2 * take], 2 * x[:2 * take]) and not bool(y[-take:].any())
    del y
    drows, dw = expert_combine_bwd(x, rows, w, sort, drows=rows)
    assert drows is rows and torch.equal(rows[tokens - take:], 2 * x[:take]) and torch.equal(rows[:take], 2 * x[take:2 * take])
    size = x[:2 * take].double().square().sum(1)
    within(dw[:2 * take, 0], size, dim * U * size, "dweights")


def test_heads_beyond_32_bit_offsets(gpu_available):
    say("far heads")
    tokens, heads, dim, sections = 70_000, 128, 256, (60, 68)
    x = torch.zeros((tokens, heads, dim), dtype=BF16, device="cuda")
    x[-8:], x[:8] = normal((8, heads, dim), BF16, 1), normal((8, heads, dim), BF16, 2)
    positions, freqs = positions_of(tokens, 2, torch.int64, 3), rotary_freqs(sections)
    ends = [(part, rotary(x[part], positions[:, part].contiguous(), freqs, sections).clone()) for part in (slice(0, 8), slice(tokens - 8, tokens))]
    rotary(x, positions, freqs, sections, out=x)
    for part, want in ends:
        assert torch.equal(x[part], want)
