"""The block operators on the GPU where a row's vectors meet between waves, and far from zero; as in the tests of their
numerics, tolerances are error bounds of the formulas."""
import numpy as np
import pytest
import torch

from all_gather_placement_amd import expert_combine_bwd, expert_sort, rotary, rotary_bwd, rotary_freqs
from test_gpu_block import framed, make_ids, untouched
from test_gpu_step import BF16, FP32, U, normal, say, uo, whole, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("choices", [2, 9])
@pytest.mark.parametrize("dim,dtype", [(257, FP32), (259, FP32), (513, FP32), (769, FP32), (1025, FP32), (2051, FP32),
                                       (513, BF16), (519, BF16), (1025, BF16), (1537, BF16), (2049, BF16), (4097, BF16)], ids=str)
def test_gradients_in_place_where_the_last_vectors_are_two_waves(gpu_available, dim, dtype, choices):
    """Rows whose last vector, which ends with the row, and the one before belong to two waves, or to two turns of
    them.  Whole numbers up to 3, and up to 2 of the weights: every product and sum is exact."""
    say("in place", dim, dtype, choices)
    sort = expert_sort(make_ids(3000, choices, 13, "some", dim), 13, align=8)
    place, source = sort.place.long(), sort.source.long()
    x, dy = whole((len(source), dim), dtype, 1, -3, 4), whole((3000, dim), dtype, 2, -3, 4)
    w = whole(place.shape, FP32, 3, -2, 3)
    real = source >= 0
    drows = torch.zeros_like(x)
    drows[real] = dy[source[real] // choices] * w.to(dtype).reshape(-1)[source[real], None]
    dw = torch.zeros_like(w)
    dw.view(-1)[source[real]] = (x[real].float() * dy[source[real] // choices].float()).sum(1)
    for _ in range(3):
        rows, buf = framed(len(source), dim, dtype, 1, 2)
        rows.copy_(x)
        got = expert_combine_bwd(dy, rows, w, sort, drows=rows)
        assert torch.equal(got[1], dw) and torch.equal(rows, drows) and untouched(buf, rows)


@pytest.mark.parametrize("kind", [torch.int64, FP32], ids=str)
@pytest.mark.parametrize("pairing", ["halves", "neighbours"])
@pytest.mark.parametrize("dtype", [FP32, BF16], ids=str)
def test_rotary_of_far_positions(gpu_available, dtype, pairing, kind):
    """Positions up to 2^62: sine and cosine of the angle in 64 bits, off by their rounding to fp32 (2^-25 of a number
    up to 1) and 2^-35 before it, however far the position is."""
    say("far positions", dtype, pairing, kind)
    exponents = np.arange(63)
    far = np.concatenate([sign * (1 << exponents) + odd for sign in (-1, 1) for odd in (-1, 0, 1)])
    positions = torch.from_numpy(far)[None].to(kind)
    freqs = rotary_freqs((9,), base=1000.0)
    x = normal((positions.shape[1], 2, 18), dtype, 1)
    a = positions.double().numpy()[0][:, None] * freqs.cpu().numpy()
    c, s = (torch.from_numpy(f(a))[:, None] for f in (np.cos, np.sin))
    u, v = (x[..., :9], x[..., 9:]) if pairing == "halves" else (x[..., 0::2], x[..., 1::2])
    u, v = u.cpu().double(), v.cpu().double()
    off = (2.0 ** -25 + 2.0 ** -35) * (u.abs() + v.abs())
    for call, sign in ((rotary, 1), (rotary_bwd, -1)):
        got = call(x, positions.cuda(), freqs, (9,), pairing).cpu()
        for g, want, size in zip((got[..., :9], got[..., 9:]) if pairing == "halves" else (got[..., 0::2], got[..., 1::2]),
                                 (u * c - sign * v * s, v * c + sign * u * s),
                                 ((u * c).abs() + (v * s).abs(), (v * c).abs() + (u * s).abs())):
            tol = off + 2 * U * (size + off)  # two products and a sum in fp32
            within(g, want, tol + uo(dtype) * (want.abs() + tol) + 1e-44, call.__name__)


@pytest.mark.parametrize("pairing", ["halves", "neighbours"])
@pytest.mark.parametrize("dtype", [FP32, BF16], ids=str)
def test_a_pair_is_turned_the_same_wherever_it_lies(gpu_available, dtype, pairing):
    """Bit for bit: in vectors that overlap, in whole ones, and alone."""
    say("pairs", dtype, pairing)
    positions, freqs = torch.arange(3000, device="cuda")[None] * 7, rotary_freqs((128,))
    u, v = normal((2, 3000, 3, 128), dtype, 1)

    def turned(first, pairs, dim):
        x = normal((3000, 3, dim), dtype, 2)
        at = torch.arange(pairs, device="cuda")
        one, two = (at, pairs + at) if pairing == "halves" else (2 * at, 2 * at + 1)
        x[..., one], x[..., two] = u[..., first:first + pairs], v[..., first:first + pairs]
        got = rotary(x, positions, freqs[first:first + pairs].contiguous(), (pairs,), pairing)
        return torch.stack([got[..., one], got[..., two]])

    want = turned(0, 128, 256)
    for first, pairs, dim in ((0, 39, 90), (40, 39, 78), (3, 21, 59), (100, 26, 52), (5, 63, 126), (90, 9, 18), (7, 2, 6)):
        assert torch.equal(turned(first, pairs, dim), want[..., first:first + pairs]), (first, pairs, dim)
    for first in (0, 1, 2, 3, 4, 5, 6, 7, 127):
        assert torch.equal(turned(first, 1, 2), want[..., first:first + 1]), first
