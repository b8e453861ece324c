"""How near the gradient norm and clipping are to their definitions: squares and sums are held in 64 bits.

The square of an fp32 or bf16 value has at most 48 bits, so it is exact in 64; a sum of n squares in any
order is off by at most (n - 1) 2^-53 of itself.  References are sums in 80 bits on the host."""
import math

import numpy as np
import pytest
import torch

from all_gather_placement_amd import clip_grad_norm, grad_clip, grad_norm
from test_gpu_step import BF16, FP32, U, normal, off_by_one, say, uo, within

pytestmark = pytest.mark.gpu

D = 2.0 ** -53


def sum_of_squares(grads):
    total = np.longdouble(0)
    for g in grads:
        total += np.square(g.double().cpu().numpy().astype(np.longdouble)).sum()
    return total


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=str)
@pytest.mark.parametrize("sizes", [[1], [2, 3], [4096 * 8], [4096 * 8 + 1], [31] * 5, [9000] * 251, [300_001], [5, 100_000, 77_777],
                                   [1000 + 17 * i for i in range(170)]], ids=lambda s: f"{len(s)}x{max(s)}")
def test_sum_of_squares_is_held_in_64_bits(gpu_available, sizes, dtype):
    say("sum of squares", len(sizes), max(sizes), dtype)
    grads = [normal((n,), dtype, 50 + i, 10.0 ** (i % 5 - 3)) for i, n in enumerate(sizes)]
    grads = [off_by_one(g) if i % 2 else g for i, g in enumerate(grads)]
    n, total = sum(sizes), sum_of_squares(grads)
    root = float(np.sqrt(total))
    sumsq = torch.full((), float("nan"), dtype=torch.float64, device="cuda")
    norm = grad_norm(grads, sumsq=sumsq)
    assert abs(np.longdouble(float(sumsq)) - total) <= n * D * total
    # the root halves the sum's error; its own rounding in 64 bits, then the one to fp32
    near = (n / 2 + 1) * D
    assert abs(float(norm) - root) <= (near + U * (1 + near)) * root
    for max_norm in (root / 3, root * 0.999):
        coef = max_norm / (root + 1e-6)
        outs = [torch.full_like(g, float("nan")) for g in grads]
        again = torch.full_like(sumsq, float("nan"))
        assert torch.equal(clip_grad_norm(grads, max_norm, outs=outs, sumsq=again), norm) and torch.equal(again, sumsq)
        given = [torch.full_like(g, float("nan")) for g in grads]
        assert torch.equal(grad_clip(grads, sumsq, max_norm, outs=given), norm)
        # the coefficient in 64 bits (three more roundings there) and its rounding to fp32, the product's, the output's
        tol = near + 3 * D + U
        tol = tol + U * (1 + tol)
        for g, o, p in zip(grads, outs, given):
            want = g.double() * coef
            within(o, want, (tol + uo(dtype) * (1 + tol)) * want.abs(), max_norm)
            assert torch.equal(o, p)


@pytest.mark.parametrize("n", [8, 5000, 40_000])
def test_small_squares_count_beside_large_ones(gpu_available, n):
    """In fp32 the small squares would vanish in the sum of any eight neighbours that hold a large one."""
    g = torch.full((n,), 2.0 ** -14, device="cuda")
    g[::8] = 1.0
    big = math.ceil(n / 8)
    want = big + (n - big) * 2.0 ** -28  # exact in 64 bits, as each partial sum
    sumsq = torch.zeros((), dtype=torch.float64, device="cuda")
    grad_norm([g], sumsq=sumsq)
    assert float(sumsq) == want
