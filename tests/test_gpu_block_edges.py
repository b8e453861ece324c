"""The block operators on the GPU where a row's vectors meet between waves, and far from zero; as in the tests of their
numerics, tolerances are error bounds of the formulas."""
import pytest
import torch

from all_gather_placement_amd import expert_combine_bwd, expert_sort
from test_gpu_block import framed, make_ids, untouched
from test_gpu_step import BF16, FP32, say, whole

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
