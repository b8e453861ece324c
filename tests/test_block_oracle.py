"""The oracle of the block operators against what is published or worked by hand (CPU)."""
import numpy as np
import torch

import block_oracle as oracle


def test_generator_known_answers():
    """The known-answer vectors that the generator's authors publish for philox4x32-10."""
    ones = 0xffffffff
    assert oracle.philox([0] * 4, [0] * 2) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    assert oracle.philox([ones] * 4, [ones] * 2) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    assert oracle.philox([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0]) == [
        0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]


def test_kept_elements():
    whole = oracle.keep(100, 0.3, 5)
    assert torch.equal(oracle.keep(60, 0.3, 5, 40), whole[40:])
    assert bool(oracle.keep(64, 0.0, 1).all()) and not bool(oracle.keep(64, 1.0, 1).any())
    # element 0 of seed 0: the low half of the first word
    u = 0x6627e8d5 & 0xffff
    assert bool(oracle.keep(1, u / 65536, 0)[0]) and not bool(oracle.keep(1, (u + 1) / 65536, 0)[0])
    kept = oracle.keep(40000, 0.25, 12345)
    # a count of 40000 draws of probability 3/4 is within six of its deviations, 86.6 each
    assert abs(int(kept.sum()) - 30000) < 6 * 87


def test_sort_by_hand():
    place, source, offsets = oracle.sort([[2, 0], [-1, 2], [0, 9]], 3, 4, 12)
    assert offsets.tolist() == [0, 4, 4, 8]
    assert place.tolist() == [[4, 0], [-1, 5], [1, -1]]
    assert source.tolist() == [1, 4, -1, -1, 0, 3, -1, -1, -1, -1, -1, -1]


def test_rotary_turns():
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    quarter = torch.full((2,), np.pi / 2, dtype=torch.float64)
    for pairing, want in (("halves", [-3.0, -2.0, 1.0, -4.0, 5.0]), ("neighbours", [-2.0, 1.0, -3.0, -4.0, 5.0])):
        out, _ = oracle.rotary(x, torch.tensor([[1], [2]]), quarter, (1, 1), pairing)
        assert torch.allclose(out, torch.tensor([[want]], dtype=torch.float64), atol=1e-12)
        back, _ = oracle.rotary(out, torch.tensor([[1], [2]]), quarter, (1, 1), pairing, inverse=True)
        assert torch.allclose(back, x.double(), atol=1e-12)
