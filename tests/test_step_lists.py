"""What counts as a list of gradients (no GPU: refusals alone)."""
import pytest

import all_gather_placement_amd as tide

torch = pytest.importorskip("torch")


def test_a_matrix_is_a_list_of_its_rows():
    """Not asked for its truth, which a tensor of more than one value does not have."""
    for call in (lambda g: tide.grad_norm(g), lambda g: tide.clip_grad_norm(g, 1.0)):
        for grads in (torch.zeros(2, 3), (torch.zeros(3), torch.zeros(2))):
            with pytest.raises(ValueError, match="grads must be on the current device"):
                call(grads)
