"""Host-side checks of the block and of the draft trees' bookkeeping. No GPU is
needed: the calls that would reach one are refused before, or recorded."""
import pytest
import torch

from gated_delta_rule_02_amd import kda as K
from gated_delta_rule_02_amd import layer

H, W = 2, 256


def mixer():
    z = torch.zeros
    bf = lambda *s: z(s, dtype=torch.bfloat16)
    return layer.KDAMixer(bf(5 * W + 8, 256), bf(W, 4), bf(W, 4), bf(W, 4), z(H), z(128), bf(256, W), H)


def test_mixer_tree_of_another_shape_is_refused():
    """x [2, 6] with parents [3, 4]: the same number of rows, other trees."""
    x = torch.zeros((2, 6, 256), dtype=torch.bfloat16)
    for shape in ((3, 4), (6, 2), (2, 5), (12,)):
        with pytest.raises(ValueError, match="parents must be"):
            mixer().decode_tree(x, torch.zeros(shape, dtype=torch.int32), None, None)
