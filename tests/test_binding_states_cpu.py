"""States that do not hold what a call reads and writes are refused by the
binding, which alone knows their sizes. No GPU is needed."""
import pytest
import torch

from gated_delta_rule_02_amd import kda as K

B, H, C, W = 4, 2, 256, 4


@pytest.mark.parametrize("state, error", [
    (torch.zeros(B - 1, H, 128, 128), ValueError),
    (torch.zeros(B, H, 128, 128, dtype=torch.bfloat16), TypeError),      # half the bytes
    (torch.zeros(2 * B, H, 128, 128, dtype=torch.bfloat16), TypeError),  # the bytes, not the type
])
def test_decode_step_state(state, error):
    q, beta, o = torch.zeros(B, H, 128), torch.zeros(B, H), torch.zeros(B, H, 128)
    with pytest.raises(error, match="state"):
        K.kda_decode_step(q, q, q, q, beta, state, o)
    with pytest.raises(ValueError, match="GPU"):  # sufficient: on to the next check
        K.kda_decode_step(q, q, q, q, beta, torch.zeros(B, H, 128, 128), o)


@pytest.mark.parametrize("state, error", [
    (torch.zeros(B - 1, W - 1, C), ValueError),
    (torch.zeros(B, W - 2, C), ValueError),
    (torch.zeros(B, W - 1, C, dtype=torch.bfloat16), TypeError),
])
def test_conv_state_update_state(state, error):
    x, w, y = torch.zeros(B, C), torch.zeros(C, W), torch.zeros(B, C)
    with pytest.raises(error, match="conv_state"):
        K.kda_conv_state_update(x, state, w, y)
    with pytest.raises(ValueError, match="GPU"):
        K.kda_conv_state_update(x, torch.zeros(B, W - 1, C), w, y)
