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


def prefill(fn, **states):
    T, Hp = 5, 2
    q, beta, o = torch.zeros(T, Hp, 128), torch.zeros(T, Hp), torch.zeros(T, Hp, 128)
    if fn is K.kda_prefill_gated:
        return fn(q, q, q, torch.zeros(T, Hp * 128), beta, torch.zeros(Hp), o, workspace=torch.zeros(16), **states)
    return fn(q, q, q, q, beta, o, **states)


@pytest.mark.parametrize("fn", [K.kda_prefill, K.kda_prefill_gated, K.kda_prefill_noalloc])
@pytest.mark.parametrize("name", ["initial_state", "final_state"])
def test_prefill_states(fn, name):
    with pytest.raises(ValueError, match=name):
        prefill(fn, **{name: torch.zeros(1, 1, 128, 128)})
    with pytest.raises(TypeError, match=name):
        prefill(fn, **{name: torch.zeros(1, 2, 128, 128, dtype=torch.bfloat16)})
    with pytest.raises(ValueError, match=name):
        prefill(fn, **{name: torch.zeros(2, 2, 128, 128)}, num_seqs=5)
    with pytest.raises(ValueError, match="GPU"):
        prefill(fn, **{name: torch.zeros(1, 2, 128, 128)})


@pytest.mark.parametrize("name", ["conv_state_in", "conv_state_out"])
def test_conv_prefill_states(name):
    x, w, y = torch.zeros(5, C), torch.zeros(C, W), torch.zeros(5, C)
    for n, shape in ((1, (1, W - 2, C)), (5, (4, W - 1, C))):
        with pytest.raises(ValueError, match=name):
            K.kda_conv_prefill(x, w, y, num_seqs=n, **{name: torch.zeros(shape)})
    with pytest.raises(TypeError, match=name):
        K.kda_conv_prefill(x, w, y, **{name: torch.zeros(1, W - 1, C, dtype=torch.bfloat16)})
    with pytest.raises(ValueError, match="GPU"):
        K.kda_conv_prefill(x, w, y, **{name: torch.zeros(1, W - 1, C)})
