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


def recorded(monkeypatch):
    """The library's calls as a list of names (nothing is computed), and the
    mixer's buffers on the CPU."""
    calls = []
    for name in ("kda_gemm", "kda_gemm_epilogue", "kda_add_rmsnorm", "kda_conv_tree", "kda_gate_prologue", "kda_decode_tree",
                 "kda_output_norm_gate", "kda_decode_tree_commit", "kda_conv_tree_commit"):
        def call(*a, _name=name, **kw):
            calls.append(_name)
            return a[4] if _name == "kda_conv_tree" else None
        monkeypatch.setattr(K, name, call)

    def buf(self, name, shape, dtype):
        key = (name, tuple(shape), dtype)
        if key not in self._bufs:
            self._bufs[key] = torch.empty(shape, dtype=dtype)
        return self._bufs[key]
    monkeypatch.setattr(layer.KDAMixer, "_buf", buf)
    return calls


@pytest.mark.parametrize("entry", ["block", "mixer"])
def test_overwritten_tree_refuses_to_commit(monkeypatch, entry):
    """After another verification of as many rows (also in trees of another
    shape) a tree's buffers hold that one's; committing it would write the wrong
    path into the states. Its last tree commits, and one of other rows as well."""
    calls = recorded(monkeypatch)
    m = mixer()
    block = layer.KDABlock(m, torch.ones(256))

    def verify(B, N):
        par = torch.zeros((B, N), dtype=torch.int32)
        if entry == "block":
            return block.decode_tree(torch.zeros((B * N, 256)), par, None, [None] * 3)[1]
        return m.decode_tree(torch.zeros((B, N, 256), dtype=torch.bfloat16), par, None, [None] * 3)[1]

    for again in ((2, 6), (3, 4)):
        first = verify(2, 6)
        second = verify(*again)
        calls.clear()
        with pytest.raises(RuntimeError, match="overwritten"):
            first.commit(None, None, [None] * 3)
        assert not calls
        second.commit(None, None, [None] * 3)
        assert calls == ["kda_decode_tree_commit"] + ["kda_conv_tree_commit"] * 3
    first = verify(2, 6)
    verify(1, 6)  # buffers of its own
    first.commit(None, None, [None] * 3)


def test_commit_takes_three_histories(monkeypatch):
    """Fewer histories than streams would leave the others where they were."""
    calls = recorded(monkeypatch)
    m = mixer()
    tree = m.decode_tree(torch.zeros((2, 6, 256), dtype=torch.bfloat16), torch.zeros((2, 6), dtype=torch.int32), None,
                         [None] * 3)[1]
    calls.clear()
    for n in (0, 2, 4):
        with pytest.raises(ValueError, match="conv_states"):
            tree.commit(None, None, [None] * n)
    assert not calls
