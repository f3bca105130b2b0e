"""Host-side checks of the block with a norm after it, the 4-bit mixer and the beam
search's bookkeeping: which calls are made on what. No GPU is needed."""
import pytest
import torch

from gated_delta_rule_02_amd import kda as K
from gated_delta_rule_02_amd import layer

H, W = 2, 256
z = torch.zeros


def bf(*shape):
    return z(shape, dtype=torch.bfloat16)


@pytest.fixture
def calls(monkeypatch):
    """The library's calls as (name, arguments); nothing is computed."""
    made = []
    for name in ("kda_gemm", "kda_gemm_epilogue", "kda_gemm_w4", "kda_w4_expand", "kda_add_rmsnorm", "kda_sandwich_rmsnorm",
                 "kda_gate_prologue", "kda_output_norm_gate", "kda_conv_state_update", "kda_decode_step", "kda_beam_select",
                 "kda_beam_reorder"):
        def call(*a, _name=name, **kw):
            made.append((_name, a, kw))
            return a[1] if _name == "kda_w4_expand" else None
        monkeypatch.setattr(K, name, call)
    monkeypatch.setattr(layer.KDAMixer, "_buf", lambda self, name, shape, dtype: torch.empty(shape, dtype=dtype))
    return made


def mixer(kind):
    rest = (bf(W, 4), bf(W, 4), bf(W, 4), z(H), z(128))
    if kind == "w4":
        weight = lambda n: K.W4Weight(z(1, dtype=torch.uint8), n, 256, 64, K.KDA_F32, False)
        return layer.KDAMixerW4(weight(5 * W + 8), weight(256), *rest, H)
    return layer.KDAMixer(bf(5 * W + 8, 256), *rest, bf(256, W), H)


def names(made):
    return [n for n, _, _ in made]


@pytest.mark.parametrize("kind", ["bf16", "w4"])
def test_block_with_a_norm_after_it_leaves_its_output(calls, kind):
    post = layer.BranchNorm(z(256), gate=z(256), gate_activation="sigmoid", residual_scale=0.5)
    block = layer.KDABlock(mixer(kind), z(256), post=post)
    hidden = z((3, 256))
    delta = block.decode(hidden, z((3, H, 128, 128)), bf(3, 3, 3, W))
    assert isinstance(delta, layer.Branch) and delta.post is post and delta.x.shape == (3, 256)
    assert "kda_sandwich_rmsnorm" not in names(calls)
    assert all(kw.get("residual") is None for n, _, kw in calls if n.startswith("kda_gemm"))
    calls.clear()
    block.finish(hidden, delta, z(256), z((3, 256)))
    (name, args, kw), = calls
    assert name == "kda_sandwich_rmsnorm" and args[0] is delta.x and args[2] is hidden and args[3] is hidden
    assert kw["gate_activation"] == "sigmoid" and kw["residual_scale"] == 0.5
    # a block without one takes such a delta as well, and adds its own output in place
    calls.clear()
    assert layer.KDABlock(mixer(kind), z(256)).decode(hidden, z((3, H, 128, 128)), bf(3, 3, 3, W), delta) is None
    assert names(calls)[0] == "kda_sandwich_rmsnorm" and calls[-1][2]["residual"] is hidden


def test_w4_mixer_expands_for_many_rows(calls):
    m = mixer("w4")
    m.projections(bf(m.EXPAND - 1, 256))
    assert names(calls) == ["kda_gemm_w4"]
    calls.clear()
    m.projections(bf(m.EXPAND, 256))
    assert names(calls) == ["kda_w4_expand", "kda_gemm_epilogue"] and calls[1][1][1].shape == (5 * W + 8, 256)


def test_beam_step_moves_every_blocks_states(calls, monkeypatch):
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=torch.float32, device=None: torch.zeros(shape, dtype=dtype))
    B, beams, V = 2, 3, 40
    blocks = [layer.KDABlock(mixer("bf16"), z(256)) for _ in range(2)]
    sts, cvs = [z((6, H, 128, 128)) for _ in blocks], [bf(3, 6, 3, W) for _ in blocks]
    s = layer.BeamSearch(blocks, z(256), bf(V, 256), B, beams, 5, sts, cvs)
    assert s.scores[:, 0].tolist() == [0, 0] and torch.isinf(s.scores[:, 1:]).all() and not s.finished.any()
    assert s.step(z((6, 256))) is s.tokens
    tail = calls[-4:]
    assert names(tail) == ["kda_gemm_epilogue", "kda_beam_select", "kda_beam_reorder", "kda_beam_reorder"]
    assert tail[1][1][0] is s.logits and tail[1][1][1] is s.scores and tail[1][1][2] is s.scores
    assert [t[1][1] is st and t[1][2] is cv for t, st, cv in zip(tail[2:], sts, cvs)] == [True, True]


@pytest.mark.parametrize("V", [40, 41, 42, 43])
def test_logits_rows_suit_the_heads_product(calls, monkeypatch, V):
    """kda_gemm_epilogue takes rows of y whose stride is a multiple of 4, whatever V is."""
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=torch.float32, device=None: torch.zeros(shape, dtype=dtype))
    s = layer.BeamSearch([layer.KDABlock(mixer("bf16"), z(256))], z(256), bf(V, 256), 2, 3, -1, [z((6, H, 128, 128))],
                         [bf(3, 6, 3, W)])
    assert s.logits.shape == (6, V) and s.logits.stride(0) % 4 == 0 and s.logits.stride(1) == 1


def test_search_refuses_what_does_not_fit_together(calls, monkeypatch):
    """Before anything is called: a step refused half-way would leave some states advanced."""
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=torch.float32, device=None: torch.zeros(shape, dtype=dtype))
    block, st, cv = layer.KDABlock(mixer("bf16"), z(256)), z((6, H, 128, 128)), bf(3, 6, 3, W)

    def search(**over):
        a = dict(blocks=[block, block], norm_weight=z(256), head=bf(40, 256), B=2, W=3, eos=5, states=[st, st], conv_states=[cv, cv])
        a.update(over)
        return layer.BeamSearch(**a)

    for bad in (dict(states=[st]), dict(conv_states=[cv]), dict(blocks=[block]), dict(blocks=[], states=[], conv_states=[]),
                dict(states=[st, st[:5]]), dict(states=[st, z((8, H, 128, 128))]), dict(states=[st, z((6, H, 128, 256))[..., :128]]),
                dict(conv_states=[cv, bf(3, 5, 3, W)]), dict(conv_states=[cv, bf(2, 6, 3, W)]), dict(conv_states=[cv, bf(3, 6, 2, W)]),
                dict(W=33, B=1), dict(W=0), dict(B=-1), dict(eos=40), dict(head=bf(40, 128)), dict(norm_weight=z(255)),
                dict(norm_weight=z(128), head=bf(40, 128))):
        with pytest.raises(ValueError):
            search(**bad)
    for bad in (dict(states=[st, bf(6, H, 128, 128)]), dict(conv_states=[cv, z((3, 6, 3, W))]), dict(head=z((40, 256))),
                dict(norm_weight=bf(256))):
        with pytest.raises(TypeError):
            search(**bad)
    s = search(states=(st, st), eos=-1)
    for hidden in (z((5, 256)), z((12, 256)), z((6, 128)), z(6 * 256)):
        with pytest.raises(ValueError, match="hidden must have shape"):
            s.step(hidden)
    assert not calls
    s.step(z((6, 256)))
    assert names(calls)[-2:] == ["kda_beam_reorder"] * 2
