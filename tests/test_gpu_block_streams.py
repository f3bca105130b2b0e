"""The block's and the mixer's scratch: a captured call keeps its own whatever
sizes are called between its replays, and calls on two streams share none."""
import numpy as np
import pytest
import torch

from gated_delta_rule_02_amd import kda as K
from gated_delta_rule_02_amd import layer, synth
from tests.gpu_util import announce, dev

pytestmark = pytest.mark.gpu

B, N, H, W = 3, 5, 2, 256


def build(fp8):
    if fp8:
        mixer = layer.KDAMixerFP8.from_host(synth.workload_layer_fp8(T=8, hidden=256, H=H, seed=41))
    else:
        mixer = layer.KDAMixer.from_host(synth.workload_layer(T=8, hidden=256, H=H, seed=41))
    w = (torch.rand(256, generator=torch.Generator().manual_seed(41)) + 0.5).cuda()
    return layer.KDABlock(mixer, w)


def draws(seed):
    """States of B sequences, one token and one tree of drafts for each."""
    g = torch.Generator().manual_seed(seed)
    state = (torch.randn((B, H, 128, 128), generator=g) * 0.1).cuda()
    conv = torch.randn((3, B, 3, W), generator=g).bfloat16().cuda()
    token, drafts = torch.randn((B, 256), generator=g).cuda(), torch.randn((B * N, 256), generator=g).cuda()
    parents = torch.tensor([[-1, 0, 0, 1, 2], [-1, -1, 1, 2, 0], [-1, 0, -2, 1, 3]], dtype=torch.int32, device="cuda")
    accepted = torch.tensor([3, 4, 4], dtype=torch.int32, device="cuda")
    return state, conv, token, drafts, parents, accepted


def other_calls(block):
    """Calls of other sizes, and new tensors in whatever memory they freed."""
    block.forward(torch.ones((70, 256), device="cuda"))
    block.mixer.forward(torch.ones((33, 256), device="cuda").bfloat16())
    rows = 2 * N
    state, conv = torch.zeros((rows, H, 128, 128), device="cuda"), torch.zeros((3, rows, 3, W), device="cuda").bfloat16()
    block.decode(torch.ones((rows, 256), device="cuda"), state, conv)
    _, tree = block.decode_tree(torch.ones((rows, 256), device="cuda"),
                                torch.zeros((2, N), dtype=torch.int32, device="cuda") - 1, state[:2], conv[:, :2].contiguous())
    tree.commit(torch.zeros(2, dtype=torch.int32, device="cuda"), state[:2], conv[:, :2].contiguous())
    junk = [torch.full((n,), float("nan"), device="cuda") for n in (64, 4096, 70 * 1288, 1 << 18) for _ in range(8)]
    torch.cuda.synchronize()
    return junk


@pytest.mark.parametrize("fp8", [False, True])
def test_captured_block_keeps_its_scratch(fp8):
    """A decode step and a tree step with its commit, captured; between the replays
    the same block prefills, decodes and verifies other sizes. Every replay equals
    the eager calls bit for bit (the same kernels on the same inputs)."""
    announce("captured block fp8=%s" % fp8)
    block = build(fp8)
    state, conv, token, drafts, parents, accepted = draws(1)

    def step(state, conv, token, drafts):
        d1 = block.decode(token, state, conv)
        d2, tree = block.decode_tree(drafts, parents, state, conv)
        tree.commit(accepted, state, conv)
        return d1, d2, tree

    eager = [t.clone() for t in (state, conv)]
    want = []
    for r in range(4):
        tk, dr = token + r, drafts - r
        d1, d2, _ = step(*eager, tk, dr)
        torch.cuda.synchronize()
        want.append([t.clone() for t in (tk, dr, *eager)] + ([d1.clone(), d2.clone()] if fp8 else []))
    kept = dict(block.mixer._bufs)
    tk, dr = token.clone(), drafts.clone()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            d1, d2, tree = step(state, conv, tk, dr)
    torch.cuda.synchronize()
    # the capture took none of the kept buffers and left none of its own to be replaced
    assert block.mixer._bufs.keys() == kept.keys() and all(block.mixer._bufs[n] is kept[n] for n in kept)
    assert not {t.data_ptr() for t in kept.values()} & {t.untyped_storage().data_ptr() for t in
                                                       (tree.k, tree.g, tree.writes, *tree.inputs)}
    for r in range(4):
        junk = other_calls(block)
        tk.copy_(token + r)
        dr.copy_(drafts - r)
        graph.replay()
        torch.cuda.synchronize()
        got = [tk, dr, state, conv] + ([d1, d2] if fp8 else [])
        assert all(torch.equal(a, b) for a, b in zip(got, want[r])), r
        del junk


def test_decode_graph_between_prefills():
    """DecodeGraph replays with prefills and decodes of other sizes between them."""
    announce("decode graph between prefills")
    block = build(False)
    mixer = block.mixer
    state, conv, token, _, _, _ = draws(2)
    x = token.bfloat16()
    s2, c2 = state.clone(), conv.clone()
    want = []
    for r in range(3):
        want.append(mixer.decode(x * (r + 1), s2, c2).clone())
    graph = layer.DecodeGraph(mixer, B, state, conv)
    for r in range(3):
        junk = other_calls(block)
        out = graph.step(x * (r + 1))
        torch.cuda.synchronize()
        assert torch.equal(out, want[r])
        del junk
    assert torch.equal(state, s2) and torch.equal(conv, c2)


@pytest.mark.parametrize("fp8", [False, True])
def test_two_streams_share_no_scratch(fp8):
    """Two streams run the same block at once, equal sizes; each sees what it sees
    alone. (The buffers are compared as well: a race need not show.)"""
    announce("two streams fp8=%s" % fp8)
    block = build(fp8)

    def work(seed):
        state, conv, token, drafts, parents, accepted = draws(seed)
        torch.cuda.synchronize()
        trees = []

        def go():
            outs = []
            for _ in range(6):
                t, d = token.clone(), drafts.clone()
                block.decode(t, state, conv)
                _, tree = block.decode_tree(d, parents, state, conv)
                tree.commit(accepted, state, conv)
                outs += [t, d]
                trees.append(tree)
            return outs + [state, conv]
        return go, trees

    alone = []
    for seed in (3, 4):
        go, _ = work(seed)
        alone.append([t.clone() for t in go()])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    both = [work(3), work(4)]
    got = []
    for s, (go, _) in zip(streams, both):
        with torch.cuda.stream(s):
            got.append(go())
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    first, second = both[0][1][-1], both[1][1][-1]
    assert first.writes.data_ptr() != second.writes.data_ptr() and first.k.data_ptr() != second.k.data_ptr()


def prefill_case(block, T, seed):
    hidden = torch.randn((T, 256), generator=torch.Generator().manual_seed(seed)).cuda()
    return hidden, torch.zeros((1, H, 128, 128), device="cuda"), torch.zeros((3, 1, 3, W), device="cuda").bfloat16()


def test_captured_prefill_keeps_its_workspace():
    """A captured prefill of the block; between the replays a longer one grows the
    binding's workspace. Every replay equals the eager call bit for bit."""
    announce("captured prefill")
    block = build(False)
    hidden, state, conv = prefill_case(block, 200, 1)
    h, s1, c1 = hidden.clone(), state.clone(), conv.clone()
    block.forward(h, final_state=s1, conv_state_out=c1)
    torch.cuda.synchronize()
    kept = dict(K._workspaces)
    buf = hidden.clone()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            block.forward(buf, final_state=state, conv_state_out=conv)
    torch.cuda.synchronize()
    assert K._workspaces.keys() == kept.keys() and all(K._workspaces[n] is kept[n] for n in kept)
    for r in range(4):
        block.forward(torch.ones((1000 + 700 * r, 256), device="cuda"))
        junk = other_calls(block)
        buf.copy_(hidden)
        state.zero_(), conv.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf, h) and torch.equal(state, s1) and torch.equal(conv, c1), r
        del junk


@pytest.mark.parametrize("how", ["current", "argument"])
def test_prefills_on_two_streams_share_no_workspace(how):
    """The same prefill on two streams at once, by the current stream or by the
    stream argument: the results are those of the call alone."""
    announce("prefill on two streams: " + how)
    T, Hc = 700, 4
    cases = []
    for seed in (5, 6):
        d = synth.core_inputs(np.random.default_rng(seed), T, Hc, bf16=True)
        cases.append([dev(d[n]) for n in ("q", "k", "v", "g", "beta")])
    def out():
        return torch.zeros((T, Hc, 128), device="cuda"), torch.zeros((1, Hc, 128, 128), device="cuda")
    alone = []
    for c in cases:
        o, st = out()
        K.kda_prefill(*c, o, final_state=st)
        torch.cuda.synchronize()
        alone.append((o, st))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[out() for _ in range(5)] for _ in cases]
    torch.cuda.synchronize()
    for r in range(5):
        for c, s, g in zip(cases, streams, got):
            if how == "argument":
                K.kda_prefill(*c, g[r][0], final_state=g[r][1], stream=s)
            else:
                with torch.cuda.stream(s):
                    K.kda_prefill(*c, g[r][0], final_state=g[r][1])
    torch.cuda.synchronize()
    for a, g in zip(alone, got):
        for o, st in g:
            assert torch.equal(o, a[0]) and torch.equal(st, a[1])
    index = torch.cuda.current_device()
    bufs = [K._workspaces[index, x.cuda_stream] for x in streams]
    assert bufs[0].data_ptr() != bufs[1].data_ptr()
