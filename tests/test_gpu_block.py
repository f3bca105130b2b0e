"""The pre-norm residual block around the token mixer, and a run of all of its
parts together: prefill, verification of a tree of drafts, commit, decode."""
import numpy as np
import pytest
import torch

from gated_delta_rule_02_amd import layer, synth
from gated_delta_rule_02_amd import kda as K
from oracle import reference as R
from tests.gpu_util import TOL_BF16, announce, dev, host64, relerr

pytestmark = pytest.mark.gpu


def build(T, seed, fp8):
    if fp8:
        d = synth.workload_layer_fp8(T=T, hidden=256, H=2, seed=seed)
        mixer = layer.KDAMixerFP8.from_host(d)
    else:
        d = synth.workload_layer(T=T, hidden=256, H=2, seed=seed)
        mixer = layer.KDAMixer.from_host(d)
    g = torch.Generator().manual_seed(seed)
    w = (torch.rand(256, generator=g) + 0.5).cuda()
    hidden = torch.randn((T, 256), generator=g).cuda() * 2
    return d, layer.KDABlock(mixer, w), hidden


def test_block_forward_matches_oracle_layer():
    """hidden grows by the oracle's layer applied to the block's own normalised
    input, which is the formula's rounded to bfloat16 (half a step, 2^-8, and
    float32's share)."""
    announce("block forward")
    d, block, hidden = build(150, 21, False)
    before = hidden.clone()
    assert block.forward(hidden) is None
    torch.cuda.synchronize()
    y = block.mixer._bufs["ny"]
    h = host64(before)
    ref_y = h / np.sqrt((h * h).mean(1, keepdims=True) + 1e-6) * host64(block.norm_weight)
    assert (np.abs(host64(y) - ref_y) <= (2.0 ** -8 + 1e-5) * np.abs(ref_y)).all()
    ref = R.layer_forward(host64(y).astype(np.float32), d["Wq"].vals, d["Wk"].vals, d["Wv"].vals, d["Wf"].vals,
                          d["Wg"].vals, d["Wb"].vals, d["Wo"].vals, d["conv_q"].vals, d["conv_k"].vals,
                          d["conv_v"].vals, d["A_log"], d["norm_w"], d["H"])
    grown = host64(hidden) - h
    # the stream itself is float32: one rounding of the sum
    assert np.max(np.abs(grown - ref)) <= TOL_BF16 * np.max(np.abs(ref)) + 2.0 ** -24 * np.max(np.abs(host64(hidden)))


def test_block_fp8_is_the_mixer_on_the_norm():
    """The W8A8 block: codes of the norm in one pass equal the two passes' (norm in
    float32, then quantized), so its output equals the mixer's on that norm bit for
    bit; the next norm adds it to the stream."""
    announce("block fp8 forward")
    _, block, hidden = build(130, 22, True)
    before = hidden.clone()
    delta = block.forward(hidden)
    y = torch.empty_like(hidden)
    K.kda_add_rmsnorm(before, block.norm_weight, y)
    out = block.mixer.forward(y)
    torch.cuda.synchronize()
    assert torch.equal(hidden, before) and torch.equal(delta, out)
    z = torch.empty(hidden.shape, dtype=torch.bfloat16, device="cuda")
    block.finish(hidden, delta, block.norm_weight, z)
    torch.cuda.synchronize()
    assert torch.equal(hidden, before + out)


N, B, H, W, T = 7, 2, 2, 256, 40
PARENTS = [[-1, 0, 0, 1, 2, -1, 4], [-1, -1, 1, 2, -2, 3, 4]]  # the second tree lacks node 4, and so 6
PATHS = [[[0], [0, 1], [0, 2], [0, 1, 3], [0, 2, 4], [5], [0, 2, 4, 6]],
         [[0], [1], [1, 2], [1, 2, 3], [], [1, 2, 3, 5], []]]


def prefilled(fp8):
    """A block whose two sequences hold a prefilled context, and drafts for them."""
    _, block, hidden = build(T, 23, fp8)
    cu = torch.tensor([0, 17, T], dtype=torch.int32, device="cuda")
    state = torch.zeros((B, H, 128, 128), device="cuda")
    conv = torch.zeros((3, B, 3, W), dtype=torch.bfloat16, device="cuda")
    block.forward(hidden, cu_seqlens=cu, cu_seqlens_host=cu.cpu(), final_state=state, conv_state_out=conv)
    drafts = torch.randn((B, N, 256), generator=torch.Generator().manual_seed(5)).cuda()
    return block, state, conv, drafts, torch.tensor(PARENTS, dtype=torch.int32, device="cuda")


def test_block_tree_step():
    """Two sequences: prefill, then a tree of drafts verified in one call. Every
    node's output equals decoding the path to it token by token, and after the
    commit of a node the states equal those of that decode; then both go on.
    Either way is within TOL_BF16 of the 64-bit chain (as every form of the layer),
    so they are within twice that of each other; an input of the convolutions is
    a bfloat16 projection, which another order of the product's sum can round to
    the neighbouring value (2^-7 of it)."""
    announce("block tree step")
    block, state, conv, drafts, par = prefilled(False)
    s0, c0 = state.clone(), conv.clone()
    hid = drafts.reshape(B * N, 256).clone()
    delta, tree = block.decode_tree(hid, par, state, conv)
    torch.cuda.synchronize()
    assert delta is None and torch.equal(state, s0) and torch.equal(conv, c0)
    got = hid.view(B, N, 256).clone()

    def decoded(b, p):
        """the path's tokens one by one on sequence b's states"""
        s, c = s0[b:b + 1].clone(), c0[:, b:b + 1].clone()
        for i in p:
            h = drafts[b, i:i + 1].clone()
            block.decode(h, s, c)
        return h, s, c

    for b in range(B):
        for i in range(N):
            if PATHS[b][i]:
                want, _, _ = decoded(b, PATHS[b][i])
                # what the block adds, not the stream it is added to
                assert relerr(host64(got[b, i] - drafts[b, i]), host64(want[0] - drafts[b, i])) < 2 * TOL_BF16, (b, i)
    tree.commit(torch.tensor([4, 5], dtype=torch.int32, device="cuda"), state, conv)
    nxt = torch.randn((B, 256), generator=torch.Generator().manual_seed(6)).cuda()
    both = nxt.clone()
    s1, c1 = state.clone(), conv.clone()
    block.decode(both, s1, c1)
    for b, i in ((0, 4), (1, 5)):
        _, s, c = decoded(b, PATHS[b][i])
        assert relerr(host64(state[b]), host64(s[0])) < 2 * TOL_BF16
        assert relerr(host64(conv[:, b]), host64(c[:, 0])) < 2.0 ** -7
        h = nxt[b:b + 1].clone()
        block.decode(h, s, c)
        assert relerr(host64(both[b] - nxt[b]), host64(h[0] - nxt[b])) < 2 * TOL_BF16


def test_block_fp8_tree_step():
    """The W8A8 block's verification and commit are the library's calls in their
    order, bit for bit (an output behind two quantizations has no closer bound
    than that: one E4M3 code is 2^-3 of its value)."""
    announce("block fp8 tree step")
    block, state, conv, drafts, par = prefilled(True)
    m = block.mixer
    hid = drafts.reshape(B * N, 256).clone()
    pending = torch.randn((B * N, 256), generator=torch.Generator().manual_seed(7)).cuda()  # of the block before
    stream = hid.clone()
    delta, tree = block.decode_tree(stream, par, state, conv, delta=pending)
    acc = torch.tensor([4, 5], dtype=torch.int32, device="cuda")
    s1, c1 = state.clone(), conv.clone()
    tree.commit(acc, s1, c1)

    bf = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")
    f = lambda *s: torch.empty(s, device="cuda")
    u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")
    xq, xs, stream2 = u8(B * N, 256), f(B * N, 2), f(B * N, 256)
    K.kda_add_rmsnorm_fp8(pending, block.norm_weight, xq, xs, residual=hid, residual_out=stream2, eps=block.eps)
    P = bf(B * N, m.W_in.shape[0])
    K.kda_gemm_fp8(xq, xs, m.W_in, m.W_in_s, P)
    cols = [P[:, i * W:(i + 1) * W] for i in range(5)] + [P[:, 5 * W:5 * W + H]]
    qkv = [K.kda_conv_tree(cols[i], conv[i], par, m.conv[i], bf(B * N, W), l2norm_group=l2, l2norm_eps=m.l2_eps)
           .view(B, N, H, 128) for i, l2 in enumerate((128, 128, 0))]
    g, beta = bf(B * N, H, 128), bf(B * N, H)
    K.kda_gate_prologue(cols[3], cols[5], m.A_log, g, beta, H, lower_bound=m.lower_bound)
    g, beta, o, writes = g.view(B, N, H, 128), beta.view(B, N, H), f(B, N, H, 128), f(B, N, H, 128)
    K.kda_decode_tree(*qkv, g, beta, par, state, o, writes, scale=m.scale, lower_bound=m.lower_bound)
    yq, ys, out = u8(B * N, W), f(B * N, H), f(B * N, 256)
    K.kda_output_norm_gate_fp8(o.view(B * N, H, 128), cols[4], m.norm_w, yq, ys, eps=m.rms_eps)
    K.kda_gemm_fp8(yq, ys, m.Wo, m.Wo_s, out)
    torch.cuda.synchronize()
    assert torch.equal(stream, stream2) and torch.equal(delta, out)
    K.kda_decode_tree_commit(qkv[1], g, writes, par, acc, state, lower_bound=m.lower_bound)
    for i in range(3):
        K.kda_conv_tree_commit(cols[i], par, acc, conv[i])
    torch.cuda.synchronize()
    assert torch.equal(state, s1) and torch.equal(conv, c1)


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_survives_a_decode_before_its_commit(fp8):
    """Decoding as many rows as the tree has, between its verification and its
    commit, leaves what the commit needs alone (of the block and of the mixer)."""
    announce("block tree, decode, commit fp8=%s" % fp8)
    block, state, conv, drafts, par = prefilled(fp8)
    acc = torch.tensor([4, 5], dtype=torch.int32, device="cuda")
    rows = B * N
    other = torch.zeros((rows, H, 128, 128), device="cuda"), torch.zeros((3, rows, 3, W), dtype=torch.bfloat16, device="cuda")
    x = torch.randn((rows, 256), generator=torch.Generator().manual_seed(9)).cuda()
    for verify, decode in (
            (lambda: block.decode_tree(drafts.reshape(rows, 256).clone(), par, state, conv)[1],
             lambda: block.decode(x.clone(), *other)),
            (lambda: block.mixer.decode_tree(drafts.bfloat16(), par, state, conv)[1],
             lambda: block.mixer.decode(x.bfloat16(), *other))):
        s1, c1, s2, c2 = state.clone(), conv.clone(), state.clone(), conv.clone()
        verify().commit(acc, s1, c1)
        tree = verify()
        decode()
        tree.commit(acc, s2, c2)
        torch.cuda.synchronize()
        assert torch.equal(s1, s2) and torch.equal(c1, c2) and not torch.equal(s1, state)


def test_calls_on_another_stream_and_without_rows():
    """On a side stream the calls run there (their result waits for that stream's
    work); no rows are no work."""
    announce("other stream, no rows")
    s = torch.cuda.Stream()
    x = torch.ones((64, 1024), device="cuda")
    w, y, y2 = torch.ones(1024, device="cuda"), torch.zeros((64, 1024), device="cuda"), torch.zeros((64, 1024), device="cuda")
    A, Bm = torch.ones((40, 512), device="cuda").bfloat16(), torch.ones((24, 512), device="cuda").bfloat16()
    C, C2 = torch.zeros((40, 24), device="cuda"), torch.zeros((40, 24), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(200):  # a queue of work before the inputs are ready
            x.mul_(1.0)
        x.mul_(3.0)
        A.mul_(2.0)
        K.kda_add_rmsnorm(x, w, y, residual=x)
        K.kda_gemm_epilogue(A, Bm, C)
    K.kda_gemm_epilogue(A, Bm, C2, stream=s)
    K.kda_add_rmsnorm(x, w, y2, residual=x, stream=s)
    torch.cuda.synchronize()
    assert (C == 1024).all() and torch.equal(C, C2) and torch.equal(y, y2)
    assert relerr(host64(y), np.ones((64, 1024))) < 1e-6
    K.kda_add_rmsnorm(x[:0], w, y[:0])
    K.kda_add_rmsnorm_fp8(x[:0], w, torch.empty((0, 1024), dtype=torch.uint8, device="cuda"), torch.empty((0, 8), device="cuda"))
    K.kda_gemm_epilogue(A[:0], Bm, C[:0], residual=C[:0])
    torch.cuda.synchronize()


def test_mixer_decode_tree_matches_decode():
    """The bare mixer: a one-node tree is a decode step (outputs to the projections'
    rounding), commits to the same states."""
    announce("mixer one-node tree")
    d = synth.workload_layer(T=3, hidden=256, H=2, seed=31)
    mixer = layer.KDAMixer.from_host(d)
    x = dev(d["x"])
    B = 3
    g = torch.Generator().manual_seed(1)
    state = (torch.randn((B, 2, 128, 128), generator=g) * 0.1).cuda()
    conv = torch.randn((3, B, 3, 256), generator=g).bfloat16().cuda()
    s2, c2 = state.clone(), conv.clone()
    par = torch.full((B, 1), -1, dtype=torch.int32, device="cuda")
    out, tree = mixer.decode_tree(x.view(B, 1, 256), par, state, conv)
    out = out.clone()
    tree.commit(torch.zeros(B, dtype=torch.int32, device="cuda"), state, conv)
    ref = mixer.decode(x, s2, c2)
    torch.cuda.synchronize()
    assert relerr(host64(out[:, 0]), host64(ref)) < TOL_BF16
    assert relerr(host64(state), host64(s2)) < 1e-5
    assert torch.equal(conv, c2)
