"""The 4-bit mixer, the block with a norm after it too, and beam search with a stack of
blocks: all of the operators together, as they are used.

Two runs whose sums are taken in another order agree to the tolerance of the mixer's own
tests (2e-3 of the largest value): a projection's bfloat16 columns may land on a neighbouring
value."""
import numpy as np
import pytest
import torch

from gated_delta_rule_02_amd import kda as K
from gated_delta_rule_02_amd import layer, synth
from tests.gpu_util import TOL_BF16, announce, host64, relerr

pytestmark = pytest.mark.gpu

BF, F, I32 = torch.bfloat16, torch.float32, torch.int32
H, WIDTH = 2, 256
U = 2.0 ** -24


def w4(N, k, seed, std=0.02):
    """A 4-bit weight whose values are exact in bfloat16 (scales are powers of two), and they."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (N, k // 2), generator=g, dtype=torch.uint8).cuda()
    scales = (2.0 ** torch.randint(-9, -7, (N, k // 64), generator=g).float()).cuda()
    w = K.kda_w4_pack(codes, scales)
    return w, K.kda_w4_expand(w, torch.empty((N, k), dtype=BF, device="cuda"))


def mixers(seed):
    """The same mixer with 4-bit and with bfloat16 weights."""
    d = synth.workload_layer(T=4, hidden=WIDTH, H=H, seed=seed)
    m = layer.KDAMixer.from_host(d)
    W_in, Wb = w4(m.W_in.shape[0], WIDTH, seed)
    Wo, Wob = w4(WIDTH, H * 128, seed + 1)
    rest = (*m.conv, m.A_log, m.norm_w, H)
    return layer.KDAMixerW4(W_in, Wo, *rest), layer.KDAMixer(Wb, *m.conv, m.A_log, m.norm_w, Wob, H)


def rows(n, seed, dtype=F):
    return torch.randn((n, WIDTH), generator=torch.Generator().manual_seed(seed)).cuda().to(dtype) * 2


def states(B):
    return torch.zeros((B, H, 128, 128), device="cuda"), torch.zeros((3, B, 3, H * 128), dtype=BF, device="cuda")


@pytest.mark.parametrize("T", [1, 5, 40, 130])
def test_w4_mixer_is_the_bf16_mixer_of_its_weights(T):
    announce("w4 mixer T=%d" % T)
    a, b = mixers(T)
    x = rows(T, T, BF)
    assert relerr(host64(a.forward(x)), host64(b.forward(x))) < TOL_BF16
    (s1, c1), (s2, c2) = states(T), states(T)
    for step in range(2):
        o1, o2 = a.decode(x, s1, c1), b.decode(x, s2, c2)
        assert relerr(host64(o1), host64(o2)) < TOL_BF16 and relerr(host64(s1), host64(s2)) < TOL_BF16
    if T % 5 == 0:
        par = torch.tensor([[-1, 0, 0, 1, 2]] * (T // 5), dtype=I32, device="cuda")
        st, cv = s1[:T // 5].clone(), c1[:, :T // 5].contiguous()
        o1, tree = a.decode_tree(x.view(T // 5, 5, WIDTH), par, st, cv)
        o2, _ = b.decode_tree(x.view(T // 5, 5, WIDTH), par, st, cv)
        assert relerr(host64(o1), host64(o2)) < TOL_BF16
        tree.commit(torch.full((T // 5,), 4, dtype=I32, device="cuda"), st, cv)


def test_w4_mixer_from_host_arrays():
    """Codes, scales and zero points on the host, an odd number of rows: the bfloat16 mixer of
    the values they stand for (powers of two as scales: exact)."""
    d = synth.workload_layer(T=4, hidden=WIDTH, H=H, seed=12)
    rng = np.random.default_rng(3)
    for name, n, k in (("Win", 5 * H * 128 + H, WIDTH), ("Wo", WIDTH, H * 128)):
        d[name + "_codes"] = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
        d[name + "_scales"] = (2.0 ** rng.integers(-9, -7, (n, k // 32))).astype(np.float32)
        d[name + "_zeros"] = rng.integers(4, 12, (n, k // 32), dtype=np.uint8)
    m = layer.KDAMixerW4.from_host(d)
    assert m.W_in.shape == (5 * H * 128 + 8, WIDTH) and m.Wo.shape == (WIDTH, H * 128)

    def values(name):
        c = np.stack([d[name + "_codes"] & 15, d[name + "_codes"] >> 4], -1).reshape(d[name + "_codes"].shape[0], -1)
        wide = lambda a: np.repeat(a.astype(np.float32), 32, 1)
        return torch.from_numpy((c - wide(d[name + "_zeros"])) * wide(d[name + "_scales"])).to(BF).cuda()
    win = torch.cat([values("Win"), torch.zeros((6, WIDTH), dtype=BF, device="cuda")])
    b = layer.KDAMixer(win, *m.conv, m.A_log, m.norm_w, values("Wo"), H)
    x = rows(9, 13, BF)
    assert relerr(host64(m.forward(x)), host64(b.forward(x))) < TOL_BF16


def test_w4_block_expanded_equals_bf16_block():
    """Above EXPAND rows the block makes the bfloat16 block's calls on the same values."""
    a, b = mixers(7)
    a.EXPAND = 64
    w = torch.ones(WIDTH, device="cuda")
    h1, h2 = rows(200, 3), rows(200, 3)
    assert layer.KDABlock(a, w).forward(h1) is None and layer.KDABlock(b, w).forward(h2) is None
    torch.cuda.synchronize()
    assert torch.equal(h1, h2)
    few = rows(30, 4)
    direct = few.clone()
    layer.KDABlock(a, w).forward(direct)
    layer.KDABlock(b, w).forward(few)
    assert relerr(host64(direct), host64(few)) < TOL_BF16


def norm64(x, w, eps):
    return x / np.sqrt((x * x).mean(1, keepdims=True) + eps) * host64(w)


@pytest.mark.parametrize("kind", ["bf16", "w4", "fp8"])
@pytest.mark.parametrize("call", ["forward", "decode", "tree"])
def test_block_with_a_norm_after_it(kind, call):
    """Two blocks and the last norm: the stream, the second block's input and the result
    follow the formula from the blocks' outputs (float32 errors of at most 200 roundings
    of each term, and the stored bfloat16's half step)."""
    announce("sandwich block %s %s" % (kind, call))
    g = torch.Generator().manual_seed(5)
    vec = lambda: (torch.rand(WIDTH, generator=g) + 0.5).cuda()
    blocks = []
    for i in range(2):
        if kind == "fp8":
            m = layer.KDAMixerFP8.from_host(synth.workload_layer_fp8(T=4, hidden=WIDTH, H=H, seed=30 + i))
        else:
            m = mixers(40 + 2 * i)[kind == "bf16"]
        post = layer.BranchNorm(vec(), gate=vec() if i else vec().to(BF), gate_activation=("sigmoid", "none")[i],
                                residual_scale=0.9, branch_scale=0.5 + i, eps=1e-5)
        blocks.append(layer.KDABlock(m, vec(), post=post))
    last = vec()
    hidden = rows(12, 6)
    h, delta, xs = host64(hidden), None, []
    par = torch.tensor([[-1, 0, 1, 1]] * 3, dtype=I32, device="cuda")
    for block in blocks:
        if call == "forward":
            delta = block.forward(hidden, delta)
        elif call == "decode":
            delta = block.decode(hidden, *states(12), delta)
        else:
            delta, tree = block.decode_tree(hidden, par, *states(3), delta)
        assert isinstance(delta, layer.Branch)
        xs.append(host64(delta.x))
    y = torch.empty((12, WIDTH), device="cuda")
    blocks[-1].finish(hidden, delta, last, y)
    torch.cuda.synchronize()
    scale = np.abs(h)
    for i, (x, block) in enumerate(zip(xs, blocks)):
        form = block.post.form
        gate = host64(form["gate"])
        gate = 1 / (1 + np.exp(-gate)) if form["gate_activation"] == "sigmoid" else gate
        branch = form["branch_scale"] * gate * norm64(x, block.post.weight, 1e-5)
        h = form["residual_scale"] * h + branch
        scale = scale + np.abs(branch)
        if i == 0 and kind != "fp8":
            ny = host64(blocks[1].mixer._bufs["ny"])
            ref = norm64(h, blocks[1].norm_weight, 1e-6)
            assert (np.abs(ny - ref) <= 2.0 ** -8 * np.abs(ref) + 300 * U * np.abs(ref).max()).all()
    assert (np.abs(host64(hidden) - h) <= 200 * U * scale).all()
    ref = norm64(h, last, 1e-6)
    assert (np.abs(host64(y) - ref) <= 500 * U * np.abs(ref).max()).all()


# ---------------------------------------------------------------- beam search
V = 60


def stack(kind, seed, n=2):
    blocks = []
    for i in range(n):
        g = torch.Generator().manual_seed(seed + i)
        vec = lambda: (torch.rand(WIDTH, generator=g) + 0.5).cuda()
        m = mixers(seed + 2 * i)[kind == "bf16"]
        blocks.append(layer.KDABlock(m, vec(), post=layer.BranchNorm(vec(), branch_scale=0.7) if kind == "w4" else None))
    g = torch.Generator().manual_seed(seed + 99)
    embed = (torch.randn((V, WIDTH), generator=g) * 2).cuda()
    last = (torch.rand(WIDTH, generator=g) + 0.5).cuda()
    head = w4(V, WIDTH, seed + 50)[kind == "bf16"]
    return blocks, embed, last, head


def search(kind, B, W, seed, eos=V - 1):
    blocks, embed, last, head = stack(kind, seed)
    sts = [states(B * W) for _ in blocks]
    return layer.BeamSearch(blocks, last, head, B, W, eos, [s for s, _ in sts], [c for _, c in sts]), embed


def sequence_run(s, embed, tokens, n):
    """The blocks' decode of a token sequence, in every of n rows (as many as the search has:
    the same forms of the products): log probabilities of every position in float64, the states."""
    sts, logp = [states(n) for _ in s.blocks], []
    y, logits = torch.empty((n, WIDTH), dtype=BF, device="cuda"), torch.empty((n, V), device="cuda")
    for token in tokens:
        hidden, delta = embed[token].repeat(n, 1), None
        for block, (st, cv) in zip(s.blocks, sts):
            delta = block.decode(hidden, st, cv, delta)
        s.blocks[-1].finish(hidden, delta, s.norm_weight, y)
        if isinstance(s.head, torch.Tensor):
            K.kda_gemm_epilogue(y, s.head, logits)
        else:
            K.kda_gemm_w4(y, s.head, logits)
        row = host64(logits)[0]
        logp.append(row - row.max() - np.log(np.exp(row - row.max()).sum()))
    return logp, sts


@pytest.mark.parametrize("kind", ["bf16", "w4"])
@pytest.mark.parametrize("B,W", [(1, 1), (2, 3), (3, 4), (5, 7)])
def test_beams_states_and_scores_are_those_of_their_sequences(kind, B, W):
    """After some steps every beam's states are bit for bit those of a decode of its tokens
    alone, and its score is the sum of their log probabilities in it. u = 2^-24: a step's
    logarithm is off by (V / 64 + 330) u (see the selection's own tests), and the sum is
    rounded once a step."""
    announce("beam search %s B=%d W=%d" % (kind, B, W))
    s, embed = search(kind, B, W, 60 + B, eos=-1)
    first = [7 + 3 * b for b in range(B)]
    paths = [[[first[b]] for _ in range(W)] for b in range(B)]
    tokens = torch.tensor(first, device="cuda").repeat_interleave(W)
    for step in range(6):
        s.step(embed[tokens].clone())
        torch.cuda.synchronize()
        par, tok = s.parents.tolist(), s.tokens.tolist()
        paths = [[paths[b][par[b][w]] + [tok[b][w]] for w in range(W)] for b in range(B)]
        tokens = s.tokens.view(-1).long()
    for b in range(B):
        assert all(s.scores[b, w] >= s.scores[b, w + 1] for w in range(W - 1))
        assert len({tuple(p) for p in paths[b]}) == W
        for w in range(W):
            path, row = paths[b][w], b * W + w
            logp, sts = sequence_run(s, embed, path[:-1], B * W)
            total = sum(logp[i][path[i + 1]] for i in range(len(path) - 1))
            assert abs(float(s.scores[b, w]) - total) <= 6 * ((V / 64 + 330) * U + U * abs(total))
            for (st, cv), mine, conv in zip(sts, s.states, s.conv_states):
                assert torch.equal(mine[row], st[row]) and torch.equal(conv[:, row], cv[:, row])


def test_captured_steps_equal_eager_ones():
    """A step captured in a graph and replayed, with eager calls of other sizes in between."""
    B, W = 2, 4
    a, embed = search("w4", B, W, 80)
    b, _ = search("w4", B, W, 80)
    other, _ = search("bf16", 5, 6, 90)
    x = torch.empty((B * W, WIDTH), device="cuda")
    x.copy_(embed[:B * W])
    a.step(x.clone())  # every kernel is loaded
    a.start()
    for st, cv in zip(a.states, a.conv_states):
        st.zero_(), cv.zero_()
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        a.step(x)
    torch.cuda.synchronize()
    tokens = torch.arange(B * W, device="cuda")
    for step in range(5):
        x.copy_(embed[tokens])
        graph.replay()
        other.step(rows(30, step))
        b.step(embed[tokens].clone())
        torch.cuda.synchronize()
        for name in ("scores", "parents", "tokens", "finished"):
            assert torch.equal(getattr(a, name), getattr(b, name)), (step, name)
        for u, v in zip(a.states + a.conv_states, b.states + b.conv_states):
            assert torch.equal(u, v)
        tokens = b.tokens.view(-1).long()


def test_ended_beams_stay():
    """Once a beam has taken eos its score stays and eos follows eos."""
    B, W = 2, 3
    s, embed = search("bf16", B, W, 95)
    tokens = torch.tensor([3, 3, 3, 4, 4, 4], device="cuda")
    s.step(embed[tokens].clone())
    s.finished[:, 0] = True  # the best beam of each ends here
    best = s.scores[:, 0].clone()
    for step in range(4):
        s.step(embed[s.tokens.view(-1).long()].clone())
        torch.cuda.synchronize()
        assert torch.equal(s.scores[:, 0], best) and bool(s.finished[:, 0].all())
        assert (s.tokens[:, 0] == V - 1).all()
        assert ((s.tokens == V - 1) <= s.finished).all()


@pytest.mark.parametrize("kind", ["bf16", "w4"])
@pytest.mark.parametrize("vocabulary", [1, 61, 62, 63, 1027])
def test_any_vocabulary(kind, vocabulary, monkeypatch):
    """Vocabularies of no whole number of 4 tokens: the logits are y head^T (256 exact products, their
    sum off by at most 2 u a term; from 4 bits 2 u (64 + 4 + 16) sum |s| |y| (32 + c + 8) with s <= 2^-8, c <=
    15), and the beams those of a selection on dense logits."""
    announce("beam search %s V=%d" % (kind, vocabulary))
    monkeypatch.setitem(globals(), "V", vocabulary)
    B, W = 2, 3
    s, embed = search(kind, B, W, 110, eos=0)
    head = s.head if kind == "bf16" else K.kda_w4_expand(s.head, torch.empty((vocabulary, WIDTH), dtype=BF, device="cuda"))
    tokens = torch.zeros(B * W, dtype=torch.int64, device="cuda")
    for step in range(3):
        before, ended = s.scores.clone(), s.finished.clone()
        s.step(embed[tokens].clone())
        torch.cuda.synchronize()
        y, w = s.y.double(), head.double().t().contiguous()
        size = y.abs() @ w.abs() if kind == "bf16" else y.abs().sum(1, keepdim=True) * (55 / 256)
        tol = 2 * U * (WIDTH + 8 if kind == "bf16" else 84) * size
        assert ((s.logits.double() - y @ w).abs() <= tol).all()
        out = [torch.empty_like(t) for t in (s.scores, s.parents, s.tokens, s.finished)]
        K.kda_beam_select(s.logits.contiguous(), before, *out[:3], finished=ended, next_finished=out[3], eos=0)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, (s.scores, s.parents, s.tokens, s.finished)))
        tokens = s.tokens.view(-1).long()


def test_mixers_share_the_expansion_of_their_weights():
    """Prefills of several 4-bit mixers, in turn and on two streams, hold no weights in bfloat16
    but one buffer a stream, as large as the largest weight, and equal the bfloat16 mixers'."""
    pairs = [mixers(120), mixers(130)]
    w, x = torch.ones(WIDTH, device="cuda"), [rows(150, 121), rows(170, 131)]
    for a, _ in pairs:
        a.EXPAND = 64

    def run(m, h):
        h = h.clone()
        assert layer.KDABlock(m, w).forward(h) is None
        return h

    want = [run(b, h) for (_, b), h in zip(pairs, x)]
    main, streams = torch.cuda.current_stream(), [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        st.wait_stream(main)
    y = torch.empty((150, WIDTH), device="cuda")
    with torch.cuda.stream(streams[0]):  # the smaller weight first: the buffer grows under work in flight
        pairs[0][0]._product(x[0].to(BF), pairs[0][0].Wo, y)
    got = []
    for _ in range(3):
        for i, (a, _) in enumerate(pairs):
            got.append((i, run(a, x[i])))
            for st in streams:
                with torch.cuda.stream(st):
                    got.append((i, run(a, x[i])))
    torch.cuda.synchronize()
    assert all(torch.equal(h, want[i]) for i, h in got)
    for a, _ in pairs:
        held = [(b.shape, b.dtype) for b in a._bufs.values()]
        assert (a.W_in.shape, BF) not in held and (a.Wo.shape, BF) not in held
    device = torch.cuda.current_device()
    for st in [main] + streams:
        assert layer._expanded[device, st.cuda_stream].numel() >= pairs[0][0].W_in.N * WIDTH


@pytest.mark.parametrize("B,W", [(1, 2), (3, 4)])
def test_search_over_a_stack_of_all_mixers(B, W):
    """W8A8, 4-bit with a norm after it, bfloat16, W8A8 with a norm after it: every way in which a block
    hands its output to the next. States and scores as in the tests above."""
    announce("beam search over all mixers B=%d W=%d" % (B, W))
    g = torch.Generator().manual_seed(140)
    vec = lambda: (torch.rand(WIDTH, generator=g) + 0.5).cuda()
    fp8 = lambda seed: layer.KDAMixerFP8.from_host(synth.workload_layer_fp8(T=4, hidden=WIDTH, H=H, seed=seed))
    post = lambda: layer.BranchNorm(vec(), gate=vec(), gate_activation="sigmoid", branch_scale=0.7)
    blocks = [layer.KDABlock(fp8(141), vec()), layer.KDABlock(mixers(142)[0], vec(), post=post()),
              layer.KDABlock(mixers(143)[1], vec()), layer.KDABlock(fp8(144), vec(), post=post())]
    embed, last, head = (torch.randn((V, WIDTH), generator=g) * 2).cuda(), vec(), w4(V, WIDTH, 145)[1]
    sts = [states(B * W) for _ in blocks]
    s = layer.BeamSearch(blocks, last, head, B, W, -1, [a for a, _ in sts], [c for _, c in sts])
    first = [5 + b for b in range(B)]
    paths = [[[first[b]] for _ in range(W)] for b in range(B)]
    tokens = torch.tensor(first, device="cuda").repeat_interleave(W)
    for step in range(4):
        s.step(embed[tokens].clone())
        torch.cuda.synchronize()
        par, tok = s.parents.tolist(), s.tokens.tolist()
        paths = [[paths[b][par[b][w]] + [tok[b][w]] for w in range(W)] for b in range(B)]
        tokens = s.tokens.view(-1).long()
    for b in range(B):
        for w in range(W):
            path, row = paths[b][w], b * W + w
            logp, own = sequence_run(s, embed, path[:-1], B * W)
            total = sum(logp[i][path[i + 1]] for i in range(len(path) - 1))
            assert abs(float(s.scores[b, w]) - total) <= 4 * ((V / 64 + 330) * U + U * abs(total))
            for (st, cv), mine, conv in zip(own, s.states, s.conv_states):
                assert torch.equal(mine[row], st[row]) and torch.equal(conv[:, row], cv[:, row])
