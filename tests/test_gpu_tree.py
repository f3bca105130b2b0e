"""Trees of drafted tokens on the GPU -- verification, commit, and the prologue
convolution along the paths -- against the recurrence followed node by node in
64 bits, a full state per node.

Tolerances, u = 2^-24. An alpha is exp of at most |lower_bound| in float32: its
argument scaled once and the hardware exponential, (8 + |lower_bound|) u; a
path's product of d of them, (10 + |lower_bound|) d u with its roundings. A read of
the state adds 128 terms, a sum over a path d of them: every term of u_i and o_i is
within c u of itself, c = 128 + 2d + 8 + (10 + |lower_bound|) d, and an error of
a write enters the writes below it with the same coefficients that the writes have.
So |error| <= c (d + 1) u M with M the formula taken on magnitudes. The state's
own error is c' u M', c' = (10 + |lower_bound|) d + d + 4. Stored bfloat16 adds 2^-8 of the value."""
import numpy as np
import pytest
import torch

from gated_delta_rule_02_amd import kda as K
from tests.gpu_util import TOL_F32, announce, host64, relerr

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F = torch.bfloat16, torch.float32


def tree(kind, N, rng):
    """parents of one tree"""
    if kind == "chain":
        return [i - 1 for i in range(N)]
    if kind == "star":
        return [-1] * N
    if kind == "none":
        return [-2] * N
    if kind == "binary":
        return [(i - 1) // 2 if i else -1 for i in range(N)]
    p = [int(rng.integers(max(-1, i - 4), i)) for i in range(N)]
    if kind == "holes":  # unused places and values that are no parent, in the middle and at the end
        for i in range(N):
            if rng.random() < 0.25:
                p[i] = int(rng.choice([-2, -5, i, i + 1, 64, 1 << 30, -(1 << 31)]))
    return p


def paths(parents):
    """Root path of every node (its own index last), [] where it is absent."""
    out = []
    for i, p in enumerate(parents):
        ok = -1 <= p < i and (p == -1 or out[p])
        out.append(([] if p == -1 else out[p]) + [i] if ok else [])
    return out


def inputs(B, N, H, xd, sd, seed, lb=-5.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    d = {}
    for n in ("q", "k"):
        x = r(B, N, H, 128)
        d[n] = (x / x.norm(dim=-1, keepdim=True)).to(xd).cuda()
    d["v"] = r(B, N, H, 128).to(xd).cuda()
    gl = -torch.nn.functional.softplus(r(B, N, H, 128) * 3)
    gl[:, :, :, :3] = -40.0  # below every floor used here
    d["g"] = gl.to(xd).cuda()
    d["beta"] = torch.sigmoid(r(B, N, H)).to(xd).cuda()
    d["state"] = (r(B, H, 128, 128) * 0.3).to(sd).cuda()
    return d


def reference(d, parents, lb=-5.0, scale=1.0):
    """o, u and states of every node, and their magnitudes, in 64 bits."""
    x = {n: host64(t) for n, t in d.items()}
    B, N, H, _ = x["q"].shape
    al = np.exp(np.maximum(x["g"], lb))
    o, u = np.zeros((B, N, H, 128)), np.zeros((B, N, H, 128))
    mo, mu, depth = np.zeros_like(o), np.zeros_like(o), np.zeros((B, N, 1, 1))
    states = {}
    for b in range(B):
        S, A = {-1: x["state"][b]}, {-1: np.abs(x["state"][b])}
        for i, p in enumerate(paths(parents[b])):
            if not p:
                continue
            up = parents[b][i]
            k, be = x["k"][b, i], x["beta"][b, i][:, None]
            Sp, Ap = al[b, i][:, :, None] * S[up], al[b, i][:, :, None] * A[up]
            u[b, i] = be * (x["v"][b, i] - np.einsum("hkv,hk->hv", Sp, k))
            mu[b, i] = be * (np.abs(x["v"][b, i]) + np.einsum("hkv,hk->hv", Ap, np.abs(k)))
            S[i] = Sp + k[:, :, None] * u[b, i][:, None, :]
            A[i] = Ap + np.abs(k)[:, :, None] * mu[b, i][:, None, :]
            o[b, i] = scale * np.einsum("hkv,hk->hv", S[i], x["q"][b, i])
            mo[b, i] = abs(scale) * np.einsum("hkv,hk->hv", A[i], np.abs(x["q"][b, i]))
            depth[b, i] = len(p)
        states[b] = (S, A)
    return o, u, mo, mu, depth, states


def verify(d, parents, od, lb=-5.0, scale=1.0, writes=True):
    B, N, H, _ = d["q"].shape
    par = torch.tensor(parents, dtype=torch.int64).to(torch.int32).cuda()
    o = torch.full((B, N, H, 128), float("nan"), dtype=od, device="cuda")
    w = torch.full((B, N, H, 128), float("nan"), device="cuda") if writes else None
    before = d["state"].clone()
    K.kda_decode_tree(d["q"], d["k"], d["v"], d["g"], d["beta"], par, d["state"], o, w, scale=scale, lower_bound=lb)
    torch.cuda.synchronize()
    assert torch.equal(before, d["state"])
    return o, w, par


def bound(depth, lb):
    lb = min(abs(lb), 45.0)  # -inf: the smallest g given is -40
    return (128 + 2 * depth + 8 + (10 + lb) * depth) * (depth + 1) * U


# (B, N, H, inputs, state, o, kind, lower bound, scale)
CASES = [
    (1, 1, 1, F, F, F, "chain", -5.0, 1.0), (2, 1, 3, BF, BF, BF, "star", -5.0, 1.0),
    (3, 7, 2, F, F, F, "random", -5.0, 0.5), (4, 8, 2, BF, F, F, "random", -5.0, 1.0),
    (2, 9, 3, BF, BF, F, "binary", -1.0, 1.0), (2, 16, 2, F, F, F, "chain", -5.0, 1.0),
    (6, 16, 1, BF, F, BF, "holes", -5.0, -2.0), (2, 17, 2, F, BF, F, "random", -5.0, 1.0),
    (5, 31, 1, BF, F, F, "holes", -5.0, 1.0), (2, 32, 2, F, F, F, "star", -5.0, 1.0),
    (2, 33, 1, BF, F, F, "binary", -5.0, 1.0), (1, 64, 2, F, F, F, "chain", -5.0, 1.0),
    (3, 64, 1, BF, BF, BF, "random", -5.0, 1.0), (2, 64, 1, F, F, F, "holes", 0.0, 1.0),
    (2, 12, 2, F, F, F, "random", float("-inf"), 1.0), (2, 5, 2, F, F, F, "none", -5.0, 1.0),
    (1, 6, 64, BF, F, F, "random", -5.0, 1.0), (130, 3, 3, BF, F, F, "random", -5.0, 1.0),
    (2, 24, 2, F, F, F, "holes", -5.0, 1.0), (2, 40, 1, BF, F, F, "random", -5.0, 1.0), (1, 48, 2, F, BF, F, "chain", -5.0, 1.0),
    (2, 49, 1, BF, BF, BF, "holes", -5.0, 1.0), (2, 57, 2, F, F, F, "binary", -5.0, 1.0),
]


@pytest.mark.parametrize("B,N,H,xd,sd,od,kind,lb,scale", CASES)
def test_decode_tree(B, N, H, xd, sd, od, kind, lb, scale):
    announce("decode_tree B=%d N=%d H=%d in=%s state=%s o=%s %s lb=%s" % (B, N, H, xd, sd, od, kind, lb))
    rng = np.random.default_rng(B * 100 + N)
    parents = [tree(kind, N, rng) for _ in range(B)]
    d = inputs(B, N, H, xd, sd, N + H)
    for b in range(B):  # what an absent node holds must not matter
        for i, p in enumerate(paths(parents[b])):
            if not p:
                for n in ("q", "k", "v", "g", "beta"):
                    d[n][b, i] = float("nan")
    o, w, _ = verify(d, parents, od, lb, scale)
    o2, _, _ = verify(d, parents, od, lb, scale, writes=False)
    assert torch.equal(o, o2)
    ro, ru, mo, mu, depth, _ = reference(d, parents, lb, scale)
    c = bound(depth, lb)
    half = 2.0 ** -8 if od == BF else 0.0
    eo = np.abs(host64(o) - ro) / np.maximum(c * mo + half * (np.abs(ro) + c * mo), 1e-300)
    eu = np.abs(host64(w) - ru) / np.maximum(c * mu, 1e-300)
    print("  o %.3f writes %.3f of the tolerance, max rel %.2e" % (eo.max(), eu.max(), relerr(host64(w), ru)), flush=True)
    assert eo.max() <= 1 and eu.max() <= 1
    if kind != "none" and od == F:
        assert relerr(host64(o), ro) < TOL_F32 and relerr(host64(w), ru) < TOL_F32


@pytest.mark.parametrize("B,N,H,xd,sd,kind,lb", [
    (1, 1, 1, F, F, "chain", -5.0), (4, 9, 2, BF, BF, "random", -5.0), (9, 16, 2, F, F, "holes", -5.0),
    (2, 33, 1, BF, F, "chain", -5.0), (2, 64, 2, F, BF, "chain", -5.0), (3, 40, 1, F, F, "binary", float("-inf")),
    (1, 64, 1, BF, F, "chain", -0.25), (67, 4, 3, BF, F, "random", -5.0),
])
def test_decode_tree_commit(B, N, H, xd, sd, kind, lb):
    """Every sequence accepts another node (each of them in turn over the calls);
    values outside the tree and absent nodes leave the state as it was."""
    announce("decode_tree_commit B=%d N=%d H=%d in=%s state=%s %s lb=%s" % (B, N, H, xd, sd, kind, lb))
    rng = np.random.default_rng(B + N)
    parents = [tree(kind, N, rng) for _ in range(B)]
    d = inputs(B, N, H, xd, sd, N)
    _, w, par = verify(d, parents, F, lb)
    ref = reference(d, parents, lb)
    for turn in range(3):
        acc = [int(x) for x in rng.integers(0, N, B)]
        if turn == 0:
            acc[0] = N - 1
        if turn == 1:
            acc[-1] = int(rng.choice([-1, N, 64, 1 << 30, -(1 << 31)]))
        state = d["state"].clone()
        K.kda_decode_tree_commit(d["k"], d["g"], w, par, torch.tensor(acc).to(torch.int32).cuda(), state, lower_bound=lb)
        torch.cuda.synchronize()
        got, was = host64(state), host64(d["state"])
        for b in range(B):
            p = paths(parents[b])[acc[b]] if 0 <= acc[b] < N else []
            if not p:
                np.testing.assert_array_equal(got[b], was[b])
                continue
            # the writes given are float32 results: their error is the verification's
            S, A = ref[5][b][0][acc[b]], ref[5][b][1][acc[b]]
            n = len(p)
            tol = (bound(n, lb) + ((10 + min(abs(lb), 45.0)) * n + n + 4) * U) * A
            if sd == BF:
                tol = tol + 2.0 ** -8 * (np.abs(S) + tol)
            assert (np.abs(got[b] - S) <= tol + 1e-300).all(), (b, float((np.abs(got[b] - S) / tol).max()))


def test_chain_equals_decode_multi():
    """A chain is what kda_decode_multi verifies: outputs, and the state of every
    prefix, to float32 rounding."""
    announce("decode_tree chain against decode_multi")
    B, N, H = 3, 6, 4
    d = inputs(B, N, H, BF, F, 8)
    parents = [tree("chain", N, None)] * B
    o, w, par = verify(d, parents, F)
    o2 = torch.empty_like(o)
    ts = torch.empty((B, N, H, 128, 128), device="cuda")
    K.kda_decode_multi(d["q"], d["k"], d["v"], d["g"], d["beta"], d["state"], o2, token_states=ts)
    assert relerr(host64(o), host64(o2)) < TOL_F32
    for i in range(N):
        s1, s2 = d["state"].clone(), d["state"].clone()
        K.kda_decode_tree_commit(d["k"], d["g"], w, par, torch.full((B,), i, dtype=torch.int32, device="cuda"), s1)
        K.kda_decode_commit(ts, torch.full((B,), i + 1, dtype=torch.int32, device="cuda"), s2)
        assert relerr(host64(s1), host64(s2)) < TOL_F32


@pytest.mark.parametrize("N", [7, 16, 30, 45, 64])
def test_decode_tree_branches_do_not_touch(N):
    """NaN and infinity in one node reach that node and what is below it, and
    nothing else, not even the last bits."""
    announce("decode_tree isolation N=%d" % N)
    d = inputs(2, N, 2, F, F, 3)
    parents = [tree("random", N, np.random.default_rng(1)), tree("binary", N, None)]
    o, w, _ = verify(d, parents, F)
    for n, bad in (("v", float("nan")), ("k", float("inf")), ("q", float("nan")), ("beta", float("nan"))):
        e = {a: t.clone() for a, t in d.items()}
        node = 2
        e[n][:, node] = bad
        o2, w2, _ = verify(e, parents, F)
        for b in range(2):
            for i, p in enumerate(paths(parents[b])):
                hit = i == node if n == "q" else node in p
                if not hit:
                    assert torch.equal(o[b, i], o2[b, i]) and torch.equal(w[b, i], w2[b, i]), (n, b, i)
                elif i == node:
                    assert not torch.isfinite(o2[b, i]).all()


def conv_reference(x, hist, parents, w, bias, silu, l2, eps=1e-6):
    """y and its tolerance (float32 arithmetic) for every node, in 64 bits."""
    B, N = len(parents), len(parents[0])
    C, W = w.shape
    y, tol = np.zeros((B * N, C)), np.zeros((B * N, C))
    for b in range(B):
        for i, p in enumerate(paths(parents[b])):
            if not p:
                continue
            win = np.concatenate([hist[b], x[b * N:(b + 1) * N][p]])[-W:]
            z = (win * w.T).sum(0) + (0 if bias is None else bias)
            t = (W + 2) * U * ((np.abs(win) * np.abs(w.T)).sum(0) + (0 if bias is None else np.abs(bias)))
            if silu:
                with np.errstate(over="ignore"):
                    t = 1.1 * t + 8 * U * (1 + np.abs(z)) * np.abs(z / (1 + np.exp(-z)))
                    z = z / (1 + np.exp(-z))
            if l2:
                zg, tg = z.reshape(-1, 128), t.reshape(-1, 128)
                r = 1 / np.sqrt((zg * zg).sum(1, keepdims=True) + eps)
                tg = tg * r + np.abs(zg * r) * (np.sqrt((tg * tg).sum(1, keepdims=True)) * r + 20 * U)
                z, t = (zg * r).reshape(-1), tg.reshape(-1)
            y[b * N + i], tol[b * N + i] = z, t
    return y, tol


# (B, N, C, W, type, kind, bias, silu, l2, padding of x rows)
CONV = [
    (1, 1, 128, 2, F, "chain", False, False, 0, 0), (3, 7, 384, 4, BF, "random", False, True, 128, 8),
    (2, 16, 2048, 4, BF, "holes", True, True, 128, 0), (2, 5, 2176, 3, F, "holes", True, True, 0, 16),
    (1, 64, 256, 8, F, "chain", True, True, 128, 0), (2, 33, 128, 8, BF, "random", False, True, 128, 24),
    (4, 6, 256, 5, BF, "star", True, False, 0, 0), (2, 9, 128, 6, F, "binary", False, True, 128, 8),
    (3, 4, 128, 7, BF, "none", True, True, 128, 0), (70, 3, 4224, 4, BF, "random", False, True, 128, 0),
]


@pytest.mark.parametrize("B,N,C,W,t,kind,bias,silu,l2,pad", CONV)
def test_conv_tree_and_commit(B, N, C, W, t, kind, bias, silu, l2, pad):
    """y against the windows along the paths; the history is not touched; the
    commit is a bit copy of the last W - 1 inputs."""
    announce("conv_tree B=%d N=%d C=%d W=%d %s %s" % (B, N, C, W, t, kind))
    rng = np.random.default_rng(N * C)
    g = torch.Generator().manual_seed(W)
    parents = [tree(kind, N, rng) for _ in range(B)]
    xf = torch.randn((B * N, C + pad), generator=g).to(t).cuda()
    for b in range(B):
        for i, p in enumerate(paths(parents[b])):
            if not p:
                xf[b * N + i] = float("nan")
    x = xf[:, :C]
    hist = torch.randn((B, W - 1, C), generator=g).to(t).cuda()
    w = (torch.randn((C, W), generator=g) * 0.5).to(t).cuda()
    bv = torch.randn(C, generator=g).to(t).cuda() if bias else None
    par = torch.tensor(parents, dtype=torch.int64).to(torch.int32).cuda()
    y = torch.full((B * N, C), float("nan"), dtype=t, device="cuda")
    before = hist.clone()
    K.kda_conv_tree(x, hist, par, w, y, bias=bv, apply_silu=silu, l2norm_group=l2)
    torch.cuda.synchronize()
    assert torch.equal(hist, before)
    ref, tol = conv_reference(host64(x), host64(hist), parents, host64(w), None if bv is None else host64(bv), silu, l2)
    if t == BF:
        tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
    assert (np.abs(host64(y) - ref) <= tol).all()
    for turn in range(3):
        acc = [int(v) for v in rng.integers(0, N, B)]
        if turn == 1:
            acc[0] = int(rng.choice([-1, N, 64, 1 << 30]))
        h2 = hist.clone()
        K.kda_conv_tree_commit(x, par, torch.tensor(acc).to(torch.int32).cuda(), h2)
        torch.cuda.synchronize()
        for b in range(B):
            p = paths(parents[b])[acc[b]] if 0 <= acc[b] < N else []
            want = torch.cat([hist[b], x[b * N:(b + 1) * N][p]])[-(W - 1):] if p else hist[b]
            assert torch.equal(h2[b].view(torch.uint8), want.contiguous().view(torch.uint8)), (b, acc[b])


def test_tree_step_captured():
    """Convolution, verification and both commits captured in one graph, replayed
    over changing inputs, trees and accepted nodes with eager work between:
    every replay equals the eager calls."""
    announce("tree step captured")
    B, N, H, W = 3, 11, 2, 4
    C = 128 * H
    wt = torch.randn(C, W).bfloat16().cuda()

    def fresh(seed):
        d = inputs(B, N, H, BF, F, seed)
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        d["parents"] = torch.tensor([tree("holes", N, rng) for _ in range(B)], dtype=torch.int64).to(torch.int32).cuda()
        d["accepted"] = torch.from_numpy(rng.integers(0, N, B)).to(torch.int32).cuda()
        d["x"] = torch.randn((B * N, C), generator=g).bfloat16().cuda()
        d["hist"] = torch.randn((B, W - 1, C), generator=g).bfloat16().cuda()
        return d

    def step(d, out):
        K.kda_conv_tree(d["x"], d["hist"], d["parents"], wt, out["y"])
        K.kda_decode_tree(d["q"], d["k"], d["v"], d["g"], d["beta"], d["parents"], d["state"], out["o"], out["w"])
        K.kda_decode_tree_commit(d["k"], d["g"], out["w"], d["parents"], d["accepted"], d["state"])
        K.kda_conv_tree_commit(d["x"], d["parents"], d["accepted"], d["hist"])

    def outs():
        return dict(y=torch.empty((B * N, C), dtype=BF, device="cuda"), o=torch.empty((B, N, H, 128), device="cuda"),
                    w=torch.empty((B, N, H, 128), device="cuda"))

    d, out = fresh(0), outs()
    step(d, out)
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        step(d, out)
    torch.cuda.current_stream().wait_stream(s)
    for i in range(1, 5):
        e, o2 = fresh(i), outs()
        for n in d:
            d[n].copy_(e[n])
        graph.replay()
        step(e, o2)
        torch.cuda.synchronize()
        for n in out:
            assert torch.equal(out[n], o2[n]), n
        for n in ("state", "hist"):
            assert torch.equal(d[n], e[n]), n


def test_tree_offsets_past_32_bits():
    """States over 4 GiB: the last sequence's rows."""
    announce("decode_tree over 4 GiB of states")
    B, N, H = 1100, 2, 64
    state = torch.zeros((B, H, 128, 128), device="cuda")
    d = inputs(1, N, H, F, F, 5)
    last = {n: torch.zeros((B,) + t.shape[1:], dtype=t.dtype, device="cuda") for n, t in d.items() if n != "state"}
    for n in last:
        last[n][-1] = d[n][0]
    state[-1] = d["state"][0]
    par = torch.tensor([[-1, 0]] * B, dtype=torch.int32, device="cuda")
    o, w = torch.empty((B, N, H, 128), device="cuda"), torch.empty((B, N, H, 128), device="cuda")
    K.kda_decode_tree(last["q"], last["k"], last["v"], last["g"], last["beta"], par, state, o, w)
    o1, w1, par1 = verify(d, [[-1, 0]], F)
    assert torch.equal(o[-1], o1[0]) and torch.equal(w[-1], w1[0])
    acc = torch.ones(B, dtype=torch.int32, device="cuda")
    K.kda_decode_tree_commit(last["k"], last["g"], w, par, acc, state)
    K.kda_decode_tree_commit(d["k"], d["g"], w1, par1, acc[:1], d["state"])
    torch.cuda.synchronize()
    assert torch.equal(state[-1], d["state"][0]) and not state[:-1].any()
