"""Beam selection and the reordering of states on the GPU against the definition,
serially in 64 bits on the CPU.

Whole numbers must be equal. Scores, u = 2^-24: a lane adds at most V / 64 + 16
exponentials (u each, relative), whose arguments x - max are rounded twice, 3 u |x
- max| each (|x - max| <= 100 where the term matters), the hardware exponential
another 2 u, and the stored score one rounding: (V / 64 + 330) u + u |score|."""
import math

import pytest
import torch

from gated_delta_rule_02_amd import kda as K
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F, I32 = torch.bfloat16, torch.float32, torch.int32
INF = float("inf")


def definition(logits, scores, finished, eos):
    """Lists per sequence of the W best (score, beam, token, finished)."""
    B, W = scores.shape
    x, V = logits.double().cpu(), logits.shape[1]
    out = []
    for b in range(B):
        rows = []
        for w in range(W):
            row, s = x[b * W + w], float(scores[b, w])
            live = math.isfinite(s) and not bool(torch.isnan(row).any()) and math.isfinite(float(row.max()))
            done = finished is not None and bool(finished[b, w])
            c = torch.full((V,), -INF, dtype=torch.float64)
            if done and math.isfinite(s):
                c[eos] = s
            elif live and not done:
                c = s + (row - row.max() - torch.log(torch.exp(row - row.max()).sum()))
            rows.append(c)
        c, order = torch.sort(torch.cat(rows), descending=True, stable=True)
        out.append([(float(c[i]), int(order[i]) // V, int(order[i]) % V) for i in range(W)])
    return out


def select(logits, scores, finished=None, eos=-1, with_flags=None, **kw):
    B, W = scores.shape
    ns = torch.full((B, W), float("nan"), device="cuda")
    p, t = (torch.full((B, W), -7, dtype=I32, device="cuda") for _ in range(2))
    nf = torch.empty((B, W), dtype=torch.bool, device="cuda") if finished is not None or with_flags else None
    K.kda_beam_select(logits, scores, ns, p, t, finished=finished, next_finished=nf, eos=eos, **kw)
    torch.cuda.synchronize()
    return ns, p, t, nf


def check(logits, scores, finished=None, eos=-1):
    ns, p, t, nf = select(logits, scores, finished, eos)
    ref = definition(logits, scores, finished, eos)
    V = logits.shape[1]
    for b, best in enumerate(ref):
        for i, (s, w, v) in enumerate(best):
            assert (int(p[b, i]), int(t[b, i])) == (w, v), (b, i, best, p[b].tolist(), t[b].tolist())
            got = float(ns[b, i])
            if math.isfinite(s):
                assert abs(got - s) <= (V / 64 + 330) * U + U * abs(s), (b, i, got, s)
            else:
                assert got == s
            if nf is not None:
                assert bool(nf[b, i]) == (bool(finished[b, w]) or v == eos)


def inputs(B, W, V, dtype, seed, std=2.5, scores=None):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((B * W, V), generator=g) * std).to(dtype).cuda()
    s = -torch.rand((B, W), generator=g) * 6 if scores is None else scores
    return x, s.cuda()


@pytest.mark.parametrize("B,W,V,dtype", [
    (1, 1, 1, F), (2, 3, 1, BF), (1, 4, 2, F), (3, 5, 7, BF), (2, 32, 5, F), (1, 8, 63, F), (2, 4, 1023, BF), (1, 4, 1024, F),
    (3, 2, 1025, F), (1, 32, 2049, BF), (2, 7, 5001, F), (1, 4, 32000, F), (5, 3, 20001, BF), (1, 16, 65537, F), (70, 4, 3001, BF),
    (1, 1, 200003, F), (300, 5, 1100, F)])
def test_select(B, W, V, dtype):
    announce("beam_select %s" % ((B, W, V, dtype),))
    check(*inputs(B, W, V, dtype, B + W + V))


@pytest.mark.parametrize("dtype", [F, BF])
def test_ties_go_to_the_lower_beam_then_the_lower_token(dtype):
    # coarse logits: many equal ones in a row; equal rows and scores: equal across beams
    g = torch.Generator().manual_seed(3)
    row = torch.randint(-3, 4, (2, 5003), generator=g).float().to(dtype)
    x = row[[0, 0, 0, 1, 1, 0, 1, 1]].cuda()
    check(x, torch.tensor([[-1.0, -1.0, -1.0, -1.0], [-2.0, -2.0, -2.5, -2.0]], device="cuda"))
    # one value throughout, and signed zeros, which are one value
    check(torch.zeros((6, 2050), dtype=dtype, device="cuda"), torch.zeros((2, 3), device="cuda"))
    z = torch.zeros((3, 4000), dtype=dtype)
    z[:, ::2] = -0.0
    check(z.cuda(), torch.zeros((1, 3), device="cuda"))


@pytest.mark.parametrize("order", ["up", "down"])
@pytest.mark.parametrize("W", [1, 5, 32])
def test_sorted_rows(order, W):
    """Ascending rows improve the list at every element, descending ones never after the first."""
    x = torch.linspace(-9, 9, 9001)
    x = (x if order == "up" else x.flip(0)).repeat(2 * W, 1) + torch.arange(2 * W)[:, None] * 0.0625
    check(x.cuda(), torch.linspace(-1, 0, 2 * W).view(2, W).cuda())


@pytest.mark.parametrize("W", [8, 32])
def test_all_of_the_best_in_one_lane_of_a_step(W):
    """Every token of the answer sits where one lane reads, above lanes of lower maxima."""
    x = torch.randn((W, 4096), generator=torch.Generator().manual_seed(1))
    for i in range(16):  # lane 5 of the first step reads 4 at a time
        x[:, i // 4 * 256 + 20 + i % 4] = 20 + i * 0.25
    check(x.cuda(), torch.zeros((1, W)).cuda())


@pytest.mark.parametrize("dtype", [F, BF])
def test_masked_logits(dtype):
    low = torch.finfo(dtype).min
    x, s = inputs(4, 3, 2500, dtype, 11)
    x[:, 100:2400] = -INF           # most tokens banned
    x[3] = -INF                     # a row with none left: dead
    x[4, 2:] = -INF                 # fewer tokens than beams
    x[5] = low                      # the type's lowest value throughout: equal offers
    x[6, :2499] = low               # masked by it, one token left
    x[7, 50] = INF                  # dead
    x[8, 2499] = float("nan")       # dead
    check(x, s)
    x[:] = -INF
    check(x, s)                     # nothing anywhere


def test_dead_beams_and_first_step():
    x, _ = inputs(3, 4, 3001, F, 12)
    s = torch.tensor([[0.0, -INF, -INF, -INF], [-INF] * 4, [float("nan"), -1.0, INF, -2.0]], device="cuda")
    check(x, s)


@pytest.mark.parametrize("eos", [0, 1, 2, 1700])
def test_finished_beams(eos):
    x, s = inputs(4, 4, 1701, F, 13)
    f = torch.tensor([[1, 0, 0, 0], [0, 1, 1, 0], [1, 1, 1, 1], [0, 0, 0, 0]], dtype=torch.bool, device="cuda")
    s[2, 1] = -INF
    x[0] = float("nan")  # an ended beam's logits are not looked at
    x[14, eos] = 50.0    # a beam that ends now
    check(x, s, f, eos)
    # without a list of the ended, the flags of those that end now
    x, s = inputs(2, 3, 1701, F, 14)
    x[1, eos] = 40.0
    ns, p, t, nf = select(x, s, None, eos, with_flags=True)
    assert torch.equal(nf, t == eos) and bool(nf.any())


def test_strided_and_unaligned_rows():
    x, s = inputs(3, 4, 3003, BF, 15)
    wide = torch.full((12, 3011), 9.0, dtype=BF, device="cuda")
    for off in (0, 1, 5):
        wide[:] = 99.0
        wide[:, off:off + 3003] = x
        a, b = select(wide[:, off:off + 3003], s), select(x, s)
        for u, v in zip(a[:3], b[:3]):
            assert torch.equal(u, v)


def test_in_place_and_captured():
    """scores and finished updated in place; a captured step replayed over new logits,
    with other calls in between that need larger workspaces."""
    B, W, V, eos = 3, 4, 2100, 9
    x, s0 = inputs(B, W, V, F, 16)
    f0 = torch.zeros((B, W), dtype=torch.bool, device="cuda")
    p, t = (torch.empty((B, W), dtype=I32, device="cuda") for _ in range(2))
    s, f, buf = s0.clone(), f0.clone(), x.clone()
    K.kda_beam_select(buf, s, s, p, t, finished=f, next_finished=f, eos=eos)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        K.kda_beam_select(buf, s, s, p, t, finished=f, next_finished=f, eos=eos)
    torch.cuda.synchronize()
    s.copy_(s0), f.copy_(f0)
    want_s, want_f = s0, f0
    for step in range(4):
        buf.copy_(inputs(B, W, V, F, 20 + step)[0])
        graph.replay()
        big, bs = inputs(40, 8, 4000, F, 30 + step)
        select(big, bs)
        ns, wp, wt, nf = select(buf, want_s, want_f, eos)
        assert torch.equal(s, ns) and torch.equal(f, nf) and torch.equal(p, wp) and torch.equal(t, wt)
        want_s, want_f = ns, nf


def test_two_streams_do_not_share_a_workspace():
    a, b = inputs(30, 8, 9000, F, 40), inputs(30, 8, 9000, F, 41)
    want = [select(*a), select(*b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for st, (x, s) in zip(streams, (a, b)):
            ns, p, t = torch.empty_like(s), *(torch.empty(s.shape, dtype=I32, device="cuda") for _ in range(2))
            K.kda_beam_select(x, s, ns, p, t, stream=st)
            got.append((ns, p, t))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for u, v in zip(g, want[i % 2][:3]):
            assert torch.equal(u, v)
    # a workspace of the caller's
    ws = torch.empty(K.kda_beam_select_workspace_bytes(30, 8, 9000), dtype=torch.uint8, device="cuda")
    for u, v in zip(select(*a, workspace=ws)[:3], want[0][:3]):
        assert torch.equal(u, v)
    with pytest.raises(K.KDAError):
        select(*a, workspace=ws[:-1])


# ---------------------------------------------------------------- states
@pytest.mark.parametrize("B,W,state,conv,dtype", [
    (1, 1, (2, 128, 128), (3, 512), F), (2, 2, (1, 128, 128), None, BF), (3, 4, (3, 128, 128), (3, 384), F),
    (2, 5, (2, 128, 128), (1, 256), BF), (4, 8, (1, 128, 128), (7, 128), F), (1, 9, (34,), (2, 8), torch.int64),
    (2, 16, (1, 128, 128), (3, 128), BF), (3, 17, (52,), (1, 40), F), (2, 32, (1, 128, 128), (3, 128), F),
    (500, 3, (12,), (3, 8), F)])
def test_reorder(B, W, state, conv, dtype):
    announce("beam_reorder %s" % ((B, W, state, conv, dtype),))
    g = torch.Generator().manual_seed(B + W)
    draw = lambda *shape: torch.randint(-1000, 1000, shape, generator=g).to(dtype).cuda()
    guard = draw(B * W + 2, *state)     # rows behind the last sequence stay
    st = guard[:B * W]
    cv = None if conv is None else torch.randn((3, B * W, *conv), generator=g).to(BF).cuda()
    for kind in ("random", "same", "first", "reverse", "bad"):
        p = torch.randint(0, W, (B, W), generator=g)
        if kind == "same":
            p = torch.arange(W).expand(B, W).clone()
        elif kind == "first":
            p.zero_()
        elif kind == "reverse":
            p = torch.arange(W - 1, -1, -1).expand(B, W).clone()
        elif kind == "bad":
            p[:, W // 2] = W
            p[0, 0] = -1
            p[B - 1, W - 1] = 2 ** 31 - 1
        before, cbefore = guard.clone(), None if cv is None else cv.clone()
        K.kda_beam_reorder(p.int().cuda(), st, cv)
        torch.cuda.synchronize()
        inside = (p >= 0) & (p < W)
        rows = (torch.arange(B)[:, None] * W + torch.where(inside, p, torch.arange(W).expand(B, W))).view(-1).cuda()
        assert torch.equal(guard[:B * W], before[:B * W][rows]) and torch.equal(guard[B * W:], before[B * W:]), kind
        if cv is not None:
            assert torch.equal(cv, cbefore[:, rows]), kind


def test_reorder_of_nothing():
    p = torch.zeros((0, 4), dtype=I32, device="cuda")
    K.kda_beam_reorder(p, torch.empty((0, 8), device="cuda"))
    K.kda_beam_reorder(torch.zeros((2, 2), dtype=I32, device="cuda"), torch.empty((4, 0), device="cuda"),
                       torch.empty((0, 4, 8), device="cuda"))


# ---------------------------------------------------------------- the logarithm
# A score that cancels its offer shows the logarithm's error whole: next_scores is near 0, where
# float32 is fine. Per term, u = 2^-24: x - m is rounded (u |x - m| of the value), the exponent (u of
# it, u |x - m| again), the hardware exponential 2 u; the largest value so far changes at most once a step
# and once between the lanes (each factor as a term: 2 u, and its distances add up to the term's own); 16
# terms are summed in 5 roundings, everything later in 64 bits.
def log_error(x, logs):
    """Error of the kernel's logarithm of every row's sum of exponentials of x - max, given it in 64 bits."""
    s = logs.float()[:, None].contiguous()
    ns, p, t, _ = select(x, s)
    return ns[:, 0].double() - (s[:, 0].double() - logs)


@pytest.mark.parametrize("rows,V,std,dtype", [(300, 8, 1.0, F), (256, 1000, 1.0, BF), (256, 1000, 5.0, F), (128, 32000, 1.0, F),
                                              (128, 32000, 2.5, BF), (5, 200003, 2.5, F)])
def test_logarithm(rows, V, std, dtype):
    announce("beam_select logarithm %s" % ((rows, V, std, dtype),))
    x = inputs(rows, 1, V, dtype, rows + V, std)[0]
    d = x.double().amax(1, keepdim=True) - x.double()
    total = torch.exp(-d).sum(1)
    mean = (torch.exp(-d) * d).sum(1) / total
    steps = -(-V // 1024)
    error = log_error(x, torch.log(total))
    print("  mean %.1e, worst %.1e" % (float(error.mean()), float(error.abs().max())), flush=True)
    assert (error.abs() <= (2 * mean + 7 + 2 * (steps + 1)) * U + 1e-13).all()


def test_exponents_are_rounded_once():
    """Rows of one distance d, at which float32's log2(e) gives a neighbour of the correctly rounded
    exponent: that moves the logarithm by more than 8 u, and all other errors stay below 5 u."""
    V, tops, log2e = 131072, 64, 1.4426950408889634
    rounded = lambda v: float(torch.tensor(v, dtype=torch.float64).float())
    logarithm = lambda exponent: math.log(tops + (V - tops) * 2.0 ** -exponent)
    ds = [i / 32 for i in range(178, 256)]
    ds = [d for d in ds if abs(logarithm(rounded(d * rounded(log2e))) - logarithm(rounded(d * log2e))) > 8 * U]
    assert len(ds) >= 5
    want = [logarithm(rounded(d * log2e)) for d in ds]
    rows = 4096  # one part a row, whose first step has a largest value for every lane
    x = (-torch.tensor(ds)).repeat(rows // len(ds) + 1)[:rows, None].to(BF).cuda().repeat(1, V)
    x[:, :8 * tops:8] = 0
    error = log_error(x, torch.tensor(want, dtype=torch.float64).repeat(rows // len(ds) + 1)[:rows].cuda())
    print("  worst %.1f u" % (float(error.abs().max()) / U), flush=True)
    assert (error.abs() <= 5 * U).all()


def test_rows_beyond_32_bits():
    """More than 2^31 logits: the last sequences' rows lie past what 32-bit offsets reach."""
    B, W, V = 271, 8, 1000003
    announce("beam_select %d x %d x %d" % (B, W, V))
    if torch.cuda.mem_get_info()[0] < (12 << 30):
        pytest.skip("takes 5 GB of device memory")
    few, s = inputs(3, W, V, BF, 50)
    x = torch.zeros((B * W, V), dtype=BF, device="cuda")
    at = (0, 134, B - 1)
    for i, b in enumerate(at):
        x[b * W:(b + 1) * W] = few[i * W:(i + 1) * W]
    scores = torch.zeros((B, W), device="cuda")
    scores[list(at)] = s
    got, want = select(x, scores), select(few, s)  # in parts of other lengths: scores of up to 32 may round otherwise
    for g, w in zip(got[:3], want[:3]):
        assert torch.equal(g[list(at)], w) if g.dtype == I32 else ((g[list(at)] - w).abs() <= 4 * U * 32).all()
    check(few, s)
