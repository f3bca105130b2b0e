"""Residual addition + RMSNorm (float32, bfloat16 and block-FP8 output) on the
GPU against the formula in 64 bits.

Tolerances, u = 2^-24 (half a float32 step, relative): h = x + r is one
rounding (u); the sum of squares adds n = K / threads-per-row terms per lane and
then at most 9 partial sums (each a rounding of a sum of positive terms, so
relative: n + 9, plus one for each square); its mean, the eps, the root and the
reciprocal add 4 more, half of what stands under the root counts; the two
products with h and w add 2. Together less than (n + 24) u relative to y,
element by element. A stored bfloat16 adds 2^-8 of the value."""
import numpy as np
import pytest
import torch

from gated_delta_rule_02_amd import kda as K
from oracle import reference as R
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6


def per_lane(k):
    return 8 * -(-k // (8 * (64 if k <= 1024 else 256)))


def half_step(dtype):
    return torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0.0


def make(M, k, xd, rd, seed, pad=0, residual=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, k + pad), generator=g).to(xd).cuda()[:, :k]
    r = (torch.randn((M, k + pad), generator=g) * 2).to(rd).cuda()[:, :k] if residual else None
    w = (torch.rand(k, generator=g) + 0.5).cuda()
    return x, r, w


def formula(x, r, w, eps=EPS):
    h = x.double().cpu() + (0 if r is None else r.double().cpu())
    return h, h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * w.double().cpu()


def near(got, ref, rel):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    worst = float(((got - ref).abs() / ref.abs().clamp(min=1e-300)).max())
    print("  worst %.2e of %.2e" % (worst, rel), flush=True)
    return bool(((got - ref).abs() <= rel * ref.abs()).all())


BF, F = torch.bfloat16, torch.float32
# (M, K, x, residual, y, padding of the rows, has residual)
CASES = [
    (1, 8, F, F, F, 0, True), (1, 4096, F, BF, BF, 0, True), (3, 1000, BF, BF, F, 8, True),
    (5, 1024, BF, F, BF, 16, False), (7, 1032, BF, BF, F, 0, True), (2, 4104, F, F, F, 8, True),
    (33, 5128, BF, BF, BF, 24, True), (4, 8192, BF, BF, F, 0, False), (3, 8200, BF, F, F, 8, True),
    (2, 40968, F, BF, F, 0, True), (4099, 136, BF, BF, BF, 0, True),
]


@pytest.mark.parametrize("M,k,xd,rd,yd,pad,res", CASES)
def test_add_rmsnorm(M, k, xd, rd, yd, pad, res):
    announce("add_rmsnorm M=%d K=%d %s %s %s pad=%d residual=%s" % (M, k, xd, rd, yd, pad, res))
    x, r, w = make(M, k, xd, rd, M + k, pad, res)
    y = torch.full((M, k + pad), float("nan"), dtype=yd, device="cuda")
    ro = torch.full((M, k + pad), float("nan"), dtype=rd, device="cuda") if res else None
    K.kda_add_rmsnorm(x, w, y[:, :k], residual=r, residual_out=None if ro is None else ro[:, :k], eps=EPS)
    torch.cuda.synchronize()
    h, ref = formula(x, r, w)
    assert near(y[:, :k], ref, (per_lane(k) + 24) * U + half_step(yd))
    assert torch.isnan(y[:, k:]).all()
    if res:
        # one float32 addition, then the storage type's rounding
        assert near(ro[:, :k], h, U + half_step(rd) * (1 + U))
        assert torch.isnan(ro[:, k:]).all()
        # in place, and without storing it: the same y
        r2, y2 = r.clone(), torch.empty_like(y)
        K.kda_add_rmsnorm(x, w, y2[:, :k], residual=r2, residual_out=r2, eps=EPS)
        y3 = torch.empty_like(y)
        K.kda_add_rmsnorm(x, w, y3[:, :k], residual=r, eps=EPS)
        assert torch.equal(r2, ro[:, :k]) and torch.equal(y2[:, :k], y[:, :k]) and torch.equal(y3[:, :k], y[:, :k])


@pytest.mark.parametrize("M,k,xd,rd,pad,res", [
    (1, 128, F, F, 0, True), (1, 4096, F, BF, 0, True), (5, 384, BF, BF, 16, True), (131, 1152, BF, F, 8, False),
    (6, 4224, BF, BF, 0, True), (2, 8320, F, BF, 8, True), (1025, 896, BF, BF, 0, True),
])
def test_add_rmsnorm_fp8(M, k, xd, rd, pad, res):
    """Codes and scales are those that kda_quantize_fp8 gives for the float32 y,
    bit for bit, and near the formula: the scale within y's tolerance and one
    division, the value within half an E4M3 step (2^-4 of it, 2^-10 among the
    subnormals)."""
    announce("add_rmsnorm_fp8 M=%d K=%d %s %s pad=%d residual=%s" % (M, k, xd, rd, pad, res))
    x, r, w = make(M, k, xd, rd, M + k, pad, res)
    x[0] *= 0  # a row without magnitude (but for its residual)
    codes = torch.full((M, k + pad), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((M, k // 128 + 3), float("nan"), device="cuda")
    ro = torch.empty_like(r) if res else None
    K.kda_add_rmsnorm_fp8(x, w, codes[:, :k], scales[:, :k // 128], residual=r, residual_out=ro, eps=EPS)
    y = torch.empty((M, k), device="cuda")
    ro2 = torch.empty_like(r) if res else None
    K.kda_add_rmsnorm(x, w, y, residual=r, residual_out=ro2, eps=EPS)
    c2, s2 = torch.empty((M, k), dtype=torch.uint8, device="cuda"), torch.empty((M, k // 128), device="cuda")
    K.kda_quantize_fp8(y, c2, s2)
    torch.cuda.synchronize()
    assert torch.equal(codes[:, :k], c2) and torch.equal(scales[:, :k // 128], s2)
    assert (codes[:, k:] == 0x55).all() and torch.isnan(scales[:, k // 128:]).all()
    if res:
        assert torch.equal(ro, ro2)
    _, ref = formula(x, r, w)
    top = ref.view(M, -1, 128).abs().amax(2)
    sref = torch.where(top > 0, top / 448, torch.ones_like(top))
    rel = (per_lane(k) + 25) * U
    assert near(scales[:, :k // 128], sref, rel)
    q = (ref.view(M, -1, 128) / sref[..., None]).view(M, k).numpy()
    dec = R.e4m3_decode(codes[:, :k].cpu().numpy())
    assert (np.abs(dec - q) <= (2.0 ** -4 + 3 * rel) * np.abs(q) + 2.0 ** -10).all()


def test_add_rmsnorm_zero_rows_and_values_outside():
    """A zero row gives zeros (eps > 0); a NaN or an infinity stays in its row and
    shows in the codes; a zero group's scale is 1; no row gets another's."""
    announce("add_rmsnorm zero, NaN and infinity")
    M, k = 6, 512
    x, r, w = make(M, k, F, F, 3)
    x[1] = 0
    r[1] = 0
    x[3, 5] = float("nan")
    x[4, 200] = float("inf")
    r[5, :128] = -x[5, :128]  # h is zero in one group
    y, codes = torch.empty_like(x), torch.empty((M, k), dtype=torch.uint8, device="cuda")
    scales = torch.empty((M, 4), device="cuda")
    K.kda_add_rmsnorm(x, w, y, residual=r)
    K.kda_add_rmsnorm_fp8(x, w, codes, scales, residual=r)
    torch.cuda.synchronize()
    assert (y[1] == 0).all() and ((codes[1] & 0x7f) == 0).all() and (scales[1] == 1).all()
    assert torch.isnan(y[3]).all() and ((codes[3] & 0x7f) == 0x7f).all() and (scales[3] == 1).all()
    assert torch.isnan(y[4, 200]) and (y[4, :200] == 0).all() and (codes[4, 200] & 0x7f) == 0x7f
    assert (scales[5, 0] == 1) and ((codes[5, :128] & 0x7f) == 0).all() and (scales[5, 1:] != 1).all()
    _, ref = formula(x, r, w)
    rows = [0, 2, 5]
    assert near(y[rows], ref[rows].where(ref[rows] != 0, torch.zeros(())), (per_lane(k) + 24) * U)


def test_add_rmsnorm_captured():
    """Captured in a HIP graph and replayed with other inputs and eager work
    between the replays: every replay equals the eager call."""
    announce("add_rmsnorm captured")
    M, k = 37, 2176
    x, r, w = make(M, k, BF, BF, 4)
    r0 = r.clone()
    codes, scales = torch.empty((M, k), dtype=torch.uint8, device="cuda"), torch.empty((M, k // 128), device="cuda")
    K.kda_add_rmsnorm_fp8(x, w, codes, scales, residual=r, residual_out=r)
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        K.kda_add_rmsnorm_fp8(x, w, codes, scales, residual=r, residual_out=r)
    torch.cuda.current_stream().wait_stream(s)
    for i in range(4):
        x2, r2, _ = make(M, k, BF, BF, 50 + i)
        x.copy_(x2)
        r.copy_(r2)
        graph.replay()
        c2, s2 = torch.empty_like(codes), torch.empty_like(scales)
        K.kda_add_rmsnorm_fp8(x2, w, c2, s2, residual=r2, residual_out=r2)
        torch.cuda.synchronize()
        assert torch.equal(codes, c2) and torch.equal(scales, s2) and torch.equal(r, r2)
