"""The norms around a block (float32, bfloat16 and block-FP8 output) on the GPU
against the formula in 64 bits.

Tolerances, u = 2^-24. A norm's factor (sum of squares over n terms a lane, at most 16
partial sums, mean, eps, root, reciprocal) is off by at most (n + 20) u; with the
two products n = x rn w by (n + 22) u. The sigmoid on the hardware exponential and
reciprocal (one ulp each): the exponential's argument is rounded twice, relative
error (2 |g| + 4) u of it, so (2 |g| + 10) u. h = rs r + bs act(g) n: relative to T
= |rs r| + |bs act(g) n| another 4 u, in all e = (n + 36 + 2 |g|) u T. y = h rh w: h's
error, and rh's, which follows that of sum h^2: by Cauchy's inequality at most
||e|| / ||h|| relative, plus (n + 22) u. A stored type adds its half step."""
import pytest
import torch

from gated_delta_rule_02_amd import kda as K
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
POST, EPS = 1e-5, 1e-6
RS, BS = 0.75, 1.25
BF, F = torch.bfloat16, torch.float32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2 if dtype != F else 0.0


def lanes(k):
    return 64 if k <= 1024 else 256 if k <= 2048 else 512 if k <= 8192 else 1024


def make(M, k, xd, rd, gate, gd, pad, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((M, k + pad), generator=g) * (torch.rand((M, 1), generator=g) * 4 + 0.1)).to(xd).cuda()[:, :k]
    r = (torch.randn((M, k + pad), generator=g) * 2).to(rd).cuda()[:, :k]
    wp, w = ((torch.rand(k, generator=g) + 0.5).cuda() for _ in range(2))
    gt = None
    if gate == "vector":
        gt = torch.randn(k, generator=g).to(gd).cuda()
    elif gate == "rows":
        gt = (torch.randn((M, k + pad), generator=g) * 2).to(gd).cuda()[:, :k]
    return x, r, wp, w, gt


def formula(x, r, wp, w, gt, act):
    """h, y and the bounds of their float32 errors."""
    M, k = x.shape
    n = 8 * -(-k // (8 * lanes(k)))
    x, r, wp, w = (t.double().cpu() for t in (x, r, wp, w))
    branch = x / torch.sqrt((x * x).mean(1, keepdim=True) + POST) * wp
    grow = torch.zeros(())
    if gt is not None:
        gt = gt.double().cpu()
        branch = branch * (torch.sigmoid(gt) if act == "sigmoid" else gt)
        grow = 2 * gt.abs() if act == "sigmoid" else grow
    h = RS * r + BS * branch
    eh = (n + 36 + grow) * U * ((RS * r).abs() + (BS * branch).abs())
    rh = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    y = h * rh * w
    rel = eh.norm(dim=1, keepdim=True) / h.norm(dim=1, keepdim=True).clamp(min=1e-300) + (n + 22) * U
    return h, eh, y, eh * rh * w + rel * y.abs()


def near(got, ref, tol, dtype):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    tol = tol + half_step(dtype) * (ref.abs() + tol)
    print("  worst %.2e of the bound" % float(((got - ref).abs() / tol.clamp(min=1e-300)).max()), flush=True)
    return bool(((got - ref).abs() <= tol).all())


# (M, K, x, residual, y, gate, gate's type, activation, padding)
CASES = [
    (1, 8, F, F, F, None, F, "none", 0), (1, 4096, F, BF, BF, "vector", F, "none", 0), (3, 1000, BF, BF, F, "rows", BF, "sigmoid", 8),
    (5, 1024, BF, F, BF, "rows", F, "none", 16), (7, 1032, BF, BF, F, "vector", BF, "sigmoid", 0),
    (2, 4104, F, F, F, "rows", F, "sigmoid", 8), (33, 5128, BF, BF, BF, "rows", BF, "sigmoid", 24),
    (4, 8192, BF, BF, F, None, F, "none", 0), (3, 8200, BF, F, F, "rows", BF, "sigmoid", 8), (2, 40968, F, BF, F, "vector", F, "none", 0),
    (4099, 136, BF, BF, BF, "vector", BF, "sigmoid", 0), (6, 16384, F, F, BF, "rows", BF, "none", 0),
    (5, 2048, F, BF, F, "rows", F, "sigmoid", 0), (3, 2056, BF, F, BF, "vector", F, "none", 8), (2, 16392, BF, BF, F, "rows", BF, "sigmoid", 0),
    (2, 32768, F, F, F, None, F, "none", 0), (3, 32776, BF, F, BF, "rows", F, "sigmoid", 8),
]


@pytest.mark.parametrize("M,k,xd,rd,yd,gate,gd,act,pad", CASES)
def test_sandwich(M, k, xd, rd, yd, gate, gd, act, pad):
    announce("sandwich %s" % ((M, k, xd, rd, yd, gate, gd, act, pad),))
    x, r, wp, w, gt = make(M, k, xd, rd, gate, gd, pad, M + k)
    y = torch.full((M, k + pad), float("nan"), dtype=yd, device="cuda")
    ro = torch.full((M, k + pad), float("nan"), dtype=rd, device="cuda")
    form = dict(gate=gt, gate_activation=act, residual_scale=RS, branch_scale=BS, post_eps=POST, eps=EPS)
    K.kda_sandwich_rmsnorm(x, wp, r, ro[:, :k], w, y[:, :k], **form)
    torch.cuda.synchronize()
    h, eh, ref, ey = formula(x, r, wp, w, gt, act)
    assert near(ro[:, :k], h, eh, rd) and near(y[:, :k], ref, ey, yd)
    assert torch.isnan(y[:, k:]).all() and torch.isnan(ro[:, k:]).all()
    # in place, and without storing the residual: the same bits
    r2, y2, y3 = r.clone(), torch.empty_like(y[:, :k]), torch.empty_like(y[:, :k])
    K.kda_sandwich_rmsnorm(x, wp, r2, r2, w, y2, **form)
    K.kda_sandwich_rmsnorm(x, wp, r, None, w, y3, **form)
    torch.cuda.synchronize()
    assert torch.equal(r2, ro[:, :k]) and torch.equal(y2, y[:, :k]) and torch.equal(y3, y[:, :k])


@pytest.mark.parametrize("M,k,xd,rd,gate,gd,act", [
    (1, 128, F, F, None, F, "none"), (3, 1024, BF, BF, "vector", F, "none"), (37, 4096, F, BF, "rows", BF, "sigmoid"),
    (5, 5120, BF, F, "rows", F, "none"), (3, 12800, BF, BF, "vector", BF, "sigmoid")])
def test_sandwich_fp8_equals_quantizing_the_float32_norm(M, k, xd, rd, gate, gd, act):
    announce("sandwich_fp8 %s" % ((M, k, xd, rd, gate, gd, act),))
    x, r, wp, w, gt = make(M, k, xd, rd, gate, gd, 0, M + k)
    r[M - 1] = 0
    x[M - 1] = 0  # an all-zero row: scale 1, codes 0
    form = dict(gate=gt, gate_activation=act, residual_scale=RS, branch_scale=BS, post_eps=POST, eps=EPS)
    y, ro, ro2 = torch.empty((M, k), device="cuda"), torch.empty_like(r), torch.empty_like(r)
    K.kda_sandwich_rmsnorm(x, wp, r, ro, w, y, **form)
    q, s = torch.empty((M, k), dtype=torch.uint8, device="cuda"), torch.empty((M, k // 128), device="cuda")
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    K.kda_quantize_fp8(y, q, s)
    K.kda_sandwich_rmsnorm_fp8(x, wp, r, ro2, w, q2, s2, **form)
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(ro, ro2)
    assert (s2[M - 1] == 1).all() and (q2[M - 1] == 0).all()


def test_a_gate_of_zero_leaves_the_plain_norm_of_the_residual():
    """rs = 1, gate 0: kda_add_rmsnorm of the residual alone (the same operations, the same bits)."""
    x, r, wp, w, _ = make(9, 2048, BF, F, None, F, 0, 3)
    y, y2, ro = torch.empty_like(r), torch.empty_like(r), torch.empty_like(r)
    K.kda_sandwich_rmsnorm(x, wp, r, ro, w, y, gate=torch.zeros(2048, device="cuda"), eps=EPS)
    K.kda_add_rmsnorm(r, w, y2, eps=EPS)
    torch.cuda.synchronize()
    assert torch.equal(ro, r) and torch.equal(y, y2)


def test_non_finite_rows_stay_in_their_rows():
    x, r, wp, w, gt = make(6, 1032, BF, F, "rows", F, 0, 4)
    y, ro = torch.empty_like(r), torch.empty_like(r)
    K.kda_sandwich_rmsnorm(x, wp, r, ro, w, y, gate=gt)
    x[2, 5] = float("nan")
    gt[4, 9] = float("inf")
    y2, ro2 = torch.empty_like(r), torch.empty_like(r)
    K.kda_sandwich_rmsnorm(x, wp, r, ro2, w, y2, gate=gt)
    keep = torch.tensor([0, 1, 3, 5], device="cuda")
    assert torch.equal(y[keep], y2[keep]) and torch.equal(ro[keep], ro2[keep])
    assert torch.isnan(y2[2]).all() and not torch.isfinite(ro2[4, 9]) and torch.isnan(y2[4, 9])
    # a call of no rows
    e = torch.empty((0, 64), device="cuda")
    K.kda_sandwich_rmsnorm(e, torch.ones(64, device="cuda"), e, None, torch.ones(64, device="cuda"), torch.empty_like(e))


@pytest.mark.parametrize("M,k", [((1 << 23) + 4099, 2176)])
def test_more_rows_than_a_launch_holds(M, k):
    """512 threads a row pass 2^32 threads at 2^23 rows: the rows beyond are as all others.
    The rows repeat a block of 4096, whose results every block has to equal bit for bit."""
    announce("sandwich_fp8 %d x %d" % (M, k))
    if torch.cuda.mem_get_info()[0] < (70 << 30):
        pytest.skip("takes 56 GB of device memory")
    n = 4096
    x, _, wp, w, gt = make(n, k, BF, BF, "vector", F, 0, 21)
    want_q, want_s = torch.empty((n, k), dtype=torch.uint8, device="cuda"), torch.empty((n, k // 128), device="cuda")
    K.kda_sandwich_rmsnorm_fp8(x, wp, x, None, w, want_q, want_s, gate=gt)
    rows = torch.empty((M, k), dtype=BF, device="cuda")
    for at in range(0, M, n):
        rows[at:at + n] = x[:M - at]
    q, s = torch.zeros((M, k), dtype=torch.uint8, device="cuda"), torch.zeros((M, k // 128), device="cuda")
    K.kda_sandwich_rmsnorm_fp8(rows, wp, rows, None, w, q, s, gate=gt)  # (the residual's rows are x's)
    whole = M // n * n
    assert all(bool((t[:whole].view(-1, n, t.shape[1])[at:at + 64] == want).all())
               for t, want in ((q, want_q), (s, want_s)) for at in range(0, M // n, 64))
    assert torch.equal(q[whole:], want_q[:M - whole]) and torch.equal(s[whole:], want_s[:M - whole])
    del rows, q, s
    torch.cuda.empty_cache()
