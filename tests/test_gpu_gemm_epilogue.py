"""C = act(A B^T + bias) + residual on the GPU against the same in 64 bits.

Tolerances, u = 2^-24: the products of bfloat16 values are exact in float32; the
accumulator takes K/32 matrix steps whose 32 products it adds with one rounding
or truncation each at most (2 u), relative to the sum of magnitudes S = |A| |B|^T
of what is added; the joined parts of K add 4 more. So the product is within
2 (K/32 + 32 + 8) u S. The bias adds one rounding, an activation's slope is at
most 1.13 and its own error (two hardware steps of an ulp each, the argument of
the exponential scaled once) 8 u (1 + |z|); the residual one more. A stored
bfloat16 adds 2^-8 of the value."""
import pytest
import torch

from gated_delta_rule_02_amd import kda as K
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F = torch.bfloat16, torch.float32
ACT = {"none": lambda z: z, "relu": torch.relu, "silu": lambda z: z * torch.sigmoid(z),
       "gelu": lambda z: z * torch.special.ndtr(z), "sigmoid": torch.sigmoid}


def make(M, N, k, seed, pad=(0, 0, 0)):
    g = torch.Generator().manual_seed(seed)
    A = torch.randn((M, k + pad[0]), generator=g).to(BF).cuda()[:, :k]
    B = (torch.randn((N, k + pad[1]), generator=g) * k ** -0.5).to(BF).cuda()[:, :k]
    bias = torch.randn(N, generator=g).cuda()
    res = torch.randn((M, N + pad[2]), generator=g).cuda()
    return A, B, bias, res


def expected(A, B, bias, act, res):
    a, b = A.double().cpu(), B.double().cpu()
    z = a @ b.t()
    S = a.abs() @ b.abs().t()
    if bias is not None:
        z = z + bias.double().cpu()
    y = ACT[act](z)
    c = y if res is None else y + res.double().cpu()
    tol = 1.13 * (2 * (A.shape[1] / 32 + 40) * U * S + U * z.abs())
    if act not in ("none", "relu"):
        tol = tol + 8 * U * (1 + z.abs())
    return c, tol + U * c.abs()


def within(got, ref, tol):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    over = float(((got - ref).abs() / tol).max())
    print("  %.3f of the tolerance" % over, flush=True)
    return over <= 1


def check(C, ref, tol):
    if C.dtype == BF:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    return within(C, ref, tol)


# (M, N, K, act, bias, residual dtype or None, C dtype, (padding of A, B, C and residual))
CASES = [
    (1, 1, 8, "none", True, F, F, (0, 0, 3)), (1, 16, 64, "relu", False, None, BF, (0, 0, 0)),
    (1, 4096, 1024, "none", False, BF, BF, (0, 0, 0)), (3, 100, 264, "silu", True, BF, F, (8, 16, 4)),
    (16, 37, 2048, "gelu", True, F, BF, (0, 8, 3)), (17, 272, 1096, "sigmoid", True, None, F, (0, 0, 0)),
    (33, 65, 512, "none", True, F, F, (8, 0, 7)), (48, 129, 4104, "silu", False, BF, BF, (0, 0, 7)),
    (64, 64, 72, "gelu", True, F, F, (0, 0, 0)), (65, 256, 320, "none", True, BF, F, (0, 0, 0)),
    (65, 61, 256, "relu", True, F, BF, (0, 0, 3)), (129, 333, 264, "silu", True, F, F, (0, 0, 3)),
    (100, 320, 256, "gelu", True, BF, BF, (8, 8, 4)), (257, 392, 192, "sigmoid", False, F, F, (0, 0, 0)),
    (300, 640, 448, "none", True, F, BF, (0, 0, 0)), (513, 772, 1088, "silu", True, BF, F, (0, 64, 12)),
]


@pytest.mark.parametrize("M,N,k,act,bias,rd,cd,pad", CASES)
def test_gemm_epilogue(M, N, k, act, bias, rd, cd, pad):
    announce("gemm_epilogue M=%d N=%d K=%d %s bias=%s res=%s C=%s pad=%s" % (M, N, k, act, bias, rd, cd, pad))
    A, B, b, res = make(M, N, k, M * 7 + N, pad)
    b = b if bias else None
    r = None if rd is None else res.to(rd)[:, :N]
    C = torch.full((M, N + pad[2]), float("nan"), dtype=cd, device="cuda")
    K.kda_gemm_epilogue(A, B, C[:, :N], bias=b, activation=act, residual=r)
    torch.cuda.synchronize()
    ref, tol = expected(A, B, b, act, r)
    assert check(C[:, :N], ref, tol)
    assert torch.isnan(C[:, N:]).all()
    if rd == cd:  # accumulated in place: the same result
        D = res.to(cd)
        edge = D[:, N:].clone()
        K.kda_gemm_epilogue(A, B, D[:, :N], bias=b, activation=act, residual=D[:, :N])
        torch.cuda.synchronize()
        assert torch.equal(D[:, :N], C[:, :N]) and torch.equal(D[:, N:], edge)


@pytest.mark.parametrize("M", [1, 16, 31, 64, 65, 128, 300])
@pytest.mark.parametrize("N,k", [(16, 64), (80, 1536), (320, 200)])
def test_gemm_epilogue_without_epilogue(M, N, k):
    """No bias, activation or residual: the plain product, for every form; run to
    run the same bits."""
    announce("gemm_epilogue plain M=%d N=%d K=%d" % (M, N, k))
    A, B, _, _ = make(M, N, k, M + N)
    C = torch.full((M, N), float("nan"), device="cuda")
    K.kda_gemm_epilogue(A, B, C)
    D = torch.empty_like(C)
    K.kda_gemm_epilogue(A, B, D)
    torch.cuda.synchronize()
    ref, tol = expected(A, B, None, "none", None)
    assert check(C, ref, tol) and torch.equal(C, D)


@pytest.mark.parametrize("M", [5, 40, 200])
def test_gemm_epilogue_far_arguments(M):
    """Arguments far out on both sides of every activation, infinities and NaN
    in single rows: they stay there, and nothing else is touched by them."""
    announce("gemm_epilogue far arguments M=%d" % M)
    N, k = 48, 128
    A, B, _, _ = make(M, N, k, 5)
    bias = torch.linspace(-200, 200, N).cuda()
    A[2, 7] = float("nan")
    A[3, 9] = float("inf")
    rows = [i for i in range(M) if i not in (2, 3)]
    for act in ACT:
        C = torch.empty((M, N), device="cuda")
        K.kda_gemm_epilogue(A, B, C, bias=bias, activation=act)
        torch.cuda.synchronize()
        ref, tol = expected(A[rows], B, bias, act, None)
        # exp of the scaled argument: 200 times its rounding
        assert within(C[rows], ref, tol + 400 * U * ref.abs() + 1e-37), act
        assert torch.isnan(C[2]).all(), act
        z = A[3].float() @ B.float().t() + bias  # +-inf
        if act in ("none", "relu", "sigmoid"):
            assert torch.equal(C[3], ACT[act](z)), act


def test_gemm_epilogue_captured():
    """Captured with the output accumulated in place, replayed with eager work
    between: every replay equals the eager call."""
    announce("gemm_epilogue captured")
    for M in (3, 130):
        N, k = 132, 384
        A, B, b, res = make(M, N, k, 1)
        C = res.clone()
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
            K.kda_gemm_epilogue(A, B, C, bias=b, activation="silu", residual=C)
        torch.cuda.current_stream().wait_stream(s)
        D = res.clone()
        for i in range(4):
            graph.replay()
            K.kda_gemm_epilogue(A, B, D, bias=b, activation="silu", residual=D)
            torch.cuda.synchronize()
            assert torch.equal(C, D)


@pytest.mark.parametrize("M,N,k", [
    (16, 4096, 136), (9, 8200, 72), (30, 4104, 200), (33, 8192, 136), (64, 4104, 72), (90, 4096, 136), (100, 8190, 72),
    (192, 4096, 200), (250, 4100, 136), (330, 4104, 72), (333, 4096, 328), (500, 4096, 136), (515, 4104, 72), (1030, 4096, 72),
    (1000, 4100, 136), (2050, 4096, 64), (4100, 4096, 128), (7000, 260, 192), (5000, 36, 72), (1, 41024, 64),
])
def test_gemm_epilogue_wide(M, N, k):
    """Sizes that fill the compute units once or several times over, in whole and
    ragged tiles: each tile form, with everything in the epilogue."""
    announce("gemm_epilogue wide M=%d N=%d K=%d" % (M, N, k))
    pad = (0, 8, -N % 4)
    A, B, b, res = make(M, N, k, M + N, pad)
    r = res[:, :N].bfloat16() if (M + N) % 3 == 0 else res[:, :N]
    if r.dtype == BF:
        r = torch.nn.functional.pad(r, (0, pad[2]))[:, :N]
    C = torch.full((M, N + pad[2]), float("nan"), dtype=BF if M % 2 else F, device="cuda")
    K.kda_gemm_epilogue(A, B, C[:, :N], bias=b, activation="silu", residual=r)
    torch.cuda.synchronize()
    ref, tol = expected(A, B, b, "silu", r)
    assert check(C[:, :N], ref, tol)
    assert torch.isnan(C[:, N:]).all()


@pytest.mark.parametrize("M,N,k", [
    (1000, 8190, 200), (2890, 2084, 72), (1500, 4104, 264), (4090, 4090, 1096), (4090, 4090, 1088), (3900, 4070, 1608),
    (1480, 3333, 264),
    (700, 8190, 136), (1900, 4100, 520), (60, 2050, 1032), (150, 4100, 72),
    (1500, 4100, 520), (2990, 2050, 520), (2050, 500, 264), (60, 1100, 72),
])
def test_gemm_epilogue_tall_tiles(M, N, k):
    """The tall and the 256 x 256 tiles (and the small ones of long K) with every edge
    ragged, K not a multiple of their step: what follows a row's last value is NaN, so a
    chunk read past K would show in every column."""
    announce("gemm_epilogue tall tiles M=%d N=%d K=%d" % (M, N, k))
    pad = (24, 16, -N % 4)
    A, B, b, res = make(M, N, k, M + N, pad)
    for x in (A, B):
        x.as_strided((x.shape[0], x.stride(0)), (x.stride(0), 1))[:, k:] = float("nan")
    C = torch.full((M, N + pad[2]), float("nan"), dtype=BF if M % 200 else F, device="cuda")
    K.kda_gemm_epilogue(A, B, C[:, :N], bias=b, activation="relu", residual=res[:, :N])
    torch.cuda.synchronize()
    ref, tol = expected(A, B, b, "relu", res[:, :N])
    assert check(C[:, :N], ref, tol)
    assert torch.isnan(C[:, N:]).all()
