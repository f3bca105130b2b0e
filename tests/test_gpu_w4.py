"""Products with 4-bit weights on the GPU against the formula in 64 bits.

Exact cases: x and the scales are small integers and powers of two, so that every
product and partial sum is an integer multiple of a power of two below 2^24 of
them: the float32 result has no rounding and must be equal bit for bit.

Other cases: u = 2^-24. The kernel sums x (16 + c) and x over a group (G terms each, a
matrix instruction may truncate: 2u a step), subtracts (16 + z) times the second,
scales, and adds K / G groups, at most 8 wavefronts' sums and the residual: an
error below 2 u (G + K / G + 16) sum_k |s| |x| (32 + c + z), and a stored
bfloat16's half step."""
import pytest
import torch

from gated_delta_rule_02_amd import kda as K
from tests.gpu_util import announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F = torch.bfloat16, torch.float32


def weight(N, k, G, sd, zeros, seed, whole=False):
    """codes [N, k/2], scales, zeros (or None) on the GPU with padded rows, and W, |s| (32 + c + z) in 64 bits."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (N, k // 2 + 4), generator=g, dtype=torch.uint8)
    if whole:
        scales = 2.0 ** torch.randint(-1, 2, (N, k // G + 1), generator=g).float()
    else:
        scales = (torch.rand((N, k // G + 1), generator=g) + 0.5) * 0.02
    scales = scales.to(sd)
    z = torch.randint(0, 16, (N, k // G + 3), generator=g, dtype=torch.uint8) if zeros else None
    c = torch.stack([codes[:, :k // 2] % 16, codes[:, :k // 2] // 16], -1).reshape(N, k).double()
    s = scales[:, :k // G].double().repeat_interleave(G, 1)
    zz = z[:, :k // G].double().repeat_interleave(G, 1) if zeros else torch.full_like(c, 8)
    dev = (codes.cuda()[:, :k // 2], scales.cuda()[:, :k // G], z.cuda()[:, :k // G] if zeros else None)
    return dev, s * (c - zz), s.abs() * (32 + c + zz)


def packed(dev):
    codes, scales, zeros = dev
    # a padded scales row has as many columns as groups: the group follows from the shapes
    return K.kda_w4_pack(codes, scales, zeros)


# (M, N, K, group, scale type, zero points, y, residual, padding of x's rows)
CASES = [
    (1, 16, 128, 128, BF, False, F, None, 0), (1, 1, 32, 32, F, True, F, None, 0), (1, 4096, 8192, 128, BF, False, BF, BF, 0),
    (2, 17, 96, 32, BF, True, BF, F, 8), (5, 4999, 4128, 32, F, True, F, None, 0), (15, 33, 192, 64, F, False, F, F, 16),
    (16, 130, 1024, 64, BF, True, F, BF, 0), (17, 257, 4160, 64, BF, True, BF, None, 8), (31, 48, 256, 128, F, True, F, None, 0),
    (32, 1001, 2048, 128, BF, False, F, F, 0), (33, 64, 160, 32, BF, False, BF, BF, 24), (63, 515, 8160, 32, F, True, F, None, 0),
    (64, 100, 384, 128, BF, True, F, F, 8), (65, 31, 640, 128, F, False, F, None, 0), (200, 79, 448, 64, BF, True, BF, F, 0),
]


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("M,N,k,G,sd,zeros,yd,rd,pad", CASES)
def test_gemm_w4(M, N, k, G, sd, zeros, yd, rd, pad, whole):
    announce("gemm_w4 %s" % ((M, N, k, G, sd, zeros, yd, rd, pad, whole),))
    dev, W, bound = weight(N, k, G, sd, zeros, M + N + k, whole)
    g = torch.Generator().manual_seed(M * 7 + k)
    if whole:  # at most 8192 * 2 * 31 * 2 / (1 / 2) < 2^21
        x = torch.randint(-2, 3, (M, k + pad), generator=g).to(BF)
        res = torch.randint(-9, 10, (M, N + 5), generator=g).to(rd) if rd else None
    else:
        x = torch.randn((M, k + pad), generator=g).to(BF)
        res = torch.randn((M, N + 5), generator=g).to(rd) if rd else None
    xc = x.cuda()[:, :k]
    w = packed(dev)
    assert (w.N, w.K, w.group) == (N, k, G)
    y = torch.full((M, N + 3), float("nan"), dtype=yd, device="cuda")
    rc = None if res is None else res.cuda()[:, :N]
    out = K.kda_gemm_w4(xc, w, y[:, :N], residual=rc)
    torch.cuda.synchronize()
    assert out.data_ptr() == y.data_ptr() and torch.isnan(y[:, N:]).all()
    xr = x[:, :k].double()
    ref = xr @ W.t() + (0 if res is None else res[:, :N].double())
    got = y[:, :N].double().cpu()
    if whole:
        assert torch.equal(got, ref.to(yd).double())
    else:
        tol = 2 * U * (G + k / G + 16) * (xr.abs() @ bound.t()) + (ref.abs() * 2.0 ** -8 if yd == BF else 0)
        print("  worst %.2e of the bound" % float(((got - ref).abs() / tol).max()), flush=True)
        assert ((got - ref).abs() <= tol).all()
    if rd is not None:  # in place: the same bits as from a residual of y's type
        a = rc.to(yd).clone()
        b = torch.empty((M, N), dtype=yd, device="cuda")
        K.kda_gemm_w4(xc, w, b, residual=a)
        K.kda_gemm_w4(xc, w, a, residual=a)
        torch.cuda.synchronize()
        assert torch.equal(a, b)


@pytest.mark.parametrize("N,k,G,sd,zeros", [(16, 128, 128, F, False), (5, 32, 32, BF, True), (130, 4160, 64, F, True),
                                            (1000, 224, 32, BF, False)])
def test_expand(N, k, G, sd, zeros):
    """Two roundings: the product to float32, then to bfloat16 (2^-8 and 2^-24 of the value)."""
    announce("w4_expand %s" % ((N, k, G, sd, zeros),))
    dev, W, _ = weight(N, k, G, sd, zeros, N + k)
    out = torch.full((N, k + 8), float("nan"), dtype=BF, device="cuda")
    K.kda_w4_expand(packed(dev), out[:, :k])
    torch.cuda.synchronize()
    assert torch.isnan(out[:, k:]).all()
    got = out[:, :k].double().cpu()
    assert ((got - W).abs() <= W.abs() * (2.0 ** -8 + 2.0 ** -23)).all()


def test_more_rows_than_a_slab_agree_with_single_rows():
    """The rows of a large call equal those of calls of one row, but for the order of the sums."""
    dev, W, bound = weight(300, 1024, 64, BF, True, 5)
    w = packed(dev)
    x = torch.randn((150, 1024), generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    y = torch.empty((150, 300), device="cuda")
    K.kda_gemm_w4(x, w, y)
    one = torch.empty((1, 300), device="cuda")
    for m in (0, 15, 16, 63, 64, 149):
        K.kda_gemm_w4(x[m:m + 1], w, one)
        tol = 4 * U * (64 + 16 + 16) * (x[m:m + 1].double().cpu().abs() @ bound.t())
        assert ((one.double() - y[m:m + 1].double()).abs().cpu() <= tol).all(), m


def test_non_finite_rows_stay_in_their_rows():
    dev, W, _ = weight(50, 256, 128, F, False, 9)
    w = packed(dev)
    x = torch.randn((20, 256), generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    clean = torch.empty((20, 50), device="cuda")
    K.kda_gemm_w4(x, w, clean)
    x[3, 7] = float("nan")
    x[18, 200] = float("inf")
    y = torch.empty((20, 50), device="cuda")
    K.kda_gemm_w4(x, w, y)
    bad = torch.tensor([3, 18], device="cuda")
    keep = torch.tensor([m for m in range(20) if m not in (3, 18)], device="cuda")
    assert torch.isnan(y[bad]).all() and torch.equal(y[keep], clean[keep])


def test_empty_and_repeated():
    dev, _, _ = weight(40, 128, 64, F, True, 4)
    w = packed(dev)
    y = torch.full((0, 40), 1.0, device="cuda")
    K.kda_gemm_w4(torch.empty((0, 128), dtype=BF, device="cuda"), w, y)
    x = torch.randn((9, 128), generator=torch.Generator().manual_seed(3)).to(BF).cuda()
    a, b = torch.empty((9, 40), device="cuda"), torch.empty((9, 40), device="cuda")
    K.kda_gemm_w4(x, w, a)
    K.kda_gemm_w4(x, w, b)
    assert torch.equal(a, b)


@pytest.mark.parametrize("M,N,k,G,sd,zeros", [
    # the forms for more rows: many row tiles, few, two turns of column tiles and odd numbers of them
    (9, 41000, 640, 128, BF, True), (16, 30000, 1184, 32, F, False), (17, 41000, 128, 64, BF, True), (20, 9000, 1152, 128, F, False), (29, 30000, 640, 32, F, True), (32, 7000, 2176, 128, BF, False),
    (33, 16000, 896, 64, F, True), (47, 41024, 256, 32, BF, True), (64, 30011, 1280, 128, BF, False), (64, 41024, 512, 32, F, True),
    (64, 20000, 2048, 64, BF, False), (97, 12345, 384, 128, F, True), (64, 3000, 8192, 32, F, True)])
def test_forms_for_more_rows(M, N, k, G, sd, zeros):
    """Exact sums (whole), against a float64 product on the GPU."""
    announce("gemm_w4 forms %s" % ((M, N, k, G, sd, zeros),))
    dev, W, _ = weight(N, k, G, sd, zeros, M + N + k, True)
    x = torch.randint(-2, 3, (M, k), generator=torch.Generator().manual_seed(k)).to(BF).cuda()
    y = torch.full((M, N), float("nan"), device="cuda")
    K.kda_gemm_w4(x, packed(dev), y)
    ref = torch.mm(x.double(), W.cuda().t().contiguous())
    assert torch.equal(y.double(), ref)


@pytest.mark.parametrize("M,N,k,G,sd,zeros", [
    # few row tiles and many column tiles, taken in turns of four with every remainder, and columns that end inside the last
    (12, 8001, 4160, 64, BF, True), (5, 4999, 4128, 32, F, True), (16, 8000, 1184, 32, F, False), (9, 8000, 1920, 128, BF, False),
    (28, 8100, 5152, 32, BF, True), (50, 4099, 8064, 128, F, True), (64, 4096, 8192, 64, BF, False), (40, 4010, 7072, 32, F, True),
    # many row tiles and two or four tiles of rows
    (31, 41024, 1216, 64, F, True), (32, 41000, 1056, 32, BF, False), (60, 40000, 704, 64, F, True),
    # as many rows as several workgroups' and one more
    (81, 12000, 352, 32, BF, False), (161, 1000, 4160, 64, F, True), (193, 9000, 1184, 32, BF, True)])
def test_rows_beside_nan(M, N, k, G, sd, zeros):
    """Exact sums (whole); NaN behind every row of x and behind the last one, which no copy may bring in."""
    announce("gemm_w4 beside NaN %s" % ((M, N, k, G, sd, zeros),))
    dev, W, _ = weight(N, k, G, sd, zeros, M + N + k, True)
    x = torch.full((M + 3, k + 8), float("nan"), dtype=BF, device="cuda")
    x[:M, :k] = torch.randint(-2, 3, (M, k), generator=torch.Generator().manual_seed(k)).to(BF).cuda()
    y = torch.full((M + 2, N), float("nan"), device="cuda")
    K.kda_gemm_w4(x[:M, :k], packed(dev), y[:M])
    ref = torch.mm(x[:M, :k].double(), W.cuda().t().contiguous())
    assert torch.equal(y[:M].double(), ref) and torch.isnan(y[M:]).all()


@pytest.mark.parametrize("M,N,k,G,sd,zeros", [(1, 500, 4096, 64, BF, True), (5, 700, 4096, 128, F, False), (1, 41024, 1024, 64, BF, True),
                                              (40, 3000, 4096, 128, F, False), (64, 16000, 1024, 32, F, True)])
def test_codes_near_their_zero_point(M, N, k, G, sd, zeros):
    """Codes within 1 of the zero point, and rows at it throughout (W = 0): the sums of (16 + c) x and
    (16 + z) x nearly cancel. The bound is that of any codes, in terms of what is summed."""
    announce("gemm_w4 near the zero point %s" % ((M, N, k, G, sd, zeros),))
    g = torch.Generator().manual_seed(N + k)
    z = torch.randint(0, 16, (N, k // G), generator=g) if zeros else torch.full((N, k // G), 8)
    zz = z.repeat_interleave(G, 1)
    c = (zz + torch.randint(-1, 2, (N, k), generator=g)).clamp(0, 15)
    c[::7] = zz[::7]
    scales = ((torch.rand((N, k // G), generator=g) + 0.5) * 0.02).to(sd)
    w = K.kda_w4_pack((c[:, 0::2] + 16 * c[:, 1::2]).to(torch.uint8).cuda(), scales.cuda(), z.to(torch.uint8).cuda() if zeros else None)
    x = torch.randn((M, k), generator=g).to(BF).cuda()
    y = torch.empty((M, N), device="cuda")
    K.kda_gemm_w4(x, w, y)
    s, c, zz = scales.cuda().double().repeat_interleave(G, 1), c.cuda().double(), zz.cuda().double()
    ref = torch.mm(x.double(), (s * (c - zz)).t().contiguous())
    tol = 2 * U * (G + k / G + 16) * torch.mm(x.double().abs(), (s * (32 + c + zz)).t().contiguous())
    error = (y.double() - ref).abs()
    print("  worst %.2e of the bound, off by %.1e of the norm" % (float((error / tol).max()), float(error.norm() / ref.norm())), flush=True)
    assert (error <= tol).all()


@pytest.mark.parametrize("M,N,k,G,zeros", [(1, 41024, 4096, 64, True), (5, 4999, 4128, 32, True), (64, 41024, 4096, 128, False),
                                           (20, 4096, 8192, 128, False), (200, 8200, 1152, 64, True)])
def test_calls_repeat_themselves(M, N, k, G, zeros):
    """The same bits in every call: after other work, on two streams at once and from a graph."""
    announce("gemm_w4 repeated %s" % ((M, N, k, G, zeros),))
    g = torch.Generator(device="cuda").manual_seed(N)
    codes = torch.randint(0, 256, (N, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    z = torch.randint(5, 11, (N, k // G), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    w = K.kda_w4_pack(codes, ((torch.rand((N, k // G), generator=g, device="cuda") + 0.5) * 0.01).to(BF), z)
    x = torch.randn((M, k), generator=g, device="cuda").to(BF)
    new = lambda: torch.full((M, N), float("nan"), device="cuda")
    want = new()
    K.kda_gemm_w4(x, w, want)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    outs = [[new() for _ in range(6)] for _ in range(3)]
    torch.cuda.synchronize()
    for i in range(6):
        K.kda_gemm_w4(x, w, outs[0][i], stream=streams[0])
        K.kda_gemm_w4(x, w, outs[1][i], stream=streams[1])
        torch.empty(1 << 28, dtype=torch.uint8, device="cuda").fill_(i)  # (other lines in the caches)
        K.kda_gemm_w4(x, w, outs[2][i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for row in outs for o in row)
    graph, y = torch.cuda.CUDAGraph(), new()
    with torch.cuda.stream(streams[0]), torch.cuda.graph(graph, stream=streams[0]):
        K.kda_gemm_w4(x, w, y)
    for i in range(3):
        torch.cuda.synchronize()
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_packed_expanded_and_used_on_another_stream():
    """All three calls with stream=, none on the current one: the same bits."""
    dev, _, _ = weight(500, 1024, 64, BF, True, 31)
    x = torch.randn((20, 1024), generator=torch.Generator().manual_seed(32)).to(BF).cuda()
    w = packed(dev)
    want, wide = torch.empty((20, 500), device="cuda"), torch.empty((500, 1024), dtype=BF, device="cuda")
    K.kda_gemm_w4(x, w, want), K.kda_w4_expand(w, wide)
    y, other = torch.empty_like(want), torch.empty_like(wide)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    w2 = K.kda_w4_pack(*dev, stream=st)
    K.kda_gemm_w4(x, w2, y, stream=st), K.kda_w4_expand(w2, other, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(w2.packed, w.packed) and torch.equal(y, want) and torch.equal(other, wide)
