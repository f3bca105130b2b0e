"""Host-side validation of the 4-bit products, the norms around a block and the
beam search's entry points: every rejected call below is refused before anything
reaches the device, with the documented status. No GPU is needed."""
import pytest
import torch

from gated_delta_rule_02_amd import kda as K
from tests.test_abi_cpu import call, fake

INVALID, UNSUPPORTED, WORKSPACE = K.KDA_ERR_INVALID_ARG, K.KDA_ERR_UNSUPPORTED, K.KDA_ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")


# ---------------------------------------------------------------- norms around a block
def sandwich(fp8=False, **over):
    a = dict(x=fake(1), x_ld=512, xd=K.KDA_BF16, wp=fake(2), pe=1e-6, g=fake(3), g_ld=512, gd=K.KDA_BF16, act=4, r=fake(4),
             r_ld=512, ro=fake(5), ro_ld=512, rd=K.KDA_BF16, rs=0.5, bs=2.0, w=fake(6), M=7, K=512, eps=1e-6, y=fake(7),
             y_ld=512, yd=K.KDA_BF16, s=fake(8), s_ld=4)
    a.update(over)
    tail = (a["y"], a["y_ld"], a["s"], a["s_ld"]) if fp8 else (a["y"], a["y_ld"], a["yd"])
    return call("kda_sandwich_rmsnorm_fp8" if fp8 else "kda_sandwich_rmsnorm", a["x"], a["x_ld"], a["xd"], a["wp"], a["pe"],
                a["g"], a["g_ld"], a["gd"], a["act"], a["r"], a["r_ld"], a["ro"], a["ro_ld"], a["rd"], a["rs"], a["bs"],
                a["w"], a["M"], a["K"], a["eps"], *tail, None)[0]


@pytest.mark.parametrize("fp8", [False, True])
def test_sandwich_rmsnorm_validation(fp8):
    assert sandwich(fp8, M=0) == K.KDA_OK  # nothing to do
    for name in ("x", "wp", "w", "r", "y"):
        assert sandwich(fp8, **{name: None}) == INVALID, name
    assert sandwich(fp8, M=-1) == INVALID and sandwich(fp8, M=1 << 31) == INVALID and sandwich(fp8, M=1 << 24) == UNSUPPORTED
    assert sandwich(fp8, K=0) == INVALID and sandwich(fp8, K=12) == UNSUPPORTED
    for name in ("x_ld", "r_ld", "ro_ld", "y_ld", "g_ld"):
        assert sandwich(fp8, **{name: 504}) == INVALID and sandwich(fp8, **{name: 516}) == INVALID, name
    for name in ("eps", "pe"):
        assert sandwich(fp8, **{name: -1.0}) == INVALID and sandwich(fp8, **{name: NAN}) == INVALID, name
    for name in ("rs", "bs"):
        assert sandwich(fp8, **{name: INF}) == INVALID and sandwich(fp8, **{name: NAN}) == INVALID, name
    for name in ("xd", "rd", "gd"):
        assert sandwich(fp8, **{name: 7}) == INVALID, name
    for act in (1, 2, 3, 5, -1):
        assert sandwich(fp8, act=act) == INVALID, act
    for name in ("x", "wp", "g", "r", "ro", "w"):
        assert sandwich(fp8, **{name: fake(9) + 8}) == INVALID, name
    # outputs over inputs, or over each other
    for i in (1, 2, 3, 4, 5, 6):
        assert sandwich(fp8, y=fake(i)) == INVALID, i
    for i in (1, 2, 3, 6, 7):
        assert sandwich(fp8, ro=fake(i)) == INVALID, i
    assert sandwich(fp8, ro=fake(4) + 16) == INVALID and sandwich(fp8, ro=fake(4), ro_ld=520) == INVALID
    if fp8:
        assert sandwich(fp8, K=520, x_ld=520, r_ld=520, ro_ld=520, y_ld=520, g_ld=520) == UNSUPPORTED
        assert sandwich(fp8, s=None) == INVALID and sandwich(fp8, s_ld=3) == INVALID
        assert sandwich(fp8, s=fake(7)) == INVALID and sandwich(fp8, s=fake(3)) == INVALID and sandwich(fp8, y=fake(9) + 4) == INVALID
    else:
        assert sandwich(fp8, yd=3) == INVALID and sandwich(fp8, y=fake(9) + 8) == INVALID


# ---------------------------------------------------------------- 4-bit weights
def pack(**over):
    a = dict(c=fake(1), ldc=128, s=fake(2), lds=4, sd=K.KDA_F32, z=fake(3), ldz=4, N=100, K=256, G=64, p=fake(4), n=1 << 29)
    a.update(over)
    return call("kda_w4_pack", a["c"], a["ldc"], a["s"], a["lds"], a["sd"], a["z"], a["ldz"], a["N"], a["K"], a["G"], a["p"],
                a["n"], None)[0]


def test_w4_pack_validation():
    for name in ("c", "s", "p"):
        assert pack(**{name: None}) == INVALID and pack(**{name: fake(9) + 8}) == INVALID, name
    assert pack(sd=2) == INVALID
    assert pack(N=0) == INVALID and pack(K=0) == INVALID and pack(G=0) == INVALID
    assert pack(N=1 << 24) == UNSUPPORTED and pack(K=1 << 20, ldc=1 << 19, lds=1 << 14, ldz=1 << 14) == UNSUPPORTED
    for group in (1, 16, 48, 256):
        assert pack(G=group) == UNSUPPORTED, group
    assert pack(K=224) == UNSUPPORTED  # groups of 64 do not fill it
    assert pack(ldc=124) == INVALID and pack(ldc=130) == INVALID and pack(lds=3) == INVALID and pack(ldz=3) == INVALID
    need = K.kda_w4_packed_bytes(100, 256, 64, K.KDA_F32, True)
    assert need == 7 * 2 * 1024 + 7 * 4 * 16 * 5
    assert pack(n=need - 1) == WORKSPACE
    for i in (1, 2, 3):
        assert pack(p=fake(i)) == INVALID, i
    assert K.kda_w4_packed_bytes(100, 256, 48) == 0 and K.kda_w4_packed_bytes(0, 256, 64) == 0


def expand(**over):
    a = dict(p=fake(1), N=100, K=256, G=64, sd=K.KDA_F32, hz=1, W=fake(2), ldw=256)
    a.update(over)
    return call("kda_w4_expand", a["p"], a["N"], a["K"], a["G"], a["sd"], a["hz"], a["W"], a["ldw"], None)[0]


def test_w4_expand_validation():
    assert expand(p=None) == INVALID and expand(W=None) == INVALID and expand(W=fake(1)) == INVALID
    assert expand(W=fake(2) + 8) == INVALID and expand(p=fake(1) + 8) == INVALID
    assert expand(ldw=248) == INVALID and expand(ldw=260) == INVALID
    assert expand(G=96) == UNSUPPORTED and expand(K=255) == UNSUPPORTED and expand(sd=9) == INVALID


def gemm(**over):
    a = dict(x=fake(1), ldx=256, xd=K.KDA_BF16, p=fake(2), G=64, sd=K.KDA_BF16, hz=0, r=fake(3), ldr=100, rd=K.KDA_F32, y=fake(4),
             ldy=100, yd=K.KDA_F32, M=9, N=100, K=256)
    a.update(over)
    return call("kda_gemm_w4", a["x"], a["ldx"], a["xd"], a["p"], a["G"], a["sd"], a["hz"], a["r"], a["ldr"], a["rd"], a["y"],
                a["ldy"], a["yd"], a["M"], a["N"], a["K"], None)[0]


def test_gemm_w4_validation():
    assert gemm(M=0) == K.KDA_OK
    for name in ("x", "p", "y"):
        assert gemm(**{name: None}) == INVALID, name
    for name in ("x", "p", "y", "r"):
        assert gemm(**{name: fake(9) + 8}) == INVALID, name
    assert gemm(xd=K.KDA_F32) == UNSUPPORTED and gemm(xd=9) == INVALID and gemm(yd=9) == INVALID and gemm(rd=9) == INVALID
    assert gemm(sd=9) == INVALID and gemm(G=16) == UNSUPPORTED and gemm(K=288, ldx=288) == UNSUPPORTED
    assert gemm(M=-1) == INVALID and gemm(M=1 << 19) == UNSUPPORTED and gemm(N=0) == INVALID
    assert gemm(ldx=248) == INVALID and gemm(ldx=260) == INVALID and gemm(ldx=1 << 22) == INVALID
    assert gemm(ldy=99) == INVALID and gemm(ldr=99) == INVALID
    assert gemm(y=fake(1)) == INVALID and gemm(y=fake(2) + 256) == INVALID
    assert gemm(r=fake(4) + 16) == INVALID                      # shifted in place
    assert gemm(r=fake(4), ldr=104) == INVALID and gemm(r=fake(4), rd=K.KDA_BF16) == INVALID


# ---------------------------------------------------------------- beam search
def select(**over):
    a = dict(x=fake(1), ld=1000, d=K.KDA_F32, s=fake(2), f=fake(3), B=3, W=4, V=1000, eos=2, ns=fake(4), p=fake(5), t=fake(6),
             nf=fake(7), ws=fake(8), n=1 << 29)
    a.update(over)
    return call("kda_beam_select", a["x"], a["ld"], a["d"], a["s"], a["f"], a["B"], a["W"], a["V"], a["eos"], a["ns"], a["p"],
                a["t"], a["nf"], a["ws"], a["n"], None)[0]


def test_beam_select_validation():
    assert select(B=0) == K.KDA_OK
    for name in ("x", "s", "ns", "p", "t"):
        assert select(**{name: None}) == INVALID and select(**{name: fake(9) + 2}) == INVALID, name
    assert select(d=5) == INVALID and select(ld=999) == INVALID
    assert select(d=K.KDA_BF16, x=fake(9) + 1) == INVALID
    assert select(B=-1) == INVALID and select(W=0) == INVALID and select(V=0) == INVALID
    assert select(W=33) == UNSUPPORTED and select(B=1 << 18) == UNSUPPORTED
    assert select(V=(1 << 30) + 1, ld=(1 << 30) + 1) == UNSUPPORTED
    assert select(eos=-1) == INVALID and select(eos=1000) == INVALID
    need = K.kda_beam_select_workspace_bytes(3, 4, 1000)
    assert need > 0 and select(n=need - 1) == WORKSPACE and select(ws=None) == WORKSPACE and select(ws=fake(8) + 8) == INVALID
    assert K.kda_beam_select_workspace_bytes(0, 4, 1000) == 0 and K.kda_beam_select_workspace_bytes(3, 33, 1000) == 0
    for out in ("ns", "p", "t", "nf", "ws"):
        assert select(**{out: fake(1)}) == INVALID, out
    assert select(p=fake(2)) == INVALID and select(nf=fake(2)) == INVALID and select(ns=fake(3)) == INVALID
    assert select(ns=fake(2) + 4) == INVALID and select(nf=fake(3) + 1) == INVALID
    for a, b in (("ns", 5), ("p", 6), ("t", 7), ("nf", 8)):
        assert select(**{a: fake(b)}) == INVALID, a


def reorder(**over):
    a = dict(p=fake(1), B=3, W=4, s=fake(2), sb=4096, c=fake(3), n=3, cb=512)
    a.update(over)
    return call("kda_beam_reorder", a["p"], a["B"], a["W"], a["s"], a["sb"], a["c"], a["n"], a["cb"], None)[0]


def test_beam_reorder_validation():
    assert reorder(B=0) == K.KDA_OK and reorder(s=None, c=None) == K.KDA_OK and reorder(sb=0, n=0) == K.KDA_OK
    assert reorder(p=None) == INVALID and reorder(p=fake(1) + 2) == INVALID
    assert reorder(s=fake(2) + 8) == INVALID and reorder(c=fake(3) + 8) == INVALID
    assert reorder(sb=4104) == INVALID and reorder(cb=520) == INVALID and reorder(sb=1 << 40) == INVALID
    assert reorder(B=-1) == INVALID and reorder(W=0) == INVALID and reorder(n=-1) == INVALID
    assert reorder(W=33) == UNSUPPORTED and reorder(B=1 << 28) == UNSUPPORTED and reorder(n=1 << 16) == UNSUPPORTED
    assert reorder(c=fake(2)) == INVALID and reorder(p=fake(2) + 64) == INVALID and reorder(p=fake(3) + 64) == INVALID


# ---------------------------------------------------------------- the binding's own checks
BF, F, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


def test_binding_refuses_other_shapes_and_types():
    z = torch.zeros
    w = K.W4Weight(z(64, dtype=U8), 16, 64, 32, K.KDA_F32, False)
    with pytest.raises(ValueError, match="x must be"):
        K.kda_gemm_w4(z((2, 32), dtype=BF), w, z((2, 16)))
    with pytest.raises(ValueError, match="y must have shape"):
        K.kda_gemm_w4(z((2, 64), dtype=BF), w, z((2, 15)))
    with pytest.raises(ValueError, match="residual must have shape"):
        K.kda_gemm_w4(z((2, 64), dtype=BF), w, z((2, 16)), residual=z((16,)).expand(3, 16))
    with pytest.raises(ValueError, match="one GPU device"):
        K.kda_gemm_w4(z((2, 64), dtype=BF), w, z((2, 16)))
    with pytest.raises(TypeError, match="out must be"):
        K.kda_w4_expand(w, z((16, 64)))
    with pytest.raises(ValueError, match="codes must be"):
        K.kda_w4_pack(z((4, 32), dtype=U8), z((5, 2)))
    with pytest.raises(ValueError, match="do not divide"):
        K.kda_w4_pack(z((4, 32), dtype=U8), z((4, 3)))
    with pytest.raises(TypeError, match="codes must be"):
        K.kda_w4_pack(z((4, 32), dtype=torch.int8), z((4, 2)))
    with pytest.raises(TypeError, match="unsupported dtype"):
        K.kda_w4_pack(z((4, 32), dtype=U8), z((4, 2), dtype=torch.float16))
    with pytest.raises(ValueError, match="zeros must have shape"):
        K.kda_w4_pack(z((4, 32), dtype=U8), z((4, 2)), z((4, 1), dtype=U8))

    x, r, wt, y = z((2, 64)), z((2, 64)), z(64), z((2, 64))
    with pytest.raises(TypeError, match="post_weight"):
        K.kda_sandwich_rmsnorm(x, z(64, dtype=BF), r, r, wt, y)
    with pytest.raises(ValueError, match="gate_activation"):
        K.kda_sandwich_rmsnorm(x, wt, r, r, wt, y, gate_activation="silu")
    with pytest.raises(ValueError, match="gate must have shape"):
        K.kda_sandwich_rmsnorm(x, wt, r, r, wt, y, gate=z(32))
    with pytest.raises(ValueError, match="gate must have shape"):
        K.kda_sandwich_rmsnorm(x, wt, r, r, wt, y, gate=z((2, 1)))
    with pytest.raises(TypeError, match="residual_out"):
        K.kda_sandwich_rmsnorm(x, wt, r, r.to(BF), wt, y)
    with pytest.raises(ValueError, match="residual must have shape"):
        K.kda_sandwich_rmsnorm(x, wt, z((3, 64)), None, wt, y)

    s, p = z((2, 3)), z((2, 3), dtype=I32)
    for bad in (dict(logits=z((5, 10))), dict(next_scores=z((3, 2))), dict(scores=z(6)), dict(finished=z((2, 2), dtype=torch.bool)),
                dict(logits=z((10, 6)).t())):
        a = dict(logits=z((6, 10)), scores=s, next_scores=s, parents=p, tokens=p)
        a.update(bad)
        with pytest.raises(ValueError):
            K.kda_beam_select(**a)
    for bad in (dict(parents=p.long()), dict(tokens=p.float()), dict(scores=s.double()), dict(finished=z((2, 3), dtype=U8)),
                dict(next_finished=z((2, 3), dtype=I32))):
        a = dict(logits=z((6, 10)), scores=s, next_scores=s, parents=p, tokens=p)
        a.update(bad)
        with pytest.raises(TypeError):
            K.kda_beam_select(**a)
    with pytest.raises(ValueError, match="workspace"):
        K.kda_beam_select(z((6, 10)), s, s, p, p, workspace="none")

    with pytest.raises(ValueError, match="state must be"):
        K.kda_beam_reorder(p, z((5, 8)))
    with pytest.raises(ValueError, match="state must be"):
        K.kda_beam_reorder(p, z((8, 6)).t())
    with pytest.raises(ValueError, match="conv_states must be"):
        K.kda_beam_reorder(p, z((6, 8)), z((6, 3)))
    with pytest.raises(TypeError, match="parents"):
        K.kda_beam_reorder(p.long(), z((6, 8)))


def test_sizes_kept_of_past_calls_are_bounded():
    """A server's batches come in many sizes: what the binding keeps of them has an end."""
    for B in range(1, 400):
        assert K._beam_bytes(B, 4, 1000 + B) == K.kda_beam_select_workspace_bytes(B, 4, 1000 + B)
    assert K._beam_bytes.cache_info().currsize <= 64


def test_norms_around_a_block_need_a_residual():
    x, w = torch.zeros((2, 64)), torch.zeros(64)
    with pytest.raises(ValueError, match="residual"):
        K.kda_sandwich_rmsnorm(x, w, None, None, w, torch.zeros((2, 64)))
