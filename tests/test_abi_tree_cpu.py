"""Host-side validation of the draft-tree entry points: every rejected call is
refused before anything reaches the device. No GPU is needed."""
import pytest
import torch

from gated_delta_rule_02_amd import kda as K
from tests.test_abi_cpu import call, fake

INVALID, UNSUPPORTED = K.KDA_ERR_INVALID_ARG, K.KDA_ERR_UNSUPPORTED
BIG = fake(20)


def tree(**over):
    a = dict(q=fake(1), k=fake(2), v=fake(3), g=fake(4), beta=fake(5), xd=K.KDA_BF16, par=fake(6), B=3, N=8, H=4, dk=128,
             dv=128, scale=1.0, lb=-5.0, s=fake(7), sd=K.KDA_F32, o=fake(8), od=K.KDA_F32, w=fake(9))
    a.update(over)
    return call("kda_decode_tree", a["q"], a["k"], a["v"], a["g"], a["beta"], a["xd"], a["par"], a["B"], a["N"], a["H"],
                a["dk"], a["dv"], a["scale"], a["lb"], a["s"], a["sd"], a["o"], a["od"], a["w"], None)[0]


def test_decode_tree_validation():
    for name in ("q", "k", "v", "g", "beta", "s", "o"):
        assert tree(**{name: None}) == INVALID, name
        assert tree(**{name: BIG + 8}) == INVALID, name
    assert tree(w=BIG + 4) == INVALID and tree(par=None) == INVALID and tree(par=BIG + 2) == INVALID
    for name in ("B", "N", "H"):
        assert tree(**{name: 0}) == INVALID, name
    assert tree(N=65) == UNSUPPORTED and tree(dk=64) == UNSUPPORTED and tree(dv=256) == UNSUPPORTED
    assert tree(B=1 << 30, H=4) == INVALID and tree(B=1, N=64, H=1 << 18) == INVALID
    assert tree(xd=2) == INVALID and tree(sd=-1) == INVALID and tree(od=7) == INVALID
    assert tree(lb=0.5) == INVALID and tree(lb=float("nan")) == INVALID
    for name in ("q", "k", "v", "g", "beta", "s", "par"):
        at = dict(q=fake(1), k=fake(2), v=fake(3), g=fake(4), beta=fake(5), s=fake(7), par=fake(6))[name]
        assert tree(o=at) == INVALID and tree(w=at) == INVALID, name
    assert tree(w=fake(8) + 1024) == INVALID


def commit(**over):
    a = dict(k=fake(2), g=fake(4), xd=K.KDA_BF16, w=fake(9), par=fake(6), acc=fake(10), B=3, N=8, H=4, dk=128, dv=128,
             lb=-5.0, s=fake(7), sd=K.KDA_F32)
    a.update(over)
    return call("kda_decode_tree_commit", a["k"], a["g"], a["xd"], a["w"], a["par"], a["acc"], a["B"], a["N"], a["H"],
                a["dk"], a["dv"], a["lb"], a["s"], a["sd"], None)[0]


def test_decode_tree_commit_validation():
    for name in ("k", "g", "w", "s"):
        assert commit(**{name: None}) == INVALID, name
        assert commit(**{name: BIG + 8}) == INVALID, name
    for name in ("par", "acc"):
        assert commit(**{name: None}) == INVALID and commit(**{name: BIG + 1}) == INVALID, name
    for name in ("B", "N", "H"):
        assert commit(**{name: 0}) == INVALID, name
    assert commit(N=65) == UNSUPPORTED and commit(dk=64) == UNSUPPORTED
    assert commit(xd=2) == INVALID and commit(sd=3) == INVALID and commit(lb=1.0) == INVALID
    for at in (fake(2), fake(4), fake(9), fake(6), fake(10)):
        assert commit(s=at) == INVALID


def conv(**over):
    a = dict(x=fake(1), ld=520, s=fake(2), par=fake(3), w=fake(4), b=fake(5), d=K.KDA_BF16, B=3, N=8, C=512, W=4, silu=1,
             l2=128, eps=1e-6, y=fake(6))
    a.update(over)
    return call("kda_conv_tree", a["x"], a["ld"], a["s"], a["par"], a["w"], a["b"], a["d"], a["B"], a["N"], a["C"], a["W"],
                a["silu"], a["l2"], a["eps"], a["y"], None)[0]


def conv_commit(**over):
    a = dict(x=fake(1), ld=520, par=fake(3), acc=fake(4), d=K.KDA_BF16, B=3, N=8, C=512, W=4, s=fake(2))
    a.update(over)
    return call("kda_conv_tree_commit", a["x"], a["ld"], a["par"], a["acc"], a["d"], a["B"], a["N"], a["C"], a["W"],
                a["s"], None)[0]


@pytest.mark.parametrize("fn", [conv, conv_commit])
def test_conv_tree_common_validation(fn):
    for name in ("x", "s", "par"):
        assert fn(**{name: None}) == INVALID and fn(**{name: BIG + 2}) == INVALID, name
    for name in ("B", "N"):
        assert fn(**{name: 0}) == INVALID, name
    assert fn(B=1 << 24, N=1) == UNSUPPORTED
    assert fn(N=65) == UNSUPPORTED and fn(C=0) == UNSUPPORTED and fn(C=192) == UNSUPPORTED
    assert fn(W=1) == UNSUPPORTED and fn(W=9) == UNSUPPORTED and fn(d=4) == INVALID
    assert fn(ld=504) == INVALID and fn(ld=516) == INVALID


def test_conv_tree_validation():
    for name in ("w", "y"):
        assert conv(**{name: None}) == INVALID and conv(**{name: BIG + 8}) == INVALID, name
    assert conv(b=BIG + 8) == INVALID and conv(l2=64) == UNSUPPORTED
    for at in (fake(1), fake(2), fake(3), fake(4), fake(5)):
        assert conv(y=at) == INVALID
    assert conv_commit(acc=None) == INVALID and conv_commit(acc=BIG + 2) == INVALID
    for at in (fake(1), fake(3), fake(4)):
        assert conv_commit(s=at) == INVALID


def test_tree_binding_refuses():
    B, N, H = 2, 5, 3
    q = torch.zeros(B, N, H, 128)
    beta, state, o = torch.zeros(B, N, H), torch.zeros(B, H, 128, 128), torch.zeros(B, N, H, 128)
    par, acc = torch.zeros(B, N, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    ok = (q, q, q, q, beta, par, state, o)

    def but(i, t):
        return ok[:i] + (t,) + ok[i + 1:]

    with pytest.raises(ValueError, match="GPU"):
        K.kda_decode_tree(*ok)
    with pytest.raises(TypeError, match="parents"):
        K.kda_decode_tree(*but(5, par.long()))
    with pytest.raises(ValueError, match="parents"):
        K.kda_decode_tree(*but(5, par[:, :4]))
    with pytest.raises(TypeError, match="k"):
        K.kda_decode_tree(*but(1, q.bfloat16()))
    with pytest.raises(ValueError, match="state"):
        K.kda_decode_tree(*but(6, state[:1]))
    with pytest.raises(ValueError, match="contiguous"):
        K.kda_decode_tree(*but(7, torch.zeros(N, B, H, 128).transpose(0, 1)))
    with pytest.raises(TypeError, match="writes"):
        K.kda_decode_tree(*ok, torch.zeros(B, N, H, 128, dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="accepted"):
        K.kda_decode_tree_commit(q, q, q, par, acc.long(), state)
    hist, w, y = torch.zeros(B, 3, 256), torch.zeros(256, 4), torch.zeros(B * N, 256)
    with pytest.raises(ValueError, match="x must"):
        K.kda_conv_tree(torch.zeros(B * N, 128), hist, par, w, y)
    with pytest.raises(ValueError, match="weight"):
        K.kda_conv_tree(torch.zeros(B * N, 256), hist, par, w[:, :3], y)
    with pytest.raises(ValueError, match="GPU"):
        K.kda_conv_tree_commit(torch.zeros(B * N, 256), par, acc, hist)


def far(i):
    """Addresses that do not overlap whatever these sizes take."""
    return i << 50


def test_tree_counts_beyond_a_launch():
    """A launch holds less than 2^32 threads: a workgroup of 256 (512 above 32
    nodes; 1,024 for the commit of a float32 state) for every sequence and head."""
    a = dict(q=far(1), k=far(2), v=far(3), g=far(4), beta=far(5), par=far(6), s=far(7), o=far(8), w=far(9), H=64)
    for N, most in ((1, 1 << 24), (32, 1 << 24), (33, 1 << 23), (64, 1 << 23)):
        assert tree(B=most // 64, N=N, **a) == UNSUPPORTED, N
        # one sequence fewer passes this check (the next, of the alignment of o, refuses it)
        assert tree(B=most // 64 - 1, N=N, **dict(a, o=far(8) + 8)) == INVALID, N
    a = dict(k=far(2), g=far(4), w=far(9), par=far(6), acc=far(10), s=far(7), H=64)
    for sd, most in ((K.KDA_F32, 1 << 22), (K.KDA_BF16, 1 << 24)):
        assert commit(B=most // 64, N=1, sd=sd, **a) == UNSUPPORTED, sd
        assert commit(B=most // 64 - 1, N=1, sd=sd, **dict(a, s=far(7) + 8)) == INVALID, sd


@pytest.mark.parametrize("b", [1, 3])
def test_conv_tree_binding_refuses_histories_of_another_batch(b):
    """conv_state of fewer (or more) sequences than the trees, dense and of the
    right type: the C entries take B from parents and would run past it."""
    B, N, C = 2, 5, 256
    x, y, w = torch.zeros(B * N, C), torch.zeros(B * N, C), torch.zeros(C, 4)
    par, acc = torch.zeros(B, N, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    hist = torch.zeros(b, 3, C)
    with pytest.raises(ValueError, match="conv_state must have shape"):
        K.kda_conv_tree(x, hist, par, w, y)
    with pytest.raises(ValueError, match="conv_state must have shape"):
        K.kda_conv_tree_commit(x, par, acc, hist)
