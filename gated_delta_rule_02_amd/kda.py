"""Thin Python binding of the C ABI in ``include/kda.h`` (ctypes).

Each function has the name of the C entry point it calls and only marshals
arguments: torch tensors become device pointers and sizes, the current HIP
stream is passed through, and a non-OK status raises ``KDAError`` with the
library's message. All computation happens in ``libkda.so``; if the library is
not built, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkda.so")

KDA_F32, KDA_BF16 = 0, 1
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "sigmoid": 4}
KDA_OK, KDA_ERR_INVALID_ARG, KDA_ERR_UNSUPPORTED, KDA_ERR_WORKSPACE, KDA_ERR_HIP = 0, -1, -2, -3, -4

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_F = ctypes.c_float
_SZ = ctypes.c_size_t

_SIGS = {
    "kda_prefill": (_I, [_P] * 5 + [_I, _I64, _I, _I, _I, _P, _P, _I, _F, _F, _P, _P, _P, _I, _P, _SZ, _P]),
    "kda_prefill_workspace_bytes": (_SZ, [_I64, _I, _I, _I, _I, _I]),
    "kda_prefill_noalloc": (_I, [_P] * 5 + [_I, _I64, _I, _I, _I, _P, _P, _I, _F, _F, _P, _P, _P, _I, _P]),
    "kda_prefill_gated": (_I, [_P] * 4 + [_I64, _P, _I64, _P, _I, _I64, _I, _I, _I, _P, _P, _I, _F, _F, _P, _P,
                                          _P, _I, _P, _SZ, _P]),
    "kda_prefill_noalloc_scratch_bytes": (_SZ, []),
    "kda_prefill_snapshots": (_I, [_P] * 5 + [_I, _I64, _I, _I, _I, _P, _P, _I, _F, _F, _P, _P, _P, _I, _P, _SZ,
                                              _I64, _I64, _P, _P]),
    "kda_prefill_segment_maps": (_I, [_P] * 4 + [_I, _I64, _I, _I, _I, _P, _P, _I, _F, _P, _P, _P, _SZ, _P]),
    "kda_affine_apply": (_I, [_P, _P, _P, _P, _I64, _I, _I, _P]),
    "kda_decode_step": (_I, [_P] * 5 + [_I, _I, _I, _I, _I, _F, _F, _P, _P, _I, _P]),
    "kda_decode_multi": (_I, [_P] * 5 + [_I, _I, _I, _I, _I, _I, _F, _F, _P, _P, _I, _P, _I, _P]),
    "kda_decode_commit": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _I, _P]),
    "kda_state_convert": (_I, [_P, _I, _P, _I, _I64, _P]),
    "kda_gemv_fp8": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _I, _I64, _I64, _I, _I, _P]),
    "kda_output_norm_gate_fp8": (_I, [_P, _I, _P, _I64, _I, _P, _I64, _I, _I, _F, _P, _P, _P]),
    "kda_quantize_fp8": (_I, [_P, _I64, _I, _I64, _I64, _P, _I64, _P, _I64, _P]),
    "kda_gemm_fp8": (_I, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _I64, _I64, _I64, _I, _P]),
    "kda_conv_state_update": (_I, [_P, _I64, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _P]),
    "kda_conv_prefill": (_I, [_P, _I64, _I64, _I, _I, _P, _P, _I, _P, _P, _P, _P, _I, _I, _F, _P, _I64, _I, _P]),
    "kda_gate_prologue": (_I, [_P, _I64, _P, _I64, _P, _I64, _I, _I, _F, _I, _P, _P, _I, _P]),
    "kda_output_norm_gate": (_I, [_P, _I, _P, _I64, _P, _I64, _I, _I, _F, _P, _I, _P]),
    "kda_gemm": (_I, [_P, _I64, _P, _I64, _P, _I64, _I64, _I64, _I64, _I, _I, _P]),
    "kda_decode_tree": (_I, [_P] * 5 + [_I, _P, _I, _I, _I, _I, _I, _F, _F, _P, _I, _P, _I, _P, _P]),
    "kda_decode_tree_commit": (_I, [_P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P, _I, _P]),
    "kda_conv_tree": (_I, [_P, _I64, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P]),
    "kda_conv_tree_commit": (_I, [_P, _I64, _P, _P, _I, _I, _I, _I, _I, _P, _P]),
    "kda_add_rmsnorm": (_I, [_P, _I64, _I, _P, _I64, _P, _I64, _I, _P, _I64, _I64, _F, _P, _I64, _I, _P]),
    "kda_add_rmsnorm_fp8": (_I, [_P, _I64, _I, _P, _I64, _P, _I64, _I, _P, _I64, _I64, _F, _P, _I64, _P, _I64, _P]),
    "kda_gemm_epilogue": (_I, [_P, _I64, _P, _I64, _P, _I, _P, _I64, _I, _P, _I64, _I64, _I64, _I64, _I, _I, _P]),
    "kda_state_bytes": (_SZ, [_I, _I, _I, _I]),
    "kda_conv_state_bytes": (_SZ, [_I, _I, _I, _I]),
    "kda_last_error": (ctypes.c_char_p, []),
    "kda_version": (_I, []),
}
EXPORTED = tuple(_SIGS)

_lib = None


class KDAError(RuntimeError):
    def __init__(self, name, status, message):
        super().__init__("%s failed with status %d: %s" % (name, status, message))
        self.status = status


def lib():
    """Load libkda.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libkda.so is not built (expected at %s); run __graft_entry__.build()" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _call(name, *args):
    rc = getattr(lib(), name)(*args)
    if rc != KDA_OK:
        raise KDAError(name, rc, lib().kda_last_error().decode())
    return rc


def _dt(t):
    if t.dtype == torch.float32:
        return KDA_F32
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    raise TypeError("unsupported dtype %s (float32 or bfloat16 expected)" % t.dtype)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on a GPU device")
    return t.data_ptr()


def _dense(t, name):
    if t is not None and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _cu(cu_seqlens, cu_seqlens_host):
    if cu_seqlens is None:
        return None, None, None
    if cu_seqlens.dtype != torch.int32:
        raise TypeError("cu_seqlens must be int32")
    host = cu_seqlens_host
    if host is None:
        host = cu_seqlens.cpu()  # one device->host copy when no mirror is given
    host = host.to(torch.int32).contiguous()
    return _ptr(_dense(cu_seqlens, "cu_seqlens")), host.data_ptr(), host


# --------------------------------------------------------------------------
_workspaces = {}


def _workspace(device, nbytes):
    """A cached device buffer of at least nbytes (one per device; grows on demand)."""
    key = torch.device(device).index
    buf = _workspaces.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _workspaces[key] = buf
    return buf


def kda_prefill(q, k, v, g, beta, o, cu_seqlens=None, cu_seqlens_host=None, num_seqs=None,
                initial_state=None, final_state=None, scale=1.0, lower_bound=-5.0,
                workspace="auto", stream=None, snapshots=None, snapshot_interval=None):
    """KDA core over packed sequences. q,k,g [T,H,128], v [T,H,128], beta [T,H]
    (one dtype), o [T,H,128] (float32 or bfloat16), states float32 [N,H,128,128].

    workspace: "auto" (a cached buffer of kda_prefill_workspace_bytes bytes, so
    bfloat16 inputs take the two-pass form), None (no workspace: single-pass
    form), or a caller-owned uint8 device tensor. Calls sharing the cached
    buffer must be ordered on one stream.

    snapshots: float32 [N, slots, H, 128, 128] with snapshot_interval (a
    multiple of 64): calls kda_prefill_snapshots, which also stores the state
    after every snapshot_interval tokens of each sequence."""
    for n_, t_ in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("o", o),
                   ("initial_state", initial_state), ("final_state", final_state), ("snapshots", snapshots)):
        _dense(t_, n_)
    T, H, dk = q.shape
    dv = v.shape[2]
    cu_dev, cu_host, keep = _cu(cu_seqlens, cu_seqlens_host)
    if num_seqs is None:
        num_seqs = (keep.numel() - 1) if keep is not None else 1
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a tensor")
        need = lib().kda_prefill_workspace_bytes(T, num_seqs, H, dk, dv, _dt(q))
        workspace = _workspace(q.device, need) if need else None
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if snapshots is None:
        _call("kda_prefill", _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _dt(q), T, H, dk, dv,
              cu_dev, cu_host, num_seqs, scale, lower_bound, _ptr(initial_state), _ptr(final_state),
              _ptr(o), _dt(o), _ptr(workspace), ws_bytes, _stream(stream))
    else:
        if snapshot_interval is None or snapshots.dim() != 5:
            raise ValueError("snapshots [N, slots, H, 128, 128] needs a snapshot_interval")
        _call("kda_prefill_snapshots", _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _dt(q), T, H, dk, dv,
              cu_dev, cu_host, num_seqs, scale, lower_bound, _ptr(initial_state), _ptr(final_state),
              _ptr(o), _dt(o), _ptr(workspace), ws_bytes, int(snapshot_interval), snapshots.shape[1],
              _ptr(snapshots), _stream(stream))
    return o


def kda_prefill_gated(q, k, v, f, b, A_log, o, cu_seqlens=None, cu_seqlens_host=None, num_seqs=None,
                      initial_state=None, final_state=None, scale=1.0, lower_bound=-5.0, workspace="auto",
                      stream=None):
    """kda_prefill with the gate prologue inside it: f rows [T, >=H*128] and
    b rows [T, >=H] (bfloat16, contiguous rows, any row stride), A_log float32
    [H] in place of g and beta. Results equal kda_gate_prologue followed by
    kda_prefill. bfloat16 q, k, v and a workspace ("auto" or a tensor)."""
    for n_, t_ in (("q", q), ("k", k), ("v", v), ("A_log", A_log), ("o", o),
                   ("initial_state", initial_state), ("final_state", final_state)):
        _dense(t_, n_)
    if f.stride(-1) != 1 or b.stride(-1) != 1:
        raise ValueError("f and b rows must be contiguous")
    T, H, dk = q.shape
    dv = v.shape[2]
    cu_dev, cu_host, keep = _cu(cu_seqlens, cu_seqlens_host)
    if num_seqs is None:
        num_seqs = (keep.numel() - 1) if keep is not None else 1
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto' or a tensor")
        need = lib().kda_prefill_workspace_bytes(T, num_seqs, H, dk, dv, _dt(q))
        workspace = _workspace(q.device, need) if need else None
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _call("kda_prefill_gated", _ptr(q), _ptr(k), _ptr(v), _ptr(f), f.stride(0), _ptr(b), b.stride(0),
          _ptr(A_log), _dt(q), T, H, dk, dv, cu_dev, cu_host, num_seqs, scale, lower_bound,
          _ptr(initial_state), _ptr(final_state), _ptr(o), _dt(o), _ptr(workspace), ws_bytes, _stream(stream))
    return o


def kda_prefill_noalloc(q, k, v, g, beta, o, cu_seqlens=None, cu_seqlens_host=None, num_seqs=None,
                        initial_state=None, final_state=None, scale=1.0, lower_bound=-5.0, stream=None):
    """kda_prefill with the library's device-resident scratch in place of a
    workspace (allocates nothing). Arguments as kda_prefill."""
    for n_, t_ in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("o", o),
                   ("initial_state", initial_state), ("final_state", final_state)):
        _dense(t_, n_)
    T, H, dk = q.shape
    dv = v.shape[2]
    cu_dev, cu_host, keep = _cu(cu_seqlens, cu_seqlens_host)
    if num_seqs is None:
        num_seqs = (keep.numel() - 1) if keep is not None else 1
    _call("kda_prefill_noalloc", _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _dt(q), T, H, dk, dv,
          cu_dev, cu_host, num_seqs, scale, lower_bound, _ptr(initial_state), _ptr(final_state),
          _ptr(o), _dt(o), _stream(stream))
    return o


def kda_prefill_noalloc_scratch_bytes():
    return lib().kda_prefill_noalloc_scratch_bytes()


def kda_prefill_workspace_bytes(num_tokens, num_seqs, H, dk=128, dv=128, in_dtype=KDA_BF16):
    return lib().kda_prefill_workspace_bytes(num_tokens, num_seqs, H, dk, dv, in_dtype)


def kda_prefill_segment_maps(k, v, g, beta, M_out, N_out, cu_seqlens=None, cu_seqlens_host=None, num_seqs=None,
                             lower_bound=-5.0, workspace="auto", stream=None):
    """Affine map S_out = M S_in + N of every segment (sequence of cu_seqlens).
    k, g [T,H,128], v [T,H,128], beta [T,H] bfloat16; M_out, N_out float32
    [N,H,128,128]. workspace as for kda_prefill (required: "auto" or a tensor)."""
    for n_, t_ in (("k", k), ("v", v), ("g", g), ("beta", beta), ("M_out", M_out), ("N_out", N_out)):
        _dense(t_, n_)
    T, H, dk = k.shape
    dv = v.shape[2]
    cu_dev, cu_host, keep = _cu(cu_seqlens, cu_seqlens_host)
    if num_seqs is None:
        num_seqs = (keep.numel() - 1) if keep is not None else 1
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto' or a tensor")
        workspace = _workspace(k.device, max(lib().kda_prefill_workspace_bytes(max(T, 1), num_seqs, H, dk, dv, _dt(k)), 16))
    ws_bytes = workspace.numel() * workspace.element_size()
    _call("kda_prefill_segment_maps", _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _dt(k), T, H, dk, dv,
          cu_dev, cu_host, num_seqs, lower_bound, _ptr(M_out), _ptr(N_out), _ptr(workspace), ws_bytes,
          _stream(stream))
    return M_out, N_out


def kda_affine_apply(M, X, Y, N=None, stream=None):
    """Y = M X (+ N) for float32 [..., 128, 128] batches (segment maps applied
    to states, or composed)."""
    for n_, t_ in (("M", M), ("X", X), ("Y", Y), ("N", N)):
        _dense(t_, n_)
    count = M.numel() // (128 * 128)
    if X.numel() != M.numel() or Y.numel() != M.numel() or (N is not None and N.numel() != M.numel()):
        raise ValueError("M, X, N and Y must hold the same number of 128 x 128 matrices")
    _call("kda_affine_apply", _ptr(M), _ptr(X), _ptr(N), _ptr(Y), count, 128, 128, _stream(stream))
    return Y


def kda_decode_step(q, k, v, g, beta, state, o, scale=1.0, lower_bound=-5.0, stream=None):
    """One token per sequence. q,k,g,v [B,H,128], beta [B,H]; state float32
    [B,H,128,128] updated in place; o [B,H,128]."""
    for n_, t_ in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("state", state), ("o", o)):
        _dense(t_, n_)
    B, H, dk = q.shape
    dv = v.shape[2]
    _call("kda_decode_step", _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _dt(q), B, H, dk, dv,
          scale, lower_bound, _ptr(state), _ptr(o), _dt(o), _stream(stream))
    return o


def kda_decode_multi(q, k, v, g, beta, state, o, token_states=None, scale=1.0, lower_bound=-5.0, stream=None):
    """Several tokens per sequence. q,k,g,v [B,Tq,H,128], beta [B,Tq,H]; state
    [B,H,128,128] in float32 or bfloat16 (its dtype is the state dtype); o
    [B,Tq,H,128]. token_states None: state becomes the state after the last
    token; else token_states [B,Tq,H,128,128] (the state's dtype) receives the
    state after every token and state is only read."""
    for n_, t_ in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("state", state), ("o", o),
                   ("token_states", token_states)):
        _dense(t_, n_)
    if token_states is not None and token_states.dtype != state.dtype:
        raise TypeError("token_states must have the state's dtype")
    B, Tq, H, dk = q.shape
    dv = v.shape[3]
    _call("kda_decode_multi", _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _dt(q), B, Tq, H, dk, dv,
          scale, lower_bound, _ptr(state), _ptr(token_states), _dt(state), _ptr(o), _dt(o), _stream(stream))
    return o


def kda_decode_commit(token_states, accepted, state, stream=None):
    """state[b] <- token_states[b, accepted[b] - 1] where 1 <= accepted[b] <= Tq
    (accepted: int32 [B] on the device; states float32 or bfloat16)."""
    for n_, t_ in (("token_states", token_states), ("accepted", accepted), ("state", state)):
        _dense(t_, n_)
    if accepted.dtype != torch.int32:
        raise TypeError("accepted must be int32")
    if token_states.dtype != state.dtype:
        raise TypeError("token_states and state must have one dtype")
    B, Tq, H, dk, dv = token_states.shape
    _call("kda_decode_commit", _ptr(token_states), _ptr(accepted), B, Tq, H, dk, dv, _ptr(state), _dt(state),
          _stream(stream))
    return state


def kda_state_convert(src, dst, stream=None):
    """dst <- src converted between float32 and bfloat16 (same number of elements)."""
    _dense(src, "src")
    _dense(dst, "dst")
    if src.numel() != dst.numel():
        raise ValueError("src and dst must have the same number of elements")
    _call("kda_state_convert", _ptr(src), _dt(src), _ptr(dst), _dt(dst), src.numel(), _stream(stream))
    return dst


def kda_conv_state_update(x, conv_state, weight, y, bias=None, apply_silu=True, l2norm_group=0,
                          l2norm_eps=1e-6, stream=None):
    """x rows [B, >=C] (row stride x.stride(0)), conv_state [B,W-1,C] (in place),
    weight [C,W], y [B,C]."""
    for n_, t_ in (("conv_state", conv_state), ("weight", weight), ("y", y), ("bias", bias)):
        _dense(t_, n_)
    if x.stride(1) != 1:
        raise ValueError("x rows must be contiguous")
    B = x.shape[0]
    C, W = weight.shape
    _call("kda_conv_state_update", _ptr(x), x.stride(0), _ptr(conv_state), _ptr(weight), _ptr(bias), _dt(x), B, C, W,
          int(bool(apply_silu)), l2norm_group, l2norm_eps, _ptr(y), _stream(stream))
    return y


def kda_conv_prefill(x, weight, y, cu_seqlens=None, cu_seqlens_host=None, num_seqs=None, bias=None,
                     conv_state_in=None, conv_state_out=None, apply_silu=True, l2norm_group=0,
                     l2norm_eps=1e-6, stream=None):
    """x rows [T, >=C] (row stride x.stride(0)), weight [C,W], y rows [T, >=C]."""
    for n_, t_ in (("weight", weight), ("bias", bias), ("conv_state_in", conv_state_in),
                   ("conv_state_out", conv_state_out)):
        _dense(t_, n_)
    if x.stride(1) != 1 or y.stride(1) != 1:
        raise ValueError("x and y rows must be contiguous")
    T = x.shape[0]
    C, W = weight.shape
    cu_dev, cu_host, keep = _cu(cu_seqlens, cu_seqlens_host)
    if num_seqs is None:
        num_seqs = (keep.numel() - 1) if keep is not None else 1
    _call("kda_conv_prefill", _ptr(x), x.stride(0), T, C, W, cu_dev, cu_host, num_seqs, _ptr(weight),
          _ptr(bias), _ptr(conv_state_in), _ptr(conv_state_out), int(bool(apply_silu)), l2norm_group,
          l2norm_eps, _ptr(y), y.stride(0), _dt(x), _stream(stream))
    return y


def kda_gate_prologue(f, b, A_log, g_out, beta_out, H, dk=128, lower_bound=-5.0, stream=None):
    """f rows [T, >=H*dk], b rows [T, >=H], A_log float32 [H]; g_out [T,H,dk], beta_out [T,H]."""
    _dense(A_log, "A_log"); _dense(g_out, "g_out"); _dense(beta_out, "beta_out")
    if f.stride(-1) != 1 or b.stride(-1) != 1:
        raise ValueError("f and b rows must be contiguous")
    T = f.shape[0]
    _call("kda_gate_prologue", _ptr(f), f.stride(0), _ptr(b), b.stride(0), _ptr(A_log), T, H, dk,
          lower_bound, _dt(f), _ptr(g_out), _ptr(beta_out), _dt(g_out), _stream(stream))
    return g_out, beta_out


def kda_output_norm_gate(o, gate, norm_weight, y, eps=1e-6, stream=None):
    """o [T,H,dv], gate rows [T, >=H*dv] (dtype of y), norm_weight float32 [dv], y [T,H*dv]."""
    _dense(o, "o"); _dense(norm_weight, "norm_weight"); _dense(y, "y")
    if gate.stride(-1) != 1:
        raise ValueError("gate rows must be contiguous")
    T, H, dv = o.shape
    _call("kda_output_norm_gate", _ptr(o), _dt(o), _ptr(gate), gate.stride(0), _ptr(norm_weight), T, H,
          dv, eps, _ptr(y), _dt(y), _stream(stream))
    return y


def kda_gemm(A, B, C, stream=None):
    """C[M,N] = A[M,K] B[N,K]^T (rows may be strided; last dims contiguous)."""
    for n_, t_ in (("A", A), ("B", B), ("C", C)):
        if t_.stride(-1) != 1:
            raise ValueError("%s rows must be contiguous" % n_)
    M, K = A.shape
    N = B.shape[0]
    _call("kda_gemm", _ptr(A), A.stride(0), _ptr(B), B.stride(0), _ptr(C), C.stride(0), M, N, K,
          _dt(A), _dt(C), _stream(stream))
    return C


def kda_gemv_fp8(x, w, w_scale, y, stream=None):
    """y[M,N] = x[M,K] W^T, W = e4m3(w) (uint8 [N,K]) x w_scale[N/128, K/128]
    blocks; x bf16, 1 <= M <= 8 (row strides allowed, last dims contiguous)."""
    for n_, t_ in (("x", x), ("w", w), ("w_scale", w_scale), ("y", y)):
        if t_.stride(-1) != 1:
            raise ValueError("%s rows must be contiguous" % n_)
    if w.dtype != torch.uint8 or w_scale.dtype != torch.float32:
        raise TypeError("w must be uint8 E4M3 codes and w_scale float32")
    M, Kd = x.shape
    N = w.shape[0]
    _call("kda_gemv_fp8", _ptr(x), x.stride(0), _ptr(w), w.stride(0), _ptr(w_scale), w_scale.stride(0),
          _ptr(y), y.stride(0), M, N, Kd, _dt(x), _dt(y), _stream(stream))
    return y


def kda_quantize_fp8(x, codes, scales, stream=None):
    """x [M,K] float32/bfloat16 -> codes uint8 [M,K] (E4M3), scales float32 [M,K/128]
    (row strides allowed, last dims contiguous)."""
    for n_, t_ in (("x", x), ("codes", codes), ("scales", scales)):
        if t_.stride(-1) != 1:
            raise ValueError("%s rows must be contiguous" % n_)
    if codes.dtype != torch.uint8 or scales.dtype != torch.float32:
        raise TypeError("codes must be uint8 and scales float32")
    M, Kd = x.shape
    _call("kda_quantize_fp8", _ptr(x), x.stride(0), _dt(x), M, Kd, _ptr(codes), codes.stride(0), _ptr(scales),
          scales.stride(0), _stream(stream))
    return codes, scales


def kda_gemm_fp8(x, x_scale, w, w_scale, y, stream=None):
    """y[M,N] = X W^T with X = e4m3(x) x x_scale[M, K/128] and W = e4m3(w) x
    w_scale[N/128, K/128] (x, w uint8 codes; row strides allowed)."""
    for n_, t_ in (("x", x), ("x_scale", x_scale), ("w", w), ("w_scale", w_scale), ("y", y)):
        if t_.stride(-1) != 1:
            raise ValueError("%s rows must be contiguous" % n_)
    if x.dtype != torch.uint8 or w.dtype != torch.uint8:
        raise TypeError("x and w must be uint8 E4M3 codes")
    if x_scale.dtype != torch.float32 or w_scale.dtype != torch.float32:
        raise TypeError("scales must be float32")
    M, Kd = x.shape
    N = w.shape[0]
    _call("kda_gemm_fp8", _ptr(x), x.stride(0), _ptr(x_scale), x_scale.stride(0), _ptr(w), w.stride(0),
          _ptr(w_scale), w_scale.stride(0), _ptr(y), y.stride(0), M, N, Kd, _dt(y), _stream(stream))
    return y


def kda_output_norm_gate_fp8(o, gate, norm_weight, y_codes, y_scales, eps=1e-6, stream=None):
    """o [T,H,128]; gate rows [T, >=H*128]; y_codes uint8 [T, H*128]; y_scales float32 [T, H]."""
    for n_, t_ in (("o", o), ("norm_weight", norm_weight), ("y_codes", y_codes), ("y_scales", y_scales)):
        _dense(t_, n_)
    if gate.stride(1) != 1:
        raise ValueError("gate rows must be contiguous")
    T, H, dv = o.shape
    _call("kda_output_norm_gate_fp8", _ptr(o), _dt(o), _ptr(gate), gate.stride(0), _dt(gate), _ptr(norm_weight),
          T, H, dv, eps, _ptr(y_codes), _ptr(y_scales), _stream(stream))
    return y_codes, y_scales


def _rows(name, t, shape, dtype=None):
    """Checks a row-strided 2-D tensor: shape, contiguous rows, dtype (if given)."""
    if t is None:
        return None
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple(shape), tuple(t.shape)))
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError("%s rows must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s" % (name, dtype))
    return t


def _ld(t):
    """Row stride of a 2-D tensor (a single row's stride means nothing: its width, rounded up)."""
    return t.stride(0) if t.shape[0] > 1 else (t.shape[1] + 15) // 16 * 16


def _call_on(name, tensors, stream, *args):
    """_call with the tensors' device current and, without a stream, that
    device's current stream; tensors on several devices are refused."""
    device = tensors[0].device
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError("%s: tensors on several devices (%s, %s)" % (name, device, t.device))
    if device.index == torch.cuda.current_device():
        return _call(name, *args, _stream(stream))
    with torch.cuda.device(device):
        return _call(name, *args, _stream(stream))


def _tensor(name, t, shape, dtype=None):
    """Checks a dense tensor: shape, contiguous, dtype (if given)."""
    if t is None:
        return None
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple(shape), tuple(t.shape)))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s" % (name, dtype))
    return _dense(t, name)


def kda_decode_tree(q, k, v, g, beta, parents, state, o, writes=None, scale=1.0, lower_bound=-5.0, stream=None):
    """Verify a tree of drafts per sequence. q,k,g,v [B,N,H,128], beta [B,N,H] (one
    dtype), parents int32 [B,N] (-1 the state, or a node before; anything else
    marks an absent node), state [B,H,128,128] (float32 or bfloat16, read only), o
    [B,N,H,128]; writes float32 [B,N,H,128] or None, for kda_decode_tree_commit."""
    if q.dim() != 4:
        raise ValueError("q must be [B, N, H, 128]")
    B, N, H, dk = q.shape
    for n_, t_, s_ in (("q", q, q.shape), ("k", k, q.shape), ("v", v, (B, N, H, v.shape[-1])), ("g", g, q.shape),
                       ("beta", beta, (B, N, H))):
        _tensor(n_, t_, s_, q.dtype)
    dv = v.shape[-1]
    _tensor("parents", parents, (B, N), torch.int32)
    _tensor("state", state, (B, H, dk, dv))
    _tensor("o", o, (B, N, H, dv))
    _tensor("writes", writes, (B, N, H, dv), torch.float32)
    _call_on("kda_decode_tree", (q, k, v, g, beta, parents, state, o, writes), stream, _ptr(q), _ptr(k), _ptr(v),
             _ptr(g), _ptr(beta), _dt(q), _ptr(parents), B, N, H, dk, dv, scale, lower_bound, _ptr(state), _dt(state),
             _ptr(o), _dt(o), _ptr(writes))
    return o


def kda_decode_tree_commit(k, g, writes, parents, accepted, state, lower_bound=-5.0, stream=None):
    """state[b] <- the state after node accepted[b] (int32 [B], device) of the tree
    that kda_decode_tree verified with these k, g and parents, and that gave
    writes; any other value of accepted leaves state[b] as it is."""
    if k.dim() != 4:
        raise ValueError("k must be [B, N, H, 128]")
    B, N, H, dk = k.shape
    dv = writes.shape[-1]
    _tensor("k", k, k.shape)
    _tensor("g", g, k.shape, k.dtype)
    _tensor("writes", writes, (B, N, H, dv), torch.float32)
    _tensor("parents", parents, (B, N), torch.int32)
    _tensor("accepted", accepted, (B,), torch.int32)
    _tensor("state", state, (B, H, dk, dv))
    _call_on("kda_decode_tree_commit", (k, g, writes, parents, accepted, state), stream, _ptr(k), _ptr(g), _dt(k),
             _ptr(writes), _ptr(parents), _ptr(accepted), B, N, H, dk, dv, lower_bound, _ptr(state), _dt(state))
    return state


def _conv_tree_sizes(x, conv_state, parents):
    B, N = parents.shape
    W, C = conv_state.shape[1] + 1, conv_state.shape[2]
    _rows("x", x, (B * N, C))
    _tensor("conv_state", conv_state, (B, W - 1, C), x.dtype)
    _tensor("parents", parents, (B, N), torch.int32)
    return B, N, C, W


def kda_conv_tree(x, conv_state, parents, weight, y, bias=None, apply_silu=True, l2norm_group=0, l2norm_eps=1e-6,
                  stream=None):
    """The prologue convolution over trees of drafts: x rows [B*N, C] (row strides
    allowed), conv_state [B,W-1,C] (read only), parents int32 [B,N] (as
    kda_decode_tree), weight [C,W], y [B*N,C]."""
    B, N, C, W = _conv_tree_sizes(x, conv_state, parents)
    _tensor("weight", weight, (C, W), x.dtype)
    _tensor("bias", bias, (C,), x.dtype)
    _tensor("y", y, (B * N, C), x.dtype)
    _call_on("kda_conv_tree", (x, conv_state, parents, weight, y, bias), stream, _ptr(x), _ld(x), _ptr(conv_state),
             _ptr(parents), _ptr(weight), _ptr(bias), _dt(x), B, N, C, W, int(bool(apply_silu)), l2norm_group,
             l2norm_eps, _ptr(y))
    return y


def kda_conv_tree_commit(x, parents, accepted, conv_state, stream=None):
    """conv_state[b] <- the last W-1 inputs of itself followed by the path to node
    accepted[b] of the tree (x, parents as for kda_conv_tree), in place."""
    B, N, C, W = _conv_tree_sizes(x, conv_state, parents)
    _tensor("accepted", accepted, (B,), torch.int32)
    _call_on("kda_conv_tree_commit", (x, parents, accepted, conv_state), stream, _ptr(x), _ld(x), _ptr(parents),
             _ptr(accepted), _dt(x), B, N, C, W, _ptr(conv_state))
    return conv_state


def _add_rmsnorm_args(x, norm_weight, residual, residual_out):
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    _rows("x", x, x.shape)
    _rows("residual", residual, x.shape)
    _rows("residual_out", residual_out, x.shape, None if residual is None else residual.dtype)
    if norm_weight.dtype != torch.float32 or tuple(norm_weight.shape) != (x.shape[1],):
        raise TypeError("norm_weight must be float32 [K]")
    r, ro = residual, residual_out
    return (_ptr(x), _ld(x), _dt(x), _ptr(r), 0 if r is None else _ld(r), _ptr(ro), 0 if ro is None else _ld(ro),
            KDA_F32 if r is None else _dt(r), _ptr(_dense(norm_weight, "norm_weight")), x.shape[0], x.shape[1])


def kda_add_rmsnorm(x, norm_weight, y, residual=None, residual_out=None, eps=1e-6, stream=None):
    """y = RMSNorm(x + residual) * norm_weight, residual_out = x + residual. x, residual,
    y [M, K] (row strides allowed; float32 or bfloat16 each), norm_weight float32
    [K]; residual_out (the residual's dtype) may be residual itself."""
    args = _add_rmsnorm_args(x, norm_weight, residual, residual_out)
    _rows("y", y, x.shape)
    _call_on("kda_add_rmsnorm", (x, norm_weight, y, residual, residual_out), stream, *args, eps, _ptr(y), _ld(y), _dt(y))
    return y


def kda_add_rmsnorm_fp8(x, norm_weight, codes, scales, residual=None, residual_out=None, eps=1e-6, stream=None):
    """kda_add_rmsnorm with y quantized as kda_quantize_fp8 does: codes uint8
    [M, K] (E4M3), scales float32 [M, K/128]; K a multiple of 128."""
    args = _add_rmsnorm_args(x, norm_weight, residual, residual_out)
    _rows("codes", codes, x.shape, torch.uint8)
    _rows("scales", scales, (x.shape[0], x.shape[1] // 128), torch.float32)
    _call_on("kda_add_rmsnorm_fp8", (x, norm_weight, codes, scales, residual, residual_out), stream, *args, eps,
             _ptr(codes), _ld(codes), _ptr(scales), _ld(scales))
    return codes, scales


def kda_gemm_epilogue(A, B, C, bias=None, activation="none", residual=None, stream=None):
    """C[M,N] = act(A[M,K] B[N,K]^T + bias) + residual (bfloat16 A and B; C and the
    residual float32 or bfloat16; rows may be strided). bias float32 [N];
    activation one of ACTIVATIONS; residual may be C itself."""
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A must be [M, K] and B [N, K]")
    if activation not in ACTIVATIONS:
        raise ValueError("activation must be one of %s (got %r)" % (sorted(ACTIVATIONS), activation))
    M, K = A.shape
    N = B.shape[0]
    _rows("A", A, (M, K))
    _rows("B", B, (N, K), A.dtype)
    _rows("C", C, (M, N))
    _rows("residual", residual, (M, N))
    if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (N,)):
        raise TypeError("bias must be float32 [N]")
    r = residual
    _call_on("kda_gemm_epilogue", (A, B, C, bias, residual), stream, _ptr(A), _ld(A), _ptr(B), _ld(B),
             _ptr(_dense(bias, "bias")), ACTIVATIONS[activation], _ptr(r), 0 if r is None else _ld(r),
             KDA_F32 if r is None else _dt(r), _ptr(C), _ld(C), M, N, K, _dt(A), _dt(C))
    return C


def kda_state_bytes(H, dk=128, dv=128, dtype=KDA_F32):
    return lib().kda_state_bytes(H, dk, dv, dtype)


def kda_conv_state_bytes(streams, W, C, dtype=KDA_BF16):
    return lib().kda_conv_state_bytes(streams, W, C, dtype)


def kda_last_error():
    return lib().kda_last_error().decode()


def kda_version():
    return lib().kda_version()
