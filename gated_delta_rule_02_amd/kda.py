"""Thin Python binding of the C ABI in ``include/kda.h`` (ctypes).

Each function has the name of the C entry point it calls and only marshals
arguments: torch tensors become device pointers and sizes, the current HIP
stream is passed through, and a non-OK status raises ``KDAError`` with the
library's message. All computation happens in ``libkda.so``; if the library is
not built, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
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
    "kda_sandwich_rmsnorm": (_I, [_P, _I64, _I, _P, _F, _P, _I64, _I, _I, _P, _I64, _P, _I64, _I, _F, _F, _P, _I64, _I64,
                                  _F, _P, _I64, _I, _P]),
    "kda_sandwich_rmsnorm_fp8": (_I, [_P, _I64, _I, _P, _F, _P, _I64, _I, _I, _P, _I64, _P, _I64, _I, _F, _F, _P, _I64,
                                      _I64, _F, _P, _I64, _P, _I64, _P]),
    "kda_w4_packed_bytes": (_SZ, [_I64, _I64, _I, _I, _I]),
    "kda_w4_pack": (_I, [_P, _I64, _P, _I64, _I, _P, _I64, _I64, _I64, _I, _P, _SZ, _P]),
    "kda_w4_expand": (_I, [_P, _I64, _I64, _I, _I, _I, _P, _I64, _P]),
    "kda_gemm_w4": (_I, [_P, _I64, _I, _P, _I, _I, _I, _P, _I64, _I, _P, _I64, _I, _I64, _I64, _I64, _P]),
    "kda_beam_select_workspace_bytes": (_SZ, [_I, _I, _I64]),
    "kda_beam_select": (_I, [_P, _I64, _I, _P, _P, _I, _I, _I64, _I64, _P, _P, _P, _P, _P, _SZ, _P]),
    "kda_beam_reorder": (_I, [_P, _I, _I, _P, _SZ, _P, _I, _SZ, _P]),
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


def _holds(name, t, dtype, n):
    """t (None: not given) is of this dtype and holds what the call reads or writes."""
    if t is not None:
        if t.dtype != dtype:
            raise TypeError("%s must be %s (got %s)" % (name, dtype, t.dtype))
        if t.numel() < n:
            raise ValueError("%s holds %d elements, the call takes %d" % (name, t.numel(), n))


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


def _workspace(device, nbytes, stream=None):
    """A device buffer of at least nbytes for a call on this stream (None: the
    current one): one kept per device and stream (grows on demand); in a captured
    call the graph's own (a kept one would be freed under its replays when it grows)."""
    if stream is not None:
        with torch.cuda.stream(stream):  # the allocator reuses a buffer in this stream's order
            return _workspace(device, nbytes)
    key = (torch.device(device).index, torch.cuda.current_stream().cuda_stream)
    if key[1] and torch.cuda.is_current_stream_capturing():  # (nothing is captured on the default stream, 0)
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    buf = _workspaces.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _workspaces[key] = buf
    return buf


def _workspace_on(t, nbytes, stream):
    """_workspace on t's device (made current for it), for the calls through _call_on."""
    index = t.get_device()
    if index < 0:
        raise ValueError("tensor must be on a GPU device")
    if stream is None and index == torch._C._cuda_getDevice():
        raw = torch._C._cuda_getCurrentRawStream(index)
        buf = _workspaces.get((index, raw))
        if buf is not None and buf.numel() >= nbytes and not (raw and torch.cuda.is_current_stream_capturing()):
            return buf
    with torch.cuda.device(index):
        return _workspace(t.device, nbytes, stream)


def kda_prefill(q, k, v, g, beta, o, cu_seqlens=None, cu_seqlens_host=None, num_seqs=None,
                initial_state=None, final_state=None, scale=1.0, lower_bound=-5.0,
                workspace="auto", stream=None, snapshots=None, snapshot_interval=None):
    """KDA core over packed sequences. q,k,g [T,H,128], v [T,H,128], beta [T,H]
    (one dtype), o [T,H,128] (float32 or bfloat16), states float32 [N,H,128,128].

    workspace: "auto" (a buffer of at least kda_prefill_workspace_bytes bytes, kept
    per stream, so bfloat16 inputs take the two-pass form), None (no workspace:
    single-pass form), or a caller-owned uint8 device tensor (calls that share it
    must be ordered on one stream).

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
    _holds("initial_state", initial_state, torch.float32, num_seqs * H * dk * dv)
    _holds("final_state", final_state, torch.float32, num_seqs * H * dk * dv)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a tensor")
        need = lib().kda_prefill_workspace_bytes(T, num_seqs, H, dk, dv, _dt(q))
        workspace = _workspace(q.device, need, stream) if need else None
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
    _holds("initial_state", initial_state, torch.float32, num_seqs * H * dk * dv)
    _holds("final_state", final_state, torch.float32, num_seqs * H * dk * dv)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto' or a tensor")
        need = lib().kda_prefill_workspace_bytes(T, num_seqs, H, dk, dv, _dt(q))
        workspace = _workspace(q.device, need, stream) if need else None
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
    _holds("initial_state", initial_state, torch.float32, num_seqs * H * dk * dv)
    _holds("final_state", final_state, torch.float32, num_seqs * H * dk * dv)
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
        need = lib().kda_prefill_workspace_bytes(max(T, 1), num_seqs, H, dk, dv, _dt(k))
        workspace = _workspace(k.device, max(need, 16), stream)
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
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and g.is_contiguous() and
            beta.is_contiguous() and state.is_contiguous() and o.is_contiguous()):
        for n_, t_ in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("state", state), ("o", o)):
            _dense(t_, n_)
    B, H, dk = q.shape
    dv = v.shape[2]
    if state.dtype is not torch.float32 or state.numel() < B * H * dk * dv:
        _holds("state", state, torch.float32, B * H * dk * dv)
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
    if not (conv_state.is_contiguous() and weight.is_contiguous() and y.is_contiguous()) or bias is not None:
        for n_, t_ in (("conv_state", conv_state), ("weight", weight), ("y", y), ("bias", bias)):
            _dense(t_, n_)
    if x.stride(1) != 1:
        raise ValueError("x rows must be contiguous")
    B = x.shape[0]
    C, W = weight.shape
    if conv_state.dtype is not x.dtype or conv_state.numel() < B * (W - 1) * C:
        _holds("conv_state", conv_state, x.dtype, B * (W - 1) * C)
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
    _holds("conv_state_in", conv_state_in, x.dtype, num_seqs * (W - 1) * C)
    _holds("conv_state_out", conv_state_out, x.dtype, num_seqs * (W - 1) * C)
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


# --------------------------------------------------------------------------
# The calls below are made once per token of a decode step, where their host
# time counts as much as the kernels': each tests all that has to hold in one
# expression and goes through the checks that name the fault only where it does not;
# the raw stream and the bound function are taken directly.
_DTYPES = {torch.float32: KDA_F32, torch.bfloat16: KDA_BF16}
_fns = {}


def _code(t, name):
    c = _DTYPES.get(t.dtype)
    if c is None:
        raise TypeError("%s: unsupported dtype %s (float32 or bfloat16 expected)" % (name, t.dtype))
    return c


def _mat(name, t, shape):
    """Row stride of a [rows, columns] tensor of this shape with contiguous rows
    (a single row's stride means nothing: its width, rounded up)."""
    if t.shape != shape:
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple(shape), tuple(t.shape)))
    ld, one = t.stride()
    if one != 1 and shape[1] != 1:
        raise ValueError("%s rows must be contiguous" % name)
    return ld if shape[0] != 1 else (shape[1] + 15) // 16 * 16


def _ld(name, t, shape):
    """_mat of a tensor that is dense as a rule."""
    return shape[1] if t.is_contiguous() and t.shape == shape else _mat(name, t, shape)


def _tensor(name, t, shape):
    """A dense tensor of this shape."""
    if t.shape != shape:
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _type(name, t, dtype):
    if t.dtype is not dtype:
        raise TypeError("%s must be %s (got %s)" % (name, dtype, t.dtype))


def _call_on(name, tensors, stream, *args):
    """_call on the device that holds all of the tensors (None left out), made
    current for the call; without a stream on that device's current one."""
    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != index:
            break
    else:
        t = tensors[0] if index < 0 else None
    if t is not None:
        raise ValueError("%s: all tensors must be on one GPU device (got %s and %s)" % (name, tensors[0].device, t.device))
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(lib(), name)
    raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if index == torch._C._cuda_getDevice():
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, raw)
    if rc != KDA_OK:
        raise KDAError(name, rc, lib().kda_last_error().decode())


def kda_decode_tree(q, k, v, g, beta, parents, state, o, writes=None, scale=1.0, lower_bound=-5.0, stream=None):
    """Verify a tree of drafts per sequence. q,k,g,v [B,N,H,128], beta [B,N,H] (one
    dtype), parents int32 [B,N] (-1 the state, or a node before; anything else
    marks an absent node), state [B,H,128,128] (float32 or bfloat16, read only), o
    [B,N,H,128]; writes float32 [B,N,H,128] or None, for kda_decode_tree_commit."""
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must be [B, N, H, 128]")
    B, N, H, dk = shape
    dv = v.shape[-1]
    vshape, xd = (B, N, H, dv), q.dtype
    if not (k.shape == shape and g.shape == shape and v.shape == vshape and beta.shape == (B, N, H) and
            parents.shape == (B, N) and state.shape == (B, H, dk, dv) and o.shape == vshape and
            k.dtype is xd and g.dtype is xd and v.dtype is xd and beta.dtype is xd and parents.dtype is torch.int32 and
            q.is_contiguous() and k.is_contiguous() and g.is_contiguous() and v.is_contiguous() and
            beta.is_contiguous() and parents.is_contiguous() and state.is_contiguous() and o.is_contiguous()):
        _tensor("q", q, shape), _tensor("k", k, shape), _tensor("g", g, shape), _tensor("v", v, vshape)
        _tensor("beta", beta, (B, N, H)), _tensor("parents", parents, (B, N)), _tensor("state", state, (B, H, dk, dv))
        _tensor("o", o, vshape)
        _type("k", k, xd), _type("g", g, xd), _type("v", v, xd), _type("beta", beta, xd)
        _type("parents", parents, torch.int32)
    if writes is not None:
        _tensor("writes", writes, vshape), _type("writes", writes, torch.float32)
    _call_on("kda_decode_tree", (q, k, v, g, beta, parents, state, o, writes), stream, q.data_ptr(), k.data_ptr(),
             v.data_ptr(), g.data_ptr(), beta.data_ptr(), _code(q, "q"), parents.data_ptr(), B, N, H, dk, dv, scale,
             lower_bound, state.data_ptr(), _code(state, "state"), o.data_ptr(), _code(o, "o"),
             None if writes is None else writes.data_ptr())
    return o


def kda_decode_tree_commit(k, g, writes, parents, accepted, state, lower_bound=-5.0, stream=None):
    """state[b] <- the state after node accepted[b] (int32 [B], device) of the tree
    that kda_decode_tree verified with these k, g and parents, and that gave
    writes; any other value of accepted leaves state[b] as it is."""
    shape = k.shape
    if len(shape) != 4:
        raise ValueError("k must be [B, N, H, 128]")
    B, N, H, dk = shape
    dv = writes.shape[-1]
    if not (g.shape == shape and writes.shape == (B, N, H, dv) and parents.shape == (B, N) and accepted.shape == (B,) and
            state.shape == (B, H, dk, dv) and g.dtype is k.dtype and writes.dtype is torch.float32 and
            parents.dtype is torch.int32 and accepted.dtype is torch.int32 and
            k.is_contiguous() and g.is_contiguous() and writes.is_contiguous() and parents.is_contiguous() and
            accepted.is_contiguous() and state.is_contiguous()):
        _tensor("k", k, shape), _tensor("g", g, shape), _tensor("writes", writes, (B, N, H, dv))
        _tensor("parents", parents, (B, N)), _tensor("accepted", accepted, (B,)), _tensor("state", state, (B, H, dk, dv))
        _type("g", g, k.dtype), _type("writes", writes, torch.float32)
        _type("parents", parents, torch.int32), _type("accepted", accepted, torch.int32)
    _call_on("kda_decode_tree_commit", (k, g, writes, parents, accepted, state), stream, k.data_ptr(), g.data_ptr(),
             _code(k, "k"), writes.data_ptr(), parents.data_ptr(), accepted.data_ptr(), B, N, H, dk, dv, lower_bound,
             state.data_ptr(), _code(state, "state"))
    return state


def _conv_tree_sizes(x, conv_state, parents):
    B, N = parents.shape
    b, w1, C = conv_state.shape
    if not (b == B and conv_state.dtype is x.dtype and parents.dtype is torch.int32 and conv_state.is_contiguous() and
            parents.is_contiguous()):
        _tensor("conv_state", conv_state, (B, w1, C)), _tensor("parents", parents, (B, N))
        _type("conv_state", conv_state, x.dtype), _type("parents", parents, torch.int32)
    return _mat("x", x, (B * N, C)), B, N, C, w1 + 1


def kda_conv_tree(x, conv_state, parents, weight, y, bias=None, apply_silu=True, l2norm_group=0, l2norm_eps=1e-6,
                  stream=None):
    """The prologue convolution over trees of drafts: x rows [B*N, C] (row strides
    allowed), conv_state [B,W-1,C] (read only), parents int32 [B,N] (as
    kda_decode_tree), weight [C,W], y [B*N,C]."""
    ld, B, N, C, W = _conv_tree_sizes(x, conv_state, parents)
    if not (weight.shape == (C, W) and y.shape == (B * N, C) and weight.dtype is x.dtype and y.dtype is x.dtype and
            weight.is_contiguous() and y.is_contiguous()):
        _tensor("weight", weight, (C, W)), _tensor("y", y, (B * N, C))
        _type("weight", weight, x.dtype), _type("y", y, x.dtype)
    if bias is not None:
        _tensor("bias", bias, (C,)), _type("bias", bias, x.dtype)
    _call_on("kda_conv_tree", (x, conv_state, parents, weight, y, bias), stream, x.data_ptr(), ld, conv_state.data_ptr(),
             parents.data_ptr(), weight.data_ptr(), None if bias is None else bias.data_ptr(), _code(x, "x"), B, N, C, W,
             1 if apply_silu else 0, l2norm_group, l2norm_eps, y.data_ptr())
    return y


def kda_conv_tree_commit(x, parents, accepted, conv_state, stream=None):
    """conv_state[b] <- the last W-1 inputs of itself followed by the path to node
    accepted[b] of the tree (x, parents as for kda_conv_tree), in place."""
    ld, B, N, C, W = _conv_tree_sizes(x, conv_state, parents)
    if not (accepted.shape == (B,) and accepted.dtype is torch.int32 and accepted.is_contiguous()):
        _tensor("accepted", accepted, (B,)), _type("accepted", accepted, torch.int32)
    _call_on("kda_conv_tree_commit", (x, parents, accepted, conv_state), stream, x.data_ptr(), ld, parents.data_ptr(),
             accepted.data_ptr(), _code(x, "x"), B, N, C, W, conv_state.data_ptr())
    return conv_state


def _add_rmsnorm_args(x, norm_weight, residual, residual_out):
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must be [M, K]")
    if norm_weight.shape != shape[1:] or norm_weight.dtype is not torch.float32 or not norm_weight.is_contiguous():
        raise TypeError("norm_weight must be dense float32 [K]")
    r = ro = None
    r_ld = ro_ld = 0
    rd = KDA_F32
    if residual is not None:
        r, r_ld, rd = residual.data_ptr(), _mat("residual", residual, shape), _code(residual, "residual")
        if residual_out is not None:
            _type("residual_out", residual_out, residual.dtype)
            ro, ro_ld = residual_out.data_ptr(), _mat("residual_out", residual_out, shape)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    return (x.data_ptr(), _mat("x", x, shape), _code(x, "x"), r, r_ld, ro, ro_ld, rd, norm_weight.data_ptr(), shape[0],
            shape[1])


def kda_add_rmsnorm(x, norm_weight, y, residual=None, residual_out=None, eps=1e-6, stream=None):
    """y = RMSNorm(x + residual) * norm_weight, residual_out = x + residual. x, residual,
    y [M, K] (row strides allowed; float32 or bfloat16 each), norm_weight float32
    [K]; residual_out (the residual's dtype) may be residual itself."""
    args = _add_rmsnorm_args(x, norm_weight, residual, residual_out)
    _call_on("kda_add_rmsnorm", (x, norm_weight, y, residual, residual_out), stream, *args, eps, y.data_ptr(),
             _mat("y", y, x.shape), _code(y, "y"))
    return y


def kda_add_rmsnorm_fp8(x, norm_weight, codes, scales, residual=None, residual_out=None, eps=1e-6, stream=None):
    """kda_add_rmsnorm with y quantized as kda_quantize_fp8 does: codes uint8
    [M, K] (E4M3), scales float32 [M, K/128]; K a multiple of 128."""
    args = _add_rmsnorm_args(x, norm_weight, residual, residual_out)
    _type("codes", codes, torch.uint8), _type("scales", scales, torch.float32)
    M, K = x.shape
    _call_on("kda_add_rmsnorm_fp8", (x, norm_weight, codes, scales, residual, residual_out), stream, *args, eps,
             codes.data_ptr(), _mat("codes", codes, x.shape), scales.data_ptr(), _mat("scales", scales, (M, K // 128)))
    return codes, scales


def kda_gemm_epilogue(A, B, C, bias=None, activation="none", residual=None, stream=None):
    """C[M,N] = act(A[M,K] B[N,K]^T + bias) + residual (bfloat16 A and B; C and the
    residual float32 or bfloat16; rows may be strided). bias float32 [N];
    activation one of ACTIVATIONS; residual may be C itself."""
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError("activation must be one of %s (got %r)" % (sorted(ACTIVATIONS), activation))
    ashape, bshape = A.shape, B.shape
    if len(ashape) != 2 or len(bshape) != 2 or ashape[1] != bshape[1]:
        raise ValueError("A must be [M, K] and B [N, K] (got %s, %s)" % (tuple(ashape), tuple(bshape)))
    M, K = ashape
    N = bshape[0]
    shape = (M, N)
    _type("B", B, A.dtype)
    pb = pr = None
    ldr, rd = 0, KDA_F32
    if bias is not None:
        _tensor("bias", bias, bshape[:1]), _type("bias", bias, torch.float32)
        pb = bias.data_ptr()
    if residual is not None:
        pr, ldr, rd = residual.data_ptr(), _mat("residual", residual, shape), _code(residual, "residual")
    _call_on("kda_gemm_epilogue", (A, B, C, bias, residual), stream, A.data_ptr(), _mat("A", A, ashape), B.data_ptr(),
             _mat("B", B, bshape), pb, act, pr, ldr, rd, C.data_ptr(), _mat("C", C, shape), M, N, K, _code(A, "A"),
             _code(C, "C"))
    return C


def _sandwich_args(x, post_weight, residual, residual_out, norm_weight, gate, gate_activation, residual_scale,
                   branch_scale, post_eps, eps):
    shape = x.shape
    if len(shape) != 2 or residual is None:
        raise ValueError("x must be [M, K], and residual given")
    M, K = shape
    act, rd, wshape = ACTIVATIONS.get(gate_activation), residual.dtype, shape[1:]
    dense = (x.is_contiguous() and residual.is_contiguous() and residual.shape == shape and
             (residual_out is residual or residual_out is not None and residual_out.is_contiguous() and
              residual_out.shape == shape and residual_out.dtype is rd))
    if not ((act == 0 or act == 4) and post_weight.shape == wshape and norm_weight.shape == wshape and
            post_weight.dtype is torch.float32 and norm_weight.dtype is torch.float32 and post_weight.is_contiguous() and
            norm_weight.is_contiguous()):
        for name, w in (("post_weight", post_weight), ("norm_weight", norm_weight)):
            if w.shape != wshape or w.dtype is not torch.float32 or not w.is_contiguous():
                raise TypeError("%s must be dense float32 [K]" % name)
        raise ValueError("gate_activation must be 'none' or 'sigmoid' (got %r)" % (gate_activation,))
    pg, g_ld, gd = None, 0, KDA_F32
    if gate is not None:
        pg, gd = gate.data_ptr(), _code(gate, "gate")
        if gate.dim() == 1:
            _tensor("gate", gate, wshape)
        else:
            g_ld = _mat("gate", gate, shape)
    x_ld = r_ld = ro_ld = K
    if not dense:
        x_ld, r_ld = _mat("x", x, shape), _mat("residual", residual, shape)
        if residual_out is not None:
            _type("residual_out", residual_out, rd)
            ro_ld = _mat("residual_out", residual_out, shape)
    return (x.data_ptr(), x_ld, _code(x, "x"), post_weight.data_ptr(), post_eps, pg, g_ld, gd, act, residual.data_ptr(),
            r_ld, None if residual_out is None else residual_out.data_ptr(), ro_ld, _code(residual, "residual"),
            residual_scale, branch_scale, norm_weight.data_ptr(), M, K, eps)


def kda_sandwich_rmsnorm(x, post_weight, residual, residual_out, norm_weight, y, gate=None, gate_activation="none",
                         residual_scale=1.0, branch_scale=1.0, post_eps=1e-6, eps=1e-6, stream=None):
    """h = residual_scale * residual + branch_scale * act(gate) * RMSNorm(x) * post_weight,
    residual_out = h, y = RMSNorm(h) * norm_weight. x, residual, y [M, K] (row strides
    allowed; float32 or bfloat16 each), the weights float32 [K]; gate [M, K] rows or
    one [K] for all (float32 or bfloat16), through 'none' or 'sigmoid'; residual_out
    (the residual's dtype, or None) may be residual itself."""
    args = _sandwich_args(x, post_weight, residual, residual_out, norm_weight, gate, gate_activation, residual_scale,
                          branch_scale, post_eps, eps)
    _call_on("kda_sandwich_rmsnorm", (x, post_weight, residual, residual_out, norm_weight, y, gate), stream, *args,
             y.data_ptr(), _ld("y", y, x.shape), _code(y, "y"))
    return y


def kda_sandwich_rmsnorm_fp8(x, post_weight, residual, residual_out, norm_weight, codes, scales, gate=None,
                             gate_activation="none", residual_scale=1.0, branch_scale=1.0, post_eps=1e-6, eps=1e-6,
                             stream=None):
    """kda_sandwich_rmsnorm with y quantized as kda_quantize_fp8 does: codes uint8
    [M, K] (E4M3), scales float32 [M, K/128]; K a multiple of 128."""
    args = _sandwich_args(x, post_weight, residual, residual_out, norm_weight, gate, gate_activation, residual_scale,
                          branch_scale, post_eps, eps)
    _type("codes", codes, torch.uint8), _type("scales", scales, torch.float32)
    M, K = shape = x.shape
    _call_on("kda_sandwich_rmsnorm_fp8", (x, post_weight, residual, residual_out, norm_weight, codes, scales, gate), stream,
             *args, codes.data_ptr(), _ld("codes", codes, shape), scales.data_ptr(), _ld("scales", scales, (M, K // 128)))
    return codes, scales


class W4Weight:
    """A packed 4-bit weight [N, K] (kda_w4_pack): one uint8 buffer with its codes,
    scales and zero points, in the layout that kda_gemm_w4 streams."""

    __slots__ = ("packed", "N", "K", "group", "scale_code", "has_zeros")

    def __init__(self, packed, N, K, group, scale_code, has_zeros):
        self.packed, self.N, self.K, self.group = packed, N, K, group
        self.scale_code, self.has_zeros = scale_code, has_zeros

    @property
    def shape(self):
        return torch.Size((self.N, self.K))

    def get_device(self):
        return self.packed.get_device()


def kda_w4_packed_bytes(N, K, group, scale_dtype=KDA_F32, has_zeros=False):
    return lib().kda_w4_packed_bytes(N, K, group, scale_dtype, int(bool(has_zeros)))


def kda_w4_pack(codes, scales, zeros=None, stream=None):
    """W[n,k] = scales[n, k/group] * (code[n,k] - zeros[n, k/group]) laid out for kda_gemm_w4
    -> W4Weight. codes uint8 [N, K/2] (the even column in the low four bits),
    scales [N, K/group] float32 or bfloat16, zeros uint8 [N, K/group] (None: 8). Once per
    weight; the inputs are not kept. Row strides allowed."""
    if codes.dim() != 2 or scales.dim() != 2 or scales.shape[0] != codes.shape[0] or scales.shape[1] < 1:
        raise ValueError("codes must be [N, K/2] and scales [N, K/group] (got %s, %s)" %
                         (tuple(codes.shape), tuple(scales.shape)))
    _type("codes", codes, torch.uint8)
    N, K = codes.shape[0], 2 * codes.shape[1]
    group, rest = divmod(K, scales.shape[1])
    if rest:
        raise ValueError("%d scales a row do not divide %d columns" % (scales.shape[1], K))
    code = _code(scales, "scales")
    pz, ldz = None, 0
    if zeros is not None:
        _type("zeros", zeros, torch.uint8)
        pz, ldz = zeros.data_ptr(), _mat("zeros", zeros, scales.shape)
    if not codes.is_cuda:
        raise ValueError("tensor must be on a GPU device")
    nbytes = kda_w4_packed_bytes(N, K, group, code, zeros is not None)
    with torch.cuda.stream(stream) if stream is not None else torch.cuda.device(codes.device):
        packed = torch.empty(nbytes, dtype=torch.uint8, device=codes.device)
    _call_on("kda_w4_pack", (codes, scales, zeros, packed), stream, codes.data_ptr(), _mat("codes", codes, codes.shape),
             scales.data_ptr(), _mat("scales", scales, scales.shape), code, pz, ldz, N, K, group, packed.data_ptr(), nbytes)
    return W4Weight(packed, N, K, group, code, zeros is not None)


def kda_w4_expand(weight, out, stream=None):
    """out [N, K] <- the packed weight's values in bfloat16 (row strides allowed)."""
    _type("out", out, torch.bfloat16)
    _call_on("kda_w4_expand", (out, weight.packed), stream, weight.packed.data_ptr(), weight.N, weight.K, weight.group,
             weight.scale_code, int(weight.has_zeros), out.data_ptr(), _mat("out", out, (weight.N, weight.K)))
    return out


def kda_gemm_w4(x, weight, y, residual=None, stream=None):
    """y[M,N] = x[M,K] W^T (+ residual) from a W4Weight (bfloat16 x; y and the residual
    float32 or bfloat16; rows may be strided). residual may be y itself."""
    xshape = x.shape
    if len(xshape) != 2 or xshape[1] != weight.K:
        raise ValueError("x must be [M, %d] (got %s)" % (weight.K, tuple(xshape)))
    M, K = xshape
    N = weight.N
    shape = (M, N)
    pr, ldr, rd = None, 0, KDA_F32
    if residual is not None:
        pr, ldr, rd = residual.data_ptr(), _ld("residual", residual, shape), _code(residual, "residual")
    packed = weight.packed
    _call_on("kda_gemm_w4", (x, packed, y, residual), stream, x.data_ptr(), K if x.is_contiguous() else _mat("x", x, xshape),
             _code(x, "x"), packed.data_ptr(), weight.group, weight.scale_code, 1 if weight.has_zeros else 0, pr, ldr, rd,
             y.data_ptr(), _ld("y", y, shape), _code(y, "y"), M, N, K)
    return y


def kda_beam_select_workspace_bytes(B, W, V):
    return lib().kda_beam_select_workspace_bytes(B, W, V)


_beam_bytes = functools.lru_cache(maxsize=64)(kda_beam_select_workspace_bytes)


def kda_beam_select(logits, scores, next_scores, parents, tokens, finished=None, next_finished=None, eos=-1,
                    workspace="auto", stream=None):
    """The W best of every sequence's W beams x V tokens by scores + log softmax(logits),
    best first, ties to the lower beam, then token. logits [B*W, V] (float32 or
    bfloat16, rows may be strided), scores and next_scores float32 [B, W] (may be one
    tensor), parents (the beam followed) and tokens int32 [B, W]; finished and
    next_finished bool [B, W] or None: a beam that has ended goes on with token eos
    at its score. workspace: "auto" (kept per stream) or a uint8 tensor of
    kda_beam_select_workspace_bytes bytes."""
    if scores.dim() != 2:
        raise ValueError("scores must be [B, W]")
    shape = scores.shape
    B, W = shape
    n, V = logits.shape
    if n != B * W:
        raise ValueError("logits must be [%d, V] for scores [%d, %d] (got %s)" % (B * W, B, W, tuple(logits.shape)))
    if not (next_scores.shape == shape and parents.shape == shape and tokens.shape == shape and
            scores.dtype is torch.float32 and next_scores.dtype is torch.float32 and parents.dtype is torch.int32 and
            tokens.dtype is torch.int32 and scores.is_contiguous() and next_scores.is_contiguous() and
            parents.is_contiguous() and tokens.is_contiguous()):
        for name, t, dtype in (("scores", scores, torch.float32), ("next_scores", next_scores, torch.float32),
                               ("parents", parents, torch.int32), ("tokens", tokens, torch.int32)):
            _tensor(name, t, shape), _type(name, t, dtype)
    pf = pn = None
    if finished is not None:
        _tensor("finished", finished, shape), _type("finished", finished, torch.bool)
        pf = finished.data_ptr()
    if next_finished is not None:
        _tensor("next_finished", next_finished, shape), _type("next_finished", next_finished, torch.bool)
        pn = next_finished.data_ptr()
    ld = logits.stride(0) if n > 1 else V
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("logits rows must be contiguous")
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto' or a tensor")
        workspace = _workspace_on(logits, _beam_bytes(B, W, V), stream)
    pw, wbytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    _call_on("kda_beam_select", (logits, scores, next_scores, parents, tokens, finished, next_finished, workspace), stream,
             logits.data_ptr(), ld, _code(logits, "logits"), scores.data_ptr(), pf, B, W, V, eos, next_scores.data_ptr(),
             parents.data_ptr(), tokens.data_ptr(), pn, pw, wbytes)
    return next_scores, parents, tokens, next_finished


def kda_beam_reorder(parents, state, conv_states=None, stream=None):
    """state[b, w] <- state[b, parents[b, w]] in place, and likewise every stream of
    conv_states. parents int32 [B, W]; state [B*W, ...] and conv_states [streams, B*W,
    ...] dense, of any dtype. A parent that is no beam leaves its row as it is."""
    shape = parents.shape
    if len(shape) != 2:
        raise ValueError("parents must be [B, W]")
    B, W = shape
    rows = B * W
    if not (parents.dtype is torch.int32 and parents.is_contiguous()):
        _tensor("parents", parents, shape), _type("parents", parents, torch.int32)
    if not state.is_contiguous() or state.dim() < 1 or state.shape[0] != rows:
        raise ValueError("state must be dense [%d, ...] for parents [%d, %d] (got %s)" % (rows, B, W, tuple(state.shape)))
    pc, streams, cbytes = None, 0, 0
    if conv_states is not None:
        cshape = conv_states.shape
        if len(cshape) < 2 or cshape[1] != rows or not conv_states.is_contiguous():
            raise ValueError("conv_states must be dense [streams, %d, ...] (got %s)" % (rows, tuple(cshape)))
        pc, streams, cbytes = conv_states.data_ptr(), cshape[0], conv_states.nbytes
    if rows == 0:
        return state
    _call_on("kda_beam_reorder", (parents, state, conv_states), stream, parents.data_ptr(), B, W, state.data_ptr(),
             state.nbytes // rows, pc, streams, cbytes // (rows * (streams or 1)))
    return state


def kda_state_bytes(H, dk=128, dv=128, dtype=KDA_F32):
    return lib().kda_state_bytes(H, dk, dv, dtype)


def kda_conv_state_bytes(streams, W, C, dtype=KDA_BF16):
    return lib().kda_conv_state_bytes(streams, W, C, dtype)


def kda_last_error():
    return lib().kda_last_error().decode()


def kda_version():
    return lib().kda_version()
