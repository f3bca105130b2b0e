"""The whole KDA token mixer of one layer, composed from the C-ABI calls.

Data flow of "Ling-3.1-flash: Grouped Routing and Two Different MLA Caches"
(flozi.net), section "KDA replaces a token list with a recurrent matrix":
hidden [T, 4096] -> q, k, v projections of width 64 x 128, each through its own
causal width-4 convolution with SiLU, q and k normalised per head -> retention +
delta-rule write + read per head -> output normalisation x sigmoid gate ->
projection back to 4096. Decay and gate projections are full rank 4096 -> 8192
and beta comes from a per-head projection ("Ling-3.1-flash: a 560B
hybrid-attention MoE, counted from its safetensors headers", section "How KDA
and MLA split the work").

Every arithmetic step runs in libkda.so; this module only holds device
buffers and sequences the calls. The six input projections are packed into one
[5*H*128 + H (+ zero rows to a multiple of 8), hidden] weight so a single GEMM
produces q|k|v|f|gate|b.
"""
from __future__ import annotations

import threading

import numpy as np
import torch

from . import kda as K

D = 128

# The expansion of a 4-bit weight (a name for KDAMixer._buf): one buffer per device and
# stream for all mixers, which their products use one after the other; one of each
# mixer's own would hold a stack's weights in bfloat16 beside their four bits. The lock keeps
# an expansion and its product together where host threads share a stream.
EXPANDED = "expanded"
_expanded = {}
_expanding = threading.Lock()


def _dev_bf16(t):
    return torch.from_numpy(np.ascontiguousarray(t.bits).view(np.int16)).view(torch.bfloat16).cuda()


class KDAMixer:
    """The mixer with bfloat16 weights. Outputs (and a DraftTree) are buffers of the
    mixer, valid until the method's next call on the same stream, or, if the call
    was captured, until the graph's next replay."""

    def __init__(self, W_in, conv_q, conv_k, conv_v, A_log, norm_w, Wo, H, scale=1.0,
                 lower_bound=-5.0, l2_eps=1e-6, rms_eps=1e-6):
        self.W_in, self.Wo = W_in, Wo
        self.conv = (conv_q, conv_k, conv_v)
        self.A_log, self.norm_w = A_log, norm_w
        self.H = H
        self.W = H * D
        self.hidden = Wo.shape[0]
        self.scale, self.lower_bound, self.l2_eps, self.rms_eps = scale, lower_bound, l2_eps, rms_eps
        self._bufs = {}
        self._device = W_in.get_device()

    @classmethod
    def from_host(cls, d):
        """Build from the seeded host weights of ``synth.workload_layer``."""
        rows = [_dev_bf16(d[n]) for n in ("Wq", "Wk", "Wv", "Wf", "Wg", "Wb")]
        pad = (-sum(r.shape[0] for r in rows)) % 8  # keep packed rows 16-byte aligned
        if pad:
            rows.append(torch.zeros((pad, rows[0].shape[1]), dtype=torch.bfloat16, device="cuda"))
        W_in = torch.cat(rows, dim=0).contiguous()
        return cls(W_in, _dev_bf16(d["conv_q"]), _dev_bf16(d["conv_k"]), _dev_bf16(d["conv_v"]),
                   torch.from_numpy(d["A_log"]).cuda(), torch.from_numpy(d["norm_w"]).cuda(),
                   _dev_bf16(d["Wo"]), d["H"])

    def flops_per_token(self):
        core = 2 * 4468736  # per chunk-head of 64 tokens -> per token-head x 64 heads / 64 tokens
        rows = 5 * self.W + self.H
        return 2 * (rows * self.W_in.shape[1] + self.Wo.shape[0] * self.Wo.shape[1]) + core * self.H // 64

    def _buf(self, name, shape, dtype):
        """Scratch of this name, kept for the next call. Every stream has its own, so
        that calls on two streams share none; a captured call's belongs to its graph
        (the capture's memory pool): a later call of another size replaces a kept
        buffer and would free what the replays use."""
        stream = torch._C._cuda_getCurrentRawStream(self._device)
        if stream:  # (nothing can be captured on the default stream, 0)
            if torch.cuda.is_current_stream_capturing():
                return torch.empty(shape, dtype=dtype, device="cuda")
        if name is EXPANDED:
            n, key = shape.numel(), (self._device, stream)
            b = _expanded.get(key)
            if b is None or b.numel() < n:
                b = _expanded[key] = torch.empty(n, dtype=dtype, device=torch.device("cuda", self._device))
            return b[:n].view(shape)
        if stream:
            name = (name, stream)
        b = self._bufs.get(name)
        if b is None or b.shape != shape or b.dtype is not dtype:
            b = torch.empty(shape, dtype=dtype, device="cuda")
            self._bufs[name] = b
        return b

    def projections(self, x, tag=""):
        """P = x W_in^T (bf16): columns q | k | v | f | gate | b."""
        T = x.shape[0]
        P = self._buf(tag + "P", (T, self.W_in.shape[0]), torch.bfloat16)
        K.kda_gemm(x, self.W_in, P)
        return P, self._columns(P)

    def _columns(self, P):
        W = self.W
        return [P[:, i * W:(i + 1) * W] for i in range(5)] + [P[:, 5 * W:5 * W + self.H]]

    def projections_of_norm(self, x, residual, norm_weight, eps, tag, post=None):
        """The columns of RMSNorm(x + residual) norm_weight W_in^T (bf16); the
        residual (or None) is updated in place. With post (a BranchNorm) x joins the
        residual through it."""
        T, hidden = x.shape
        y = self._buf("ny", (T, hidden), torch.bfloat16)
        if post is None:
            K.kda_add_rmsnorm(x, norm_weight, y, residual=residual, residual_out=residual, eps=eps)
        else:
            K.kda_sandwich_rmsnorm(x, post.weight, residual, residual, norm_weight, y, eps=eps, **post.form)
        P = self._buf(tag + "nP", (T, self.W_in.shape[0]), torch.bfloat16)
        K.kda_gemm_epilogue(y, self.W_in, P)
        return self._columns(P)

    def output_into(self, o, gp, hidden, tag):
        """hidden += (RMSNorm(o) x w x sigmoid(gate)) W_o^T, in the product's epilogue."""
        y = self._buf(tag + "y", (o.shape[0], self.W), torch.bfloat16)
        K.kda_output_norm_gate(o, gp, self.norm_w, y, eps=self.rms_eps)
        K.kda_gemm_epilogue(y, self.Wo, hidden, residual=hidden)

    def output_branch(self, o, gp, tag):
        """output's result alone, through the product that has forms for few rows."""
        T = o.shape[0]
        y = self._buf(tag + "y", (T, self.W), torch.bfloat16)
        K.kda_output_norm_gate(o, gp, self.norm_w, y, eps=self.rms_eps)
        out = self._buf(tag + "out", (T, self.hidden), torch.float32)
        K.kda_gemm_epilogue(y, self.Wo, out)
        return out

    def output(self, o, gp, tag=""):
        """y = RMSNorm(o) x w x sigmoid(gate) (bf16), out = y W_o^T (float32)."""
        T = o.shape[0]
        y = self._buf(tag + "y", (T, self.W), torch.bfloat16)
        K.kda_output_norm_gate(o, gp, self.norm_w, y, eps=self.rms_eps)
        out = self._buf(tag + "out", (T, self.hidden), torch.float32)
        K.kda_gemm(y, self.Wo, out)
        return out, y

    def forward(self, x, cu_seqlens=None, cu_seqlens_host=None, initial_state=None, final_state=None,
                conv_state_in=None, conv_state_out=None, return_parts=False):
        """x [T, hidden] bf16 (packed sequences if cu_seqlens is given) ->
        out [T, hidden] float32. Optional conv states are [3, N, 3, H*128]."""
        P, cols = self.projections(x)
        o, qkv = self._core(cols, cu_seqlens, cu_seqlens_host, initial_state, final_state, conv_state_in, conv_state_out)
        out, y = self.output(o, cols[4])
        if return_parts:
            return out, dict(q=qkv[0], k=qkv[1], v=qkv[2], o=o, y=y, P=P)
        return out

    def _core(self, cols, cu_seqlens=None, cu_seqlens_host=None, initial_state=None, final_state=None,
              conv_state_in=None, conv_state_out=None):
        """Convolutions, gate and prefill of the projection columns -> o, (q, k, v)."""
        qp, kp, vp, fp, _, bp = cols
        T, H, W = qp.shape[0], self.H, self.W
        qkv = []
        for i, (src, l2) in enumerate(((qp, D), (kp, D), (vp, 0))):
            y = self._buf("c%d" % i, (T, W), torch.bfloat16)
            K.kda_conv_prefill(src, self.conv[i], y, cu_seqlens=cu_seqlens, cu_seqlens_host=cu_seqlens_host,
                               conv_state_in=None if conv_state_in is None else conv_state_in[i],
                               conv_state_out=None if conv_state_out is None else conv_state_out[i],
                               apply_silu=True, l2norm_group=l2, l2norm_eps=self.l2_eps)
            qkv.append(y.view(T, H, D))
        # the gate prologue runs inside the prefill: g and beta are formed from
        # the f and b columns of P in registers and never stored
        o = self._buf("o", (T, H, D), torch.float32)
        K.kda_prefill_gated(qkv[0], qkv[1], qkv[2], fp, bp, self.A_log, o, cu_seqlens=cu_seqlens,
                            cu_seqlens_host=cu_seqlens_host, initial_state=initial_state,
                            final_state=final_state, scale=self.scale, lower_bound=self.lower_bound)
        return o, qkv

    def decode(self, x, state, conv_states):
        """One token per sequence: x [B, hidden] bf16; state float32 [B, H, 128, 128]
        and conv_states bf16 [3, B, 3, H*128] are updated in place. Returns
        out [B, hidden] float32."""
        _, cols = self.projections(x)
        o = self._core_decode(cols, state, conv_states)
        out, _ = self.output(o, cols[4], tag="d")
        return out

    def _core_decode(self, cols, state, conv_states):
        qp, kp, vp, fp, _, bp = cols
        B, H, W = qp.shape[0], self.H, self.W
        qkv = []
        for i, (src, l2) in enumerate(((qp, D), (kp, D), (vp, 0))):
            y = self._buf("dc%d" % i, (B, W), torch.bfloat16)
            K.kda_conv_state_update(src, conv_states[i], self.conv[i], y, apply_silu=True,
                                    l2norm_group=l2, l2norm_eps=self.l2_eps)
            qkv.append(y.view(B, H, D))
        g = self._buf("dg", (B, H, D), torch.bfloat16)
        beta = self._buf("dbeta", (B, H), torch.bfloat16)
        K.kda_gate_prologue(fp, bp, self.A_log, g, beta, H, D, lower_bound=self.lower_bound)
        o = self._buf("do", (B, H, D), torch.float32)
        K.kda_decode_step(qkv[0], qkv[1], qkv[2], g, beta, state, o, scale=self.scale,
                          lower_bound=self.lower_bound)
        return o

    def decode_tree(self, x, parents, state, conv_states):
        """Verify a tree of drafted tokens per sequence: x [B, N, hidden] bf16,
        parents int32 [B, N] (as kda_decode_tree), state [B, H, 128, 128]
        (float32 or bfloat16) and conv_states bf16 [3, B, 3, H*128] only read.
        Returns out [B, N, hidden] float32 and the DraftTree that commits an
        accepted path (both valid until the next call on this stream)."""
        B, N, hidden = x.shape
        if parents.shape != (B, N):
            raise ValueError("parents must be [%d, %d] as x (got %s)" % (B, N, tuple(parents.shape)))
        _, cols = self.projections(x.reshape(B * N, hidden), tag="t")  # the commit reads them: not decode's buffer
        o, tree = self._core_tree(cols, parents, state, conv_states)
        out, _ = self.output(o.view(B * N, self.H, D), cols[4], tag="t")
        return out.view(B, N, hidden), tree

    def _core_tree(self, cols, parents, state, conv_states):
        qp, kp, vp, fp, _, bp = cols
        B, N = parents.shape
        H, W = self.H, self.W
        qkv = []
        for i, (src, l2) in enumerate(((qp, D), (kp, D), (vp, 0))):
            y = self._buf("tc%d" % i, (B * N, W), torch.bfloat16)
            K.kda_conv_tree(src, conv_states[i], parents, self.conv[i], y, apply_silu=True, l2norm_group=l2,
                            l2norm_eps=self.l2_eps)
            qkv.append(y.view(B, N, H, D))
        g = self._buf("tg", (B * N, H, D), torch.bfloat16)
        beta = self._buf("tbeta", (B * N, H), torch.bfloat16)
        K.kda_gate_prologue(fp, bp, self.A_log, g, beta, H, D, lower_bound=self.lower_bound)
        o = self._buf("to", (B, N, H, D), torch.float32)
        writes = self._buf("tw", (B, N, H, D), torch.float32)
        tree = DraftTree(self, parents, (qp, kp, vp), qkv[1], g.view(B, N, H, D), writes, g)
        K.kda_decode_tree(qkv[0], qkv[1], qkv[2], tree.g, beta.view(B, N, H), parents, state, o, writes, scale=self.scale,
                          lower_bound=self.lower_bound)
        return o, tree


class DraftTree:
    """What a mixer's verification of a tree leaves for its commit (buffers of
    the mixer: valid until its next verification on the same stream; once another
    has overwritten them it refuses to commit)."""

    def __init__(self, mixer, parents, inputs, k, g, writes, buffer):
        self.mixer, self.parents, self.inputs, self.k, self.g, self.writes = mixer, parents, inputs, k, g, writes
        # `buffer`, a buffer of the verification that every next one with as many
        # rows overwrites, names the tree that it holds
        self.buffer, self.token = buffer, object()
        buffer.tree = self.token

    def commit(self, accepted, state, conv_states):
        """state and conv_states (those that were verified against) advance in place
        along the path to node accepted[b] (int32 [B]; any other value: unchanged)."""
        if self.buffer.tree is not self.token:
            raise RuntimeError("the mixer has verified another tree since: this one's buffers are overwritten")
        if len(conv_states) != len(self.inputs):
            raise ValueError("conv_states must hold the q, k and v histories (got %d)" % len(conv_states))
        K.kda_decode_tree_commit(self.k, self.g, self.writes, self.parents, accepted, state,
                                 lower_bound=self.mixer.lower_bound)
        for x, cs in zip(self.inputs, conv_states):
            K.kda_conv_tree_commit(x, self.parents, accepted, cs)


class BranchNorm:
    """How a block's output x joins the residual stream h in a block with a norm after
    it too: h = residual_scale h + branch_scale act(gate) RMSNorm(x) weight. weight
    float32 [width]; gate a learned [width] vector (float32 or bfloat16) or None, through
    gate_activation ('none' or 'sigmoid')."""

    def __init__(self, weight, gate=None, gate_activation="none", residual_scale=1.0, branch_scale=1.0, eps=1e-6):
        self.weight = weight
        self.form = dict(gate=gate, gate_activation=gate_activation, residual_scale=residual_scale,
                         branch_scale=branch_scale, post_eps=eps)


class Branch:
    """A block's output still to be joined to the residual stream through its norm."""

    __slots__ = ("x", "post")

    def __init__(self, x, post):
        self.x, self.post = x, post


class KDABlock:
    """A mixer in its pre-norm residual block: hidden += mixer(RMSNorm(hidden) norm_weight).

    The residual stream `hidden` (bfloat16 or float32 rows) is updated in place.
    With bfloat16 or 4-bit weights the output projection adds into it (the product's
    epilogue). With block-FP8 weights the block's output is returned as `delta`,
    and the next block adds it while it normalises: one pass then updates the
    stream, norms it and quantizes the projections' input. So every method takes
    the delta still to be added (None: nothing) and returns the one it leaves
    (None: added; else a buffer of the mixer, valid until that method's next call on
    the same stream); `finish` adds a last one.

    With `post` (a BranchNorm) the output is normalised, gated and scaled before it is
    added: every kind of mixer then returns a delta (a Branch), and the next block's
    norm takes both norms in one pass."""

    def __init__(self, mixer, norm_weight, eps=1e-6, post=None):
        self.mixer, self.norm_weight, self.eps, self.post = mixer, norm_weight, eps, post

    def _enter(self, hidden, delta, tag=""):
        """hidden += delta in place; the projections of its norm -> their columns."""
        m = self.mixer
        if isinstance(delta, Branch):
            return m.projections_of_norm(delta.x, hidden, self.norm_weight, self.eps, tag, post=delta.post)
        x, residual = (hidden, None) if delta is None else (delta, hidden)
        return m.projections_of_norm(x, residual, self.norm_weight, self.eps, tag)

    def _leave(self, o, gp, hidden, tag):
        if self.post is None:
            return self.mixer.output_into(o, gp, hidden, tag=tag)
        return Branch(self.mixer.output_branch(o, gp, tag), self.post)

    def forward(self, hidden, delta=None, **states):
        """Prefill: hidden [T, width] rows, states as KDAMixer.forward's arguments."""
        cols = self._enter(hidden, delta)
        o, _ = self.mixer._core(cols, **states)
        return self._leave(o, cols[4], hidden, "b")

    def decode(self, hidden, state, conv_states, delta=None):
        """One token per sequence: hidden [B, width], states (as KDAMixer.decode's,
        float32) updated in place."""
        cols = self._enter(hidden, delta)
        o = self.mixer._core_decode(cols, state, conv_states)
        return self._leave(o, cols[4], hidden, "bd")

    def decode_tree(self, hidden, parents, state, conv_states, delta=None):
        """A tree of drafts per sequence: hidden [B * N, width], states as
        KDAMixer.decode_tree's. Returns (delta, DraftTree)."""
        cols = self._enter(hidden, delta, tag="t")  # the commit reads them: not decode's buffer
        o, tree = self.mixer._core_tree(cols, parents, state, conv_states)
        return self._leave(o.view(hidden.shape[0], self.mixer.H, D), cols[4], hidden, "bt"), tree

    def finish(self, hidden, delta, norm_weight, y):
        """After the last block: y = RMSNorm(hidden + delta) norm_weight, hidden += delta."""
        if delta is None:
            return K.kda_add_rmsnorm(hidden, norm_weight, y, eps=self.eps)
        if isinstance(delta, Branch):
            return K.kda_sandwich_rmsnorm(delta.x, delta.post.weight, hidden, hidden, norm_weight, y, eps=self.eps,
                                          **delta.post.form)
        return K.kda_add_rmsnorm(delta, norm_weight, y, residual=hidden, residual_out=hidden, eps=self.eps)


class BeamSearch:
    """Beam search with a stack of blocks: B sequences of W beams, a token each a step.

    blocks KDABlocks, norm_weight [width] the norm after the last, head [V, width] (a
    bfloat16 tensor or a W4Weight) the vocabulary's projection, eos the end token (-1: no
    beam ends); states float32 [B * W, H,
    128, 128] and conv_states bf16 [3, B * W, 3, H*128] of every block, updated in place:
    row b * W + w is beam w of sequence b. `start` makes beam 0 of every sequence the
    one that lives (prefill its row; the first step spreads it over the others). After a
    step scores float32, parents (the beam followed), tokens int32 and finished bool
    [B, W] hold the new beams, best first; they and `logits` [B * W, V] (its rows padded to a
    multiple of 4, as the head's product asks) are overwritten by the next. What does not
    fit together is refused here or before a step's first call: a call refused in the middle
    of a step would leave the states of the blocks before it advanced."""

    def __init__(self, blocks, norm_weight, head, B, W, eos, states, conv_states):
        blocks, states, conv_states = list(blocks), list(states), list(conv_states)
        if not blocks or len(states) != len(blocks) or len(conv_states) != len(blocks):
            raise ValueError("a state and a history of every block, one block at least (got %d blocks, %d states, %d histories)" %
                             (len(blocks), len(states), len(conv_states)))
        if B < 0 or not 1 <= W <= 32:
            raise ValueError("B >= 0 sequences of 1 to 32 beams (got %d, %d)" % (B, W))
        if not isinstance(head, K.W4Weight):
            K._type("head", head, torch.bfloat16)
        if eos >= head.shape[0]:
            raise ValueError("eos must be a token below %d, or negative: none (got %d)" % (head.shape[0], eos))
        K._type("norm_weight", norm_weight, torch.float32), K._tensor("norm_weight", norm_weight, head.shape[1:])
        for block, state, conv in zip(blocks, states, conv_states):
            m = block.mixer
            if m.hidden != head.shape[1]:
                raise ValueError("the head is %d wide, a block %d" % (head.shape[1], m.hidden))
            K._type("state", state, torch.float32), K._tensor("state", state, (B * W, m.H, D, D))
            K._type("conv_states", conv, torch.bfloat16)
            K._tensor("conv_states", conv, (3, B * W, m.conv[0].shape[1] - 1, m.W))
        self.blocks, self.norm_weight, self.head, self.eos = blocks, norm_weight, head, eos
        self.states, self.conv_states = states, conv_states
        new = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device="cuda")
        V, width = head.shape
        self.scores, self.finished = new(B, W), new(B, W, dtype=torch.bool)
        self.parents, self.tokens = new(B, W, dtype=torch.int32), new(B, W, dtype=torch.int32)
        self.logits, self.y = new(B * W, (V + 3) // 4 * 4)[:, :V], new(B * W, width, dtype=torch.bfloat16)
        self.start()

    def start(self):
        self.scores.fill_(float("-inf"))
        self.scores[:, 0] = 0
        self.finished.fill_(False)

    def step(self, hidden):
        """hidden [B * W, width] (bfloat16 or float32, changed in place): the embeddings of
        the last step's tokens. Chooses the next ones and moves the beams' states."""
        if hidden.shape != self.y.shape:  # fewer rows would advance some of the beams alone
            raise ValueError("hidden must have shape %s (got %s)" % (tuple(self.y.shape), tuple(hidden.shape)))
        delta = None
        for block, state, conv in zip(self.blocks, self.states, self.conv_states):
            delta = block.decode(hidden, state, conv, delta)
        self.blocks[-1].finish(hidden, delta, self.norm_weight, self.y)
        if isinstance(self.head, K.W4Weight):
            K.kda_gemm_w4(self.y, self.head, self.logits)
        else:
            K.kda_gemm_epilogue(self.y, self.head, self.logits)
        finished = self.finished if self.eos >= 0 else None
        K.kda_beam_select(self.logits, self.scores, self.scores, self.parents, self.tokens, finished=finished,
                          next_finished=finished, eos=self.eos)
        for state, conv in zip(self.states, self.conv_states):
            K.kda_beam_reorder(self.parents, state, conv)
        return self.tokens


class DecodeGraph:
    """One decode step of a mixer captured as a HIP graph: the step's kernels
    (projections, the three conv updates, gate, decode step, epilogue, output
    projection) are replayed without a host launch each, which at a few
    sequences is a large part of the step. The graph reads x from, and writes
    out to, its own buffers and updates the given state and conv states in
    place, so each replay advances those sequences by one token. The calls
    enqueue no memset (the library never does), and the step's buffers are the
    graph's own, so other calls of the mixer may run between replays."""

    def __init__(self, mixer, B, state, conv_states):
        self.x = torch.zeros((B, mixer.hidden), dtype=torch.bfloat16, device="cuda")
        self.state, self.conv_states = state, conv_states
        # an eager step on copies: every kernel is loaded before the capture
        mixer.decode(self.x, state.clone(), conv_states.clone())
        torch.cuda.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            with torch.cuda.graph(self.graph, stream=s):
                self.out = mixer.decode(self.x, state, conv_states)
        torch.cuda.current_stream().wait_stream(s)

    def step(self, x):
        """Copy x [B, hidden] in, replay, return the output buffer."""
        self.x.copy_(x)
        self.graph.replay()
        return self.out


class KDAMixerFP8(KDAMixer):
    """The same mixer with its projections in block FP8 (W8A8): E4M3 weights
    in 128 x 128 blocks with float32 block scales, as the release stores them,
    and activations quantized dynamically ("Ling-3.1-flash: Grouped Routing
    and Two Different MLA Caches", section "Production boundaries"). The input
    x is quantized per (token, 128 channels) by kda_quantize_fp8 and the
    epilogue writes its output quantized per (token, head)
    (kda_output_norm_gate_fp8); both projections run kda_gemm_fp8 (weight
    streaming up to 8 tokens, the FP8 matrix cores beyond)."""

    def __init__(self, Win_codes, Win_scales, Wo_codes, Wo_scales, conv_q, conv_k, conv_v, A_log, norm_w, H,
                 **kw):
        super().__init__(Win_codes, conv_q, conv_k, conv_v, A_log, norm_w, Wo_codes, H, **kw)
        self.W_in_s, self.Wo_s = Win_scales, Wo_scales

    @classmethod
    def from_host(cls, d):
        """Build from the seeded host weights of ``synth.workload_layer_fp8``."""
        u8 = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        # packed rows padded with zero codes to a multiple of 8 (16-byte aligned
        # column slices of the projection output), with block scales to match
        codes, scales = d["Win_codes"], d["Win_scales"]
        pad = (-codes.shape[0]) % 8
        if pad:
            codes = np.concatenate([codes, np.zeros((pad, codes.shape[1]), np.uint8)])
        need = (codes.shape[0] + 127) // 128
        if scales.shape[0] < need:
            scales = np.concatenate([scales, np.ones((need - scales.shape[0], scales.shape[1]), np.float32)])
        return cls(u8(codes), u8(scales), u8(d["Wo_codes"]), u8(d["Wo_scales"]),
                   _dev_bf16(d["conv_q"]), _dev_bf16(d["conv_k"]), _dev_bf16(d["conv_v"]),
                   torch.from_numpy(d["A_log"]).cuda(), torch.from_numpy(d["norm_w"]).cuda(), d["H"])

    def projections(self, x, tag=""):
        """x quantized per (token, 128 channels), then P = X W_in^T (bf16)."""
        T, hidden = x.shape
        xq = self._buf("xq", (T, hidden), torch.uint8)
        xs = self._buf("xs", (T, hidden // 128), torch.float32)
        K.kda_quantize_fp8(x, xq, xs)
        P = self._buf(tag + "P", (T, self.W_in.shape[0]), torch.bfloat16)
        K.kda_gemm_fp8(xq, xs, self.W_in, self.W_in_s, P)
        return P, self._columns(P)

    def projections_of_norm(self, x, residual, norm_weight, eps, tag, post=None):
        """As KDAMixer's, the norm quantized in the same pass."""
        T, hidden = x.shape
        xq = self._buf("nq", (T, hidden), torch.uint8)
        xs = self._buf("ns", (T, hidden // 128), torch.float32)
        if post is None:
            K.kda_add_rmsnorm_fp8(x, norm_weight, xq, xs, residual=residual, residual_out=residual, eps=eps)
        else:
            K.kda_sandwich_rmsnorm_fp8(x, post.weight, residual, residual, norm_weight, xq, xs, eps=eps, **post.form)
        P = self._buf(tag + "nP", (T, self.W_in.shape[0]), torch.bfloat16)
        K.kda_gemm_fp8(xq, xs, self.W_in, self.W_in_s, P)
        return self._columns(P)

    def output_branch(self, o, gp, tag):
        return self.output(o, gp, tag)[0]

    def output_into(self, o, gp, hidden, tag):
        """The block's output, left for the next norm to add."""
        return self.output_branch(o, gp, tag)

    def output(self, o, gp, tag=""):
        """The epilogue quantized per (token, head), then out = Y W_o^T (float32)."""
        T = o.shape[0]
        yq = self._buf(tag + "yq", (T, self.W), torch.uint8)
        ys = self._buf(tag + "ys", (T, self.H), torch.float32)
        K.kda_output_norm_gate_fp8(o, gp, self.norm_w, yq, ys, eps=self.rms_eps)
        out = self._buf(tag + "out", (T, self.hidden), torch.float32)
        K.kda_gemm_fp8(yq, ys, self.Wo, self.Wo_s, out)
        return out, (yq, ys)


class KDAMixerW4(KDAMixer):
    """The same mixer with its projections in 4 bits (kda_w4_pack): W_in [5*H*128 + H (+
    zero rows to a multiple of 8), hidden] and Wo [hidden, H*128] are W4Weights. Below
    EXPAND rows (decode, draft trees, beams) the products read the packed weights; a
    prefill expands each to bfloat16 before its product, in a scratch that all mixers of a
    device and stream share (in every call anew: the weights' roundings to bfloat16 are the
    difference between the two)."""

    # Rows from which expanding pays; direct | expanded, us: with 41,024 x 4096 weights 512
    # rows 219 | 296, 768 338 | 318, 1,024 433 | 415; with 4096 x 8192 80 | 88 for 768, 100 | 92
    EXPAND = 768

    def __init__(self, W_in, Wo, conv_q, conv_k, conv_v, A_log, norm_w, H, **kw):
        super().__init__(W_in, conv_q, conv_k, conv_v, A_log, norm_w, Wo, H, **kw)

    @classmethod
    def from_host(cls, d):
        """Build from host arrays: the convolutions, A_log, norm_w and H as in
        ``synth.workload_layer``, and for both weights (Win, Wo) kda_w4_pack's inputs:
        codes uint8 [N, K/2], scales float32 [N, K/group] and, where given, zeros uint8."""
        def packed(name, pad):
            parts = [d[name + "_codes"], d[name + "_scales"], d.get(name + "_zeros")]
            # rows of zero scale up to a multiple of 8 (16-byte aligned columns of the output)
            rows = (-parts[0].shape[0]) % 8 if pad else 0
            parts = [None if p is None else np.concatenate([p, np.zeros((rows, p.shape[1]), p.dtype)]) for p in parts]
            return K.kda_w4_pack(*(None if p is None else torch.from_numpy(p).cuda() for p in parts))
        return cls(packed("Win", True), packed("Wo", False), _dev_bf16(d["conv_q"]), _dev_bf16(d["conv_k"]),
                   _dev_bf16(d["conv_v"]), torch.from_numpy(d["A_log"]).cuda(), torch.from_numpy(d["norm_w"]).cuda(), d["H"])

    def _product(self, x, w, y, residual=None):
        if x.shape[0] < self.EXPAND:
            return K.kda_gemm_w4(x, w, y, residual=residual)
        with _expanding:
            W = K.kda_w4_expand(w, self._buf(EXPANDED, w.shape, torch.bfloat16))
            return K.kda_gemm_epilogue(x, W, y, residual=residual)

    def projections(self, x, tag=""):
        P = self._buf(tag + "P", (x.shape[0], self.W_in.N), torch.bfloat16)
        self._product(x, self.W_in, P)
        return P, self._columns(P)

    def projections_of_norm(self, x, residual, norm_weight, eps, tag, post=None):
        T, hidden = x.shape
        y = self._buf("ny", (T, hidden), torch.bfloat16)
        if post is None:
            K.kda_add_rmsnorm(x, norm_weight, y, residual=residual, residual_out=residual, eps=eps)
        else:
            K.kda_sandwich_rmsnorm(x, post.weight, residual, residual, norm_weight, y, eps=eps, **post.form)
        P = self._buf(tag + "nP", (T, self.W_in.N), torch.bfloat16)
        self._product(y, self.W_in, P)
        return self._columns(P)

    def output_into(self, o, gp, hidden, tag):
        y = self._buf(tag + "y", (o.shape[0], self.W), torch.bfloat16)
        K.kda_output_norm_gate(o, gp, self.norm_w, y, eps=self.rms_eps)
        self._product(y, self.Wo, hidden, residual=hidden)

    def output_branch(self, o, gp, tag):
        return self.output(o, gp, tag)[0]

    def output(self, o, gp, tag=""):
        T = o.shape[0]
        y = self._buf(tag + "y", (T, self.W), torch.bfloat16)
        K.kda_output_norm_gate(o, gp, self.norm_w, y, eps=self.rms_eps)
        out = self._buf(tag + "out", (T, self.hidden), torch.float32)
        self._product(y, self.Wo, out)
        return out, y
