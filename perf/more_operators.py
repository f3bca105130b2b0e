"""Operators of a beam-search decoding step over blocks with 4-bit weights, as cases to measure.

``run`` computes a case either in plain torch operations (``own`` false) or by
the calls a user makes of the library (``own`` true). Four kinds of case:

w4        y = x W^T (+ residual) with W = scale (code - zero) from 4-bit codes,
          one scale (and zero point) per row and group of columns
sandwich  h = residual_scale residual + branch_scale act(gate) RMSNorm(x) and
          y = RMSNorm(h): the norm after a block, its gate and residual scale, and
          the norm before the next one; y in bfloat16, float32 or E4M3 with scales
beam      the best continuations of a batch of beams over the vocabulary
reorder   recurrent states and convolution histories moved to the beams chosen
"""
import math

import torch

own = False

D = 128  # channels of a head
EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # output projection of one decoding sequence: latency of a single token
        dict(name="w4_1x4096x8192", kind="w4", M=1, N=4096, K=8192, G=128, s="bf16", zeros=False, residual=True, y="bf16"),
        # packed input projection of one decoding sequence, with zero points in groups of 64
        dict(name="w4_1x41024x4096", kind="w4", M=1, N=41024, K=4096, G=64, s="bf16", zeros=True, residual=False, y="bf16"),
        # a few beams through a projection of odd sizes, groups of 32 with float32 scales
        dict(name="w4_5x4999x4128", kind="w4", M=5, N=4999, K=4128, G=32, s="f32", zeros=True, residual=False, y="f32"),
        # packed input projection of a serving batch of 16 sequences of 4 beams
        dict(name="w4_64x41024x4096", kind="w4", M=64, N=41024, K=4096, G=128, s="bf16", zeros=False, residual=False, y="bf16"),
        # between two W8A8 blocks, one token of one sequence: latency of a single row
        dict(name="sandwich_fp8_1x4096", kind="sandwich", M=1, K=4096, x="f32", r="bf16", y="fp8", gate="vector", act="none"),
        # a ragged prefill chunk at an odd width, a gate of the tokens' own
        dict(name="sandwich_bf16_1237x5128", kind="sandwich", M=1237, K=5128, x="bf16", r="bf16", y="bf16", gate="rows", act="sigmoid"),
        # the layer workload's prefill, 8,192 tokens of width 4,096, one token short of whole tiles, float32 stream
        dict(name="sandwich_fp8_8191x4096", kind="sandwich", M=8191, K=4096, x="f32", r="f32", y="fp8", gate="none", act="none"),
        # one sequence of four beams, its first steps: latency
        dict(name="beam_1x4x32000", kind="beam", B=1, W=4, V=32000, t="f32", finished=False, first=True),
        # a few sequences with an odd number of beams and an odd vocabulary, some beams ended
        dict(name="beam_7x5x50257", kind="beam", B=7, W=5, V=50257, t="bf16", finished=True, first=False),
        # a full serving batch
        dict(name="beam_64x8x131072", kind="beam", B=64, W=8, V=131072, t="f32", finished=True, first=False),
        # one sequence of four beams, bfloat16 states: latency
        dict(name="reorder_1x4_bf16", kind="reorder", B=1, W=4, H=64, taps=4, s="bf16"),
        # the decode workload's 256 float32 states as 64 sequences of four beams
        dict(name="reorder_64x4_f32", kind="reorder", B=64, W=4, H=64, taps=4, s="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["w4", "sandwich", "beam", "reorder"])
    if kind == "w4":
        G = rng.choice([32, 64, 128])
        return dict(kind=kind, M=_log(rng, 1, 64), N=_log(rng, 64, 40000), K=G * _log(rng, 2, 4096 // G), G=G,
                    s=rng.choice(["f32", "bf16", "bf16"]), zeros=rng.random() < 0.5, residual=rng.random() < 0.3,
                    y=rng.choice(["f32", "bf16"]))
    if kind == "sandwich":
        y = rng.choice(["fp8", "bf16", "f32"])
        K = 128 * _log(rng, 1, 64) if y == "fp8" else 8 * _log(rng, 4, 1024)
        return dict(kind=kind, M=_log(rng, 1, min(8191, 16777216 // K)), K=K, x=rng.choice(["f32", "bf16"]),
                    r=rng.choice(["f32", "bf16"]), y=y, gate=rng.choice(["none", "vector", "rows"]),
                    act=rng.choice(["none", "sigmoid"]))
    if kind == "beam":
        W, V = _log(rng, 1, 16), _log(rng, 1000, 160000)
        return dict(kind=kind, B=_log(rng, 1, min(64, 64000000 // (W * V))), W=W, V=V, t=rng.choice(["f32", "bf16"]),
                    finished=rng.random() < 0.6, first=rng.random() < 0.2)
    W, H = _log(rng, 2, 16), _log(rng, 4, 64)
    return dict(kind=kind, B=_log(rng, 1, min(96, 192 // W)), W=W, H=H, taps=rng.choice([3, 4, 4, 8]),
                s=rng.choice(["f32", "bf16"]))


# ------------------------------------------------------------------ inputs
class _Draws:
    """Seeded values on the GPU."""

    def __init__(self, seed):
        self.gen = torch.Generator(device="cuda").manual_seed(seed % (1 << 62) + 1)

    def normal(self, *shape, std=1.0):
        return torch.randn(shape, generator=self.gen, device="cuda") * std

    def uniform(self, *shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=self.gen, device="cuda") * (hi - lo) + lo

    def whole(self, hi, *shape, lo=0, dtype=torch.int32):
        return torch.randint(lo, hi, shape, generator=self.gen, device="cuda", dtype=dtype)


def prepare(case, seed):
    c, d, s = case, _Draws(seed), dict(case)
    kind = c["kind"]
    if kind == "w4":
        M, N, K, G = c["M"], c["N"], c["K"], c["G"]
        s["x"] = d.normal(M, K).bfloat16()
        s["codes"] = d.whole(256, N, K // 2, dtype=torch.uint8)  # the even column in the low four bits
        s["scales"] = (d.uniform(N, K // G, lo=0.5, hi=1.5) * (0.2 / K ** 0.5)).to(TYPES[c["s"]])
        s["zero_points"] = d.whole(11, N, K // G, lo=5, dtype=torch.uint8) if c["zeros"] else None
        s["res"] = d.normal(M, N).to(TYPES[c["y"]]) if c["residual"] else None
        s["out"] = torch.empty((M, N), dtype=TYPES[c["y"]], device="cuda")
        if own:  # a program lays its weights out once, when it loads them
            from gated_delta_rule_02_amd import kda as K_
            s["weight"] = K_.kda_w4_pack(s["codes"], s["scales"], s["zero_points"])
    elif kind == "sandwich":
        M, K = c["M"], c["K"]
        s["x"] = (d.normal(M, K) * d.uniform(M, 1, lo=0.1, hi=4.0)).to(TYPES[c["x"]])
        s["res"] = (d.normal(M, K) * d.uniform(M, 1, lo=0.5, hi=4.0)).to(TYPES[c["r"]])
        s["res_out"] = torch.empty_like(s["res"])
        s["w_post"], s["w"] = d.uniform(K, lo=0.5, hi=1.5), d.uniform(K, lo=0.5, hi=1.5)
        # a learned vector, or columns of the tokens' own packed projections
        s["gate_v"] = None
        if c["gate"] == "vector":
            s["gate_v"] = d.normal(K)
        elif c["gate"] == "rows":
            s["gate_v"] = d.normal(M, K + 64).bfloat16()[:, 64:]
        s["residual_scale"], s["branch_scale"] = 0.875, 0.625
        if c["y"] == "fp8":
            s["codes"] = torch.empty((M, K), dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty((M, K // 128), device="cuda")
        else:
            s["out"] = torch.empty((M, K), dtype=TYPES[c["y"]], device="cuda")
    elif kind == "beam":
        B, W, V = c["B"], c["W"], c["V"]
        logits = d.normal(B * W, V, std=2.5)
        logits[:, V // 3:V // 3 + V // 50] = float("-inf")  # tokens the caller bans
        s["logits"] = logits.to(TYPES[c["t"]])
        s["scores"] = -d.uniform(B, W, lo=0.0, hi=8.0).sort(-1).values
        if c["first"]:  # one live beam a sequence
            s["scores"][:, 1:] = float("-inf")
        s["eos"] = V - 1
        s["ended"] = d.uniform(B, W) < 0.2 if c["finished"] else None
        s["new_scores"] = torch.empty((B, W), device="cuda")
        s["parents"] = torch.empty((B, W), dtype=torch.int32, device="cuda")
        s["tokens"] = torch.empty((B, W), dtype=torch.int32, device="cuda")
        s["new_ended"] = torch.empty((B, W), dtype=torch.bool, device="cuda") if c["finished"] else None
    else:
        B, W, H, C = c["B"], c["W"], c["H"], c["H"] * D
        s["state"] = d.normal(B * W, H, D, D, std=0.1).to(TYPES[c["s"]])
        s["hist"] = d.normal(3, B * W, c["taps"] - 1, C).bfloat16()
        s["parents"] = d.whole(W, B, W)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    from gated_delta_rule_02_amd import kda as K
    kind = s["kind"]
    if kind == "w4":
        return K.kda_gemm_w4(s["x"], s["weight"], s["out"], residual=s["res"])
    if kind == "sandwich":
        form = dict(gate=s["gate_v"], gate_activation=s["act"], residual_scale=s["residual_scale"],
                    branch_scale=s["branch_scale"], post_eps=EPS, eps=EPS)
        if s["y"] == "fp8":
            K.kda_sandwich_rmsnorm_fp8(s["x"], s["w_post"], s["res"], s["res_out"], s["w"], s["codes"], s["scales"], **form)
            return [s["codes"].view(torch.float8_e4m3fn), s["scales"], s["res_out"]]
        K.kda_sandwich_rmsnorm(s["x"], s["w_post"], s["res"], s["res_out"], s["w"], s["out"], **form)
        return [s["out"], s["res_out"]]
    if kind == "beam":
        K.kda_beam_select(s["logits"], s["scores"], s["new_scores"], s["parents"], s["tokens"], finished=s["ended"],
                          next_finished=s["new_ended"], eos=s["eos"])
        return [s["new_scores"], s["parents"], s["tokens"], s["new_ended"]]
    K.kda_beam_reorder(s["parents"], s["state"], s["hist"])
    return [s["state"], s["hist"]]


def _plain(s):
    kind = s["kind"]
    if kind == "w4":
        N, K, G = s["N"], s["K"], s["G"]
        w = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).view(N, K // G, G).float()
        w = w - (8.0 if s["zero_points"] is None else s["zero_points"].float()[:, :, None])
        y = s["x"].float() @ (w * s["scales"].float()[:, :, None]).view(N, K).t()
        if s["res"] is not None:
            y = y + s["res"].float()
        return y.to(s["out"].dtype)
    if kind == "sandwich":
        x = s["x"].float()
        n = x * (1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)) * s["w_post"]
        if s["gate_v"] is not None:
            g = s["gate_v"].float()
            n = n * (1 / (1 + torch.exp(-g)) if s["act"] == "sigmoid" else g)
        h = s["residual_scale"] * s["res"].float() + s["branch_scale"] * n
        y = h * (1 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)) * s["w"]
        r = h.to(s["res"].dtype)
        if s["y"] != "fp8":
            return [y.to(TYPES[s["y"]]), r]
        y = y.view(y.shape[0], -1, 128)
        top = y.abs().amax(-1)
        scale = torch.where(top > 0, top / 448, torch.ones_like(top))
        q = (y / scale[..., None]).clamp(-448, 448).view(s["codes"].shape)
        return [q.to(torch.float8_e4m3fn), scale, r]
    if kind == "beam":
        B, W, V = s["B"], s["W"], s["V"]
        # 64 bits: the order of two continuations may hang on their last places
        x = s["logits"].double().view(B, W, V)
        top = x.amax(-1, keepdim=True)
        cand = s["scores"].double()[:, :, None] + (x - top - torch.log(torch.exp(x - top).sum(-1, keepdim=True)))
        place = torch.arange(W * V, device=x.device)
        if s["ended"] is not None:  # an ended beam goes on as it is
            alone = torch.where(place[:V] == s["eos"], s["scores"].double()[:, :, None], -math.inf)
            cand = torch.where(s["ended"][:, :, None], alone, cand)
        cand = torch.where(cand != cand, -math.inf, cand).view(B, W * V)
        free = torch.ones_like(cand, dtype=torch.bool)
        scores, picks = [], []
        for _ in range(W):
            best = torch.where(free, cand, -math.inf).amax(-1, keepdim=True)
            at = torch.where(free & (cand == best), place, W * V).amin(-1, keepdim=True)
            free.scatter_(1, at, False)
            scores.append(best)
            picks.append(at)
        picks = torch.cat(picks, -1)
        parents, tokens = (picks // V).int(), (picks % V).int()
        ended = None
        if s["ended"] is not None:
            ended = torch.gather(s["ended"], 1, picks // V) | (tokens == s["eos"])
        return [torch.cat(scores, -1).float(), parents, tokens, ended]
    B, W = s["parents"].shape
    rows = (torch.arange(B, device="cuda")[:, None] * W + s["parents"]).view(-1)
    s["state"].copy_(s["state"][rows])
    s["hist"].copy_(s["hist"][:, rows])
    return [s["state"], s["hist"]]


# ------------------------------------------------------------------ cost
def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "fp8": 1}
    if c["kind"] == "w4":
        M, N, K, G = c["M"], c["N"], c["K"], c["G"]
        groups = N * (K // G) * (size[c["s"]] + (1 if c["zeros"] else 0))
        return {"bytes": N * K // 2 + groups + 2 * M * K + M * N * size[c["y"]] * (2 if c["residual"] else 1),
                "flops": 2 * M * N * K}
    if c["kind"] == "sandwich":
        n = c["M"] * c["K"]
        gate = {"none": 0, "vector": 4 * c["K"], "rows": 2 * n}[c["gate"]]
        b = n * (size[c["x"]] + size[c["y"]] + 2 * size[c["r"]]) + 8 * c["K"] + gate
        return {"bytes": b + (n // 32 if c["y"] == "fp8" else 0), "flops": 14 * n}
    if c["kind"] == "beam":
        n = c["B"] * c["W"] * c["V"]
        return {"bytes": n * size[c["t"]], "flops": 4 * n}
    # parents are drawn independently: all beams but one of a sequence move on average, from
    # the beams that at least one of the W - 1 others chose
    W = c["W"]
    rows = c["B"] * ((W - 1) + W * (1 - (1 - 1 / W) ** (W - 1)))
    return {"bytes": int(rows * (c["H"] * D * D * size[c["s"]] + 3 * (c["taps"] - 1) * c["H"] * D * 2)), "flops": 0}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The operators' definitions followed in 64 bits, group by group, sequence by sequence."""
    s = prepare(case, seed)
    kind = s["kind"]
    if kind == "w4":
        N, K, G = s["N"], s["K"], s["G"]
        codes = torch.empty((N, K), dtype=torch.float64, device="cuda")
        codes[:, 0::2] = (s["codes"] % 16).double()
        codes[:, 1::2] = (s["codes"] // 16).double()
        y = torch.zeros((s["M"], N), dtype=torch.float64, device="cuda")
        if s["res"] is not None:
            y += s["res"].double()
        for g in range(K // G):
            at = slice(g * G, (g + 1) * G)
            zero = 8 if s["zero_points"] is None else s["zero_points"][:, g:g + 1].double()
            y += torch.mm(s["x"][:, at].double(), (codes[:, at] - zero).t().contiguous()) * s["scales"][:, g].double()
        return y
    if kind == "sandwich":
        def norm(v, w):
            return v / (v.pow(2).sum(1, keepdim=True) / v.shape[1] + EPS).sqrt() * w.double()

        branch = norm(s["x"].double(), s["w_post"])
        if s["gate_v"] is not None:
            branch = branch * (torch.sigmoid(s["gate_v"].double()) if s["act"] == "sigmoid" else s["gate_v"].double())
        h = s["res"].double() * s["residual_scale"] + branch * s["branch_scale"]
        y = norm(h, s["w"])
        if s["y"] != "fp8":
            return [y, h]
        scale = y.unflatten(1, (-1, 128)).abs().max(2).values / 448
        scale[scale == 0] = 1
        return [(y.unflatten(1, (-1, 128)) / scale[:, :, None]).flatten(1), scale, h]
    if kind == "beam":
        B, W, V = s["B"], s["W"], s["V"]
        scores = torch.empty((B, W), dtype=torch.float64, device="cuda")
        flat = torch.empty((B, W), dtype=torch.int64, device="cuda")
        for b in range(B):
            rows = []
            for w in range(W):
                score = s["scores"][b, w].double()
                if s["ended"] is not None and bool(s["ended"][b, w]):
                    row = torch.full((V,), -math.inf, dtype=torch.float64, device="cuda")
                    row[s["eos"]] = score
                else:
                    row = torch.log_softmax(s["logits"][b * W + w].double(), 0) + score
                rows.append(torch.nan_to_num(row, nan=-math.inf, posinf=math.inf, neginf=-math.inf))
            order = torch.sort(torch.cat(rows), descending=True, stable=True)
            scores[b], flat[b] = order.values[:W], order.indices[:W]
        parents, tokens = torch.div(flat, V, rounding_mode="floor"), flat.remainder(V)
        ended = None
        if s["ended"] is not None:
            ended = s["ended"].gather(1, parents).logical_or(tokens.eq(s["eos"]))
        return [scores, parents.int(), tokens.int(), ended]
    state, hist, W = s["state"].clone(), s["hist"].clone(), s["W"]
    for b, chosen in enumerate(s["parents"].tolist()):
        for i, j in enumerate(chosen):
            state[b * W + i] = s["state"][b * W + j]
            hist[:, b * W + i] = s["hist"][:, b * W + j]
    return [state.double(), hist.double()]
