"""The operators around the FP4 mixture-of-experts layer, case by case: the
router that gives it its expert ids and weights, the FP8 linear map with a
scale per block of 128 that its shared expert and neighbouring projections
are made of, and the norms before and after the block fused with its gate
and residual.

``run`` computes a case in elementary torch operations, or, with ``own`` set,
with this package's kernels.  ``exact`` gives the values of the definition in
64 bits.  Shapes are those of the package's workloads (H 2560 / 4096 / 7168,
E 128 / 256 / 512) or powers of two next to them.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
FP8_MAX = 448.0
BLOCK = 128


def listed():
    return [
        # one token of a decode step through a grouped sigmoid router: latency alone
        dict(name="route_m1_e256_groups", op="route", M=1, H=7168, E=256, k=8, weight="bf16", scoring="sigmoid",
             bias=True, groups=8, top_groups=4, renorm=True, scale=1.5, logits=False),
        # a ragged decode batch over many experts, fp32 router weights, probabilities not renormalised, logits kept
        dict(name="route_m37_e512_fp32", op="route", M=37, H=2560, E=512, k=10, weight="fp32", scoring="softmax",
             bias=False, groups=1, top_groups=1, renorm=False, scale=1.0, logits=True),
        # a prefill chunk of the E128 layer
        dict(name="route_m4096_e128", op="route", M=4096, H=4096, E=128, k=8, weight="bf16", scoring="softmax",
             bias=False, groups=1, top_groups=1, renorm=True, scale=1.0, logits=False),
        # a long prefill through the grouped sigmoid router
        dict(name="route_m16384_e256_groups", op="route", M=16384, H=7168, E=256, k=8, weight="bf16",
             scoring="sigmoid", bias=True, groups=8, top_groups=4, renorm=True, scale=1.5, logits=False),
        # shared expert's gate and up for one token: the weights are read once
        dict(name="fp8_m1_gated", op="fp8", M=1, K=7168, N=2048, fn="silu"),
        # small projection of a few tokens, widths that are no whole blocks
        dict(name="fp8_m7_k320", op="fp8", M=7, K=320, N=2560, fn="none"),
        # a ragged mid-size batch
        dict(name="fp8_m100_k4096", op="fp8", M=100, K=4096, N=4096, fn="none"),
        # shared expert's down projection in a prefill chunk
        dict(name="fp8_m4096_k2048", op="fp8", M=4096, K=2048, N=4096, fn="none"),
        # shared expert's gate and up in a long prefill, clamped activation
        dict(name="fp8_m8192_gated", op="fp8", M=8192, K=7168, N=2048, fn="swigluoai"),
        # the norm before the block, one token
        dict(name="norm_m1_pre", op="norm", M=1, H=7168, residual="bf16", weight="bf16", branch=0, post=False,
             gate="none", gate_sigmoid=False, pre=True, residual_scale=1.0, branch_scale=1.0, offset=0.0),
        # norm after a block with a gate per channel, then the next block's norm, prefill chunk
        dict(name="norm_m4096_post_pre", op="norm", M=4096, H=4096, residual="bf16", weight="bf16", branch=1,
             post=True, gate="channel", gate_sigmoid=False, pre=True, residual_scale=1.0, branch_scale=0.5,
             offset=1.0),
        # routed and shared expert outputs summed, gated per token, onto an fp32 residual, long prefill
        dict(name="norm_m16384_fp32", op="norm", M=16384, H=7168, residual="fp32", weight="fp32", branch=2,
             post=True, gate="token", gate_sigmoid=True, pre=True, residual_scale=0.75, branch_scale=1.0,
             offset=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "fp8", "norm"])
    if op == "route":
        M, H = _log(rng, 1, 16384), 32 * _log(rng, 8, 224)
        groups = rng.choice([1, 1, 4, 8])
        E = groups * max(4, _log(rng, 8, 512) // groups)
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(16, top_groups * (E // groups)))
        # a call costs no more than the largest listed one
        M = max(1, min(M, 16384 * 7168 * 256 // (H * max(E, 256))))
        return dict(op="route", M=M, H=H, E=E, k=k, weight=rng.choice(["bf16", "bf16", "fp32"]),
                    scoring=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                    top_groups=top_groups, renorm=rng.random() < 0.7, scale=rng.choice([1.0, 1.5, 2.0]),
                    logits=rng.random() < 0.3)
    if op == "fp8":
        M, K, N = _log(rng, 1, 8192), 8 * _log(rng, 16, 896), 8 * _log(rng, 16, 896)
        fn = rng.choice(["none", "none", "silu", "gelu_tanh", "swigluoai", "relu2"])
        wide = 1 if fn in ("none", "relu2") else 2
        M = max(1, min(M, 8192 * 7168 * 4096 // (K * N * wide)))
        return dict(op="fp8", M=M, K=K, N=N, fn=fn)
    M, H = _log(rng, 1, 16384), 8 * _log(rng, 16, 1024)
    M = max(1, min(M, 16384 * 7168 // (2 * H)))
    branch = rng.choice([0, 1, 1, 2])
    return dict(op="norm", M=M, H=H, residual=rng.choice(["bf16", "fp32"]), weight=rng.choice(["bf16", "fp32"]),
                branch=branch, post=branch > 0 and rng.random() < 0.7,
                gate=rng.choice(["none", "channel", "token", "full"]) if branch else "none",
                gate_sigmoid=rng.random() < 0.5, pre=branch == 0 or rng.random() < 0.7,
                residual_scale=rng.choice([1.0, 0.75]), branch_scale=rng.choice([1.0, 0.5]),
                offset=rng.choice([0.0, 1.0]))


# ---------------------------------------------------------------- inputs

def _type(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _hidden(g, M, H):
    """Normed hidden states: unit variance with a spread over channels and a few large ones."""
    channel = torch.exp(0.4 * _normal(g, H))
    channel[torch.randint(0, H, (max(1, H // 512),), generator=g, device=DEV)] *= 8.0
    return (_normal(g, M, H) * channel).to(torch.bfloat16)


def _act(case):
    return (1.702, 1.0, 7.0) if case["fn"] == "swigluoai" else (0.0, 0.0, 0.0)


def _rows(case):
    return case["N"] if case["fn"] in ("none", "relu2") else 2 * case["N"]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "route":
        M, H, E = case["M"], case["H"], case["E"]
        s["x"] = _hidden(g, M, H)
        s["w"] = (_normal(g, E, H) / math.sqrt(2.0 * H)).to(_type(case["weight"]))
        s["bias"] = 0.05 * _normal(g, E) if case["bias"] else None
        if own:
            from block_scaled_fp4_gather_amd import block

            desc = block.RouterDesc(E, H, case["k"], max_tokens=M, weight=case["weight"], scoring=case["scoring"],
                                    groups=case["groups"], top_groups=case["top_groups"], renorm=case["renorm"],
                                    scale=case["scale"])
            s["router"] = block.Router(desc, s["w"], bias=s["bias"])
    elif case["op"] == "fp8":
        M, K, N, R = case["M"], case["K"], case["N"], _rows(case)
        halves, nb, kb = R // N, -(-N // BLOCK), -(-K // BLOCK)
        s["x"] = _hidden(g, M, K)
        w = torch.zeros(halves, nb * BLOCK, kb * BLOCK, device=DEV)
        w[:, :N, :K] = _normal(g, halves, N, K) * torch.exp(0.3 * _normal(g, halves, N, 1)) / math.sqrt(K)
        blocks = w.view(halves, nb, BLOCK, kb, BLOCK)
        scale = blocks.abs().amax(dim=(2, 4)).clamp_min(1e-12) / FP8_MAX
        codes = (blocks / scale[:, :, None, :, None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
        codes = codes.view(torch.uint8).view(halves, nb * BLOCK, kb * BLOCK)[:, :N, :K]
        s["codes"] = codes.reshape(R, K).contiguous()          # E4M3 bytes; gated: gate rows, then up rows
        s["scales"] = scale.reshape(halves * nb, kb).contiguous()  # a block row per 128 rows of each half
        if own:
            from block_scaled_fp4_gather_amd import block

            alpha, beta, limit = _act(case)
            desc = block.Fp8Desc(K, N, max_tokens=M, fn=case["fn"], alpha=alpha, beta=beta, limit=limit)
            s["linear"] = block.Fp8Linear(desc, s["codes"], s["scales"])
    else:
        M, H = case["M"], case["H"]
        wt = _type(case["weight"])
        s["h"] = (1.7 * _hidden(g, M, H).float()).to(_type(case["residual"]))
        s["y"] = (0.3 * _hidden(g, M, H).float()).to(torch.bfloat16) if case["branch"] >= 1 else None
        s["y2"] = (0.2 * _hidden(g, M, H).float()).to(torch.bfloat16) if case["branch"] >= 2 else None
        shape = {"none": None, "channel": (H,), "token": (M, 1), "full": (M, H)}[case["gate"]]
        s["gate"] = None if shape is None else (1.0 + 0.3 * _normal(g, *shape)).to(wt)
        around = 1.0 - case["offset"]
        s["post"] = (around + 0.2 * _normal(g, H)).to(wt) if case["post"] else None
        s["pre"] = (around + 0.2 * _normal(g, H)).to(wt) if case["pre"] else None
    return s


# ---------------------------------------------------------------- the framework's calls

def _run_own(s):
    from block_scaled_fp4_gather_amd import block

    c = s["case"]
    if c["op"] == "route":
        if c["logits"]:
            logits = torch.empty((c["M"], c["E"]), dtype=torch.float32, device=DEV)
            ids, w = s["router"](s["x"], logits=logits)
            return dict(ids=ids, w=w, logits=logits)
        ids, w = s["router"](s["x"])
        return dict(ids=ids, w=w)
    if c["op"] == "fp8":
        return dict(y=s["linear"](s["x"]))
    h, x = block.block_norm(s["h"], s["y"], s["y2"], gate=s["gate"], post_weight=s["post"], pre_weight=s["pre"],
                            eps=1e-6, residual_scale=c["residual_scale"], branch_scale=c["branch_scale"],
                            weight_offset=c["offset"], gate_sigmoid=c["gate_sigmoid"])
    return dict(h=h, x=x)


# ---------------------------------------------------------------- plain forms

def _run_route(s):
    """Scores in 64 bits: which experts are taken turns on differences far below what 32 bits keep of a sum over H."""
    c = s["case"]
    M, E, k = c["M"], c["E"], c["k"]
    logits = s["x"].double() @ s["w"].double().t()
    e = torch.exp(logits - logits.amax(1, keepdim=True))
    p = e / e.sum(1, keepdim=True) if c["scoring"] == "softmax" else 1.0 / (1.0 + torch.exp(-logits))
    biased = p + s["bias"].double() if s["bias"] is not None else p
    order = biased if s["bias"] is not None else logits
    if c["groups"] > 1:
        per = E // c["groups"]
        top2 = biased.view(M, c["groups"], per).sort(dim=2, descending=True)[0][..., :2].sum(2)
        taken = top2.sort(dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        keep = torch.zeros(M, c["groups"], dtype=torch.bool, device=DEV).scatter_(1, taken, True)
        order = order.masked_fill(~keep.repeat_interleave(per, 1), -math.inf)
    ids = order.sort(dim=1, descending=True, stable=True)[1][:, :k]
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    out = dict(ids=ids.to(torch.int32), w=(w * c["scale"]).float())
    if c["logits"]:
        out["logits"] = logits.float()
    return out


def _quantised(x):
    """x rounded to E4M3 with one power-of-two scale per 128 values: the least one that brings the block within 448."""
    M, K = x.shape
    b = torch.nn.functional.pad(x.float(), (0, -K % BLOCK)).view(M, -1, BLOCK)
    bits = b.abs().amax(2, keepdim=True).view(torch.int32)
    # amax = (1 + m 2^-23) 2^(e - 127) and 448 = 1.75 2^8: the scale's biased exponent is e - 8, or one more past 1.75
    byte = torch.clamp((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000), min=0)
    inverse = ((254 - byte) << 23).view(torch.float32)
    return ((b * inverse).to(torch.float8_e4m3fn).float() / inverse).view(M, -1)[:, :K]


def _activation(c, g, u):
    if c["fn"] == "silu":
        return g / (1.0 + torch.exp(-g)) * u
    if c["fn"] == "gelu_tanh":
        return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g))) * u
    alpha, beta, limit = _act(c)
    g, u = g.clamp(max=limit), u.clamp(-limit, limit)
    return g / (1.0 + torch.exp(-alpha * g)) * (u + beta)


def _run_fp8(s):
    c = s["case"]
    N, K, R = c["N"], c["K"], _rows(c)
    up = s["scales"].view(R // N, -1, s["scales"].shape[1]).repeat_interleave(BLOCK, 1)[:, :N]
    up = up.repeat_interleave(BLOCK, 2)[:, :, :K].reshape(R, K)
    w = s["codes"].view(torch.float8_e4m3fn).float() * up
    y = _quantised(s["x"]) @ w.t()
    if c["fn"] == "relu2":
        y = y.clamp(min=0.0) ** 2
    elif c["fn"] != "none":
        y = _activation(c, y[:, :N], y[:, N:])
    return dict(y=y.to(torch.bfloat16))


def _rms(v, weight, offset):
    n = v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6)
    return n * (weight.float() + offset)


def _run_norm(s):
    c = s["case"]
    h = s["h"]
    out = dict(h=None, x=None)
    if c["branch"]:
        b = s["y"].float() + s["y2"].float() if c["branch"] > 1 else s["y"].float()
        if c["post"]:
            b = _rms(b, s["post"], c["offset"])
        if s["gate"] is not None:
            gate = s["gate"].float()
            b = b * (1.0 / (1.0 + torch.exp(-gate)) if c["gate_sigmoid"] else gate)
        h = (c["residual_scale"] * h.float() + c["branch_scale"] * b).to(h.dtype)
        out["h"] = h
    if c["pre"]:
        out["x"] = _rms(h.float(), s["pre"], c["offset"]).to(torch.bfloat16)
    return out


def run(state):
    if own:
        return _run_own(state)
    return {"route": _run_route, "fp8": _run_fp8, "norm": _run_norm}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_route(c, s):
    M, E, G = c["M"], c["E"], c["groups"]
    z = torch.einsum("mh,eh->me", s["x"].to(torch.float64), s["w"].to(torch.float64))
    if c["scoring"] == "softmax":
        p = torch.softmax(z, dim=-1)
    else:
        p = torch.sigmoid(z)
    t = p.clone()
    if s["bias"] is not None:
        t = t + s["bias"].to(torch.float64)[None]
    rank = t if s["bias"] is not None else z
    if G > 1:
        best = torch.topk(t.reshape(M, G, E // G), 2, dim=2).values.sum(-1)
        floor = torch.topk(best, c["top_groups"], dim=1).values[:, -1:]
        rank = torch.where((best >= floor)[:, :, None].expand(M, G, E // G).reshape(M, E), rank,
                           torch.full_like(rank, -torch.inf))
    ids = torch.topk(rank, c["k"], dim=1, sorted=True).indices
    w = torch.take_along_dim(p, ids, dim=1)
    w = c["scale"] * (w / w.sum(-1, keepdim=True) if c["renorm"] else w)
    out = dict(ids=ids.to(torch.int32), w=w)
    if c["logits"]:
        out["logits"] = z
    return out


def _power_of_two(n):
    return ((n.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_fp8(c, s):
    M, K, N, R = c["M"], c["K"], c["N"], _rows(c)
    kb = -(-K // BLOCK)
    x = torch.zeros(M, kb * BLOCK, dtype=torch.float64, device=DEV)
    x[:, :K] = s["x"].to(torch.float64)
    x = x.reshape(M, kb, BLOCK)
    top = x.abs().max(dim=2, keepdim=True).values
    part, n = torch.frexp(top / FP8_MAX)  # top / 448 = part 2^n with part in [0.5, 1)
    step = _power_of_two(torch.where(part > 0.5, n, n - 1).clamp(min=-127))  # the least one with top <= 448 step
    # E4M3: 4 significant bits, steps of 2^-9 below 2^-6, to the nearest, halves to even
    v = x / step
    ulp = _power_of_two(torch.frexp(v.abs().clamp(min=2.0 ** -6)).exponent - 4)
    x = (torch.round(v / ulp) * ulp * step).reshape(M, kb * BLOCK)[:, :K]
    w = s["codes"].view(torch.float8_e4m3fn).to(torch.float64)
    of_row = (torch.arange(R, device=DEV) // N) * (-(-N // BLOCK)) + (torch.arange(R, device=DEV) % N) // BLOCK
    of_col = torch.arange(K, device=DEV) // BLOCK
    w = w * s["scales"].to(torch.float64)[of_row][:, of_col]
    y = torch.mm(x, w.T)
    if c["fn"] == "relu2":
        y = torch.where(y > 0, y * y, torch.zeros_like(y))
    elif c["fn"] == "silu":
        y = y[:, :N] * torch.sigmoid(y[:, :N]) * y[:, N:]
    elif c["fn"] == "gelu_tanh":
        y = torch.nn.functional.gelu(y[:, :N], approximate="tanh") * y[:, N:]
    elif c["fn"] == "swigluoai":
        alpha, beta, limit = _act(c)
        gate, lin = torch.clamp_max(y[:, :N], limit), torch.clamp(y[:, N:], min=-limit, max=limit)
        y = gate * torch.sigmoid(alpha * gate) * (lin + beta)
    return dict(y=y)


def _exact_norm(c, s):
    def normed(v, weight):
        return v / torch.sqrt(torch.sum(v ** 2, dim=-1, keepdim=True) / v.shape[-1] + 1e-6) * (
            weight.to(torch.float64) + c["offset"])

    h, out = s["h"].to(torch.float64), dict(h=None, x=None)
    if c["branch"]:
        b = s["y"].to(torch.float64)
        if s["y2"] is not None:
            b = b + s["y2"].to(torch.float64)
        if s["post"] is not None:
            b = normed(b, s["post"])
        if s["gate"] is not None:
            gate = s["gate"].to(torch.float64)
            b = (torch.sigmoid(gate) if c["gate_sigmoid"] else gate) * b
        h = c["residual_scale"] * h + c["branch_scale"] * b
        out["h"] = h
        h = h.to(_type(c["residual"])).to(torch.float64)  # the next norm reads the residual as it is stored
    if s["pre"] is not None:
        out["x"] = normed(h, s["pre"])
    return out


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"route": _exact_route, "fp8": _exact_fp8, "norm": _exact_norm}[case["op"]](case, s)


def work(case):
    """Bytes: each input once, each output once.  Flops: the products' multiply-adds, or the norm's per value."""
    M = case["M"]
    if case["op"] == "route":
        H, E = case["H"], case["E"]
        wb = 2 if case["weight"] == "bf16" else 4
        by = 2 * M * H + wb * E * H + 8 * M * case["k"] + (4 * E if case["bias"] else 0)
        return dict(bytes=by + (4 * M * E if case["logits"] else 0), flops=2 * M * E * H)
    if case["op"] == "fp8":
        K, N, R = case["K"], case["N"], _rows(case)
        blocks = (R // N) * -(-N // BLOCK) * -(-K // BLOCK)
        return dict(bytes=2 * M * K + R * K + 4 * blocks + 2 * M * N, flops=2 * M * R * K)
    H = case["H"]
    rb, wb = (2 if case["residual"] == "bf16" else 4), (2 if case["weight"] == "bf16" else 4)
    by = M * H * (rb + 2 * case["branch"] + (rb if case["branch"] else 0) + (2 if case["pre"] else 0))
    by += H * wb * (int(case["post"]) + int(case["pre"]))
    by += wb * {"none": 0, "channel": H, "token": M, "full": M * H}[case["gate"]]
    return dict(bytes=by, flops=M * H * (4 + 6 * int(case["branch"] > 0)))
