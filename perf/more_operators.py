"""Operators from 16 and 32 bits to the FP4 experts and around them, case by
case: the block-scaled 4-bit quantisation that makes the layer's weights, the
linear map over MXFP4 weights and MXFP4 activations, the products grouped by
expert over ragged rows with their gradients, and the grouping, gathering and
weighted joining of the routes that go with them.

``run`` computes a case in elementary torch operations, or, with ``own`` set,
with this package's kernels.  ``exact`` gives the values of the definition in
64 bits.  Shapes are those of the package's workloads (H 2560 / 4096 / 7168,
I 256 / 320 / 1536, E 128 / 256 / 512) or powers of two next to them.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
GROUP = {"mxfp4": 32, "nvfp4": 16}


def listed():
    return [
        # one token's hidden state to MXFP4 and back: latency alone
        dict(name="quant_mxfp4_m1", op="quant", fmt="mxfp4", E=1, R=1, K=7168, dtype="bf16"),
        # fp32 master weights of some experts to NVFP4, a global scale per expert, and back (a check of what it costs)
        dict(name="quant_nvfp4_e64_fp32", op="quant", fmt="nvfp4", E=64, R=640, K=2560, dtype="fp32"),
        # hidden states of a long prefill to MXFP4 and back
        dict(name="quant_mxfp4_m16384", op="quant", fmt="mxfp4", E=1, R=16384, K=7168, dtype="bf16"),
        # shared expert's gate and up for one token: the weights are read once
        dict(name="fp4_m1_gated", op="fp4", M=1, K=7168, N=2048, fn="silu", given=False),
        # small projection of a ragged decode batch, widths that are no whole blocks
        dict(name="fp4_m37_k320", op="fp4", M=37, K=320, N=2560, fn="none", given=False),
        # mid-size batch whose quantised form is there already (several maps of the same tokens)
        dict(name="fp4_m512_k4096_given", op="fp4", M=512, K=4096, N=4096, fn="none", given=True),
        # shared expert's gate and up in a long prefill, clamped activation
        dict(name="fp4_m8192_gated", op="fp4", M=8192, K=7168, N=2048, fn="swigluoai", given=False),
        # one token through its 8 experts' gate and up in bf16: weights of 8 of 256 experts
        dict(name="grouped_decode_e256", op="grouped", tokens=1, k=8, E=256, K=7168, N=512, mode="forward", dead=0),
        # forward and backward of a small ragged batch, some rows of it in no group
        dict(name="grouped_train_e32", op="grouped", tokens=515, k=4, E=32, K=2560, N=640, mode="train", dead=45),
        # forward and backward of the down projection, a training batch over 128 experts
        dict(name="grouped_train_e128", op="grouped", tokens=4096, k=8, E=128, K=1536, N=4096, mode="train", dead=0),
        # routes of one token: grouped, gathered and joined
        dict(name="routes_m1_e256", op="routes", M=1, k=8, E=256, H=7168, train=False, invalid=0.0),
        # routes of a training batch, with the gradients of hidden states, expert outputs and weights
        dict(name="routes_m4096_e128", op="routes", M=4096, k=8, E=128, H=4096, train=True, invalid=0.02),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "fp4", "fp4", "grouped", "grouped", "routes"])
    if op == "quant":
        E, K = rng.choice([1, 1, _log(rng, 2, 64)]), 32 * _log(rng, 4, 256)
        R = max(1, min(_log(rng, 1, 16384), 16384 * 7168 // (2 * E * K)))
        return dict(op="quant", fmt=rng.choice(["mxfp4", "nvfp4"]), E=E, R=R, K=K, dtype=rng.choice(["bf16", "fp32"]))
    if op == "fp4":
        M, K, N = _log(rng, 1, 8192), 32 * _log(rng, 4, 224), 8 * _log(rng, 16, 896)
        fn = rng.choice(["none", "none", "silu", "gelu_tanh", "swigluoai", "relu2"])
        # a call costs no more than the largest listed one
        M = max(1, min(M, 8192 * 7168 * 4096 // (K * N * _halves(fn))))
        return dict(op="fp4", M=M, K=K, N=N, fn=fn, given=rng.random() < 0.3)
    if op == "grouped":
        E, k = _log(rng, 1, 256), 1
        k = rng.randint(1, min(8, E))
        K, N = 8 * _log(rng, 16, 896), 8 * _log(rng, 16, 512)
        tokens = _log(rng, 1, 4096)
        tokens = max(1, min(tokens, 4096 * 8 * 1536 * 4096 // (k * K * N)))
        E = max(k, min(E, 128 * 1536 * 4096 // (K * N)))
        return dict(op="grouped", tokens=tokens, k=k, E=E, K=K, N=N,
                    mode=rng.choice(["forward", "train", "train", "weight_fp32"]),
                    dead=rng.choice([0, 0, _log(rng, 1, 64)]))
    E = _log(rng, 4, 512)
    k, H = rng.randint(1, min(10, E)), 8 * _log(rng, 16, 896)
    M = max(1, min(_log(rng, 1, 8192), 4096 * 8 * 4096 // (k * H)))
    return dict(op="routes", M=M, k=k, E=E, H=H, train=rng.random() < 0.5, invalid=rng.choice([0.0, 0.05]))


# ---------------------------------------------------------------- inputs

def _type(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def _halves(fn):
    return 1 if fn in ("none", "relu2") else 2


def _act(case):
    return (1.702, 1.0, 7.0) if case["fn"] == "swigluoai" else (0.0, 0.0, 0.0)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _hidden(g, M, H):
    """Normed hidden states: unit variance with a spread over channels and a few large ones."""
    channel = torch.exp(0.4 * _normal(g, H))
    channel[torch.randint(0, H, (max(1, H // 512),), generator=g, device=DEV)] *= 8.0
    return (_normal(g, M, H) * channel).to(torch.bfloat16)


def _ids(g, M, k, E):
    """k distinct experts per token, some experts more loved than others."""
    return (_normal(g, M, E) + 0.5 * _normal(g, E)).topk(k, dim=1).indices.to(torch.int32)


def _codes(g, rows, K):
    """MXFP4 weights as checkpoints hold them: E2M1 nibbles and a scale byte per 32."""
    codes = torch.randint(0, 256, (rows, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    middle = 125 - int(math.log2(math.sqrt(K) * 2.5))
    scales = torch.randint(middle - 1, middle + 2, (rows, K // 32), generator=g, device=DEV, dtype=torch.uint8)
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "quant":
        E, R, K = case["E"], case["R"], case["K"]
        shape = (E, R, K) if E > 1 else (R, K)
        if case["dtype"] == "fp32":
            scale = torch.exp(0.3 * _normal(g, E * R, 1)) * 0.02
            s["x"] = (_normal(g, E * R, K) * scale).view(shape)
        else:
            s["x"] = _hidden(g, E * R, K).view(shape)
    elif case["op"] == "fp4":
        M, K, N = case["M"], case["K"], case["N"]
        s["codes"], s["scales"] = _codes(g, _halves(case["fn"]) * N, K)
        s["x"] = _hidden(g, M, K)
        if case["given"]:
            q, byte = _mxfp4(s["x"].float())
            nibble = _nibbles(q)
            s["given"] = (nibble[:, 0::2] | nibble[:, 1::2] << 4), byte.to(torch.uint8)
        if own:
            from block_scaled_fp4_gather_amd import experts

            alpha, beta, limit = _act(case)
            desc = experts.Fp4Desc(K, N, max_tokens=M, fn=case["fn"], alpha=alpha, beta=beta, limit=limit)
            s["linear"] = experts.Fp4Linear(desc, s["codes"], s["scales"])
    elif case["op"] == "grouped":
        E, K, N, k = case["E"], case["K"], case["N"], case["k"]
        rows = case["tokens"] * k
        counts = torch.bincount(_ids(g, case["tokens"], k, E).flatten(), minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["x"] = _hidden(g, rows + case["dead"], K)
        s["dy"] = (0.1 * _normal(g, rows + case["dead"], N)).to(torch.bfloat16)
        if case["mode"] != "weight_fp32":
            s["w"] = torch.empty(E, N, K, device=DEV, dtype=torch.bfloat16)
            for e in range(E):
                s["w"][e] = _normal(g, N, K) / math.sqrt(K)
        if case["mode"] == "train":
            s["x"].requires_grad_()
            s["w"].requires_grad_()
    else:
        M, k, E, H = case["M"], case["k"], case["E"], case["H"]
        ids = _ids(g, M, k, E)
        lost = torch.rand(M, k, generator=g, device=DEV) < case["invalid"]
        s["ids"] = torch.where(lost, torch.full_like(ids, -1), ids)
        s["x"] = _hidden(g, M, H)
        s["y"] = _hidden(g, M * k, H)
        w = torch.rand(M, k, generator=g, device=DEV) + 0.05
        s["w"] = w / w.sum(1, keepdim=True)
        s["dxg"] = (0.1 * _normal(g, M * k, H)).to(torch.bfloat16)
        s["dout"] = (0.1 * _normal(g, M, H)).to(torch.bfloat16)
        if case["train"]:
            for name in ("x", "y", "w"):
                s[name].requires_grad_()
    return s


# ---------------------------------------------------------------- the framework's calls

def _run_own(s):
    from block_scaled_fp4_gather_amd import experts

    c = s["case"]
    if c["op"] == "quant":
        q = experts.fp4_quantize(s["x"], c["fmt"])
        out = dict(values=experts.fp4_dequantize(q, c["fmt"], dtype=s["x"].dtype))
        if c["fmt"] == "nvfp4":
            out["global_scale"] = q.global_scale
        return out
    if c["op"] == "fp4":
        return dict(y=s["linear"](quantized=s["given"]) if c["given"] else s["linear"](s["x"]))
    if c["op"] == "grouped":
        if c["mode"] == "weight_fp32":
            return dict(dw=experts.grouped_weight_grad(s["dy"], s["x"], s["offsets"], dtype=torch.float32))
        y = experts.grouped_linear(s["x"], s["w"], s["offsets"])
        if c["mode"] == "forward":
            return dict(y=y)
        dx, dw = torch.autograd.grad(y, (s["x"], s["w"]), s["dy"])
        return dict(y=y.detach(), dx=dx, dw=dw)
    groups = experts.group_routes(s["ids"], c["E"])
    xg = experts.gather_routes(s["x"], groups)
    out = experts.combine_routes(s["y"], groups, s["w"])
    r = dict(offsets=groups.offsets, order=groups.order, place=groups.place, xg=xg.detach(), out=out.detach())
    if c["train"]:
        (r["dx"],) = torch.autograd.grad(xg, (s["x"],), s["dxg"])
        r["dy"], r["dw"] = torch.autograd.grad(out, (s["y"], s["w"]), s["dout"])
    return r


# ---------------------------------------------------------------- plain forms

def _e2m1(a):
    """Magnitudes rounded to nearest-even E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6), at most 6."""
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).to(a.dtype)
    return (torch.round(a / step) * step).clamp(max=6.0)


def _mxfp4(x):
    """Blocks of 32 of x (fp32) in MXFP4: values over their scale, and the scale bytes."""
    b = x.view(*x.shape[:-1], -1, 32)
    # 2^(floor(log2 amax) - 2): its byte is amax's exponent field less 2
    byte = ((b.abs().amax(-1).view(torch.int32) >> 23) - 2).clamp(min=0)
    v = torch.ldexp(b.double(), (127 - byte)[..., None])
    return (torch.sign(v) * _e2m1(v.abs())).view(x.shape), byte


def _nibbles(q):
    """E2M1 codes of values."""
    a = q.abs()
    return (torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
            | (torch.signbit(q).to(torch.uint8) << 3))


def _e4m3(v):
    """Non-negative v (64 bits) rounded to nearest-even E4M3, at most 448."""
    step = torch.exp2((torch.frexp(v)[1].clamp(min=-5) - 4).double())
    return (torch.round(v / step) * step).clamp(max=448.0)


def _run_quant(s):
    c, x = s["case"], s["x"]
    if c["fmt"] == "mxfp4":
        q, byte = _mxfp4(x.float())
        scale = torch.exp2((byte - 127).double())[..., None]
        return dict(values=(q.view(*byte.shape, 32) * scale).view(x.shape).to(x.dtype))
    b = x.double().view(c["E"], c["R"], -1, 16)
    g = (b.abs().amax((1, 2, 3)) / (6 * 448)).float()
    whole = g.double()[:, None, None]
    scale = _e4m3(b.abs().amax(-1) / (6 * whole))
    unit = (scale * whole)[..., None]
    v = torch.where(unit > 0, b / unit, torch.zeros_like(b))
    q = torch.sign(v) * _e2m1(v.abs())
    # code times block scale is exact in 32 bits, the global scale rounds it
    values = (q * scale[..., None]).float() * g[:, None, None, None]
    return dict(values=values.view(x.shape).to(x.dtype), global_scale=g)


def _e2m1_of_bytes(codes):
    nibble = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV)
    v = table[(nibble & 7).int()]
    return torch.where(nibble > 7, -v, v)


def _of_bytes(codes, scales):
    return _e2m1_of_bytes(codes) * torch.exp2(scales.float() - 127).repeat_interleave(32, 1)


def _activation(c, y):
    if c["fn"] == "none":
        return y
    if c["fn"] == "relu2":
        return y.clamp(min=0.0) ** 2
    g, u = y[:, :c["N"]], y[:, c["N"]:]
    if c["fn"] == "silu":
        return g / (1.0 + torch.exp(-g)) * u
    if c["fn"] == "gelu_tanh":
        return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g))) * u
    alpha, beta, limit = _act(c)
    g, u = g.clamp(max=limit), u.clamp(-limit, limit)
    return g / (1.0 + torch.exp(-alpha * g)) * (u + beta)


def _run_fp4(s):
    c = s["case"]
    if c["given"]:
        x = _of_bytes(*s["given"])
    else:
        q, byte = _mxfp4(s["x"].float())
        x = (q * torch.exp2((byte - 127).double()).repeat_interleave(32, 1)).float()
    y = x @ _of_bytes(s["codes"], s["scales"]).t()
    return dict(y=_activation(c, y).to(torch.bfloat16))


def _run_grouped(s):
    c = s["case"]
    E, N, K = c["E"], c["N"], c["K"]
    x, dy = s["x"].detach(), s["dy"]
    rows = x.shape[0]
    at = s["offsets"].tolist()
    mode = c["mode"]
    out = {}
    if mode != "weight_fp32":
        w = s["w"].detach()
        out["y"] = torch.zeros(rows, N, device=DEV, dtype=torch.bfloat16)
        if mode == "train":
            out["dx"] = torch.zeros(rows, K, device=DEV, dtype=torch.bfloat16)
    if mode != "forward":
        out["dw"] = torch.zeros(E, N, K, device=DEV, dtype=torch.bfloat16 if mode == "train" else torch.float32)
    for e in range(E):
        a, b = at[e], at[e + 1]
        if a == b:
            continue
        if mode != "weight_fp32":
            we = w[e].float()
            out["y"][a:b] = (x[a:b].float() @ we.t()).to(torch.bfloat16)
            if mode == "train":
                out["dx"][a:b] = (dy[a:b].float() @ we).to(torch.bfloat16)
        if mode != "forward":
            out["dw"][e] = (dy[a:b].float().t() @ x[a:b].float()).to(out["dw"].dtype)
    return out


def _run_routes(s):
    c = s["case"]
    M, k, E, H = c["M"], c["k"], c["E"], c["H"]
    R = M * k
    ids = s["ids"].flatten().long()
    ok = (ids >= 0) & (ids < E)
    key = torch.where(ok, ids, torch.full_like(ids, E))
    order = key.sort(stable=True)[1]
    counts = (key[:, None] == torch.arange(E, device=DEV)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    live = torch.arange(R, device=DEV) < offsets[-1]
    place = torch.empty_like(order)
    place[order] = torch.arange(R, device=DEV)
    place = torch.where(ok, place, torch.full_like(place, -1))
    order = torch.where(live, order, torch.full_like(order, -1))
    x, y, w = s["x"].detach(), s["y"].detach(), s["w"].detach()
    token = order.clamp(min=0) // k
    xg = torch.where(live[:, None], x[token], torch.zeros_like(x[:1]))
    okj, at = ok.view(M, k), place.clamp(min=0).view(M, k)
    acc = torch.zeros(M, H, device=DEV)
    for j in range(k):
        acc += torch.where(okj[:, j, None], w[:, j, None] * y[at[:, j]].float(), torch.zeros_like(acc[:1]))
    r = dict(offsets=offsets.to(torch.int32), order=order.to(torch.int32), place=place.view(M, k).to(torch.int32),
             xg=xg, out=acc.to(torch.bfloat16))
    if c["train"]:
        dx, dw = torch.zeros(M, H, device=DEV), torch.zeros(M, k, device=DEV)
        dout = s["dout"].float()
        for j in range(k):
            dx += torch.where(okj[:, j, None], s["dxg"][at[:, j]].float(), torch.zeros_like(dx[:1]))
            dw[:, j] = torch.where(okj[:, j], (dout * y[at[:, j]].float()).sum(1), torch.zeros_like(dw[:, j]))
        wr = w.flatten()[order.clamp(min=0)]
        r["dx"] = dx.to(torch.bfloat16)
        r["dy"] = torch.where(live[:, None], wr[:, None] * dout[token], torch.zeros_like(dout[:1])).to(torch.bfloat16)
        r["dw"] = dw
    return r


def run(state):
    if own:
        return _run_own(state)
    return {"quant": _run_quant, "fp4": _run_fp4, "grouped": _run_grouped,
            "routes": _run_routes}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definition in 64 bits

_MIDDLES = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
_VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _nearest_e2m1(v):
    """By counting the midpoints below a magnitude; a value on one goes to the even code."""
    mids = torch.tensor(_MIDDLES, dtype=torch.float64, device=DEV)
    a = v.abs().contiguous()
    below, upto = torch.bucketize(a, mids), torch.bucketize(a, mids, right=True)
    code = torch.where(upto % 2 == 0, upto, below)
    return torch.copysign(torch.tensor(_VALUES, dtype=torch.float64, device=DEV)[code], v)


def _power_below(a):
    """floor(log2 a) of positive 64-bit values."""
    return ((a.view(torch.int64) >> 52) & 2047) - 1023


def _pow2(n):
    return ((n + 1023) << 52).view(torch.float64)


def _exact_mx(x):
    """x [.., K] as the values of its MXFP4 form."""
    b = x.to(torch.float64).reshape(-1, 32)
    top = b.abs().max(1, keepdim=True).values
    step = _pow2(torch.where(top > 0, _power_below(top) - 2, torch.full_like(top, -127, dtype=torch.int64)).clamp(min=-127))
    return (_nearest_e2m1(b / step) * step).reshape(x.shape)


def _exact_quant(c, s):
    x = s["x"]
    if c["fmt"] == "mxfp4":
        return dict(values=_exact_mx(x))
    E = c["E"]
    flat = x.to(torch.float64).reshape(E, -1)
    g = (flat.abs().max(1).values / 2688.0).to(torch.float32)  # the scale that is stored has 32 bits
    blocks = flat.reshape(E, -1, 16)
    ratio = blocks.abs().max(2).values / (6.0 * g.to(torch.float64)[:, None])
    # E4M3: steps of an eighth of the power of two below, of 2^-9 under 2^-6
    ulp = _pow2(_power_below(ratio.clamp(min=2.0 ** -6)) - 3)
    scale = torch.minimum(torch.round(ratio / ulp) * ulp, torch.full_like(ratio, 448.0))
    unit = (scale * g.to(torch.float64)[:, None])[:, :, None]
    values = torch.where(unit > 0, _nearest_e2m1(blocks / unit.clamp(min=1e-300)) * unit, torch.zeros_like(blocks))
    return dict(values=values.reshape(x.shape), global_scale=g.to(torch.float64))


def _exact_bytes(codes, scales):
    n = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.int64, device=DEV)
    n[:, 0::2], n[:, 1::2] = codes % 16, codes // 16
    v = torch.tensor(_VALUES + [-v for v in _VALUES], dtype=torch.float64, device=DEV)[n]
    return (v.reshape(n.shape[0], -1, 32) * _pow2(scales.to(torch.int64) - 127)[:, :, None]).reshape(n.shape)


def _exact_fp4(c, s):
    N = c["N"]
    x = _exact_bytes(*s["given"]) if c["given"] else _exact_mx(s["x"])
    y = torch.mm(x, _exact_bytes(s["codes"], s["scales"]).T)
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


def _exact_grouped(c, s):
    """One expert at a time, rows taken by a mask."""
    rows = s["x"].shape[0]
    group = torch.bucketize(torch.arange(rows, device=DEV, dtype=torch.int32), s["offsets"][1:], right=True)
    x, dy = s["x"].detach().to(torch.float64), s["dy"].to(torch.float64)
    y = dx = dw = None
    if c["mode"] != "weight_fp32":
        y = torch.zeros(rows, c["N"], dtype=torch.float64, device=DEV)
    if c["mode"] == "train":
        dx = torch.zeros(rows, c["K"], dtype=torch.float64, device=DEV)
    if c["mode"] != "forward":
        dw = torch.zeros(c["E"], c["N"], c["K"], dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        mine = (group == e).nonzero().flatten()
        xe, ge = x[mine], dy[mine]
        if y is not None:
            we = s["w"][e].detach().to(torch.float64)
            y[mine] = torch.mm(xe, we.T)
            if dx is not None:
                dx[mine] = torch.mm(ge, we)
        if dw is not None:
            dw[e] = torch.mm(ge.T, xe)
    return {n: v for n, v in (("y", y), ("dx", dx), ("dw", dw)) if v is not None}


def _exact_routes(c, s):
    M, k, E = c["M"], c["k"], c["E"]
    R = M * k
    ids = s["ids"].reshape(-1).to(torch.int64)
    # an expert's routes in the order of their index: sorted by expert * R + index
    valid = (ids >= 0) & (ids < E)
    slots = torch.arange(R, device=DEV)
    listed_slots = (ids[valid] * R + slots[valid]).sort().values % R
    n = listed_slots.numel()
    order = torch.full((R,), -1, dtype=torch.int64, device=DEV)
    order[:n] = listed_slots
    place = torch.full((R,), -1, dtype=torch.int64, device=DEV)
    place[listed_slots] = slots[:n]
    offsets = torch.searchsorted(ids[listed_slots].contiguous(), torch.arange(E + 1, device=DEV))
    x, y = s["x"].detach().to(torch.float64), s["y"].detach().to(torch.float64)
    w = s["w"].detach().to(torch.float64).reshape(-1)
    xg = torch.zeros(R, c["H"], dtype=torch.float64, device=DEV)
    xg[:n] = x[listed_slots // k]
    out = torch.zeros_like(x).index_add_(0, listed_slots // k, y[:n] * w[listed_slots][:, None])
    r = dict(offsets=offsets.to(torch.int32), order=order.to(torch.int32), place=place.to(torch.int32).reshape(M, k),
             xg=xg, out=out)
    if c["train"]:
        dxg, dout = s["dxg"].to(torch.float64), s["dout"].to(torch.float64)
        r["dx"] = torch.zeros_like(x).index_add_(0, listed_slots // k, dxg[:n])
        r["dy"] = torch.zeros_like(y)
        r["dy"][:n] = dout[listed_slots // k] * w[listed_slots][:, None]
        dw = torch.zeros(R, dtype=torch.float64, device=DEV)
        dw[listed_slots] = (dout[listed_slots // k] * y[:n]).sum(1)
        r["dw"] = dw.reshape(M, k)
    return r


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    with torch.no_grad():
        return {"quant": _exact_quant, "fp4": _exact_fp4, "grouped": _exact_grouped,
                "routes": _exact_routes}[case["op"]](case, s)


def work(case):
    """Bytes: each input once, each output once.  Flops: the products' multiply-adds, or a few per value."""
    if case["op"] == "quant":
        n = case["E"] * case["R"] * case["K"]
        size = 4 if case["dtype"] == "fp32" else 2
        held = n // 2 + n // GROUP[case["fmt"]]
        # x read, codes and scales written, both read again, values written; NVFP4's global scale needs x once before
        return dict(bytes=n * size * (3 if case["fmt"] == "nvfp4" else 2) + 2 * held, flops=8 * n)
    if case["op"] == "fp4":
        M, K, N, R = case["M"], case["K"], case["N"], _halves(case["fn"]) * case["N"]
        x = M * (K // 2 + K // 32) if case["given"] else 2 * M * K
        return dict(bytes=x + R * (K // 2 + K // 32) + 2 * M * N, flops=2 * M * R * K)
    if case["op"] == "grouped":
        E, K, N, rows = case["E"], case["K"], case["N"], case["tokens"] * case["k"]
        T = rows + case["dead"]
        hit = E * (1.0 - (1.0 - case["k"] / E) ** case["tokens"])  # experts that get a row, expected
        by, products = 0, 0
        if case["mode"] != "weight_fp32":
            by += 2 * rows * K + 2 * hit * N * K + 2 * T * N
            products += 1
        if case["mode"] == "train":
            by += 2 * rows * N + 2 * hit * N * K + 2 * T * K + 2 * rows * (N + K) + 2 * E * N * K
            products += 2
        if case["mode"] == "weight_fp32":
            by += 2 * rows * (N + K) + 4 * E * N * K
            products += 1
        return dict(bytes=int(by), flops=2 * products * rows * K * N)
    M, k, H = case["M"], case["k"], case["H"]
    R = M * k
    by = 12 * R + 2 * M * H + 2 * R * H + 2 * R * H + 4 * R + 2 * M * H
    if case["train"]:  # gradients: dxg to dx; dout and y to dy and dw
        by += 2 * R * H + 2 * M * H + 2 * M * H + 4 * R * H + 8 * R
    return dict(bytes=by, flops=2 * R * H * (4 if case["train"] else 1))
