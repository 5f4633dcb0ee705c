"""64-bit references of FP4 quantisation, the MXFP4 linear map, grouped
products and the routes' grouping, written from their definitions in
include/moe_fp4.h, on the CPU."""
from __future__ import annotations

import math

import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()  # bytes 0 to 0x7E


def nearest(v, table):
    """Index of the nearest entry of an ascending table, a value between two to
    the even index, past the last to the last."""
    mids = (table[1:] + table[:-1]) / 2
    v = v.contiguous()
    upto, below = torch.bucketize(v, mids, right=True), torch.bucketize(v, mids)
    return torch.where(upto % 2 == 0, upto, below)


def pack(nibbles):
    return (nibbles[..., 0::2] | nibbles[..., 1::2] << 4).to(torch.uint8)


def unpack(codes):
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    return torch.where(n > 7, -E2M1[n & 7], E2M1[n & 7])


def quantize(x, fmt, g=None):
    """codes, scale bytes and (NVFP4) global scales [E] of x [E][R][K]."""
    E, R, K = x.shape
    G = 32 if fmt == "mxfp4" else 16
    b = x.double().view(E, R, K // G, G)
    bad = ~torch.isfinite(b).all(-1)
    safe = torch.where(bad[..., None], torch.zeros_like(b), b)
    amax = safe.abs().amax(-1)
    if fmt == "mxfp4":
        e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, torch.full_like(amax, -127, dtype=torch.int32)).clamp(min=-127)
        byte = torch.where(bad, torch.full_like(e, 255), e + 127)
        unit = torch.ldexp(torch.ones_like(amax), e)
    else:
        if g is None:
            finite = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).double()
            g = (finite.abs().amax((1, 2)) / 2688).float()
        gd = g.double().view(E, 1, 1)
        ok = torch.isfinite(gd) & (gd >= 0)
        six = torch.where(ok & (gd > 0), 6 * gd, torch.ones_like(gd))
        byte = torch.where(ok & (gd > 0), nearest(amax / six, E4M3), torch.zeros_like(amax, dtype=torch.int64))
        unit = E4M3[byte] * gd
        byte = torch.where(bad | ~ok, torch.full_like(byte, 0x7F), byte)
        bad = bad | ~ok
    u = torch.where(unit > 0, unit, torch.ones_like(unit))[..., None]
    v = torch.where(unit[..., None] > 0, safe / u, torch.zeros_like(safe))
    code = nearest(v.abs(), E2M1)
    # a value that is given no scale has no sign either; a negative one that rounds to zero keeps its own
    sign = torch.signbit(safe) & (unit[..., None] > 0)
    code = torch.where(bad[..., None], torch.full_like(code, 7), code | sign.long() << 3)
    return pack(code.view(E, R, K)), byte.view(E, R, -1).to(torch.uint8), g


def scale_values(scales, fmt):
    s = scales.long()
    if fmt == "mxfp4":
        return torch.where(s == 255, torch.full(s.shape, math.nan, dtype=torch.float64),
                           torch.ldexp(torch.ones(s.shape, dtype=torch.float64), s - 127))
    return torch.cat([E4M3, torch.tensor([math.nan], dtype=torch.float64)])[s]


def dequantize(codes, scales, fmt, g=None):
    """Values in 64 bits, the global scale not applied."""
    G = 32 if fmt == "mxfp4" else 16
    return unpack(codes) * scale_values(scales, fmt).repeat_interleave(G, -1)


def linear(xc, xs, wc, ws):
    """Products and, of their magnitudes, the sum."""
    x, w = dequantize(xc, xs, "mxfp4"), dequantize(wc, ws, "mxfp4")
    return x @ w.t(), x.abs() @ w.abs().t()


def group(ids, E):
    M, k = ids.shape
    flat = ids.flatten().tolist()
    rows = [r for e in range(E) for r in range(M * k) if flat[r] == e]
    offsets = [0]
    for e in range(E):
        offsets.append(offsets[-1] + sum(1 for v in flat if v == e))
    order = rows + [-1] * (M * k - len(rows))
    place = [-1] * (M * k)
    for p, r in enumerate(rows):
        place[r] = p
    i32 = torch.int32
    return (torch.tensor(offsets, dtype=i32), torch.tensor(order, dtype=i32),
            torch.tensor(place, dtype=i32).view(M, k))


def grouped(x, w, offsets):
    """y of x [T][K] and w [E][N][K], and the sum of the terms' magnitudes."""
    T, E, N = x.shape[0], w.shape[0], w.shape[1]
    y, s = torch.zeros(T, N, dtype=torch.float64), torch.zeros(T, N, dtype=torch.float64)
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        xe, we = x[a:b].double(), w[e].double()
        y[a:b], s[a:b] = xe @ we.t(), xe.abs() @ we.abs().t()
    return y, s


def grouped_grad(dy, x, offsets):
    E = len(offsets) - 1
    dw = torch.zeros(E, dy.shape[1], x.shape[1], dtype=torch.float64)
    s = torch.zeros_like(dw)
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        d, xe = dy[a:b].double(), x[a:b].double()
        dw[e], s[e] = d.t() @ xe, d.abs().t() @ xe.abs()
    return dw, s
