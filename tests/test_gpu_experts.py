"""FP4 quantisation, the MXFP4 linear map, products grouped by expert and the
routes' grouping against 64-bit references, and a layer made of them."""
from __future__ import annotations

import math

import pytest
import torch

import block_ref
import experts_ref as ref
from block_scaled_fp4_gather_amd import block, experts, moe
from gpu_util import say

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8  # half a step of bf16, relative
FP32 = 2.0 ** -24
NAN, INF = math.nan, math.inf


@pytest.fixture(autouse=True)
def _announce(request):
    say(f"\n[gpu] {request.node.nodeid}")
    yield


def rand(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g)


def spread(seed, *shape):
    """Values over many powers of two, blocks of zeros among them."""
    x = rand(seed, *shape) * torch.exp2(torch.round(3 * rand(seed + 1, *shape[:-1], 1)))
    x[..., : shape[-1] // 4] *= torch.exp2(torch.round(2 * rand(seed + 2, *shape[:-1], shape[-1] // 4)))
    flat = x.view(-1, 16)
    flat[::7] = 0.0
    return x


# ---------------------------------------------------------------- quantisation

@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 32), (5, 320), (3, 7, 96), (2, 130, 1056), (33, 4096)])
def test_quantize_bit_exact(fmt, dtype, shape):
    x = spread(1, *shape).to(dtype)
    q = experts.fp4_quantize(x.cuda(), fmt)
    x3 = x if x.dim() == 3 else x[None]
    codes, scales, g = ref.quantize(x3, fmt)
    assert torch.equal(q.scales.cpu().view(scales.shape), scales)
    assert torch.equal(q.codes.cpu().view(codes.shape), codes)
    if fmt == "nvfp4":
        assert torch.equal(q.global_scale.cpu(), g)
    else:
        assert q.global_scale is None


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_quantize_ties_and_ends(fmt):
    """Quotients on midpoints of E2M1, next to them by a unit in the last place,
    and magnitudes from the smallest subnormal to the largest number; with a
    global scale that is no power of two, one that is, and ends of fp32."""
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0])
    for g in ([None] if fmt == "mxfp4" else [0.7311, 0.5, 2.0 ** -100, 2.0 ** 100, 1e-40, 1e-3, 0.0]):
        rows = []
        for e in (-120, -40, 0, 3, 100):
            v = mids * 2.0 ** e * (1.0 if g is None else float(torch.tensor(g))) * (1.0 if g is None or e else 1.125)
            v = v.float()
            near = [v, torch.nextafter(v, torch.full_like(v, INF)), torch.nextafter(v, torch.zeros_like(v)), -v]
            row = torch.cat(near + [torch.zeros(64 - 4 * len(mids))])
            rows.append(row)
            top = torch.cat([row[:15], (6.0 * v[4] / mids[4]).view(1)] * 4)
            rows.append(top)
        rows.append(torch.tensor([1e-45, -1e-45, 3.4e38, 1e-38] * 16))
        rows.append(torch.tensor([1e-45, -1e-45, 0.0, 1e-42] * 16))
        x = torch.stack(rows)
        x = torch.where(torch.isfinite(x), x, torch.full_like(x, 3e38))
        gt = None if g is None else torch.tensor([g])
        q = experts.fp4_quantize(x.cuda(), fmt, None if gt is None else gt.cuda())
        codes, scales, _ = ref.quantize(x[None], fmt, gt)
        assert torch.equal(q.scales.cpu(), scales[0]), (fmt, g)
        assert torch.equal(q.codes.cpu(), codes[0]), (fmt, g)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_quantize_keeps_nan_and_infinity_in_their_block(fmt, dtype):
    x = rand(4, 2, 40, 128)
    x[0, 3, 17], x[0, 4, 100], x[1, 0, 0], x[1, 39, 127] = NAN, INF, -INF, NAN
    x[1, 7] = NAN
    x = x.to(dtype)
    q = experts.fp4_quantize(x.cuda(), fmt)
    codes, scales, g = ref.quantize(x, fmt)
    assert torch.equal(q.scales.cpu(), scales) and torch.equal(q.codes.cpu(), codes)
    back = experts.fp4_dequantize(q, fmt, torch.float32).cpu()
    assert int(torch.isnan(back).sum()) == int((scales == (255 if fmt == "mxfp4" else 127)).sum()) * experts.GROUP[fmt]
    if fmt == "nvfp4":
        assert torch.equal(q.global_scale.cpu(), g)
        for bad in (-1.0, NAN, INF):
            q = experts.fp4_quantize(x.cuda(), fmt, torch.tensor([1.0, bad]).cuda())
            assert bool((q.scales[1] == 0x7F).all()) and bool((q.codes[1] == 0x77).all())
            assert bool((q.scales[0] != 0x7F).any())


def test_quantize_strides_and_empty():
    whole = rand(5, 3, 10, 256).bfloat16().cuda()
    part = whole[:, :, 64:160]
    for fmt in ("mxfp4", "nvfp4"):
        got, want = experts.fp4_quantize(part, fmt), experts.fp4_quantize(part.contiguous(), fmt)
        assert all(a is None or torch.equal(a, b) for a, b in zip(got, want))
        row, want = experts.fp4_quantize(whole[1, 4:5, 32:64], fmt), experts.fp4_quantize(whole[1, 4:5, 32:64].contiguous(), fmt)
        assert torch.equal(row.codes, want.codes)
        q = experts.fp4_quantize(whole[:, :0], fmt)
        assert q.codes.shape == (3, 0, 128) and experts.fp4_dequantize(q, fmt).shape == (3, 0, 256)
    with pytest.raises(ValueError):
        experts.fp4_quantize(whole.transpose(1, 2), "mxfp4")
    with pytest.raises(moe.MoeFp4Error):
        experts.fp4_quantize(whole[0][:, :48], "mxfp4")
    with pytest.raises(moe.MoeFp4Error):
        experts.fp4_quantize(whole[:, :, 4:100], "mxfp4")  # 8-byte aligned
    with pytest.raises(ValueError):
        experts.fp4_quantize(whole, "nvfp4", torch.ones(2).cuda())


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_dequantize_every_code_and_scale(fmt):
    """All codes under all scale bytes; bf16 outputs are the fp32 ones, rounded."""
    G = experts.GROUP[fmt]
    scales = torch.arange(256, dtype=torch.uint8).view(64, 4)
    if fmt == "nvfp4":
        scales = (scales & 0x7F)  # E4M3 scales have no sign
    codes = torch.arange(16, dtype=torch.uint8).repeat(64, 4 * G // 16)
    packed = codes[:, 0::2] | codes[:, 1::2] << 4
    g = torch.tensor([0.0123]) if fmt == "nvfp4" else None
    q = experts.Fp4Tensor(packed.cuda(), scales.cuda(), None if g is None else g.cuda())
    got = experts.fp4_dequantize(q, fmt, torch.float32).cpu()
    want = ref.dequantize(packed, scales, fmt).float()
    if g is not None:
        want = want * g
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))
    low = experts.fp4_dequantize(q, fmt).cpu()
    assert torch.equal(torch.nan_to_num(low), torch.nan_to_num(want.bfloat16()))


# ---------------------------------------------------------------- linear map

def weights(seed, rows, K):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (rows, K // 2), generator=g, dtype=torch.uint8)
    mid = 125 - int(math.log2(math.sqrt(K) * 2.5))
    return codes, torch.randint(mid - 2, mid + 3, (rows, K // 32), generator=g, dtype=torch.uint8)


def make_linear(M, K, N, fn, seed=7):
    alpha, beta, limit = (1.702, 1.0, 7.0) if fn == "swigluoai" else (0.0, 0.0, 0.0)
    desc = experts.Fp4Desc(K, N, M, fn, alpha, beta, limit)
    codes, scales = weights(seed, desc.rows, K)
    return experts.Fp4Linear(desc, codes.cuda(), scales.cuda()), codes, scales


def linear_bound(y, s, N, fn, K, args=(0.0, 0.0, 0.0)):
    """Outputs of exact sums y of terms with magnitudes that sum to s, and how
    far fp32 sums may be off: the K / 128 instructions of an output, their joins
    (16 waves) and what an instruction does within 2^-22 of the magnitudes each;
    through the activation by its slopes (|silu'|, |gelu'| and |g sigmoid(a g)|'
    are below 1.2), its own arithmetic within 2^-18, and the rounding to bf16.
    A relative error holds for normal numbers only: below 2^-126 a step of bf16 is
    2^-133 whatever the value, and an instruction may take a sum there as zero, so
    each of them adds 2^-126."""
    d = (K / 128 + 20) * (2.0 ** -22 * s + 2.0 ** -126)
    if fn == "none":
        out, tol = y, d
    elif fn == "relu2":
        out = block_ref.activation(fn, y, None)
        tol = 2 * y.abs() * d + d * d
    else:
        g, u = y[:, :N], y[:, N:]
        dg, du = d[:, :N], d[:, N:]
        out = block_ref.activation(fn, g, u, *args)
        one = g.abs() + dg
        uu = u.abs() + abs(args[1]) + du
        tol = 1.2 * dg * uu + one * du + 2.0 ** -18 * one * uu
    return out, tol + BF16 * out.abs()


def check_linear(lin, codes, scales, x, rows=None, quantized=False):
    d = lin.desc
    q = experts.fp4_quantize(x.cuda())
    y = lin(quantized=q) if quantized else lin(x.cuda())
    torch.cuda.synchronize()
    pick = slice(None) if rows is None else rows
    exact, s = ref.linear(q.codes.cpu()[pick], q.scales.cpu()[pick], codes, scales)
    want, tol = linear_bound(exact, s, d.N, d.fn, d.K, (d.alpha, d.beta, d.limit))
    err = (y.cpu()[pick].double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    return y


LINEAR = [
    # M, K, N, fn
    (1, 32, 8, "none"), (1, 7168, 256, "silu"), (2, 4096, 264, "none"), (3, 288, 24, "relu2"), (4, 7168, 64, "gelu_tanh"),
    (4, 8224, 40, "swigluoai"), (5, 320, 256, "none"), (16, 2560, 72, "silu"), (17, 96, 200, "none"), (33, 544, 1000, "silu"),
    (64, 1024, 136, "swigluoai"), (100, 160, 520, "relu2"), (129, 256, 2064, "none"), (300, 1568, 1032, "gelu_tanh"),
    (515, 64, 4104, "none"), (1100, 512, 1024, "silu"), (2049, 768, 4096, "none"), (1025, 288, 8200, "silu"),
]


@pytest.mark.parametrize("M,K,N,fn", LINEAR)
def test_linear(M, K, N, fn):
    lin, codes, scales = make_linear(M, K, N, fn)
    x = (rand(3, M, K) * torch.exp(0.4 * rand(4, K))).bfloat16()
    rows = None if M * N * K < 2 ** 31 else torch.tensor([0, 1, 15, 16, 127, 128, 255, 256, M - 2, M - 1])
    y = check_linear(lin, codes, scales, x, rows)
    assert torch.equal(lin(quantized=experts.fp4_quantize(x.cuda())), y) or M <= 4  # few tokens: other launches, other joins
    assert torch.equal(lin(x.cuda()), y)


# 256 x 256 tiles: above 768 of 128 x 128.
@pytest.mark.parametrize("M,K,N,fn", [(2100, 320, 6200, "none"), (3100, 96, 4000, "relu2"), (1100, 544, 8200, "swigluoai"),
                                      (1030, 64, 5800, "gelu_tanh")])
def test_linear_large_tiles(M, K, N, fn):
    lin, codes, scales = make_linear(M, K, N, fn)
    x = (rand(3, M, K) * torch.exp(0.4 * rand(4, K))).bfloat16()
    rows = torch.cat([torch.arange(0, M, 67), torch.tensor([1, 31, 32, 63, 64, 255, 256, 1023, 1024, M - 2, M - 1])])
    y = check_linear(lin, codes, scales, x, rows)
    x[1, 40], x[0, 5] = NAN, INF
    z = lin(x.cuda())
    assert bool(torch.isnan(z[:2]).all() if fn in ("none", "relu2") else torch.isnan(z[:2]).any())
    assert torch.equal(z[2:], y[2:])


@pytest.mark.parametrize("M", [1, 4, 37, 600])
def test_linear_given_codes(M):
    lin, codes, scales = make_linear(M, 1312, 1056, "silu")
    check_linear(lin, codes, scales, rand(5, M, 1312).bfloat16(), quantized=True)


def test_linear_smaller_batches_and_none():
    lin, codes, scales = make_linear(700, 640, 520, "none")
    for M in (700, 1, 33, 0, 260):
        x = rand(M, M, 640).bfloat16()
        if M:
            check_linear(lin, codes, scales, x)
        else:
            assert lin(x.cuda()).shape == (0, 520)


@pytest.mark.parametrize("M", [2, 20, 700])
def test_linear_nan_stays_with_its_token(M):
    lin, codes, scales = make_linear(M, 512, 264, "none")
    x = rand(6, M, 512).bfloat16()
    clean = lin(x.cuda())
    x[1, 40], x[0, 500] = NAN, INF
    y = lin(x.cuda())
    assert bool(torch.isnan(y[:2]).all())
    assert torch.equal(y[2:], clean[2:])


def test_linear_zeros_and_large_scales():
    """A token of zeros gives zeros; the ends of the scales' range multiply as they should."""
    lin, codes, scales = make_linear(6, 256, 32, "none")
    x = torch.zeros(6, 256)
    x[1], x[2], x[3] = 1e38, 1e-38, 1e-40
    y = check_linear(lin, codes, scales, x.bfloat16())
    assert bool((y[0] == 0).all())


def test_linear_leaves_borders_alone():
    for M, K, N in ((1, 7168, 40), (37, 320, 264), (300, 256, 1032)):
        lin, codes, scales = make_linear(M, K, N, "none")
        lin.workspace.fill_(0xFF)
        big = torch.full((M + 16, N), 7.0, dtype=torch.bfloat16, device="cuda")
        out = lin(rand(8, M, K).bfloat16().cuda(), out=big[8:M + 8])
        assert bool((big[:8] == 7).all()) and bool((big[M + 8:] == 7).all())
        assert torch.equal(out, lin(rand(8, M, K).bfloat16().cuda()))


# ---------------------------------------------------------------- routes

GROUPS = [(1, 1, 1), (1, 8, 256), (7, 3, 5), (512, 8, 128), (513, 8, 128), (1100, 4, 64), (4097, 1, 3), (300, 4, 1030),
          (257, 4, 4096), (3000, 8, 512)]


def make_ids(M, k, E, seed=1, lost=0.1):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, E, (M, k), generator=g)
    wild = torch.tensor([-1, E, -2 ** 31, 2 ** 31 - 1])[torch.randint(0, 4, (M, k), generator=g)]
    return torch.where(torch.rand(M, k, generator=g) < lost, wild, ids)


@pytest.mark.parametrize("M,k,E", GROUPS)
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_group_routes(M, k, E, dtype):
    """The same expert twice in a token is two routes."""
    ids = make_ids(M, k, E)
    got = experts.group_routes(ids.to(dtype).cuda(), E)
    for name, a, b in zip(got._fields, got, ref.group(ids, E) if E < 600 else group_sorted(ids, E)):
        assert torch.equal(a.cpu(), b), name


def group_sorted(ids, E):
    flat = ids.flatten()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = key.sort(stable=True)[1]
    n = int((key < E).sum())
    place = torch.full_like(order, -1)
    place[order[:n]] = torch.arange(n)
    offsets = torch.searchsorted(key[order].contiguous(), torch.arange(E + 1))
    order[n:] = -1
    return offsets.int(), order.int(), place.view(ids.shape).int()


def test_group_routes_ends():
    none = experts.group_routes(torch.full((50, 3), -1, dtype=torch.int64).cuda(), 9)
    assert bool((none.offsets == 0).all()) and bool((none.order == -1).all()) and bool((none.place == -1).all())
    one = experts.group_routes(torch.full((2000, 5), 8, dtype=torch.int32).cuda(), 9)
    assert one.offsets.tolist() == [0] * 9 + [10000]
    assert torch.equal(one.order.cpu(), torch.arange(10000, dtype=torch.int32))
    empty = experts.group_routes(torch.zeros((0, 4), dtype=torch.int32).cuda(), 9)
    assert empty.offsets.tolist() == [0] * 10
    big = torch.tensor([[2 ** 32, 1], [-2 ** 40, 2 ** 33 + 1]])  # int64 ids are not cut to 32 bits
    assert experts.group_routes(big.cuda(), 4).place.tolist() == [[-1, 0], [-1, -1]]


ROWS = [(1, 1, 8, 1), (1, 8, 7168, 256), (5, 3, 24, 7), (130, 4, 520, 16), (40, 10, 2056, 9), (700, 2, 4096, 30)]


@pytest.mark.parametrize("M,k,H,E", ROWS)
def test_gather_and_combine(M, k, H, E):
    ids = make_ids(M, k, E, seed=M, lost=0.2)
    groups = experts.group_routes(ids.cuda(), E)
    _, order, place = ref.group(ids, E)
    R = M * k
    x, y, w = rand(1, M, H).bfloat16(), rand(2, R, H).bfloat16(), rand(3, M, k)
    y[order < 0] = NAN  # rows of no route are not read
    xg = experts.gather_routes(x.cuda(), groups)
    want = torch.where((order >= 0)[:, None], x[order.clamp(min=0).long() // k], torch.zeros(1, dtype=torch.bfloat16))
    assert torch.equal(xg.cpu(), want)
    for ww in (w, None):
        out = experts.combine_routes(y.cuda(), groups, None if ww is None else ww.cuda())
        rows = y[place.clamp(min=0).long()].double()
        f = torch.ones(M, k, dtype=torch.float64) if ww is None else ww.double()
        t = torch.where((place >= 0)[..., None], f[..., None] * rows, torch.zeros(1, dtype=torch.float64))
        tol = BF16 * t.sum(1).abs() + (k + 1) * FP32 * t.abs().sum(1)
        assert bool(((out.cpu().double() - t.sum(1)).abs() <= tol).all())


@pytest.mark.parametrize("M,k,H,E", ROWS + [(1030, 1, 64, 8), (300, 4, 1000, 12)])
def test_route_gradients(M, k, H, E):
    ids = make_ids(M, k, E, seed=M + 1, lost=0.2)
    groups = experts.group_routes(ids.cuda(), E)
    _, order, place = ref.group(ids, E)
    R = M * k
    x = rand(1, M, H).bfloat16().cuda().requires_grad_()
    y = rand(2, R, H).bfloat16()
    y[order < 0] = NAN
    y = y.cuda().requires_grad_()
    w = rand(3, M, k).cuda().requires_grad_()
    dxg, dout = rand(4, R, H).bfloat16(), rand(5, M, H).bfloat16()
    (dx,) = torch.autograd.grad(experts.gather_routes(x, groups), x, dxg.cuda())
    dy, dw = torch.autograd.grad(experts.combine_routes(y, groups, w), (y, w), dout.cuda())
    has, at = (place >= 0), place.clamp(min=0).long()
    t = torch.where(has[..., None], dxg[at].double(), torch.zeros(1, dtype=torch.float64))
    tol = BF16 * t.sum(1).abs() + (k + 1) * FP32 * t.abs().sum(1)
    assert bool(((dx.cpu().double() - t.sum(1)).abs() <= tol).all())
    live = (order >= 0)
    slot = order.clamp(min=0).long()
    want = torch.where(live[:, None], w.detach().cpu().flatten()[slot, None] * dout[slot // k].float(), torch.zeros(1))
    assert torch.equal(dy.cpu(), want.bfloat16())
    prod = torch.where(has[..., None], dout[:, None].double() * y.detach().cpu()[at].double(), torch.zeros(1, dtype=torch.float64))
    tol = (H / 64 + 24) * FP32 * prod.abs().sum(2)
    assert bool(((dw.cpu().double() - prod.sum(2)).abs() <= tol).all())
    # without weights the gradient is a gather; a gradient that is a broadcast scalar
    (d1,) = torch.autograd.grad(experts.combine_routes(y, groups).sum(), y)
    assert torch.equal(d1.cpu(), live[:, None].expand(R, H).bfloat16())


# ---------------------------------------------------------------- grouped products

def make_offsets(counts, before=0):
    return torch.cat([torch.tensor([before]), before + torch.tensor(counts).cumsum(0)]).int()


GROUPED = [
    # counts, rows before and after them, K, N
    ([1], 0, 0, 8, 8), ([0, 1, 0], 0, 0, 72, 16), ([3, 0, 5, 1], 2, 9, 64, 136), ([0, 0], 0, 5, 40, 24),
    ([17, 1, 0, 16, 33], 0, 0, 264, 520), ([130, 127, 128, 0, 1], 3, 0, 128, 256), ([300, 5, 257], 0, 70, 328, 392),
    ([256, 512], 0, 0, 192, 264), ([700, 20], 40, 1, 72, 1032), ([1] * 70, 0, 0, 136, 48), ([0] * 300 + [40], 0, 0, 200, 64),
    ([260, 0, 411, 130], 0, 0, 1000, 520),
]


def dot_bound(s, n):
    """fp32 sums of n products on the bf16 matrix instruction, 32 at a time:
    within (n / 64 + 5) 2^-22 of the sum of their magnitudes."""
    return (n / 64 + 5) * 2.0 ** -22 * s


@pytest.mark.parametrize("counts,before,after,K,N", GROUPED)
def test_grouped_linear_and_gradients(counts, before, after, K, N):
    E, T = len(counts), before + sum(counts) + after
    off = make_offsets(counts, before)
    x, w, dy = rand(1, T, K).bfloat16(), (rand(2, E, N, K) / math.sqrt(K)).bfloat16(), rand(3, T, N).bfloat16()
    x[off[-1]:], dy[:before] = NAN, NAN  # rows of no expert are not read
    y, s = ref.grouped(x, w, off)
    xd, wd, o = x.cuda().requires_grad_(), w.cuda().requires_grad_(), off.cuda()
    got = experts.grouped_linear(xd, wd, o)
    err = (got.detach().cpu().double() - y).abs()
    assert bool((err <= dot_bound(s, K) + BF16 * y.abs()).all())
    dx, dw = torch.autograd.grad(got, (xd, wd), dy.cuda())
    ex, sx = ref.grouped(dy, w.transpose(1, 2), off)
    assert bool(((dx.cpu().double() - ex).abs() <= dot_bound(sx, N) + BF16 * ex.abs()).all())
    ew, sw = ref.grouped_grad(dy, x, off)
    n = max(counts)
    assert bool(((dw.cpu().double() - ew).abs() <= dot_bound(sw, n) + BF16 * ew.abs()).all())
    d32 = experts.grouped_weight_grad(dy.cuda(), x.cuda(), o, dtype=torch.float32)
    assert bool(((d32.cpu().double() - ew).abs() <= dot_bound(sw, n)).all())
    # the same bits again, and without a gradient
    with torch.no_grad():
        assert torch.equal(experts.grouped_linear(xd, wd, o), got.detach())
    assert torch.equal(torch.autograd.grad(experts.grouped_linear(xd, wd, o), wd, dy.cuda())[0], dw)


def test_grouped_gradient_against_differences():
    """With small whole numbers every sum is exact, so the differences of the
    outputs along a direction are those of the gradients to the last bit."""
    g = torch.Generator().manual_seed(3)
    whole = lambda *s: torch.randint(-1, 2, s, generator=g).bfloat16().cuda()
    off = make_offsets([20, 0, 45, 3], 1).cuda()
    x, w, dy, vx, vw = whole(72, 64), whole(4, 40, 64), whole(72, 40), whole(72, 64), whole(4, 40, 64)
    x.requires_grad_(), w.requires_grad_()
    dx, dw = torch.autograd.grad(experts.grouped_linear(x, w, off), (x, w), dy)
    with torch.no_grad():
        base = experts.grouped_linear(x, w, off).double()
        along_x = ((experts.grouped_linear(x + vx, w, off).double() - base) * dy.double()).sum()
        along_w = ((experts.grouped_linear(x, w + vw, off).double() - base) * dy.double()).sum()
    assert float(along_x) == float((dx.double() * vx.double()).sum())
    assert float(along_w) == float((dw.double() * vw.double()).sum())


def test_grouped_wild_offsets_stay_in_range():
    """Offsets out of range or order give no access out of range: the borders of
    the outputs stay as they are."""
    T, K, N, E = 96, 64, 72, 4
    x, w = rand(1, T, K).bfloat16().cuda(), rand(2, E, N, K).bfloat16().cuda()
    for off in ([-5, 10, 3, 200, 2 ** 30], [50, 40, 30, 20, 10], [-2 ** 31, 0, 2 ** 31 - 1, -1, 7]):
        big = torch.full((T + 32, N), 7.0, dtype=torch.bfloat16, device="cuda")
        o = torch.tensor(off, dtype=torch.int32).cuda()
        experts.grouped_linear(x, w, o, out=big[16:T + 16])
        assert bool((big[:16] == 7).all()) and bool((big[T + 16:] == 7).all())
        experts.grouped_weight_grad(rand(3, T, N).bfloat16().cuda(), x, o)


def test_grouped_no_rows():
    w = rand(2, 3, 16, 24).bfloat16().cuda().requires_grad_()
    x = torch.zeros(0, 24, dtype=torch.bfloat16, device="cuda").requires_grad_()
    off = torch.zeros(4, dtype=torch.int32).cuda()
    y = experts.grouped_linear(x, w, off)
    dx, dw = torch.autograd.grad(y, (x, w), torch.zeros_like(y))
    assert y.shape == (0, 16) and dx.shape == (0, 24) and bool((dw == 0).all())


def test_grouped_nan_stays_in_its_row_and_expert():
    off = make_offsets([100, 60, 0, 200]).cuda()
    x, w = rand(1, 360, 128).bfloat16().cuda(), rand(2, 4, 136, 128).bfloat16().cuda()
    clean, dy = experts.grouped_linear(x, w, off), rand(3, 360, 136).bfloat16().cuda()
    cw = experts.grouped_weight_grad(dy, x, off)
    x[130, 5] = NAN
    y, dw = experts.grouped_linear(x, w, off), experts.grouped_weight_grad(dy, x, off)
    keep = torch.arange(360) != 130
    assert bool(torch.isnan(y[130]).all()) and torch.equal(y[keep], clean[keep])
    assert bool(torch.isnan(dw[1, :, 5]).all())
    dw[1, :, 5] = cw[1, :, 5]
    assert torch.equal(dw, cw)


# Ragged groups at the borders of the launches' variants: 256 x 256 tiles (many
# experts, or many rows), one-step contractions, tails of every row fragment, and
# few rows with K shared by 1, 2 and 4 waves.
SOME = [0, 1, 2, 5, 0, 3]
VARIANTS = [
    # counts, rows before and after them, K, N
    (SOME * 40 + [600, 257, 64, 33, 96, 161, 225, 31, 255, 256], 3, 7, 72, 264), (SOME * 11 + [400, 200], 0, 2, 328, 1032),
    ([70, 0, 1] * 23, 0, 0, 64, 1288), ([1] * 130, 5, 0, 24, 520), ([9000, 0, 11000], 1, 40, 72, 1000),
    ([0] * 258 + [3], 0, 0, 520, 264), ([2, 0, 0, 31, 16], 5, 3, 2056, 40), ([1], 0, 0, 4104, 8), ([5] * 20, 1, 0, 520, 72),
    ([1, 0, 1, 17], 0, 300, 1032, 136), ([0, 2] * 150, 0, 0, 1096, 16), ([16, 15], 0, 0, 8, 2056),
]


@pytest.mark.parametrize("counts,before,after,K,N", VARIANTS)
def test_grouped_variants(counts, before, after, K, N):
    test_grouped_linear_and_gradients(counts, before, after, K, N)


@pytest.mark.parametrize("E,T,K,N", [(4, 96, 64, 72), (300, 700, 72, 264), (6, 9, 1032, 72), (3, 700, 64, 1032)])
def test_grouped_wild_offsets_in_every_variant(E, T, K, N):
    x, w, dy = rand(1, T, K).bfloat16().cuda(), rand(2, E, N, K).bfloat16().cuda(), rand(3, T, N).bfloat16().cuda()
    g = torch.Generator().manual_seed(E)
    for low, high in ((-50, T + 50), (-2 ** 31, 2 ** 31 - 1)):
        off = torch.randint(low, high, (E + 1,), generator=g).int().cuda()
        for a, b, layout in ((x, N, 0), (dy, K, 1)):
            big = torch.full((T + 32, b), 7.0, dtype=torch.bfloat16, device="cuda")
            experts._grouped(a, w, off, layout, big[16:T + 16])
            assert bool((big[:16] == 7).all()) and bool((big[T + 16:] == 7).all())
        big = torch.full((E + 2, N, K), 7.0, device="cuda")
        experts.grouped_weight_grad(dy, x, off, torch.float32, out=big[1:E + 1])
        assert bool((big[0] == 7).all()) and bool((big[E + 1] == 7).all())


@pytest.mark.parametrize("T", [5, 600])
def test_grouped_weights_past_32_bits(T):
    """300 experts of 2048 x 4096: 5 GB of weights and of their gradient."""
    E, N, K = 300, 2048, 4096
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda")
    w[0], w[-1] = rand(1, N, K).bfloat16(), rand(2, N, K).bfloat16()
    x, dy = rand(3, T, K).bfloat16(), rand(4, T, N).bfloat16()
    off = make_offsets([2] + [0] * (E - 2) + [T - 2])
    small = torch.tensor([0, 2, T], dtype=torch.int32)
    both = w[[0, E - 1]].cpu()
    y = experts.grouped_linear(x.cuda(), w, off.cuda())
    ey, sy = ref.grouped(x, both, small)
    assert bool(((y.cpu().double() - ey).abs() <= dot_bound(sy, K) + BF16 * ey.abs()).all())
    dx = experts._grouped(dy.cuda(), w, off.cuda(), experts.WEIGHT_IN_OUT)
    ex, sx = ref.grouped(dy, both.transpose(1, 2), small)
    assert bool(((dx.cpu().double() - ex).abs() <= dot_bound(sx, N) + BF16 * ex.abs()).all())
    w.fill_(7.0)
    dw = experts.grouped_weight_grad(dy.cuda(), x.cuda(), off.cuda(), out=w)
    assert not bool(dw[1:-1].any())
    ew, sw = ref.grouped_grad(dy, x, small)
    assert bool(((dw[[0, E - 1]].cpu().double() - ew).abs() <= dot_bound(sw, T) + BF16 * ew.abs()).all())


def test_grouped_rows_past_32_bits():
    """600000 rows of 4096 values, of which the last 300 are not zero."""
    T, K, N, n = 600000, 4096, 8, 300
    x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    tail, dtail = rand(1, n, K).bfloat16(), rand(2, n, N).bfloat16()
    x[-n:], dy[-n:] = tail, dtail
    w = (rand(3, 2, N, K) / 64).bfloat16()
    off = torch.tensor([0, T - 100, T], dtype=torch.int32)
    small = torch.tensor([0, n - 100, n], dtype=torch.int32)
    y = experts.grouped_linear(x, w.cuda(), off.cuda())
    ey, sy = ref.grouped(tail, w, small)
    assert bool(((y[-n:].cpu().double() - ey).abs() <= dot_bound(sy, K) + BF16 * ey.abs()).all()) and not bool(y[:-n].any())
    dx = experts._grouped(dy, w.cuda(), off.cuda(), experts.WEIGHT_IN_OUT)
    ex, sx = ref.grouped(dtail, w.transpose(1, 2), small)
    assert bool(((dx[-n:].cpu().double() - ex).abs() <= dot_bound(sx, N) + BF16 * ex.abs()).all()) and not bool(dx[:-n].any())
    dw = experts.grouped_weight_grad(dy, x, off.cuda())
    ew, sw = ref.grouped_grad(dtail, tail, small)
    # zeros add nothing: 300 products that are not
    assert bool(((dw.cpu().double() - ew).abs() <= dot_bound(sw, n) + BF16 * ew.abs()).all())


def test_grouped_gradients_one_at_a_time():
    """Only x or only w asks for a gradient; the output's may be strided or broadcast."""
    off = make_offsets([20, 0, 45], 2).cuda()
    x, w = rand(1, 70, 64).bfloat16().cuda(), rand(2, 3, 40, 64).bfloat16().cuda()
    dy = rand(3, 40, 70).bfloat16().cuda().t()
    xr, wr = x.clone().requires_grad_(), w.clone().requires_grad_()
    dx, dw = torch.autograd.grad(experts.grouped_linear(xr, wr, off), (xr, wr), dy)
    assert torch.equal(torch.autograd.grad(experts.grouped_linear(xr, w, off), xr, dy)[0], dx)
    assert torch.equal(torch.autograd.grad(experts.grouped_linear(x, wr, off), wr, dy)[0], dw)
    assert torch.equal(dw, experts.grouped_weight_grad(dy.contiguous(), x, off))
    (ones,) = torch.autograd.grad(experts.grouped_linear(x, wr, off).sum(), wr)
    assert torch.equal(ones, experts.grouped_weight_grad(torch.ones_like(dy).contiguous(), x, off))


# ---------------------------------------------------------------- long arrays

def test_quantize_past_32_bits():
    x = torch.zeros(40000, 65536, dtype=torch.bfloat16, device="cuda")
    tail = spread(1, 7, 65536).bfloat16()
    x[-7:] = tail
    codes, scales, _ = ref.quantize(tail[None], "mxfp4")
    q = experts.fp4_quantize(x)
    assert torch.equal(q.codes[-7:].cpu(), codes[0]) and torch.equal(q.scales[-7:].cpu(), scales[0])
    back = experts.fp4_dequantize(q)
    assert torch.equal(back[-7:].cpu(), ref.dequantize(codes[0], scales[0], "mxfp4").bfloat16())
    del back, q
    codes, scales, g = ref.quantize(tail[None], "nvfp4")
    q = experts.fp4_quantize(x, "nvfp4")
    assert torch.equal(q.global_scale.cpu(), g)
    assert torch.equal(q.codes[-7:].cpu(), codes[0]) and torch.equal(q.scales[-7:].cpu(), scales[0])


def test_linear_past_32_bits():
    """The last features of 2^31 weights, and the last tokens of 2^31 values."""
    K, N = 65536, 32768
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device="cuda")
    scales = torch.randint(112, 118, (N, K // 32), generator=g, dtype=torch.uint8, device="cuda")
    x = torch.zeros(34000, K, dtype=torch.bfloat16, device="cuda")
    x[-3:] = rand(2, 3, K).bfloat16()
    for M, rows in ((3, slice(N - 40, N)), (300, slice(N - 24, N)), (34000, slice(0, 8))):
        part = experts.Fp4Desc(K, N if M < 1000 else 8, M)
        lin = experts.Fp4Linear(part, codes[:part.N], scales[:part.N])
        q = experts.fp4_quantize(x[-3:])
        y = lin(x[-M:])
        exact, s = ref.linear(q.codes.cpu(), q.scales.cpu(), codes[rows].cpu(), scales[rows].cpu())
        want, tol = linear_bound(exact, s, 0, "none", K)
        assert bool(((y[-3:, rows].cpu().double() - want).abs() <= tol).all())
        assert not bool(y[:-3].any())


def test_routes_past_32_bits():
    M, k, H, E = 300000, 4, 2048, 64
    ids = make_ids(M, k, E)
    groups = experts.group_routes(ids.cuda(), E)
    x = torch.randn(M, H, device="cuda").bfloat16()
    xg = experts.gather_routes(x, groups)
    pick = torch.tensor([0, 1, M * k // 2, int(groups.offsets[-1]) - 1, M * k - 1])
    for p in pick.tolist():
        r = int(groups.order[p])
        assert torch.equal(xg[p], x[r // k] if r >= 0 else torch.zeros_like(x[0]))
    w = rand(3, M, k).cuda()
    out = experts.combine_routes(xg, groups, w)
    f = torch.where(groups.place >= 0, w, torch.zeros_like(w)).double()
    for t in (0, 7, M - 2, M - 1):  # rows of a token are its own x again
        terms = f[t].sum() * x[t].double()
        tol = BF16 * terms.abs() + (k + 1) * FP32 * f[t].abs().sum() * x[t].double().abs()
        assert bool(((out[t].double() - terms).abs() <= tol).all())


# ---------------------------------------------------------------- together

def bf16_layer(x, ids, w, w13, w2):
    E, I = w13.shape[0], w13.shape[1] // 2
    groups = experts.group_routes(ids, E)
    h = experts.grouped_linear(experts.gather_routes(x, groups), w13, groups.offsets).float()
    a = (torch.nn.functional.silu(h[:, :I]) * h[:, I:]).bfloat16()
    return experts.combine_routes(experts.grouped_linear(a, w2, groups.offsets), groups, w)


def layer_inputs(M, H, I, E, k, seed=1):
    w13 = (rand(seed, E, 2 * I, H) / math.sqrt(H)).bfloat16().cuda()
    w2 = (rand(seed + 1, E, H, I) / math.sqrt(I)).bfloat16().cuda()
    x = rand(seed + 2, M, H).bfloat16().cuda()
    router = block.Router(block.RouterDesc(E, H, k, M), (rand(seed + 3, E, H) / math.sqrt(H)).bfloat16().cuda())
    ids, w = router(x)
    return x, ids, w, w13, w2


def test_layer_of_bf16_experts_trains():
    """Router, grouping, products and join together: outputs and gradients
    against the same layer in 64 bits.  Each bf16 rounding on the way (h, a, y
    and their gradients) is relative 2^-8 of its value; all told the norm of a
    result is off by no more than 4 of them."""
    M, H, I, E, k = 70, 128, 96, 16, 4
    x, ids, w, w13, w2 = layer_inputs(M, H, I, E, k)
    ids[3, 1], ids[69, 0] = -1, E
    leaves = [t.clone().requires_grad_() for t in (x, w, w13, w2)]
    dout = rand(9, M, H).bfloat16().cuda()
    out = bf16_layer(leaves[0], ids, *leaves[1:])
    grads = torch.autograd.grad(out, leaves, dout)
    ex = [t.detach().cpu().double().requires_grad_() for t in leaves]
    want = torch.zeros(M, H, dtype=torch.float64)
    for j in range(k):
        for e in range(E):
            rows = (ids[:, j].cpu() == e).nonzero().flatten()
            h = ex[0][rows] @ ex[2][e].t()
            y = (torch.nn.functional.silu(h[:, :I]) * h[:, I:]) @ ex[3][e].t()
            want = want.index_add(0, rows, ex[1][rows, j, None] * y)
    exact = torch.autograd.grad(want, ex, dout.cpu().double())
    for name, a, b in (("out", out, want), *zip(("dx", "dw", "dw13", "dw2"), grads, exact)):
        rel = float((a.detach().cpu().double() - b.detach()).norm() / b.detach().norm())
        assert rel <= 4 * BF16, (name, rel)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_fp4_layer_from_float(fmt):
    """The FP4 layer of bf16 experts is that of their quantised forms, bit for
    bit, and the bf16 layer on the values those stand for agrees with it."""
    M, H, I, E, k = 40, 256, 128, 8, 2
    x, ids, w, w13, w2 = layer_inputs(M, H, I, E, k, seed=21)
    desc = moe.Desc(fmt, E, H, I, k, M)
    layer = moe.Fp4MoE.from_float(desc, w13, w2)
    q13, q2 = experts.fp4_quantize(w13, fmt), experts.fp4_quantize(w2, fmt)
    same = moe.Fp4MoE(desc, q13.codes, q13.scales, q2.codes, q2.scales, q13.global_scale, q2.global_scale)
    out = layer(x, ids, w)
    assert torch.equal(out, same(x, ids, w))
    back = [experts.fp4_dequantize(q, fmt) for q in (q13, q2)]
    other = bf16_layer(x, ids, w, *back)
    rel = float((out.double() - other.double()).norm() / other.double().norm())
    # roundings of the bf16 layer's h, a, y and of NVFP4's values to bf16
    assert rel <= 4 * BF16, rel


def test_fp4_linear_as_a_shared_expert():
    M, H, I, E, k = 24, 256, 128, 8, 2
    x, ids, w, w13, w2 = layer_inputs(M, H, I, E, k, seed=31)
    layer = moe.Fp4MoE.from_float(moe.Desc("mxfp4", E, H, I, k, M), w13, w2)
    router = block.Router(block.RouterDesc(E, H, k, M), (rand(34, E, H) / math.sqrt(H)).bfloat16().cuda())
    up = experts.Fp4Linear.from_float(experts.Fp4Desc(H, I, M, fn="silu"), w13[0])
    down = experts.Fp4Linear.from_float(experts.Fp4Desc(I, H, M), w2[0].float())
    pre = (1 + 0.2 * rand(35, H)).bfloat16().cuda()
    h, _ = block.Fp4MoEBlock(layer, router, pre, shared_up=up, shared_down=down)(x)
    _, n = block.block_norm(x, pre_weight=pre)
    ids, w = router(n)
    want, _ = block.block_norm(x, layer(n, ids, w), down(up(n)))
    assert torch.equal(h, want)


# ---------------------------------------------------------------- streams and graphs

def everything(x, ids, w, w13, w2, lin, dout, stream=None):
    """One call of each, given a stream or not."""
    kw = dict(stream=stream)
    E = w13.shape[0]
    groups = experts.group_routes(ids, E, **kw)
    xg = experts.gather_routes(x, groups, **kw)
    h = experts.grouped_linear(xg, w13, groups.offsets, **kw)
    q = experts.fp4_quantize(h, "nvfp4", **kw)
    back = experts.fp4_dequantize(q, "nvfp4", **kw)
    dw = experts.grouped_weight_grad(back, xg, groups.offsets, dtype=torch.float32, **kw)
    out = experts.combine_routes(xg, groups, w, **kw)
    return out, lin(out, **kw), h, dw, q.codes, q.scales, q.global_scale, *groups


def test_calls_on_a_given_stream():
    x, ids, w, w13, w2 = layer_inputs(50, 128, 64, 8, 3, seed=41)
    lin, _, _ = make_linear(50, 128, 64, "none")
    dout = rand(2, 50, 128).bfloat16().cuda()
    want = everything(x, ids, w, w13, w2, lin, dout)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(10_000_000)
    x2 = x.clone()
    side.wait_stream(torch.cuda.current_stream())
    got = everything(x2, ids, w, w13, w2, lin, dout, stream=side)
    del x2
    filler = torch.full((50, 128), 3.0, dtype=torch.bfloat16, device="cuda")  # must not take x2's place too early
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and bool((filler == 3).all())
    # a raw stream address, and a gradient taken later
    y = x.clone().requires_grad_()
    groups = experts.group_routes(ids, 8, stream=side.cuda_stream)
    side.synchronize()
    out = experts.gather_routes(y, groups, stream=side)
    side.synchronize()
    out.backward(torch.ones_like(out))
    torch.cuda.synchronize()
    assert torch.equal(y.grad, (groups.place >= 0).sum(1, keepdim=True).expand(50, 128).bfloat16())


@pytest.mark.parametrize("where", ["cpu", "cuda"])
def test_made_from_floats_on_a_given_stream(where):
    """In order with the current stream before and after: the weights are still
    on their way when the objects are made, which are used at once."""
    M, H, I, E, k = 20, 128, 64, 8, 3
    x, ids, w, w13, w2 = layer_inputs(M, H, I, E, k, seed=61)
    x = x.detach()
    desc, up = moe.Desc("nvfp4", E, H, I, k, M), experts.Fp4Desc(H, I, M, fn="silu")
    want = moe.Fp4MoE.from_float(desc, w13, w2)(x, ids, w), experts.Fp4Linear.from_float(up, w13[0])(x)
    side = torch.cuda.Stream()
    given = [t.detach().to(where) for t in (w13, w2)]
    torch.cuda.synchronize()
    torch.cuda._sleep(10_000_000)
    if where == "cuda":
        late = [torch.zeros_like(t) for t in given]
        for a, b in zip(late, given):
            a.copy_(b)
        given = late
    layer = moe.Fp4MoE.from_float(desc, *given, stream=side)
    linear = experts.Fp4Linear.from_float(up, given[0][0], stream=side.cuda_stream)
    del given
    got = layer(x, ids, w), linear(x)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_captured_and_replayed():
    """A forward and backward pass in a graph, replayed on new inputs with eager
    work in between, against eager calls."""
    M, H, I, E, k = 60, 128, 64, 8, 3
    x, ids, w, w13, w2 = layer_inputs(M, H, I, E, k, seed=51)
    lin, _, _ = make_linear(M, H, 72, "silu")
    dout = rand(3, M, H).bfloat16().cuda()

    def step():
        leaves = [t.detach().requires_grad_() for t in (x, w, w13, w2)]
        out = bf16_layer(leaves[0], ids, *leaves[1:])
        grads = torch.autograd.grad(out, leaves, dout)
        q = experts.fp4_quantize(out.detach(), "nvfp4")
        return out.detach(), *grads, lin(out.detach()), *q

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        x.copy_(rand(60 + i, M, H).bfloat16())
        ids.copy_(make_ids(M, k, E, seed=i).int())
        w13.mul_(1.125)
        graph.replay()
        got = [t.clone() for t in held]
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), i
