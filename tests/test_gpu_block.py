"""The operators around the expert layer (router, FP8 linear map, fused block
norms, and the block made of them) against 64-bit references."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import block_ref as ref
import oracle
from block_scaled_fp4_gather_amd import block, moe, synth
from gpu_util import compare, make_layer, say

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8  # half a step of bf16, relative
FP32 = 2.0 ** -24


@pytest.fixture(autouse=True)
def _announce(request):
    say(f"\n[gpu] {request.node.nodeid}")
    yield


def rand(seed, *shape):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g)


def hidden(seed, M, H):
    """Rows with a spread over channels and a few large values."""
    x = rand(seed, M, H) * torch.exp(0.4 * rand(seed + 1, H))
    x[:, :: max(1, H // 3)] *= 6.0
    return x.bfloat16()


# ---------------------------------------------------------------- router

def make_router(E, H, k, M, weight="bf16", bias=None, seed=3, w=None, **kw):
    if w is None:
        w = rand(seed, E, H) / math.sqrt(2 * H)
    w = w.to(torch.bfloat16 if weight == "bf16" else torch.float32)
    desc = block.RouterDesc(E, H, k, M, weight=weight, **kw)
    return block.Router(desc, w.cuda(), None if bias is None else bias.cuda()), w


def check_routes(router, w, x, bias=None, logits=True):
    d = router.desc
    M = x.shape[0]
    lg = torch.full((M, d.E), math.nan, device="cuda") if logits else None
    ids, wt = router(x.cuda(), logits=lg)
    torch.cuda.synchronize()
    rid, rw, z = ref.route(x, w, d.k, d.scoring, bias, d.groups, d.top_groups, d.renorm, d.scale)
    assert torch.equal(ids.cpu(), rid)
    # an fp32 logit is off by at most a rounding of 2^-22 per 32 products of a
    # slice, on partial sums of at most ||x|| ||w||; weights follow with twice that
    planes = 3 if d.weight == "fp32" else 1
    delta = (0.5 * (d.H / 32) * planes + 5) * 2.0 ** -22 * x.double().norm(dim=1, keepdim=True) * w.double().norm(dim=1).max()
    assert bool(((wt.cpu().double() - rw).abs() <= rw.abs() * (4 * delta + 2 ** -22) + 1e-37).all())
    if logits:
        assert bool(((lg.cpu().double() - z).abs() <= delta + z.abs() * FP32).all())
        return ids, wt, lg
    return ids, wt


ROUTES = [
    # M, H, E, k, weight, scoring, bias, groups, top_groups, renorm, scale
    (1, 8, 1, 1, "bf16", "softmax", False, 1, 1, True, 1.0),
    (1, 256, 8, 2, "bf16", "softmax", False, 1, 1, True, 1.0),
    (3, 40, 5, 5, "fp32", "sigmoid", True, 1, 1, True, 2.0),
    (1, 7168, 256, 8, "bf16", "sigmoid", True, 8, 4, True, 1.5),
    (16, 4096, 128, 8, "fp32", "softmax", True, 1, 1, False, 1.0),
    (17, 2560, 512, 10, "fp32", "softmax", False, 1, 1, False, 1.0),
    (33, 1000, 65, 7, "bf16", "sigmoid", False, 13, 5, True, 1.0),
    (65, 520, 200, 16, "bf16", "softmax", True, 4, 2, True, 1.0),
    (100, 264, 129, 64, "bf16", "softmax", False, 1, 1, True, 1.0),
    (200, 2048, 384, 6, "fp32", "softmax", False, 64, 3, False, 0.5),
    (300, 328, 512, 8, "bf16", "sigmoid", True, 16, 1, False, 1.0),
    (1500, 520, 256, 8, "bf16", "sigmoid", True, 8, 4, True, 1.5),
    (257, 776, 96, 8, "bf16", "softmax", False, 1, 1, True, 1.0),
    (700, 1000, 100, 4, "fp32", "softmax", False, 1, 1, False, 1.0),
    (1000, 72, 300, 8, "fp32", "sigmoid", True, 1, 1, True, 1.0),
    (2000, 1096, 64, 2, "bf16", "softmax", True, 1, 1, True, 1.0),
    (1025, 40, 512, 5, "bf16", "sigmoid", False, 8, 2, True, 1.0),
    (600, 416, 444, 6, "bf16", "softmax", True, 4, 4, True, 1.0),
    (270, 648, 241, 10, "fp32", "softmax", True, 1, 1, True, 1.0),
]


@pytest.mark.parametrize("M,H,E,k,weight,scoring,biased,groups,top_groups,renorm,scale", ROUTES)
def test_route(M, H, E, k, weight, scoring, biased, groups, top_groups, renorm, scale):
    bias = 0.05 * rand(9, E) if biased else None
    router, w = make_router(E, H, k, M, weight, bias, scoring=scoring, groups=groups, top_groups=top_groups,
                            renorm=renorm, scale=scale)
    check_routes(router, w, hidden(M, M, H), bias)
    # fewer tokens on the same router, without logits
    check_routes(router, w, hidden(M + 7, max(1, M // 3), H), bias, logits=False)


@pytest.mark.parametrize("weight", ["bf16", "fp32"])
@pytest.mark.parametrize("scoring,biased,groups,top_groups", [
    ("softmax", False, 1, 1), ("sigmoid", True, 1, 1), ("softmax", True, 1, 1), ("sigmoid", False, 8, 3),
    ("sigmoid", True, 8, 3), ("softmax", False, 8, 3), ("softmax", True, 8, 3)])
def test_route_near_ties(weight, scoring, biased, groups, top_groups):
    """Experts that are copies of each other (equal logits: the lowest index
    first) or off by one step in one weight, far below what fp32 sums keep."""
    E, H, M = 64, 1024, 40
    w = rand(11, E, H) / math.sqrt(2 * H)
    w = w.bfloat16() if weight == "bf16" else w
    for e in range(8, E):  # every expert a near copy of one of eight
        w[e] = w[e % 8]
        if e % 3:
            c = (37 * e) % H
            w[e, c] = w[e, c] * (1 + 2.0 ** -7) if weight == "bf16" else w[e, c] * (1 + 2.0 ** -20)
    bias = (0.02 * rand(12, 8)).repeat(E // 8) if biased else None
    router, w = make_router(E, H, 12, M, weight, bias, w=w, scoring=scoring, groups=groups, top_groups=top_groups)
    check_routes(router, w, hidden(21, M, H), bias)


def test_route_masks_and_empty_rows():
    """A bias of -infinity takes an expert out; a token with fewer than k left
    gets ids of -1 and weights of 0, one whose groups are all masked nothing.
    A row of zeros ties everywhere; a NaN row takes nothing."""
    E, H, M, k = 48, 320, 9, 6
    x = hidden(5, M, H)
    x[3] = 0
    for groups, top_groups, left in ((1, 1, 4), (6, 2, 10), (6, 2, 0)):
        bias = torch.full((E,), -math.inf)
        bias[torch.arange(left) * 4 % E] = 0.01 * torch.arange(left).float()
        router, w = make_router(E, H, k, M, "bf16", bias, scoring="sigmoid", groups=groups, top_groups=top_groups)
        ids, wt, _ = check_routes(router, w, x, bias)
        if left == 0:
            assert bool((ids == -1).all()) and bool((wt == 0).all())
    for scoring in ("softmax", "sigmoid"):
        for bias in (None, 0.05 * rand(4, E)):
            router, w = make_router(E, H, k, M, "bf16", bias, scoring=scoring)
            check_routes(router, w, x, bias)
            bad = x.clone()
            bad[4, 17] = math.nan
            ids, wt = router(bad.cuda())
            good, gw = router(x.cuda())
            assert bool((ids[4] == -1).all()) and bool((wt[4] == 0).all())
            rest = [i for i in range(M) if i != 4]
            assert torch.equal(ids[rest], good[rest]) and torch.equal(wt[rest], gw[rest])


def test_route_infinite_bias_and_large_values():
    E, H, M, k = 40, 256, 6, 5
    bias = 0.05 * rand(4, E)
    bias[7], bias[30] = math.inf, math.inf
    for scoring in ("sigmoid", "softmax"):
        router, w = make_router(E, H, k, M, "bf16", bias, scoring=scoring)
        ids, _, _ = check_routes(router, w, hidden(2, M, H), bias)
        assert bool((ids[:, 0] == 7).all()) and bool((ids[:, 1] == 30).all())
    # logits of +-1e4: saturated scores, told apart by the logits
    router, w = make_router(E, H, k, M, "bf16", scoring="sigmoid", renorm=True)
    check_routes(router, w, (hidden(2, M, H).float() * 2.0 ** 14).bfloat16())


@pytest.mark.parametrize("M,E,H,k,weight,groups,top_groups", [
    (5, 48, 520, 6, "bf16", 1, 1), (40, 300, 1024, 8, "fp32", 1, 1), (400, 128, 264, 4, "bf16", 8, 4)])
def test_route_bias_that_evens_a_softmax(M, E, H, k, weight, groups, top_groups):
    """A bias that makes all scores of some tokens alike but for its rounding to
    fp32, while their probabilities differ: the sum over all experts decides."""
    x = hidden(91, M, H)
    w = rand(92, E, H) / math.sqrt(2 * H)
    w = w.bfloat16() if weight == "bf16" else w
    p = torch.softmax(x[M // 2].double() @ w.double().t(), 0)
    bias = (0.1 - p).float()
    x[0] = x[M // 2]
    router, w = make_router(E, H, k, M, weight, bias, w=w, groups=groups, top_groups=top_groups)
    check_routes(router, w, x, bias)


@pytest.mark.parametrize("scoring,biased,groups,top_groups,weight", [
    ("softmax", False, 1, 1, "bf16"), ("softmax", True, 1, 1, "fp32"), ("softmax", True, 8, 3, "bf16"),
    ("sigmoid", True, 8, 3, "fp32"), ("sigmoid", False, 1, 1, "bf16")])
def test_route_without_a_bound(scoring, biased, groups, top_groups, weight):
    """Squares of x that overflow leave no bound on the logits' errors, and ones
    that vanish a loose one: still the exact experts.  An infinity in x makes
    logits infinite: a softmax over them takes nothing."""
    E, H, M, k = 104, 520, 7, 6
    bias = 0.05 * rand(4, E) if biased else None
    g = torch.Generator().manual_seed(31)
    x = hidden(30, M, H)
    w = rand(29, E, H) / math.sqrt(2 * H)
    x[1] = (x[1].float() * 2.0 ** 64).bfloat16()
    x[4] = (x[4].float() * 2.0 ** -100).bfloat16()
    x[5] = 0
    x[5, 7] = 2.0 ** -130
    x[3, 9] = math.inf
    x[6] = torch.where(torch.rand(H, generator=g) < 0.5, x[6].float() * 2.0 ** 62, x[6].float()).bfloat16()
    # rows of +-2^64 saturate every score: only the logits' order is left, so no bias there
    rows = list(range(M)) if not biased and groups == 1 else [0, 2, 3, 4, 5]
    router, w = make_router(E, H, k, M, weight, bias, w=w, scoring=scoring, groups=groups, top_groups=top_groups)
    ids, wt = router(x.cuda())
    rid, rw, _ = ref.route(x, w, k, scoring, bias, groups, top_groups, True, 1.0)
    assert torch.equal(ids.cpu()[rows], rid[rows])
    if scoring == "softmax":
        assert bool((ids[3] == -1).all())
    assert bool(torch.isfinite(wt).all())


def test_route_is_the_same_alone_and_in_a_batch():
    E, H, k = 256, 2560, 8
    bias = 0.05 * rand(1, E)
    router, _ = make_router(E, H, k, 600, "bf16", bias, scoring="sigmoid", groups=8, top_groups=4)
    x = hidden(77, 600, H).cuda()
    ids, _ = router(x)
    for m in (0, 1, 299, 599):
        one, _ = router(x[m:m + 1])
        assert torch.equal(one[0], ids[m])
    for n in (2, 17, 40, 130):
        few, _ = router(x[:n])
        assert torch.equal(few, ids[:n])


# ---------------------------------------------------------------- FP8 linear

def fp8_weights(seed, rows, K, N):
    g = torch.Generator().manual_seed(seed)
    halves = rows // N
    codes = torch.randint(0, 256, (rows, K), generator=g, dtype=torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x3A  # no NaN
    scales = torch.exp(rand(seed + 1, halves * (-(-N // 128)), -(-K // 128))) * 1e-3
    return codes, scales


ACT = dict(swigluoai=dict(alpha=1.702, beta=1.0, limit=7.0))

FP8 = [
    # M, K, N, fn
    (1, 8, 8, "none"), (1, 128, 64, "silu"), (2, 136, 24, "none"), (1, 7168, 512, "silu"), (3, 320, 2560, "none"),
    (3, 7168, 264, "silu"), (4, 5128, 40, "none"), (5, 1000, 40, "gelu_tanh"), (8, 2560, 320, "relu2"), (13, 512, 136, "swigluoai"), (16, 256, 128, "none"),
    (17, 256, 128, "none"), (31, 392, 200, "silu"), (40, 2048, 96, "none"), (64, 128, 512, "relu2"),
    (65, 640, 264, "none"), (100, 1536, 328, "gelu_tanh"), (129, 264, 520, "swigluoai"), (256, 512, 512, "none"),
    (300, 1024, 776, "silu"), (520, 384, 256, "none"), (1030, 256, 1288, "none"), (700, 200, 648, "swigluoai"),
    (1500, 264, 1544, "swigluoai"), (2050, 392, 1032, "none"), (1200, 1160, 2056, "silu"),  # for the small ones
    (3100, 136, 4120, "none"), (2900, 648, 2056, "silu"), (3000, 1160, 4096, "relu2"),  # enough for the large tiles
]


@pytest.mark.parametrize("M,K,N,fn", FP8)
def test_fp8_linear(M, K, N, fn):
    desc = block.Fp8Desc(K, N, M, fn=fn, **ACT.get(fn, {}))
    codes, scales = fp8_weights(M + K, desc.rows, K, N)
    lin = block.Fp8Linear(desc, codes, scales)
    for m in {M, max(1, M // 2)}:
        x = hidden(m, m, K)
        y = lin(x.cuda()).cpu().double()
        want, tol = ref.fp8_linear(x, codes, scales, N, fn, **ACT.get(fn, {}))
        bad = (y - want).abs() > tol + (want.abs() + tol) * BF16 + 2.0 ** -133
        assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} outputs off, first at {bad.nonzero()[0].tolist()}"


def test_fp8_quantisation_borders():
    """Identity weights give back the quantised x: block maxima on both sides
    of 448 times a power of two, zero blocks, rounding ties, tiny and huge
    values."""
    K = 256
    codes = torch.zeros(K, K, dtype=torch.uint8)
    codes[torch.arange(K), torch.arange(K)] = 0x38  # 1.0
    scales = torch.ones(2, 2)
    x = torch.zeros(21, K)
    x[0, :5] = torch.tensor([448.0, 1.0, 1.0625, 1.1875, -0.015])
    x[1, :5] = torch.tensor([450.0, 1.0, 1.0625, 1.1875, -0.015])
    x[2, 128:131] = torch.tensor([2.0 ** -100, 2.0 ** -104, -2.0 ** -110])
    x[3, 0] = 3e38
    x[4, 0], x[4, 200] = 2.0 ** -133, 1.0
    x[5:] = rand(3, 16, K) * torch.exp(3 * rand(4, 16, 1))
    x = x.bfloat16()
    for M in (21, 3):
        lin = block.Fp8Linear(block.Fp8Desc(K, K, M), codes, scales)
        y = lin(x[:M].cuda()).cpu()
        want = ref.quantise(x[:M])
        # E4M3 times a power of two is a bf16 value unless it is below the normal range
        normal = want.abs() >= 2.0 ** -126
        assert torch.equal(y.double()[normal], want[normal])
        assert bool((y.double()[~normal].abs() <= 2.0 ** -126).all())


def test_fp8_nan_stays_in_its_token():
    M, K, N = 40, 384, 136
    desc = block.Fp8Desc(K, N, M, fn="silu")
    codes, scales = fp8_weights(1, desc.rows, K, N)
    lin = block.Fp8Linear(desc, codes, scales)
    x = hidden(8, M, K)
    good = lin(x.cuda())
    x[7, 200], x[21, 3] = math.nan, math.inf
    bad = lin(x.cuda())
    rest = [i for i in range(M) if i not in (7, 21)]
    assert bool(bad[[7, 21]].isnan().all()) and torch.equal(bad[rest], good[rest])
    one = lin(x[7:8].cuda())
    assert bool(one.isnan().all())


# ---------------------------------------------------------------- block norm

NORMS = [
    # M, H, residual, weight, branch, post, gate, sigmoid, pre
    (1, 8, "bf16", "bf16", 0, False, None, False, True), (1, 7168, "bf16", "bf16", 0, False, None, False, True),
    (5, 7168, "fp32", "fp32", 2, True, "token", True, True), (9, 512, "bf16", "fp32", 1, True, "channel", False, True),
    (7, 520, "fp32", "bf16", 1, True, "full", True, False), (3, 1024, "bf16", "bf16", 1, False, None, False, True),
    (4, 1032, "bf16", "bf16", 2, True, "channel", True, True), (6, 2048, "fp32", "fp32", 1, False, "token", False, False),
    (2, 2056, "bf16", "bf16", 1, True, "full", False, True), (33, 4096, "bf16", "bf16", 1, True, "channel", False, True),
    (3, 5000, "bf16", "fp32", 2, True, "token", False, True), (2, 8200, "fp32", "bf16", 1, True, "channel", True, True),
    (3, 16384, "bf16", "bf16", 1, True, None, False, True), (2, 16392, "fp32", "fp32", 2, True, "full", False, True),
    (1, 32768, "bf16", "bf16", 1, True, "token", True, True), (1000, 264, "bf16", "bf16", 1, True, "token", False, True),
]


@pytest.mark.parametrize("M,H,residual,weight,branch,post,gate,sig,pre", NORMS)
def test_block_norm(M, H, residual, weight, branch, post, gate, sig, pre):
    T = {"bf16": torch.bfloat16, "fp32": torch.float32}
    h = (2 * rand(1, M, H)).to(T[residual])
    y = hidden(2, M, H) if branch else None
    y2 = hidden(3, M, H) if branch > 1 else None
    shape = {None: None, "channel": (H,), "token": (M, 1), "full": (M, H)}[gate]
    g = None if shape is None else (1 + rand(4, *shape)).to(T[weight])
    pw = (1 + 0.2 * rand(5, H)).to(T[weight]) if post else None
    nw = (0.1 * rand(6, H)).to(T[weight]) if pre else None
    kw = dict(eps=1e-5, residual_scale=0.75, branch_scale=1.5, weight_offset=0.5, gate_sigmoid=sig)
    dev = [None if t is None else t.cuda() for t in (h, y, y2, g, pw, nw)]
    before = [None if t is None else t.clone() for t in dev]
    h2, x = block.block_norm(dev[0], dev[1], dev[2], gate=dev[3], post_weight=dev[4], pre_weight=dev[5], **kw)
    for a, b in zip(dev, before):
        assert a is None or torch.equal(a, b)
    stored = None if h2 is None else h2.cpu()
    want, mag, wx = ref.norm(h, y, y2, g, pw, nw, 1e-5, 0.75, 1.5, 0.5, sig, stored)
    # The mean of squares: at most 32 values in a row per lane and 10 levels of
    # a tree, each within 2^-24, half of that in its root; a dozen roundings of
    # products, sums, the root, the sigmoid's exponential and quotient after it.
    part = 64 * FP32
    if branch:
        step = FP32 if residual == "fp32" else BF16
        assert bool(((stored.double() - want).abs() <= mag * part * (1 + step) + want.abs() * step).all())
    if pre:
        assert bool(((x.cpu().double() - wx).abs() <= wx.abs() * (part + BF16 * (1 + part)) + 1e-38).all())
    if branch and pre:
        # the fused norm of h' is the norm of h' on its own, bit for bit
        assert torch.equal(block.block_norm(h2, pre_weight=dev[5], eps=1e-5, weight_offset=0.5)[1], x)
        # in place
        hin = dev[0].clone()
        h3, x3 = block.block_norm(hin, dev[1], dev[2], gate=dev[3], post_weight=dev[4], pre_weight=dev[5], h_out=hin, **kw)
        assert h3 is hin and torch.equal(h3, h2) and torch.equal(x3, x)


def test_block_norm_zero_and_nan_rows():
    M, H = 4, 640
    h = rand(1, M, H).bfloat16()
    y = hidden(2, M, H)
    y[1] = 0
    h[2] = 0
    y[2] = 0
    y[3, 5] = math.nan
    w = torch.ones(H, dtype=torch.bfloat16)
    h2, x = block.block_norm(h.cuda(), y.cuda(), post_weight=w.cuda(), pre_weight=w.cuda())
    assert torch.equal(h2[1].cpu(), h[1]) and bool((h2[2] == 0).all()) and bool((x[2] == 0).all())
    assert bool(h2[3].isnan().all()) and bool(x[3].isnan().all()) and bool(torch.isfinite(x[:3]).all())


# ---------------------------------------------------------------- together

def make_block(M, k=8, seed=0, shared=True):
    wl = synth.WORKLOADS["tiny_mxfp4"].replace(E=64, H=512, I=128, M=M, k=k)
    d = synth.generate(wl)
    layer = make_layer("mxfp4", d, k, M)
    H = wl.H
    bias = 0.05 * rand(seed + 1, wl.E)
    router, rw = make_router(wl.E, H, k, M, "fp32", bias, scoring="sigmoid", groups=8, top_groups=4, scale=1.5)
    up = block.Fp8Desc(H, 384, M, fn="silu")
    down = block.Fp8Desc(384, H, M)
    uc, us = fp8_weights(seed + 2, up.rows, H, 384)
    dc, ds = fp8_weights(seed + 3, H, 384, H)
    us, ds = us * 0.2, ds * 0.2
    su, sd = (block.Fp8Linear(up, uc, us), block.Fp8Linear(down, dc, ds)) if shared else (None, None)
    pre, post = (1 + 0.1 * rand(seed + 4, H)).bfloat16(), (1 + 0.1 * rand(seed + 5, H)).bfloat16()
    blk = block.Fp4MoEBlock(layer, router, pre.cuda(), post.cuda(), su, sd, residual_scale=0.9, branch_scale=0.5)
    return blk, d, (uc, us, dc, ds), pre, post


@pytest.mark.parametrize("M", [1, 5, 40, 200])
def test_whole_block(M):
    """Norm, router, experts, shared expert and the gated residual as a user
    runs them: every step against its reference on the step's own input."""
    blk, d, (uc, us, dc, ds), pre, post = make_block(M)
    H = blk.layer.desc.H
    h = rand(31, M, H).bfloat16()
    gate = (0.5 * rand(32, M, 1)).bfloat16()
    nxt = (1 + 0.1 * rand(33, H)).bfloat16()
    h2, x2 = blk(h.cuda(), gate=gate.cuda(), gate_sigmoid=True, next_weight=nxt.cuda())
    # the same steps one by one
    _, x = block.block_norm(h.cuda(), pre_weight=pre.cuda())
    ids, w = blk.router(x)
    y = blk.layer(x, ids, w)
    s1 = blk.shared_up(x)
    s2 = blk.shared_down(s1)
    h3, x3 = block.block_norm(h.cuda(), y, s2, gate=gate.cuda(), gate_sigmoid=True, post_weight=post.cuda(),
                              pre_weight=nxt.cuda(), residual_scale=0.9, branch_scale=0.5)
    assert torch.equal(h2, h3) and torch.equal(x2, x3)
    # experts against the oracle on the router's routes
    dm = dict(d, x=x.view(torch.int16).cpu().numpy().view(np.uint16), ids=ids.cpu().numpy(), w=w.cpu().numpy())
    acc, _ = oracle.forward_f32("mxfp4", dm)
    compare(y.view(torch.int16).cpu().numpy().view(np.uint16), acc, f"block M={M}")
    for got, xin, c, s, N, fn in ((s1, x, uc, us, 384, "silu"), (s2, s1, dc, ds, H, "none")):
        want, tol = ref.fp8_linear(xin.cpu(), c, s, N, fn)
        assert bool(((got.cpu().double() - want).abs() <= tol + (want.abs() + tol) * BF16 + 2.0 ** -133).all())
    want, mag, _ = ref.norm(h, y.cpu(), s2.cpu(), gate, post, None, 1e-6, 0.9, 0.5, 0.0, True)
    assert bool(((h2.cpu().double() - want).abs() <= mag * 64 * FP32 * 1.01 + want.abs() * BF16).all())


def test_captured_block_replays():
    """The whole block captured into a graph and replayed on new inputs, with
    eager calls of the same block in between."""
    for M in (3, 150):
        blk, *_ = make_block(M)
        H = blk.layer.desc.H
        nxt = torch.ones(H, dtype=torch.bfloat16, device="cuda")
        inputs = [rand(40 + i, M, H).bfloat16().cuda() for i in range(4)]
        want = [tuple(t.clone() for t in blk(h, next_weight=nxt)) for h in inputs]
        static = inputs[0].clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            blk(static, next_weight=nxt)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = blk(static, next_weight=nxt)
        for i in (1, 3, 0, 2, 1):
            static.copy_(inputs[i])
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[0], want[i][0]) and torch.equal(out[1], want[i][1])
            eager = blk(inputs[(i + 1) % 4], next_weight=nxt)
            torch.cuda.synchronize()
            assert torch.equal(eager[0], want[(i + 1) % 4][0])


def test_other_stream_and_empty_batch():
    M = 24
    blk, *_ = make_block(M)
    H = blk.layer.desc.H
    h = rand(50, M, H).bfloat16().cuda()
    nxt = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    want = blk(h, next_weight=nxt)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = blk(h, next_weight=nxt, stream=s)
    raw = blk(h, next_weight=nxt, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(raw[1], want[1])
    e0, e1 = blk(h[:0], next_weight=nxt)
    assert e0.shape == (0, H) and e1.shape == (0, H)
    torch.cuda.synchronize()


BAND = 4096


def _banded(shape, dtype, fill=0xA5):
    n = math.prod(shape) * torch.empty(0, dtype=dtype).element_size()
    big = torch.full((BAND + -(-n // 256) * 256 + BAND,), fill, dtype=torch.uint8, device="cuda")
    return big, n, big[BAND:BAND + n].view(dtype).view(shape)


def _intact(big, n, fill=0xA5):
    torch.cuda.synchronize()
    return bool((big[:BAND] == fill).all()) and bool((big[BAND + n:] == fill).all())


@pytest.mark.parametrize("M", [1, 7, 19, 70, 300])
def test_writes_stay_inside(M):
    """Outputs and workspaces lie inside larger allocations whose bytes before
    and after stay as they were; rows behind the last token are not written."""
    E, H, k = 72, 392, 5
    router, _ = make_router(E, H, k, M, "fp32")
    x = hidden(1, M, H).cuda()
    bands = [_banded((M, k), torch.int32), _banded((M, k), torch.float32), _banded((M, E), torch.float32),
             _banded((block.router_workspace_bytes(router.desc, M),), torch.uint8)]
    router.workspace = bands[3][2]
    router._at = router._at[0], bands[3][2].data_ptr(), bands[3][1]
    router(x, bands[0][2], bands[1][2], bands[2][2])
    assert all(_intact(b, n) for b, n, _ in bands)
    for fn, N in (("silu", 136), ("none", 264)):
        desc = block.Fp8Desc(H, N, M, fn=fn)
        lin = block.Fp8Linear(desc, *fp8_weights(2, desc.rows, H, N))
        o, w = _banded((M, N), torch.bfloat16), _banded((block.fp8_workspace_bytes(desc, M),), torch.uint8)
        lin.workspace = w[2]
        lin._at = lin._at[0], w[2].data_ptr(), w[1]
        lin(x, out=o[2])
        assert _intact(*o[:2]) and _intact(*w[:2])
    ho, xo = _banded((M, H), torch.float32), _banded((M, H), torch.bfloat16)
    wt = torch.ones(H, device="cuda")
    block.block_norm(x.float(), x, post_weight=wt, pre_weight=wt, h_out=ho[2], x_out=xo[2])
    assert _intact(*ho[:2]) and _intact(*xo[:2])


def test_offsets_past_32_bits():
    """300000 tokens of 7168 values, 4.3 GB: the same 100 rows over and over give
    the same outputs over and over, the last ones too."""
    M, H, n = 300000, 7168, 100
    rows = hidden(60, n, H).cuda()
    x = rows.repeat(M // n, 1)

    def alike(t):
        t = t.view(M // n, n, -1)
        return bool((t == t[0]).all())

    router, _ = make_router(8, H, 3, M, scoring="sigmoid")
    ids, w = router(x)
    few, _ = router(rows)
    assert alike(ids) and alike(w) and torch.equal(ids[:n], few)
    desc = block.Fp8Desc(H, 24, M, fn="silu")
    y = block.Fp8Linear(desc, *fp8_weights(61, desc.rows, H, 24))(x)
    assert alike(y) and bool(y.isfinite().all())
    del y
    gate = torch.full((M, 1), 0.5, dtype=torch.bfloat16, device="cuda")
    one = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    h, xo = block.block_norm(x, x, gate=gate, post_weight=one, pre_weight=one)
    assert alike(h) and alike(xo)
