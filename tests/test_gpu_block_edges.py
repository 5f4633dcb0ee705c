"""The operators around the layer at the ends of their documented ranges."""
from __future__ import annotations

import math

import pytest
import torch

import block_ref as ref
from block_scaled_fp4_gather_amd import block
from gpu_util import say
from test_gpu_block import fp8_weights, hidden, make_router, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    say(f"\n[gpu] {request.node.nodeid}")
    yield


@pytest.mark.parametrize("M", [1, 40, 40000])  # quantised in the product's launch, few tokens, tiles
def test_fp8_products_are_cut_as_the_header_says(M):
    """256 + t - 256: t in a group of 8 with the 256s is cut towards zero to a
    multiple of 2^-13 * 256 = 1 / 32; in a group of its own it is whole."""
    K, N = 128, 64
    codes = torch.zeros(N, K, dtype=torch.uint8)
    codes[:, :] = 0x38  # 1.0
    codes[:, 2] = 0xB8  # -1.0
    codes[1::2, 1] = 0xB8
    lin = block.Fp8Linear(block.Fp8Desc(K, N, M), codes, torch.ones(1, 1))
    t = torch.tensor([1.875 * 2.0 ** (8 - j) for j in range(1, 15)], dtype=torch.float64)
    x = torch.zeros(len(t), 2, K, dtype=torch.float64)
    x[:, :, 0] = x[:, :, 2] = 256.0
    x[:, 0, 1] = t   # in the 256s' group
    x[:, 1, 9] = t   # in the next one
    cut = torch.floor(t * 32) / 32
    assert bool((cut[:10] == t[:10]).all()) and cut[10:].tolist() == [7 / 32, 3 / 32, 1 / 32, 0.0]
    want = torch.stack([cut, t], 1).view(-1, 1) * torch.ones(N, dtype=torch.float64)
    want[::2, 1::2] *= -1  # both signs
    x, rows = x.view(-1, K).bfloat16(), torch.arange(M) % (2 * len(t))
    for start in range(2 * len(t)) if M == 1 else (0,):
        at = (rows + start) % (2 * len(t))
        y = lin(x[at].cuda()).cpu()
        assert torch.equal(y.double(), want[at])


def test_block_norm_of_more_rows_than_a_launch_has_threads():
    """2^26 rows of 8 values and a few more, 64 threads a row: past the 2^32
    threads of one launch."""
    M, H, n = (1 << 26) + 1031, 8, 1031
    rows = rand(80, n, H).bfloat16().cuda()
    h = torch.zeros(M, H, dtype=torch.bfloat16, device="cuda")
    h[:n], h[-n:] = rows, rows
    h[1 << 25:(1 << 25) + n] = rows
    w = (1 + 0.1 * rand(81, H)).bfloat16().cuda()
    want = block.block_norm(rows, pre_weight=w)[1]
    x = block.block_norm(h, pre_weight=w)[1]
    for at in (0, 1 << 25, M - n):
        assert torch.equal(x[at:at + n], want)
    assert bool((x[n:1 << 25] == 0).all()) and bool((x[(1 << 25) + n:M - n] == 0).all())


@pytest.mark.parametrize("M", [40, 300])
@pytest.mark.parametrize("xe,we", [(0, -83), (0, -100), (60, -120), (-110, 20)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_near_ties_of_tiny_values(scoring, xe, we, M):
    """Weights whose squares vanish in 32 bits, or whose terms of bf16 fall
    below its normal numbers, and hidden states of that kind: without a bias
    the order is that of the logits, however small."""
    E, H = 64, 1024
    w = rand(11, E, H) / math.sqrt(2 * H)
    for e in range(8, E):
        w[e] = w[e % 8]
        if e % 3:
            c = (37 * e) % H
            w[e, c] = w[e, c] * (1 + 2.0 ** -20)
    w = w * 2.0 ** we
    x = (rand(21, M, H) * 2.0 ** xe).bfloat16()
    router, w = make_router(E, H, 12, M, "fp32", None, w=w, scoring=scoring)
    ids, _ = router(x.cuda())
    rid, _, _ = ref.route(x, w, 12, scoring)
    assert torch.equal(ids.cpu(), rid)


@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("biased,groups", [(False, 8), (True, 8), (True, 1)])
def test_route_softmax_of_logits_off_by_more_than_an_exponent(M, biased, groups):
    """Logits near 2^40, which fp32 holds to 2^16, while what decides is a
    difference of 1 between the two largest: the later of two near copies, in
    another group, is e times as probable."""
    E, H = 64, 520
    x = (rand(70, M, H) * 2.0 ** 36).bfloat16()
    x[:, 17] = 128.0
    w = (0.25 * rand(71, E, H)).bfloat16()
    top = (x[:, :16].sign().float() * 8).bfloat16()  # expert 3 and its copy 61 stand out for the rows of x[0]'s signs
    x[:, :16] = x[:, :16].abs() * top[0].sign()
    w[3, :16] = top[0]
    w[3, 17] = 1.0
    w[61] = w[3]
    w[61, 17] = 1.0 + 2.0 ** -7
    bias = torch.full((E,), 0.125) if biased else None
    router, w = make_router(E, H, 1, M, "bf16", bias, w=w, scoring="softmax", groups=groups, top_groups=1)
    ids, _ = router(x.cuda())
    rid, _, z = ref.route(x, w, 1, "softmax", bias, groups, 1)
    assert bool((rid == 61).all()) and torch.equal(z[:, 61] - z[:, 3], torch.ones(M, dtype=torch.float64))
    assert torch.equal(ids.cpu(), rid)


@pytest.mark.parametrize("H", [264, 4096, 16384])
@pytest.mark.parametrize("h_in,x_in", [("h", "y"), ("y", "h"), ("y2", "y"), ("h", "y2"), (None, "h"), ("y", None)])
def test_block_norm_over_its_inputs(H, h_in, x_in):
    """Outputs in the place of h, y and y2: what they are elsewhere."""
    M = 5
    t = {n: rand(i, M, H).bfloat16().cuda() for i, n in enumerate(("h", "y", "y2"))}
    w = (1 + 0.1 * rand(7, H)).bfloat16().cuda()
    gate = (1 + 0.1 * rand(8, M, H)).bfloat16().cuda()
    kw = dict(gate=gate, post_weight=w, pre_weight=w, residual_scale=0.75)
    want = block.block_norm(t["h"], t["y"], t["y2"], **kw)
    got = block.block_norm(t["h"], t["y"], t["y2"], h_out=t.get(h_in), x_out=t.get(x_in), **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert h_in is None or got[0] is t[h_in]
    assert x_in is None or got[1] is t[x_in]


def logits_coefficient(E, H, planes, M):
    """The kernel's bound on a logit's error over the magnitudes of its
    products, from the plan of a call: chains of 8 instructions of four groups
    each, a group's cuts, the sums over chains, waves and slices."""
    blocks = -(-H // 32)
    if M <= 256:
        kb, unit, splits = blocks, 4, -(-blocks // 32)
    else:
        kb, unit = -(-blocks // 8) * 8, 8 // planes
        wide = E > 128 and planes == 1
        tiles = -(-M // (128 if wide or planes == 3 else 64)) * -(-E // (256 if wide else 128))
        splits = min(8, max(1, (256 if wide else 512) // tiles))
    units = -(-kb // unit)
    per = -(-units // min(splits, units)) * unit
    return (4 * 8 + 8 + per * planes // 4 + 4 + -(-kb // per)) * 2.0 ** -24


LOGITS = [  # M, H, E, weight: every kernel of the logits, in one slice and in several
    (5, 512, 40, "bf16"), (16, 7168, 256, "bf16"), (30, 4096, 100, "fp32"), (200, 2560, 200, "bf16"),
    (256, 7168, 300, "fp32"), (257, 7168, 64, "bf16"), (300, 7168, 256, "bf16"), (300, 2560, 512, "fp32"),
    (17000, 1096, 100, "bf16"), (17000, 2048, 256, "bf16"), (16500, 1096, 130, "fp32"),
]


@pytest.mark.parametrize("signs", ["mixed", "alike"])
@pytest.mark.parametrize("M,H,E,weight", LOGITS)
def test_logits_are_within_the_bound_that_the_choice_goes_by(M, H, E, weight, signs):
    """Values of very different sizes, of both signs and of one, where cuts
    towards zero add up.  Recomputed logits are exact."""
    x = rand(1, M, H) * torch.exp2(3 * rand(2, 1, H))
    w = rand(3, E, H) * torch.exp2(rand(4, E, H)) / math.sqrt(H)
    if signs == "alike":
        x, w = x.abs(), w.abs()
    x = x.bfloat16()
    router, w = make_router(E, H, min(E, 4), M, weight, None, w=w)
    lg = torch.empty(M, E, device="cuda")
    router(x.cuda(), logits=lg)
    rows = torch.unique(torch.cat([torch.arange(0, M, max(1, M // 300)), torch.arange(max(0, M - 70), M)]))
    xd, wd = x[rows].double(), w.double()
    z = xd @ wd.t()
    bound = logits_coefficient(E, H, 3 if weight == "fp32" else 1, M) * xd.norm(dim=1, keepdim=True) * wd.norm(dim=1).max()
    off = (lg.cpu().double()[rows] - z).abs()
    say(f"  largest error over the bound {float((off / bound).max()):.3f}, over the magnitudes' "
        f"{float((off / (bound / (xd.norm(dim=1, keepdim=True) * wd.norm(dim=1).max()) * (xd.abs() @ wd.abs().t()))).max()):.3f}")
    assert bool((off <= bound + z.abs() * 2.0 ** -24).all())


@pytest.mark.parametrize("scoring,biased,groups,top_groups", [
    ("softmax", False, 1, 1), ("sigmoid", True, 1, 1), ("sigmoid", True, 8, 3), ("softmax", True, 8, 3)])
@pytest.mark.parametrize("M,H,E,weight", [
    (300, 1024, 64, "bf16"), (300, 256, 64, "bf16"), (17000, 1024, 64, "bf16"),     # tiles of 64 x 128
    (300, 1024, 200, "bf16"), (300, 256, 200, "bf16"), (17000, 520, 200, "bf16"),   # of 128 x 256
    (300, 1024, 64, "fp32"), (300, 64, 200, "fp32"), (8500, 1024, 200, "fp32")])    # of three planes
def test_route_near_ties_of_many_tokens(M, H, E, weight, scoring, biased, groups, top_groups):
    """Near copies of eight experts, as in the few tokens' test, through the
    tiled kernels with several slices of H and with one."""
    w = rand(11, E, H) / math.sqrt(2 * H)
    w = w.bfloat16() if weight == "bf16" else w
    for e in range(8, E):
        w[e] = w[e % 8]
        if e % 3:
            c = (37 * e) % H
            w[e, c] = w[e, c] * (1 + (2.0 ** -7 if weight == "bf16" else 2.0 ** -20))
    bias = (0.02 * rand(12, 8)).repeat(E // 8) if biased else None
    x = hidden(21, min(M, 600), H).repeat(-(-M // 600), 1)[:M] if M > 600 else hidden(21, M, H)
    router, w = make_router(E, H, 12, M, weight, bias, w=w, scoring=scoring, groups=groups, top_groups=top_groups)
    ids, wt = router(x.cuda())
    # Copies of an expert have one logit.  A product over all experts does not
    # give them that (it may sum some columns in another order: 2^-52 apart,
    # seen once in 600 rows), so it is taken over the distinct ones; the
    # identity passes it on as it is.
    kinds, of = torch.unique(w, dim=0, return_inverse=True)
    z = (x[:600].double() @ kinds.double().t())[:, of]
    rid, rw, _ = ref.route(z, torch.eye(E), 12, scoring, bias, groups, top_groups)
    at = torch.arange(M) % 600
    assert torch.equal(ids.cpu(), rid[at])
    delta = logits_coefficient(E, H, 3 if weight == "fp32" else 1, M) * float(x.double().norm(dim=1).max() * w.double().norm(dim=1).max())
    # a weight is a quotient of p and their sum, each within e^delta of its own, and a few roundings
    assert bool(((wt.cpu().double() - rw[at]).abs() <= rw[at] * (4 * delta + 2.0 ** -22)).all())


def test_a_long_prompt_in_sampled_rows():
    """The largest plans whole: 16384 tokens through the grouped router of 256
    experts, 8192 through the gated FP8 map.  Rows at the borders of tiles and
    some between them, each against 64 bits."""
    M, H, E = 16384, 7168, 256
    bias = 0.05 * rand(9, E)
    x = hidden(90, M, H)
    router, w = make_router(E, H, 8, M, "bf16", bias, scoring="sigmoid", groups=8, top_groups=4, scale=1.5)
    ids, wt = router(x.cuda())
    rows = torch.unique(torch.cat([torch.arange(0, M, 257), torch.arange(127, M, 1024), torch.arange(128, M, 1024),
                                   torch.arange(M - 5, M)]))
    rid, rw, _ = ref.route(x[rows], w, 8, "sigmoid", bias, 8, 4, True, 1.5)
    assert torch.equal(ids.cpu()[rows], rid)
    delta = logits_coefficient(E, H, 1, M) * float(x[rows].double().norm(dim=1).max() * w.double().norm(dim=1).max())
    assert bool(((wt.cpu().double()[rows] - rw).abs() <= rw * (4 * delta + 2.0 ** -22)).all())
    M, K, N = 8192, 7168, 2048
    act = dict(alpha=1.702, beta=1.0, limit=7.0)
    desc = block.Fp8Desc(K, N, M, fn="swigluoai", **act)
    codes, scales = fp8_weights(91, desc.rows, K, N)
    y = block.Fp8Linear(desc, codes, scales)(x[:M].cuda()).cpu().double()
    rows = torch.unique(torch.cat([torch.arange(0, M, 409), torch.arange(255, M, 2048), torch.arange(256, M, 2048),
                                   torch.tensor([M - 1])]))
    want, tol = ref.fp8_linear(x[rows], codes, scales, N, "swigluoai", **act)
    assert bool(((y[rows] - want).abs() <= tol + (want.abs() + tol) * 2.0 ** -8 + 2.0 ** -133).all())


@pytest.mark.parametrize("weight,scoring,biased", [("fp32", "sigmoid", True), ("bf16", "softmax", False)])
@pytest.mark.parametrize("M", [1, 37, 300])
def test_route_at_the_largest_sizes(M, weight, scoring, biased):
    """65536 values, 512 experts in 64 groups, 64 experts a token."""
    E, H, k = 512, 65536, 64
    bias = 0.05 * rand(9, E) if biased else None
    x = hidden(1, M, H)
    w = (rand(3, E, H) / math.sqrt(2 * H)).to(torch.bfloat16 if weight == "bf16" else torch.float32)
    router, w = make_router(E, H, k, M, weight, bias, w=w, scoring=scoring, groups=64, top_groups=9)
    ids, wt = router(x.cuda())
    rid, rw, _ = ref.route(x, w, k, scoring, bias, 64, 9)
    assert torch.equal(ids.cpu(), rid)
    delta = logits_coefficient(E, H, 3 if weight == "fp32" else 1, M) * float(x.double().norm(dim=1).max() * w.double().norm(dim=1).max())
    assert bool(((wt.cpu().double() - rw).abs() <= rw * (4 * delta + 2.0 ** -22)).all())


def test_route_of_a_million_tokens():
    E, H, k, M = 16, 64, 3, 1 << 20
    x = hidden(1, M, H)
    router, w = make_router(E, H, k, M, "bf16", None, scoring="sigmoid")
    ids, _ = router(x.cuda())
    rid, _, z = ref.route(x, w, k, "sigmoid")
    assert torch.equal(ids.cpu(), rid)


@pytest.mark.parametrize("M", [1, 3, 16, 40, 300])
def test_fp8_longest_rows(M):
    K, N = 1 << 20, 8
    codes, scales = fp8_weights(4, N, K, N)
    x = hidden(5, M, K)
    y = block.Fp8Linear(block.Fp8Desc(K, N, M), codes, scales)(x.cuda()).cpu().double()
    want, tol = ref.fp8_linear(x, codes, scales, N)
    assert bool(((y - want).abs() <= tol + (want.abs() + tol) * 2.0 ** -8).all())


@pytest.mark.parametrize("M", [1, 20])
def test_fp8_most_rows(M):
    """2^26 outputs of 8 values with gate and up, the last ones at their place."""
    K, N = 8, 1 << 26
    g = torch.Generator(device="cuda").manual_seed(6)
    codes = torch.randint(0, 120, (2 * N, K), generator=g, dtype=torch.uint8, device="cuda")
    scales = torch.rand(2 * N // 128, 1, generator=g, device="cuda") + 0.5
    x = torch.eye(8)[torch.arange(M) % 8].bfloat16()  # one value a token: one weight an output, and no cut
    y = block.Fp8Linear(block.Fp8Desc(K, N, M, fn="relu2"), codes[:N], scales[:N // 128])(x.cuda())
    for m in range(M):
        c = m % 8
        v = codes[:N, c].view(torch.float8_e4m3fn).float().view(-1, 128) * scales[:N // 128]
        assert torch.equal(y[m].view(-1, 128), (v * v).bfloat16()), m
    del y, v
    y = block.Fp8Linear(block.Fp8Desc(K, N, M, fn="silu"), codes, scales)(x.cuda())
    for m in range(0, M, 7):
        c = m % 8
        gate, up = (codes[i * N:(i + 1) * N, c].view(torch.float8_e4m3fn).float().view(-1, 128) *
                    scales[i * (N // 128):(i + 1) * (N // 128)] for i in (0, 1))
        want = gate / (1 + torch.exp(-gate)) * up
        # the activation within 2^-16 as elsewhere, and the rounding to bf16
        assert bool(((y[m].view(-1, 128).float() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -15)).all()), m


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("k", [1, 3])
def test_route_with_infinite_and_nan_weights(k, biased, renorm, scoring):
    """Experts with a weight of -infinity, of +infinity or of NaN next to
    ordinary ones: logits of +-infinity and NaN by the sign of x.  An infinity
    that a bias has taken weighs nothing; no weight is NaN."""
    E, H, M = 12, 264, 16
    x = hidden(33, M, H)
    x[:, 5] = x[:, 5].abs() + 1
    x[::2, 9] = 2.0
    x[1::2, 9] = -2.0
    w = rand(34, E, H) / math.sqrt(2 * H)
    w[2, 5] = -math.inf          # -infinity for every token
    w[7, 5] = -math.inf
    if scoring == "sigmoid":     # a softmax has no probabilities then
        w[4, 9] = math.inf       # by turns
        w[9, 100] = math.nan
    bias = 0.05 * rand(35, E) if biased else None
    if biased:
        bias[2] = bias[7] = 8.0  # these first
    router, w = make_router(E, H, k, M, "fp32", bias, w=w, scoring=scoring, renorm=renorm)
    ids, wt = router(x.cuda())
    rid, rw, _ = ref.route(x, w, k, scoring, bias, renorm=renorm)
    assert torch.equal(ids.cpu(), rid)
    if biased:
        assert bool((ids[:, 0].cpu() == (2 if bias[2] >= bias[7] else 7)).all())
    assert bool(torch.isfinite(wt).all())
    # exact logits, weights in 64 bits but for an fp32 sum of 12 terms
    assert bool(((wt.cpu().double() - rw).abs() <= rw * 16 * 2.0 ** -23).all())
