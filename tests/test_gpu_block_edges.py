"""The operators around the layer at the ends of their documented ranges."""
from __future__ import annotations

import math

import pytest
import torch

import block_ref as ref
from block_scaled_fp4_gather_amd import block
from gpu_util import say
from test_gpu_block import make_router, rand

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
