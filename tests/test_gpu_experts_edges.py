"""Ends of the ranges that include/moe_fp4.h gives for FP4 quantisation, the
MXFP4 linear map, grouped products and the routes' calls."""
from __future__ import annotations

import pytest
import torch

import experts_ref as ref
from block_scaled_fp4_gather_amd import block, experts
from gpu_util import say
from test_gpu_experts import BF16, linear_bound, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    say(f"\n[gpu] {request.node.nodeid}")
    yield


# ---------------------------------------------------------------- very wide maps

def wide_map(M, N, fn="none", K=32):
    """A map whose outputs are exact: one block of 32, so that an output is a sum
    of 32 quarters of whole numbers below 36, times a power of two."""
    g = torch.Generator(device="cuda").manual_seed(N)
    desc = experts.Fp4Desc(K, N, M, fn)
    codes = torch.empty(desc.rows, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(desc.rows, K // 32, dtype=torch.uint8, device="cuda")
    for a in range(0, desc.rows, 1 << 24):
        codes[a:a + (1 << 24)].random_(0, 256, generator=g)
        scales[a:a + (1 << 24)].random_(120, 126, generator=g)
    return experts.Fp4Linear(desc, codes, scales), codes, scales


def values(codes, scales):
    return experts.fp4_dequantize((codes, scales), "mxfp4", torch.float32)


def check_wide(lin, codes, scales, x, rows):
    """Every output of the given rows, those that the call did not write
    among them; nothing around the outputs is touched."""
    M, N = x.shape[0], lin.desc.N
    big = torch.full((M * N + 2048,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = big[1024:-1024].view(M, N)
    out.fill_(float("nan"))
    lin(x, out=out)
    assert bool((big[:1024] == 7).all()) and bool((big[-1024:] == 7).all())
    q = experts.fp4_quantize(x[rows].contiguous())
    xv = values(q.codes, q.scales)
    for a in range(0, N, 1 << 20):
        want = (xv @ values(codes[a:a + (1 << 20)], scales[a:a + (1 << 20)]).t()).bfloat16()
        assert torch.equal(out[rows, a:a + (1 << 20)], want), a
    last = slice(N - 24, N)
    exact, _ = ref.linear(q.codes.cpu(), q.scales.cpu(), codes[last].cpu(), scales[last].cpu())
    assert torch.equal(out[rows, last].cpu(), exact.bfloat16())


# Outputs of 256 tokens that are 2^30 bytes, and past them: 2^31 and 2^32, with a
# last tile that is cut; of 32 tokens that are 2^31 bytes, and past them.
@pytest.mark.parametrize("M,N", [(257, 1 << 21), (257, (1 << 21) + 8), (300, 4194312), (256, 1 << 23), (70, 1 << 25),
                                 (70, (1 << 25) + 8), (33, 1 << 26)])
def test_linear_of_very_many_features(M, N):
    lin, codes, scales = wide_map(M, N)
    rows = torch.tensor(sorted({0, 1, 31, 32, M // 2, M - 2, M - 1}), device="cuda")
    check_wide(lin, codes, scales, rand(2, M, 32).bfloat16().cuda(), rows)


def test_linear_of_very_many_features_and_tokens():
    """2^35 outputs, in more than 2^32 threads."""
    M, N = 513, 1 << 26
    lin, codes, scales = wide_map(M, N)
    check_wide(lin, codes, scales, rand(2, M, 32).bfloat16().cuda(), torch.tensor([0, 63, 64, 511, 512], device="cuda"))


# Gated: outputs past 2^31 bytes in a tile; and up to the most features, whose
# weights' subtiles need 2^32 threads of the few-token kernel.
@pytest.mark.parametrize("M,N", [(300, (1 << 22) + 8), (1, (1 << 26) - 16), (2, (1 << 26) - 8), (4, 1 << 26), (5, 1 << 26),
                                 (20, 1 << 26)])
def test_gated_linear_of_very_many_features(M, N):
    lin, codes, scales = wide_map(M, N, "silu")
    x = rand(2, M, 32).bfloat16().cuda()
    out = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    lin(x, out=out)
    assert not any(bool(torch.isnan(row).any()) for row in out)
    q = experts.fp4_quantize(x)
    some = torch.cat([torch.arange(40), torch.arange(N // 2 - 20, N // 2 + 20), torch.arange(N - 40, N)])
    both = torch.cat([some, N + some]).cuda()
    exact, s = ref.linear(q.codes.cpu(), q.scales.cpu(), codes[both].cpu(), scales[both].cpu())
    want, tol = linear_bound(exact, s, len(some), "silu", 32)
    assert bool(((out[:, some.cuda()].cpu().double() - want).abs() <= tol).all())


# ---------------------------------------------------------------- every bf16 value

def test_quantize_every_bf16_value():
    """All finite bf16 values under every scale that a block can give them: next
    to largest magnitudes 2^e and 1.9921875 2^e of the same exponent and of larger
    ones.  A linear map whose weights are a one in each row gives the values back,
    whichever kernel quantises its tokens; it may take those below 2^-126 as zeros."""
    bits = torch.arange(65536, dtype=torch.int32)
    every = bits.to(torch.int16).view(torch.bfloat16)
    every = every[torch.isfinite(every)]
    rows = []
    mag = every.abs().float()
    exponent = torch.where(mag > 0, torch.frexp(mag)[1] - 1, torch.full_like(bits[: len(every)], -133)).clamp(min=-133)
    for up in (0, 1, 2, 3, 4, 9):
        for m in (1.0, 1.9921875):
            top = torch.ldexp(torch.full_like(mag, m), (exponent + up).clamp(max=127)).bfloat16()
            keep = mag <= top.float()
            block_ = torch.zeros(len(every), 32, dtype=torch.bfloat16)
            block_[:, 0], block_[:, 1], block_[:, 31] = top, every, -every
            rows.append(block_[keep])
    x = torch.cat(rows)
    x = x[: len(x) // 8 * 8].view(-1, 256)
    q = experts.fp4_quantize(x.cuda())
    codes, scales, _ = ref.quantize(x[None], "mxfp4")
    assert torch.equal(q.scales.cpu(), scales[0]) and torch.equal(q.codes.cpu(), codes[0])
    assert bool((scales == 0).any()) and int(scales.max()) == 252
    f32 = experts.fp4_quantize(x.float().cuda())
    assert torch.equal(f32.codes, q.codes) and torch.equal(f32.scales, q.scales)
    ones = experts.Fp4Linear.from_float(experts.Fp4Desc(256, 256, len(x)), torch.eye(256))
    v, xd = values(q.codes, q.scales), x.cuda()
    tiny = v.abs() < 2.0 ** -126
    for M, most in ((len(x), 1), (16, 200), (3, 400)):  # tiles, and one launch for up to 4 tokens
        step = max(len(x) // most, M)
        for a in range(0, len(x) - M + 1, step):
            y = ones(xd[a:a + M]).float()
            assert bool(((y == v[a:a + M]) | (tiny[a:a + M] & (y.abs() < 2.0 ** -126))).all()), (M, a)


# ---------------------------------------------------------------- activations

@pytest.mark.parametrize("M", [1, 3, 20, 100, 600, 2100])
@pytest.mark.parametrize("kind", ["fp4", "fp8"])
def test_gelu_of_negative_gates(kind, M):
    """GELU keeps its digits where it is nearly zero.  The gates -(a + c / 2 + b / 8)
    are exact, 4 to 9.75; z = sqrt(2 / pi) (g + 0.044715 g^3) goes through seven
    roundings of 2^-24 and the exponential's argument through two more, and
    |2 z| is below 81: 81 * 9 * 2^-24 < 2^-14 of the value."""
    K, N = 128, 2048
    x = torch.zeros(M, K)
    x[:, 0], x[:, 1], x[:, 2] = 1.0, 0.125, 0.5
    g = torch.Generator().manual_seed(M)
    pick = torch.randint(0, 8, (N, 3), generator=g)
    pick[:, 0] = torch.randint(6, 8, (N,), generator=g)  # 4 or 6
    w = torch.zeros(2 * N, K)
    w[:N, :3] = -ref.E2M1[pick].float()
    w[N:, 0] = 1.0
    if kind == "fp4":
        lin = experts.Fp4Linear.from_float(experts.Fp4Desc(K, N, M, "gelu_tanh"), w.cuda())
        q = experts.fp4_quantize(w.cuda())
        assert torch.equal(values(q.codes, q.scales).cpu(), w)
    else:
        lin = block.Fp8Linear(block.Fp8Desc(K, N, M, "gelu_tanh"), w.to(torch.float8_e4m3fn).cuda(),
                              torch.ones(2 * (N // 128), K // 128, device="cuda"))
    y = lin(x.bfloat16().cuda()).cpu().double()
    gate = (x.double() @ w.double().t())[:, :N]
    z = 0.7978845608028654 * (gate + 0.044715 * gate ** 3)
    want = gate / (1 + torch.exp(-2 * z))
    err = (y - want).abs() / want.abs()
    assert float(err.max()) <= BF16 + 2.0 ** -14
