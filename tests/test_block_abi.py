"""Refusals of the operators around the expert layer: bad arguments are
rejected before any HIP call (so these run without a GPU)."""
from __future__ import annotations

import ctypes
import time

import pytest
import torch

from block_scaled_fp4_gather_amd import block, moe

EINVAL, EUNSUPPORTED, EWORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    return moe.lib()


def _router(**kw):
    base = dict(E=64, H=256, k=4, max_tokens=8)
    return block.RouterDesc(**{**base, **kw})


def _sized(fn, desc):
    n = ctypes.c_size_t()
    return fn(ctypes.byref(desc.c()), ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,status", [
    (dict(), 0), (dict(E=0), EINVAL), (dict(H=0), EINVAL), (dict(H=252), EINVAL), (dict(k=0), EINVAL),
    (dict(k=65), EINVAL), (dict(E=128, k=65), EUNSUPPORTED), (dict(E=513), EUNSUPPORTED), (dict(E=512), 0),
    (dict(H=65544), EUNSUPPORTED), (dict(max_tokens=-1), EINVAL), (dict(max_tokens=(1 << 20) + 1), EUNSUPPORTED),
    (dict(weight=2), EINVAL), (dict(scoring=2), EINVAL), (dict(groups=0), EINVAL), (dict(groups=3), EINVAL),
    (dict(groups=64), EINVAL), (dict(groups=8, top_groups=9), EINVAL), (dict(groups=8, top_groups=0), EINVAL),
    (dict(groups=32, top_groups=1, k=4), EINVAL), (dict(groups=32, top_groups=2, k=4), 0),
    (dict(E=512, groups=128, k=1), EUNSUPPORTED), (dict(scale=float("nan")), EINVAL),
    (dict(scale=float("inf")), EINVAL),
])
def test_router_descriptor(L, kw, status):
    assert _sized(L.moe_fp4_router_prepared_bytes, _router(**kw))[0] == status


def test_router_sizes(L):
    """bf16 bytes once, fp32 as three planes; the workspace covers every M."""
    _, n = _sized(L.moe_fp4_router_prepared_bytes, _router(E=100, H=264))
    assert n >= 2 * 112 * 288 + 4 * 100
    _, n3 = _sized(L.moe_fp4_router_prepared_bytes, _router(E=100, H=264, weight="fp32"))
    assert n3 >= 6 * 112 * 288 + 4 * 100
    last = 0
    for cap in (1, 5, 16, 17, 100, 1000, 4096, 20000, 40000):
        ws = block.router_workspace_bytes(_router(E=256, H=7168, max_tokens=cap), 1)
        assert ws >= last and ws >= 4 * cap * 257
        last = ws


def test_route_rejects_before_launch(L):
    d = _router()
    ref = ctypes.byref(d.c())
    need = block.router_workspace_bytes(d, 8)

    P, X, I, W, G, S = (1 << b for b in range(20, 26))  # far enough apart

    def call(M=8, prepared=P, x=X, bias=None, ids=I, w=W, logits=None, ws=S, n=need):
        return L.moe_fp4_route(ref, prepared, x, M, bias, ids, w, logits, ws, n, None)

    assert call(M=0) == 0
    assert call(M=9) == EINVAL and call(M=-1) == EINVAL
    for name in ("prepared", "x", "ids", "w", "ws"):
        assert call(**{name: None}) == EINVAL
    assert call(prepared=P + 128) == EINVAL and call(x=X + 8) == EINVAL and call(ids=I + 2) == EINVAL
    assert call(w=W + 2) == EINVAL and call(bias=6) == EINVAL and call(logits=G + 2) == EINVAL
    assert call(ws=S + 128) == EINVAL
    # outputs on each other or on what is read, and x on the workspace
    assert call(w=I + 124) == EINVAL and call(logits=W - 2044) == EINVAL and call(logits=I) == EINVAL
    assert call(ids=X + 4092) == EINVAL and call(w=P) == EINVAL and call(logits=S + need - 4) == EINVAL
    assert call(bias=I - 252) == EINVAL and call(x=S) == EINVAL
    assert call(n=need - 1) == EWORKSPACE
    assert L.moe_fp4_router_prepare(ref, None, 256, 1 << 30, None) == EINVAL
    assert L.moe_fp4_router_prepare(ref, 8, 256, 1 << 30, None) == EINVAL
    assert L.moe_fp4_router_prepare(ref, 16, 256, 16, None) == EWORKSPACE


@pytest.mark.parametrize("kw,status", [
    (dict(), 0), (dict(K=0), EINVAL), (dict(N=0), EINVAL), (dict(K=124), EINVAL), (dict(N=20), EINVAL),
    (dict(max_tokens=-1), EINVAL), (dict(max_tokens=(1 << 20) + 1), EUNSUPPORTED), (dict(fn=4), EINVAL),
    (dict(fn=-2), EINVAL), (dict(fn="swigluoai"), EINVAL), (dict(fn="swigluoai", alpha=1.0, limit=7.0), 0),
    (dict(fn="swigluoai", alpha=1.0, beta=float("nan"), limit=7.0), EINVAL), (dict(K=1 << 16, N=1 << 15), EUNSUPPORTED),
    (dict(K=(1 << 20) + 8, N=8), EUNSUPPORTED), (dict(K=1 << 20, N=8), 0),
])
def test_fp8_descriptor(L, kw, status):
    desc = block.Fp8Desc(**{**dict(K=128, N=64, max_tokens=8), **kw})
    assert _sized(L.moe_fp4_fp8_prepared_bytes, desc)[0] == status


def test_fp8_linear_rejects_before_launch(L):
    d = block.Fp8Desc(128, 64, 8)
    ref = ctypes.byref(d.c())
    need = block.fp8_workspace_bytes(d, 8)

    def call(M=8, prepared=256, x=1 << 14, out=1 << 16, ws=1 << 18, n=need):
        return L.moe_fp4_fp8_linear(ref, prepared, x, M, out, ws, n, None)

    assert call(M=0) == 0
    assert call(M=9) == EINVAL and call(M=-1) == EINVAL
    for name in ("prepared", "x", "out", "ws"):
        assert call(**{name: None}) == EINVAL
    assert call(prepared=128) == EINVAL and call(x=(1 << 14) + 8) == EINVAL and call(out=(1 << 16) + 8) == EINVAL
    assert call(ws=(1 << 18) + 128) == EINVAL
    assert call(out=1 << 14) == EINVAL and call(out=(1 << 14) + 2 * 8 * 128 - 16) == EINVAL  # overlaps x
    assert call(out=1 << 18) == EINVAL and call(x=(1 << 18) + 256) == EINVAL and call(out=512) == EINVAL
    assert call(n=need - 1) == EWORKSPACE
    assert L.moe_fp4_fp8_prepare(ref, 16, None, 256, 1 << 30, None) == EINVAL
    assert L.moe_fp4_fp8_prepare(ref, 16, 16, 256, 16, None) == EWORKSPACE


def test_block_norm_rejects_before_launch(L):
    H, M = 64, 4
    n = M * H

    def call(M=M, h=1 << 12, y=1 << 14, y2=None, gate=None, post=None, pre=1 << 20, ho=1 << 16, xo=1 << 18, **kw):
        d = dict(H=H, rt=0, wt=0, kind=0, sig=0, eps=1e-6, rs=1.0, bs=1.0, off=0.0)
        d.update(kw)
        c = block._NormDesc(*d.values())
        return L.moe_fp4_block_norm(ctypes.byref(c), M, h, y, y2, gate, post, pre, ho, xo, None)

    assert call(M=0) == 0
    for bad in (dict(M=-1), dict(H=0), dict(H=60), dict(rt=2), dict(wt=2), dict(kind=4), dict(sig=2),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(rs=float("inf")), dict(bs=float("nan")),
                dict(off=float("inf")), dict(h=None), dict(ho=None), dict(xo=None), dict(pre=None),
                dict(y=None), dict(y=None, ho=None, y2=1 << 15), dict(y=None, ho=None, post=1 << 21),
                dict(y=None, ho=None, pre=None, xo=None), dict(kind=1), dict(gate=1 << 22),
                dict(h=(1 << 12) + 8), dict(xo=(1 << 18) + 2), dict(kind=1, gate=(1 << 22) + 2),
                dict(kind=2, gate=(1 << 22) + 1), dict(kind=2, wt=1, gate=(1 << 22) + 2),
                dict(ho=(1 << 12) + 16),              # a shifted residual
                dict(rt=1, ho=1 << 14),               # fp32 residual over the bf16 branch
                dict(xo=1 << 16),                     # both outputs in one place
                dict(ho=(1 << 20) - 2 * n + 16)):     # over the weights
        assert call(**bad) == EINVAL, bad
    assert call(H=32776) == EUNSUPPORTED
    assert L.moe_fp4_block_norm(None, M, 16, None, None, None, None, 16, None, 16, None) == EINVAL


def test_binding_refuses_what_does_not_fit():
    h = torch.zeros(2, 64)
    with pytest.raises(ValueError):
        block.block_norm(h.double(), pre_weight=torch.ones(64))
    with pytest.raises(ValueError):
        block.block_norm(h, pre_weight=torch.ones(64))  # not on a GPU
    with pytest.raises(ValueError):
        block.block_norm(h, h.bfloat16(), gate=torch.ones(3), pre_weight=torch.ones(64))


def _route_floats(E, H, planes, M):
    """What a call of M tokens keeps, by the plan of its slices: f32 logits per
    slice, token and expert (to a multiple of 16), and a norm per slice and
    token."""
    blocks = (H + 31) // 32
    if M <= 256:
        kb, unit, splits = blocks, 4, (blocks + 31) // 32
    else:
        kb, unit = (blocks + 7) // 8 * 8, 8 // planes
        be = 128 if E <= 128 or planes == 3 else 256
        bm = 128 if be == 256 or planes == 3 else 64
        tiles = -(-M // bm) * -(-E // be)
        splits = min(8, max(1, (256 if be == 256 else 512) // tiles))
    units = -(-kb // unit)
    per = -(-units // min(splits, units)) * unit
    return -(-kb // per) * M * (-(-E // 16) * 16 + 1)


@pytest.mark.parametrize("E,H,weight", [(256, 7168, "bf16"), (128, 4096, "bf16"), (512, 2560, "fp32"), (8, 8, "fp32"),
                                        (100, 264, "bf16"), (300, 65536, "bf16"), (130, 1000, "fp32"), (512, 520, "bf16")])
def test_router_workspace_is_the_most_that_any_call_needs(E, H, weight):
    planes, most, M = 3 if weight == "fp32" else 1, 0, 0
    for cap in (1, 15, 16, 100, 256, 257, 300, 511, 600, 1000, 1030, 2047, 4096, 5000, 8200, 16384, 20000, 32768, 33000,
                40000):
        while M < cap:
            M += 1
            most = max(most, _route_floats(E, H, planes, M))
        need = -(-4 * most // 256) * 256
        assert block.router_workspace_bytes(block.RouterDesc(E, H, 1, cap, weight=weight), 1) == need, cap


def test_route_takes_the_host_no_longer_for_a_large_capacity(L):
    """A call refused at its last check (a workspace of one byte too few) takes
    on the host what it takes whatever max_tokens is: at most twice as long,
    and half a microsecond."""
    best = []
    for cap in (1, 4096, 32768, 1 << 20):
        d = block.RouterDesc(256, 7168, 8, cap, scoring="sigmoid")
        need = block.router_workspace_bytes(d, 1)
        P, X, I, W, S = (1 << b for b in (28, 30, 31, 32, 40))
        args = (ctypes.byref(d.c()), P, X, 1, None, I, W, None, S, need - 1, None)
        times = []
        for _ in range(15):
            t = time.perf_counter()
            for _ in range(400):
                status = L.moe_fp4_route(*args)
            times.append((time.perf_counter() - t) / 400)
        assert status == EWORKSPACE
        best.append(min(times))
    assert max(best) <= 2 * best[0] + 0.5e-6, best


def test_workspaces_and_prepared_weights_lie_apart_from_what_is_read(L):
    d = _router()
    ref = ctypes.byref(d.c())
    need, prep = block.router_workspace_bytes(d, 8), block.router_prepared_bytes(d)
    P, X, I, W, S = (1 << b for b in range(20, 25))

    def route(prepared=P, bias=None, ws=S):
        return L.moe_fp4_route(ref, prepared, X, 8, bias, I, W, None, ws, need, None)

    assert route(ws=P) == EINVAL and route(ws=P + prep - 256) == EINVAL  # over the prepared weights
    assert route(bias=S + need - 4) == EINVAL and route(bias=S - 252) == EINVAL  # the bias in it
    assert L.moe_fp4_router_prepare(ref, P, P, 1 << 30, None) == EINVAL
    assert L.moe_fp4_router_prepare(ref, P - 2 * 64 * 256 + 16, P, 1 << 30, None) == EINVAL  # the weights' last bytes
    assert L.moe_fp4_router_prepare(ref, P + prep - 16, P, 1 << 30, None) == EINVAL
    f = block.Fp8Desc(264, 136, 8, fn="silu")
    ref = ctypes.byref(f.c())
    need, prep = block.fp8_workspace_bytes(f, 8), block.fp8_prepared_bytes(f)
    assert L.moe_fp4_fp8_linear(ref, P, X, 8, I, P + prep - 256, need, None) == EINVAL
    assert L.moe_fp4_fp8_linear(ref, P, X, 8, I, P, need, None) == EINVAL
    assert L.moe_fp4_fp8_prepare(ref, P - 272 * 264 + 16, X, P, 1 << 30, None) == EINVAL  # the codes' last bytes
    assert L.moe_fp4_fp8_prepare(ref, X, P - 4 * 4 * 3 + 4, P, 1 << 30, None) == EINVAL  # the scales' last
    assert L.moe_fp4_fp8_prepare(ref, X, P + prep - 4, P, 1 << 30, None) == EINVAL


@pytest.mark.parametrize("N,fn,status", [(1 << 26, "silu", 0), (1 << 26, "none", 0), ((1 << 26) + 8, "none", EUNSUPPORTED),
                                         (1 << 27, "silu", EUNSUPPORTED)])
def test_fp8_rows_that_a_launch_has_threads_for(L, N, fn, status):
    assert _sized(L.moe_fp4_fp8_prepared_bytes, block.Fp8Desc(8, N, 1, fn=fn))[0] == status


@pytest.mark.parametrize("out", ["h_out", "x_out"])
def test_block_norm_writes_over_no_gate(L, out):
    """A gate of [M][H] in the residual's type is no place for an output."""
    H, M = 64, 4
    at = dict(h=1 << 12, y=1 << 14, gate=1 << 16, pre=1 << 18, h_out=1 << 20, x_out=1 << 22)
    at[out] = at["gate"]
    c = block._NormDesc(H, 0, 0, block.GATE_FULL, 0, 1e-6, 1.0, 1.0, 0.0)
    assert L.moe_fp4_block_norm(ctypes.byref(c), M, at["h"], at["y"], None, at["gate"], None, at["pre"], at["h_out"],
                                at["x_out"], None) == EINVAL
