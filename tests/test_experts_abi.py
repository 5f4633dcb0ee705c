"""Refusals and sizes of FP4 quantisation, the MXFP4 linear map, grouped
products and the routes' calls: bad arguments are rejected before any HIP
call (so these run without a GPU)."""
from __future__ import annotations

import contextlib
import ctypes
import types

import pytest
import torch
from torch.autograd import forward_ad

from block_scaled_fp4_gather_amd import experts, moe

EINVAL, EUNSUPPORTED, EWORKSPACE = 1, 2, 3
A, B, C, D, E, F, G = (1 << b for b in range(24, 31))  # far enough apart


@pytest.fixture(scope="module")
def L():
    return moe.lib()


def caller(fn, base):
    def call(**kw):
        assert not set(kw) - set(base)
        return fn(*{**base, **kw}.values(), None)
    return call


def test_quantize_rejects_before_launch(L):
    call = caller(L.moe_fp4_quantize, dict(fmt=1, type=0, x=A, experts=2, rows=3, cols=64, ld=64, codes=B, scales=C,
                                           g=None, g_out=None, ws=None, n=0))
    assert call(rows=0) == 0 and call(experts=0, x=None) == 0
    for kw in (dict(fmt=0), dict(fmt=3), dict(type=2), dict(experts=-1), dict(rows=-1), dict(cols=0), dict(cols=48),
               dict(ld=56), dict(ld=68), dict(x=None), dict(codes=None), dict(scales=None), dict(x=A + 8),
               dict(codes=B + 8), dict(g=D), dict(g_out=D), dict(codes=A + 752), dict(scales=A), dict(scales=B + 191)):
        assert call(**kw) == EINVAL, kw
    assert call(cols=1 << 21, ld=1 << 21) == EUNSUPPORTED and call(rows=1 << 40) == EUNSUPPORTED
    nv = caller(L.moe_fp4_quantize, dict(fmt=2, type=1, x=A, experts=2, rows=3, cols=48, ld=52, codes=B, scales=C,
                                         g=None, g_out=D, ws=E, n=2048))
    for kw in (dict(g=F), dict(g_out=None), dict(ws=None), dict(ws=E + 128), dict(cols=40), dict(ld=50), dict(g_out=D + 2),
               dict(g_out=A + 1196), dict(ws=A), dict(ws=C), dict(g_out=C + 16)):
        assert nv(**kw) == EINVAL, kw
    assert nv(n=2047) == EWORKSPACE
    n = ctypes.c_size_t()
    assert L.moe_fp4_quantize_workspace_bytes(2, 2, ctypes.byref(n)) == 0 and n.value == 2048
    assert L.moe_fp4_quantize_workspace_bytes(1, 2, ctypes.byref(n)) == 0 and n.value == 0
    assert L.moe_fp4_quantize_workspace_bytes(3, 2, ctypes.byref(n)) == EINVAL


def test_dequantize_rejects_before_launch(L):
    call = caller(L.moe_fp4_dequantize, dict(fmt=2, type=0, codes=A, scales=B, g=C, experts=2, rows=3, cols=48, out=D))
    assert call(rows=0) == 0
    for kw in (dict(fmt=0), dict(type=-1), dict(cols=40), dict(g=None), dict(fmt=1, cols=64), dict(codes=None),
               dict(scales=None), dict(out=None), dict(out=D + 8), dict(codes=A + 4), dict(out=B), dict(out=C)):
        assert call(**kw) == EINVAL, kw


def _sized(fn, desc, *args):
    n = ctypes.c_size_t()
    return fn(ctypes.byref(desc.c()), *args, ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,status", [
    (dict(), 0), (dict(K=0), EINVAL), (dict(N=0), EINVAL), (dict(K=48), EINVAL), (dict(N=20), EINVAL),
    (dict(max_tokens=-1), EINVAL), (dict(max_tokens=(1 << 20) + 1), EUNSUPPORTED), (dict(fn=4), EINVAL),
    (dict(fn=-2), EINVAL), (dict(fn="swigluoai"), EINVAL), (dict(fn="swigluoai", alpha=1.0, limit=7.0), 0),
    (dict(fn="swigluoai", alpha=1.0, beta=float("nan"), limit=7.0), EINVAL),
    (dict(K=1 << 16, N=1 << 16), EUNSUPPORTED), (dict(K=(1 << 20) + 32, N=8), EUNSUPPORTED), (dict(K=1 << 20, N=8), 0),
    (dict(K=32, N=(1 << 26) + 8), EUNSUPPORTED),
])
def test_linear_descriptor(L, kw, status):
    desc = experts.Fp4Desc(**{**dict(K=128, N=64, max_tokens=8), **kw})
    assert _sized(L.moe_fp4_linear_prepared_bytes, desc)[0] == status
    assert _sized(L.moe_fp4_linear_workspace_bytes, desc, 0)[0] == status


def test_linear_rejects_before_launch(L):
    d = experts.Fp4Desc(96, 64, 8)
    ref = ctypes.byref(d.c())
    need = experts.linear_workspace_bytes(d, 8)
    assert _sized(L.moe_fp4_linear_workspace_bytes, d, 9)[0] == EINVAL
    call = caller(L.moe_fp4_linear, dict(d=ref, prepared=A, x=B, M=8, out=C, ws=D, n=need))
    assert call(M=0) == 0
    for kw in (dict(M=9), dict(M=-1), dict(prepared=None), dict(x=None), dict(out=None), dict(ws=None), dict(prepared=A + 128),
               dict(x=B + 8), dict(out=C + 8), dict(ws=D + 128), dict(out=B), dict(out=A), dict(ws=B), dict(ws=A),
               dict(out=D + need - 256)):
        assert call(**kw) == EINVAL, kw
    assert call(n=need - 1) == EWORKSPACE
    given = caller(L.moe_fp4_linear_quantized, dict(d=ref, prepared=A, codes=B, scales=E, M=8, out=C, ws=D, n=need))
    for kw in (dict(codes=None), dict(scales=None), dict(codes=B + 8), dict(out=E), dict(ws=E), dict(out=B), dict(M=9)):
        assert given(**kw) == EINVAL, kw
    size = experts.linear_prepared_bytes(d)
    prep = caller(L.moe_fp4_linear_prepare, dict(d=ref, codes=A, scales=B, prepared=C, n=size))
    for kw in (dict(codes=None), dict(scales=None), dict(prepared=None), dict(codes=A + 8), dict(prepared=C + 128),
               dict(prepared=A), dict(prepared=B)):
        assert prep(**kw) == EINVAL, kw
    assert prep(n=size - 1) == EWORKSPACE


def test_group_routes_rejects_before_launch(L):
    n = ctypes.c_size_t()
    assert L.moe_fp4_group_routes_workspace_bytes(3000, 4, 64, ctypes.byref(n)) == 0
    need = n.value
    call = caller(L.moe_fp4_group_routes, dict(ids=A, M=3000, k=4, E=64, offsets=B, order=C, place=D, ws=E, n=need))
    for kw in (dict(ids=None), dict(M=-1), dict(k=0), dict(E=0), dict(offsets=None), dict(order=None), dict(place=None),
               dict(ws=None), dict(ids=A + 2), dict(ws=E + 128), dict(order=A), dict(place=C + 4), dict(offsets=D + 47996),
               dict(ws=C)):
        assert call(**kw) == EINVAL, kw
    assert call(n=need - 1) == EWORKSPACE
    assert call(E=4097) == EUNSUPPORTED and call(M=(1 << 20) + 1) == EUNSUPPORTED
    assert L.moe_fp4_group_routes_i64(A + 4, 3000, 4, 64, B, C, D, E, need, None) == EINVAL
    # the workspace grows with the blocks that the routes make
    last = 0
    for M in (1, 1024, 1025, 5000, 1 << 20):
        assert L.moe_fp4_group_routes_workspace_bytes(M, 4, 64, ctypes.byref(n)) == 0
        assert n.value >= last
        last = n.value
    assert last >= 1024 * 64 * 4


def test_rows_of_routes_reject_before_launch(L):
    call = caller(L.moe_fp4_gather_routes, dict(x=A, order=B, M=5, k=3, H=64, out=C))
    assert call(M=0) == 0
    for kw in (dict(x=None), dict(order=None), dict(out=None), dict(M=-1), dict(k=0), dict(H=0), dict(H=60), dict(x=A + 8),
               dict(order=B + 2), dict(out=C + 8), dict(out=A), dict(out=B)):
        assert call(**kw) == EINVAL, kw
    assert call(H=(1 << 15) + 8) == EUNSUPPORTED and call(M=1 << 21) == EUNSUPPORTED
    call = caller(L.moe_fp4_combine_routes, dict(y=A, place=B, w=D, M=5, k=3, H=64, out=C))
    for kw in (dict(y=None), dict(place=None), dict(out=None), dict(H=60), dict(y=A + 8), dict(w=D + 2), dict(out=A),
               dict(out=B), dict(out=D), dict(place=B + 1)):
        assert call(**kw) == EINVAL, kw
    call = caller(L.moe_fp4_combine_routes_grad, dict(d=A, y=B, place=C, order=D, w=E, M=5, k=3, H=64, dy=F, dw=G))
    for kw in (dict(d=None), dict(y=None), dict(place=None), dict(order=None), dict(w=None), dict(dy=None), dict(dw=None),
               dict(dy=B), dict(dy=A), dict(dw=E), dict(dw=F + 1916), dict(dy=F + 8), dict(dw=G + 2)):
        assert call(**kw) == EINVAL, kw


def test_grouped_rejects_before_launch(L):
    def desc(E=4, K=64, N=32, layout=0):
        return ctypes.byref(experts._GroupedDesc(E, K, N, layout))

    call = caller(L.moe_fp4_grouped_linear, dict(d=desc(), x=A, rows=10, w=B, offsets=C, y=D))
    assert call(rows=0) == 0
    for kw in (dict(d=None), dict(d=desc(E=0)), dict(d=desc(K=60)), dict(d=desc(N=4)), dict(d=desc(layout=2)),
               dict(rows=-1), dict(x=None), dict(w=None), dict(offsets=None), dict(y=None), dict(x=A + 8),
               dict(offsets=C + 2), dict(y=A), dict(y=B), dict(y=C), dict(w=B + 8)):
        assert call(**kw) == EINVAL, kw
    assert call(d=desc(E=4097)) == EUNSUPPORTED and call(rows=(1 << 22) + 1) == EUNSUPPORTED
    assert call(d=desc(K=(1 << 20) + 8)) == EUNSUPPORTED and call(d=desc(N=(1 << 20) + 8)) == EUNSUPPORTED
    call = caller(L.moe_fp4_grouped_weight_grad, dict(d=desc(), type=0, dy=A, x=B, rows=10, offsets=C, dw=D))
    for kw in (dict(type=2), dict(d=desc(layout=1)), dict(dy=None), dict(x=None), dict(offsets=None), dict(dw=None),
               dict(dw=A), dict(dw=B), dict(dw=C), dict(dw=D + 8), dict(rows=-1)):
        assert call(**kw) == EINVAL, kw


def test_python_refusals():
    cpu = torch.zeros(4, 64, dtype=torch.bfloat16)
    for f in (lambda: experts.fp4_quantize(cpu), lambda: experts.group_routes(torch.zeros(4, 2, dtype=torch.int32), 8),
              lambda: experts.grouped_linear(cpu, torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(3).int()),
              lambda: experts.fp4_quantize(cpu.half()), lambda: experts.fp4_quantize(cpu, "fp4"),
              lambda: experts.fp4_quantize(cpu[0]), lambda: experts.group_routes(torch.zeros(4, 2), 8)):
        with pytest.raises(ValueError):
            f()


def test_forward_mode_derivatives_are_refused():
    """A dual tensor requires no gradient, so nothing else keeps its tangent from
    getting lost; with or without one that does beside it, and where gradients
    are switched off."""
    bf = torch.zeros(4, 64, dtype=torch.bfloat16)
    w3, off = torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    groups = experts.RouteGroups(off, torch.zeros(4, dtype=torch.int32), torch.zeros(4, 1, dtype=torch.int32))
    cases = [(experts.gather_routes, (bf, groups), (0,)), (experts.combine_routes, (bf, groups, torch.zeros(4, 1)), (0, 2)),
             (experts.grouped_linear, (bf, w3, off), (0, 1)), (experts.grouped_weight_grad, (bf, bf, off), (0, 1))]
    for f, args, inputs in cases:
        for i in inputs:
            for other in (False, True):
                given = [a.clone().requires_grad_() if other and isinstance(a, torch.Tensor) and a.is_floating_point() else a
                         for a in args]
                with forward_ad.dual_level():
                    given[i] = forward_ad.make_dual(args[i].clone(), torch.ones_like(args[i]))
                    for grad in (False, True):
                        with torch.set_grad_enabled(grad), pytest.raises(NotImplementedError, match="forward-mode"):
                            f(*given)
        with forward_ad.dual_level(), pytest.raises(ValueError, match="not on a GPU"):  # no tangent: the checks as ever
            f(*args)


class _OnSecond:
    """Stands for a dense tensor on the second of two GPUs."""
    device = torch.device("cuda:1")
    shape = (4, 64)

    def __init__(self, dtype=torch.uint8):
        self.dtype = dtype

    data_ptr = lambda self: A
    is_contiguous = lambda self: True
    numel = lambda self: 256
    element_size = lambda self: 1


def test_layer_calls_follow_their_tensors_to_another_device(monkeypatch):
    """What Fp4MoE and its from_float call on another device than the current one
    runs there, on that device's current stream, or on the stream that is given."""
    current, seen = [0], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], torch.device(d).index
        yield
        current[0] = before

    class Library:
        def __getattr__(self, name):
            return lambda *args: seen.append((name, current[0], args[-1].value)) or 0

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda d=None: types.SimpleNamespace(cuda_stream=1000 + (current[0] if d is None else torch.device(d).index)))
    monkeypatch.setattr(moe, "lib", lambda: Library())
    t, desc = _OnSecond(), moe.Desc("mxfp4", 2, 64, 32, 1, 4)
    i32, i64 = _OnSecond(torch.int32), _OnSecond(torch.int64)
    calls = {
        "moe_fp4_prepare": lambda s: moe.prepare(desc, t, t, t, t, None, None, t, s),
        "moe_fp4_unprepare": lambda s: moe.unprepare(desc, t, t, t, t, t, None, None, s),
        "moe_fp4_forward": lambda s: moe.forward(desc, t, t, i32, t, t, t, s),
        "moe_fp4_forward_i64": lambda s: moe.forward(desc, t, t, i64, t, t, t, s),
        "moe_fp4_forward_ex": lambda s: moe.forward(desc, t, t, i32, t, t, t, s, moe.Tuning()),
        "moe_fp4_forward_noalloc": lambda s: moe.forward_noalloc(desc, t, t, i32, t, t, s),
        "moe_fp4_dequant_export": lambda s: moe.dequant_export(desc, t, 0, 0, t, s),
        "moe_fp4_mxfp8_quantize": lambda s: moe.mxfp8_quantize(t, t, t, s),
    }
    for name, call in calls.items():
        for stream, address in ((None, 1001), (77, 77), (types.SimpleNamespace(cuda_stream=78), 78)):
            call(stream)
            assert seen.pop() == (name, 1, address) and current == [0]


@pytest.mark.parametrize("fmt,fn", [("mxfp4", "silu"), ("nvfp4", "silu"), ("mxfp4", "relu2")])
def test_layer_refuses_weights_of_another_shape(fmt, fn):
    """The library knows the descriptor alone: smaller weights than it says would
    be read past their end."""
    E, H, I, G = 4, 128, 64, experts.GROUP[fmt]
    desc = moe.Desc(fmt, E, H, I, 2, 8, fn=fn)
    rows = I if fn == "relu2" else 2 * I
    w13, w2 = torch.zeros(E, rows, H), torch.zeros(E, H, I)
    for a, b in ((w13[:3], w2), (w13, w2[:3]), (w13[:, :I // 2], w2), (w13[..., :64], w2), (w13, w2[..., :32]),
                 (w13.transpose(1, 2) if rows != H else w13[:, 1:], w2), (w13, w2.transpose(1, 2)), (w13[0], w2)):
        with pytest.raises(ValueError, match="want"):
            moe.Fp4MoE.from_float(desc, a, b, device="cuda:0")
    parts = [torch.zeros(E, rows, H // 2, dtype=torch.uint8), torch.zeros(E, rows, H // G, dtype=torch.uint8),
             torch.zeros(E, H, I // 2, dtype=torch.uint8), torch.zeros(E, H, I // G, dtype=torch.uint8)]
    parts += [torch.ones(E), torch.ones(E)] if fmt == "nvfp4" else []
    for i in range(len(parts)):
        for short in (parts[i][:-1], parts[i].flatten()[1:], parts[i].numpy()[1:]):
            with pytest.raises(ValueError, match="want"):
                moe.Fp4MoE(desc, *parts[:i], short, *parts[i + 1:], device="cuda:0")
