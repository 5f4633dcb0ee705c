"""From 16- and 32-bit experts to FP4 ones, and beside them
(include/moe_fp4.h, last part):

``fp4_quantize``, ``fp4_dequantize``  MXFP4 / NVFP4 codes and scales of bf16 or fp32 tensors, and back
``Fp4Linear``       linear map over MXFP4 weights and MXFP4 activations
``group_routes``    a router's routes sorted by expert
``gather_routes``   rows of hidden states in that order (with its gradient)
``grouped_linear``  products grouped by expert over ragged rows (with their gradients)
``grouped_weight_grad``  the weights' gradient by itself, bf16 or fp32
``combine_routes``  weighted sum of a token's expert outputs (with its gradients)

so that a layer of bf16 experts is

    groups = group_routes(ids, E)
    h = grouped_linear(gather_routes(x, groups), w13, groups.offsets)
    y = grouped_linear(activation(h), w2, groups.offsets)
    out = combine_routes(y, groups, w)

and ``moe.Fp4MoE.from_float`` makes the FP4 layer of the same weights.

Argument marshalling only, as in ``moe``; every step runs in the HIP library.
Calls run on the current stream of the tensors' device unless given one.  A
graph that captures a backward pass takes its leaves' gradients by
``torch.autograd.grad``, or of leaves that no eager graph holds any more.
Gradients are those of reverse mode: tensors with a forward-mode tangent are
refused.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad

from . import moe
from .block import _TORCH_TYPES, FNS, _device, _empty, _launch, _need, _sized

_VP, _SZ, _I32, _I64, _F32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
GROUP = {"mxfp4": 32, "nvfp4": 16}  # values per block scale
WEIGHT_OUT_IN, WEIGHT_IN_OUT = 0, 1


class _LinearDesc(ctypes.Structure):
    _fields_ = [("in_features", _I32), ("out_features", _I32), ("max_tokens", _I32), ("act_fn", _I32),
                ("act_alpha", _F32), ("act_beta", _F32), ("act_limit", _F32)]


class _GroupedDesc(ctypes.Structure):
    _fields_ = [("num_experts", _I32), ("in_features", _I32), ("out_features", _I32), ("weight_layout", _I32)]


_P = ctypes.POINTER
moe.declare({
    "moe_fp4_quantize_workspace_bytes": ([_I32, _I64, _P(_SZ)], ctypes.c_int),
    "moe_fp4_quantize": ([_I32, _I32, _VP, _I64, _I64, _I32, _I64, _VP, _VP, _VP, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "moe_fp4_dequantize": ([_I32, _I32, _VP, _VP, _VP, _I64, _I64, _I32, _VP, _VP], ctypes.c_int),
    "moe_fp4_linear_prepared_bytes": ([_P(_LinearDesc), _P(_SZ)], ctypes.c_int),
    "moe_fp4_linear_prepare": ([_P(_LinearDesc), _VP, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "moe_fp4_linear_workspace_bytes": ([_P(_LinearDesc), _I32, _P(_SZ)], ctypes.c_int),
    "moe_fp4_linear": ([_P(_LinearDesc), _VP, _VP, _I32, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "moe_fp4_linear_quantized": ([_P(_LinearDesc), _VP, _VP, _VP, _I32, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "moe_fp4_group_routes_workspace_bytes": ([_I32, _I32, _I32, _P(_SZ)], ctypes.c_int),
    "moe_fp4_group_routes": ([_VP, _I32, _I32, _I32, _VP, _VP, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "moe_fp4_group_routes_i64": ([_VP, _I32, _I32, _I32, _VP, _VP, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "moe_fp4_gather_routes": ([_VP, _VP, _I32, _I32, _I32, _VP, _VP], ctypes.c_int),
    "moe_fp4_combine_routes": ([_VP, _VP, _VP, _I32, _I32, _I32, _VP, _VP], ctypes.c_int),
    "moe_fp4_combine_routes_grad": ([_VP, _VP, _VP, _VP, _VP, _I32, _I32, _I32, _VP, _VP, _VP], ctypes.c_int),
    "moe_fp4_grouped_linear": ([_P(_GroupedDesc), _VP, _I32, _VP, _VP, _VP, _VP], ctypes.c_int),
    "moe_fp4_grouped_weight_grad": ([_P(_GroupedDesc), _I32, _VP, _VP, _I32, _VP, _VP, _VP], ctypes.c_int),
})


def _on(stream, call, *tensors):
    """call() with `stream` current, the tensors kept until it is past them."""
    stream = moe.as_stream(stream, tensors[0].device)
    for t in tensors:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
    with torch.cuda.stream(stream):
        return call()


def _check_gpu(t, what):
    if not t.is_cuda:
        raise ValueError(f"{what} is on {t.device}, not on a GPU")


def _no_tangents(name, *tensors):
    """Refuses dual tensors, whose derivative would get lost: they require no gradient."""
    if forward_ad._current_level >= 0 and any(
            t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise NotImplementedError(f"{name} has no forward-mode derivative")


# ---------------------------------------------------------------- quantisation

class Fp4Tensor(NamedTuple):
    """E2M1 codes uint8 [.., K / 2], block scales uint8 [.., K / 32] (MXFP4) or
    [.., K / 16] (NVFP4), and NVFP4's fp32 global scales [E]."""
    codes: torch.Tensor
    scales: torch.Tensor
    global_scale: Optional[torch.Tensor] = None


def _shape3(shape):
    if len(shape) == 2:
        return 1, shape[0], shape[1]
    if len(shape) == 3:
        return tuple(shape)
    raise ValueError(f"want [rows][cols] or [experts][rows][cols], got {list(shape)}")


def fp4_quantize(x, fmt: str = "mxfp4", global_scale=None, stream=None) -> Fp4Tensor:
    """MXFP4 or NVFP4 form of x [rows][cols] or [experts][rows][cols], bf16 or
    fp32 (moe_fp4_quantize).  Rows may be apart (a slice of columns), experts
    follow each other at whole rows.  NVFP4: global_scale fp32 [experts] ([1] for
    [rows][cols]), by default taken from x."""
    if stream is not None:
        return _on(stream, lambda: fp4_quantize(x, fmt, global_scale), x, global_scale)
    E, R, K = _shape3(x.shape)
    if x.dtype not in _TORCH_TYPES or fmt not in GROUP:
        raise ValueError(f"fp4_quantize makes mxfp4 or nvfp4 of bf16 and fp32, got {fmt} of {x.dtype}")
    _check_gpu(x, "x")
    index = x.get_device()
    ld = K if x.numel() == 0 else x.stride(-2) if R > 1 else x.stride(0) if E > 1 else K
    if x.numel() and ((K > 1 and x.stride(-1) != 1) or (E > 1 and x.stride(0) != R * ld)):
        raise ValueError(f"x: want rows of consecutive values, experts at whole rows, got strides {list(x.stride())}")
    dev, lead, G = x.device, x.shape[:-1], GROUP[fmt]
    codes = torch.empty((*lead, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((*lead, K // G), dtype=torch.uint8, device=dev)
    given = made = ws = None
    need = 0
    if fmt == "nvfp4" and global_scale is None:
        n = _SZ()
        moe.check("moe_fp4_quantize_workspace_bytes",
                  moe.lib().moe_fp4_quantize_workspace_bytes(moe.NVFP4, E, ctypes.byref(n)))
        need = n.value
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        # an expert without values has no largest one
        made = torch.empty(E, dtype=torch.float32, device=dev) if R else torch.zeros(E, dtype=torch.float32, device=dev)
    elif global_scale is not None:
        given = _need(global_scale, "global_scale", torch.float32, (E,), index)
    _launch(index, None, moe.lib().moe_fp4_quantize, (
        moe.FORMATS[fmt], _TORCH_TYPES[x.dtype], x.data_ptr(), E, R, K, ld, codes.data_ptr(), scales.data_ptr(), given,
        None if made is None else made.data_ptr(), None if ws is None else ws.data_ptr(), need), ())
    return Fp4Tensor(codes, scales, made if made is not None else global_scale)


def fp4_dequantize(q, fmt: str = "mxfp4", dtype=torch.bfloat16, stream=None):
    """The values of an Fp4Tensor (or of a tuple of its parts), bf16 or fp32."""
    codes, scales, global_scale = q if len(q) == 3 else (*q, None)
    if stream is not None:
        return _on(stream, lambda: fp4_dequantize(q, fmt, dtype), codes, scales, global_scale)
    if dtype not in _TORCH_TYPES or fmt not in GROUP:
        raise ValueError(f"fp4_dequantize makes bf16 or fp32 of mxfp4 and nvfp4, got {dtype} of {fmt}")
    _check_gpu(codes, "codes")
    index = codes.get_device()
    lead, K = codes.shape[:-1], 2 * codes.shape[-1]
    E, R, _ = _shape3((*lead, K))
    out = torch.empty((*lead, K), dtype=dtype, device=codes.device)
    _launch(index, None, moe.lib().moe_fp4_dequantize, (
        moe.FORMATS[fmt], _TORCH_TYPES[dtype], _need(codes, "codes", torch.uint8, codes.shape, index),
        _need(scales, "scales", torch.uint8, (*lead, K // GROUP[fmt]), index),
        None if global_scale is None else _need(global_scale, "global_scale", torch.float32, (E,), index),
        E, R, K, out.data_ptr()), ())
    return out


# ---------------------------------------------------------------- linear map

@dataclasses.dataclass(frozen=True)
class Fp4Desc:
    """Shape of an MXFP4 linear map from K to N features; `fn` "none" or an
    activation of the layer ("silu", "gelu_tanh", "swigluoai" over gate and up
    rows, so 2 N weight rows; "relu2" over N)."""
    K: int
    N: int
    max_tokens: int
    fn: str = "none"
    alpha: float = 0.0
    beta: float = 0.0
    limit: float = 0.0

    @property
    def rows(self) -> int:
        return self.N if self.fn in ("none", "relu2") else 2 * self.N

    def c(self) -> _LinearDesc:
        return _LinearDesc(self.K, self.N, self.max_tokens, FNS.get(self.fn, self.fn), self.alpha, self.beta,
                           self.limit)


def linear_prepared_bytes(desc: Fp4Desc) -> int:
    return _sized("moe_fp4_linear_prepared_bytes", desc.c())


def linear_workspace_bytes(desc: Fp4Desc, M: int) -> int:
    return _sized("moe_fp4_linear_workspace_bytes", desc.c(), M)


class Fp4Linear:
    """Prepared MXFP4 weights (codes uint8 [rows][K / 2], scales uint8
    [rows][K / 32]) plus a workspace on one device, made on `stream` (in order
    with the current one).  Calls share the workspace: run them on one stream, or
    order them.  Takes the place of block.Fp8Linear in a block.Fp4MoEBlock."""

    def __init__(self, desc: Fp4Desc, codes: torch.Tensor, scales: torch.Tensor, device="cuda", stream=None):
        self.desc = desc
        dev = self.device = _device(device)
        stream = moe.as_stream(stream, dev)
        self._c = desc.c()
        self._ref = ctypes.byref(self._c)
        with moe.preparing(stream, dev, codes, scales) as made:
            codes, scales = codes.to(dev).contiguous(), scales.to(dev).contiguous()
            ca = _need(codes, "codes", torch.uint8, (desc.rows, desc.K // 2), dev.index)
            sa = _need(scales, "scales", torch.uint8, (desc.rows, desc.K // 32), dev.index)
            self.prepared = torch.empty(linear_prepared_bytes(desc), dtype=torch.uint8, device=dev)
            self.workspace = torch.empty(linear_workspace_bytes(desc, desc.max_tokens), dtype=torch.uint8, device=dev)
            self._at = self.prepared.data_ptr(), self.workspace.data_ptr(), self.workspace.numel()
            _launch(dev.index, stream, moe.lib().moe_fp4_linear_prepare,
                    (self._ref, ca, sa, self._at[0], self.prepared.numel()), (codes, scales, self.prepared))
            made += self.prepared, self.workspace
        self._linear, self._quantized = moe.lib().moe_fp4_linear, moe.lib().moe_fp4_linear_quantized

    @classmethod
    def from_float(cls, desc: Fp4Desc, weight: torch.Tensor, device="cuda", stream=None):
        """The map of a bf16 or fp32 weight [rows][K], quantised on the GPU."""
        dev = _device(device)
        with moe.preparing(moe.as_stream(stream, dev), dev, weight) as made:
            q = fp4_quantize(weight.to(dev).contiguous(), "mxfp4")
            linear = cls(desc, q.codes, q.scales, dev)
            made += linear.prepared, linear.workspace
        return linear

    def __call__(self, x=None, out=None, stream=None, quantized=None):
        """bf16 [M][N] of x bf16 [M][K], or of `quantized`, the Fp4Tensor (or its
        codes and scales) that fp4_quantize(x) gives."""
        d, dev = self.desc, self.device
        at = dev.index
        if (x is None) == (quantized is None):
            raise ValueError("want x or quantized")
        if x is None:
            codes, scales = quantized[:2]
            M = codes.shape[0]
            given = (_need(codes, "codes", torch.uint8, (M, d.K // 2), at),
                     _need(scales, "scales", torch.uint8, (M, d.K // 32), at))
            fn, used = self._quantized, (codes, scales)
        else:
            M = x.shape[0]
            given = _need(x, "x", torch.bfloat16, (M, d.K), at),
            fn, used = self._linear, (x,)
        if stream is not None:
            stream = moe.as_stream(stream, dev)
        if out is None:
            out = _empty((M, d.N), torch.bfloat16, dev, stream)
        pa, sa, sn = self._at
        _launch(at, stream, fn, (self._ref, pa, *given, M, _need(out, "out", torch.bfloat16, (M, d.N), at), sa, sn),
                (*used, out, self.prepared, self.workspace))
        return out


# ---------------------------------------------------------------- routes

class RouteGroups(NamedTuple):
    """Routes sorted by expert: expert e has the rows offsets[e] ..
    offsets[e + 1] - 1; order [M * k] holds a row's route (token * k + slot, -1:
    none) and place [M][k] a route's row (-1: its id is no expert)."""
    offsets: torch.Tensor
    order: torch.Tensor
    place: torch.Tensor


@functools.lru_cache(maxsize=256)
def _group_workspace(M, k, E):
    n = _SZ()
    moe.check("moe_fp4_group_routes_workspace_bytes",
              moe.lib().moe_fp4_group_routes_workspace_bytes(M, k, E, ctypes.byref(n)))
    return n.value


def group_routes(ids, num_experts: int, stream=None) -> RouteGroups:
    """Groups ids int32 or int64 [M][k] by expert (moe_fp4_group_routes)."""
    if stream is not None:
        return _on(stream, lambda: group_routes(ids, num_experts), ids)
    if ids.dtype not in (torch.int32, torch.int64) or ids.dim() != 2:
        raise ValueError(f"ids: want int32 or int64 [M][k], got {ids.dtype} {list(ids.shape)}")
    _check_gpu(ids, "ids")
    M, k = ids.shape
    dev, index = ids.device, ids.get_device()
    need = _group_workspace(M, k, num_experts)
    # one allocation: offsets, order and place; and the workspace
    ints = torch.empty(num_experts + 1 + 2 * M * k, dtype=torch.int32, device=dev)
    offsets, order, place = ints.split((num_experts + 1, M * k, M * k))
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    fn = moe.lib().moe_fp4_group_routes if ids.dtype is torch.int32 else moe.lib().moe_fp4_group_routes_i64
    _launch(index, None, fn, (_need(ids, "ids", ids.dtype, (M, k), index), M, k, num_experts, offsets.data_ptr(),
                              order.data_ptr(), place.data_ptr(), ws.data_ptr(), need), ())
    return RouteGroups(offsets, order, place.view(M, k))


def _gather(x, order, k):
    M, H = x.shape
    index = x.get_device()
    out = torch.empty((M * k, H), dtype=torch.bfloat16, device=x.device)
    _launch(index, None, moe.lib().moe_fp4_gather_routes, (
        _need(x, "x", torch.bfloat16, (M, H), index), _need(order, "order", torch.int32, (M * k,), index), M, k, H,
        out.data_ptr()), ())
    return out


def _combine(y, place, w):
    M, k = place.shape
    index, H = y.get_device(), y.shape[-1]
    out = torch.empty((M, H), dtype=torch.bfloat16, device=y.device)
    _launch(index, None, moe.lib().moe_fp4_combine_routes, (
        _need(y, "y", torch.bfloat16, (M * k, H), index), _need(place, "place", torch.int32, (M, k), index),
        None if w is None else _need(w, "w", torch.float32, (M, k), index), M, k, H, out.data_ptr()), ())
    return out


class _GatherRoutes(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, order, place):
        ctx.save_for_backward(place)
        return _gather(x, order, place.shape[1])

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d):
        place, = ctx.saved_tensors
        return _combine(d.contiguous(), place, None), None, None


class _CombineRoutes(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, order, place, w):
        ctx.save_for_backward(y, order, place, w)
        return _combine(y, place, w)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d):
        y, order, place, w = ctx.saved_tensors
        if w is None:
            return _gather(d.contiguous(), order, place.shape[1]), None, None, None
        dy, dw = _combine_grad(d.contiguous(), y, order, place, w)
        return dy, None, None, dw


def _combine_grad(d, y, order, place, w):
    M, k = place.shape
    index, H = y.get_device(), y.shape[-1]
    dy, dw = torch.empty_like(y), torch.empty_like(w)
    _launch(index, None, moe.lib().moe_fp4_combine_routes_grad, (
        _need(d, "the output's gradient", torch.bfloat16, (M, H), index), y.data_ptr(), place.data_ptr(),
        order.data_ptr(), w.data_ptr(), M, k, H, dy.data_ptr(), dw.data_ptr()), ())
    return dy, dw


def gather_routes(x, groups: RouteGroups, stream=None):
    """Rows of x bf16 [M][H] in the order of the groups, bf16 [M * k][H]; zeros
    in the rows of no route.  Differentiable in x."""
    if stream is not None:
        return _on(stream, lambda: gather_routes(x, groups), x, *groups)
    _no_tangents("gather_routes", x)
    _check_gpu(x, "x")
    if x.dim() != 2 or groups.place.shape[0] != x.shape[0]:
        raise ValueError(f"x: want [{groups.place.shape[0]}][H], got {list(x.shape)}")
    if x.requires_grad and torch.is_grad_enabled():
        return _GatherRoutes.apply(x, groups.order, groups.place)
    return _gather(x, groups.order, groups.place.shape[1])


def combine_routes(y, groups: RouteGroups, w=None, stream=None):
    """Weighted sum of each token's rows of y bf16 [M * k][H], bf16 [M][H]; w
    fp32 [M][k] (ones if left out).  Differentiable in y and w."""
    if stream is not None:
        return _on(stream, lambda: combine_routes(y, groups, w), y, w, *groups)
    _no_tangents("combine_routes", y, w)
    _check_gpu(y, "y")
    if torch.is_grad_enabled() and (y.requires_grad or (w is not None and w.requires_grad)):
        return _CombineRoutes.apply(y, groups.order, groups.place, w)
    return _combine(y, groups.place, w)


# ---------------------------------------------------------------- grouped products

@functools.lru_cache(maxsize=256)
def _grouped_desc(*fields):
    return ctypes.byref(_GroupedDesc(*fields))


def _grouped(x, w, offsets, layout, out=None):
    """y of x and w [E][N][K], or of w [E][K][N] with WEIGHT_IN_OUT."""
    E, a, b = w.shape
    N, K = (a, b) if layout == WEIGHT_OUT_IN else (b, a)
    T, index = x.shape[0], x.get_device()
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=x.device)
    _launch(index, None, moe.lib().moe_fp4_grouped_linear, (
        _grouped_desc(E, K, N, layout), _need(x, "x", torch.bfloat16, (T, K), index), T,
        _need(w, "w", torch.bfloat16, (E, a, b), index), _need(offsets, "offsets", torch.int32, (E + 1,), index),
        _need(out, "out", torch.bfloat16, (T, N), index)), ())
    return out


class _GroupedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets):
        ctx.save_for_backward(x, w, offsets)
        return _grouped(x, w, offsets, WEIGHT_OUT_IN)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d):
        x, w, offsets = ctx.saved_tensors
        d = d.contiguous()
        dx = _grouped(d, w, offsets, WEIGHT_IN_OUT) if ctx.needs_input_grad[0] else None
        dw = grouped_weight_grad(d, x, offsets) if ctx.needs_input_grad[1] else None
        return dx, dw, None


def grouped_linear(x, w, offsets, out=None, stream=None):
    """y[t] = w[e(t)] x[t], bf16 [T][N], of x bf16 [T][K] and w bf16 [E][N][K],
    where rows offsets[e] .. offsets[e + 1] - 1 (int32 [E + 1], on the GPU) are
    expert e's; rows of no expert are zeros.  Differentiable in x and w (without
    `out`)."""
    if stream is not None:
        return _on(stream, lambda: grouped_linear(x, w, offsets, out), x, w, offsets, out)
    _no_tangents("grouped_linear", x, w)
    _check_gpu(x, "x")
    if w.dim() != 3 or x.dim() != 2:
        raise ValueError(f"want x [T][K] and w [E][N][K], got {list(x.shape)} and {list(w.shape)}")
    if torch.is_grad_enabled() and (x.requires_grad or w.requires_grad):
        if out is not None:
            raise ValueError("out: not where a gradient is wanted")
        return _GroupedLinear.apply(x, w, offsets)
    return _grouped(x, w, offsets, WEIGHT_OUT_IN, out)


def grouped_weight_grad(dy, x, offsets, dtype=torch.bfloat16, out=None, stream=None):
    """dw[e] = sum over e's rows of dy[t] x[t]^T, [E][N][K] in bf16 or fp32, of dy
    bf16 [T][N] and x bf16 [T][K]; zeros for an expert without rows."""
    if stream is not None:
        return _on(stream, lambda: grouped_weight_grad(dy, x, offsets, dtype, out), dy, x, offsets, out)
    _no_tangents("grouped_weight_grad", dy, x)
    _check_gpu(dy, "dy")
    if dtype not in _TORCH_TYPES or dy.dim() != 2 or x.dim() != 2:
        raise ValueError(f"want bf16 or fp32 of dy [T][N] and x [T][K], got {dtype} of {list(dy.shape)} and {list(x.shape)}")
    T, N = dy.shape
    K, E, index = x.shape[1], offsets.shape[0] - 1, dy.get_device()
    if out is None:
        out = torch.empty((E, N, K), dtype=dtype, device=dy.device)
    _launch(index, None, moe.lib().moe_fp4_grouped_weight_grad, (
        _grouped_desc(E, K, N, WEIGHT_OUT_IN), _TORCH_TYPES[dtype], _need(dy, "dy", torch.bfloat16, (T, N), index),
        _need(x, "x", torch.bfloat16, (T, K), index), T, _need(offsets, "offsets", torch.int32, (E + 1,), index),
        _need(out, "out", dtype, (E, N, K), index)), ())
    return out
