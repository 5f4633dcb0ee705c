"""The operators around the expert layer (include/moe_fp4.h, second part):

``Router``      ids and weights for ``moe.Fp4MoE`` from the hidden states
``Fp8Linear``   linear map over E4M3 weights with a scale per block of 128
``block_norm``  the norms before and after a block, with its gate and residual
``Fp4MoEBlock`` all of them around a layer: norm, router, routed experts,
                shared expert, gated residual

Argument marshalling only, as in ``moe``; every step runs in the HIP library.
Calls run on the current stream of the tensors' device unless given one.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools

import torch

from . import moe

TYPES = {"bf16": 0, "fp32": 1}
_TORCH_TYPES = {torch.bfloat16: 0, torch.float32: 1}
SCORING = {"softmax": 0, "sigmoid": 1}
FN_NONE = -1
FNS = dict(moe.ACT_FNS, none=FN_NONE)
GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL = 0, 1, 2, 3

_VP, _SZ, _I32, _F32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_float


class _RouterDesc(ctypes.Structure):
    _fields_ = [("num_experts", _I32), ("hidden", _I32), ("top_k", _I32), ("max_tokens", _I32),
                ("weight_type", _I32), ("scoring", _I32), ("num_groups", _I32), ("top_groups", _I32),
                ("renormalize", _I32), ("scale", _F32)]


class _Fp8Desc(ctypes.Structure):
    _fields_ = [("in_features", _I32), ("out_features", _I32), ("max_tokens", _I32), ("act_fn", _I32),
                ("act_alpha", _F32), ("act_beta", _F32), ("act_limit", _F32)]


class _NormDesc(ctypes.Structure):
    _fields_ = [("hidden", _I32), ("residual_type", _I32), ("weight_type", _I32), ("gate", _I32),
                ("gate_sigmoid", _I32), ("eps", _F32), ("residual_scale", _F32), ("branch_scale", _F32),
                ("weight_offset", _F32)]


_P = ctypes.POINTER
moe.declare({
    "moe_fp4_router_prepared_bytes": ([_P(_RouterDesc), _P(_SZ)], ctypes.c_int),
    "moe_fp4_router_prepare": ([_P(_RouterDesc), _VP, _VP, _SZ, _VP], ctypes.c_int),
    "moe_fp4_router_workspace_bytes": ([_P(_RouterDesc), _I32, _P(_SZ)], ctypes.c_int),
    "moe_fp4_route": ([_P(_RouterDesc), _VP, _VP, _I32, _VP, _VP, _VP, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "moe_fp4_fp8_prepared_bytes": ([_P(_Fp8Desc), _P(_SZ)], ctypes.c_int),
    "moe_fp4_fp8_prepare": ([_P(_Fp8Desc), _VP, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "moe_fp4_fp8_workspace_bytes": ([_P(_Fp8Desc), _I32, _P(_SZ)], ctypes.c_int),
    "moe_fp4_fp8_linear": ([_P(_Fp8Desc), _VP, _VP, _I32, _VP, _VP, _SZ, _VP], ctypes.c_int),
    "moe_fp4_block_norm": ([_P(_NormDesc), _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP], ctypes.c_int),
})


@dataclasses.dataclass(frozen=True)
class RouterDesc:
    """Shape of a router: E experts, k of them per token; `weight` the type of
    its weights ("bf16" or "fp32"), `scoring` "softmax" or "sigmoid", `groups`
    and `top_groups` the group limit (1: none), `renorm` whether a token's
    weights are divided by their sum, `scale` what multiplies them."""
    E: int
    H: int
    k: int
    max_tokens: int
    weight: str = "bf16"
    scoring: str = "softmax"
    groups: int = 1
    top_groups: int = 1
    renorm: bool = True
    scale: float = 1.0

    def c(self) -> _RouterDesc:
        return _RouterDesc(self.E, self.H, self.k, self.max_tokens, TYPES.get(self.weight, self.weight),
                           SCORING.get(self.scoring, self.scoring), self.groups, self.top_groups,
                           int(self.renorm), self.scale)


@dataclasses.dataclass(frozen=True)
class Fp8Desc:
    """Shape of an FP8 linear map from K to N features; `fn` "none" or an
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

    def c(self) -> _Fp8Desc:
        return _Fp8Desc(self.K, self.N, self.max_tokens, FNS.get(self.fn, self.fn), self.alpha, self.beta,
                        self.limit)


def _sized(name: str, c, *args) -> int:
    n = _SZ()
    moe.check(name, getattr(moe.lib(), name)(ctypes.byref(c), *args, ctypes.byref(n)))
    return n.value


def router_prepared_bytes(desc: RouterDesc) -> int:
    return _sized("moe_fp4_router_prepared_bytes", desc.c())


def router_workspace_bytes(desc: RouterDesc, M: int) -> int:
    return _sized("moe_fp4_router_workspace_bytes", desc.c(), M)


def fp8_prepared_bytes(desc: Fp8Desc) -> int:
    return _sized("moe_fp4_fp8_prepared_bytes", desc.c())


def fp8_workspace_bytes(desc: Fp8Desc, M: int) -> int:
    return _sized("moe_fp4_fp8_workspace_bytes", desc.c(), M)


# A call of a few tokens takes about as long on the host as on the GPU, so the
# checks below look things up by index (the current stream's address and the
# current device) instead of through objects made for each call.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _need(t: torch.Tensor, what: str, dtype, shape, index: int) -> int:
    """Address of a dense tensor after checking its type, shape and device."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what}: want contiguous {dtype} {list(shape)}, "
                         f"got {'' if t.is_contiguous() else 'strided '}{t.dtype} {list(t.shape)}")
    if t.get_device() != index or not t.is_cuda:
        raise ValueError(f"{what} is on {t.device}, not on {'a GPU' if index < 0 else f'cuda:{index}'}")
    return t.data_ptr()


def _empty(shape, dtype, device, stream):
    """Memory that belongs to the stream that writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _empty_like(t, dtype, stream):
    """The same of t's shape, in half the host's time where the type is t's too."""
    if stream is None:
        return torch.empty_like(t) if t.dtype is dtype else torch.empty_like(t, dtype=dtype)
    with torch.cuda.stream(stream):
        return torch.empty_like(t, dtype=dtype)


def _launch(index: int, stream, fn, args, tensors) -> None:
    """fn(*args, stream address) with device `index` current, which launches go
    by.  `tensors` are kept until an explicitly given stream is past the call."""
    s = _raw_stream(index) if stream is None else stream.cuda_stream
    if _current_device() == index:
        status = fn(*args, s)
    else:
        with torch.cuda.device(index):
            status = fn(*args, s)
    if status != 0:
        moe.check(fn.__name__, status)
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _device(device) -> torch.device:
    d = torch.device(device)
    return d if d.index is not None else torch.device(d.type, torch.cuda.current_device())


class Router:
    """Prepared router weights plus a workspace on one device, made on `stream`
    (in order with the current one).  Calls share the workspace: run them on
    one stream, or order them."""

    def __init__(self, desc: RouterDesc, weight: torch.Tensor, bias: torch.Tensor | None = None, device="cuda",
                 stream=None):
        self.desc = desc
        dev = self.device = _device(device)
        stream = moe.as_stream(stream, dev)
        self._c = desc.c()
        self._ref = ctypes.byref(self._c)
        dtype = {"bf16": torch.bfloat16, "fp32": torch.float32}[desc.weight]
        if weight.dtype is not dtype:
            raise ValueError(f"router weights are {weight.dtype}, the descriptor says {dtype}")
        with moe.preparing(stream, dev, weight, bias) as made:
            weight = weight.to(dev).contiguous()
            at = _need(weight, "weight", dtype, (desc.E, desc.H), dev.index)
            self.bias = None if bias is None else bias.to(device=dev, dtype=torch.float32).contiguous()
            self._bias_at = None if bias is None else _need(self.bias, "bias", torch.float32, (desc.E,), dev.index)
            self.prepared = torch.empty(router_prepared_bytes(desc), dtype=torch.uint8, device=dev)
            self.workspace = torch.empty(router_workspace_bytes(desc, desc.max_tokens), dtype=torch.uint8, device=dev)
            self._at = self.prepared.data_ptr(), self.workspace.data_ptr(), self.workspace.numel()
            _launch(dev.index, stream, moe.lib().moe_fp4_router_prepare,
                    (self._ref, at, self._at[0], self.prepared.numel()), (weight, self.prepared))
            made += self.bias, self.prepared, self.workspace
        self._route = moe.lib().moe_fp4_route

    def __call__(self, x, ids=None, w=None, logits=None, stream=None):
        """ids int32 [M][k] and w fp32 [M][k] of x bf16 [M][H]; fills `logits`
        fp32 [M][E] if given."""
        d, dev = self.desc, self.device
        at = dev.index
        M = x.shape[0]
        if stream is not None:
            stream = moe.as_stream(stream, dev)
        if ids is None:
            ids = _empty((M, d.k), torch.int32, dev, stream)
        if w is None:
            w = _empty((M, d.k), torch.float32, dev, stream)
        pa, sa, sn = self._at
        _launch(at, stream, self._route, (
            self._ref, pa, _need(x, "x", torch.bfloat16, (M, d.H), at), M, self._bias_at,
            _need(ids, "ids", torch.int32, (M, d.k), at), _need(w, "w", torch.float32, (M, d.k), at),
            None if logits is None else _need(logits, "logits", torch.float32, (M, d.E), at), sa, sn),
            (x, ids, w, logits, self.bias, self.prepared, self.workspace))
        return ids, w


class Fp8Linear:
    """Prepared FP8 weights plus a workspace on one device, made on `stream`
    (in order with the current one).  Calls share the workspace: run them on
    one stream, or order them."""

    def __init__(self, desc: Fp8Desc, codes: torch.Tensor, scales: torch.Tensor, device="cuda", stream=None):
        self.desc = desc
        dev = self.device = _device(device)
        stream = moe.as_stream(stream, dev)
        self._c = desc.c()
        self._ref = ctypes.byref(self._c)
        halves = desc.rows // desc.N
        if codes.dtype is torch.float8_e4m3fn:
            codes = codes.view(torch.uint8)
        with moe.preparing(stream, dev, codes, scales) as made:
            codes, scales = codes.to(dev).contiguous(), scales.to(dev).contiguous()
            ca = _need(codes, "codes", torch.uint8, (desc.rows, desc.K), dev.index)
            sa = _need(scales, "scales", torch.float32, (halves * (-(-desc.N // 128)), -(-desc.K // 128)), dev.index)
            self.prepared = torch.empty(fp8_prepared_bytes(desc), dtype=torch.uint8, device=dev)
            self.workspace = torch.empty(fp8_workspace_bytes(desc, desc.max_tokens), dtype=torch.uint8, device=dev)
            self._at = self.prepared.data_ptr(), self.workspace.data_ptr(), self.workspace.numel()
            _launch(dev.index, stream, moe.lib().moe_fp4_fp8_prepare,
                    (self._ref, ca, sa, self._at[0], self.prepared.numel()), (codes, scales, self.prepared))
            made += self.prepared, self.workspace
        self._linear = moe.lib().moe_fp4_fp8_linear

    def __call__(self, x, out=None, stream=None):
        """bf16 [M][N] of x bf16 [M][K]."""
        d, dev = self.desc, self.device
        at = dev.index
        M = x.shape[0]
        if stream is not None:
            stream = moe.as_stream(stream, dev)
        if out is None:
            out = _empty((M, d.N), torch.bfloat16, dev, stream)
        pa, sa, sn = self._at
        _launch(at, stream, self._linear, (
            self._ref, pa, _need(x, "x", torch.bfloat16, (M, d.K), at), M,
            _need(out, "out", torch.bfloat16, (M, d.N), at), sa, sn), (x, out, self.prepared, self.workspace))
        return out


@functools.lru_cache(maxsize=256)
def _norm_desc(*fields):
    return ctypes.byref(_NormDesc(*fields))


def block_norm(h, y=None, y2=None, *, gate=None, post_weight=None, pre_weight=None, eps=1e-6, residual_scale=1.0,
               branch_scale=1.0, weight_offset=0.0, gate_sigmoid=False, h_out=None, x_out=None, stream=None):
    """The norms before and after a block (moe_fp4_block_norm).

    h: residual [M][H], bf16 or fp32; y, y2: the branch's outputs, bf16
    [M][H]; gate: [H] (per channel), [M][1] (per token) or [M][H], of the
    weights' type; post_weight, pre_weight: [H], bf16 or fp32.  Returns the
    new residual (None without y) and the normed hidden states (None without
    pre_weight).  h_out may be h."""
    M, H = h.shape
    at = h.get_device()
    if stream is not None:
        stream = moe.as_stream(stream, h.device)
    wt = next((t.dtype for t in (pre_weight, post_weight, gate) if t is not None), torch.bfloat16)
    if h.dtype not in _TORCH_TYPES or wt not in _TORCH_TYPES:
        raise ValueError(f"block_norm takes bf16 and fp32, got {h.dtype} and {wt}")
    kind, shape = GATE_NONE, None
    if gate is not None:
        shape = gate.shape
        if shape == (H,):
            kind = GATE_CHANNEL
        elif shape == (M, H):
            kind = GATE_FULL
        elif shape == (M, 1):
            kind = GATE_TOKEN
        else:
            raise ValueError(f"gate {list(shape)}: want [{H}], [{M}, 1] or [{M}, {H}]")
    rows = (M, H)
    if y is not None and h_out is None:
        h_out = _empty_like(h, h.dtype, stream)
    if pre_weight is not None and x_out is None:
        x_out = _empty_like(h, torch.bfloat16, stream)
    bf16 = torch.bfloat16
    _launch(at, stream, moe.lib().moe_fp4_block_norm, (
        _norm_desc(H, _TORCH_TYPES[h.dtype], _TORCH_TYPES[wt], kind, int(gate_sigmoid), eps, residual_scale,
                   branch_scale, weight_offset), M,
        _need(h, "h", h.dtype, rows, at),
        None if y is None else _need(y, "y", bf16, rows, at),
        None if y2 is None else _need(y2, "y2", bf16, rows, at),
        None if gate is None else _need(gate, "gate", wt, shape, at),
        None if post_weight is None else _need(post_weight, "post_weight", wt, (H,), at),
        None if pre_weight is None else _need(pre_weight, "pre_weight", wt, (H,), at),
        None if h_out is None else _need(h_out, "h_out", h.dtype, rows, at),
        None if x_out is None else _need(x_out, "x_out", bf16, rows, at)),
        (h, y, y2, gate, post_weight, pre_weight, h_out, x_out))
    return h_out, x_out


class Fp4MoEBlock:
    """A mixture-of-experts block around an ``moe.Fp4MoE`` layer:

        x  = norm(h; pre_weight)
        h' = residual_scale h + branch_scale gate * norm(experts(x) + shared(x); post_weight)

    with the routes from `router` and, where given, a shared expert of two
    FP8 maps (`shared_up` with a gated or other activation, `shared_down`);
    without post_weight the branch joins as it is.  Called with h, it returns
    h' and, given `next_weight`, the next block's normed input."""

    def __init__(self, layer: moe.Fp4MoE, router: Router, pre_weight, post_weight=None, shared_up: Fp8Linear = None,
                 shared_down: Fp8Linear = None, eps=1e-6, residual_scale=1.0, branch_scale=1.0, weight_offset=0.0):
        d, r = layer.desc, router.desc
        if (r.E, r.H, r.k) != (d.E, d.H, d.k):
            raise ValueError(f"router E{r.E} H{r.H} k{r.k} does not fit the layer's E{d.E} H{d.H} k{d.k}")
        if (shared_up is None) != (shared_down is None):
            raise ValueError("a shared expert has both its maps or none")
        if shared_up is not None and (shared_up.desc.K, shared_down.desc.K, shared_down.desc.N) != (
                d.H, shared_up.desc.N, d.H):
            raise ValueError("the shared expert's maps do not fit the layer")
        self.layer, self.router, self.shared_up, self.shared_down = layer, router, shared_up, shared_down
        self.pre_weight, self.post_weight = pre_weight, post_weight
        self.kw = dict(eps=eps, residual_scale=residual_scale, branch_scale=branch_scale,
                       weight_offset=weight_offset)

    def _held(self):
        """What the block's steps read and write of their own."""
        yield from (self.pre_weight, self.post_weight, self.router.bias)
        for part in (self.layer, self.router, self.shared_up, self.shared_down):
            if part is not None:
                yield from (part.prepared, part.workspace)

    def __call__(self, h, x=None, gate=None, gate_sigmoid=False, next_weight=None, h_out=None, stream=None):
        """h [M][H]; x: its normed form where the block before gave it."""
        stream = moe.as_stream(stream, h.device)
        if stream is not None:
            for t in (h, x, gate, next_weight, h_out, *self._held()):
                if t is not None:
                    t.record_stream(stream)
            with torch.cuda.stream(stream):
                return self(h, x, gate, gate_sigmoid, next_weight, h_out)
        with torch.cuda.device(h.device):
            if x is None:
                _, x = block_norm(h, pre_weight=self.pre_weight, eps=self.kw["eps"],
                                  weight_offset=self.kw["weight_offset"])
            ids, w = self.router(x)
            y = self.layer(x, ids, w)
            y2 = None if self.shared_up is None else self.shared_down(self.shared_up(x))
            return block_norm(h, y, y2, gate=gate, gate_sigmoid=gate_sigmoid, post_weight=self.post_weight,
                              pre_weight=next_weight, h_out=h_out, **self.kw)
