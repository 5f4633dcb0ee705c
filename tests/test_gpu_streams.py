"""Objects of the framework made and called on a stream of the user's."""
from __future__ import annotations

import contextlib
import math

import pytest
import torch

from block_scaled_fp4_gather_amd import block, moe, synth
from gpu_util import say, to_dev
from test_gpu_block import fp8_weights, hidden, make_block, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    say(f"\n[gpu] {request.node.nodeid}")
    yield


def late(t):
    """t on the GPU, as a tensor whose bytes come late on the current stream."""
    src = t.cuda()
    out = torch.zeros_like(src)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    return out.copy_(src)


class RouterBuild:
    E, H, k, M = 40, 328, 4, 9

    def weights(self, put):
        w = rand(3, self.E, self.H).float() / math.sqrt(2 * self.H)
        # a transposed weight and a bf16 bias: both are copied by the constructor
        return put(w.t().contiguous()).t(), put((0.05 * rand(9, self.E)).bfloat16())

    def __call__(self, tensors, stream=None):
        desc = block.RouterDesc(self.E, self.H, self.k, self.M, weight="fp32", scoring="sigmoid")
        router = block.Router(desc, *tensors, stream=stream)
        ids, w = router(hidden(1, self.M, self.H).cuda())
        # operands and norms, then from the next multiple of 256 the rows; the bytes between are not written
        end = 3 * -(-self.E // 16) * (-(-self.H // 256) * 8) * 1024 + 4 * self.E
        rows = -(-end // 256) * 256
        return router.prepared[:end], router.prepared[rows:rows + 4 * self.E * self.H], router.bias, ids, w


class Fp8Build:
    K, N, M = 392, 264, 9

    def weights(self, put):
        codes, scales = fp8_weights(5, self.N, self.K, self.N)
        return put(codes.t().contiguous()).t(), put(scales.t().contiguous()).t()

    def __call__(self, tensors, stream=None):
        lin = block.Fp8Linear(block.Fp8Desc(self.K, self.N, self.M), *tensors, stream=stream)
        # columns of padding in the scales are not written; the scales show in the output
        return lin.prepared[:16 * -(-self.N // 16) * 128 * -(-self.K // 128)], lin(hidden(2, self.M, self.K).cuda())


class LayerBuild:
    def __init__(self):
        self.wl = synth.WORKLOADS["tiny_mxfp4"].replace(M=3)
        self.d = synth.generate(self.wl)

    def weights(self, put):
        # all four are strided: the constructor copies them
        return [put(torch.from_numpy(self.d[n]).transpose(1, 2).contiguous()).transpose(1, 2)
                for n in ("w13_codes", "w13_scales", "w2_codes", "w2_scales")]

    def __call__(self, tensors, stream=None):
        w = self.wl
        layer = moe.Fp4MoE(moe.Desc(w.fmt, w.E, w.H, w.I, w.k, w.M), *tensors, stream=stream)
        y = layer(to_dev(self.d["x"]).view(torch.bfloat16), to_dev(self.d["ids"]), to_dev(self.d["w"]))
        back = [torch.empty(self.d[n].shape, dtype=torch.uint8, device="cuda")
                for n in ("w13_codes", "w13_scales", "w2_codes", "w2_scales")]
        moe.unprepare(layer.desc, layer.prepared, *back, None, None)
        return *back, y


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("weights_on_side", [False, True])
@pytest.mark.parametrize("build", [RouterBuild(), Fp8Build(), LayerBuild()], ids=["router", "fp8", "layer"])
def test_made_on_a_side_stream(build, weights_on_side, raw):
    """Weights that are still being written when the constructor is called, on
    the current stream or on the one it is given: the same prepared bytes and
    outputs as without streams."""
    want = build(build.weights(lambda t: t.cuda()))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side) if weights_on_side else contextlib.nullcontext():
        tensors = build.weights(late)
    got = build(tensors, side.cuda_stream if raw else side)
    del tensors
    torch.cuda.synchronize()
    assert len(want) == len(got) and all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("shared", [False, True])
def test_a_block_dropped_behind_its_call_is_kept_for_the_stream(shared, monkeypatch):
    """A call on a stream of the user's marks everything that its steps touch as
    used there, so that none of it is reused before the stream is past it."""
    M = 5
    blk, *_ = make_block(M, shared=shared)
    h = rand(50, M, blk.layer.desc.H).bfloat16().cuda()
    want, _ = blk(h)
    torch.cuda.synchronize()
    side, used, record = torch.cuda.Stream(), set(), torch.Tensor.record_stream

    def note(t, stream):
        if stream.cuda_stream == side.cuda_stream:
            used.add(t.data_ptr())
        return record(t, stream)

    monkeypatch.setattr(torch.Tensor, "record_stream", note)
    side.wait_stream(torch.cuda.current_stream())
    got, _ = blk(h, stream=side)
    parts = [blk.layer, blk.router] + ([blk.shared_up, blk.shared_down] if shared else [])
    held = [t for p in parts for t in (p.prepared, p.workspace)] + [blk.router.bias, blk.pre_weight, blk.post_weight, h]
    assert all(t.data_ptr() in used for t in held)
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("M", [3, 40, 700])
def test_captured_router_with_a_softmax_and_a_bias(M):
    """Three launches, the last of which finds its tokens by what the second
    left in the ids: captured, replayed on new inputs, with eager calls of the
    same router between the replays."""
    E, H, k = 96, 520, 6
    w = (rand(92, E, H) / math.sqrt(2 * H)).bfloat16()
    xs = [hidden(91 + i, M, H).cuda() for i in range(4)]
    p = torch.softmax(xs[1][M // 2].cpu().double() @ w.double().t(), 0)
    bias = (0.1 - p).float()  # evens the scores of one token of xs[1]: all its logits decide
    router = block.Router(block.RouterDesc(E, H, k, M), w.cuda(), bias.cuda())
    want = [tuple(t.clone() for t in router(x)) for x in xs]
    static = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        router(static)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids, wt = router(static)
    for i in (1, 0, 1, 3, 2, 1):
        static.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ids, want[i][0]) and torch.equal(wt, want[i][1])
        eager = router(xs[(i + 1) % 4])
        torch.cuda.synchronize()
        assert torch.equal(eager[0], want[(i + 1) % 4][0]) and torch.equal(eager[1], want[(i + 1) % 4][1])
