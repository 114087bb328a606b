"""The 4-bit layers and the basis solve on a stream that is not torch's current one: the
memory of what they make, while the current stream is behind."""

import numpy as np
import pytest
import torch

from wam_asp_w4a4_amd import synth
from wam_asp_w4a4_amd.layer import PackedLayer, SvdqLayer, forward_group, top_eigenspace

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _busy():
    """Some milliseconds of work on the current stream."""
    a = torch.ones((8192, 8192), dtype=torch.bfloat16, device=DEV)
    b = torch.empty_like(a)
    for _ in range(12):
        torch.mm(a, a, out=b)


@pytest.mark.parametrize("other", ["a side stream", "the default stream"])
def test_memory_of_calls_on_another_stream(other):
    """Blocks that the current stream freed are still to be written by it, and a result is
    still to be read.  Neither may be handed to a call on another stream."""
    lay = synth.make_layer("s", 80, 256, 384, 32, seed=1, dtype="f32")
    packed = [PackedLayer.pack(lay.w, lay.s, lay.v, b, DEV) for b in (lay.b, None)]
    int4 = SvdqLayer.pack_host(lay.w, lay.s, 0, None).to(DEV)
    a = torch.randn((256, 256), device=DEV)
    g, v0 = a @ a.t() / 256, torch.randn((256, 16), device=DEV)
    x = torch.from_numpy(np.ascontiguousarray(lay.x)).to(DEV)
    x2 = torch.randn_like(x)

    def calls(x, stream=None):
        return [packed[0].forward(x, stream=stream), packed[0].forward(x, "bf16", stream=stream),
                *forward_group(packed, x, stream=stream), int4.forward(x, stream=stream),
                *top_eigenspace(g, v0, 8, 4, stream=stream)]

    want, want2 = calls(x), calls(x2)
    torch.cuda.synchronize()
    side, cur = torch.cuda.Stream(), torch.cuda.default_stream()
    if other == "the default stream":
        side, cur = cur, side
        assert side.cuda_stream == 0
    cur.wait_stream(side)
    with torch.cuda.stream(cur):
        _busy()
        trash = [torch.empty_like(t) for t in want for _ in range(2)]
        for t in trash:
            t.fill_(3)
        del trash, t
        got = calls(x, side.cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        # read late, on the current stream, and freed before that
        _busy()
        late = [t.clone() for t in got]
        del got
        again = calls(x2, side.cuda_stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(late, want))
        assert all(torch.equal(a, b) for a, b in zip(again, want2))


def test_the_stream_that_a_handle_stands_for():
    from wam_asp_w4a4_amd.layer import _made_for
    dev, side = torch.device("cuda:0"), torch.cuda.Stream()
    for cur, other in ((torch.cuda.default_stream(), side), (side, torch.cuda.default_stream())):
        with torch.cuda.stream(cur):
            for handle, want in ((None, cur), (cur.cuda_stream, cur), (other.cuda_stream, other)):
                with _made_for(handle, dev):
                    assert torch.cuda.current_stream().cuda_stream == want.cuda_stream
            assert torch.cuda.current_stream() == cur


def test_a_forked_stream_inside_a_capture():
    """Calls on a stream that joined a capture make their tensors in the graph's memory:
    replays give the eager results, with eager work in between."""
    from wam_asp_w4a4_amd.fp8 import Fp8Layer
    from wam_asp_w4a4_amd.norm import gated_norm, gated_norm_backward
    torch.manual_seed(7)
    layer = Fp8Layer.pack(torch.randn((300, 640), device=DEV), torch.randn(300, device=DEV))
    x, dy = torch.randn((200, 640), device=DEV), torch.randn((200, 300), device=DEV)
    w = torch.randn(640, device=DEV)

    def calls(stream=None):
        h, n = gated_norm(x, x, post="rms", weight=w, stream=stream)
        return [h, n, layer.forward(n, stream=stream), *layer.backward(dy, n, stream=stream),
                *gated_norm_backward(x, n, h, x, post="rms", weight=w, need=("dx", "weight"), stream=stream)[::4]]

    calls()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        cur = torch.cuda.current_stream()
        side.wait_stream(cur)
        got = calls(side.cuda_stream)
        cur.wait_stream(side)
    for i in range(4):
        x.copy_(torch.randn_like(x) * (i + 1))
        dy.copy_(torch.randn_like(dy))
        want = calls()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        trash = [torch.full_like(t, 9.0) for t in want for _ in range(3)]
        del trash, want
