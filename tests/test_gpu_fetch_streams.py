"""A layer fetched, run and released on a stream of its own while the current stream
allocates and writes: the weights' memory is not handed out under the passes."""
import pytest
import torch

from gpu_util import dev, say

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def test_fetch_and_release_beside_the_current_stream(Z):
    K, N, M, S = 320, 512, 256, 128 * 1024
    gen = torch.Generator(device=dev())
    gen.manual_seed(3)
    flat = (torch.randn(2 * S, generator=gen, device=dev()) * 0.1).to(BF)
    shards = [flat[:S].clone(), flat[S:].clone()]
    x = torch.randn(M, K, generator=gen, device=dev()).to(BF)
    offsets, numels = [24, 24 + K * N], [K * N, N]
    say("fetch beside the current stream", K, N, M)
    want = Z.zero_linear_forward(x, flat[24:24 + K * N].view(N, K).clone(), flat[24 + K * N:][:N].clone())
    layer = Z.FlatLinear(offsets, numels, 0, 1, K, N)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for it in range(8):
        # a block that the current stream still writes must not become the fetch's
        busy = torch.full((K * N,), float("nan"), dtype=BF, device=dev())
        held = busy.data_ptr()
        del busy
        layer.fetch(shards, S, stream=side)
        assert layer.w.data_ptr() != held
        got.append(layer.forward(x, stream=side)[0])
        held = layer.w.data_ptr()
        layer.release()
        # and the released weights not the current stream's while the pass may read them
        after = [torch.full((K * N,), float("nan"), dtype=BF, device=dev()) for _ in range(3)]
        assert held not in [t.data_ptr() for t in after]
    torch.cuda.synchronize()
    for y in got:
        assert torch.equal(y, want)


def test_fetched_ahead_and_used_on_the_current_stream(Z):
    """The next layer fetched on a side stream while the current stream runs this one."""
    K, N, M, S = 256, 256, 192, 1 << 16
    gen = torch.Generator(device=dev())
    gen.manual_seed(4)
    flat = (torch.randn(4 * S, generator=gen, device=dev()) * 0.1).to(BF)
    shards = [flat[r * S:(r + 1) * S].clone() for r in range(4)]
    numels = [K * N] * 3
    offsets = [0, K * N, 2 * K * N]
    layers = [Z.FlatLinear(offsets, numels, i, None, K, N) for i in range(3)]
    say("fetch ahead", K, N, M)
    x = torch.randn(M, K, generator=gen, device=dev()).to(BF)
    want = x
    for i in range(3):
        want = Z.zero_linear_forward(want, flat[offsets[i]:offsets[i] + K * N].view(N, K).clone())
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    for it in range(4):
        h = x
        layers[0].fetch(shards, S, stream=side)
        for i in range(3):
            main.wait_stream(side)
            if i < 2:
                layers[i + 1].fetch(shards, S, stream=side)
            h, _ = layers[i].forward(h)
            layers[i].release()
        assert torch.equal(h, want)


def test_captured_fetch_on_a_side_stream(Z):
    """Fetch on a forked stream, pass and release inside one graph: every replay copies what
    the shards hold then."""
    K, N, M, S = 136, 264, 40, 1 << 15
    gen = torch.Generator(device=dev())
    gen.manual_seed(5)
    shards = [torch.empty(S, dtype=BF, device=dev()) for _ in range(2)]
    x = torch.randn(M, K, generator=gen, device=dev()).to(BF)
    layer = Z.FlatLinear([16, 16 + K * N], [K * N, N], 0, 1, K, N)
    side = torch.cuda.Stream()
    say("captured fetch", K, N, M)

    def run():
        cur = torch.cuda.current_stream()
        side.wait_stream(cur)
        layer.fetch(shards, S, stream=side)
        cur.wait_stream(side)
        y, _ = layer.forward(x)
        layer.release()
        side.wait_stream(cur)
        layer.fetch(shards, S, stream=side)
        cur.wait_stream(side)
        z, _ = layer.forward(x, residual=y)
        layer.release()
        return z

    for s in shards:
        s.zero_()
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for it in range(4):
        flat = (torch.randn(2 * S, generator=gen, device=dev()) * 0.1).to(BF)
        shards[0].copy_(flat[:S])
        shards[1].copy_(flat[S:])
        graph.replay()
        w, b = flat[16:16 + K * N].view(N, K).clone(), flat[16 + K * N:][:N].clone()
        want = Z.zero_linear_forward(x, w, b, residual=Z.zero_linear_forward(x, w, b))
        torch.cuda.synchronize()
        assert torch.equal(out, want), it
        assert torch.equal(run(), want), it
