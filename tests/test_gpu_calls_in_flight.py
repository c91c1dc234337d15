"""Calls that overlap in time: graphs replayed beside eager calls on other
streams, each with buffers of its own, give what they give alone, bit for bit."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu
TURNS = 12
CALLS = 40    # eager calls a turn: more than any pool of scratch that wraps


@pytest.fixture(scope="module")
def fq():
    import scaled_quantize_fp8_warp_gb300 as fq
    yield fq
    assert fq.device_status() == fq.OK


def normal(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).bfloat16().cuda()


def beside(calls):
    """Each call (a function that fills and returns tensors of its own) alone,
    then the first two as graphs replayed on streams of their own while the
    others are made again and again on two further streams."""
    alone = [[t.clone() for t in f()] for f in calls]
    torch.cuda.synchronize()
    graphs = []
    for f in calls[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = f()
        graphs.append((g, out))
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(TURNS):
        torch.cuda.synchronize()
        for _, out in graphs:
            for t in out:
                t.view(torch.uint8).zero_()
        torch.cuda.synchronize()
        got = []
        for i in range(CALLS):
            for (g, _), s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
            for k, f in enumerate(calls[2:]):
                with torch.cuda.stream(streams[2 + k % 2]):
                    got.append((2 + k, [t.clone() for t in f()]))
        torch.cuda.synchronize()
        got += [(k, out) for k, (_, out) in enumerate(graphs)]
        for k, out in got:
            for a, b in zip(alone[k], out):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), k


def test_linears_that_find_their_amax(fq):
    w = fq.fp4_quantize(normal((512, 2048), 1, 0.02), fq.NVFP4)[0]

    def linear(M, seed):
        x, y = normal((M, 2048), seed, 1.0 + seed), torch.empty((M, 512), dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(fq.fp4_linear_workspace_size(fq.NVFP4, M, 512, 2048), dtype=torch.uint8,
                         device="cuda")
        return lambda: (fq.fp4_linear(x, w, workspace=ws, out=y),)

    def amax(M, seed):
        x, a = normal((M, 2048), seed, 1.0 + seed), torch.empty(1, device="cuda")
        return lambda: (fq.fp4_amax(x, out=a),)
    beside([linear(500, 2), amax(900, 3), linear(300, 4), amax(700, 5)])


def test_8_bit_casts(fq):
    """Per-tensor scaling in one call (small) and in two, and a cast whose
    tiles are claimed as CTAs come free (large)."""
    def current(shape, seed):
        x = normal(shape, seed, 1.0 + seed)
        q, a, s = (torch.empty(shape, dtype=torch.uint8, device="cuda"), torch.empty(1, device="cuda"),
                   torch.empty(1, device="cuda"))

        def run():
            fq.fp8_quantize_tensor_current(x, fq.E4M3, q=q, amax=a, scale=s)
            return q, a, s
        return run

    def tiles(shape, seed):
        x = normal(shape, seed)
        q = torch.empty(shape, dtype=torch.uint8, device="cuda")
        s = torch.empty((shape[1] // 128, shape[0]), device="cuda")

        def run():
            fq.fp8_quantize_tile1x128(x, fq.E4M3, q=q, q_scales=s)
            return q, s
        return run
    beside([current((640, 1024), 1), current((4096, 4096), 2), current((512, 2048), 3), current((300, 4096), 4)])
    beside([tiles((16384, 4096), 5), current((256, 4096), 6), tiles((16384, 4096), 7), tiles((8192, 8192), 8)])


def test_more_streams_than_slots(fq):
    """Streams past the first 128 of a process have no scratch of their own."""
    x = [normal((600, 2048), k, 1.0 + k) for k in range(4)]
    want = [t.abs().max().float() for t in x]
    handles = [ctypes.c_uint64() for _ in range(150)]   # torch's own pool repeats after 32
    for h in handles:
        assert int(torch.cuda.cudart().cudaStreamCreate(ctypes.addressof(h))) == 0
    streams = [torch.cuda.ExternalStream(h.value) for h in handles]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i % 4, fq.fp4_amax(x[i % 4]), fq.fp8_quantize_tensor_current(x[i % 4], fq.E4M3)))
    torch.cuda.synchronize()
    for k, a, b in got:
        assert a.item() == want[k].item() and b[2].item() == want[k].item()
