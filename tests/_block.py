"""Helpers of the GPU tests of the norm, the 8-bit projection, the convolution
and the state space scan: seeded inputs and the elementwise bound
    |got - ref| <= half * |ref| + coef * mag
where half is half a step of the output's type (one rounding) and mag the fp64
reference's sum of magnitudes: coef is the relative error of the terms and of
their fp32 summation."""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24, torch.float8_e4m3fn: 2.0 ** -4}
DEV = "cuda"


def rnd(*shape, seed=0, scale=1.0, shift=0.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(1000 * seed + len(shape))
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype).to(DEV)


def d64(*ts):
    return [None if t is None else t.double() for t in ts]


def held(name, got, ref, mag, coef, half=None):
    assert tuple(got.shape) == tuple(ref.shape), (name, got.shape, ref.shape)
    half = HALF[got.dtype] if half is None else half
    got = got.double()
    assert bool(torch.isfinite(got).all()), name
    err, bound = (got - ref).abs(), half * ref.abs() + coef * mag + 1e-38
    worst = float((err / bound).max()) if got.numel() else 0.0
    print("%s: worst error / bound %.3f" % (name, worst), flush=True)
    assert worst <= 1.0, (name, worst)


def replayed(call, outputs):
    """A captured call replayed three times, eager work and a synchronisation
    between, every replay bit for bit the eager result."""
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for name, g, w in zip(outputs, got, want):
            assert torch.equal(g, w), name
        again = call()
        torch.cuda.synchronize()
        for name, g, w in zip(outputs, again, want):
            assert torch.equal(g, w), name
