"""The one-token calls as a server makes them: norm, convolution and scan of a layer captured into a graph whose states
go on from replay to replay, with eager calls between, on a stream of their own, inputs given by name."""

import pytest

from selective_cases import host
from test_gpu_scan_selective import L  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,C,G,N,K", [(3, 70, 2, 16, 4), (1, 256, 1, 5, 2)], ids=str)
def test_captured_tokens(L, B, C, G, N, K, dtype):  # noqa: F811
    import torch
    ty = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape, ty=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda").to(ty)

    weight, taps, bias, A, D = normal(C), normal(C, K), normal(C), -normal(C, N).abs(), normal(C)
    maps = [normal(B, G, N, ty=ty) for _ in range(2)]
    tokens = [normal(B, C, ty=ty) for _ in range(5)]
    start = normal(B, K - 1, C, ty=ty), normal(B, C, N)

    def step(x, tail, state):
        n, s = L.rms_norm_add(x=x, weight=weight, residual=x)
        u = L.short_conv_decode_step(x=n, weight=taps, state=tail, bias=bias)
        y = L.scan_selective_decode_step(u=u, dt=n, A=A, B=maps[0], C=maps[1], state=state, D=D, z=s, dt_bias=bias)
        return n, s, u, y

    want, tail, state = [], start[0].clone(), start[1].clone()
    for x in tokens:
        want.append([host(t).tobytes() for t in (*step(x, tail, state), tail, state)])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x, tail, state = tokens[0].clone(), start[0].clone(), start[1].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step(x, tail, state)
        for t, w in zip(tokens, want):
            x.copy_(t)
            graph.replay()
            assert [host(v).tobytes() for v in (*out, tail, state)] == w
            step(t, start[0].clone(), start[1].clone())
