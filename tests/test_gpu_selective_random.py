"""The selective scan, the short convolution and the norm on seeded random sizes with their options on and off,
against the float64 oracle; runs beside another stream's work give the same bits.  Tolerances as for the
fixed shapes."""

import numpy as np
import pytest

import test_gpu_rms_norm as norm
import test_gpu_scan_selective as scan
import test_gpu_short_conv as conv
from selective_cases import host, make_conv, make_rms, make_scan
from test_gpu_scan_selective import INS, L, to_gpu  # noqa: F401

pytestmark = pytest.mark.gpu


def log_int(rng, lo, hi):
    return int(round(np.exp(rng.uniform(np.log(lo), np.log(hi)))))


def ragged(rng, B, T):
    return [int(x) for x in rng.integers(0, T + 1, B)] if rng.random() < 0.5 else None


@pytest.mark.parametrize("seed", range(40))
def test_scan(L, seed):  # noqa: F811
    rng = np.random.default_rng(100 + seed)
    B, T, G = int(rng.integers(1, 6)), log_int(rng, 1, 400), int(rng.integers(1, 5))
    C, N = G * log_int(rng, 16 // G + 1, 300 // G), log_int(rng, 1, 128)
    drop = tuple(n for n in ("D", "z", "dt_bias") if rng.random() < 0.3)
    scan.check(L, (B, T, C, G, N), ("f32", "bf16")[seed % 2], softplus=rng.random() < 0.7, state=rng.random() < 0.5,
               lengths=ragged(rng, B, T), drop=drop, seed=seed, gstate=rng.random() < 0.5)


@pytest.mark.parametrize("seed", range(40))
def test_conv(L, seed):  # noqa: F811
    rng = np.random.default_rng(200 + seed)
    B, T, C, K = int(rng.integers(1, 20)), log_int(rng, 1, 400), log_int(rng, 16, 1200), int(rng.integers(1, 9))
    conv.check(L, B, T, C, K, ("f32", "bf16")[seed % 2], act=("silu", "none")[seed // 2 % 2], bias=rng.random() < 0.7,
               state=rng.random() < 0.5, lengths=ragged(rng, B, T), seed=seed)


@pytest.mark.parametrize("seed", range(40))
def test_norm(L, seed):  # noqa: F811
    rng = np.random.default_rng(300 + seed)
    N, C = log_int(rng, 1, 3000), log_int(rng, 16, 8192)
    norm.check(L, min(N, 4000000 // C), C, *norm.TYPES[seed % 3], residual=rng.random() < 0.7, gsum=rng.random() < 0.7,
               seed=seed)


def test_runs_agree(L):  # noqa: F811
    """A training step of each, four times, every other one beside a product of matrices on another stream."""
    import torch
    from selective_cases import dev
    g = to_gpu(make_scan(3, 700, 200, 2, 20, 1), "f32")
    c = conv.to_gpu(make_conv(3, 700, 200, 4, 2), "f32")
    r = {n: dev(x, None) for n, x in make_rms(3000, 1000, 3).items()}
    big = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()

    def step():
        kw = {n: g[n] for n in ("D", "z", "dt_bias")}
        y, s, ck = L.scan_selective_ckpt(*(g[n] for n in INS), state=g["s_in"], **kw)
        out = [y, s, *L.scan_selective_backward(*(g[n] for n in INS), g["gy"], state=g["s_in"], gstate=g["gs_out"], ckpt=ck,
                                                **kw)]
        out += L.short_conv_act(c["x"], c["weight"], bias=c["bias"], state=c["s_in"])
        out += L.short_conv_act_backward(c["x"], c["weight"], c["gy"], bias=c["bias"], state=c["s_in"], gstate=c["gs_out"])
        y, s = L.rms_norm_add(r["x"], r["weight"], residual=r["residual"])
        return out + [y, s, *L.rms_norm_add_backward(s, r["weight"], r["gy"], gsum=r["gsum"])]

    want = None
    for i in range(4):
        if i % 2:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                for _ in range(4):
                    big @ big
        got = [host(t).tobytes() for t in step()]
        torch.cuda.synchronize()
        want = want or got
        assert got == want
