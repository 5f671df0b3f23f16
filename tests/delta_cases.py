"""Seeded inputs and comparisons shared by the gated delta rule's and the group norm's tests."""

import numpy as np

# Error measures.  rms_err: largest error of an element relative to the larger of the element
# and the RMS of its whole tensor.
#
# Tolerances, from the number formats.  float32 results (every result of a float32 call, states
# and parameter gradients of any call): 1e-4, the library's float32 gate.  bfloat16 results: the
# final rounding is at most 2^-9 of the element; before it, an output is a sum of products whose
# operands were rounded to bfloat16 once each (2^-9 relative, at most four roundings in a chain
# of products), errors of either sign over sums of at least 16 terms, of which the largest of
# some 10^6 elements may reach five standard deviations of the RMS: 2^-9 (1 + 4 * 5 / sqrt(16) / 2)
# < 2^-6.
TOL_F32 = 1e-4
TOL_BF16 = 2.0 ** -6


def rms_err(out, ref):
    out, ref = np.asarray(out, np.float64), np.asarray(ref, np.float64)
    assert out.shape == ref.shape, (out.shape, ref.shape)
    if ref.size == 0:
        return 0.0
    rms = np.sqrt(np.mean(ref * ref))
    e = np.abs(out - ref) / np.maximum(np.maximum(np.abs(ref), rms), 1e-30)
    return float(np.max(e)) if np.all(np.isfinite(e)) else float("inf")


def bf16_round(x):
    """float32 values rounded to bfloat16 (nearest, ties to even), kept as float32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32)
    return u.view(np.float32)


def make_delta(B, T, Hk, Hv, Dk, Dv, seed, dtype="f32", decay=0.1, grads=False):
    """Unit-norm q and k, v ~ N(0,1), g = -decay softplus(N(0,1)), beta = sigmoid(N(0,1)), states
    and upstream gradients ~ N(0,1); rounded to the call's type."""
    rng = np.random.default_rng(seed)
    rnd = bf16_round if dtype == "bf16" else (lambda x: x.astype(np.float32))

    def unit(*shape):
        x = rng.standard_normal(shape)
        return rnd(x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-6))

    d = {"q": unit(B, T, Hk, Dk), "k": unit(B, T, Hk, Dk), "v": rnd(rng.standard_normal((B, T, Hv, Dv))),
         "g": rnd(-decay * np.log1p(np.exp(rng.standard_normal((B, T, Hv))))),
         "beta": rnd(1 / (1 + np.exp(-rng.standard_normal((B, T, Hv))))),
         "s_in": rng.standard_normal((B, Hv, Dk, Dv)).astype(np.float32)}
    if grads:
        d["go"] = rnd(rng.standard_normal((B, T, Hv, Dv)))
        d["gs_out"] = rng.standard_normal((B, Hv, Dk, Dv)).astype(np.float32)
    return d


def make_norm(N, C, seed, dtype="f32", mean=0.0):
    rng = np.random.default_rng(seed)
    rnd = bf16_round if dtype == "bf16" else (lambda x: x.astype(np.float32))
    return {"x": rnd(rng.standard_normal((N, C)) + mean), "gate": rnd(2 * rng.standard_normal((N, C))),
            "gout": rnd(rng.standard_normal((N, C))),
            "weight": (1 + 0.3 * rng.standard_normal(C)).astype(np.float32),
            "bias": (0.3 * rng.standard_normal(C)).astype(np.float32)}


def to_dev(x, dtype=None):
    import torch
    if x is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def host(t):
    import torch
    torch.cuda.synchronize()
    return None if t is None else t.float().cpu().numpy()
