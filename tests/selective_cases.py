"""Seeded inputs and comparisons shared by the tests of the selective scan, the short convolution
and the root-mean-square norm."""

import numpy as np

from delta_cases import bf16_round, host, rms_err, to_dev  # noqa: F401

# Tolerances (rms_err: an element's error relative to the larger of it and its tensor's RMS).
#
# float32 results (every result of a float32 call; states and sums over tokens of any call).  A
# state's step rounds five times (its decay's argument, the exponential, d u, d u B, the
# multiply-add), 2^-24 each; over at most 400 tokens without decay that adds up to 400 * 5 * 2^-24 =
# 1.2e-4 if all went one way and grew no sum; of either sign it is sqrt(400) * 5 * 2^-24 = 6e-6 of
# the RMS, ten times that for the largest of a million elements and sums of 128 states.  1e-4, the
# library's float32 gate, holds both; the 2-norm over a whole tensor is held to 1e-5.
#
# bfloat16 results: float32 until the final rounding, half a step: 2^-8 of the value, and 1e-4.
TOL_F32 = 1e-4
NORM_F32 = 1e-5
TOL_BF16 = 2.0 ** -8 + 1e-4


def norm_err(out, ref):
    out, ref = np.asarray(out, np.float64), np.asarray(ref, np.float64)
    return float(np.linalg.norm(out - ref) / max(np.linalg.norm(ref), 1e-30))


def check_one(name, out, ref, bf16, terms=None):
    """``terms``: where ``ref`` is a difference, an array of its size holding what it is a difference
    of.  Each term is rounded to float32 a few times (k steps), so the difference is off by up to k 2^-24
    of the larger term whatever is left of it: both measures then take the terms' RMS for that of a
    difference that is smaller."""
    assert np.all(np.isfinite(out)), name
    out, ref = np.asarray(out, np.float64), np.asarray(ref, np.float64)
    floor = 0.0 if terms is None else np.sqrt(np.mean(np.square(np.asarray(terms, np.float64))))
    whole = np.sqrt(ref.size) * floor
    err = rms_err(out, ref) if not floor else float(np.max(np.abs(out - ref) / np.maximum(np.abs(ref), max(
        floor, np.sqrt(np.mean(ref * ref))))))
    assert err <= (TOL_BF16 if bf16 else TOL_F32), (name, err)
    if not bf16 and ref.size:
        err = float(np.linalg.norm(out - ref) / max(np.linalg.norm(ref), whole, 1e-30))
        assert err <= NORM_F32, (name, err)


def rounder(dtype):
    return bf16_round if dtype == "bf16" else (lambda x: np.asarray(x, np.float32))


def make_scan(B, T, C, G, N, seed, dtype="f32", softplus=True, rate=1.0):
    """Inputs of a state space layer: A from -1 to -N (times ``rate``), steps from 1e-3 to 1e-1."""
    rng = np.random.default_rng(seed)
    rnd = rounder(dtype)
    n = rng.standard_normal
    step = np.exp(rng.uniform(np.log(1e-3), np.log(1e-1), C))
    d = {"u": rnd(n((B, T, C))), "A": (-rate * np.arange(1, N + 1) * np.exp(0.1 * n((C, N)))).astype(np.float32),
         "B": rnd(n((B, T, G, N))), "C": rnd(n((B, T, G, N))), "D": n(C).astype(np.float32), "z": rnd(n((B, T, C))),
         "s_in": n((B, C, N)).astype(np.float32), "gy": rnd(n((B, T, C))), "gs_out": n((B, C, N)).astype(np.float32)}
    if softplus:
        d["dt"] = rnd(0.5 * n((B, T, C)))
        d["dt_bias"] = (step + np.log(-np.expm1(-step))).astype(np.float32)
    else:
        d["dt"] = rnd(step * np.exp(0.5 * n((B, T, C))))
        d["dt_bias"] = (1e-3 * np.abs(n(C))).astype(np.float32)
    return d


def make_conv(B, T, C, K, seed, dtype="f32"):
    rng = np.random.default_rng(seed)
    rnd = rounder(dtype)
    n = rng.standard_normal
    return {"x": rnd(n((B, T, C))), "weight": n((C, K)).astype(np.float32), "bias": n(C).astype(np.float32),
            "s_in": rnd(n((B, K - 1, C))), "gy": rnd(n((B, T, C))), "gs_out": rnd(n((B, K - 1, C)))}


def make_rms(N, C, seed, dtype="f32", rtype="f32"):
    rng = np.random.default_rng(seed)
    n = rng.standard_normal
    rnd, rr = rounder(dtype), rounder(rtype)
    return {"x": rnd(n((N, C))), "residual": rr(2 * n((N, C))), "weight": (1 + 0.3 * n(C)).astype(np.float32),
            "gy": rnd(n((N, C))), "gsum": rr(n((N, C)))}


def dev(x, dtype):
    return to_dev(x, dtype)


def lens(x):
    return None if x is None else to_dev(np.asarray(x, np.int32))
