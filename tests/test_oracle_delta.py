"""Pins of the float64 oracle of the gated delta rule and the group norm: closed forms, an
independent evaluation, and central differences of every gradient."""

import numpy as np
import pytest

from oracle import delta
from delta_cases import make_delta, make_norm

INS = ("q", "k", "v", "g", "beta")


def f64(d):
    return {n: x.astype(np.float64) for n, x in d.items()}


def test_state_is_a_product_of_token_matrices():
    # S_T = sum_j (prod_{t>j} M_t) beta_j k_j v_j^T + (prod_t M_t) S_in, M_t = a_t (I - beta_t k_t k_t^T)
    d = f64(make_delta(2, 9, 1, 2, 5, 3, 1))
    _, S = delta.gated_delta_forward(*(d[n] for n in INS), s_in=d["s_in"])
    for b in range(2):
        for h in range(2):
            ref = d["s_in"][b, h]
            for t in range(9):
                k, bt = d["k"][b, t, 0], d["beta"][b, t, h]
                M = np.exp(d["g"][b, t, h]) * (np.eye(5) - bt * np.outer(k, k))
                ref = M @ ref + bt * np.outer(k, d["v"][b, t, h])
            np.testing.assert_allclose(S[b, h], ref, rtol=1e-12, atol=1e-13)


def test_orthonormal_keys_recall_their_values():
    d = f64(make_delta(1, 6, 1, 1, 6, 4, 2))
    d["k"] = np.linalg.qr(np.random.default_rng(0).standard_normal((6, 6)))[0][None, :, None]
    d["q"] = np.repeat(d["k"][:, 2:3], 6, axis=1)
    o, _ = delta.gated_delta_forward(d["q"], d["k"], d["v"], 0 * d["g"], 0 * d["beta"] + 1, scale=1.0)
    np.testing.assert_allclose(o[0, :2], 0, atol=1e-12)
    np.testing.assert_allclose(o[0, 2:, 0], np.repeat(d["v"][0, 2:3, 0], 4, axis=0), atol=1e-12)


def test_a_cleared_state_forgets_and_a_long_row_equals_its_pieces():
    d = f64(make_delta(2, 10, 2, 2, 4, 4, 3))
    args = [d[n] for n in INS]
    o, S = delta.gated_delta_forward(*args, s_in=d["s_in"])
    o1, S1 = delta.gated_delta_forward(*(x[:, :4] for x in args), s_in=d["s_in"])
    o2, S2 = delta.gated_delta_forward(*(x[:, 4:] for x in args), s_in=S1)
    np.testing.assert_allclose(np.concatenate([o1, o2], 1), o, rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(S2, S, rtol=1e-12, atol=1e-14)
    g = d["g"].copy()
    g[:, 4] = -np.inf
    cut = delta.gated_delta_forward(d["q"], d["k"], d["v"], g, d["beta"], s_in=d["s_in"])[0][:, 4:]
    fresh = delta.gated_delta_forward(*(x[:, 4:] for x in args))[0]
    np.testing.assert_allclose(cut, fresh, rtol=1e-12, atol=1e-14)


def test_lengths_equal_shorter_rows():
    d = f64(make_delta(3, 7, 1, 2, 4, 3, 4, grads=True))
    lens = [7, 0, 3]
    args = [d[n] for n in INS]
    o, S = delta.gated_delta_forward(*args, s_in=d["s_in"], lengths=lens)
    gs = delta.gated_delta_backward(*args, d["go"], d["s_in"], d["gs_out"], lens)
    for b, n in enumerate(lens):
        cut = [x[b:b + 1, :n] for x in args]
        ob, Sb = delta.gated_delta_forward(*cut, s_in=d["s_in"][b:b + 1])
        np.testing.assert_allclose(o[b:b + 1, :n], ob, atol=1e-14)
        assert np.all(o[b, n:] == 0)
        np.testing.assert_allclose(S[b:b + 1], Sb, atol=1e-14)
        gb = delta.gated_delta_backward(*cut, d["go"][b:b + 1, :n], d["s_in"][b:b + 1], d["gs_out"][b:b + 1])
        for x, y in zip(gs[:5], gb[:5]):
            np.testing.assert_allclose(x[b:b + 1, :n], y, atol=1e-13)
            assert np.all(x[b, n:] == 0)
        np.testing.assert_allclose(gs[5][b:b + 1], gb[5], atol=1e-13)


def differences(f, x, step=1e-5):
    g = np.empty_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        keep = x[i]
        x[i] = keep + step
        up = f()
        x[i] = keep - step
        g[i] = (up - f()) / (2 * step)
        x[i] = keep
    return g


@pytest.mark.parametrize("Hv", [1, 2])
def test_delta_gradients_against_differences(Hv):
    d = f64(make_delta(2, 5, 1, Hv, 3, 2, 5, grads=True))
    lens = [5, 3]

    def loss():
        o, S = delta.gated_delta_forward(*(d[n] for n in INS), s_in=d["s_in"], lengths=lens)
        return np.sum(o * d["go"]) + np.sum(S * d["gs_out"])

    got = delta.gated_delta_backward(*(d[n] for n in INS), d["go"], d["s_in"], d["gs_out"], lens)
    for name, g in zip(INS + ("s_in",), got):
        np.testing.assert_allclose(g, differences(loss, d[name]), rtol=1e-7, atol=1e-8, err_msg=name)


@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("gated", [False, True])
def test_norm_gradients_against_differences(gated, act):
    d = f64(make_norm(3, 12, 6))
    gate = d["gate"] if gated else None

    def loss():
        return np.sum(delta.group_norm_act(d["x"], 3, d["weight"], d["bias"], gate, act) * d["gout"])

    got = delta.group_norm_act_backward(d["x"], 3, d["weight"], d["bias"], d["gout"], gate, act)
    for name, g in zip(("x", "weight", "bias") + (("gate",) if gated else ()), got):
        np.testing.assert_allclose(g, differences(loss, d[name]), rtol=1e-6, atol=1e-8, err_msg=name)


def test_norm_of_each_group_is_standard():
    d = make_norm(4, 30, 7, mean=50.0)
    y = delta.group_norm_act(d["x"], 5, np.ones(30), np.zeros(30), act="none", eps=0.0).reshape(4, 5, 6)
    np.testing.assert_allclose(y.mean(-1), 0, atol=1e-9)
    np.testing.assert_allclose((y * y).mean(-1), 1, rtol=1e-9)
