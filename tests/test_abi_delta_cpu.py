"""Host-only argument checks of the gated delta rule's and the group norm's entry points: every
call below returns before any HIP call."""

import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "linear_recurrence_rnn_amd", "liblinrec.so")

OK, INVALID, WORKSPACE, UNSUPPORTED = 0, 1, 2, 3
F32, BF16 = 0, 1
P = ctypes.c_void_p(0x100000)  # aligned, never dereferenced
ODD = ctypes.c_void_p(0x100001)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.fail("liblinrec.so is not built (run python -m linear_recurrence_rnn_amd.build)")
    from linear_recurrence_rnn_amd import binding
    return binding.load()


def delta_call(lib, shape=(2, 70, 1, 2, 16, 16), dtype=F32, q=P, lengths=None, s_in=None, o=P, s_out=None, ws=P,
               nws=1 << 40):
    return lib.gated_delta_forward(*shape, dtype, q, P, P, P, P, lengths, s_in, 1.0, o, s_out, ws, nws, None)


@pytest.mark.parametrize("shape", [(-1, 4, 1, 1, 8, 8), (1, -4, 1, 1, 8, 8), (1, 4, -1, 1, 8, 8), (1, 4, 2, 3, 8, 8),
                                   (1, 4, 0, 3, 8, 8), (1, 4, 1, 1, 0, 8), (1, 4, 1, 1, 129, 8), (1, 4, 1, 1, 8, 0),
                                   (1, 4, 1, 1, 8, 257), (1 << 40, 1 << 40, 1, 1, 8, 8)], ids=str)
def test_delta_sizes(lib, shape):
    assert delta_call(lib, shape) == INVALID
    assert lib.linrec_last_error()
    assert lib.gated_delta_workspace_size(*shape, F32, 0, 0) == 0


def test_delta_arguments(lib):
    assert delta_call(lib, dtype=2) == INVALID
    assert delta_call(lib, q=None) == INVALID
    assert delta_call(lib, o=None) == INVALID
    assert delta_call(lib, q=ODD) == UNSUPPORTED
    assert delta_call(lib, dtype=BF16, q=ODD) == UNSUPPORTED
    for name in ("lengths", "s_in", "s_out"):
        assert delta_call(lib, **{name: ctypes.c_void_p(0x100002)}) == UNSUPPORTED
    assert delta_call(lib, (1 << 30, 1, 1, 1, 1, 1)) == UNSUPPORTED
    assert delta_call(lib, (0, 70, 1, 2, 16, 16), q=None) == OK
    assert delta_call(lib, (2, 70, 0, 0, 16, 16), q=None) == OK
    assert delta_call(lib, (2, 0, 1, 2, 16, 16), q=None) == OK  # no state to pass on


def test_decode_arguments(lib):
    def call(shape=(2, 1, 2, 16, 16), dtype=F32, q=P, s_in=P, o=P, s_out=P):
        return lib.gated_delta_decode_step(*shape, dtype, q, P, P, P, P, s_in, 1.0, o, s_out, None)
    assert call(shape=(-1, 1, 2, 16, 16)) == INVALID
    assert call(shape=(2, 2, 3, 16, 16)) == INVALID
    assert call(dtype=7) == INVALID
    assert call(q=None) == INVALID
    assert call(s_out=None) == INVALID
    assert call(s_in=ctypes.c_void_p(0x100002)) == UNSUPPORTED
    assert call(shape=(0, 1, 2, 16, 16), q=None) == OK


def test_norm_arguments(lib):
    def fwd(N=4, C=64, G=4, dtype=F32, x=P, w=P, gate=None, eps=1e-5, act=1, out=P):
        return lib.group_norm_act(N, C, G, dtype, x, w, P, gate, eps, act, out, None)
    assert fwd(N=-1) == INVALID
    assert fwd(G=0) == INVALID
    assert fwd(G=5) == INVALID
    assert fwd(dtype=9) == INVALID
    assert fwd(act=2) == INVALID
    assert fwd(eps=-1.0) == INVALID
    assert fwd(eps=float("nan")) == INVALID
    assert fwd(C=1 << 14, G=1) == UNSUPPORTED
    assert fwd(x=None) == INVALID
    assert fwd(w=None) == INVALID
    assert fwd(gate=ODD) == UNSUPPORTED
    assert fwd(N=0, x=None) == OK

    need = lib.group_norm_act_backward_workspace_size(4, 64, 4)
    assert need > 0 and lib.group_norm_act_backward_workspace_size(4, 64, 5) == 0

    def bwd(N=4, C=64, gate=None, ggate=None, gout=P, gw=P, ws=P, nws=need):
        return lib.group_norm_act_backward(N, C, 4, F32, P, P, P, gate, gout, 1e-5, 1, P, gw, P, ggate, ws, nws, None)
    assert bwd(gate=P) == INVALID
    assert bwd(ggate=P) == INVALID
    assert bwd(gout=None) == INVALID
    assert bwd(gw=None) == INVALID
    assert bwd(gw=ODD) == UNSUPPORTED
    assert bwd(nws=need - 1) == WORKSPACE
    assert bwd(ws=None) == INVALID
    assert bwd(N=0, gw=None) == INVALID


def test_checkpoint_and_backward_arguments(lib):
    shape = (2, 70, 1, 2, 16, 16)
    nck = lib.gated_delta_checkpoint_size(*shape, F32, 0)
    full = lib.gated_delta_workspace_size(*shape, F32, 0, 1)
    assert 0 < nck < full
    assert lib.gated_delta_checkpoint_size(*shape, BF16, 0) < lib.gated_delta_checkpoint_size(*shape, BF16, 1) == nck
    assert lib.gated_delta_checkpoint_size(2, 70, 1, 2, 16, 300, F32, 0) == 0

    def keep(ckpt=P, n=nck, o=P):
        return lib.gated_delta_forward_ckpt(*shape, F32, P, P, P, P, P, None, None, 1.0, o, None, ckpt, n, None)
    assert keep(n=nck - 1) == WORKSPACE
    assert keep(ckpt=None) == INVALID
    assert keep(ckpt=ctypes.c_void_p(0x100004)) == UNSUPPORTED
    assert keep(o=None) == INVALID

    def bwd(ckpt=None, n=nck, go=P, gq=P, gs_in=None, gs_out=None, ws=P, nws=full, sizes=shape):
        return lib.gated_delta_backward(*sizes, F32, P, P, P, P, P, None, None, 1.0, ckpt, n, go, gs_out, gq, P, P, P,
                                        P, gs_in, ws, nws, None)
    assert bwd(nws=full - 1) == WORKSPACE
    assert bwd(ckpt=P, nws=full - nck - 1) == WORKSPACE
    assert bwd(ckpt=P, n=nck - 1) == WORKSPACE
    assert bwd(go=None) == INVALID
    assert bwd(gq=None) == INVALID
    assert bwd(gq=ODD) == UNSUPPORTED
    assert bwd(gs_in=ODD) == UNSUPPORTED
    assert bwd(gs_in=P) == INVALID  # without s_in
    assert bwd(gs_out=ODD) == UNSUPPORTED
    assert bwd(ws=None) == INVALID
    assert bwd(sizes=(0, 70, 1, 2, 16, 16), go=None) == OK
    assert bwd(sizes=(2, 70, 1, 2, 16, 0)) == INVALID
