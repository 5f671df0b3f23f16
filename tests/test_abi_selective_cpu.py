"""Host-only argument checks of the selective scan's, the short convolution's and the
root-mean-square norm's entry points: every call below returns before any HIP call."""

import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "linear_recurrence_rnn_amd", "liblinrec.so")

OK, INVALID, WORKSPACE, UNSUPPORTED = 0, 1, 2, 3
F32, BF16 = 0, 1
P = ctypes.c_void_p(0x100000)  # aligned, never dereferenced
ODD = ctypes.c_void_p(0x100001)
HALF = ctypes.c_void_p(0x100002)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.fail("liblinrec.so is not built (run python -m linear_recurrence_rnn_amd.build)")
    from linear_recurrence_rnn_amd import binding
    return binding.load()


SHAPE = (2, 70, 12, 2, 16)


def fwd(lib, shape=SHAPE, dtype=F32, u=P, A=P, D=None, z=None, bias=None, lengths=None, s_in=None, y=P, s_out=None, ws=P,
        nws=1 << 50):
    return lib.linrec_scan_selective(*shape, dtype, u, P, A, P, P, D, z, bias, 1, lengths, s_in, y, s_out, ws, nws, None)


@pytest.mark.parametrize("shape", [(-1, 4, 8, 1, 8), (1, -4, 8, 1, 8), (1, 4, -8, 1, 8), (1, 4, 8, 3, 8), (1, 4, 8, 0, 8),
                                   (1, 4, 8, -1, 8), (1, 4, 8, 1, 0), (1, 4, 8, 1, 129)], ids=str)
def test_scan_sizes(lib, shape):
    assert fwd(lib, shape) == INVALID
    assert lib.linrec_last_error()
    assert lib.linrec_scan_selective_workspace_size(*shape, F32, 0) == 0
    assert lib.linrec_scan_selective_checkpoint_size(*shape, F32) == 0


@pytest.mark.parametrize("shape", [((1 << 20) + 1, 1, 1, 1, 1), (1, (1 << 30) + 1, 1, 1, 1), (1, 1, (1 << 22) + 1, 1, 1),
                                   (1, 1, 1 << 22, 1, 17), (1, 1, 1 << 21, 1 << 21, 9), (1 << 18, 1, 1 << 13, 1, 4), (1 << 20, 1, 8, 8, 1),
                                   (1 << 20, 1 << 30, 1, 1, 1), (1, 1 << 30, 1 << 15, 1, 1), (1 << 62, 1 << 62, 1, 1, 1)],
                         ids=str)
def test_scan_limits(lib, shape):
    assert fwd(lib, shape) == UNSUPPORTED
    assert lib.linrec_scan_selective_workspace_size(*shape, F32, 0) == 0


def test_scan_arguments(lib):
    assert fwd(lib, dtype=2) == INVALID
    assert fwd(lib, u=None) == INVALID
    assert fwd(lib, A=None) == INVALID
    assert fwd(lib, y=None) == INVALID
    assert fwd(lib, u=ODD) == UNSUPPORTED
    assert fwd(lib, u=HALF) == UNSUPPORTED
    assert fwd(lib, dtype=BF16, u=ODD) == UNSUPPORTED
    assert fwd(lib, dtype=BF16, z=ODD) == UNSUPPORTED
    for name in ("D", "bias", "lengths", "s_in", "s_out"):
        assert fwd(lib, dtype=BF16, **{name: HALF}) == UNSUPPORTED
    need = lib.linrec_scan_selective_workspace_size(*SHAPE, F32, 0)
    assert need > 0
    assert fwd(lib, nws=need - 1) == WORKSPACE
    assert fwd(lib, ws=None) == INVALID
    assert fwd(lib, ws=ctypes.c_void_p(0x100008)) == UNSUPPORTED
    assert fwd(lib, (0, 70, 12, 2, 16), u=None) == OK
    assert fwd(lib, (2, 70, 0, 2, 16), u=None) == OK
    assert fwd(lib, (2, 0, 12, 2, 16), u=None) == OK  # no state to pass on


def test_scan_step_arguments(lib):
    def call(shape=(2, 12, 2, 16), dtype=F32, u=P, s_in=P, y=P, s_out=P):
        return lib.linrec_scan_selective_decode_step(*shape, dtype, u, P, P, P, P, None, None, None, 1, s_in, y, s_out, None)
    assert call(shape=(-1, 12, 2, 16)) == INVALID
    assert call(shape=(2, 12, 5, 16)) == INVALID
    assert call(dtype=7) == INVALID
    assert call(u=None) == INVALID
    assert call(s_out=None) == INVALID
    assert call(s_in=HALF) == UNSUPPORTED
    assert call(shape=(0, 12, 2, 16), u=None) == OK


def test_scan_training_arguments(lib):
    nck = lib.linrec_scan_selective_checkpoint_size(*SHAPE, F32)
    nws = lib.linrec_scan_selective_workspace_size(*SHAPE, F32, 0)
    full = lib.linrec_scan_selective_workspace_size(*SHAPE, F32, 1)
    kept = lib.linrec_scan_selective_workspace_size(*SHAPE, F32, 2)
    assert nck >= 2 * 5 * 12 * 16 * 4 and 0 < kept < full

    def keep(ckpt=P, n=nck, y=P, ws=P, w=nws):
        return lib.linrec_scan_selective_ckpt(*SHAPE, F32, P, P, P, P, P, None, None, None, 1, None, None, y, None, ckpt, n,
                                              ws, w, None)
    assert keep(n=nck - 1) == WORKSPACE
    assert keep(ckpt=None) == INVALID
    assert keep(ckpt=ctypes.c_void_p(0x100004)) == UNSUPPORTED
    assert keep(y=None) == INVALID
    assert keep(w=nws - 1) == WORKSPACE

    def bwd(sizes=SHAPE, D=None, gD=None, z=None, gz=None, bias=None, gbias=None, s_in=None, ckpt=None, n=nck, gy=P, gu=P,
            gA=P, gs_out=None, gs_in=None, ws=P, w=full):
        return lib.linrec_scan_selective_backward(*sizes, F32, P, P, P, P, P, D, z, bias, 1, None, s_in, ckpt, n, gy, gs_out,
                                                  gu, P, gA, P, P, gD, gz, gbias, gs_in, ws, w, None)
    assert bwd(w=full - 1) == WORKSPACE
    assert bwd(ckpt=P, w=kept - 1) == WORKSPACE
    assert bwd(ckpt=P, n=nck - 1) == WORKSPACE
    for pair in (("D", "gD"), ("z", "gz"), ("bias", "gbias")):
        for name in pair:
            assert bwd(**{name: P}) == INVALID
    assert bwd(gy=None) == INVALID
    assert bwd(gu=None) == INVALID
    assert bwd(gA=None) == INVALID
    assert bwd(gu=ODD) == UNSUPPORTED
    assert bwd(z=P, gz=ODD) == UNSUPPORTED
    assert bwd(gA=HALF) == UNSUPPORTED
    assert bwd(gs_in=P) == INVALID  # without s_in
    assert bwd(gs_out=ODD) == UNSUPPORTED
    assert bwd(ws=None) == INVALID
    assert bwd(sizes=(2, 70, 0, 2, 16), gy=None, gA=None) == OK
    # Blocks of the backward beyond its grid.
    wide = (1 << 10, 1 << 20, 1, 1, 1)
    assert fwd(lib, wide, nws=0) == WORKSPACE
    assert bwd(sizes=wide) == UNSUPPORTED
    assert lib.linrec_scan_selective_workspace_size(*wide, F32, 1) == 0


def test_conv_arguments(lib):
    def fwd(B=2, T=9, C=12, K=4, dtype=F32, x=P, w=P, bias=None, act=1, lengths=None, s_in=None, y=P, s_out=None):
        return lib.short_conv_act(B, T, C, K, dtype, x, w, bias, act, lengths, s_in, y, s_out, None)
    for bad in (dict(B=-1), dict(T=-1), dict(C=-1), dict(K=0), dict(K=9), dict(dtype=3), dict(act=2), dict(x=None),
                dict(w=None), dict(y=None)):
        assert fwd(**bad) == INVALID, bad
    for bad in (dict(x=HALF), dict(dtype=BF16, x=ODD), dict(w=HALF), dict(bias=HALF), dict(lengths=HALF), dict(s_in=HALF),
                dict(dtype=BF16, s_out=ODD), dict(B=(1 << 20) + 1), dict(T=(1 << 30) + 1), dict(C=(1 << 24) + 1),
                dict(B=1 << 20, T=1 << 30), dict(T=1 << 30, C=1 << 10), dict(B=1 << 62, T=1 << 62, C=1 << 62)):
        assert fwd(**bad) == UNSUPPORTED, bad
    assert fwd(B=0, x=None) == OK
    assert fwd(C=0, x=None) == OK
    assert fwd(T=0, x=None, y=None) == OK

    def step(K=4, x=P, s_in=P, s_out=P, dtype=F32):
        return lib.short_conv_decode_step(2, 12, K, dtype, x, P, None, 1, s_in, P, s_out, None)
    assert step(s_out=None) == INVALID
    assert step(K=9) == INVALID
    assert step(x=None) == INVALID
    assert step(s_in=HALF) == UNSUPPORTED

    need = lib.short_conv_act_backward_workspace_size(2, 9, 12, 4, F32)
    assert need > 0 and lib.short_conv_act_backward_workspace_size(2, 9, 12, 9, F32) == 0

    def bwd(B=2, C=12, bias=None, gbias=None, s_in=None, gy=P, gs_out=None, gx=P, gw=P, gs_in=None, ws=P, nws=need):
        return lib.short_conv_act_backward(B, 9, C, 4, F32, P, P, bias, 1, None, s_in, gy, gs_out, gx, gw, gbias, gs_in, ws,
                                           nws, None)
    for bad in (dict(bias=P), dict(gbias=P), dict(gy=None), dict(gx=None), dict(gw=None), dict(gs_in=P),
                dict(s_in=P, gs_in=P, gs_out=P), dict(ws=None), dict(B=0, gw=None)):
        assert bwd(**bad) == INVALID, bad
    for bad in (dict(gw=HALF), dict(gx=HALF), dict(gs_out=HALF), dict(ws=ctypes.c_void_p(0x100008))):
        assert bwd(**bad) == UNSUPPORTED, bad
    assert bwd(nws=need - 1) == WORKSPACE
    assert bwd(C=0, gw=None) == OK


def test_rms_arguments(lib):
    def fwd(N=4, C=64, dtype=F32, rtype=F32, x=P, res=None, w=P, eps=1e-5, y=P, s=None):
        return lib.rms_norm_add(N, C, dtype, rtype, x, res, w, eps, y, s, None)
    for bad in (dict(N=-1), dict(C=-1), dict(dtype=9), dict(rtype=9), dict(rtype=BF16), dict(eps=-1.0),
                dict(eps=float("nan")), dict(x=None), dict(w=None), dict(y=None), dict(res=P), dict(s=P),
                dict(N=1 << 62)):
        assert fwd(**bad) == INVALID, bad
    for bad in (dict(C=8193), dict(x=HALF), dict(dtype=BF16, x=ODD), dict(dtype=BF16, res=HALF, s=P), dict(w=HALF)):
        assert fwd(**bad) == UNSUPPORTED, bad
    assert fwd(N=0, x=None) == OK
    assert fwd(C=0, x=None) == OK
    need = lib.rms_norm_add_backward_workspace_size(4, 64)
    assert need > 0 and lib.rms_norm_add_backward_workspace_size(4, 8193) == 0

    def bwd(N=4, dtype=F32, rtype=F32, s=P, gy=P, gsum=None, gx=None, gs=P, gw=P, ws=P, nws=need):
        return lib.rms_norm_add_backward(N, 64, dtype, rtype, s, P, gy, gsum, 1e-5, gx, gs, gw, ws, nws, None)
    for bad in (dict(s=None), dict(gy=None), dict(gs=None), dict(gw=None), dict(gx=P), dict(ws=None), dict(N=0, gw=None),
                dict(dtype=BF16, rtype=BF16, gx=P), dict(dtype=F32, rtype=BF16)):
        assert bwd(**bad) == INVALID, bad
    for bad in (dict(gsum=HALF), dict(gw=HALF), dict(dtype=BF16, gx=ODD)):
        assert bwd(**bad) == UNSUPPORTED, bad
    assert bwd(nws=need - 1) == WORKSPACE
