"""What the state-space block's operators refuse, at the C entries and in the binding, without a GPU: every check comes
before anything is enqueued.  And the sizes of their workspaces at the ends of their ranges."""

import ctypes

import pytest
import torch

import layer_rnn_forward_amd as R
from layer_rnn_forward_amd._binding import _SsmGrads, _SsmInputs

INVALID, UNSUPPORTED, SMALL = -1, -2, -3
SOME = 1 << 20          # an address (multiple of 256) that no refused call follows
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return R.load_library()


def test_norm(lib):
    n = ctypes.c_size_t()
    for args, want in (((4, 8), 0), ((0, 0), 0), ((-1, 8), INVALID), ((4, -8), INVALID), ((4, 1 << 20), UNSUPPORTED),
                       ((1 << 30, 8), UNSUPPORTED)):
        assert lib.rnn_norm_workspace_size(*args, ctypes.byref(n)) == want, args
    assert lib.rnn_norm_workspace_size(4, 8, None) == INVALID
    assert R.rnn_norm_workspace_size(1 << 29, (1 << 20) - 1) >= (1 << 20) * 4 * 2

    def fwd(kind=0, wt=0, M=4, D=8, x=SOME, eps=1e-5, y=SOME):
        return lib.rnn_norm_forward(None, kind, wt, M, D, x, None, None, None, eps, y, None, None)

    for bad in (dict(kind=2), dict(kind=-1), dict(wt=2), dict(M=-1), dict(D=-1), dict(x=None), dict(y=None), dict(eps=-1e-5),
                dict(eps=NAN), dict(eps=INF)):
        assert fwd(**bad) == INVALID, bad
    assert fwd(D=1 << 20) == UNSUPPORTED and fwd(M=0) == 0 and fwd(D=0) == 0
    size = R.rnn_norm_workspace_size(4, 8)

    def bwd(kind=0, wt=0, M=4, D=8, s=SOME, st=SOME, dy=SOME, dw=SOME, ws=SOME, n=size):
        return lib.rnn_norm_backward(None, kind, wt, M, D, s, None, st, dy, None, SOME, dw, None, ws, n)

    for bad in (dict(kind=2), dict(wt=-1), dict(M=-1), dict(D=-1), dict(s=None), dict(st=None), dict(dy=None), dict(ws=None), dict(ws=SOME + 16)):
        assert bwd(**bad) == INVALID, bad
    assert bwd(n=size - 1) == SMALL and bwd(D=0) == 0 and bwd(M=1 << 30) == UNSUPPORTED


def test_conv(lib):
    n = ctypes.c_size_t()
    for args, want in (((4, 2, 8, 4), 0), ((0, 0, 0, 1), 0), ((-1, 2, 8, 4), INVALID), ((4, -2, 8, 4), INVALID), ((4, 2, -8, 4), INVALID),
                       ((4, 2, 8, 0), INVALID), ((4, 2, 8, 9), UNSUPPORTED), ((4, 1 << 15, 1 << 15, 4), UNSUPPORTED),
                       ((1 << 30, 1, 1, 4), UNSUPPORTED), ((1, 1 << 24, 1, 4), UNSUPPORTED), ((1 << 29, 1 << 10, 1, 4), 0)):
        assert lib.rnn_conv_workspace_size(*args, ctypes.byref(n)) == want, args
    assert lib.rnn_conv_workspace_size(4, 2, 8, 4, None) == INVALID

    def fwd(act=1, wt=0, T=4, B=2, C=8, K=4, x=SOME, ldx=8, w=SOME, y=SOME, ldy=8):
        return lib.rnn_conv_forward(None, act, wt, T, B, C, K, x, ldx, w, None, None, None, y, ldy, None)

    def step(act=1, wt=0, B=2, C=8, K=4, x=SOME, ldx=8, w=SOME, y=SOME, ldy=8):
        return lib.rnn_conv_step(None, act, wt, B, C, K, x, ldx, w, None, None, y, ldy, None)

    size = R.rnn_conv_workspace_size(4, 2, 8, 4)

    def bwd(act=1, wt=0, T=4, B=2, C=8, K=4, x=SOME, ldx=8, w=SOME, dy=SOME, lddy=8, lddx=8, ws=SOME, n=size):
        return lib.rnn_conv_backward(None, act, wt, T, B, C, K, x, ldx, w, None, None, None, dy, lddy, None, SOME, lddx, SOME,
                                     None, None, ws, n)

    for call in (fwd, step, bwd):
        for bad in (dict(act=0), dict(act=2), dict(act=4), dict(act=-1), dict(wt=2), dict(B=-1), dict(C=-1), dict(K=0), dict(x=None), dict(w=None),
                    dict(ldx=7)):
            assert call(**bad) == INVALID, (call, bad)
        assert call(K=9) == UNSUPPORTED and call(B=1 << 15, C=1 << 15, ldx=1 << 15) == UNSUPPORTED
    assert fwd(T=-1) == INVALID and fwd(y=None) == INVALID and fwd(ldy=7) == INVALID and step(y=None) == INVALID
    assert fwd(B=0) == 0 and fwd(C=0, ldx=0, ldy=0) == 0 and step(B=0) == 0
    for bad in (dict(T=-1), dict(dy=None), dict(lddy=7), dict(lddx=7), dict(ws=None), dict(ws=SOME + 128)):
        assert bwd(**bad) == INVALID, bad
    assert bwd(n=size - 1) == SMALL


def inputs(**other):
    v = dict(u=SOME, delta=SOME, z=SOME, Bm=SOME, Cm=SOME, ldu=8, lddelta=8, ldz=8, ldB=4, ldC=4, A=SOME, D=SOME, delta_bias=SOME)
    return _SsmInputs(**(v | other))


def test_ssm(lib):
    n = ctypes.c_size_t()
    for args, want in (((4, 2, 8, 4, 1, 0), 0), ((4, 2, 8, 4, 2, 1), 0), ((0, 0, 0, 1, 1, 1), 0), ((-1, 2, 8, 4, 1, 0), INVALID),
                       ((4, -2, 8, 4, 1, 0), INVALID), ((4, 2, -8, 4, 1, 0), INVALID), ((4, 2, 8, 0, 1, 0), INVALID), ((4, 2, 8, 4, 0, 0), INVALID),
                       ((4, 2, 8, 4, 3, 0), INVALID), ((4, 2, 8, 4, 1, 2), INVALID), ((4, 2, 8, 4, 1, -1), INVALID), ((4, 2, 8, 65, 1, 0), UNSUPPORTED),
                       ((4, 1 << 15, 1 << 15, 4, 1, 0), UNSUPPORTED), ((1 << 30, 1, 8, 4, 1, 0), UNSUPPORTED), ((4, 1, 1 << 22, 4, 1, 0), UNSUPPORTED),
                       ((1, 1 << 24, 8, 4, 1, 0), UNSUPPORTED), ((1, 1 << 20, 64, 4, 64, 0), UNSUPPORTED), ((4, 1 << 14, 1 << 12, 16, 1, 1), 0)):
        assert lib.rnn_ssm_workspace_size(*args, ctypes.byref(n)) == want, args
    assert lib.rnn_ssm_workspace_size(4, 2, 8, 4, 1, 0, None) == INVALID
    # the states before every 8th step, 16 of them a channel
    assert R.rnn_ssm_workspace_size(1 << 20, 4, 1 << 10, 16, 1, "full") >= (1 << 17) * 4 * (1 << 10) * 16 * 4
    size, full = R.rnn_ssm_workspace_size(4, 2, 8, 4), R.rnn_ssm_workspace_size(4, 2, 8, 4, 1, "full")

    def fwd(mode=0, wt=0, save=0, T=4, B=2, E=8, N=4, G=1, ins=inputs(), y=SOME, ldy=8, ws=SOME, n=full):
        return lib.rnn_ssm_forward(None, mode, wt, save, T, B, E, N, G, ins and ctypes.byref(ins), None, None, y, ldy, None, ws, n)

    def step(mode=0, wt=0, B=2, E=8, N=4, G=1, ins=inputs(), y=SOME, ldy=8):
        return lib.rnn_ssm_step(None, mode, wt, B, E, N, G, ins and ctypes.byref(ins), None, y, ldy, None)

    def bwd(mode=0, wt=0, T=4, B=2, E=8, N=4, G=1, ins=inputs(), dy=SOME, lddy=8, grads=_SsmGrads(), ws=SOME, n=full):
        return lib.rnn_ssm_backward(None, mode, wt, T, B, E, N, G, ins and ctypes.byref(ins), None, dy, lddy, None,
                                    grads and ctypes.byref(grads), ws, n)

    big = 1 << 28
    for call in (fwd, bwd):
        assert call(ins=inputs(ldu=big)) == UNSUPPORTED and call(ins=inputs(ldC=big)) == UNSUPPORTED      # B * ld > 2^28
    for call in (fwd, step, bwd):
        for bad in (dict(mode=2), dict(mode=-1), dict(wt=2), dict(B=-1), dict(E=-1), dict(N=0), dict(G=3), dict(G=0), dict(ins=None),
                    *[dict(ins=inputs(**{k: None})) for k in ("u", "delta", "Bm", "Cm", "A")],
                    *[dict(ins=inputs(**{k: v})) for k, v in (("ldu", 7), ("lddelta", 0), ("ldz", -8), ("ldB", 3), ("ldC", 3))]):
            assert call(**bad) == INVALID, (call, bad)
        assert call(N=65) == UNSUPPORTED and call(B=1 << 24) == UNSUPPORTED and call(E=1 << 22) == UNSUPPORTED
    for bad in (dict(T=-1), dict(save=2), dict(y=None), dict(ldy=7), dict(ws=None), dict(ws=SOME + 64)):
        assert fwd(**bad) == INVALID, bad
    assert fwd(n=size - 1) == SMALL and fwd(save=1, n=full - 1) == SMALL and fwd(B=0) == 0 and step(B=0) == 0
    assert step(y=None) == INVALID and step(ldy=7) == INVALID
    for bad in (dict(T=-1), dict(dy=None), dict(lddy=7), dict(grads=None), dict(ws=None), dict(ws=SOME + 64),
                dict(ins=inputs(z=None), grads=_SsmGrads(dz=SOME, lddz=8)), dict(grads=_SsmGrads(du=SOME, lddu=7)),
                dict(grads=_SsmGrads(dBm=SOME, lddB=3))):
        assert bwd(**bad) == INVALID, bad
    assert bwd(n=full - 1) == SMALL and bwd(grads=_SsmGrads(ddelta=SOME, ldddelta=big)) == UNSUPPORTED


def test_binding_refuses_host_tensors_and_wrong_arguments():
    x, v = torch.zeros(4, 2, 8), torch.zeros(8)
    rows, w, A, bc = torch.zeros(4, 8), torch.zeros(8, 4), torch.zeros(8, 4), torch.zeros(4, 2, 4)
    for call in (lambda: R.rnn_norm_forward("batch", rows, None, v, None, rows), lambda: R.rnn_norm_forward("rms", rows, None, v, None, rows),
                 lambda: R.rnn_norm_backward("rms", rows, v, rows[:, :2], rows, None, rows, None, None),
                 lambda: R.rnn_conv_forward("gelu", x, w, None, None, None, x, None), lambda: R.rnn_conv_forward("silu", x, w, None, None, None, x, None),
                 lambda: R.rnn_conv_step("silu", rows, w, None, None, rows, None),
                 lambda: R.rnn_conv_backward("silu", x, w, None, None, None, x, None, x, None, None, None),
                 lambda: R.rnn_ssm_forward("exp", x, x, A, bc, bc, v, x, v, None, None, x, None, rows),
                 lambda: R.rnn_ssm_forward("softplus", x, x, A, bc, bc, v, x, v, None, None, x, None, rows),
                 lambda: R.rnn_ssm_step("softplus", rows, rows, A, rows[:, :4], rows[:, :4], v, rows, v, None, rows, None),
                 lambda: R.rnn_ssm_forward("softplus", x, x, A, bc[..., :3], bc, v, x, v, None, None, x, None, rows),
                 lambda: R.rnn_norm_forward("rms", rows.double(), None, v, None, rows), lambda: R.rnn_conv_forward("silu", rows, w, None, None, None, x, None),
                 lambda: R.rnn_ssm_workspace_size(4, 2, 8, 4, 1, "int8"), lambda: R.rnn_ssm_workspace_size(1 << 32, 1, 1, 1),
                 lambda: R.rnn_norm_workspace_size(1 << 31, 1), lambda: R.rnn_conv_workspace_size(1, 1, 1 << 40, 4)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        R.rnn_norm_forward("rms", None, None, None, None, rows)
    with pytest.raises(R.RNNError):
        R.rnn_ssm_workspace_size(4, 2, 8, 4, 3)
