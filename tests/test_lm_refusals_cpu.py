"""What the language-model operators refuse, at the C entries and in the binding, without a GPU: every check
comes before anything is enqueued."""

import ctypes

import pytest
import torch

import layer_rnn_forward_amd as R

INVALID, UNSUPPORTED, SMALL = -1, -2, -3
P = ctypes.c_void_p
SOME = 1 << 20          # an address (multiple of 256) that no refused call follows


@pytest.fixture(scope="module")
def lib():
    return R.load_library()


def test_scan_sizes(lib):
    n = ctypes.c_size_t()
    for args, want in (((4, 2, 8, 1), 0), ((0, 0, 0, 2), 0), ((-1, 2, 8, 1), INVALID), ((4, -2, 8, 1), INVALID),
                       ((4, 2, -8, 1), INVALID), ((4, 2, 8, 3), INVALID), ((4, 2, 8, 0), INVALID),
                       ((4, 1 << 15, 1 << 15, 1), UNSUPPORTED), ((4, 1 << 30, 1 << 30, 2), UNSUPPORTED)):
        assert lib.rnn_scan_workspace_size(*args, ctypes.byref(n)) == want, args
    assert lib.rnn_scan_workspace_size(4, 2, 8, 1, None) == INVALID
    assert R.rnn_scan_workspace_size(1000, 4, 64, 2) >= R.rnn_scan_workspace_size(10, 4, 64, 2)
    with pytest.raises(R.RNNError):
        R.rnn_scan_workspace_size(-1, 1, 1)


def test_scan_calls(lib):
    ws = R.rnn_scan_workspace_size(4, 2, 8, 1)

    def fwd(mode=0, wt=0, T=4, B=2, H=8, D=1, g=SOME, y=SOME, w=SOME, n=ws):
        return lib.rnn_scan_forward(None, mode, wt, T, B, H, D, g, None, None, y, None, w, n)

    def bwd(mode=0, wt=0, T=4, B=2, H=8, D=1, g=SOME, dy=SOME, dg=SOME, w=SOME, n=ws):
        return lib.rnn_scan_backward(None, mode, wt, T, B, H, D, g, None, None, dy, None, dg, None, w, n)

    for call in (fwd, bwd):
        for bad in (dict(mode=2), dict(mode=-1), dict(wt=2), dict(T=-1), dict(B=-1), dict(H=-1), dict(D=3), dict(g=None),
                    dict(w=None), dict(w=SOME + 16)):
            assert call(**bad) == INVALID, bad
        assert call(n=ws - 1) == SMALL
        assert call(B=0) == 0                       # nothing to do
    assert fwd(y=None) == INVALID and bwd(dy=None) == INVALID and bwd(dg=None) == INVALID
    step = lambda mode=0, wt=0, B=2, H=8, g=SOME, hy=SOME: lib.rnn_scan_step(None, mode, wt, B, H, g, None, None, hy)  # noqa: E731
    for bad in (dict(mode=5), dict(wt=-1), dict(B=-1), dict(H=-1), dict(g=None), dict(hy=None)):
        assert step(**bad) == INVALID, bad
    assert step(B=1 << 15, H=1 << 15) == UNSUPPORTED and step(B=0) == 0


def test_ffn_sizes(lib):
    n = ctypes.c_size_t()
    for f in (lib.rnn_ffn_workspace_size, lib.rnn_ffn_reserve_size):
        for args, want in (((4, 8, 16, 1, 1), 0), ((0, 8, 16, 0, 2), 0), ((-1, 8, 16, 1, 1), INVALID),
                           ((4, -8, 16, 1, 1), INVALID), ((4, 8, -1, 1, 1), INVALID), ((4, 8, 16, 2, 1), INVALID),
                           ((4, 8, 16, 1, 3), INVALID), ((4, 8, 16, 1, -1), INVALID), ((4, 1 << 24, 16, 1, 1), UNSUPPORTED),
                           ((4, 8, 1 << 24, 1, 1), UNSUPPORTED), ((1 << 30, 8, 8, 1, 1), UNSUPPORTED)):
            assert f(*args, ctypes.byref(n)) == want, args
        assert f(4, 8, 16, 1, 1, None) == INVALID
    assert R.rnn_ffn_reserve_size(64, 32, 96, "bf16", "none") == 0
    # 8-bit checkpoints: x and two projections, a byte a value and one for 32
    small, full = (R.rnn_ffn_reserve_size(4096, 1024, 4096, "bf16", s) for s in ("int8", "full"))
    assert 4096 * (1024 + 2 * 4096) <= small < 1.05 * 4096 * (1024 + 2 * 4096) and full > 1.9 * small / 1.2


def test_ffn_calls(lib):
    M, D, F = 4, 8, 16
    for save in (0, 1, 2):
        ws = R.rnn_ffn_workspace_size(M, D, F, "bf16", ["none", "full", "int8"][save])
        rs = R.rnn_ffn_reserve_size(M, D, F, "bf16", ["none", "full", "int8"][save])

        def fwd(act=1, wt=1, save=save, M=M, D=D, F=F, x=SOME, wi=SOME, wo=SOME, y=SOME, w=SOME, n=ws, r=SOME, m=rs):
            return lib.rnn_ffn_forward(None, act, wt, save, M, D, F, x, wi, wo, y, w, n, r, m)

        def bwd(act=1, wt=1, save=save, M=M, D=D, F=F, x=SOME, wi=SOME, wo=SOME, dy=SOME, w=SOME, n=ws, r=SOME, m=rs):
            return lib.rnn_ffn_backward(None, act, wt, save, M, D, F, x, wi, wo, dy, SOME, SOME, SOME, w, n, r, m)

        for call in (fwd,) + ((bwd,) if save else ()):
            for bad in (dict(act=3), dict(act=-1), dict(wt=2), dict(save=3), dict(M=-1), dict(D=-1), dict(F=-1),
                        dict(wi=None), dict(wo=None), dict(w=None), dict(w=SOME + 128)):
                assert call(**bad) == INVALID, (save, bad)
            assert call(n=ws - 1) == SMALL
            if save:
                assert call(r=None) == INVALID and call(r=SOME + 8) == INVALID and call(m=rs - 1) == SMALL
        assert fwd(x=None) == INVALID and fwd(y=None) == INVALID
        assert fwd(M=0) == 0
        if save:
            assert bwd(dy=None) == INVALID
        if save == 1:
            assert bwd(x=None) == INVALID
    assert lib.rnn_ffn_backward(None, 1, 1, 0, M, D, F, SOME, SOME, SOME, SOME, SOME, SOME, SOME, SOME, 1 << 30, SOME,
                                1 << 30) == INVALID      # nothing was saved


def test_checkpoint_calls(lib):
    n = ctypes.c_size_t()
    assert lib.rnn_checkpoint_size(3, 33, ctypes.byref(n)) == 0 and n.value == 3 * 33 + 3 * 2
    assert lib.rnn_checkpoint_size(1 << 20, 1 << 14, ctypes.byref(n)) == 0 and n.value == (1 << 34) + (1 << 29)
    for args, want in (((-1, 4), INVALID), ((4, -1), INVALID), ((4, 1 << 30), UNSUPPORTED)):
        assert lib.rnn_checkpoint_size(*args, ctypes.byref(n)) == want
    assert lib.rnn_checkpoint_size(3, 33, None) == INVALID
    store = lambda wt=0, r=3, c=33, x=SOME, k=SOME, b=105: lib.rnn_checkpoint_store(None, wt, r, c, x, k, b)  # noqa: E731
    load = lambda wt=0, r=3, c=33, x=SOME, k=SOME, b=105: lib.rnn_checkpoint_load(None, wt, r, c, k, b, x)  # noqa: E731
    for call in (store, load):
        for bad in (dict(wt=2), dict(r=-1), dict(c=-1), dict(x=None), dict(k=None), dict(k=SOME + 1)):
            assert call(**bad) == INVALID, bad
        assert call(b=104) == SMALL and call(r=0, b=0, x=None, k=None) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    g, h = torch.zeros(3, 2, 16), torch.zeros(1, 2, 8)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device"):
        R.rnn_scan_forward("gated", g, h, None, torch.zeros(3, 2, 8), h, ws)
    with pytest.raises(ValueError, match="mode"):
        R.rnn_scan_forward("lstm", g, h, None, torch.zeros(3, 2, 8), h, ws)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        R.rnn_scan_forward("gated", g.double(), h, None, torch.zeros(3, 2, 8), h, ws)
    with pytest.raises(ValueError, match="dimensions"):
        R.rnn_scan_step("gated", g, h, None, h)
    with pytest.raises(ValueError, match="even"):
        R.rnn_scan_step("gated", torch.zeros(2, 7), None, None, torch.zeros(2, 3))
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="act"):
        R.rnn_ffn_forward("relu", x, x, x, x, ws)
    with pytest.raises(ValueError, match="save"):
        R.rnn_ffn_forward("silu", x, x, x, x, ws, "fp8")
    with pytest.raises(ValueError, match="device"):
        R.rnn_ffn_forward("silu", x, torch.zeros(32, 8), torch.zeros(8, 16), x, ws)
    with pytest.raises(TypeError):
        R.rnn_checkpoint_store([1.0], ws)
    with pytest.raises(ValueError, match="device"):
        R.rnn_checkpoint_load(ws, x)
    with pytest.raises(ValueError):
        R.rnn_ffn_workspace_size(1, 1, 1, "fp16")
