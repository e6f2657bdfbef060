"""The scan where the products of its coefficients leave fp32's range although no state does: steps that grow and
fall by many powers of two, with and without resets (a = 0), both passes.  Tolerances as in the scan's own tests
(derived there for any coefficients)."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import layer_rnn_forward_amd as R  # noqa: E402
from tests import test_gpu_lm_scan as scan  # noqa: E402

pytestmark = pytest.mark.gpu


def path(T, rate, resets, down, rng):
    """Exponents of the states' scale before every step and after the last, within -100 .. 100, and the steps that reset."""
    e, reset = np.empty(T + 1), np.zeros(T, bool)
    at, way = (100.0, -1) if down else (-100.0, 1)
    for t in range(T):
        e[t] = at
        nxt = at + way * rate
        if abs(nxt) > 100:
            if resets:
                reset[t], nxt = True, -100.0 * way
            else:
                way, nxt = -way, at
        elif resets and rng.random() < 0.004:
            reset[t], nxt = True, -100.0 * way
        at = nxt
    e[T] = at
    return e, reset


def make(dtype, T, B, H, rate, resets, down, add, seed=0):
    """One direction; states of scale 2^e[t], gradients of scale 2^-e[t]."""
    rng = np.random.default_rng([seed, T, B, H, rate, resets, down])
    e, reset = path(T, rate, resets, down, rng)
    a = np.exp2(np.diff(e))[:, None, None] * rng.choice([-1.0, 1.0], size=(T, B, H))
    a[reset] = 0
    b = rng.normal(size=(T, B, H)) * np.exp2(e[1:])[:, None, None] * (0.25 if add else 0.0)
    b[reset] = rng.normal(size=b[reset].shape) * np.exp2(e[1:][reset])[:, None, None]
    dy = rng.normal(size=(T, B, H)) * np.exp2(-e[1:])[:, None, None]
    dt = scan.DT[dtype]
    return dict(mode="linear", dtype=dtype, T=T, B=B, H=H, dirs=1, lengths=None,
                g=torch.tensor(np.concatenate([a, b], 2)).to(dt), dy=torch.tensor(dy).to(dt),
                h0=torch.tensor(rng.normal(size=(1, B, H)) * 2.0 ** e[0]).float(),
                dhy=torch.tensor(rng.normal(size=(1, B, H)) * 2.0 ** -e[T]).float())


def check(got, want):
    """scan.check, but for gradients that lie beyond fp32 (a large state meets a large gradient at a reset)."""
    want = {k: (ref, np.where(np.abs(ref) + tol < 2.0 ** 127, tol, np.inf)) for k, (ref, tol) in want.items()}
    got = {k: torch.where(torch.from_numpy(want[k][1]).isinf().to(v.device), 0.0, v.double()) for k, v in got.items()}
    scan.check(got, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rate", [1, 3, 12, 60])
@pytest.mark.parametrize("resets", [False, True])
@pytest.mark.parametrize("down", [False, True])
@pytest.mark.parametrize("add", [False, True])
def test_states_in_range(dtype, rate, resets, down, add):
    print("CASE scan range", dtype, rate, resets, down, add, flush=True)
    for T in (100, 700, 2500):
        c = make(dtype, T, 2, 70, rate, resets, down, add)
        check(scan.run(c), scan.expected(c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_reset_after_growth(dtype):
    """Growth from a state of zero leaves nothing behind once a = 0 and b = 1 are reached."""
    T, H = 700, 64
    g = torch.zeros(T, 1, 2 * H)
    g[:, :, :H] = 1e30
    g[-40, :, :H], g[-40, :, H:] = 0.0, 1.0
    g[-39:, :, :H] = 0.5
    y, hy = torch.empty(T, 1, H, device="cuda", dtype=scan.DT[dtype]), torch.empty(1, 1, H, device="cuda")
    ws = torch.empty(R.rnn_scan_workspace_size(T, 1, H, 1), dtype=torch.uint8, device="cuda")
    R.rnn_scan_forward("linear", g.to(scan.DT[dtype]).cuda(), None, None, y, hy, ws)
    assert (y[:-40] == 0).all() and (y[-40] == 1).all() and (hy == 2.0 ** -39).all()


def test_one_channel_beyond_the_range_leaves_the_others_alone():
    """Channels next to one that grows have bitwise the results they have without it."""
    c = scan.make("linear", "f32", 1500, 2, 70, 1)
    want = scan.run(c)
    hot = make("f32", 1500, 2, 70, 3, True, False, True)
    for k, cols in (("g", (5, 75)), ("dy", (5,)), ("h0", (5,)), ("dhy", (5,))):
        for i in cols:
            c[k][..., 0, i] = hot[k][..., 0, i]
    got = scan.run(c)
    check(got, scan.expected(c))
    for k in want:
        a, b = got[k].clone(), want[k].clone()
        for i in ((5, 75) if k == "dg" else (5,)):
            a[..., 0, i] = b[..., 0, i] = 0
        assert torch.equal(a, b), k


def test_repeats_are_bitwise():
    c = make("bf16", 3000, 2, 150, 3, True, False, True)
    a = scan.run(c)
    for _ in range(4):
        b = scan.run(c)
        for k in a:
            assert torch.equal(a[k], b[k]), k


def run_some():
    out = {}
    for i, (dtype, T, rate, down) in enumerate([("bf16", 3000, 3, False), ("f32", 3000, 12, False), ("bf16", 2000, 3, True)]):
        print("case", i, flush=True)
        got = scan.run(make(dtype, T, 2, 150, rate, True, down, True, seed=1))
        out |= {f"{i}.{k}": v.float().cpu().numpy() for k, v in got.items()}
    return out


@pytest.mark.timeout(300)
def test_perturbed_order_is_bitwise_equal(tmp_path):
    from layer_rnn_forward_amd.build import PERTURB_LIB
    assert os.path.exists(PERTURB_LIB), "the perturbed test build is missing (run build())"
    ref, out = run_some(), tmp_path / "perturbed.npz"
    r = subprocess.run([sys.executable, "-u", os.path.abspath(__file__), str(out)], env=dict(os.environ, RNN_LIB=PERTURB_LIB),
                       cwd=ROOT, capture_output=True, text=True, timeout=240)
    print(r.stdout[-2000:], r.stderr[-2000:], flush=True)
    assert r.returncode == 0 and "perturb" in r.stdout.splitlines()[0]
    got = np.load(out)
    assert sorted(got.files) == sorted(ref)
    for k, v in ref.items():
        assert np.array_equal(got[k].view(np.uint32), v.view(np.uint32)), k


if __name__ == "__main__":
    print("library", R.lib_path(), flush=True)
    np.savez(sys.argv[1], **run_some())
