"""Normalisation of rows on the GPU against the definition in 64 bits; tolerances are the oracle's bounds on an evaluation
in fp32 and half a step of the output's type."""

import pytest
import torch

import layer_rnn_forward_amd as R
from oracle.bounds import check
from tests.block_gpu import norm_case, norm_run, norm_want, numbers, room

pytestmark = pytest.mark.gpu


def compare(kind, c, dtype, eps=1e-5):
    got, want = norm_run(kind, c, eps), norm_want(kind, c, eps)
    for k, v in want.items():
        if k == "total":
            assert torch.equal(got[k].cpu(), v)
        else:
            check(k, got[k], v, "f32" if k in ("dweight", "dbias") else dtype)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,D", [(1, 1), (3, 2), (1, 64), (5, 63), (16, 800), (2, 2048), (130, 257), (33, 1357), (7, 4096), (3, 8192),
                                 (2, 8195), (1500, 40), (1025, 513), (1030, 1100)])
def test_rows(kind, dtype, M, D):
    print("CASE norm", kind, dtype, M, D, flush=True)
    compare(kind, norm_case(M, D, dtype, residual=(M + D) % 2 == 0), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,D", [(2, 32768), (3, 32769), (2, 100001)])
def test_long_rows(dtype, M, D):
    for residual in (True, False):
        compare("layer", norm_case(M, D, dtype, residual=residual), dtype)
    compare("rms", norm_case(M, D, dtype), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_parameters(dtype):
    for weight, bias in ((False, True), (True, False), (False, False)):
        compare("layer", norm_case(37, 300, dtype, weight=weight, bias=bias), dtype)


def test_far_from_zero():
    """A mean of 1000 with a deviation of 1: nothing cancels in the sum of squares about the mean."""
    compare("layer", norm_case(9, 777, "f32", residual=False, spread=1000.0), "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [300, 2050, 40000])
def test_total_in_place(dtype, D):
    """The residual stream updated in place, from either side, and dx over dtotal."""
    c = norm_case(21, D, dtype)
    want = norm_run("layer", c)
    for which in ("x", "residual"):
        g = {k: v.cuda() for k, v in c.items()}
        y, stats = torch.empty_like(g["x"]), torch.empty(21, 2, device="cuda")
        R.rnn_norm_forward("layer", g["x"], g["residual"], g["weight"], g["bias"], y, g[which], stats)
        assert torch.equal(y, want["y"]) and torch.equal(g[which], want["total"])
        R.rnn_norm_backward("layer", g[which], g["weight"], stats, g["dy"], g["dtotal"], g["dtotal"], None, None)
        assert torch.equal(g["dtotal"], want["dx"])


def test_not_wanted_gradients():
    c = norm_case(50, 130, "bf16")
    want = norm_run("layer", c)
    g = {k: v.cuda() for k, v in c.items()}
    y, total, stats = torch.empty_like(g["x"]), torch.empty_like(g["x"]), torch.empty(50, 2, device="cuda")
    R.rnn_norm_forward("layer", g["x"], g["residual"], g["weight"], g["bias"], y, total, stats)
    ws = room(R.rnn_norm_workspace_size(50, 130))
    for name in ("dx", "dweight", "dbias"):
        out = {k: torch.empty_like(want[k]) if k == name else None for k in ("dx", "dweight", "dbias")}
        R.rnn_norm_backward("layer", total, g["weight"], stats, g["dy"], g["dtotal"], out["dx"], out["dweight"], out["dbias"], ws)
        assert torch.equal(out[name], want[name])


def test_no_rows():
    """The parameters' gradients over no rows are zero."""
    x, w = torch.empty(0, 24, device="cuda"), torch.ones(24, device="cuda")
    R.rnn_norm_forward("rms", x, None, w, None, x, None, None)
    dw, db = torch.full_like(w, 3.0), torch.full_like(w, 3.0)
    R.rnn_norm_backward("rms", x, w, torch.empty(0, 2, device="cuda"), x, None, x, dw, db, room(R.rnn_norm_workspace_size(0, 24)))
    assert not dw.any() and not db.any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinities_stay_in_their_row(dtype):
    c = norm_case(12, 700, dtype, residual=False)
    want = norm_run("layer", c)
    c["x"][3, 40], c["x"][7, 699] = float("inf"), float("nan")
    got = norm_run("layer", c)
    rows = [i for i in range(12) if i not in (3, 7)]
    for k in ("y", "dx"):
        assert torch.equal(got[k][rows], want[k][rows]) and got[k][[3, 7]].isnan().all()
    assert got["dweight"].isnan().all() and torch.equal(got["dbias"], want["dbias"])


def test_misaligned_rows():
    """Rows that start at any element."""
    for dtype in (torch.float32, torch.bfloat16):
        base = numbers(3, (1 + 5 * 333,)).to(dtype).cuda()
        x, y = base[1:].view(5, 333), torch.empty(1 + 5 * 333, dtype=dtype, device="cuda")[1:].view(5, 333)
        want = torch.empty_like(x)
        R.rnn_norm_forward("rms", x.clone(), None, None, None, want)
        R.rnn_norm_forward("rms", x, None, None, None, y)
        assert torch.equal(y, want)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,D", [(600, 8195), (300, 16384), (150, 16400)])
def test_several_long_rows_a_workgroup(kind, dtype, M, D):
    """Workgroups of 1024 lanes that walk several rows, and sums by columns over every 64th row."""
    print("CASE norm", kind, dtype, M, D, flush=True)
    compare(kind, norm_case(M, D, dtype, seed=3), dtype)
