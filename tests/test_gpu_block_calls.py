"""How the state-space block's operators are called: repeated, on other streams, two at once, captured into a graph and
replayed, through the interpreted entries, together as one block."""

import pytest
import torch

import layer_rnn_forward_amd as R
from layer_rnn_forward_amd import _binding
from oracle.bounds import check
from tests.block_gpu import (INPUTS, conv_case, conv_run, conv_want, gpu, norm_case, norm_run, room, ssm_case, ssm_run,
                             ssm_want)

pytestmark = pytest.mark.gpu


def passes():
    """Every entry once or more, with several segments and several workgroups a sum."""
    out = {}
    for dtype in ("f32", "bf16"):
        out |= {f"norm.{dtype}.{k}": v for k, v in norm_run("layer", norm_case(700, 900, dtype)).items()}
        out |= {f"conv.{dtype}.{k}": v for k, v in conv_run("silu", conv_case(150, 3, 300, 4, dtype, [150, 3, 77])).items()}
        out |= {f"ssm.{dtype}.{k}": v for k, v in ssm_run("softplus", ssm_case(400, 2, 90, 16, 1, dtype, [400, 130])).items()}
        x = torch.linspace(-2, 2, 60, device="cuda").view(3, 20).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
        s, y = torch.zeros(3, 3, 20, dtype=x.dtype, device="cuda"), torch.empty_like(x)
        R.rnn_conv_step("silu", x, torch.full((20, 4), 0.5, device="cuda"), None, s, y, s)
        h, A = torch.ones(3, 20, 4, device="cuda"), -torch.ones(20, 4, device="cuda")
        out |= {f"steps.{dtype}.y": y, f"steps.{dtype}.s": s, f"steps.{dtype}.h": h}
        R.rnn_ssm_step("softplus", x, x, A, x[:, :4], x[:, 4:8], None, x, None, h, y, h)
    return out


def same(got, want):
    assert got.keys() == want.keys()
    for k, v in want.items():
        assert torch.equal(got[k], v), k


def test_repeated_calls_are_bitwise_equal():
    same(passes(), passes())


def test_interpreted_calls(monkeypatch):
    want = passes()
    assert type(_binding._CALL).__name__ == "module", "the compiled entries are not built"
    monkeypatch.setattr(_binding, "_CALL", _binding._Interpreted("a test"))
    with pytest.warns(RuntimeWarning, match="_call.so"):
        got = passes()
    same(got, want)


def test_other_streams_and_two_calls_at_once():
    want = passes()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(passes())
    torch.cuda.synchronize()
    for g in got:
        same(g, want)


class Block:
    """A state-space block over x [T, B, D], forward and backward, from the library's calls and plain products; buffers
    are kept, so that it can be captured."""

    def __init__(self, T, B, D, E, N, K, dtype, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def n(*shape, std=1.0, dt=torch.float32):
            return (torch.randn(*shape, device="cuda", generator=g) * std).to(dt)

        self.sizes, self.dt = (T, B, D, E, N, K), dtype
        self.x, self.res, self.dy = n(T * B, D, dt=dtype), n(T * B, D, dt=dtype), n(T * B, D, dt=dtype)
        self.weight, self.w_in, self.w_bc = n(D), n(2 * E, D, std=D ** -0.5, dt=dtype), n(2 * N, E, std=E ** -0.5, dt=dtype)
        self.w_dt, self.w_out = n(E, E, std=0.1 * E ** -0.5, dt=dtype), n(D, E, std=E ** -0.5, dt=dtype)
        self.cw, self.cb, self.dtb, self.skip = n(E, K, std=0.5), n(E, std=0.1), n(E) - 3, n(E)
        self.A = -torch.rand(E, N, device="cuda", generator=g) * N
        e = lambda *s, dt=dtype: torch.empty(s, dtype=dt, device="cuda")  # noqa: E731
        f = torch.float32
        self.total, self.n, self.stats = e(T * B, D), e(T * B, D), e(T * B, 2, dt=f)
        self.xz, self.u, self.delta, self.bc = e(T, B, 2 * E), e(T, B, E), e(T, B, E), e(T, B, 2 * N)
        self.y, self.hy, self.sy = e(T, B, E), e(B, E, N, dt=f), e(K - 1, B, E)
        self.dxz, self.du, self.ddelta, self.dbc = e(T, B, 2 * E), e(T, B, E), e(T, B, E), e(T, B, 2 * N)
        self.dA, self.dD, self.ddtb, self.dcw = e(E, N, dt=f), e(E, dt=f), e(E, dt=f), e(E, K, dt=f)
        self.dcb, self.dweight, self.dx, self.out = e(E, dt=f), e(D, dt=f), e(T * B, D), e(T * B, D)
        self.wn, self.wc = room(R.rnn_norm_workspace_size(T * B, D)), room(R.rnn_conv_workspace_size(T, B, E, K))
        self.ws = room(R.rnn_ssm_workspace_size(T, B, E, N, 1, "full"))

    def run(self):
        T, B, D, E, N, K = self.sizes
        rows = T * B
        R.rnn_norm_forward("rms", self.x, self.res, self.weight, None, self.n, self.total, self.stats)
        torch.mm(self.n, self.w_in.t(), out=self.xz.view(rows, -1))
        R.rnn_conv_forward("silu", self.xz[..., :E], self.cw, self.cb, None, None, self.u, self.sy)
        u = self.u.view(rows, E)
        torch.mm(u, self.w_dt.t(), out=self.delta.view(rows, E))
        torch.mm(u, self.w_bc.t(), out=self.bc.view(rows, -1))
        args = (self.u, self.delta, self.A, self.bc[..., :N], self.bc[..., N:], self.skip, self.xz[..., E:], self.dtb)
        R.rnn_ssm_forward("softplus", *args, None, None, self.y, self.hy, self.ws, "full")
        torch.mm(self.y.view(rows, E), self.w_out.t(), out=self.out)
        dy = (self.dy @ self.w_out).view(T, B, E)
        R.rnn_ssm_backward("softplus", *args, None, None, dy, None, self.du, self.ddelta, self.dA, self.dbc[..., :N],
                           self.dbc[..., N:], self.dD, self.dxz[..., E:], self.ddtb, None, self.ws)
        du = self.du.view(rows, E) + self.ddelta.view(rows, E) @ self.w_dt + self.dbc.view(rows, -1) @ self.w_bc
        R.rnn_conv_backward("silu", self.xz[..., :E], self.cw, self.cb, None, None, du.view(T, B, E), None,
                            self.dxz[..., :E], self.dcw, self.dcb, None, self.wc)
        dn = self.dxz.view(rows, -1) @ self.w_in
        R.rnn_norm_backward("rms", self.total, self.weight, self.stats, dn, self.dy, self.dx, self.dweight, None, self.wn)
        return [self.out, self.hy, self.sy, self.total, self.dx, self.dA, self.dD, self.ddtb, self.dcw, self.dcb, self.dweight]


def test_block_gradients():
    """float32: the block's gradients against autograd of the plain formulas in float64."""
    b = Block(37, 2, 24, 40, 16, 4, torch.float32)
    got = b.run()
    T, B, D, E, N, K = b.sizes
    p = {k: getattr(b, k).double().cpu().requires_grad_(True) for k in ("x", "weight", "cw", "cb", "dtb", "skip", "A")}
    w_in, w_bc, w_dt, w_out = (getattr(b, k).double().cpu() for k in ("w_in", "w_bc", "w_dt", "w_out"))
    total = p["x"] + b.res.double().cpu()
    n = total * torch.rsqrt(total.square().mean(1, keepdim=True) + 1e-5) * p["weight"]
    xz = (n @ w_in.t()).view(T, B, -1)
    v, z = xz[..., :E], xz[..., E:]
    pad = torch.cat([torch.zeros(K - 1, B, E, dtype=torch.float64), v])
    u = torch.nn.functional.silu(p["cb"] + sum(p["cw"][:, k] * pad[k:k + T] for k in range(K)))
    d = torch.nn.functional.softplus(u @ w_dt.t() + p["dtb"])
    bc = u @ w_bc.t()
    h, ys = torch.zeros(B, E, N, dtype=torch.float64), []
    for t in range(T):
        h = torch.exp(d[t][..., None] * p["A"]) * h + (d[t] * u[t])[..., None] * bc[t][:, None, :N]
        ys.append((h * bc[t][:, None, N:]).sum(-1) + p["skip"] * u[t])
    out = (torch.stack(ys) * torch.nn.functional.silu(z)).view(T * B, E) @ w_out.t()
    dy = b.dy.double().cpu()
    grads = torch.autograd.grad((out, total), list(p.values()), (dy, dy))
    want = dict(zip(p, grads)) | {"out": out, "hy": h}
    named = dict(zip(("out", "hy", "sy", "total", "x", "A", "skip", "dtb", "cw", "cb", "weight"), got))
    for k, v in want.items():
        # sums of a few hundred terms in fp32, through six operators: 2^-24 times a few thousand
        assert (named[k].double().cpu() - v.detach()).norm() <= 2.0 ** -12 * v.detach().norm(), k


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_block_in_a_graph(dtype):
    """Captured once, replayed several times on new inputs with other work between: bitwise the eager results."""
    b = Block(300, 2, 64, 96, 16, 4, dtype)
    b.run()                                            # the library products' handles and workspaces
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = b.run()
    for seed in (1, 2, 3):
        other = Block(300, 2, 64, 96, 16, 4, dtype, seed)
        want = [t.clone() for t in other.run()]
        for k in ("x", "res", "dy"):
            getattr(b, k).copy_(getattr(other, k))
        for k in ("weight", "w_in", "w_bc", "w_dt", "w_out", "cw", "cb", "dtb", "skip", "A"):
            getattr(b, k).copy_(getattr(other, k))
        for t in outs:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for i, (got, w) in enumerate(zip(outs, want)):
            assert torch.equal(got, w), (seed, i)


def test_no_work_is_left_on_other_streams():
    """A call's results are there for work that follows on its stream."""
    c = ssm_case(500, 2, 70, 16, 1, "f32")
    want = ssm_run("softplus", c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = {k: v.clone() for k, v in ssm_run("softplus", c).items()}
    s.synchronize()
    same(got, want)


def test_misaligned_tensors():
    """Tensors that start at any element of their type."""
    for dtype in ("f32", "bf16"):
        c = ssm_case(70, 2, 21, 13, 1, dtype)
        want = ssm_want("softplus", c)
        for k in ("u", "delta", "Bm", "Cm", "z", "dy", "A", "h0", "D"):
            flat = torch.empty(c[k].numel() + 1, dtype=c[k].dtype)
            flat[1:] = c[k].reshape(-1)
            c[k] = flat                                # shifted on the device
        g = {k: gpu(v) for k, v in c.items()}
        shapes = {"u": (70, 2, 21), "delta": (70, 2, 21), "z": (70, 2, 21), "dy": (70, 2, 21), "Bm": (70, 2, 13),
                  "Cm": (70, 2, 13), "A": (21, 13), "h0": (2, 21, 13), "D": (21,)}
        for k, s in shapes.items():
            g[k] = g[k][1:].view(s)
        y = torch.empty(70 * 2 * 21 + 1, dtype=g["u"].dtype, device="cuda")[1:].view(70, 2, 21)
        hy = torch.empty(2 * 21 * 13 + 1, device="cuda")[1:].view(2, 21, 13)
        R.rnn_ssm_forward("softplus", *(g[k] for k in INPUTS), g["h0"], None, y, hy,
                          room(R.rnn_ssm_workspace_size(70, 2, 21, 13)))
        check("y", y, want["y"], dtype)
        check("hy", hy, want["hy"])
        c = conv_case(40, 2, 37, 4, dtype)
        want = conv_want("silu", c)
        x = torch.empty(40 * 2 * 37 + 1, dtype=c["x"].dtype, device="cuda")[1:].view(40, 2, 37)
        x.copy_(c["x"])
        y = torch.empty(40 * 2 * 37 + 1, dtype=x.dtype, device="cuda")[1:].view(40, 2, 37)
        R.rnn_conv_forward("silu", x, gpu(c["w"]), gpu(c["bias"]), gpu(c["s0"]), None, y, None)
        check("y", y, want["y"], dtype)


def test_binding_refuses_other_layouts_and_types():
    x, w = torch.zeros(6, 2, 8, device="cuda"), torch.zeros(8, 4, device="cuda")
    A, bc, ws = torch.zeros(8, 4, device="cuda"), torch.zeros(6, 2, 4, device="cuda"), room(1 << 16)
    apart = torch.zeros(6, 3, 8, device="cuda")[:, :2]            # rows of a step lie closer than the steps' last and first
    every = torch.zeros(6, 2, 16, device="cuda")[..., ::2]
    over = torch.zeros(19, device="cuda").as_strided((6, 2, 8), (2, 1, 1))
    half, host = x.bfloat16(), x.cpu()

    def conv(x=x, y=x, w=w):
        R.rnn_conv_forward("silu", x, w, None, None, None, y, None)

    def ssm(u=x, delta=x, Bm=bc, Cm=bc, y=x, h0=None):
        R.rnn_ssm_forward("softplus", u, delta, A, Bm, Cm, None, None, None, h0, None, y, None, ws)

    conv(y=torch.empty_like(x))
    ssm(y=torch.empty_like(x))
    for bad in (apart, every, over, x[:5], x[..., :7], half, host):
        for call in (lambda: conv(y=bad), lambda: ssm(delta=bad), lambda: ssm(y=bad)):
            with pytest.raises(ValueError):
                call()
    for bad in (w.t().contiguous().t(), w.bfloat16(), w[:7]):
        with pytest.raises(ValueError):
            conv(w=bad)
    for bad in (bc[..., :3], bc.bfloat16(), bc.cpu()):
        with pytest.raises(ValueError):
            ssm(Cm=bad)
    with pytest.raises(ValueError):
        ssm(h0=torch.zeros(2, 4, 8, device="cuda"))
    with pytest.raises(R.RNNError):
        R.rnn_ssm_forward("softplus", x, x, A, bc, bc, None, None, None, None, None, x.clone(), None, ws[1:])
    with pytest.raises(R.RNNError):
        R.rnn_ssm_forward("softplus", x, x, A, bc, bc, None, None, None, None, None, x.clone(), None, ws[:512], "full")


def test_calls_keep_their_place_on_the_stream():
    """Inputs that arrive on a stream behind a long product, calls behind them, copies of the results behind those, and
    nothing of the host between: every call waits for what comes before it and is done for what follows."""
    c, n, v = ssm_case(500, 2, 70, 16, 1, "f32", seed=4), norm_case(300, 700, "f32", seed=4), conv_case(200, 3, 300, 4, "f32", seed=4)
    want = {f"ssm.{k}": t for k, t in ssm_run("softplus", c).items()}
    want |= {f"norm.{k}": t for k, t in norm_run("layer", n).items()}
    want |= {f"conv.{k}": t for k, t in conv_run("silu", v).items()}
    sources = {f"{p}.{k}": gpu(t) for p, d in (("ssm", c), ("norm", n), ("conv", v)) for k, t in d.items() if t is not None}
    g = {k: torch.full_like(t, float("nan")) for k, t in sources.items()}
    out = {k: torch.full_like(t, 7.0) for k, t in want.items()}
    stats, big = torch.full((300, 2), 7.0, device="cuda"), torch.randn(4096, 4096, device="cuda")
    sizes = (R.rnn_ssm_workspace_size(500, 2, 70, 16, 1, "full"), R.rnn_norm_workspace_size(300, 700), R.rnn_conv_workspace_size(200, 3, 300, 4))
    ws, wn, wc = (room(s) for s in sizes)
    copies = {k: torch.empty_like(t) for k, t in want.items()}
    args = [g.get(f"ssm.{k}") for k in INPUTS]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(8):
            big @ big
        for k, t in sources.items():
            g[k].copy_(t)
        R.rnn_ssm_forward("softplus", *args, g["ssm.h0"], None, out["ssm.y"], out["ssm.hy"], ws, "full")
        R.rnn_ssm_backward("softplus", *args, g["ssm.h0"], None, g["ssm.dy"], g["ssm.dhy"],
                           *(out[f"ssm.{k}"] for k in ("du", "ddelta", "dA", "dBm", "dCm", "dD", "dz", "ddelta_bias", "dh0")), ws)
        R.rnn_norm_forward("layer", g["norm.x"], g["norm.residual"], g["norm.weight"], g["norm.bias"], out["norm.y"], out["norm.total"], stats)
        R.rnn_norm_backward("layer", out["norm.total"], g["norm.weight"], stats, g["norm.dy"], g["norm.dtotal"], out["norm.dx"],
                            out["norm.dweight"], out["norm.dbias"], wn)
        x = (g["conv.x"], g["conv.w"], g["conv.bias"], g["conv.s0"], None)
        R.rnn_conv_forward("silu", *x, out["conv.y"], out["conv.sy"])
        R.rnn_conv_backward("silu", *x, g["conv.dy"], g["conv.dsy"], *(out[f"conv.{k}"] for k in ("dx", "dw", "dbias", "ds0")), wc)
        for k, t in out.items():
            copies[k].copy_(t)
    s.synchronize()
    same(copies, want)


def test_workspaces_do_for_fewer_steps_and_rows():
    """One workspace each, sized for the longest sequences of the largest batch, for all calls of a server."""
    T, B, E, N, K = 700, 4, 90, 16, 4
    ws, wc = room(R.rnn_ssm_workspace_size(T, B, E, N, 1, "full")), room(R.rnn_conv_workspace_size(T, B, E, K))
    for t, b in ((700, 4), (545, 4), (33, 4), (65, 3), (699, 1), (1, 2), (512, 2)):
        c, v = ssm_case(t, b, E, N, 1, "f32", seed=t), conv_case(t, b, E, K, "f32", seed=t)
        want, g = ssm_run("softplus", c), {k: gpu(x) for k, x in c.items()}
        got = {k: torch.full_like(x, 7.0) for k, x in want.items()}
        args = [g[k] for k in INPUTS]
        R.rnn_ssm_forward("softplus", *args, g["h0"], None, got["y"], got["hy"], ws, "full")
        R.rnn_ssm_backward("softplus", *args, g["h0"], None, g["dy"], g["dhy"],
                           *(got[k] for k in ("du", "ddelta", "dA", "dBm", "dCm", "dD", "dz", "ddelta_bias", "dh0")), ws)
        same(got, want)
        want, g = conv_run("silu", v), {k: gpu(x) for k, x in v.items()}
        dw, db = torch.full_like(want["dw"], 7.0), torch.full_like(want["dbias"], 7.0)
        R.rnn_conv_backward("silu", g["x"], g["w"], g["bias"], g["s0"], None, g["dy"], g["dsy"], None, dw, db, None, wc)
        assert torch.equal(dw, want["dw"]) and torch.equal(db, want["dbias"])
