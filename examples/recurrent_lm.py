"""A small recurrent language model on the gated scan or the selective state-space scan, the gated feed-forward block
and 8-bit checkpoints.

    python examples/recurrent_lm.py [--steps 300] [--period 2] [--mixer scan|ssm]

Each block is  x + mixer(norm(x))  followed by  x + ffn(norm(x)); the mixer is  scan(x W_g)  or a state-space block
(projection, causal convolution, state-space scan with its gate, projection).  Training keeps the blocks' inputs and
projections in 8 bits; generation runs one token at a time on the recurrent state.  The data are sequences that repeat
a random phrase, so that the model has to remember."""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import layer_rnn_forward_amd as R  # noqa: E402


def room(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


class Scan(torch.autograd.Function):
    """y, hy = scan(x W^T, h0) over x [T, B, D]; x is kept in 8 bits, the gates as they are."""

    @staticmethod
    def forward(ctx, x, w, h0):
        T, B, D = x.shape
        H = w.shape[0] // 2
        g = (x.view(T * B, D) @ w.t()).view(T, B, 2 * H)
        y, hy = torch.empty(T, B, H, dtype=x.dtype, device="cuda"), torch.empty_like(h0)
        ctx.ws = room(R.rnn_scan_workspace_size(T, B, H, 1))
        R.rnn_scan_forward("gated", g, h0, None, y, hy, ctx.ws)
        ctx.kept = room(R.rnn_checkpoint_size(T * B, D))
        R.rnn_checkpoint_store(x.reshape(T * B, D), ctx.kept)
        ctx.save_for_backward(w, h0, g)
        return y, hy

    @staticmethod
    def backward(ctx, dy, dhy):
        w, h0, g = ctx.saved_tensors
        T, B, H2 = g.shape
        dg, dh0 = torch.empty_like(g), torch.empty_like(h0)
        R.rnn_scan_backward("gated", g, h0, None, dy.contiguous(), dhy.contiguous(), dg, dh0, ctx.ws)
        x = torch.empty(T * B, w.shape[1], dtype=g.dtype, device="cuda")
        R.rnn_checkpoint_load(ctx.kept, x)
        dg = dg.view(T * B, H2)
        return (dg @ w).view(T, B, -1), dg.t().contiguous() @ x, dh0


class FeedForward(torch.autograd.Function):
    """The gated feed-forward block over rows x [M, D], its activations kept in 8 bits."""

    @staticmethod
    def forward(ctx, x, w_in, w_out):
        M, D, F, dt = x.shape[0], x.shape[1], w_out.shape[1], "bf16" if x.dtype == torch.bfloat16 else "f32"
        y, ctx.ws = torch.empty_like(x), room(R.rnn_ffn_workspace_size(M, D, F, dt, "int8"))
        ctx.reserve = room(R.rnn_ffn_reserve_size(M, D, F, dt, "int8"))
        R.rnn_ffn_forward("silu", x, w_in, w_out, y, ctx.ws, "int8", ctx.reserve)
        ctx.save_for_backward(w_in, w_out)
        return y

    @staticmethod
    def backward(ctx, dy):
        w_in, w_out = ctx.saved_tensors
        dy = dy.contiguous()
        dx, dw_in, dw_out = torch.empty_like(dy), torch.empty_like(w_in), torch.empty_like(w_out)
        R.rnn_ffn_backward("silu", None, w_in, w_out, dy, dx, dw_in, dw_out, ctx.ws, "int8", ctx.reserve)
        return dx, dw_in, dw_out


class Norm(torch.autograd.Function):
    """Root-mean-square normalisation of rows."""

    @staticmethod
    def forward(ctx, x):
        rows = x.contiguous().view(-1, x.shape[-1])
        y, stats = torch.empty_like(rows), torch.empty(rows.shape[0], 2, device="cuda")
        R.rnn_norm_forward("rms", rows, None, None, None, y, None, stats, 1e-6)
        ctx.save_for_backward(rows, stats)
        return y.view(x.shape)

    @staticmethod
    def backward(ctx, dy):
        rows, stats = ctx.saved_tensors
        dx = torch.empty_like(rows)
        R.rnn_norm_backward("rms", rows, None, stats, dy.contiguous().view(rows.shape), None, dx, None, None)
        return dx.view(dy.shape)


norm = Norm.apply


class Conv(torch.autograd.Function):
    """y, sy = silu(causal convolution of x [T, B, C] that goes on from s0)."""

    @staticmethod
    def forward(ctx, x, w, bias, s0):
        y, sy = torch.empty(x.shape, dtype=x.dtype, device="cuda"), torch.empty_like(s0)
        R.rnn_conv_forward("silu", x, w, bias, s0, None, y, sy)
        ctx.save_for_backward(x, w, bias, s0)
        return y, sy

    @staticmethod
    def backward(ctx, dy, dsy):
        x, w, bias, s0 = ctx.saved_tensors
        dx, dw, db, ds0 = torch.empty_like(dy), torch.empty_like(w), torch.empty_like(bias), torch.empty_like(s0)
        ws = room(R.rnn_conv_workspace_size(*x.shape, w.shape[1]))
        R.rnn_conv_backward("silu", x, w, bias, s0, None, dy.contiguous(), dsy.contiguous(), dx, dw, db, ds0, ws)
        return dx, dw, db, ds0


class StateSpace(torch.autograd.Function):
    """y, hy of the selective state-space scan over u, delta, z [T, B, E], Bm and Cm [T, B, N]."""

    @staticmethod
    def forward(ctx, u, delta, A, Bm, Cm, D, z, delta_bias, h0):
        y, hy = torch.empty_like(u), torch.empty_like(h0)
        ctx.ws = room(R.rnn_ssm_workspace_size(*u.shape, A.shape[1], 1, "full"))
        R.rnn_ssm_forward("softplus", u, delta, A, Bm, Cm, D, z, delta_bias, h0, None, y, hy, ctx.ws, "full")
        ctx.save_for_backward(u, delta, A, Bm, Cm, D, z, delta_bias, h0)
        return y, hy

    @staticmethod
    def backward(ctx, dy, dhy):
        saved = ctx.saved_tensors
        grads = [torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in saved]
        R.rnn_ssm_backward("softplus", *saved, None, dy.contiguous(), dhy.contiguous(), *grads, ctx.ws)
        return tuple(grads)


class Model(torch.nn.Module):
    """mixer "ssm": blocks of 2 * width channels with `state` states each, a convolution over `taps` steps."""

    def __init__(self, vocab=64, width=256, hidden=512, blocks=2, dtype=torch.bfloat16, mixer="scan", state=16, taps=4):
        super().__init__()
        self.width, self.blocks, self.dtype, self.mixer, self.state, self.taps = width, blocks, dtype, mixer, state, taps

        def weight(rows, cols):
            return torch.nn.Parameter(torch.randn(rows, cols, device="cuda") * cols ** -0.5)

        self.embed = torch.nn.Parameter(torch.randn(vocab, width, device="cuda"))
        if mixer == "scan":
            self.gates = torch.nn.ParameterList(weight(2 * width, width) for _ in range(blocks))
        else:
            E, rank = 2 * width, max(1, width // 16)
            self.rank = rank
            self.w_xz = torch.nn.ParameterList(weight(2 * E, width) for _ in range(blocks))
            self.taps_w = torch.nn.ParameterList(weight(E, taps) for _ in range(blocks))
            self.taps_b = torch.nn.ParameterList(torch.zeros(E, device="cuda") for _ in range(blocks))
            self.w_dbc = torch.nn.ParameterList(weight(rank + 2 * state, E) for _ in range(blocks))
            self.w_delta = torch.nn.ParameterList(weight(E, rank) for _ in range(blocks))
            # softplus of it: steps between 0.001 and 0.1
            self.delta_b = torch.nn.ParameterList(torch.log(torch.expm1(10 ** torch.linspace(-3, -1, E, device="cuda")))
                                                  for _ in range(blocks))
            self.A_log = torch.nn.ParameterList(torch.arange(1.0, state + 1, device="cuda").log().repeat(E, 1)
                                                for _ in range(blocks))
            self.skip = torch.nn.ParameterList(torch.ones(E, device="cuda") for _ in range(blocks))
            self.w_mix = torch.nn.ParameterList(weight(width, E) for _ in range(blocks))
        self.w_in = torch.nn.ParameterList(weight(2 * hidden, width) for _ in range(blocks))
        self.w_out = torch.nn.ParameterList(weight(width, hidden) for _ in range(blocks))
        self.head = weight(vocab, width)

    def states(self, B):
        if self.mixer == "scan":
            return [torch.zeros(1, B, self.width, device="cuda") for _ in range(self.blocks)]
        E = 2 * self.width
        return [(torch.zeros(self.taps - 1, B, E, dtype=self.dtype, device="cuda"),
                 torch.zeros(B, E, self.state, device="cuda")) for _ in range(self.blocks)]

    def mix(self, i, x, state):
        """The i-th block's mixer over x [T, B, width]: y, state."""
        if self.mixer == "scan":
            return Scan.apply(x, self.gates[i].to(self.dtype), state)
        def times(v, w):
            return (v.reshape(-1, v.shape[-1]) @ w.to(self.dtype).t()).view(*v.shape[:-1], -1)
        E, N = 2 * self.width, self.state
        xz = times(x, self.w_xz[i])
        u, sy = Conv.apply(xz[..., :E], self.taps_w[i], self.taps_b[i], state[0])
        dbc = times(u, self.w_dbc[i])
        delta, Bm, Cm = dbc.split((self.rank, N, N), -1)
        y, hy = StateSpace.apply(u, times(delta, self.w_delta[i]), -self.A_log[i].exp(), Bm, Cm, self.skip[i], xz[..., E:],
                                 self.delta_b[i], state[1])
        return times(y, self.w_mix[i]), (sy, hy)

    def mix_step(self, i, x, state):
        """One token a row: x [B, width] -> y; the state is updated in place."""
        def times(v, w):
            return v @ w.to(self.dtype).t()
        if self.mixer == "scan":
            y = torch.empty_like(x)
            R.rnn_scan_step("gated", times(x, self.gates[i]), state[0], y, state[0])
            return y
        E, N = 2 * self.width, self.state
        xz = times(x, self.w_xz[i])
        u = torch.empty(x.shape[0], E, dtype=self.dtype, device="cuda")
        R.rnn_conv_step("silu", xz[:, :E], self.taps_w[i], self.taps_b[i], state[0], u, state[0])
        dbc = times(u, self.w_dbc[i])
        delta, Bm, Cm = dbc.split((self.rank, N, N), -1)
        y = torch.empty_like(u)
        R.rnn_ssm_step("softplus", u, times(delta, self.w_delta[i]), -self.A_log[i].exp(), Bm, Cm, self.skip[i], xz[:, E:],
                       self.delta_b[i], state[1], y, state[1])
        return times(y, self.w_mix[i])

    def forward(self, tokens, states):
        """tokens [T, B] -> logits [T, B, vocab] in float32, states."""
        T, B = tokens.shape
        x, out = self.embed[tokens].to(self.dtype), []
        for i in range(self.blocks):
            y, state = self.mix(i, norm(x), states[i])
            x = x + y
            f = FeedForward.apply(norm(x).view(T * B, -1), self.w_in[i].to(self.dtype), self.w_out[i].to(self.dtype))
            x = x + f.view(T, B, -1)
            out.append(state)
        return norm(x).float() @ self.head.t(), out

    @torch.no_grad()
    def step(self, tokens, states, ws):
        """One token a row: tokens [B] -> logits [B, vocab]; states are updated in place."""
        x = self.embed[tokens].to(self.dtype)
        for i in range(self.blocks):
            x = x + self.mix_step(i, norm(x), states[i])
            f = torch.empty_like(x)
            R.rnn_ffn_forward("silu", norm(x), self.w_in[i].to(self.dtype), self.w_out[i].to(self.dtype), f, ws)
            x = x + f
        return norm(x).float() @ self.head.t()


def phrases(T, B, vocab, period, gen):
    p = torch.randint(0, vocab, (period, B), device="cuda", generator=gen)
    return p.repeat(-(-T // period), 1)[:T]


def train(model, steps, T=96, B=16, period=1, lr=3e-3, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    opt = torch.optim.Adam(model.parameters(), lr=lr)
    vocab, losses = model.embed.shape[0], []
    for _ in range(steps):
        tokens = phrases(T + 1, B, vocab, period, gen)
        logits, _ = model(tokens[:-1], model.states(B))
        loss = torch.nn.functional.cross_entropy(logits.reshape(-1, vocab), tokens[1:].reshape(-1))
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


@torch.no_grad()
def generate(model, prompt, count):
    """prompt [T, B] -> the `count` tokens that follow, greedily."""
    B = prompt.shape[1]
    logits, states = model(prompt, model.states(B))
    dt = "bf16" if model.dtype == torch.bfloat16 else "f32"
    ws = room(R.rnn_ffn_workspace_size(B, model.width, model.w_out[0].shape[1], dt))
    token, out = logits[-1].argmax(-1), []
    for _ in range(count):
        out.append(token)
        token = model.step(token, states, ws).argmax(-1)
    return torch.stack(out)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=300)
    ap.add_argument("--period", type=int, default=2, help="length of the phrases")
    ap.add_argument("--mixer", choices=("scan", "ssm"), default="scan")
    args = ap.parse_args()
    torch.manual_seed(0)
    model = Model(mixer=args.mixer)
    losses = train(model, args.steps, period=args.period)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} over {args.steps} steps")
    prompt = phrases(24, 4, 64, args.period, torch.Generator(device="cuda").manual_seed(7))
    said = generate(model, prompt, 12)
    right = (said == prompt[:12]).float().mean().item()
    print(f"generated {said.shape[0]} tokens a row, {100 * right:.0f} % as the phrase goes on")


if __name__ == "__main__":
    main()
