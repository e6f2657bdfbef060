"""A small recurrent language model on the gated scan, the gated feed-forward block and 8-bit checkpoints.

    python examples/recurrent_lm.py [--steps 300] [--period 2]

Each block is  x + scan(x W_g)  followed by  x + ffn(x).  Training keeps the blocks' inputs and projections in
8 bits; generation runs one token at a time on the recurrent state.  The data are sequences that repeat a random
phrase, so that the model has to remember."""

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


def norm(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class Model(torch.nn.Module):
    def __init__(self, vocab=64, width=256, hidden=512, blocks=2, dtype=torch.bfloat16):
        super().__init__()
        self.width, self.blocks, self.dtype = width, blocks, dtype

        def weight(rows, cols):
            return torch.nn.Parameter(torch.randn(rows, cols, device="cuda") * cols ** -0.5)

        self.embed = torch.nn.Parameter(torch.randn(vocab, width, device="cuda"))
        self.gates = torch.nn.ParameterList(weight(2 * width, width) for _ in range(blocks))
        self.w_in = torch.nn.ParameterList(weight(2 * hidden, width) for _ in range(blocks))
        self.w_out = torch.nn.ParameterList(weight(width, hidden) for _ in range(blocks))
        self.head = weight(vocab, width)

    def states(self, B):
        return [torch.zeros(1, B, self.width, device="cuda") for _ in range(self.blocks)]

    def forward(self, tokens, states):
        """tokens [T, B] -> logits [T, B, vocab] in float32, states."""
        T, B = tokens.shape
        x, out = self.embed[tokens].to(self.dtype), []
        for i in range(self.blocks):
            y, hy = Scan.apply(norm(x), self.gates[i].to(self.dtype), states[i])
            x = x + y
            f = FeedForward.apply(norm(x).view(T * B, -1), self.w_in[i].to(self.dtype), self.w_out[i].to(self.dtype))
            x = x + f.view(T, B, -1)
            out.append(hy)
        return norm(x).float() @ self.head.t(), out

    @torch.no_grad()
    def step(self, tokens, states, ws):
        """One token a row: tokens [B] -> logits [B, vocab]; states are updated in place."""
        x = self.embed[tokens].to(self.dtype)
        for i in range(self.blocks):
            g, y = norm(x) @ self.gates[i].to(self.dtype).t(), torch.empty_like(x)
            R.rnn_scan_step("gated", g, states[i][0], y, states[i][0])
            x = x + y
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
    args = ap.parse_args()
    torch.manual_seed(0)
    model = Model()
    losses = train(model, args.steps, period=args.period)
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} over {args.steps} steps")
    prompt = phrases(24, 4, 64, args.period, torch.Generator(device="cuda").manual_seed(7))
    said = generate(model, prompt, 12)
    right = (said == prompt[:12]).float().mean().item()
    print(f"generated {said.shape[0]} tokens a row, {100 * right:.0f} % as the phrase goes on")


if __name__ == "__main__":
    main()
