"""The example language model with state-space blocks: gradients against a plain model's in float64, and generation by
single tokens that follows the whole sequence."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "recurrent_lm.py")


@pytest.fixture(scope="module")
def lm():
    spec = importlib.util.spec_from_file_location("recurrent_lm", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def plain(model, tokens):
    """The same model from elementary operations in float64 on the host, without 8-bit rounding."""
    p = {k: v.detach().double().cpu().requires_grad_(True) for k, v in model.named_parameters()}
    tokens = tokens.cpu()
    T, B = tokens.shape
    E, N, K = 2 * model.width, model.state, model.taps
    silu = torch.nn.functional.silu

    def norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    x = p["embed"][tokens]
    for i in range(model.blocks):
        v, z = (norm(x) @ p[f"w_xz.{i}"].t()).chunk(2, -1)
        padded = torch.cat([torch.zeros(K - 1, B, E, dtype=torch.float64), v])
        u = silu(p[f"taps_b.{i}"] + sum(p[f"taps_w.{i}"][:, k] * padded[k:k + T] for k in range(K)))
        delta, Bm, Cm = (u @ p[f"w_dbc.{i}"].t()).split((model.rank, N, N), -1)
        d = torch.nn.functional.softplus(delta @ p[f"w_delta.{i}"].t() + p[f"delta_b.{i}"])
        A, h, ys = -p[f"A_log.{i}"].exp(), torch.zeros(B, E, N, dtype=torch.float64), []
        for t in range(T):
            h = torch.exp(d[t][..., None] * A) * h + (d[t] * u[t])[..., None] * Bm[t][:, None]
            ys.append((h * Cm[t][:, None]).sum(-1) + p[f"skip.{i}"] * u[t])
        x = x + (torch.stack(ys) * silu(z)) @ p[f"w_mix.{i}"].t()
        g, up = (norm(x) @ p[f"w_in.{i}"].t()).chunk(2, -1)
        x = x + (silu(g) * up) @ p[f"w_out.{i}"].t()
    return norm(x) @ p["head"].t(), p


def test_gradients_are_the_models(lm):
    """float32: what is left is the rounding to 8 bits of the feed-forward blocks' kept activations (2^-7 of a group's
    largest; 2^-6 of a gradient's norm bounds it, as for the model with scans)."""
    torch.manual_seed(1)
    model = lm.Model(vocab=20, width=64, hidden=96, dtype=torch.float32, mixer="ssm", state=8)
    tokens = torch.randint(0, 20, (73, 3), device="cuda")
    logits, _ = model(tokens[:-1], model.states(3))
    loss = torch.nn.functional.cross_entropy(logits.reshape(-1, 20), tokens[1:].reshape(-1))
    loss.backward()
    want, p = plain(model, tokens[:-1])
    assert (logits.double().cpu() - want).norm() <= 1e-5 * want.norm()
    ref = torch.nn.functional.cross_entropy(want.reshape(-1, 20), tokens[1:].reshape(-1).cpu())
    ref.backward()
    for k, v in model.named_parameters():
        assert (v.grad.double().cpu() - p[k].grad).norm() <= 2.0 ** -6 * p[k].grad.norm(), k


def test_it_trains_and_generates(lm):
    """Runs in bf16: finite losses, and tokens of the vocabulary."""
    torch.manual_seed(0)
    model = lm.Model(vocab=16, width=128, hidden=256, mixer="ssm")
    losses = lm.train(model, 4, T=70, B=8)
    assert torch.tensor(losses).isfinite().all()
    said = lm.generate(model, lm.phrases(12, 8, 16, 1, torch.Generator(device="cuda").manual_seed(3)), 6)
    assert said.shape == (6, 8) and ((said >= 0) & (said < 16)).all()


def test_steps_follow_the_sequence(lm):
    """float32: logits of a prompt's last tokens by single steps are those of the whole sequence."""
    torch.manual_seed(2)
    model = lm.Model(vocab=20, width=64, hidden=96, dtype=torch.float32, mixer="ssm")
    tokens = torch.randint(0, 20, (90, 3), device="cuda")
    with torch.no_grad():
        whole, _ = model(tokens, model.states(3))
        _, states = model(tokens[:84], model.states(3))
        ws = lm.room(lm.R.rnn_ffn_workspace_size(3, 64, 96, "f32"))
        for t in range(84, 90):
            got = model.step(tokens[t], states, ws)
            assert (got - whole[t]).abs().max() <= 1e-4 * whole[t].abs().max()
