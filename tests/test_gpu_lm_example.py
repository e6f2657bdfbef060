"""The example language model: gradients against a plain model's in float64, a loss that falls, and generation by
single tokens that follows the scan."""

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

    def norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    x = p["embed"][tokens]
    for i in range(model.blocks):
        a, q = (norm(x) @ p[f"gates.{i}"].t()).chunk(2, -1)
        a, n = torch.sigmoid(a), torch.tanh(q)
        h, ys = torch.zeros(B, model.width, dtype=torch.float64), []
        for t in range(T):
            h = a[t] * h + (1 - a[t]) * n[t]
            ys.append(h)
        x = x + torch.stack(ys)
        g, u = (norm(x) @ p[f"w_in.{i}"].t()).chunk(2, -1)
        x = x + (torch.nn.functional.silu(g) * u) @ p[f"w_out.{i}"].t()
    return norm(x) @ p["head"].t(), p


def test_gradients_are_the_models(lm):
    """float32: what is left is the rounding to 8 bits of the kept activations (of groups of 32 values, 2^-7 of the
    largest; a gradient is a sum over many of them with independent errors, so 2^-6 of its norm bounds it)."""
    torch.manual_seed(1)
    model = lm.Model(vocab=20, width=64, hidden=96, dtype=torch.float32)
    tokens = torch.randint(0, 20, (33, 3), device="cuda")
    logits, _ = model(tokens[:-1], model.states(3))
    loss = torch.nn.functional.cross_entropy(logits.reshape(-1, 20), tokens[1:].reshape(-1))
    loss.backward()
    want, p = plain(model, tokens[:-1])
    assert (logits.double().cpu() - want).norm() <= 1e-5 * want.norm()
    ref = torch.nn.functional.cross_entropy(want.reshape(-1, 20), tokens[1:].reshape(-1).cpu())
    ref.backward()
    for k, v in model.named_parameters():
        got = v.grad.double().cpu()
        assert (got - p[k].grad).norm() <= 2.0 ** -6 * p[k].grad.norm(), k


def test_it_learns_and_generates(lm):
    torch.manual_seed(0)
    model = lm.Model(vocab=16, width=128, hidden=256)
    losses = lm.train(model, 60, T=40, B=8)
    assert losses[-1] < 0.5 * losses[0]
    prompt = lm.phrases(12, 8, 16, 1, torch.Generator(device="cuda").manual_seed(3))
    assert (lm.generate(model, prompt, 6) == prompt[:6]).float().mean() > 0.9


def test_steps_follow_the_scan(lm):
    """float32: logits of a prompt's last tokens by single steps are those of the whole sequence."""
    torch.manual_seed(2)
    model = lm.Model(vocab=20, width=64, hidden=96, dtype=torch.float32)
    tokens = torch.randint(0, 20, (50, 3), device="cuda")
    with torch.no_grad():
        whole, _ = model(tokens, model.states(3))
        _, states = model(tokens[:44], model.states(3))
        ws = lm.room(lm.R.rnn_ffn_workspace_size(3, 64, 96, "f32"))
        for t in range(44, 50):
            got = model.step(tokens[t], states, ws)
            assert (got - whole[t]).abs().max() <= 1e-4 * whole[t].abs().max()
