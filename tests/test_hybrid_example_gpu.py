"""examples/hybrid_decoder.py: the layers together, as a decoder and in training."""
import importlib.util
import os

import pytest
import torch
import torch.nn.functional as nnf

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "hybrid_decoder", os.path.join(ROOT, "examples", "hybrid_decoder.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("batch,prompt,steps", [(1, 1, 5), (3, 70, 9), (2, 130, 4)])
def test_decoding_equals_a_prefill_of_the_same_tokens(example, batch, prompt, steps):
    """Logits of the decode steps against one pass over prompt and generated tokens. Between
    the two, activations round to bf16 (2^-8) in a dozen places of three layers: 3e-2 of
    the logits' size covers twice their square-root sum."""
    dev = torch.device("cuda:0")
    model = example.HybridDecoder(dev)
    gen = torch.Generator().manual_seed(prompt)
    tokens = torch.randint(0, example.VOCAB, (batch, prompt), generator=gen).to(dev)
    out, logits = model.generate(tokens, steps)
    whole = torch.cat([tokens, out[:, :-1]], 1)
    again = model.forward(whole, example.Cache(batch, whole.shape[1], dev))[:, prompt - 1:]
    rms = again.float().pow(2).mean().sqrt()
    assert torch.isfinite(logits).all()
    assert (logits.float() - again.float()).pow(2).mean().sqrt() <= 3e-2 * rms


def test_training_lowers_the_loss(example):
    losses = example.train(torch.device("cuda:0"))
    assert losses[-1] < 0.8 * losses[0]


@pytest.mark.parametrize("batch,prompt,tail,steps", [(1, 16, 1, 4), (5, 70, 9, 6), (3, 15, 30, 3),
                                                     (2, 200, 1, 4)])
def test_shared_prompt_equals_whole_sequences(example, batch, prompt, tail, steps):
    """Logits behind one prompt against a prefill of every whole sequence by itself. Between the
    two, activations round to bf16 (2^-8) in a dozen places of three layers: 3e-2 of the logits'
    size covers twice their square-root sum."""
    dev = torch.device("cuda:0")
    model = example.NormedDecoder(dev)
    gen = torch.Generator().manual_seed(prompt)
    first = torch.randint(0, example.VOCAB, (prompt,), generator=gen).to(dev)
    tails = torch.randint(0, example.VOCAB, (batch, tail), generator=gen).to(dev)
    out, logits = model.generate_shared(first, tails, steps)
    whole = torch.cat([first.expand(batch, -1), tails, out[:, :-1]], 1)
    cache = example.Cache(batch, whole.shape[1], dev)
    again = model.forward(whole, cache)[:, prompt + tail - 1:]
    rms = again.float().pow(2).mean().sqrt()
    assert torch.isfinite(logits).all()
    assert (logits.float() - again.float()).pow(2).mean().sqrt() <= 3e-2 * rms


def test_gradients_through_gate_norms_and_scan(example):
    """A recurrent layer with its gate, between two residual norms, trained in 32 bits: every
    gradient against the same formulas in 64 bits. Each operator's results are within 1e-5 of
    the sizes that make them up (2e-5 the scan's); through five of them, and products of 64
    terms, 5e-4 of a gradient's largest value is used."""
    dev, B, T, H, D = torch.device("cuda:0"), 2, 70, 4, 16
    W = H * D
    gen = torch.Generator().manual_seed(5)

    def leaf(*shape, size=1.0):
        return (torch.randn(*shape, generator=gen) * size).to(dev).requires_grad_(True)

    x, y = leaf(B, T, W), leaf(B, T, W)
    w_in, w_out = leaf(W, 3 * W, size=W ** -0.5), leaf(W, W, size=W ** -0.5)
    vectors = [(1 + 0.2 * torch.randn(n, generator=gen)).to(dev).requires_grad_(True)
               for n in (W, W, D, W, W)]
    leaves = [x, y, w_in, w_out, *vectors]
    target = torch.randn(B, T, W, generator=gen).to(dev)

    def run(residual, y, w_in, w_out, w1, s1, wg, w2, s2, join, scan, gated):
        out, residual = join(residual, y, w1, s1)
        value, decay, gate = (out @ w_in).chunk(3, -1)
        h = scan(value, nnf.logsigmoid(decay + 2.0))
        h = gated(h.unflatten(-1, (H, D)), gate.unflatten(-1, (H, D)), wg).flatten(-2)
        out, residual = join(residual, h @ w_out, w2, s2)
        return ((out * target.to(out.dtype)).sum() + (residual ** 2).sum()) / out.numel()

    def norm(t):
        return t / torch.sqrt(t.pow(2).mean(-1, keepdim=True) + 1e-6)

    def plain_scan(value, g):
        a, state, out = g.exp(), 0, []
        for t in range(T):
            state = a[:, t] * state + (1 - a[:, t]) * value[:, t]
            out.append(state)
        return torch.stack(out, 1)

    def plain_join(r, y, w, s):
        r = r + s * y
        return norm(r) * w, r

    loss = run(*leaves, example.ResidualNorm.apply, example.LinearScan.apply,
               example.GatedNorm.apply)
    got = torch.autograd.grad(loss, leaves)
    exact = [t.detach().double().requires_grad_(True) for t in leaves]
    want = torch.autograd.grad(
        run(*exact, plain_join, plain_scan, lambda o, z, w: norm(o) * w * nnf.silu(z)), exact)
    for g, e in zip(got, want):
        assert (g.double() - e).abs().max() <= 5e-4 * e.abs().max()


@pytest.mark.parametrize("prompt", [1, 16, 32, 33, 47])
def test_several_continuations_of_one_prompt(example, prompt):
    """No tails: every sequence begins with the prompt's own next token, whole pages or not.
    The bound as above."""
    dev, batch, steps = torch.device("cuda:0"), 3, 4
    model = example.NormedDecoder(dev)
    gen = torch.Generator().manual_seed(prompt)
    first = torch.randint(0, example.VOCAB, (prompt,), generator=gen).to(dev)
    tails = torch.empty(batch, 0, dtype=torch.long, device=dev)
    out, logits = model.generate_shared(first, tails, steps)
    assert out.shape == (batch, steps) and logits.shape == (batch, steps, example.VOCAB)
    whole = torch.cat([first.expand(batch, -1), out[:, :-1]], 1)
    again = model.forward(whole, example.Cache(batch, whole.shape[1], dev))[:, prompt - 1:]
    rms = again.float().pow(2).mean().sqrt()
    assert torch.isfinite(logits).all()
    assert (logits.float() - again.float()).pow(2).mean().sqrt() <= 3e-2 * rms
    with pytest.raises(ValueError, match="nothing to continue"):
        model.generate_shared(first[:0], tails, steps)
