"""examples/hybrid_decoder.py: the layers together, as a decoder and in training."""
import importlib.util
import os

import pytest
import torch

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
