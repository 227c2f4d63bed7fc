"""The example that trains and serves a model from the operators around the scan.

Served token by token or in one pass, the same prompt gives the same logits but for the order of fp32 sums: such a
difference moves a bfloat16 value by at most a step (2^-8) and about one in 2^5 of the e4m3 values made from
bfloat16 ones that are a step off by a step of theirs (2^-3). That is 2^-3 2^-2.5 = 2^-5.5 of the norm for an
operand all of whose values are a step off, which adds to the sum of squares for each of the 2 x layers + 1
products: sqrt(5) 2^-5.5 = 0.05 for two layers."""
import importlib.util
import os

import pytest
import torch

from state_space_sequence_complex_gb300 import block

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("gated_block", os.path.join(ROOT, "examples", "gated_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_pattern_on_the_cpu():
    tokens, first = example().pattern(257, 3, 50, device="cpu")
    assert tokens.shape == first.shape == (3, 50) and first.dtype == torch.uint8
    assert torch.equal(first[0].nonzero().flatten(), torch.tensor([0, 21, 42]))
    assert torch.equal(tokens[:, 7:], tokens[:, :-7]) and int(tokens.max()) < 257


@pytest.mark.gpu
def test_trains_and_continues():
    losses, right = example().main(["--steps", "60"])
    assert losses[-1] < 0.5 * losses[0]
    assert right > 0.5


@pytest.mark.gpu
@pytest.mark.parametrize("B,T,more", [(3, 70, 5), (1, 1, 3), (2, 200, 2)])
def test_tokens_follow_the_whole_pass(B, T, more):
    ex = example()
    model = ex.Model(vocab=301, width=192, channels=136, layers=2, seed=4)
    weights = ex.Weights8(model)
    prompt = torch.randint(0, 301, (B, T), generator=torch.Generator().manual_seed(1)).cuda()
    said, logits = ex.generate(model, prompt, more, weights)
    assert said.shape == (B, more) and logits.shape == (B, more, 301)
    whole = ex.Pass(model, weights, B, T + more - 1)
    whole.tokens.copy_(torch.cat([prompt, said[:, :-1]], 1).flatten())
    with torch.no_grad():
        want = whole()[:, T - 1:]
    e = float((logits.double() - want.double()).norm() / want.double().norm())
    assert e <= 0.05, e
    for s in whole.scans:
        assert not hasattr(s, "status") or s.status() == 0
    assert all(p.status() == 0 for p in (*whole.to_in, *whole.to_out, whole.to_logits))
