"""The cache, the tree attention and the verification together: examples/speculative_decode.py."""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "speculative_decode.py")
    spec = importlib.util.spec_from_file_location("speculative_decode", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def decode(example, model, prompts, parents, temperature=0.0, tokens=40):
    out, steps, _ = example.Decoder(model, prompts, tokens, parents, temperature).run(tokens)
    for text, prompt in zip(out, prompts):
        assert text[:len(prompt)] == list(prompt)
        assert all(0 <= t < model.vocab for t in text)
    return [text[len(prompt):] for text, prompt in zip(out, prompts)], steps


@pytest.mark.parametrize("lengths", [[5], [1, 77, 16, 130]])
def test_trees_give_the_tokens_of_single_steps(example, lengths):
    rng = np.random.default_rng(len(lengths))
    model = example.Model()
    prompts = [rng.integers(0, model.vocab, size=n) for n in lengths]
    alone, steps_alone = decode(example, model, prompts, example.CHAIN)
    trees, steps_trees = decode(example, model, prompts, example.TREE)
    assert steps_trees < steps_alone  # drafts are accepted
    for a, t in zip(alone, trees):
        n = min(len(a), len(t))
        assert n >= 2 and a[:n] == t[:n]


def test_sampled_decoding_runs(example):
    rng = np.random.default_rng(9)
    model = example.Model()
    prompts = [rng.integers(0, model.vocab, size=n) for n in (20, 3)]
    _, steps = decode(example, model, prompts, example.TREE, temperature=0.7)
    assert steps > 0
