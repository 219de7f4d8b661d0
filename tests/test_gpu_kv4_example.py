"""The parallel-sampling example runs, and its samples share their prompts' pages."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("bits", [4, 8])
def test_samples_share_pages(bits):
    import parallel_sampling as example

    prompts, samples, tokens, page = [list(range(5, 75)), list(range(100, 149)), [7] * 32], 4, 20, 16
    s = example.Sampler(prompts, samples, tokens, bits=bits, page=page)
    text = s.run(tokens)
    assert text.shape == (12, tokens + 1) and int(text.min()) >= 0 and int(text.max()) < s.vocab
    lengths = [len(p) + tokens for p in prompts for _ in range(samples)]
    assert s.lengths.tolist() == lengths
    assert s.pool.held.tolist() == [-(-n // page) for n in lengths]
    # a prompt's whole pages once; of each sample the others
    want = sum(len(p) // page for p in prompts) + sum(-(-n // page) for n in lengths) - samples * sum(len(p) // page for p in prompts)
    assert int((s.pool.refs > 0).sum()) == want
    refs = s.pool.refs.new_zeros(s.pool.pages)
    for b in range(12):
        refs[s.pool.table[b, :int(s.pool.held[b])].long()] += 1
    assert (refs == s.pool.refs).all()
