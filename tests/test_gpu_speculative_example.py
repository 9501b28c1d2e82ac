"""The operators of a decoding step together, as examples/speculative_decoding.py
uses them: at temperature 0 every token is the most likely one after what came
before it, as one pass over the whole sequence sees it, and the cache holds
what it should.

Tolerance, derived: a logit is a sum over activations that are rounded to BF16
about 20 times on the way (3 layers, some 6 roundings each, relative 2^-9,
independent): relative 2^-9 sqrt(20) < 0.01 of the logits' spread, 3 -- 0.03; two
passes differ by sqrt(2) of that, and 0.3 is 7 of those. A token read from a
wrong cache row would be some 3 spreads (about 9) below the best."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import speculative_decoding
    return speculative_decoding


@pytest.fixture(scope="module")
def model(ex):
    return ex.Model()


def prompt_of(model, n):
    return torch.randint(0, model.vocab, (2, n), dtype=torch.int32, generator=torch.Generator().manual_seed(n)).cuda()


@pytest.mark.parametrize("speculate", [False, True])
@pytest.mark.parametrize("n", [2, 40, 200])
def test_greedy_tokens_are_the_most_likely(ex, model, n, speculate):
    print("[gpu-case] speculative greedy", n, speculate, flush=True)
    prompt = prompt_of(model, n)
    decoder = ex.Decoder(model, 2, temperature=0.0)
    out, steps = ex.generate(decoder, prompt, 48, speculate=speculate)
    assert steps == 48 if not speculate else steps < 40
    assert int(decoder.cache.status) == 0
    whole = torch.cat([prompt, torch.tensor(out, dtype=torch.int32, device="cuda")], 1)
    order = torch.arange(whole.shape[1], dtype=torch.int32, device="cuda").repeat(2, 1)
    logits, _ = ex.Decoder(model, 2).forward(whole, order, None, model.layers)      # an empty cache: one chain
    after = logits[:, n - 1:-1]
    got = after.gather(2, whole[:, n:, None].long())[..., 0]
    assert (got >= after.amax(-1) - 0.3).all()


def test_cache_after_sampling(ex, model):
    """Pages, counts and lengths after steps whose trees were partly accepted."""
    print("[gpu-case] speculative sampling", flush=True)
    decoder = ex.Decoder(model, 2, temperature=1.0)
    pending = decoder.prefill(prompt_of(model, 33))
    total = torch.full((2,), 32, dtype=torch.int32)
    for _ in range(12):
        pending, _, count = decoder.step(pending)
        total += count.cpu()
        assert ((pending >= 0) & (pending < model.vocab)).all()
    c = decoder.cache
    assert c.lens.cpu().tolist() == total.tolist() and int(c.status) == 0
    held = c.table[c.table >= 0]
    assert held.numel() == int(((total + 15) // 16).sum()) == int(c.refs.sum()) and held.unique().numel() == held.numel()
