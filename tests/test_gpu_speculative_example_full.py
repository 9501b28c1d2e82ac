"""examples/speculative_decoding.py when its cache is full: an error, not tokens
decoded without the rows that did not fit."""
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


@pytest.mark.parametrize("speculate", [False, True])
def test_a_full_cache_is_an_error(ex, speculate):
    print("[gpu-case] speculative, full cache", speculate, flush=True)
    model = ex.Model(layers=2)
    prompt = torch.zeros(2, 40, dtype=torch.int32, device="cuda")
    decoder = ex.Decoder(model, 2, max_len=64)
    with pytest.raises(RuntimeError):
        ex.generate(decoder, prompt, 48, speculate=speculate)
    with pytest.raises(RuntimeError):
        ex.Decoder(model, 2, max_len=32).prefill(prompt)
