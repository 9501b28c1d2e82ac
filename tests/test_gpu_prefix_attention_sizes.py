"""enc_prefix_attention without groups, and calls of many sizes in one workspace,
against the formula in 64 bits (tolerances: test_gpu_prefix_attention.py)."""
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_prefix_attention import Case  # noqa: E402
from test_gpu_prefix_attention_scores import SHAPES  # noqa: E402

BF, FP = torch.bfloat16, torch.float16


def say(*a):
    print("[gpu-case]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def E():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from lossless_weight_compression_amd import enc
    enc.lib()
    return enc


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_no_groups(E, shape, dt):
    """Nothing is shared: the same results from every sequence's own rows."""
    say("prefix without groups", shape, dt)
    Case(*SHAPES[shape], dt, seed=61).check(E, starts=[0], shared=[])


def test_no_groups_prompt(E):
    """A prompt's nodes, all heads of 64 and of 256, behind a long history."""
    say("prefix without groups, prompt")
    for D, T in ((64, 17), (64, 200), (256, 100)):
        Case([(0, [700]), (0, [33])], T, 4, 2, D, 16, seed=62).check(E, mask=False, starts=[0], shared=[])
