"""enc_cache_commit given counts that no call left behind."""
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_cache_pages import Both, i32  # noqa: E402


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


@pytest.mark.parametrize("refs", [0, -1])
def test_a_held_page_that_counts_as_free_is_refused(E, refs):
    """Its rows would be the next sequence's too: nothing is changed, -4."""
    say("cache, held page with count", refs)
    t = Both(E, 2, 6, 8, 16, 4, 3, seed=7)
    t.commit([0], t.paths(1, 5, [5]), [5])
    page = int(t.c.table[0, 0])
    t.c.refs[page] = refs
    t.r.refs[page] = refs
    draft = torch.zeros((2, 2, 4, 16), dtype=torch.int16, device="cuda")
    status = E.enc_cache_commit(t.c, i32([1, 0]), draft, i32(np.zeros((2, 4))), i32([3, 1]))
    assert int(status) == -4
    t.same()
    t.c.refs[page] = t.r.refs[page] = 1             # put right, the same call goes through
    t.commit([1, 0], t.paths(2, 4, [3, 1]), [3, 1])
