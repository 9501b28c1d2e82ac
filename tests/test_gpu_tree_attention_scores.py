"""enc_tree_attention over the whole range of scales and scores, in every
kernel that a call can reach, against the formula in 64 bits.

Tolerances: those derived in test_gpu_tree_attention.py, where nothing else is
said."""
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_tree_attention import Case  # noqa: E402


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


# rows that share a KV head: T H / G
SHAPES = {
    "4 rows, a strip to a wave": (2, 1, 8, 2, 128, [90, 0], 16),
    "12 rows, a strip to a wave": (2, 3, 8, 2, 128, [70, 0], 16),
    "8 rows, heads of 200": (1, 4, 4, 2, 200, [130], 16),
    "6 rows, four heads to a workgroup": (128, 3, 8, 4, 64, [b * 7 % 90 for b in range(128)], 16),
    "28 rows, four heads to a workgroup": (128, 7, 16, 4, 128, [b * 7 % 90 for b in range(128)], 16),
    "49 rows, four waves of 16, many sequences": (128, 7, 28, 4, 128, [b * 7 % 90 for b in range(128)], 16),
    "20 rows, four waves of 16": (2, 5, 8, 2, 128, [500, 0], 16),
    "40 rows, four waves of 16": (2, 10, 8, 2, 64, [70, 300], 20),
    "40 rows, heads of 256": (2, 10, 8, 2, 256, [0, 90], 16),
    "100 rows, eight waves of 16": (1, 25, 8, 2, 128, [300], 16),
    "100 rows, heads of 256": (1, 25, 8, 2, 256, [90], 16),
    "100 rows, four waves of 32": (32, 25, 16, 4, 64, [b * 7 % 90 for b in range(32)], 16),
    "132 rows, eight waves of 32": (2, 33, 4, 1, 128, [300, 0], 16),
    "256 rows, eight waves of 32": (1, 64, 8, 2, 128, [700], 64),
}


@pytest.mark.parametrize("scale", [0.0, -1.0])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_scale_zero_or_negative(E, shape, dt, scale):
    """With scale 0 every node has the mean of what it sees, whatever it does not see."""
    say("attention scale", scale, shape, dt)
    c = Case(*SHAPES[shape], dt, seed=31)
    c.scale *= scale
    c.check(E)
    c.seen[:, c.T // 2] = False                     # a node that sees no other, nor itself
    c.check(E, nodes=[c.T - b % 2 for b in range(c.B)])
