"""enc_qk_norm_rope at the edge of the rotated values."""
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("rot", [2, 4, 6, 8, 12, 20, 34, 90])
def test_values_past_the_rotation_are_only_converted(E, rot, adjacent):
    """Without a norm, a value that is not turned stays as it is, next to
    infinities and NaN too."""
    say("rope, values past the rotation", rot, adjacent)
    rng = np.random.default_rng(rot)
    x = torch.from_numpy(rng.standard_normal((6, 3, 96)).astype(np.float32)).cuda()
    bad = [float("inf"), -float("inf"), float("nan")]
    for t in range(6):
        x[t, :, rot + (5 * t) % (96 - rot)] = bad[t % 3]
    ang = torch.from_numpy(rng.standard_normal((8, rot // 2)).astype(np.float32)).cuda()
    table = torch.cat([ang.cos(), ang.sin()], 1)
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    q, k, _ = E.enc_qk_norm_rope(x, x[:, :2], None, pos, table, adjacent=adjacent, norm=False, out_dtype=torch.float32)
    for got, want in ((q, x), (k, x[:, :2])):
        assert torch.equal(got[..., rot:].nan_to_num(7.0), want[..., rot:].nan_to_num(7.0))
        assert torch.equal(got[..., rot:].isnan(), want[..., rot:].isnan())
        assert got[..., :rot].isfinite().all()
