"""enc_prefix_attention without groups, and calls of many sizes in one workspace,
against the formula in 64 bits (tolerances: test_gpu_prefix_attention.py)."""
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_prefix_attention import Case, compare  # noqa: E402
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


def test_one_workspace_for_all(E):
    """A workspace of the largest call serves smaller ones, which write nothing past it; a call that needs more than it
    is given is refused."""
    say("prefix workspace")
    T, H, G, D = 10, 8, 2, 128
    biggest = Case([(90, [i % 5 for i in range(8)])] * 4, T, H, G, D, 16, seed=63)
    starts = torch.zeros(5, dtype=torch.int32, device="cuda")
    size = E.enc_prefix_attention_workspace_bytes(biggest.q, biggest.kn, torch.from_numpy(biggest.table), biggest.kc, starts)
    room = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    for members, groups, nodes in ((8, 4, 10), (8, 1, 10), (1, 1, 10), (4, 4, 10), (8, 4, 1), (2, 1, 1), (3, 2, 4), (1, 4, 1)):
        c = Case([(90, [i % 5 for i in range(members)])] * groups, nodes, H, G, D, 16, seed=64)
        say("prefix workspace", members, groups, nodes)
        want, wl, magnitude = c.want()
        for kw in (dict(), dict(starts=[0], shared=[])):
            out, lse = c.run(E, ws=room[:size], **kw)
            compare(out, lse, want, wl, magnitude)
    assert (room[size:] == 0xA5).all()
    with pytest.raises(E.EncError):
        biggest.run(E, ws=room[:1024])
