"""enc_verify_tree over vocabularies whose rows no longer fit the lanes'
registers (above 262144 values): equal, number for number, to the definition."""
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_verify_tree import compare, make  # noqa: E402


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


@pytest.mark.parametrize("spins", ["", "0"])
@pytest.mark.parametrize("point", [False, True])
@pytest.mark.parametrize("B,T,V,dt", [
    (2, 6, 262144, torch.float32),       # the largest that fits
    (2, 6, 262145, torch.float32),
    (3, 5, 300007, torch.bfloat16),
    (1, 7, 1000003, torch.float32),
    (1, 4, 1 << 22, torch.float16),      # the largest there is
])
def test_vocabularies_above_the_registers(E, monkeypatch, B, T, V, dt, point, spins):
    say("verify large vocabulary", B, T, V, dt, point, spins)
    if spins:
        monkeypatch.setenv("ENC_VERIFY_SPINS", spins)
    ws = None
    rejected = 0
    for seed in range(2):
        # 16-bit types hold what a softmax over this many values gives as multiples of little
        parents, tokens, p, q, u = make(B, T, V, dt, 50 + seed, width=T, near=1.5)
        parents[0, 1:] = 0                                  # all children of one node: rejections in a row
        u[0, 1:] = 0.999
        if ws is None:
            ws = E.verify_tree_workspace(torch.from_numpy(tokens).cuda(), p.cuda())
        want = compare(E, parents, tokens, p, None if point else q, u, ws=ws)
        rejected += int((want[1] < T).sum())
        u0 = u.copy()
        u0[:, 0] = [0.0, 0.9999999, 0.25][:B]
        compare(E, parents, tokens, p, None if point else q, u0, ws=ws)
    assert rejected and not ws.any()


@pytest.mark.parametrize("spins", ["0", "2"])
def test_workgroups_that_give_up_leave_the_workspace_zero(E, monkeypatch, spins):
    """Many sequences whose workgroups stop waiting at their first sum, then the
    same workspace with all the patience there is, in turn."""
    say("verify, impatient then patient", spins)
    parents, tokens, p, q, u = make(24, 3, 66000, torch.float32, 60, near=1.5)
    c = [torch.from_numpy(a).cuda() for a in (parents, tokens)] + [p.cuda(), q.cuda(), torch.from_numpy(u).cuda()]
    ws = E.verify_tree_workspace(c[1], c[2])
    want = [t.clone() for t in E.enc_verify_tree(*c)]
    for _ in range(20):
        monkeypatch.setenv("ENC_VERIFY_SPINS", spins)
        got = E.enc_verify_tree(*c, ws=ws)
        monkeypatch.delenv("ENC_VERIFY_SPINS")
        again = E.enc_verify_tree(*c, ws=ws)
        assert all(torch.equal(a, b) for a, b in zip(want, got)) and all(torch.equal(a, b) for a, b in zip(want, again))
    assert not ws.any()
