"""enc_verify_tree on the GPU: equal, number for number, to the definition."""
import sys

import numpy as np
import pytest

import step_ref as ref

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


def make(B, T, V, dt, seed, width=3, near=0.6):
    rng = np.random.default_rng([31, seed, B, T, V])
    x = rng.standard_normal((B, T, V)).astype(np.float32) * 2.5
    y = x + near * rng.standard_normal((B, T, V)).astype(np.float32)
    soft = lambda z: torch.softmax(torch.from_numpy(z).double(), -1).to(dt)  # noqa: E731
    p, q = soft(x), soft(y)
    parents = np.full((B, T), -1, np.int32)
    tokens = np.zeros((B, T), np.int32)
    for b in range(B):
        for i in range(1, T):
            parents[b, i] = rng.integers(max(0, i - width), i)
            w = q[b, parents[b, i]].double().numpy()
            tokens[b, i] = rng.choice(V, p=w / w.sum())
    return parents, tokens, p, q, rng.random((B, T), dtype=np.float32)


def compare(E, parents, tokens, p, q, u, nodes=None, **kw):
    c = lambda a: None if a is None else (a if isinstance(a, torch.Tensor) else torch.from_numpy(a)).cuda()  # noqa: E731
    got = E.enc_verify_tree(c(parents), c(tokens), c(p), c(q), c(u), nodes=c(nodes), **kw)
    torch.cuda.synchronize()
    f = lambda t: None if t is None else t.float().cpu().numpy()  # noqa: E731
    want = ref.verify(parents, tokens, f(p), f(q), u, nodes)
    for g, w, name in zip(got, want, ("path", "count", "token")):
        assert np.array_equal(g.cpu().numpy(), w), (name, g.cpu().numpy().tolist(), w.tolist())
    return want


@pytest.mark.parametrize("point", [False, True])
@pytest.mark.parametrize("B,T,V,dt", [
    (1, 1, 1, torch.float32), (2, 1, 100, torch.bfloat16), (3, 2, 257, torch.float32), (5, 6, 1000, torch.float16),
    (4, 9, 4097, torch.float32), (3, 16, 32000, torch.bfloat16), (1, 6, 128256, torch.float32),
    (2, 24, 20011, torch.float16), (300, 4, 4500, torch.float32), (1, 256, 300, torch.float32),
    (20, 5, 65537, torch.float32),
])
def test_against_definition(E, B, T, V, dt, point):
    say("verify", B, T, V, dt, point)
    parents, tokens, p, q, u = make(B, T, V, dt, 1)
    compare(E, parents, tokens, p, None if point else q, u)


def test_every_way_a_walk_can_end(E):
    say("verify many walks")
    lengths = set()
    for seed in range(6):
        parents, tokens, p, q, u = make(64, 8, 50, torch.float32, 100 + seed, near=0.2 + 0.3 * seed)
        lengths |= set(compare(E, parents, tokens, p, q, u)[1].tolist())
        compare(E, parents, tokens, p, None, u)
    assert {1, 2, 3, 4} <= lengths


def test_nodes_chains_and_workspace_reuse(E):
    say("verify nodes, reuse")
    parents, tokens, p, q, u = make(6, 7, 9000, torch.float32, 2, width=1)
    ws = E.verify_tree_workspace(torch.from_numpy(tokens).cuda(), p.cuda())
    for nodes in ([7, 0, 3, 1, -2, 50], None, [1] * 6):
        n = None if nodes is None else np.array(nodes, np.int32)
        compare(E, parents, tokens, p, q, u, nodes=n, ws=ws)
    assert not ws.any()


@pytest.mark.parametrize("spins", ["0", "1", "3"])
def test_workgroups_that_do_not_wait(E, monkeypatch, spins):
    """With no patience, workgroups compute the others' sums themselves."""
    say("verify spins", spins)
    monkeypatch.setenv("ENC_VERIFY_SPINS", spins)
    parents, tokens, p, q, u = make(4, 9, 70000, torch.float32, 3)
    ws = E.verify_tree_workspace(torch.from_numpy(tokens).cuda(), p.cuda())
    for _ in range(3):
        compare(E, parents, tokens, p, q, u, ws=ws)
        compare(E, parents, tokens, p, None, u, ws=ws)
    assert not ws.any()


def test_strange_inputs(E):
    """Rows of zeros, NaN, infinities and negative values, tokens and parents out
    of range, equal rows (an empty difference), and the ends of u."""
    say("verify strange inputs")
    parents, tokens, p, q, u = make(12, 5, 700, torch.float32, 4)
    p[0] = 0
    p[1, :, ::3] = float("nan")
    p[2, :, 5] = float("inf")
    p[3] = -p[3]
    q[4] = p[4]
    u[4, 1:] = 1.0                                  # u q < r fails although q = r: max(r - q, 0) is empty
    tokens[5, 1:] = [-1, 700, 2 ** 31 - 1, -2 ** 31]
    parents[6, 1:] = [5, -3, 2 ** 30, -1]
    q[7] = 0
    u[8] = [0.0, 1.0, 0.0, 2.0, -1.0]
    u[9] = 1.0
    u[10] = float("nan")
    q[11] = float("nan")
    with np.errstate(invalid="ignore"):
        want = compare(E, parents, tokens, p, q, u)
        compare(E, parents, tokens, p, None, u)
    assert want[2][0] == -1


def test_strided_and_unaligned_rows(E):
    say("verify strides")
    parents, tokens, p, q, u = make(3, 5, 1001, torch.bfloat16, 5)
    big = torch.zeros(3, 6, 1010, dtype=torch.bfloat16, device="cuda")
    big[:, 1:, 3:1004] = p.cuda()
    other = torch.zeros(5, 3, 1001, dtype=torch.bfloat16, device="cuda")
    other[:] = q.cuda().transpose(0, 1)
    compare(E, parents, tokens, big[:, 1:, 3:1004], other.transpose(0, 1), u)


def test_another_stream_and_a_graph(E):
    say("verify stream, graph")
    parents, tokens, p, q, u = make(3, 6, 30000, torch.float32, 6)
    c = [torch.from_numpy(a).cuda() for a in (parents, tokens)] + [p.cuda(), q.cuda(), torch.from_numpy(u).cuda()]
    want = [t.clone() for t in E.enc_verify_tree(*c)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = E.enc_verify_tree(*c, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    ws = E.verify_tree_workspace(c[1], c[2])
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        held = E.enc_verify_tree(*c, ws=ws)
    for rep in range(3):
        c[4].copy_(torch.rand(3, 6))
        want = [t.clone() for t in E.enc_verify_tree(*c)]
        for t in held:
            t.fill_(-9)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held)), rep
