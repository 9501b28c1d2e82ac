"""Rotation and the cache's calls in a captured graph, replayed with eager work
between the replays: equal to the eager calls every time."""
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


def captured(call):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    return g


def test_rotation(E):
    say("rope in a graph")
    x = torch.randn(40, 12, 64, device="cuda")
    q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
    ang = torch.randn(100, 32, device="cuda")
    table, pos = torch.cat([ang.cos(), ang.sin()], 1), torch.arange(40, dtype=torch.int32, device="cuda")
    out = tuple(torch.empty(t.shape, dtype=torch.bfloat16, device="cuda") for t in (q, k, v))
    g = captured(lambda: E.enc_qk_norm_rope(q, k, v, pos, table, out=out))
    for rep in range(4):
        x.normal_()
        pos.add_(rep)
        want = E.enc_qk_norm_rope(q, k, v, pos, table)
        for t in out:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out)), rep


def test_cache(E):
    """Fork, commit with copy on write and truncate in one graph."""
    say("cache in a graph")
    i32 = lambda a: torch.from_numpy(np.array(a, np.int32)).cuda()  # noqa: E731
    caches = [E.Cache.empty(4, 64, 8, (32,), 4, 20, dtype=torch.int16) for _ in "ab"]
    caches[1].data.copy_(caches[0].data.random_(-999, 999))
    draft = torch.zeros(4, 2, 6, 32, dtype=torch.int16, device="cuda")
    path, count, seqs = i32([[0, 1, 2, 3, 4, 5], [0, 2, 4, 5, 0, 0]]), i32([6, 4]), i32([0, 1])
    src, dst, cut = i32([0, 1]), i32([2, 3]), i32([7, 0])
    ws = [E.cache_workspace(c, path) for c in caches]

    def step(c, w):
        E.enc_cache_fork(c, src, dst)
        E.enc_cache_commit(c, seqs, draft, path, count, ws=w)
        E.enc_cache_truncate(c, dst, cut)

    step(caches[1], ws[1])                          # as captured() does once on the other
    g = captured(lambda: step(caches[0], ws[0]))
    for rep in range(6):
        draft.random_(-999, 999)
        count.copy_(torch.tensor([6 - rep % 3, 1 + rep % 4], dtype=torch.int32))
        step(caches[1], ws[1])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert int(caches[0].status) == int(caches[1].status) == 0
        a, b = caches
        assert all(torch.equal(getattr(a, n), getattr(b, n)) for n in ("table", "lens", "refs")), rep
        for s in range(4):                          # every held row (the first pass's drafts were zeros in both)
            n = int(a.lens[s])
            pages = a.table[s, :-(-n // 8)].long()
            assert torch.equal(a.data[:, pages].reshape(4, -1, 32)[:, :n], b.data[:, pages].reshape(4, -1, 32)[:, :n]), rep
