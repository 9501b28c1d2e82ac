"""enc_cache_commit / _fork / _truncate on the GPU: table, lengths, counts and
every byte of the data equal to the plain bookkeeping's after each call."""
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


def i32(a):
    return torch.from_numpy(np.array(a, np.int32)).cuda()


class Both:
    """The cache on the device and as plain arrays, driven by the same calls."""

    def __init__(self, E, planes, pages, page, row, seqs, max_pages, seed=0):
        self.E, self.rng = E, np.random.default_rng([41, seed, pages, page])
        self.c = E.Cache.empty(planes, pages, page, (row,), seqs, max_pages, dtype=torch.int16)
        self.c.data.copy_(torch.from_numpy(self.rng.integers(-2 ** 15, 2 ** 15, self.c.data.shape).astype(np.int16)))
        self.r = ref.Pages(self.c.data.cpu().numpy(), *(t.cpu().numpy() for t in (self.c.table, self.c.lens, self.c.refs)))
        self.row = row

    def same(self):
        torch.cuda.synchronize()
        for name in ("table", "lens", "refs", "data"):
            assert np.array_equal(getattr(self.c, name).cpu().numpy(), getattr(self.r, name)), name

    def commit(self, seqs, path, count):
        path = np.array(path, np.int32)
        draft = self.rng.integers(-2 ** 15, 2 ** 15, (self.r.data.shape[0],) + path.shape + (self.row,)).astype(np.int16)
        status = self.E.enc_cache_commit(self.c, i32(seqs), torch.from_numpy(draft).cuda(), torch.from_numpy(path).cuda(),
                                         i32(count))
        want = self.r.commit(seqs, draft, path, count)
        assert int(status) == want
        self.same()
        return want

    def fork(self, src, dst):
        self.E.enc_cache_fork(self.c, i32(src), i32(dst))
        self.r.fork(src, dst)
        self.same()

    def truncate(self, seqs, lens):
        self.E.enc_cache_truncate(self.c, i32(seqs), i32(lens))
        self.r.truncate(seqs, lens)
        self.same()

    def paths(self, n, T, counts):
        p = np.full((n, T), -1, np.int32)
        for b in range(n):
            p[b, :counts[b]] = np.sort(self.rng.permutation(T)[:counts[b]])
        return p


@pytest.mark.parametrize("page,row,T", [(1, 8, 5), (8, 8, 5), (16, 24, 33), (20, 136, 7), (64, 1024, 256)])
def test_a_long_life(E, page, row, T):
    """Appends, forks, cuts and frees in a random order."""
    say("cache life", page, row, T)
    S, M = 6, -(-4 * T // page) + 3
    t = Both(E, 3, S * M, page, row, S, M, seed=page)
    for step in range(25):
        what = t.rng.integers(0, 4)
        if what <= 1:
            n = int(t.rng.integers(1, S + 1))
            seqs = t.rng.permutation(S)[:n].tolist()
            room = [M * page - int(t.r.lens[s]) for s in seqs]
            counts = [int(min(t.rng.integers(0, T + 1), r)) for r in room]
            t.commit(seqs, t.paths(n, T, counts), counts)
        elif what == 2:
            order = t.rng.permutation(S)
            k = int(t.rng.integers(1, 4))
            t.fork([int(order[0])] * k, order[1:1 + k].tolist())
        else:
            n = int(t.rng.integers(1, S + 1))
            seqs = t.rng.permutation(S)[:n].tolist()
            t.truncate(seqs, [int(t.rng.integers(0, t.r.lens[s] + 2)) for s in seqs])
    t.truncate(list(range(S)), [0] * S)
    assert not t.r.refs.any() and (t.r.table == -1).all()


def test_shared_last_pages_are_copied_once_each(E):
    say("cache copy on write")
    t = Both(E, 2, 40, 16, 64, 8, 4, seed=1)
    t.commit([0], t.paths(1, 20, [20]), [20])
    t.fork([0] * 5, [1, 2, 3, 4, 5])
    t.truncate([3], [18])                            # a shared page, less of it
    t.truncate([4], [16])                            # no partly filled page
    t.commit([0, 1, 3, 4, 5], t.paths(5, 6, [2, 6, 1, 3, 0]), [2, 6, 1, 3, 0])
    t.commit([2, 5], t.paths(2, 6, [1, 1]), [1, 1])


def test_refusals_change_nothing(E):
    say("cache refusals")
    t = Both(E, 2, 6, 8, 16, 4, 3, seed=2)
    assert t.commit([0, 1], t.paths(2, 12, [12, 9]), [12, 9]) == 0          # 4 of 6 pages
    assert t.commit([2, 3], t.paths(2, 20, [17, 1]), [17, 1]) == 2           # 4 needed, 2 free
    assert t.commit([0, 1], t.paths(2, 20, [12, 16]), [12, 16]) == -3        # 25 tokens: past the end
    assert t.commit([0, 4], t.paths(2, 4, [1, 1]), [1, 1]) == -1
    assert t.commit([-1, 2], t.paths(2, 4, [1, 1]), [1, 1]) == -1
    assert t.commit([0, 2], t.paths(2, 4, [1, 1]), [1, 5]) == -2
    assert t.commit([0, 2], t.paths(2, 4, [1, 1]), [-1, 1]) == -2
    assert t.commit([0, 2], [[0, 4, 0, 0], [0, 0, 0, 0]], [2, 1]) == -2
    assert t.commit([0, 2], [[0, -1, 0, 0], [0, 0, 0, 0]], [2, 1]) == -2
    assert t.commit([0], [[3, 3, 0, 1]], [4]) == 0
    t.fork([0, 9, 1, 2], [2, 3, 1, -5])              # only the first pair is one
    t.truncate([7, -1, 1], [0, 0, 4])
    t.truncate([1, 0], [100, -3])                    # longer than it is: as it was; below 0: freed


def test_many_pages_and_sequences(E):
    say("cache many")
    S = 1500
    t = Both(E, 1, 70000, 4, 8, S, 6, seed=3)
    t.commit(list(range(S)), t.paths(S, 9, [9] * S), [9] * S)
    t.truncate(list(range(0, S, 3)), [2] * (S // 3))
    t.commit(list(range(S - 1, -1, -1)), t.paths(S, 9, [5] * S), [5] * S)


def test_rows_of_other_layouts_and_streams(E):
    """Draft planes and sequences apart from each other, cache planes apart, a
    workspace used again, another stream."""
    say("cache layouts")
    rng = np.random.default_rng(5)
    store = torch.from_numpy(rng.integers(-99, 99, (5, 2, 10, 16, 2, 8)).astype(np.int16)).cuda()
    data = store[:, 1]                               # planes of a larger array
    table, lens, refs = i32(np.full((3, 4), -1)), i32(np.zeros(3)), i32(np.zeros(10))
    c = E.Cache(data, table, lens, refs)
    r = ref.Pages(data.cpu().numpy(), *(x.cpu().numpy() for x in (table, lens, refs)))
    draft = torch.from_numpy(rng.integers(-99, 99, (5, 3, 4, 6, 2, 8)).astype(np.int16)).cuda()[:, :2, 1]
    path, count = np.array([[0, 3, 5, -1, -1, -1], [1, 2, 3, 4, 5, 0]], np.int32), [3, 6]
    ws = E.cache_workspace(c, torch.from_numpy(path).cuda())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            ws.fill_(0xFF)
            st = E.enc_cache_commit(c, i32([2, 0]), draft, torch.from_numpy(path).cuda(), i32(count), ws=ws)
            assert r.commit([2, 0], draft.cpu().numpy(), path, count) == int(st)
    side.synchronize()
    assert np.array_equal(data.cpu().numpy(), r.data) and np.array_equal(table.cpu().numpy(), r.table)
    assert np.array_equal(refs.cpu().numpy(), r.refs) and np.array_equal(lens.cpu().numpy(), r.lens)


def test_a_workspace_on_the_host_is_refused(E):
    say("cache workspace on the host")
    t = Both(E, 1, 4, 4, 8, 1, 4, seed=6)
    draft = torch.zeros((1, 1, 2, 8), dtype=torch.int16, device="cuda")
    with pytest.raises(ValueError):
        E.enc_cache_commit(t.c, i32([0]), draft, i32([[0, 1]]), i32([2]), ws=torch.empty(4096, dtype=torch.uint8))
    t.same()
