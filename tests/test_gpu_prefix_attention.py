"""enc_prefix_attention and enc_cache_shared on the GPU against the formula in 64
bits (each row over all the keys it sees, whoever shares them).

Tolerance, derived: with u the rounding unit of the type (2^-8 BF16, 2^-11
FP16), the result's rounding is u |o|; each weight p is rounded to that type
(u p |v| each, at most); scores are fp32 sums of at most 256 exact products,
off by less than 256 2^-24 sum |q k| scale, which for the inputs here (|q|,
|k| about 1 a value) is below 2^-11 absolute and so relative in p. Together
|err| <= u |o| + (u + 2^-10) sum p |v|, and the log-sum-exp is off by less than
2^-11 + 2^-20 |lse|."""
import ctypes
import sys

import numpy as np
import pytest

import step_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
U = {BF: 2.0 ** -8, FP: 2.0 ** -11}


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


def dev(a, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype))).cuda()


class Case:
    """groups: [(prefix, [tail, ...]), ...]; the sequences of a group share its prefix's whole pages, and have equal
    rows up to its end."""

    def __init__(self, groups, T, H, G, D, page, dt=BF, seed=0, width=None, extra=2):
        rng = np.random.default_rng([33, seed, T, H, G, D, page])
        self.T, self.H, self.G, self.D, self.page, self.dt = T, H, G, D, page, dt
        lens, rows, used = [], [], 0
        self.starts, self.shared = [0], []
        copies = []
        for prefix, tails in groups:
            full = prefix // page
            common = list(range(used, used + full))
            used += full
            first = None
            for tail in tails:
                n = -(-(prefix % page + tail) // page)
                rows.append(common + list(range(used, used + n)))
                if prefix % page:
                    if first is None:
                        first = used
                    else:
                        copies.append((first, used, prefix % page))
                used += n
                lens.append(prefix + tail)
            self.starts.append(len(lens))
            self.shared.append(prefix)
        self.B, self.lens = len(lens), np.array(lens, np.int32)
        n_pages = used + extra
        order = rng.permutation(n_pages)
        self.table = np.full((self.B, width or max([len(r) for r in rows] + [1])), -1, np.int32)
        for s, r in enumerate(rows):
            self.table[s, :len(r)] = order[r]
        t = lambda *shape: torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dt).cuda()  # noqa: E731
        B = self.B
        self.q, self.kn, self.vn = t(B, T, H, D), t(B, T, G, D), t(B, T, G, D)
        self.kc, self.vc = t(n_pages, page, G, D), t(n_pages, page, G, D)
        for a, b, n in copies:
            for c in (self.kc, self.vc):
                c[int(order[b]), :n] = c[int(order[a]), :n]
        parents = np.full((B, T), -1, np.int32)
        for i in range(1, T):
            parents[:, i] = rng.integers(0, i, B)
        self.seen = ref.ancestors(parents)
        self.scale = D ** -0.5

    def run(self, E, mask=True, seqs=None, nodes=None, starts=None, shared=None, **kw):
        out, lse = E.enc_prefix_attention(
            self.q, self.kn, self.vn, self.kc, self.vc, dev(self.table), dev(self.lens),
            dev(self.starts if starts is None else starts), dev(self.shared if shared is None else shared),
            mask=dev(ref.mask_words(self.seen), np.int64) if mask else None, seqs=None if seqs is None else dev(seqs),
            nodes=None if nodes is None else dev(nodes), scale=self.scale, return_lse=True, **kw)
        torch.cuda.synchronize()
        return out, lse

    def want(self, mask=True, seqs=None, nodes=None):
        d = lambda x: x.double().cpu().numpy()  # noqa: E731
        seen = self.seen if mask else np.tril(np.ones((self.T, self.T), bool))[None].repeat(self.B, 0)
        return ref.tree_attention(d(self.q), d(self.kn), d(self.vn), d(self.kc), d(self.vc), self.table, self.lens, seen,
                                  self.scale, seqs, nodes)

    def check(self, E, starts=None, shared=None, **kw):
        out, lse = self.run(E, starts=starts, shared=shared, **kw)
        want, wl, size = self.want(**kw)
        compare(out, lse, want, wl, size)
        return out, lse


def compare(out, lse, want, wl, size):
    u = U[out.dtype]
    g, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    bad = ~(np.abs(g - want) <= u * np.abs(want) + (u + 2.0 ** -10) * size + 1e-30)
    assert not bad.any(), "%d of %d outside, worst %g" % (bad.sum(), bad.size, np.nanmax(np.abs(g - want)))
    fin = np.isfinite(wl)
    assert np.array_equal(fin, np.isfinite(gl))
    assert (np.abs(gl - wl)[fin] <= 2.0 ** -11 + 2.0 ** -20 * np.abs(wl[fin])).all()
    assert (gl[~fin] == -np.inf).all() and (g[~fin] == 0).all()


@pytest.mark.parametrize("groups,T,H,G,D,page,dt", [
    ([(1, [0, 0])], 1, 1, 1, 64, 16, BF),                              # the smallest call
    ([(0, [0, 5])], 1, 2, 1, 64, 16, BF),                              # nothing in common
    ([(31, [1, 0, 3])], 1, 4, 1, 128, 16, FP),                         # around a strip of 32
    ([(33, [31, 32])], 1, 8, 2, 128, 16, BF),
    ([(1021, [3, 0, 17, 40])], 1, 32, 8, 128, 16, BF),
    ([(128, [1, 1]), (64, [5]), (200, [9, 0, 33, 7])], 1, 8, 2, 64, 16, FP),
    ([(500, list(range(20)))], 1, 8, 2, 128, 64, BF),                  # 80 rows: two tiles
    ([(130, [40, 2, 0]), (77, [5, 6])], 5, 4, 2, 64, 1, BF),           # trees, pages of one token
    ([(129, [4, 60]), (40, [9, 9, 9])], 7, 6, 2, 96, 20, FP),          # pages that end inside a strip
    ([(300, [0, 10, 33])], 33, 4, 1, 128, 48, BF),                     # 132 own rows: tiles of a sequence
    ([(90, [5, 70])], 256, 2, 1, 64, 16, FP),                          # the largest tree
    ([(100, [5, 70, 1])], 3, 2, 1, 256, 16, BF),
    ([(100, [5, 70])], 40, 2, 1, 256, 16, FP),
    ([(70, [20, 45])], 4, 3, 3, 8, 16, BF),                            # heads smaller than a fragment
    ([(60, [7, 8, 9])], 1, 7, 1, 80, 16, FP),
    ([(77, [1] * 9)], 9, 4, 2, 200, 32, BF),
    ([(3, [2, 1])], 2, 2, 1, 64, 4096, BF),                            # a page larger than the history
    ([(3000, [40, 100])], 1, 4, 4, 128, 16, BF),
])
def test_against_formula(E, groups, T, H, G, D, page, dt):
    say("prefix", groups, T, H, G, D, page, dt)
    Case(groups, T, H, G, D, page, dt).check(E)


@pytest.mark.parametrize("T", [1, 2, 40])
def test_chain_without_a_mask(E, T):
    say("chain", T)
    Case([(100, [3, 50]), (33, [0, 1])], T, 4, 2, 128, 16, seed=1).check(E, mask=False)


@pytest.mark.parametrize("D,dt,T", [(64, BF, 2), (128, FP, 2), (256, BF, 2), (64, FP, 10), (128, BF, 10), (256, FP, 10),
                                    (64, BF, 30), (128, BF, 30), (96, FP, 30)])
def test_any_shared_length(E, D, dt, T):
    """Fewer tokens than the rows agree in, none, more than the shortest has, negative: results stay the same."""
    say("shared lengths", D, T)
    c = Case([(100, [0, 3, 40]), (65, [1, 2])], T, 4, 2, D, 16, dt, seed=2)
    for shared in ([100, 65], [99, 1], [0, 0], [32, 64], [31, 33], [-7, 65], [1, -2 ** 31]):
        c.check(E, shared=shared)
    c = Case([(100, [0, 3, 40])], 1, 4, 2, D, 16, dt, seed=3)
    c.check(E, shared=[2 ** 31 - 1])                                   # the shortest has 100, and all agree in them


def test_groups_of_any_kind(E):
    """All sequences agree in 90 tokens, so every way to group them is right: entries of no group, empty groups, groups
    of one, starts out of range or not ascending."""
    say("groups")
    c = Case([(90, [0, 5, 33, 7, 64, 1, 2, 20])], 2, 4, 2, 64, 16, seed=4)
    for starts in ([0, 8], [0, 3, 8], [2, 5], [0, 0, 0, 8, 8], [0, 1, 2, 3, 4, 5, 6, 7, 8], [8, 8], [0, 0], [3, 100],
                   [-5, 2, 7], [0, 6, 3, 8], [5, 1, 0, 8], [0, 8, 0, 8, 0, 8], [2 ** 31 - 1, -2 ** 31], [0]):
        c.check(E, starts=starts, shared=[90] * (len(starts) - 1))


def test_sequences_by_index_and_live_nodes(E):
    say("seqs, nodes")
    c = Case([(90, [0, 5, 33]), (40, [7, 64])], 9, 4, 2, 64, 16, seed=5)
    c.check(E, seqs=[2, 0, 1, 4, 3], nodes=[9, 4, 3, 12, 0])
    c.check(E, seqs=[0, 0, 0, 3, 3], nodes=[0, 1, -5, 9, 9])
    # an index outside the table has no cached tokens, and so its group none in common
    c.check(E, seqs=[2, 7, 1, 4, -1], nodes=[9, 4, 3, 2, 1])


def test_rows_that_see_nothing(E):
    say("empty rows")
    c = Case([(0, [0, 0]), (50, [0, 20])], 6, 4, 2, 128, 16, seed=6)
    c.seen[:, 2] = False
    c.seen[:, 4, :] = False
    c.check(E)


def test_table_far_wider_than_the_histories(E):
    say("wide table")
    Case([(700, [30, 0, 500])], 3, 8, 2, 128, 16, seed=7, width=4000).check(E)


@pytest.mark.parametrize("T", [5, 20, 40])
def test_table_that_could_hold_long_histories(E, T):
    """What a table can hold chooses the tiles of groups of some 20, 80 and more rows, never the result."""
    say("room", T)
    for width in (None, 1100, 2100):                                   # pages of 16: up to 17600 and 33600 tokens
        Case([(100, [0, 3, 40]), (70, [10])], T, 4, 2, 128, 16, seed=19, width=width).check(E)


@pytest.mark.parametrize("T", [2, 8, 20, 40])
def test_strangers_leave_rows_alone(E, T):
    """NaN and infinities in pages' unused rows, in pages of nobody, and in nodes that a row does not see."""
    say("strangers", T)
    c = Case([(100, [0, 3, 40]), (70, [10])], T, 4, 2, 128, 16, seed=8)
    used = set()
    for s in range(c.B):
        for j in range(int(c.lens[s])):
            used.add((int(c.table[s, j // 16]), j % 16))
    for p in range(c.kc.shape[0]):
        for r in range(16):
            if (p, r) not in used:
                c.kc[p, r] = float("nan") if r % 2 else float("inf")
                c.vc[p, r] = float("inf") if r % 2 else float("nan")
    c.check(E)
    clean, clean_lse = c.run(E)
    c.seen[:, :, T - 1] = False
    c.seen[:, T - 1, T - 1] = True
    before, _ = c.run(E)
    c.vn[:, T - 1] = float("inf")
    c.kn[1, T - 1] = float("nan")
    out, _ = c.run(E)
    assert torch.equal(out[:, :T - 1], before[:, :T - 1])
    # the row that sees them; a sequence's NaN is its own
    assert out[1, T - 1].isnan().all() and (out[0, T - 1] == float("inf")).all()


@pytest.mark.parametrize("T", [1, 8, 30])
def test_a_row_depends_on_nothing_but_its_own(E, T):
    """Large and infinite queries of one sequence change nothing in the others, to the bit."""
    say("rows", T)
    c = Case([(300, [0, 3, 40, 7, 9])], T, 8, 2, 128, 16, seed=9)
    want, wl = c.run(E)
    c.q[2] *= 1000.0
    c.q[3, 0, 1] = float("inf")
    got, gl = c.run(E)
    for b in (0, 1, 4):
        assert torch.equal(got[b], want[b]) and torch.equal(gl[b], wl[b])


@pytest.mark.parametrize("T", [3, 10, 30])                                # up to 16 rows of a group, 64, more
@pytest.mark.parametrize("scale", [0.0, -0.1, 30.0, 1e-30, 1e30, -1e38, 3e38])
def test_scales(E, scale, T):
    """Any finite scale. With large ones one key takes all: then inputs are whole numbers, so that scores are exact."""
    say("scale", scale, T)
    c = Case([(90, [0, 20]), (40, [3, 3, 3])], T, 4, 2, 64, 16, seed=10)
    if abs(scale) > 1:
        for t in (c.q, c.kn, c.kc):
            t.copy_(t.mul(2).round())
    c.scale = scale
    out, lse = c.run(E)
    want, wl, size = c.want()
    u = U[c.dt]
    assert (np.abs(out.double().cpu().numpy() - want) <= u * np.abs(want) + (u + 2.0 ** -10) * size + 1e-30).all()
    fin = np.isfinite(wl) & (np.abs(wl) < 3e38)
    assert (np.abs(lse.double().cpu().numpy() - wl)[fin] <= 2.0 ** -11 + 2.0 ** -20 * np.abs(wl[fin])).all()


def test_strides(E):
    """Heads before tokens in the cache; q, k and v as parts of one projection; outputs with gaps that stay."""
    say("strides")
    c = Case([(100, [0, 3, 40]), (33, [8, 8])], 4, 8, 2, 64, 16, seed=11)
    want, wl = c.run(E)
    B, T, H, G, D = c.B, c.T, c.H, c.G, c.D
    packed = torch.cat([c.q, c.kn, c.vn], 2)
    c.q, c.kn, c.vn = packed[:, :, :H], packed[:, :, H:H + G], packed[:, :, H + G:]
    c.kc, c.vc = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (c.kc, c.vc))
    room = torch.full((B, T, H + 3, D), 5.0, dtype=c.dt, device="cuda")
    got, gl = c.run(E, out=room[:, :, :H])
    assert torch.equal(got, want) and torch.equal(gl, wl) and (room[:, :, H:] == 5).all()


def test_many_groups_and_one_large(E):
    """More groups, and more sequences in a group, than the plan looks at in one go."""
    say("many groups")
    Case([(17, [1, 2])] * 1100, 1, 1, 1, 64, 16, seed=12).check(E)
    Case([(40, [0, 1] * 700)], 1, 2, 1, 64, 16, seed=13).check(E)


def test_long_prefix(E):
    """Pieces of many strips, more of them than a wave joins at once: against fp64 on the device."""
    say("long prefix")
    for D, dt, T in ((128, BF, 1), (64, FP, 8), (256, BF, 1)):
        c = Case([(40000, [100, 0, 700]), (1, [2])], T, 4, 1, D, 64, dt, seed=14)
        out, lse = c.run(E)
        for b in range(c.B):
            n = int(c.lens[b])
            pages = torch.from_numpy(c.table[b, :-(-n // 64)]).long().cuda()
            k = torch.cat([c.kc[pages, :, 0].reshape(-1, D)[:n], c.kn[b, :, 0]]).double()
            v = torch.cat([c.vc[pages, :, 0].reshape(-1, D)[:n], c.vn[b, :, 0]]).double()
            x = torch.matmul(c.q[b].double(), k.T) * c.scale
            x[:, :, n:] = x[:, :, n:].masked_fill(~torch.from_numpy(c.seen[b]).cuda()[:, None], -np.inf)
            wl = torch.logsumexp(x, -1)
            p = (x - wl[..., None]).exp()
            compare(out[b], lse[b], torch.matmul(p, v).cpu().numpy(), wl.cpu().numpy(), torch.matmul(p, v.abs()).cpu().numpy())


def test_cache_above_4_gib(E):
    """Pages whose rows lie beyond 2^32 bytes and 2^31 elements."""
    say("4 GiB")
    small = Case([(100, [0, 30, 5])], 1, 8, 2, 128, 16, seed=15)
    want, wl = small.run(E)
    n = 600000                                                         # 600000 x 16 x 2 x 128 x 2 bytes: 4.9 GB
    step = (n - 1) // small.kc.shape[0]
    big = [torch.empty(n, 16, 2, 128, dtype=BF, device="cuda") for _ in range(2)]
    at = n - 1 - step * np.arange(small.kc.shape[0])
    for b, s in zip(big, (small.kc, small.vc)):
        b[torch.from_numpy(at).cuda()] = s
    small.kc, small.vc = big
    small.table = np.where(small.table >= 0, at[np.maximum(small.table, 0)], -1).astype(np.int32)
    got, gl = small.run(E)
    assert torch.equal(got, want) and torch.equal(gl, wl)


def test_workspace_stream_and_graph(E):
    """Equal bits from a used workspace, on another stream, and from a captured call whose lengths, groups and values
    change between replays."""
    say("graph")
    c = Case([(200, [0, 30, 5, 60]), (64, [1, 100])], 2, 8, 2, 128, 16, seed=16, width=40)
    want, wl = c.run(E)
    ws = E.prefix_attention_workspace(c.q, c.kn, dev(c.table), c.kc, dev(c.starts))
    ws.fill_(0xFF)
    got, gl = c.run(E, ws=ws)
    assert torch.equal(got, want) and torch.equal(gl, wl)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, gl = c.run(E, stream=other)
    assert torch.equal(got, want) and torch.equal(gl, wl)
    table, lens, starts, shared = dev(c.table), dev(c.lens), dev(c.starts), dev(c.shared)
    mask = dev(ref.mask_words(c.seen), np.int64)
    out = torch.empty_like(c.q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, lse = E.enc_prefix_attention(c.q, c.kn, c.vn, c.kc, c.vc, table, lens, starts, shared, mask=mask, scale=c.scale,
                                        return_lse=True, out=out, ws=ws)
    for step, (cut, st, sh) in enumerate([(0, [0, 4, 6], [200, 64]), (30, [0, 3, 6], [150, 0]), (1, [0, 6, 6], [0, 9]),
                                          (63, [2, 4, 5], [100, 64]), (0, [0, 4, 6], [200, 64])]):
        c.lens = np.maximum(np.array([200, 230, 205, 260, 65, 164], np.int32) - cut, 0)
        c.starts, c.shared = st, sh
        lens.copy_(dev(c.lens))
        starts.copy_(dev(st))
        shared.copy_(dev(sh))
        c.q.normal_()
        graph.replay()
        torch.cuda.synchronize()
        want, wl = c.run(E)
        assert torch.equal(out, want) and torch.equal(lse, wl)
        c.check(E)


def test_against_tree_attention(E):
    """The same call without sharing."""
    say("tree attention")
    c = Case([(300, [0, 3, 40]), (100, [8, 8])], 4, 8, 2, 128, 16, seed=17)
    out, lse = c.run(E)
    same, same_lse = E.enc_tree_attention(c.q, c.kn, c.vn, c.kc, c.vc, dev(c.table), dev(c.lens),
                                          mask=dev(ref.mask_words(c.seen), np.int64), scale=c.scale, return_lse=True)
    want, wl, size = c.want()
    compare(same, same_lse, want, wl, size)
    assert (lse - same_lse).abs().max() < 2.0 ** -10


def test_far_scores(E):
    """Scores that differ by little where they are large: whole numbers up to 2^16 and beyond, in every kernel."""
    say("far scores")
    for T in (1, 8, 30):
        c = Case([(200, [0, 9, 40])], T, 4, 2, 64, 16, seed=19)
        for t in (c.q, c.kn, c.kc):
            t.copy_(t.mul(2).round())
        c.q[..., 0], c.kn[..., 0], c.kc[..., 0] = 256.0, 256.0, 256.0      # 65536 in every score
        c.q[..., 1] *= 64
        c.scale = 0.125
        c.check(E)


def test_no_groups_no_pointers(E):
    """groups = 0: starts and shared may be NULL."""
    say("no groups")
    c = Case([(60, [0, 3])], 2, 4, 2, 64, 16, seed=20)
    want, _ = c.run(E, starts=[0], shared=[])
    out = torch.empty_like(c.q)
    table, lens, mask = dev(c.table), dev(c.lens), dev(ref.mask_words(c.seen), np.int64)
    ws = E.prefix_attention_workspace(c.q, c.kn, table, c.kc, dev([0]))
    a = E.EncPrefixAttentionArgs()
    t = a.t
    t.d_q, t.d_k_new, t.d_v_new, t.d_k_cache, t.d_v_cache, t.d_out = (x.data_ptr() for x in (c.q, c.kn, c.vn, c.kc, c.vc, out))
    t.d_table, t.d_lens, t.d_mask = table.data_ptr(), lens.data_ptr(), mask.data_ptr()
    for n, x in (("q", c.q), ("k_new", c.kn), ("v_new", c.vn), ("out", out)):
        for m, st in zip(("batch", "node", "head"), x.stride()):
            setattr(t, n + "_" + m, st)
    t.cache_page, t.cache_token, t.cache_head = c.kc.stride()[:3]
    t.batch, t.nodes, t.q_heads, t.kv_heads, t.head_dim, t.dtype = c.B, c.T, c.H, c.G, c.D, 1
    t.n_pages, t.page_size, t.max_pages, t.max_seqs, t.scale = c.kc.shape[0], 16, c.table.shape[1], c.B, c.scale
    assert E.lib().enc_prefix_attention(ctypes.byref(a), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_binding_refusals(E):
    say("refusals")
    c = Case([(30, [0, 3])], 2, 4, 2, 64, 16, seed=18)
    args = lambda **kw: [kw.get(n, d) for n, d in (  # noqa: E731
        ("q", c.q), ("kn", c.kn), ("vn", c.vn), ("kc", c.kc), ("vc", c.vc), ("table", dev(c.table)), ("lens", dev(c.lens)),
        ("starts", dev(c.starts)), ("shared", dev(c.shared)))]
    for bad in (dict(starts=dev([])), dict(shared=dev([1, 2])), dict(starts=dev([0, 2], np.int64)), dict(vc=c.kc[:1]),
                dict(lens=dev([1])), dict(kn=c.kn.float()), dict(shared=torch.zeros(1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            E.enc_prefix_attention(*args(**bad))
    with pytest.raises(E.EncError):
        E.enc_prefix_attention(*args(), ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(E.EncError):
        E.enc_prefix_attention(*args(), scale=float("nan"))
    out, lse = E.enc_prefix_attention(*args(q=c.q[:0], kn=c.kn[:0], vn=c.vn[:0]), return_lse=True)
    assert out.shape == (0, 2, 4, 64) and lse.shape == (0, 2, 4)


# ------------------------------------------------------------------ what sequences share
def shared_want(table, lens, page, seqs, starts):
    B = len(seqs)
    top, out = 0, []
    ends = []
    for s in starts:
        top = max(top, min(max(s, 0), B))
        ends.append(top)
    for a, b in zip(ends, ends[1:]):
        group = [int(s) for s in seqs[a:b]]
        if not group or any(not 0 <= s < len(lens) for s in group):
            out.append(0)
            continue
        least = min(min(max(int(lens[s]), 0), table.shape[1] * page) for s in group)
        n = 0
        while n < -(-least // page) and table[group[0], n] >= 0 and all(table[s, n] == table[group[0], n] for s in group):
            n += 1
        out.append(min(n * page, least))
    return out


@pytest.mark.parametrize("entries,page", [(1, 16), (40, 1), (2500, 16)])
def test_cache_shared(E, entries, page):
    say("shared", entries, page)
    rng = np.random.default_rng([5, entries, page])
    S = 12
    base = rng.permutation(entries * S).reshape(S, entries).astype(np.int32)
    table = base.copy()
    for s in range(1, S):                                              # leading entries of an earlier sequence
        n = int(rng.integers(0, entries + 1))
        table[s, :n] = table[s - 1, :n]
    lens = rng.integers(0, entries * page + 1, S).astype(np.int32)
    lens[3] = entries * page
    for s in range(S):
        table[s, -(-int(lens[s]) // page):] = -1
    cache = E.Cache(torch.zeros(1, entries * S, page, 8, dtype=BF, device="cuda"), dev(table), dev(lens),
                    torch.ones(entries * S, dtype=torch.int32, device="cuda"))
    for seqs, starts in ((range(S), [0, S]), (range(S), [0, 2, 4, 4, 9, S]), ([3, 3, 3], [0, 3]), (range(S), list(range(S + 1))),
                         ([0, 1, 99, 2, 3, -1], [0, 2, 3, 5, 6]), (range(S), [5, 2, 9, 4, 100, -3]), ([], [0, 0]), (range(4), [0])):
        got = E.enc_cache_shared(cache, dev(list(seqs)), dev(starts))
        assert got.tolist() == shared_want(table, lens, page, list(seqs), starts), (list(seqs), starts)


def test_cache_shared_after_forks(E):
    """What fork and commit leave: whole pages stay shared, the copied last one does not."""
    say("forks")
    cache = E.Cache.empty(2, 40, 16, (2, 64), 5, 8)
    one = lambda *x: dev(list(x))  # noqa: E731
    draft = torch.randn(2, 1, 70, 2, 64, device="cuda").to(BF)
    E.enc_cache_commit(cache, one(0), draft, torch.arange(70, dtype=torch.int32, device="cuda")[None], one(70))
    E.enc_cache_fork(cache, one(0, 0, 0), one(1, 2, 3))
    seqs, starts = one(0, 1, 2, 3), one(0, 4)
    assert E.enc_cache_shared(cache, seqs, starts).tolist() == [70]
    rows = torch.randn(2, 2, 3, 2, 64, device="cuda").to(BF)
    path = torch.arange(3, dtype=torch.int32, device="cuda").repeat(2, 1)
    E.enc_cache_commit(cache, one(1, 2), rows, path, one(3, 1))
    assert int(cache.status) == 0
    assert E.enc_cache_shared(cache, seqs, starts).tolist() == [64]
    assert E.enc_cache_shared(cache, one(0, 3), one(0, 2)).tolist() == [70]
    E.enc_cache_truncate(cache, one(3), one(20))
    assert E.enc_cache_shared(cache, seqs, starts).tolist() == [20]
    assert E.enc_cache_shared(cache, one(0, 4), one(0, 2)).tolist() == [0]
