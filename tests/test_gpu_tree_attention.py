"""enc_tree_attention on the GPU against the formula in 64 bits.

Tolerance, derived: with u the rounding unit of the type (2^-8 BF16, 2^-11
FP16), the result's rounding is u |o|; each weight p is rounded to that type
(u p |v| each, at most); scores are fp32 sums of at most 256 exact products,
off by less than 256 2^-24 sum |q k| scale, which for the inputs here (|q|,
|k| about 1 a value) is below 2^-11 absolute and so relative in p. Together
|err| <= u |o| + (u + 2^-10) sum p |v|, and the log-sum-exp is off by less than
2^-11 + 2^-20 |lse|."""
import sys

import numpy as np
import pytest

import step_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


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


class Case:
    def __init__(self, B, T, H, G, D, lens, page, dt=torch.bfloat16, seed=0, extra_pages=2, width=None):
        rng = np.random.default_rng([21, seed, B, T, H, G, D, page])
        self.B, self.T, self.H, self.G, self.D, self.page = B, T, H, G, D, page
        self.lens = np.array(lens, np.int32)
        S = len(lens)
        need = [-(-n // page) for n in lens]
        n_pages = sum(need) + extra_pages
        order = rng.permutation(n_pages)
        self.table = np.full((S, width or max(max(need), 1)), -1, np.int32)
        at = 0
        for s in range(S):
            self.table[s, :need[s]] = order[at:at + need[s]]
            at += need[s]
        t = lambda *shape: torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dt).cuda()  # noqa: E731
        self.q, self.kn, self.vn = t(B, T, H, D), t(B, T, G, D), t(B, T, G, D)
        self.kc, self.vc = t(n_pages, page, G, D), t(n_pages, page, G, D)
        parents = np.full((B, T), -1, np.int32)
        for i in range(1, T):
            parents[:, i] = rng.integers(0, i, B)
        self.seen = ref.ancestors(parents)
        self.scale = D ** -0.5

    def run(self, E, mask=True, seqs=None, nodes=None, **kw):
        c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        out, lse = E.enc_tree_attention(self.q, self.kn, self.vn, self.kc, self.vc, c(self.table), c(self.lens),
                                        mask=c(ref.mask_words(self.seen)) if mask else None,
                                        seqs=None if seqs is None else c(np.array(seqs, np.int32)),
                                        nodes=None if nodes is None else c(np.array(nodes, np.int32)),
                                        scale=self.scale, return_lse=True, **kw)
        torch.cuda.synchronize()
        return out, lse

    def want(self, mask=True, seqs=None, nodes=None):
        d = lambda x: x.double().cpu().numpy()  # noqa: E731
        seen = self.seen if mask else np.tril(np.ones((self.T, self.T), bool))[None].repeat(self.B, 0)
        return ref.tree_attention(d(self.q), d(self.kn), d(self.vn), d(self.kc), d(self.vc), self.table, self.lens, seen,
                                  self.scale, seqs, nodes)

    def check(self, E, **kw):
        out, lse = self.run(E, **kw)
        kw.pop("ws", None)
        want, wl, size = self.want(**kw)
        u = U[out.dtype]
        g, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        bad = ~(np.abs(g - want) <= u * np.abs(want) + (u + 2.0 ** -10) * size + 1e-30)
        assert not bad.any(), "%d of %d outside, worst %g" % (bad.sum(), bad.size, np.nanmax(np.abs(g - want)))
        fin = np.isfinite(wl)
        assert np.array_equal(fin, np.isfinite(gl))
        assert (np.abs(gl - wl)[fin] <= 2.0 ** -11 + 2.0 ** -20 * np.abs(wl[fin])).all()
        assert (gl[~fin] == -np.inf).all() and (g[~fin] == 0).all()
        return out, lse


@pytest.mark.parametrize("B,T,H,G,D,lens,page,dt", [
    (1, 1, 1, 1, 64, [0], 16, torch.bfloat16),              # nothing cached: the node itself
    (1, 1, 4, 1, 128, [1], 16, torch.bfloat16),
    (2, 1, 8, 2, 128, [31, 33], 16, torch.float16),         # around a strip of 32
    (3, 1, 32, 8, 128, [1021, 64, 500], 16, torch.bfloat16),
    (2, 5, 4, 2, 64, [17, 100], 1, torch.bfloat16),         # pages of one token
    (2, 7, 6, 2, 96, [40, 129], 20, torch.float16),         # pages that end inside a tile
    (1, 16, 4, 1, 128, [300], 48, torch.bfloat16),
    (2, 33, 4, 4, 64, [65, 0], 7, torch.float16),
    (1, 64, 8, 2, 128, [700], 64, torch.bfloat16),          # 256 rows a KV head: four waves of them
    (1, 100, 7, 1, 64, [130], 16, torch.bfloat16),          # 700 rows: several tiles
    (1, 256, 2, 1, 64, [40], 16, torch.bfloat16),           # the largest tree
    (2, 3, 2, 1, 256, [50, 3], 16, torch.bfloat16),
    (1, 40, 2, 1, 256, [90], 16, torch.float16),
    (2, 4, 3, 3, 8, [20, 45], 16, torch.bfloat16),          # heads smaller than a fragment
    (1, 6, 2, 2, 80, [77], 16, torch.float16),
    (1, 9, 4, 2, 200, [77], 32, torch.bfloat16),
    (1, 2, 2, 1, 64, [3], 4096, torch.bfloat16),            # a page larger than the history
])
def test_against_formula(E, B, T, H, G, D, lens, page, dt):
    say("attention", B, T, H, G, D, lens, page, dt)
    Case(B, T, H, G, D, lens, page, dt).check(E)


@pytest.mark.parametrize("T", [1, 2, 40])
def test_chain_without_a_mask(E, T):
    say("attention chain", T)
    Case(2, T, 4, 2, 128, [50, 0], 16, seed=1).check(E, mask=False)


def test_table_far_wider_than_the_histories(E):
    say("attention wide table")
    Case(2, 5, 8, 2, 128, [70, 3000], 16, seed=2, width=4000).check(E)


def test_sequences_by_index_and_live_nodes(E):
    say("attention seqs, nodes")
    c = Case(4, 9, 4, 2, 64, [10, 200, 33], 16, seed=3)
    # an index outside the table: no cached tokens; live nodes clamped to [0, 9]
    c.check(E, seqs=[2, 1, 7, -1], nodes=[9, 4, 3, 12])
    c.check(E, seqs=[0, 0, 1, 2], nodes=[0, 1, -5, 9])


def test_rows_that_see_nothing(E):
    say("attention empty rows")
    c = Case(2, 6, 4, 2, 128, [0, 20], 16, seed=4)
    c.seen[:, 2] = False
    c.seen[:, 4, :] = False
    c.check(E)


def test_any_mask_not_only_trees(E):
    say("attention random mask")
    c = Case(2, 70, 4, 2, 64, [0, 45], 16, seed=5)
    c.seen = np.random.default_rng(5).random(c.seen.shape) < 0.3
    c.check(E)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,H,D", [(6, 4, 128), (40, 4, 64), (5, 2, 256), (6, 2, 40)])
def test_nonfinite_where_a_row_may_not_look(E, dt, T, H, D):
    """Infinities and NaN behind the history's end, in pages of nobody and in
    nodes that a row does not see leave it alone; rows that see them get what
    the formula gives."""
    say("attention non-finite", dt, T, H, D)
    c = Case(2, T, H, 2, D, [45, 0], 16, dt, seed=6)
    base, blse = c.check(E)
    used = np.zeros((c.kc.shape[0], 16), bool)
    for j in range(45):
        used[c.table[0, j // 16], j % 16] = True
    for x, bad in ((c.kc, float("nan")), (c.vc, float("inf"))):
        x[torch.from_numpy(~used).cuda()] = bad
    out, lse = c.run(E)
    assert torch.equal(out, base) and torch.equal(lse, blse)
    j = 3
    c.vn[:, j, :, 1] = float("inf")
    c.vn[:, j, :, 3] = float("nan")
    c.vn[:, j, :, D - 1] = -float("inf")
    out, _ = c.run(E)
    sees = torch.from_numpy(c.seen[:, :, j]).cuda()
    assert torch.equal(out[~sees], base[~sees])
    rows = out[sees].float()
    assert rows[..., 3].isnan().all() and (rows[..., 1] == float("inf")).all() and (rows[..., D - 1] == -float("inf")).all()
    keep = [d for d in range(D) if d not in (1, 3, D - 1)]
    assert torch.equal(out[sees][..., keep], base[sees][..., keep])
    c.kn[:, j] = float("nan")
    out, _ = c.run(E)
    assert torch.equal(out[~sees], base[~sees]) and out[sees].isnan().all()


def test_infinity_in_the_last_cached_row(E):
    say("attention infinite value in a partial strip")
    c = Case(1, 3, 2, 1, 64, [37], 16, seed=7)
    c.vc[c.table[0, 36 // 16], 36 % 16, 0, 5] = float("inf")
    out, _ = c.run(E)
    assert (out[..., 5] == float("inf")).all() and out[..., :5].isfinite().all() and out[..., 6:].isfinite().all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_sharp_scores_and_lowest_values(E, dt):
    """One key that outweighs all others by far, anywhere in the history, and
    scores at the type's lowest value."""
    say("attention sharp", dt)
    for at in (0, 31, 32, 150, 299):
        c = Case(1, 4, 2, 1, 64, [300], 16, dt, seed=8)
        c.kc[c.table[0, at // 16], at % 16, 0] = 30 * c.q[0, 0, 0]
        out, lse = c.run(E)
        assert (out[0, 0, 0].float() - c.vc[c.table[0, at // 16], at % 16, 0].float()).abs().max() <= 2 * U[dt] * 4
    c = Case(1, 2, 2, 1, 64, [64], 16, dt, seed=9)
    c.q[:] = 0
    c.q[..., 0] = 1
    c.kc[..., 0] = torch.finfo(dt).min
    c.kn[..., 0] = torch.finfo(dt).min
    c.scale = 1.0
    out, _ = c.run(E)       # equal scores, however low: the mean of what is seen
    want, _, size = c.want()
    assert (np.abs(out.double().cpu().numpy() - want) <= U[dt] * np.abs(want) + (U[dt] + 2.0 ** -10) * size).all()


def test_strides_and_orders(E):
    say("attention strides")
    c = Case(2, 5, 4, 2, 64, [45, 80], 16, seed=10)
    base, _ = c.check(E)
    n = c.kc.shape[0]
    both = torch.zeros(n, 2, 2, 16, 64, dtype=c.kc.dtype, device="cuda")   # page, (K, V), head, token, value
    both[:, 0], both[:, 1] = c.kc.transpose(1, 2), c.vc.transpose(1, 2)
    c.kc, c.vc = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    packed = torch.zeros(2, 5, 8, 64, dtype=c.q.dtype, device="cuda")
    packed[:, :, :4], packed[:, :, 4:6], packed[:, :, 6:] = c.q, c.kn, c.vn
    c.q, c.kn = packed[:, :, :4], packed[:, :, 4:6]
    c.vn = c.vn.transpose(1, 2).contiguous().transpose(1, 2)               # other strides than k_new
    store = torch.full((2, 5, 6, 64), 7.0, dtype=c.q.dtype, device="cuda")
    out, _ = c.run(E, out=store[:, :, 1:5])
    assert torch.equal(out, base) and (store[:, :, 0] == 7).all() and (store[:, :, 5] == 7).all()


def test_table_entries_outside_are_not_followed(E):
    say("attention bad table")
    c = Case(2, 3, 2, 1, 64, [45, 80], 16, seed=11)
    base, _ = c.run(E)
    c.table[0, 1], c.table[0, 2] = -3, 2 ** 30
    out, _ = c.run(E)
    assert torch.equal(out[1], base[1])
    c.lens[0] = 2 ** 31 - 1                        # clamped to the table
    c.run(E)
    c.lens[0] = -7
    assert c.run(E)[0].isfinite().all()


def test_equal_inputs_give_equal_bits_and_shared_workspaces(E):
    say("attention repeat")
    a, b = Case(1, 4, 8, 2, 128, [2000], 16, seed=12), Case(1, 4, 8, 2, 128, [2000], 16, seed=13)
    dev = lambda c: (c.q, c.kn, torch.from_numpy(c.table).cuda(), c.kc)  # noqa: E731
    ws = E.tree_attention_workspace(*dev(a))
    ws.fill_(0xFF)                                 # any contents
    first = a.run(E, ws=ws)[0].clone()
    b.run(E, ws=ws)
    assert torch.equal(a.run(E, ws=ws)[0], first)


def test_in_a_graph(E):
    say("attention in a graph")
    c = Case(2, 5, 8, 2, 128, [700, 90], 16, seed=14)
    d = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    table, lens, mask = d(c.table), d(c.lens), d(ref.mask_words(c.seen))
    ws = E.tree_attention_workspace(c.q, c.kn, table, c.kc)
    out = torch.empty_like(c.q)
    call = lambda: E.enc_tree_attention(c.q, c.kn, c.vn, c.kc, c.vc, table, lens, mask=mask, out=out, ws=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for rep in range(3):
        lens.copy_(torch.tensor([700 - 100 * rep, 90 + rep], dtype=torch.int32))   # the history moves on
        c.lens = lens.cpu().numpy()
        eager = c.run(E)[0]
        out.fill_(float("nan"))
        ws.fill_(0x55)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), rep


def test_offsets_past_32_bits(E):
    """A cache above 4 GiB: rows whose byte offset does not fit 32 bits."""
    say("attention large cache")
    pages, page, G, D = 20000, 128, 1, 1024 // 4
    kc = torch.zeros(pages, page, G, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    assert kc.numel() * 2 > 1 << 30
    rng = np.random.default_rng(15)
    table = np.array([[19999, 0, 16384, 8192]], np.int32)
    small_k, small_v = (torch.from_numpy(rng.standard_normal((4, page, G, D)).astype(np.float32)).bfloat16().cuda()
                        for _ in "kv")
    kc[torch.from_numpy(table[0]).long().cuda()], vc[torch.from_numpy(table[0]).long().cuda()] = small_k, small_v
    q = torch.randn(1, 2, 2, D, device="cuda").bfloat16()
    kn, vn = torch.randn(1, 2, 1, D, device="cuda").bfloat16(), torch.randn(1, 2, 1, D, device="cuda").bfloat16()
    lens = torch.tensor([500], dtype=torch.int32, device="cuda")
    wide = kc.view(pages // 8, page * 8, G, D)[:, :page], vc.view(pages // 8, page * 8, G, D)[:, :page]
    want = E.enc_tree_attention(q, kn, vn, small_k, small_v, torch.arange(4, dtype=torch.int32, device="cuda")[None], lens)[0]
    got = E.enc_tree_attention(q, kn, vn, kc, vc, torch.from_numpy(table).cuda(), lens)[0]
    assert torch.equal(got, want)
    # the same through a strided view whose pages are 8 times as far apart
    t2 = torch.tensor([[2048, 0, 1024, 512]], dtype=torch.int32, device="cuda")
    wide[0][t2[0].long()], wide[1][t2[0].long()] = small_k, small_v
    got = E.enc_tree_attention(q, kn, vn, wide[0], wide[1], t2, lens)[0]
    assert torch.equal(got, want)


MANY = [(128, 3, 8, 4, 128, torch.bfloat16),    # 6 rows to a KV head, four heads to a workgroup
        (128, 5, 8, 4, 72, torch.float16),      # 10, heads of 72
        (128, 7, 16, 4, 128, torch.bfloat16),   # 28
        (130, 8, 12, 4, 64, torch.float16),     # 24, a batch that ends inside a wave
        (128, 2, 8, 4, 200, torch.bfloat16),    # 4, heads of 200
        (128, 4, 20, 5, 128, torch.bfloat16),   # five KV heads: not in fours
        (32, 25, 16, 4, 128, torch.bfloat16),   # 100, two to a wave's fragments
        (32, 25, 16, 4, 40, torch.float16),
        (40, 30, 16, 4, 64, torch.bfloat16)]    # 120


@pytest.mark.parametrize("B,T,H,G,D,dt", MANY)
def test_many_sequences(E, B, T, H, G, D, dt):
    say("attention, many sequences", B, T, H, G, D, dt)
    c = Case(B, T, H, G, D, [700 if b == 5 else b * 7 % 90 for b in range(B)], 16, dt, seed=5)
    live = [(b * 5) % (T + 1) for b in range(B)]
    c.check(E)
    c.check(E, nodes=live)


@pytest.mark.parametrize("B,T,H,G,D,dt", MANY)
def test_many_sequences_nonfinite_where_a_row_may_not_look(E, B, T, H, G, D, dt):
    say("attention, many sequences, NaN", B, T, H, G, D, dt)
    c = Case(B, T, H, G, D, [700 if b == 5 else b * 7 % 90 for b in range(B)], 16, dt, seed=6)
    c.seen[:, :T - 1, T - 1] = False
    clean, clean_lse = c.run(E)
    c.kn[:, T - 1], c.vn[:, T - 1] = float("nan"), float("inf")
    out, lse = c.run(E)
    assert torch.equal(out[:, :T - 1], clean[:, :T - 1]) and torch.equal(lse[:, :T - 1], clean_lse[:, :T - 1])
    assert torch.isnan(out[:, T - 1].float()).all()
