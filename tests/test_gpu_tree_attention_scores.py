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


# ------------------------------------------------------------------ large scores
# Queries and keys are small whole numbers times powers of two, so that q.k is
# exact in 32 bits and the kernels' scores are the definition's but for the
# product with the scale. Rows up to 16 (32 in large batches) round that
# product, by 2^-24 of the score at most, in each weight: |err| grows by 2^-23
# max |score| sum p |v|. The wide kernel does not.
WIDE = [s for s in SHAPES if "waves" in s or "256" in s]
NARROW = [s for s in SHAPES if s not in WIDE]


class Whole(Case):
    """q.k = 2^exp n + at, n whole and small; `at` a column of its own."""

    def __init__(self, shape, dt, seed, exp=0):
        super().__init__(*SHAPES[shape], dt, seed=seed)
        g = torch.Generator().manual_seed(seed)
        small = lambda x: torch.randint(-1, 2, x.shape, generator=g).to(x.dtype).cuda()  # noqa: E731
        self.a, self.b = exp // 2, exp - exp // 2
        self.q, self.kn, self.kc = small(self.q) * 2.0 ** self.a, small(self.kn) * 2.0 ** self.b, small(self.kc) * 2.0 ** self.b
        self.g = g

    def column(self, d, q, k, spread=0, step=1):
        """Column d of every query q, of every key k - step {0 .. spread}."""
        for x in (self.kn, self.kc):
            x[..., d] = k - step * torch.randint(0, spread + 1, x.shape[:-1], generator=self.g).to(x.dtype).cuda()
        self.q[..., d] = q

    def verdict(self, E, slack=0.0, **kw):
        """As Case.check, with `slack` more for the weights."""
        out, lse = self.run(E, **kw)
        want, wl, size = self.want(**kw)
        u = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[out.dtype]
        g, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        bad = ~(abs(g - want) <= u * abs(want) + (u + 2.0 ** -10 + slack) * size + 1e-30)
        assert not bad.any(), "%d of %d outside" % (bad.sum(), bad.size)
        fin = abs(wl) < float("inf")
        assert (abs(gl - wl)[fin] <= 2.0 ** -11 + 2.0 ** -20 * abs(wl[fin])).all()
        assert (gl[~fin] == -float("inf")).all() and (g[~fin] == 0).all()


def extra(shape, top):
    return 0.0 if shape in WIDE else 2.0 ** -23 * top


@pytest.mark.parametrize("dt,exp", [(torch.bfloat16, e) for e in (20, 27, 30, 100, 120)]
                         + [(torch.float16, e) for e in (20, 27, 30)])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_large_scores(E, shape, dt, exp):
    """n is some 10 and the scale near 0.1: scores about 1e6, 1e8, 1e9, 1e30,
    1e36. The largest outweighs all others; equal ones share."""
    say("attention large scores", shape, dt, exp)
    c = Whole(shape, dt, 41, exp)
    c.verdict(E)
    c.scale *= -1
    c.verdict(E)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("bits", [14, 18, 20, 22])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_smooth_weights_far_from_zero(E, shape, bits, sign, dt):
    """All scores far from 0 together, their differences ordinary ones."""
    say("attention scores far from 0", shape, bits, sign, dt)
    c = Whole(shape, dt, 42)
    c.column(0, 2.0 ** (bits // 2), sign * 2.0 ** (bits - bits // 2))
    c.verdict(E, extra(shape, (2.0 ** bits + 300) * c.scale))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_where_the_arithmetic_changes(E, shape, sign, dt):
    """Scores of 2^16 powers of two, some keys on each side, in every part."""
    say("attention scores around 2^16", shape, sign, dt)
    c = Whole(shape, dt, 43)
    c.scale = 128 ** -0.5                          # 2^16 at q.k = 513935
    c.column(0, 512.0, sign * 1004.0)              # 514048
    c.column(1, 1.0, 0.0, 127, sign * 2)           # down to 513794
    c.verdict(E, extra(shape, 514348 * c.scale))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("down", [False, True])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_scores_that_grow_along_the_history(E, shape, down, dt):
    """Each page's keys outweigh the page's before (or after) by far, from
    ordinary scores to 2^22."""
    say("attention growing scores", shape, down, dt)
    c = Whole(shape, dt, 44)
    c.q[..., 0] = 2.0 ** 11
    c.kn[..., 0] = 0 if down else 2.0 ** 11
    for row, n in zip(c.table, c.lens):
        held = row[:-(-n // c.page)]
        for i, page in enumerate(held):
            at = len(held) - 1 - i if down else i
            c.kc[int(page), :, :, 0] = 2.0 ** min(at, 11) if at else 0
    c.verdict(E, extra(shape, (2.0 ** 22 + 300) * c.scale))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_lowest_values(E, shape, dt):
    """Scores at the type's lowest value, all of them: the mean of what is seen."""
    say("attention lowest values", shape, dt)
    c = Case(*SHAPES[shape], dt, seed=45)
    c.q[:] = 0
    c.q[..., 0] = 1
    c.kc[..., 0] = torch.finfo(dt).min
    c.kn[..., 0] = torch.finfo(dt).min
    c.scale = 1.0
    Whole.verdict(c, E)
    c.q[..., 0] = -1                               # and at the highest
    Whole.verdict(c, E)


@pytest.mark.parametrize("scale", [1e-38, 1e30, 3.4e38])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_scales_at_the_ends(E, shape, scale):
    say("attention scale", scale, shape)
    c = Whole(shape, torch.bfloat16, 46, 0 if scale < 1 else -120)
    c.scale = scale
    c.verdict(E)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_one_key_that_outweighs_all(E, shape, dt):
    say("attention sharp", shape, dt)
    for part in (0.0, 0.3, 0.99):
        c = Case(*SHAPES[shape], dt, seed=47)
        b = int(c.lens.argmax())
        at = int(part * c.lens[b])
        page, row = int(c.table[b, at // c.page]), at % c.page
        c.kc[page, row, 0] = 30 * c.q[b, 0, 0]
        out, _ = c.run(E)
        # every other score is 30 |q|^2 scale - 6 |q| or more below, far past 2^-24
        assert (out[b, 0, 0].float() - c.vc[page, row, 0].float()).abs().max() <= 2.0 ** -7 * 4


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", NARROW)
def test_only_the_result_is_rounded(E, shape, dt):
    """Up to 16 rows (32 in large batches) weights count in more than 16 bits.
    Scores are exact here, exponentials good to 2^-19 of themselves, what is
    left of a weight in two parts is 2^-18, and a sum of n fp32 terms is off by
    n 2^-24 at most (130 keys): 2^-15 of sum p |v| bounds them all, beside the
    result's own rounding, 2^-8 (BF16) or 2^-11 of it, or 2^-25 in FP16."""
    say("attention rounding", shape, dt)
    c = Whole(shape, dt, 48)
    out, _ = c.run(E)
    want, _, size = c.want()
    u = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[dt]
    g = out.double().cpu().numpy()
    bad = ~(abs(g - want) <= u * abs(want) + 2.0 ** -15 * size + (2.0 ** -25 if dt == torch.float16 else 0))
    assert not bad.any(), "%d of %d outside" % (bad.sum(), bad.size)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", list(SHAPES))
def test_infinite_cached_values(E, shape, dt):
    """Every row of the sequence sees them: infinities of the value's sign, no
    number where both meet or a value is none, and nothing anywhere else."""
    say("attention infinite cached values", shape, dt)
    c = Case(*SHAPES[shape], dt, seed=49)
    base, lse = c.run(E)
    b = int(c.lens.argmax())
    n = int(c.lens[b])
    inf = float("inf")
    at = lambda t: (int(c.table[b, t // c.page]), t % c.page)  # noqa: E731
    for t, d, x in ((0, 1, inf), (n // 2, 3, -inf), (n - 1, 6, inf), (3, 9, inf), (n - 2, 9, -inf), (n // 3, 12, float("nan"))):
        c.vc[at(t) + (slice(None), d)] = x
    out, l2 = c.run(E)
    assert torch.equal(lse, l2)
    got = out[b].float()
    assert (got[..., 1] == inf).all() and (got[..., 3] == -inf).all() and (got[..., 6] == inf).all()
    assert got[..., [9, 12]].isnan().all()
    rest = [d for d in range(c.D) if d not in (1, 3, 6, 9, 12)]
    # finite places differ at most by what rounding the weights does
    u = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[dt]
    want, _, size = c.want()
    bad = ~(abs(out.double().cpu().numpy() - want) <= u * abs(want) + (u + 2.0 ** -10) * size + 1e-30)
    assert not bad[b][..., rest].any()
    others = [i for i in range(c.B) if i != b]
    assert torch.equal(out[others], base[others])


@pytest.mark.parametrize("x", [float("inf"), 1e4])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", [s for s in SHAPES if SHAPES[s][1] > 1])
def test_keys_that_a_row_does_not_see(E, shape, dt, x):
    """Scores of infinity, or large ones, in other rows change nothing, to the bit."""
    say("attention, keys of other rows", shape, dt, x)
    c = Case(*SHAPES[shape], dt, seed=50)
    j = c.T // 2
    c.seen[:, j, j] = True
    base, lse = c.run(E)
    c.kn[:, j, :, 5] = x
    out, l2 = c.run(E)
    sees = torch.from_numpy(c.seen[:, :, j]).cuda()
    assert bool(sees.any()) and not bool(sees.all())
    assert torch.equal(out[~sees], base[~sees]) and torch.equal(l2[~sees], lse[~sees])
