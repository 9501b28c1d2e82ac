"""enc_sample on the GPU against its definition in 64 bits.

Tokens and the set that is kept have to be equal: cumulative sums on either side
are off by some 2^-33 of a weight, at random, and a border between two tokens lies
that close to a random u, or to a top-p, in less than 1e-5 of the rows. Borders that are met
exactly are tested where both sides' arithmetic is exact (equal logits).
Probabilities are a quotient of fp64 values, rounded to fp32 (2^-24), then to
the output's type; the sum's weights are rounded to 2^-33 each (a whole number of
2^-32 that is at least 2^32), exponents of up to 2^10 are fp64: 2^-32 in all. Below e^-47 of the greatest (2^-67) a probability may be 0."""
import itertools
import sys

import numpy as np
import pytest

import continuation_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF: 2.0 ** -8, FP: 2.0 ** -11, F32: 2.0 ** -24}
TINY = {BF: 0.0, FP: 2.0 ** -25, F32: 0.0}


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


def settings_of(n, T=None, k=None, p=None, m=None):
    """Lists (or None) -> keyword arguments for the call."""
    f = lambda x, dt: None if x is None else torch.tensor(x, dtype=dt, device="cuda")  # noqa: E731
    return dict(temperature=f(T, F32), top_k=f(k, torch.int32), top_p=f(p, F32), min_p=f(m, F32))


def check(E, logits, u, T=None, k=None, p=None, m=None, probs_dtype=F32, **kw):
    rows, V = logits.shape
    s = settings_of(rows, T, k, p, m)
    token, probs = E.enc_sample(logits, u, return_probs=True, probs_dtype=probs_dtype, **s, **kw)
    torch.cuda.synchronize()
    alone, none = E.enc_sample(logits, u, **s)
    assert none is None and torch.equal(alone, token)
    l, got, uu = logits.double().cpu().numpy(), probs.double().cpu().numpy(), u.double().cpu().numpy()
    at = lambda name, r, otherwise: otherwise if s[name] is None else float(s[name][r // (rows // len(s[name]))])  # noqa: E731
    for r in range(rows):
        setting = at("temperature", r, 1.0), int(at("top_k", r, 0)), at("top_p", r, 1.0), at("min_p", r, 0.0)
        e = ref.kept_weights(l[r], *setting)
        ur = min(max(uu[r], 0.0), 1.0) if uu[r] == uu[r] else 0.0
        assert int(token[r]) == ref.draw(e, ur), (r, setting, uu[r])
        want = e / max(e.sum(), 1e-300)
        bound = want * (U[probs_dtype] + 2.0 ** -24 + 2.0 ** -32) + TINY[probs_dtype] + 2.0 ** -67 + 2.0 ** -149
        bad = ~(np.abs(got[r] - want) <= bound)
        assert not bad.any(), (r, setting, int(bad.sum()), np.nonzero(bad)[0][:4], got[r][bad][:4], want[bad][:4])
    return token, probs


def rows_of(rows, V, dtype=F32, seed=0, sigma=3.0):
    g = torch.Generator().manual_seed(seed)
    return (sigma * torch.randn(rows, V, generator=g)).to(dtype).cuda(), torch.rand(rows, generator=g).cuda()


MIX = dict(T=[1.0, 0.7, 1.3, 0.0, 0.5, 1.0, 2.0, 0.9], k=[0, 50, 1, 7, 3, 1000, 0, 20],
           p=[0.9, 0.95, 1.0, 0.5, 0.99, 0.8, 0.3, 1.0], m=[0.0, 0.05, 0.0, 0.3, 0.0, 0.01, 0.2, 0.1])


@pytest.mark.parametrize("V", [1, 2, 3, 63, 257, 1000, 4089, 4096, 4097, 16384, 32003, 50001, 128256])
def test_sizes(E, V):
    say("sizes", V)
    l, u = rows_of(8, V, seed=V)
    check(E, l, u)
    check(E, l, u, **MIX)


@pytest.mark.parametrize("dtype,probs_dtype", itertools.product((F32, BF, FP), repeat=2))
@pytest.mark.parametrize("V", [777, 20000])
def test_types(E, dtype, probs_dtype, V):
    say("types", dtype, probs_dtype, V)
    l, u = rows_of(8, V, dtype, 3)
    check(E, l, u, probs_dtype=probs_dtype, **MIX)


@pytest.mark.parametrize("names", [c for n in range(1, 5) for c in itertools.combinations("Tkpm", n)])
@pytest.mark.parametrize("sigma", [0.5, 4.0])
def test_each_filter(E, names, sigma):
    say("filters", names, sigma)
    l, u = rows_of(8, 30000, seed=5, sigma=sigma)
    check(E, l, u, **{n: MIX[n] for n in names})


@pytest.mark.parametrize("V", [1, 2, 7, 4501])
@pytest.mark.parametrize("dtype,pad,lead", [(F32, 3, 0), (F32, 0, 1), (BF, 5, 3), (FP, 1, 7), (BF, 0, 0), (F32, 4, 0)])
def test_strides_and_alignment(E, dtype, pad, lead, V):
    """Rows longer than they need be, any base: neighbours are neither read as logits nor written."""
    say("strides", dtype, pad, lead, V)
    rows = 5
    buf = torch.full((lead + rows * (V + pad) + 8,), 60.0, dtype=dtype, device="cuda")
    l = buf[lead:lead + rows * (V + pad)].view(rows, V + pad)[:, :V]
    src, u = rows_of(rows, V, dtype, 11)
    l.copy_(src)
    out = torch.full((lead + rows * (V + pad) + 8,), 7.0, dtype=dtype, device="cuda")
    probs = out[lead:lead + rows * (V + pad)].view(rows, V + pad)
    check(E, l, u, T=[0.8] * 5, k=[40, 0, 3, 0, 0], p=[0.9, 0.9, 1.0, 0.5, 1.0], probs_dtype=dtype, probs=probs[:, :V])
    assert (probs[:, V:] == 7).all() and (out[:lead] == 7).all() and (out[lead + rows * (V + pad):] == 7).all()


@pytest.mark.parametrize("V", [10, 1000, 5000, 40000])
def test_equal_logits(E, V):
    """All weights 1: borders are met exactly, ties go to the lowest index; more of them than are gathered."""
    say("equal", V)
    l = torch.full((8, V), -3.7, device="cuda")
    u = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0 - 2.0 ** -24, 1.0, 0.5, 0.125], device="cuda")
    check(E, l, u)
    check(E, l, u, p=[0.5, 0.25, 0.125, 0.75, 0.5, 0.5, 0.0, 0.0625])
    check(E, l, u, k=[1, 2, V // 2, V - 1, V, V + 5, -3, V // 2 + 1])
    check(E, l, u, k=[4, 8, V // 2 // 2 * 2, 0, 2, 1, 6, 10], p=[0.5, 0.25, 0.5, 0.5, 0.5, 0.5, 1.0, 0.5], m=[1.0] * 8)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_coarse_logits(E, dtype):
    """Few distinct values, thousands of each: cuts inside ties."""
    say("coarse", dtype)
    l, u = rows_of(8, 60000, F32, 21)
    l = (torch.round(l * 2) / 2).to(dtype)
    check(E, l, u, **MIX)
    check(E, l, u, k=[100, 1000, 3000, 5000, 20000, 59999, 10, 2])
    check(E, l, u, T=[3.0] * 8, k=[30000] * 8, p=[0.1, 0.3, 0.5, 0.7, 0.9, 0.99, 0.999, 0.01])


def test_flat_and_sharp(E):
    """Temperatures from almost none to infinite."""
    say("flat")
    l, u = rows_of(8, 20000, F32, 22)
    T = [1e-6, 1e-3, 0.05, 20.0, 1e3, 1e6, 1e-38, 3e38]
    check(E, l, u, T=T)
    check(E, l, u, T=T, p=[0.9] * 8)
    check(E, l, u, T=T, k=[300] * 8, p=[0.5] * 8, m=[0.1] * 8)
    same = torch.zeros(2, 5000, device="cuda")
    check(E, same, u[:2], T=[float("inf"), float("inf")], p=[0.5, 1.0])
    mixed = l[:2, :5000].clone()
    token, probs = E.enc_sample(mixed, u[:2], temperature=torch.full((2,), float("inf"), device="cuda"), return_probs=True)
    assert torch.allclose(probs, torch.full_like(probs, 1 / 5000), rtol=1e-6)
    assert token.tolist() == [int(float(x) * 5000) for x in u[:2].double()]


def test_special_values(E):
    """NaN, infinities, rows without anything, zeros of both signs, the largest finite values."""
    say("special")
    l, u = rows_of(12, 6000, F32, 23)
    nan, inf = float("nan"), float("inf")
    l[0, ::2] = nan
    l[1, :5990] = -inf
    l[2] = -inf
    l[3] = nan
    l[4, 17] = inf
    l[5, 100::1000] = inf
    l[6] = 0.0
    l[6, ::3] = -0.0
    l[7] *= 1e37
    l[8] = 3.4e38
    l[8, 5] = -3.4e38
    l[9, 1:] = -inf
    l[10, :] = nan
    l[10, 4000] = -1e30
    l[11] *= 1e-42
    for kw in (dict(), dict(k=[2] * 12), dict(p=[0.5] * 12), dict(m=[0.5] * 12), dict(T=[0.0] * 12),
               dict(T=[0.5] * 12, k=[900] * 12, p=[0.9] * 12, m=[0.001] * 12)):
        token, probs = check(E, l, u, **kw)
        assert token[2] == token[3] == -1 and not probs[2:4].any()
        assert token[9] == 0 and token[10] == 4000 and token[4] == 17


def test_odd_settings(E):
    """Settings outside their ranges, NaN among them, and numbers u at and past their ends."""
    say("settings")
    l, u = rows_of(8, 3000, F32, 24)
    nan, inf = float("nan"), float("inf")
    u = torch.tensor([0.0, 1.0, nan, -1.0, 2.0, inf, 1.0 - 2.0 ** -24, 1e-30], device="cuda")
    token, _ = check(E, l, u)
    token, probs = E.enc_sample(l, u, temperature=torch.full((8,), nan, device="cuda"), return_probs=True)
    assert torch.equal(token.long(), l.argmax(1)) and torch.equal(probs, torch.nn.functional.one_hot(l.argmax(1), 3000).float())
    token, _ = check(E, l, u, T=[-1.0] * 8)
    token, probs = check(E, l, u, k=[-5, 0, 2 ** 31 - 1, -2 ** 31, 3000, 2999, 3001, 1], p=[1.5, inf, 1.0, 2.0, 1.0, 1.0, 1.0, 1.0],
                         m=[-1.0, -inf, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0])
    a = E.enc_sample(l, u, return_probs=True)
    for name in ("top_p", "min_p"):
        b = E.enc_sample(l, u, return_probs=True, **{name: torch.full((8,), nan, device="cuda")})
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check(E, l, u, p=[0.0, -1.0, 1e-30, 1e-7, 1.0 - 2.0 ** -24, 0.999999, -inf, 0.5])
    check(E, l, u, m=[1.0, 1.5, inf, 1e-30, 0.999, 1e-10, 1e-20, 0.5])


def test_settings_of_several_rows(E):
    say("shared settings")
    l, u = rows_of(12, 2000, F32, 25)
    for n in (1, 2, 3, 4, 6, 12):
        check(E, l, u, T=MIX["T"][:n] if n <= 8 else [0.9] * n, k=([50, 3, 0, 10, 5, 1] * 2)[:n], p=[0.9] * n)


def test_large_vocabulary(E):
    say("2^22")
    g = torch.Generator(device="cuda").manual_seed(4)
    l = 2.0 * torch.randn(2, 1 << 22, device="cuda", generator=g)
    u = torch.tensor([0.3, 0.9], device="cuda")
    check(E, l, u, T=[1.0, 0.8], k=[0, 100000], p=[0.9, 0.95])
    check(E, l.bfloat16(), u, T=[1.0, 0.8], k=[0, 100000], p=[0.9, 0.95])


def test_many_rows(E):
    """More rows than the workspace holds at a time; a row's answer does not depend on the others."""
    say("many rows")
    l, u = rows_of(2500, 300, F32, 26)
    s = dict(temperature=torch.full((2500,), 0.8, device="cuda"), top_p=torch.full((2500,), 0.9, device="cuda"))
    token, probs = E.enc_sample(l, u, return_probs=True, **s)
    for r in (0, 1, 1023, 1024, 2047, 2048, 2499):
        one = {n: t[r:r + 1] for n, t in s.items()}
        t1, p1 = E.enc_sample(l[r:r + 1], u[r:r + 1], return_probs=True, **one)
        assert torch.equal(t1, token[r:r + 1]) and torch.equal(p1, probs[r:r + 1])
    want = torch.tensor([ref.draw(ref.kept_weights(x, float(np.float32(0.8)), 0, float(np.float32(0.9)), 0.0), float(w))
                         for x, w in zip(l.double().cpu().numpy(), u.double().cpu().numpy())])
    assert torch.equal(token.cpu().long(), want)


def test_rows_alone_and_together(E):
    """Segments are shorter for few rows: probabilities have the same bits."""
    say("alone")
    l, u = rows_of(64, 128256, BF, 27)
    s = settings_of(64, T=[0.9] * 64, p=[0.9] * 64, k=[500] * 64)
    token, probs = E.enc_sample(l, u, return_probs=True, **s)
    for r in (0, 31, 63):
        t1, p1 = E.enc_sample(l[r:r + 1], u[r:r + 1], return_probs=True, **{n: t[:1] if t is not None else None for n, t in s.items()})
        assert torch.equal(t1, token[r:r + 1]) and torch.equal(p1, probs[r:r + 1])


def test_distribution(E):
    """Equally spaced u: each token as often as its probability says, to one."""
    say("distribution")
    n = 4096
    l = torch.randn(50, generator=torch.Generator().manual_seed(2)).cuda().expand(n, 50)
    u = (torch.arange(n, device="cuda") + 0.5) / n
    token, probs = E.enc_sample(l, u, top_k=torch.tensor([20], dtype=torch.int32, device="cuda"), return_probs=True)
    count = torch.bincount(token.long(), minlength=50).double()
    assert (count - probs[0].double() * n).abs().max() <= 1.0 + 1e-3


def test_stream_graph_and_workspace(E):
    """On another stream; captured, replayed with other logits; a used workspace; repeated calls give equal bits."""
    say("graph")
    l, u = rows_of(16, 50000, F32, 28)
    s = settings_of(16, T=MIX["T"] * 2, k=MIX["k"] * 2, p=MIX["p"] * 2, m=MIX["m"] * 2)
    want = E.enc_sample(l, u, return_probs=True, **s)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    got = E.enc_sample(l, u, return_probs=True, stream=other, **s)
    other.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    ws = E.sample_workspace(l)
    ws.fill_(0xFF)
    probs = torch.empty_like(l)
    got = E.enc_sample(l, u, ws=ws, probs=probs, **s)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], probs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token, _ = E.enc_sample(l, u, ws=ws, probs=probs, **s)
    for i in range(4):
        l.normal_().mul_(1.0 + i)
        u.uniform_()
        graph.replay()
        torch.cuda.synchronize()
        want = E.enc_sample(l, u, return_probs=True, **s)
        assert torch.equal(want[0], token) and torch.equal(want[1], probs)


def test_binding_refusals(E):
    say("refusals")
    l, u = rows_of(6, 100, F32, 29)
    f = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    for bad in (dict(u=u[:5]), dict(u=u.double()), dict(temperature=f(4)), dict(temperature=f(3), top_p=f(2)), dict(top_k=f(6)),
                dict(temperature=f(0)), dict(u=u.cpu()), dict(probs=f(100)), dict(ws=torch.zeros(16, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            E.enc_sample(l, **{"u": u, **bad})
    with pytest.raises(TypeError):
        E.enc_sample(l.double(), u)
    with pytest.raises(E.EncError):
        E.enc_sample(l)                                       # nothing is asked for
    with pytest.raises(E.EncError):
        E.enc_sample(l, u, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    token, probs = E.enc_sample(l[:0], u[:0], return_probs=True)
    assert token.shape == (0,) and probs.shape == (0, 100)
