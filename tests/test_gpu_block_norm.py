"""enc_block_norm on the GPU against the formula in 64 bits.

Tolerance, derived: a sum of squares runs through at most 32 values of a thread
(4 chunks of 8), 6 steps in a wave and 16 over the waves: 54 roundings of 2^-24,
halved by the square root: 27, and 3 for the quotient, the root and eps. Products
with the factor, the weight (1 + w: one more), the gate, the two scales and the
sum add 6 more: 36 roundings, below 2^-18 of |a h| + |s g z|. x carries that
through its own norm (continuation_ref.block_norm gives the magnitude) and adds
as many roundings: 2^-17. Then each result is rounded once to its type."""
import itertools
import sys

import numpy as np
import pytest

import continuation_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF: 2.0 ** -8, FP: 2.0 ** -11, F32: 2.0 ** -24}


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


def near(got, want, size, slack, what):
    u = U[got.dtype]
    bound = u * np.abs(want) + slack * size + (2.0 ** -25 if got.dtype == FP else 1e-37)
    g = got.double().cpu().numpy()
    bad = ~(np.abs(g - want) <= bound)
    assert not bad.any(), "%s: %d of %d outside, worst %g" % (what, bad.sum(), bad.size, np.nanmax(np.abs(g - want)))


def case(tokens, width, ty, th, tw, seed=0, pad=0, lead=0):
    """y, h on the device, rows `pad` values longer than they need be, the first `lead` values in."""
    g = torch.Generator().manual_seed(seed)
    def rows(n, dtype, scale):
        t = torch.zeros(max(n * (width + pad), 1) + lead, dtype=dtype, device="cuda")
        v = t[lead:lead + n * (width + pad)].view(n, width + pad)[:, :width]
        v.copy_((scale * torch.randn(n, width, generator=g)).to(dtype))
        return v
    weight = lambda: (1 + 0.2 * torch.randn(width, generator=g)).to(tw).cuda()  # noqa: E731
    return rows(tokens, ty, 1.7), rows(tokens, th, 4.0), weight(), weight(), g, rows


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def check(E, y, h, gate, w_post, w_pre, post, offset=False, a=1.0, s=1.0, eps=1e-6, **kw):
    tokens = h.shape[0]
    every = None if gate is None else f64(gate if gate.dim() == 2 else gate[None])
    if every is not None:
        every = every.repeat(tokens // every.shape[0], 0)
    want_h, want_x, size_h, size_x = ref.block_norm(f64(y), f64(h), every, f64(w_post), f64(w_pre), post, a, s, eps, offset)
    got_h, got_x = E.enc_block_norm(h, y, gate=gate, w_post=w_post, w_pre=w_pre, post_norm=post, h_scale=a, y_scale=s,
                                    eps=eps, unit_offset=offset, **kw)
    torch.cuda.synchronize()
    near(got_h, want_h, size_h, 2.0 ** -18, "h'")
    near(got_x, want_x, size_x, 2.0 ** -17, "x")
    return got_h, got_x


@pytest.mark.parametrize("tokens,width", [
    (1, 1), (1, 4096), (3, 7), (5, 8), (2, 63), (4, 64), (9, 513), (792, 2560), (33, 1537), (1, 8192), (2, 8200), (2, 8191),
    (1, 16384), (3, 16392), (1, 32768), (2, 32767), (1030, 1024), (1025, 1000), (1024, 2049)])
def test_sizes(E, tokens, width):
    say("sizes", tokens, width)
    y, h, wq, wp, g, rows = case(tokens, width, F32, F32, BF)
    check(E, y, h, None, None, wp, False)
    check(E, y, h, rows(1, BF, 0.5)[0], wq, wp, True, s=0.25)


@pytest.mark.parametrize("ty,th,tw,to", [c for c in itertools.product((F32, BF, FP), repeat=4) if len(set(c)) < 3 or c[0] is F32])
@pytest.mark.parametrize("width", [128, 131])
def test_types(E, ty, th, tw, to, width):
    say("types", ty, th, tw, to, width)
    y, h, wq, wp, g, rows = case(5, width, ty, th, tw, 1)
    check(E, y, h, rows(5, tw, 0.5), wq, wp, True, out_dtype=to)


@pytest.mark.parametrize("rows_of_gates", [1, 2, 3, 12])
@pytest.mark.parametrize("offset", [False, True])
def test_gates_and_offset(E, rows_of_gates, offset):
    say("gates", rows_of_gates, offset)
    y, h, wq, wp, g, rows = case(12, 96, BF, BF, BF, 2)
    check(E, y, h, rows(rows_of_gates, F32, 0.5), wq, wp, True, offset=offset, a=1.5, s=-0.75)
    check(E, y, h, rows(rows_of_gates, FP, 0.5), None, None, True, offset=offset)
    check(E, y, h, rows(rows_of_gates, FP, 0.5), None, wp, False, offset=offset)


@pytest.mark.parametrize("pad,lead", [(8, 0), (8, 8), (3, 0), (0, 1), (5, 3)])
def test_strides_and_alignment(E, pad, lead):
    """Rows longer than the width, bases that are not 16-byte aligned: what lies between rows stays as it is."""
    say("strides", pad, lead)
    y, h, wq, wp, g, rows = case(6, 256, BF, F32, F32, 3, pad, lead)
    gate = rows(2, BF, 0.3)
    out = torch.full((6 * (256 + pad) + lead,), 7.0, dtype=BF, device="cuda")
    h_out = torch.full((6 * (256 + pad) + lead,), 7.0, dtype=F32, device="cuda")
    view = lambda t: t[lead:].view(6, 256 + pad)  # noqa: E731
    check(E, y, h, gate, wq, wp, True, out=view(out)[:, :256], h_out=view(h_out)[:, :256])
    assert (view(out)[:, 256:] == 7).all() and (view(h_out)[:, 256:] == 7).all()
    assert (out[:lead] == 7).all() and (h_out[:lead] == 7).all()


def test_in_place_and_parts(E):
    """h' over h; only h'; only x; without y; nothing to do."""
    say("in place")
    y, h, wq, wp, g, rows = case(7, 640, F32, F32, BF, 4)
    want_h, want_x = check(E, y, h, None, wq, wp, True)
    copy = h.clone()
    got_h, got_x = E.enc_block_norm(copy, y, w_post=wq, w_pre=wp, post_norm=True, h_out=copy)
    assert got_h is copy and torch.equal(copy, want_h) and torch.equal(got_x, want_x)
    only_h, nothing = E.enc_block_norm(h, y, w_post=wq, post_norm=True, pre_norm=False)
    assert nothing is None and torch.equal(only_h, want_h)
    same, x = E.enc_block_norm(h, w_pre=wp)
    assert same is h
    check(E, None, h, None, None, wp, False)
    scaled, _ = check(E, None, h, None, None, wp, False, a=0.5)
    assert torch.equal(scaled, 0.5 * h)
    again, none = E.enc_block_norm(h, pre_norm=False)
    assert again is h and none is None
    e_h, e_x = E.enc_block_norm(h[:0], y[:0])
    assert e_h.shape == e_x.shape == (0, 640)


def test_special_rows(E):
    """Infinities, NaN and zeros stay in their rows; a row of zeros with eps 0 is NaN, with eps > 0 zero."""
    say("special")
    y, h, wq, wp, g, rows = case(8, 200, F32, F32, BF, 5)
    clean = E.enc_block_norm(h, y, w_post=wq, w_pre=wp, post_norm=True)
    y[1, 5], h[3, 7], y[5] = float("inf"), float("nan"), 0.0
    got = E.enc_block_norm(h, y, w_post=wq, w_pre=wp, post_norm=True)
    for r in (0, 2, 4, 6, 7):
        assert torch.equal(got[0][r], clean[0][r]) and torch.equal(got[1][r], clean[1][r])
    assert got[1][1].isnan().all() and got[1][3].isnan().all()
    assert got[0][1, 5].isnan() and torch.equal(got[0][1, :5], h[1, :5])    # an infinite mean: the rest is 0
    assert torch.equal(got[0][5], h[5])
    zero = torch.zeros_like(h)
    _, x = E.enc_block_norm(zero, eps=0.0)
    assert x.isnan().all()
    _, x = E.enc_block_norm(zero, eps=1e-6)
    assert (x == 0).all()


def test_large_and_small_values(E):
    """Values at both ends of what squares allow in fp32."""
    say("large values")
    for scale in (1e-15, 1e15):
        y, h, wq, wp, g, rows = case(3, 300, F32, F32, F32, 6)
        check(E, y * scale, h * scale, None, wq, wp, True, eps=0.0)


def test_many_rows(E):
    """More rows than one launch takes, and an array above 4 GiB."""
    say("many rows")
    n = (1 << 21) + 3
    h = torch.randn(n, 8, device="cuda", dtype=F32)
    got, x = E.enc_block_norm(h, h, y_scale=0.5)
    part = torch.cat([torch.arange(64), torch.arange(n - 64, n), torch.arange((1 << 21) - 32, (1 << 21) + 3)]).cuda()
    want_h, want_x, size_h, size_x = ref.block_norm(f64(h[part]), f64(h[part]), None, None, None, False, 1.0, 0.5, 1e-6, False)
    near(got[part], want_h, size_h, 2.0 ** -18, "h'")
    near(x[part], want_x, size_x, 2.0 ** -17, "x")
    del h, got, x
    h = torch.randn(70000, 16384, device="cuda", dtype=F32)       # 4.6 GB
    got, x = E.enc_block_norm(h, h, y_scale=0.5)
    part = torch.tensor([0, 65535, 65536, 69999]).cuda()
    want_h, want_x, size_h, size_x = ref.block_norm(f64(h[part]), f64(h[part]), None, None, None, False, 1.0, 0.5, 1e-6, False)
    near(got[part], want_h, size_h, 2.0 ** -18, "h'")
    near(x[part], want_x, size_x, 2.0 ** -17, "x")


def test_another_stream(E):
    say("stream")
    y, h, wq, wp, g, rows = case(64, 1000, BF, F32, BF, 7)
    want = E.enc_block_norm(h, y, w_post=wq, w_pre=wp, post_norm=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = E.enc_block_norm(h, y, w_post=wq, w_pre=wp, post_norm=True, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graph(E):
    """Captured and replayed, with other values in the same buffers each time."""
    say("graph")
    y, h, wq, wp, g, rows = case(40, 768, F32, F32, BF, 8)
    x = torch.empty(40, 768, dtype=BF, device="cuda")
    ho = torch.empty_like(h)
    E.enc_block_norm(h, y, w_post=wq, w_pre=wp, post_norm=True, h_out=ho, out=x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        E.enc_block_norm(h, y, w_post=wq, w_pre=wp, post_norm=True, h_out=ho, out=x)
    for i in range(4):
        y.normal_()
        graph.replay()
        want = E.enc_block_norm(h, y, w_post=wq, w_pre=wp, post_norm=True)
        torch.cuda.synchronize()
        assert torch.equal(ho, want[0]) and torch.equal(x, want[1])


def test_binding_refusals(E):
    say("refusals")
    y, h, wq, wp, g, rows = case(6, 64, BF, F32, BF, 9)
    for bad in (dict(y=y[:5]), dict(y=y[:, :32]), dict(gate=rows(4, BF, 1.0)), dict(w_pre=wp[:32]), dict(y=y.cpu()),
                dict(w_pre=wp, pre_norm=False), dict(out=y.new_empty(6, 64), pre_norm=False),
                dict(h_out=torch.empty(6, 64, dtype=BF, device="cuda")), dict(y=y.t().contiguous().t())):
        with pytest.raises(ValueError):
            E.enc_block_norm(h, **bad)
    with pytest.raises(TypeError):
        E.enc_block_norm(h, y, w_post=wq, w_pre=wp.float(), post_norm=True)
    with pytest.raises(TypeError):
        E.enc_block_norm(h, y.double())
    for bad in (dict(w_post=wq), dict(gate=wq), dict(post_norm=True), dict(eps=-1.0), dict(h_scale=float("nan"))):
        with pytest.raises(E.EncError):
            E.enc_block_norm(h, **bad)
