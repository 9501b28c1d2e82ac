"""enc_qk_norm_rope on the GPU against the formula in 64 bits.

Tolerance, derived: the result is rounded once to the output's type (u = 2^-8
BF16, 2^-11 FP16, 2^-24 FP32, plus half the least subnormal of FP16), and the
fp32 arithmetic before it -- a sum of at most 512 squares, a square root, a
quotient, at most four products and a sum -- is off by less than 2^-17 of the
products' magnitude (512 rounding steps of 2^-24 halved by the square root are
2^-16 in the worst case; squares are summed 8 to a lane and then in a tree, 14
steps deep, so 20 steps of 2^-24 in all bound it: < 2^-19)."""
import sys

import numpy as np
import pytest

import step_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


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


def rope_table(n, rot):
    ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def check(got, want, size, what):
    u = U[got.dtype]
    bound = u * np.abs(want) + 2.0 ** -19 * size + (2.0 ** -25 if got.dtype == torch.float16 else 1e-30)
    g = got.double().cpu().numpy()
    bad = ~(np.abs(g - want) <= bound)
    assert not bad.any(), "%s: %d of %d outside, worst %g" % (what, bad.sum(), bad.size, np.nanmax(np.abs(g - want)))


@pytest.mark.parametrize("tokens,hq,hkv,dim,rot,src,dst,adjacent", [
    (1, 32, 8, 128, 128, torch.float32, torch.bfloat16, False),
    (1, 1, 1, 8, 8, torch.float32, torch.float32, True),
    (7, 3, 1, 64, 32, torch.bfloat16, torch.bfloat16, True),
    (33, 7, 2, 80, 40, torch.float32, torch.float16, False),      # halves of 20: no multiple of 8
    (5, 4, 4, 96, 6, torch.float16, torch.float16, False),        # a rotation of 6 values
    (5, 4, 4, 96, 6, torch.bfloat16, torch.float16, True),
    (19, 5, 5, 256, 256, torch.float16, torch.float32, False),
    (4, 2, 1, 512, 500, torch.float32, torch.bfloat16, False),
    (3, 2, 1, 24, 0, torch.float32, torch.bfloat16, False),       # no rotation
    (300, 4, 2, 72, 72, torch.bfloat16, torch.float32, False),
])
def test_against_formula(E, tokens, hq, hkv, dim, rot, src, dst, adjacent):
    say("rope", tokens, hq, hkv, dim, rot, src, dst, adjacent)
    rng = np.random.default_rng([11, tokens, dim, rot])
    make = lambda h: torch.from_numpy(rng.standard_normal((tokens, h, dim)).astype(np.float32)).to(src).cuda()  # noqa: E731
    q, k, v = make(hq), make(hkv), make(hkv)
    w = [torch.from_numpy((1 + 0.2 * rng.standard_normal(dim)).astype(np.float32)).to(torch.bfloat16).cuda() for _ in "qk"]
    table = rope_table(1000, rot) if rot else None
    pos = rng.integers(0, 1000, tokens).astype(np.int32)
    got = E.enc_qk_norm_rope(q, k, v, torch.from_numpy(pos).cuda() if rot else None,
                             torch.from_numpy(table).cuda() if rot else None, w[0], w[1], eps=1e-5,
                             adjacent=adjacent, out_dtype=dst)
    torch.cuda.synchronize()
    for x, wt, g, name in ((q, w[0], got[0], "q"), (k, w[1], got[1], "k")):
        want, size = ref.norm_rope(x.double().cpu().numpy(), wt.double().cpu().numpy(), table, pos, 1e-5, adjacent)
        check(g, want, size, name)
    assert torch.equal(got[2], v.to(torch.float32).to(dst))


def test_no_norm_no_weight_no_v(E):
    say("rope without norm, weights, v")
    rng = np.random.default_rng(12)
    q, k = (torch.from_numpy(rng.standard_normal((9, h, 128)).astype(np.float32)).cuda() for h in (4, 2))
    table, pos = rope_table(64, 128), rng.integers(0, 64, 9).astype(np.int32)
    qo, ko, vo = E.enc_qk_norm_rope(q, k, None, torch.from_numpy(pos).cuda(), torch.from_numpy(table).cuda(), norm=False,
                                    out_dtype=torch.float32)
    assert vo is None
    for x, g in ((q, qo), (k, ko)):
        want, size = ref.norm_rope(x.double().cpu().numpy(), None, table, pos, 0.0, False, norm=False)
        check(g, want, size, "no norm")


def test_strides_in_place_and_rows_of_zeros(E):
    say("rope strided, in place")
    rng = np.random.default_rng(13)
    x = torch.from_numpy(rng.standard_normal((10, 3 + 2 + 2, 64)).astype(np.float32)).to(torch.bfloat16).cuda()
    x[4, 1] = 0                                    # a head of zeros stays zero (eps keeps it finite)
    before = x.clone()
    table, pos = rope_table(64, 64), rng.integers(0, 64, 10).astype(np.int32)
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    q, k, v = x[:, :3], x[:, 3:5], x[:, 5:]        # one packed projection, worked on in place
    E.enc_qk_norm_rope(q, k, v, torch.from_numpy(pos).cuda(), torch.from_numpy(table).cuda(), w, w, out=(q, k, v))
    torch.cuda.synchronize()
    for part, sl in (("q", slice(0, 3)), ("k", slice(3, 5))):
        want, size = ref.norm_rope(before[:, sl].double().cpu().numpy(), np.ones(64), table, pos, 1e-6, False)
        check(x[:, sl], want, size, part)
    assert torch.equal(x[:, 5:], before[:, 5:]) and not x[4, 1].any()
    # tokens from a transposed buffer: head-major rows
    y = before.transpose(0, 1).contiguous().transpose(0, 1)
    a = E.enc_qk_norm_rope(y[:, :3], y[:, 3:5], None, torch.from_numpy(pos).cuda(), torch.from_numpy(table).cuda(), w, w)
    assert torch.equal(a[0], x[:, :3]) and torch.equal(a[1], x[:, 3:5])


def test_positions_outside_the_table_give_nan(E):
    say("rope positions outside")
    x = torch.ones(4, 2, 64, device="cuda")
    table = torch.from_numpy(rope_table(16, 32)).cuda()
    pos = torch.tensor([0, 16, -1, 15], dtype=torch.int32, device="cuda")
    q, k, v = E.enc_qk_norm_rope(x, x, x, pos, table)
    assert q.isnan().all(-1).all(-1).tolist() == [False, True, True, False]
    assert k.isnan().any(-1).any(-1).tolist() == [False, True, True, False]
    assert torch.equal(v, x.to(torch.bfloat16))


def test_infinities_stay_in_their_head(E):
    say("rope infinities")
    x = torch.ones(3, 4, 64, device="cuda")
    x[1, 2, 5] = float("inf")
    table, pos = torch.from_numpy(rope_table(16, 64)).cuda(), torch.arange(3, dtype=torch.int32, device="cuda")
    q, _, _ = E.enc_qk_norm_rope(x, x[:, :1].contiguous(), None, pos, table)
    clean = E.enc_qk_norm_rope(torch.ones_like(x), x[:, :1].contiguous(), None, pos, table)[0]
    same = (q == clean).all(-1)
    assert not same[1, 2] and int(same.sum()) == 11


def test_another_stream_and_empty(E):
    say("rope on another stream; no tokens")
    x = torch.randn(50, 4, 128, device="cuda")
    table, pos = torch.from_numpy(rope_table(64, 128)).cuda(), torch.arange(50, dtype=torch.int32, device="cuda")
    want = E.enc_qk_norm_rope(x, x, x, pos, table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = E.enc_qk_norm_rope(x, x, x, pos, table, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    E.enc_qk_norm_rope(x[:0], x[:0], x[:0], pos[:0], table)


def test_more_tokens_than_one_grid_holds(E):
    say("2^24 + 5 tokens of three heads of 8 values")
    tokens, big = 2 ** 24 + 5, 2 ** 23
    q = torch.randn(tokens, 2, 8, device="cuda", dtype=torch.bfloat16)
    k = torch.randn(tokens, 1, 8, device="cuda", dtype=torch.bfloat16)
    table = torch.from_numpy(rope_table(64, 8)).cuda()
    pos = (torch.arange(tokens, device="cuda") % 64).int()
    qo, ko, _ = E.enc_qk_norm_rope(q, k, None, pos, table)
    for at in (0, big - 2, 2 * big - 2, tokens - 5):
        part = slice(at, at + 5)
        one_q, one_k, _ = E.enc_qk_norm_rope(q[part], k[part], None, pos[part], table)
        assert torch.equal(qo[part], one_q) and torch.equal(ko[part], one_k)
