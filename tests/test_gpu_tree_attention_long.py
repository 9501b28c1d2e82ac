"""enc_tree_attention where a workgroup goes through many stages of keys in one
go, and over caches above 4 GiB, in every kernel that a call can reach.

Against the formula in 64 bits on the device; tolerances as derived in
test_gpu_tree_attention.py."""
import sys

import numpy as np
import pytest

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


def definition(q, kn, vn, kc, vc, table, lens, scale):
    """Out, log-sum-exp and sum p |v|, in float64; node i sees nodes 0 .. i."""
    B, T, H, D = q.shape
    page, G = kc.shape[1:3]
    out, size = torch.zeros(B, T, H, D, dtype=torch.float64, device="cuda"), torch.zeros(B, T, H, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, T, H, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(lens[b])
        used = table[b, :-(-n // page)].long()
        hidden = torch.ones(T, T, dtype=torch.bool, device="cuda").triu(1)
        for g in range(G):
            k = torch.cat([kc[used, :, g].reshape(-1, D)[:n], kn[b, :, g]]).double()
            v = torch.cat([vc[used, :, g].reshape(-1, D)[:n], vn[b, :, g]]).double()
            for h in range(g * (H // G), (g + 1) * (H // G)):
                x = torch.matmul(q[b, :, h].double(), k.T) * scale
                x[:, n:][hidden] = -float("inf")
                lse[b, :, h] = torch.logsumexp(x, -1)
                p = (x - lse[b, :, h, None]).exp()
                out[b, :, h], size[b, :, h] = torch.matmul(p, v), torch.matmul(p, v.abs())
    return out, lse, size


def compare(got, lse, want, wl, size):
    u = U[got.dtype]
    bad = ~((got.double() - want).abs() <= u * want.abs() + (u + 2.0 ** -10) * size + 1e-30)
    assert not bad.any(), "%d of %d outside" % (int(bad.sum()), bad.numel())
    assert ((lse.double() - wl).abs() <= 2.0 ** -11 + 2.0 ** -20 * wl.abs()).all()


def parts_of(E, q, kn, table, kc):
    """How many equal parts a call's keys are cut into (its workspace holds
    that many and one more a sequence, of head_dim + 2 floats a row)."""
    B, T, H, D = q.shape
    return round(E.enc_tree_attention_workspace_bytes(q, kn, table, kc) / (T * H * (D + 2) * 4)) - B


def tensors(B, T, H, G, D, pages, page, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    return t(B, T, H, D), t(B, T, G, D), t(B, T, G, D), t(pages, page, G, D), t(pages, page, G, D)


# keys in a stage, batch, nodes, query and KV heads, head_dim, tokens
DEEP = {
    "four waves, a strip to a wave, heads of 128": (128, 1, 3, 512, 128, 128, 6000),
    "four waves, a strip to a wave, heads of 96": (128, 1, 2, 256, 128, 96, 6000),
    "four waves, a strip to a wave, heads of 64": (128, 1, 3, 512, 128, 64, 7500),
    "four waves, a strip to a wave, heads of 256": (128, 1, 1, 256, 128, 256, 2500),
    "four heads, heads of 64": (32, 8, 3, 256, 64, 64, 2500),
    "four heads, heads of 128": (32, 8, 4, 128, 64, 128, 1700),
    "four heads, heads of 256": (32, 8, 4, 64, 64, 256, 900),
    "four heads, 32 rows, heads of 64": (32, 8, 8, 256, 64, 64, 2000),
    "four heads, 24 rows, heads of 128": (32, 8, 12, 128, 64, 128, 1300),
    "four waves of 16, heads of 64": (64, 1, 5, 256, 64, 64, 5000),
    "four waves of 16, heads of 128": (32, 1, 5, 256, 64, 128, 2500),
    "four waves of 16, heads of 256": (32, 1, 5, 256, 64, 256, 2500),
    "four waves of 16, 64 rows, heads of 72": (32, 1, 16, 256, 64, 72, 2500),
    "eight waves of 16, heads of 64": (64, 1, 25, 256, 64, 64, 2500),
    "eight waves of 16, heads of 128": (64, 1, 25, 256, 64, 128, 2500),
    "eight waves of 16, heads of 256": (32, 1, 25, 256, 64, 256, 1300),
    "four waves of 32, heads of 64": (64, 2, 25, 256, 64, 64, 2500),
    "four waves of 32, heads of 128": (32, 2, 25, 256, 64, 128, 1300),
    "eight waves of 32, heads of 64": (64, 1, 33, 256, 64, 64, 2500),
    "eight waves of 32, heads of 128": (64, 1, 64, 256, 64, 128, 2500),
    "eight waves of 32, two tiles, heads of 104": (64, 1, 65, 128, 32, 104, 2500),
}


@pytest.mark.parametrize("page,dt", [(16, torch.bfloat16), (21, torch.float16)])   # the page of a wave's rows; each lane's own
@pytest.mark.parametrize("case", list(DEEP))
def test_many_stages_in_one_go(E, case, page, dt):
    say("attention, many stages:", case, page, dt)
    keys, B, T, H, G, D, length = DEEP[case]
    most = -(-length // page)
    q, kn, vn, kc, vc = tensors(B, T, H, G, D, B * most + 3, page, dt, 61)
    table = torch.randperm(B * most + 3, generator=torch.Generator().manual_seed(62))[:B * most].view(B, most).int().cuda()
    lens = torch.tensor([length - 37 * b for b in range(B)], dtype=torch.int32)
    parts = parts_of(E, q, kn, table, kc)
    assert parts >= 1 and int(lens.sum()) // keys >= 7 * parts, parts
    out, lse = E.enc_tree_attention(q, kn, vn, kc, vc, table, lens.cuda(), return_lse=True)
    compare(out, lse, *definition(q, kn, vn, kc, vc, table, lens, D ** -0.5))


# batch, nodes, query and KV heads, head_dim
FAR = {
    "2 rows": (1, 2, 2, 1, 256),
    "8 rows, two heads": (1, 4, 4, 2, 128),
    "four heads to a workgroup": (128, 2, 8, 4, 64),
    "40 rows": (1, 20, 2, 1, 256),
    "40 rows, two heads": (1, 20, 4, 2, 128),
    "100 rows": (1, 50, 4, 2, 128),
    "200 rows, four heads": (1, 100, 8, 4, 64),
}


@pytest.mark.parametrize("page", [128, 125])     # the page of a wave's rows; each lane's own
@pytest.mark.parametrize("case", list(FAR))
def test_caches_above_4_gib(E, case, page):
    """Rows on both sides of 2^31 and 2^32 bytes from the cache's start; where
    an offset wraps, other values lie."""
    say("attention, cache above 4 GiB:", case, page)
    B, T, H, G, D = FAR[case]
    per = page * G * D * 2                        # bytes of a page
    pages = (1 << 32) // per + 2000
    q, kn, vn, small_k, small_v = tensors(B, T, H, G, D, 8, page, torch.bfloat16, 63)
    kc = torch.zeros(pages, page, G, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    assert kc.numel() * 2 > 1 << 32
    held = [pages - 1, 0, (1 << 31) // per - 1, (1 << 31) // per + 1, (1 << 32) // per - 1, (1 << 32) // per + 1, 1,
            (1 << 32) // per]                     # the last one straddles 2^32 unless pages divide it
    kc[held], vc[held] = small_k, small_v
    lens = torch.tensor([8 * page - 3 * b for b in range(B)], dtype=torch.int32, device="cuda")
    near = torch.arange(8, dtype=torch.int32, device="cuda").repeat(B, 1)
    far = torch.tensor(held, dtype=torch.int32, device="cuda").repeat(B, 1)
    want = E.enc_tree_attention(q, kn, vn, small_k, small_v, near, lens)[0]
    got = E.enc_tree_attention(q, kn, vn, kc, vc, far, lens)[0]
    assert torch.equal(got, want)
    if page == 128 and G == 1:                    # and through strides that pass 2^32 bytes in few pages
        t = torch.tensor([[0, 3, 1, 2]], dtype=torch.int32, device="cuda")
        step = pages // 4
        wide = [x[:4 * step].view(4, step * page, G, D)[:, :page] for x in (kc, vc)]
        assert (3 * wide[0].stride(0)) * 2 > 3 << 30
        wide[0][t[0].long()], wide[1][t[0].long()] = small_k[:4], small_v[:4]
        lens[:] = 4 * page - 5
        want = E.enc_tree_attention(q, kn, vn, small_k, small_v, near[:, :4].contiguous(), lens)[0]
        assert torch.equal(E.enc_tree_attention(q, kn, vn, *wide, t, lens)[0], want)
