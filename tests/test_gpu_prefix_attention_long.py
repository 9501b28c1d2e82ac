"""enc_prefix_attention where a workgroup goes through many stages of shared
keys in one go, so that every buffer is filled and read again, in every kernel
that a call can reach.

Against the formula in 64 bits on the device; tolerances as derived in
test_gpu_prefix_attention.py."""
import sys

import numpy as np
import pytest

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


def pieces_of(prefix, rows, tile, kv_heads):
    """Strips of 32 keys in each piece of one group's shared tokens (as the plan cuts them)."""
    units, tiles, slots = -(-prefix // 32), -(-rows // tile), max((512 if tile == 16 else 256) // kv_heads, 1)
    size = max(-(-(-(-tiles * units // slots)) // 4) * 4, 4)
    return [min(size, units - at) for at in range(0, units, size)]


# sequences, nodes, query and KV heads, head_dim, rows of a tile; shared tokens are chosen for the stages of a piece
KERNELS = {
    "16 rows, heads of 64": (2, 1, 64, 16, 64, 16),
    "16 rows, heads of 128": (2, 2, 64, 16, 128, 16),
    "16 rows, heads of 256": (2, 1, 64, 16, 256, 16),
    "64 rows, heads of 64": (10, 1, 64, 16, 64, 64),
    "64 rows, heads of 96": (10, 1, 64, 16, 96, 64),
    "64 rows, heads of 128": (10, 1, 64, 16, 128, 64),
    "64 rows, heads of 200": (10, 1, 64, 16, 200, 64),
    "64 rows, heads of 256": (10, 1, 64, 16, 256, 64),
    "128 rows, heads of 64": (35, 1, 64, 16, 64, 128),
    "128 rows, heads of 96": (35, 1, 64, 16, 96, 128),
    "128 rows, heads of 128": (35, 1, 64, 16, 128, 128),
    "two tiles of 64, trees, heads of 256": (3, 10, 64, 16, 256, 64),
    "two tiles of 128, trees, heads of 128": (5, 10, 64, 16, 128, 128),
}


@pytest.mark.parametrize("dt", [BF, FP])
# stages of 64 keys in a piece, whole ones in the last piece, and tokens behind them
@pytest.mark.parametrize("stages,last,past", [(6, 3, 0), (8, 6, 1), (10, 7, 33), (12, 10, 63)])
@pytest.mark.parametrize("case", list(KERNELS))
def test_many_stages_in_one_go(E, case, stages, last, past, dt):
    B, T, H, G, D, tile = KERNELS[case]
    page, per = 20, T * (H // G)
    tiles, slots = -(-B * per // tile), (512 if tile == 16 else 256) // G
    # as many pieces as there is room for; the last is shorter
    prefix = ((slots // tiles - 1) * stages + last) * 64 + past
    pieces = pieces_of(prefix, B * per, tile, G)
    assert pieces[0] == 2 * stages and pieces[-1] < 2 * stages
    say("prefix, many stages:", case, prefix, dt)
    g = torch.Generator(device="cuda").manual_seed(70 + stages)
    t = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    whole, own = prefix // page, 2
    n_pages = whole + own * B
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(71)).int()
    table = torch.stack([torch.cat([order[:whole], order[whole + own * b:whole + own * (b + 1)]]) for b in range(B)])
    lens = torch.tensor([prefix + b % 7 for b in range(B)], dtype=torch.int32)
    q, kn, vn, kc, vc = t(B, T, H, D), t(B, T, G, D), t(B, T, G, D), t(n_pages, page, G, D), t(n_pages, page, G, D)
    for c in (kc, vc):                                          # a prompt's last rows, copied
        for b in range(1, B):
            c[int(table[b, whole]), :prefix % page] = c[int(table[0, whole]), :prefix % page]
    starts, shared = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, B], [prefix]))
    out, lse = E.enc_prefix_attention(q, kn, vn, kc, vc, table.cuda(), lens.cuda(), starts, shared, return_lse=True)
    hidden = torch.ones(T, T, dtype=torch.bool, device="cuda").triu(1)
    u = U[dt]
    for b in range(0, B, max(B // 3, 1)):                        # rows of every tile's waves
        n = int(lens[b])
        pages = table[b].long().cuda()
        for h in range(G):
            k = torch.cat([kc[pages, :, h].reshape(-1, D)[:n], kn[b, :, h]]).double()
            v = torch.cat([vc[pages, :, h].reshape(-1, D)[:n], vn[b, :, h]]).double()
            at = slice(h * (H // G), (h + 1) * (H // G))
            x = torch.matmul(q[b, :, at].reshape(-1, D).double(), k.T).view(T, H // G, -1) * D ** -0.5
            x[:, :, n:] = x[:, :, n:].masked_fill(hidden[:, None], -np.inf)
            wl = torch.logsumexp(x, -1)
            p = (x - wl[..., None]).exp()
            want, size = torch.matmul(p, v), torch.matmul(p, v.abs())
            bad = ~((out[b, :, at].double() - want).abs() <= u * want.abs() + (u + 2.0 ** -10) * size + 1e-30)
            assert not bad.any(), "%d of %d outside" % (int(bad.sum()), bad.numel())
            assert ((lse[b, :, at].double() - wl).abs() <= 2.0 ** -11 + 2.0 ** -20 * wl.abs()).all()
