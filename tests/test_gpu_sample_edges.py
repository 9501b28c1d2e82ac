"""enc_sample where roundings of fp64 sums, or a second rounding of a result,
would show."""
import sys

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


@pytest.mark.parametrize("depth", [30.0, 38.0, 42.0, 45.0])
@pytest.mark.parametrize("rows,V", [(1, 128256), (16, 128256), (64, 128256), (16, 32003), (300, 5000)])
def test_last_token(E, rows, V, depth):
    """u of 1 names the last kept token, also where it and many before it weigh less than a sum's rounding."""
    say("u = 1", rows, V, depth)
    g = torch.Generator().manual_seed(int(depth))
    logits = 3.0 * torch.randn(rows, V, generator=g)
    tail = V // 3
    logits[:, -tail:] = logits.max(1, keepdim=True)[0] - depth
    last = V - 1 - torch.arange(rows) % 3                     # the very last ones are not kept in some rows
    for r in range(rows):
        logits[r, int(last[r]) + 1:] = -float("inf")
    token, _ = E.enc_sample(logits.cuda(), torch.ones(rows, device="cuda"))
    assert torch.equal(token.cpu(), last.int())


def test_equal_rows(E):
    """Equal rows give equal tokens and probabilities, at cuts of every size."""
    say("equal rows")
    g = torch.Generator().manual_seed(7)
    row = 2.0 * torch.randn(1, 50000, generator=g)
    p = (torch.arange(1, 257) / 257.0).float().repeat_interleave(4)
    u = torch.rand(256, generator=g).repeat_interleave(4)
    token, probs = E.enc_sample(row.repeat(1024, 1).cuda(), u.cuda(), top_p=p.cuda(), return_probs=True)
    token, probs = token.view(256, 4), probs.view(256, 4, -1)
    assert (token == token[:, :1]).all() and (probs == probs[:, :1]).all()


def test_one_workspace_for_all(E):
    """A workspace of the largest batch serves smaller ones, which write nothing past it."""
    say("sampling workspace")
    g = torch.Generator().manual_seed(8)
    logits, u = (3.0 * torch.randn(40, 128256, generator=g)).cuda(), torch.rand(40, generator=g).cuda()
    p = torch.full((1,), 0.9, device="cuda")
    size = E.enc_sample_workspace_bytes(40, 128256)
    room = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    want, _ = E.enc_sample(logits, u, top_p=p)
    for rows in (40, 32, 31, 30, 16, 1):
        token, _ = E.enc_sample(logits[:rows], u[:rows], top_p=p, ws=room[:size])
        assert torch.equal(token, want[:rows])
    assert (room[size:] == 0xA5).all()


@pytest.mark.parametrize("n,dtype,want", [
    # 1 / n = 381 / (2^28 - 1): just above the half between 190 and 191 2^-27
    (704555, torch.bfloat16, 191 * 2.0 ** -27),
    # 1 / n = 1801 / (2^25 - 1): just above the half between 900 and 901 2^-24
    (18631, torch.float16, 901 * 2.0 ** -24),
    # 1 / n = 251 / (2^25 + 1): just below the half between 125 and 126 2^-24
    (133683, torch.float16, 125 * 2.0 ** -24),
])
@pytest.mark.parametrize("logits_dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_probabilities_are_rounded_once(E, n, dtype, want, logits_dtype):
    """Equal probabilities that fp32 puts on a half of the output's type, where they are not."""
    say("probabilities", n, dtype, logits_dtype)
    _, probs = E.enc_sample(torch.zeros(1, n, dtype=logits_dtype, device="cuda"), return_probs=True, probs_dtype=dtype)
    assert (probs.double() == want).all()
