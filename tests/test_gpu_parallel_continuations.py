"""A run of the operators together: examples/parallel_continuations.py, its
steps' logits against the same model in plain fp32 torch, its tokens against the
filters' definition, and its bookkeeping.

Tolerance, derived: activations are rounded to BF16 (2^-8 relative) at four
places of a layer (the norm before each product, q / k / v, the attention's
weights and its result, the gated product), 3 layers deep, 7 roundings a layer,
each passed on by products with gain about 1 (random weights scaled by 1 / sqrt
of the fan-in; later layers by 0.4): errors add like independent ones, sqrt(21)
2^-9 of the logits' spread (rounding is uniform: a half of 2^-8 at most, a third
of that in the mean square), below 2^-6.5. Twice that bounds the relative
difference of all logits together."""
import os
import sys

import numpy as np
import pytest

import continuation_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import parallel_continuations
    return parallel_continuations


def plain_logits(E, m, tokens):
    """fp32 logits after the last of tokens [B, n], without a cache."""
    if not hasattr(m, "decoded"):
        def dense(coded):
            stream, info, n = coded
            return E.enc_decompress(stream, info).view(torch.bfloat16).view(n, -1).float()
        m.decoded = [{k: dense(b[k]) for k in ("qkv", "o", "up", "down")} for b in m.blocks], dense(m.head)
    blocks, head = m.decoded
    B, n = tokens.shape
    norm = lambda x: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    h = m.embedding[tokens.long()].float()
    half = m.head_dim // 2
    cos, sin = m.angles[:n, None, :half], m.angles[:n, None, half:]
    rotate = lambda x: torch.cat([x[..., :half] * cos - x[..., half:] * sin,  # noqa: E731
                                  x[..., half:] * cos + x[..., :half] * sin], -1)
    for w in blocks:
        q, k, v = (norm(h) @ w["qkv"].T).view(B, n, -1, m.head_dim).split((m.heads, m.kv_heads, m.kv_heads), 2)
        q, k = rotate(norm(q)), rotate(norm(k))
        k, v = (x.repeat_interleave(m.heads // m.kv_heads, 2).transpose(1, 2).contiguous() for x in (k, v))
        s = torch.matmul(q.transpose(1, 2).contiguous(), k.transpose(2, 3).contiguous()) * m.head_dim ** -0.5
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -float("inf"))
        h = h + torch.matmul(s.softmax(-1), v).transpose(1, 2).reshape(B, n, -1) @ w["o"].T
        gate, up = (norm(h) @ w["up"].T).split(m.ffn, -1)
        h = h + (torch.nn.functional.silu(gate) * up) @ w["down"].T
    return norm(h[:, -1]) @ head.T


def test_steps_against_plain_torch(example):
    print("[gpu-case] continuations", flush=True)
    E = example.enc
    model = example.Model(seed=3)
    prompt = torch.randint(0, model.vocab, (3, 45), dtype=torch.int32, generator=torch.Generator().manual_seed(2)).cuda()
    c = example.Continuations(model, 3, 5, max_len=256, seed=4)
    pending = c.prefill(prompt)
    text = prompt.repeat_interleave(5, 0)
    rng = torch.Generator(device="cuda").manual_seed(4)
    for step in range(20):
        token, logits = c.step(pending)
        want = plain_logits(E, model, text)
        assert (logits - want).norm() <= 2 * 2.0 ** -6.5 * want.norm(), step
        u = torch.rand(c.batch, generator=rng, device="cuda")
        for b in range(c.batch):
            e = ref.kept_weights(logits[b].double().cpu().numpy(), float(np.float32(0.8)), 50, float(np.float32(0.95)),
                                 float(np.float32(0.02)))
            assert int(token[b]) == ref.draw(e, float(u[b])), (step, b)
        text = torch.cat([text, token[:, None]], 1)
        pending = token
    assert c.cache.lens[3:].tolist() == [64] * 15 and c.cache.lens[:3].tolist() == [44] * 3
    assert E.enc_cache_shared(c.cache, c.seqs, c.starts).tolist() == [32] * 3      # two whole pages of each prompt
    # the pages of the prompts (3 each), and 2 more for every continuation
    assert int((c.cache.refs > 0).sum()) == 3 * 3 + 15 * 2


def test_example_runs(example, capsys):
    print("[gpu-case] example", flush=True)
    example.main()
    assert "16 continuations of 48 tokens" in capsys.readouterr().out
