"""Several continuations of one prompt, from a small transformer whose weights
stay compressed.

    python examples/parallel_continuations.py

The prompt is run once; every continuation is a fork that shares its pages. A
step decodes one token of each:

    enc_block_norm        residual sum, the norm after a block and before the next
    enc_decompress_gemm_nt  every product with a weight, from the coded weights
    enc_qk_norm_rope      head norms, rotation
    enc_cache_shared      how many cached tokens the continuations have in common
    enc_prefix_attention  their attention; common rows are read once for all
    enc_sample            temperature, top-k, top-p, min-p, and the next tokens
    enc_cache_commit      the step's rows become cache rows
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from lossless_weight_compression_amd import enc  # noqa: E402
from speculative_decoding import Model  # noqa: E402


class Continuations:
    """`prompts` prompts with `each` continuations of each."""

    def __init__(self, model, prompts, each, page=16, max_len=1024, seed=0, temperature=0.8, top_k=50, top_p=0.95, min_p=0.02):
        m = self.model = model
        self.prompts, self.each, self.batch = prompts, each, prompts * each
        entries = max_len // page
        # the prompts' own sequences come first, their continuations behind them
        self.cache = enc.Cache.empty(2 * m.layers, (prompts + self.batch) * entries, page, (m.kv_heads, m.head_dim),
                                     prompts + self.batch, entries)
        ints = lambda t: t.to(torch.int32).cuda()  # noqa: E731
        self.roots = ints(torch.arange(prompts))
        self.seqs = ints(prompts + torch.arange(self.batch))
        self.starts = ints(each * torch.arange(prompts + 1))
        self.rng = torch.Generator(device="cuda").manual_seed(seed)
        # one setting for each continuation
        full = lambda x, dt: torch.full((self.batch,), x, dtype=dt, device="cuda")  # noqa: E731
        self.settings = dict(temperature=full(temperature, torch.float32), top_k=full(top_k, torch.int32),
                             top_p=full(top_p, torch.float32), min_p=full(min_p, torch.float32))

    def forward(self, tokens, seqs, starts, shared):
        """Logits after every token of [B, T] new ones, and their K and V rows in every plane."""
        m = self.model
        B, T = tokens.shape
        rows = torch.empty(2 * m.layers, B, T, m.kv_heads, m.head_dim, dtype=torch.bfloat16, device="cuda")
        order = torch.arange(T, dtype=torch.int32, device="cuda")
        positions = (self.cache.lens[seqs.long(), None] + order).view(-1)
        h = m.embedding[tokens.long()].float().view(B * T, m.hidden)
        y = None                                            # the last block's result, not yet in h
        for layer in range(m.layers):
            w = m.blocks[layer]
            h, x = enc.enc_block_norm(h, y, h_out=None if y is None else h)
            q, k, v = m.product(x, w["qkv"]).view(B * T, -1, m.head_dim).split((m.heads, m.kv_heads, m.kv_heads), 1)
            k_new, v_new = rows[2 * layer], rows[2 * layer + 1]
            q, _, _ = enc.enc_qk_norm_rope(
                q, k, v, positions, m.angles, w["qw"], w["kw"],
                out=(torch.empty(B * T, m.heads, m.head_dim, dtype=torch.bfloat16, device="cuda"),
                     k_new.view(B * T, m.kv_heads, m.head_dim), v_new.view(B * T, m.kv_heads, m.head_dim)))
            a, _ = enc.enc_prefix_attention(q.view(B, T, m.heads, m.head_dim), k_new, v_new, self.cache.data[2 * layer],
                                            self.cache.data[2 * layer + 1], self.cache.table, self.cache.lens, starts, shared,
                                            seqs=seqs)
            h, x = enc.enc_block_norm(h, m.product(a.view(B * T, -1), w["o"]), h_out=h)
            gate, up = m.product(x, w["up"]).split(m.ffn, 1)
            y = m.product((torch.nn.functional.silu(gate) * up).to(torch.bfloat16), w["down"])
        _, x = enc.enc_block_norm(h, y, h_out=h)
        return m.product(x, m.head).view(B, T, m.vocab), rows

    def commit(self, seqs, rows):
        B, T = rows.shape[1:3]
        order = torch.arange(T, dtype=torch.int32, device="cuda").repeat(B, 1)
        enc.enc_cache_commit(self.cache, seqs, rows, order, torch.full((B,), T, dtype=torch.int32, device="cuda"))
        if int(self.cache.status):                          # nothing was appended: what followed would miss these rows
            raise RuntimeError("the cache refused the rows: %d" % int(self.cache.status))

    def prefill(self, prompt):
        """Run prompts [prompts, n], all but their last tokens, fork them, and return those."""
        nobody = torch.zeros(1, dtype=torch.int32, device="cuda")
        for at in range(0, prompt.shape[1] - 1, enc.ENC_TREE_MAX_NODES):
            part = prompt[:, at:min(at + enc.ENC_TREE_MAX_NODES, prompt.shape[1] - 1)]
            _, rows = self.forward(part, self.roots, nobody, nobody[:0])
            self.commit(self.roots, rows)
        enc.enc_cache_fork(self.cache, self.roots.repeat_interleave(self.each), self.seqs)
        return prompt[:, -1].repeat_interleave(self.each)

    def step(self, pending):
        """The next token of every continuation, and the logits it was drawn from."""
        shared = enc.enc_cache_shared(self.cache, self.seqs, self.starts)
        logits, rows = self.forward(pending[:, None], self.seqs, self.starts, shared)
        token, _ = enc.enc_sample(logits[:, 0], torch.rand(self.batch, generator=self.rng, device="cuda"), **self.settings)
        self.commit(self.seqs, rows)
        return token, logits[:, 0]


def generate(continuations, prompt, n):
    pending = continuations.prefill(prompt)
    out = []
    for _ in range(n):
        pending, _ = continuations.step(pending)
        out.append(pending)
    return torch.stack(out, 1)


def main():
    model = Model()
    prompt = torch.randint(0, model.vocab, (2, 100), dtype=torch.int32, generator=torch.Generator().manual_seed(1)).cuda()
    c = Continuations(model, 2, 8)
    tokens = generate(c, prompt, 48)
    shared = enc.enc_cache_shared(c.cache, c.seqs, c.starts).tolist()
    print("%d continuations of %d tokens; each prompt's share %s cached tokens; %d of %d pages used"
          % (tokens.shape[0], tokens.shape[1], shared, int((c.cache.refs > 0).sum()), c.cache.refs.numel()))


if __name__ == "__main__":
    main()
