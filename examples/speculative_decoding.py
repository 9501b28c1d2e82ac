"""Speculative decoding with a small transformer whose weights stay compressed.

    python examples/speculative_decoding.py

Each step drafts a tree of tokens with the model's first layer, runs the whole
model once over the tree, and keeps what the target accepts. Every product with
a weight is the fused decompress-GEMM on the coded weights; between them run
the operators of one decoding step:

    enc_qk_norm_rope     q, k norms, rotation, v: fp32 GEMM rows -> BF16 draft rows
    enc_tree_attention   the tree's nodes over the paged cache and the tree
    enc_verify_tree      accepted nodes and the next token, from random numbers
    enc_cache_commit     accepted rows become cache rows

The accepted tokens are distributed as if they had been drawn from the whole
model one at a time; at temperature 0 they are the most likely ones (where two
are equally likely up to the rounding of BF16 activations, either).
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from lossless_weight_compression_amd import enc  # noqa: E402


class Model:
    """Random BF16 weights in linear-layer layout, coded once."""

    def __init__(self, hidden=512, layers=3, heads=8, kv_heads=2, head_dim=64, ffn=1024, vocab=2048, max_pos=4096,
                 seed=0, device="cuda"):
        self.hidden, self.layers, self.heads, self.kv_heads, self.head_dim = hidden, layers, heads, kv_heads, head_dim
        self.ffn, self.vocab = ffn, vocab
        g = torch.Generator().manual_seed(seed)

        def coded(n, k, scale):
            w = (torch.randn(n, k, generator=g) * scale * k ** -0.5).to(torch.bfloat16).to(device)
            return enc.enc_compress(w, 512) + (n,)

        qkv = (heads + 2 * kv_heads) * head_dim
        self.blocks = []
        for layer in range(layers):
            s = 1.0 if layer == 0 else 0.4          # later layers correct the first one
            self.blocks.append(dict(qkv=coded(qkv, hidden, 1.0), o=coded(hidden, heads * head_dim, s),
                                    up=coded(2 * ffn, hidden, 1.0), down=coded(hidden, ffn, s),
                                    qw=torch.ones(head_dim, dtype=torch.bfloat16, device=device),
                                    kw=torch.ones(head_dim, dtype=torch.bfloat16, device=device)))
        self.embedding = (torch.randn(vocab, hidden, generator=g)).to(torch.bfloat16).to(device)
        self.head = coded(vocab, hidden, 3.0)
        angle = torch.arange(max_pos)[:, None] * 10000.0 ** (-torch.arange(0, head_dim, 2) / head_dim)
        self.angles = torch.cat([angle.cos(), angle.sin()], 1).float().to(device)

    @staticmethod
    def product(x, coded):
        stream, info, n = coded
        return enc.enc_decompress_gemm_nt(x, stream, info, n)

    @staticmethod
    def norm(x):
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Decoder:
    """B sequences with their cache, drafting trees of up to `nodes` nodes."""

    def __init__(self, model, batch, nodes=8, page=16, max_len=1024, seed=0, temperature=1.0):
        m = self.model = model
        self.batch, self.nodes, self.temperature = batch, nodes, temperature
        entries = max_len // page
        self.cache = enc.Cache.empty(2 * m.layers, batch * entries, page, (m.kv_heads, m.head_dim), batch, entries)
        self.seqs = torch.arange(batch, dtype=torch.int32, device="cuda")
        self.rng = torch.Generator(device="cuda").manual_seed(seed)

    def uniform(self, *shape):
        return torch.rand(shape, generator=self.rng, device="cuda")

    def probabilities(self, logits):
        if self.temperature == 0:
            return torch.nn.functional.one_hot(logits.argmax(-1), logits.shape[-1]).float()
        return torch.softmax(logits / self.temperature, -1)

    def forward(self, tokens, depth, seen, layers):
        """Logits after every node of the trees, and the nodes' K and V rows in
        every plane: tokens, depth [B, T]; seen: mask words or None (a chain)."""
        m = self.model
        B, T = tokens.shape
        x = m.embedding[tokens.long()].float().view(B * T, m.hidden)
        positions = (self.cache.lens[:, None] + depth).view(-1).to(torch.int32)
        rows = torch.empty(2 * layers, B, T, m.kv_heads, m.head_dim, dtype=torch.bfloat16, device="cuda")
        for layer in range(layers):
            w = m.blocks[layer]
            y = m.product(m.norm(x), w["qkv"]).view(B * T, -1, m.head_dim)
            q, k, v = y.split((m.heads, m.kv_heads, m.kv_heads), 1)
            k_new, v_new = rows[2 * layer], rows[2 * layer + 1]
            q, _, _ = enc.enc_qk_norm_rope(
                q, k, v, positions, m.angles, w["qw"], w["kw"],
                out=(torch.empty(B * T, m.heads, m.head_dim, dtype=torch.bfloat16, device="cuda"),
                     k_new.view(B * T, m.kv_heads, m.head_dim), v_new.view(B * T, m.kv_heads, m.head_dim)))
            a, _ = enc.enc_tree_attention(q.view(B, T, m.heads, m.head_dim), k_new, v_new, self.cache.data[2 * layer],
                                          self.cache.data[2 * layer + 1], self.cache.table, self.cache.lens, mask=seen)
            x = x + m.product(a.view(B * T, -1), w["o"])
            gate, up = m.product(m.norm(x), w["up"]).split(m.ffn, 1)
            x = x + m.product((torch.nn.functional.silu(gate) * up).to(torch.bfloat16), w["down"])
        return m.product(m.norm(x), m.head).view(B, T, m.vocab), rows

    def commit(self, rows, path, count):
        enc.enc_cache_commit(self.cache, self.seqs, rows, path, count)

    def prefill(self, prompt):
        """Cache a prompt [B, n], all but its last token, and return that one."""
        for at in range(0, prompt.shape[1] - 1, enc.ENC_TREE_MAX_NODES):
            part = prompt[:, at:min(at + enc.ENC_TREE_MAX_NODES, prompt.shape[1] - 1)]
            n = part.shape[1]
            order = torch.arange(n, dtype=torch.int32, device="cuda").repeat(self.batch, 1)
            _, rows = self.forward(part, order, None, self.model.layers)
            self.commit(rows, order, torch.full((self.batch,), n, dtype=torch.int32, device="cuda"))
            if int(self.cache.status):
                raise RuntimeError("the cache refused the prompt's rows: %d" % int(self.cache.status))
        return prompt[:, -1].contiguous()

    def plain_step(self, pending):
        """One token a sequence, without drafts: nodes = 1."""
        zero = torch.zeros(self.batch, 1, dtype=torch.int32, device="cuda")
        logits, rows = self.forward(pending[:, None], zero, None, self.model.layers)
        path, count, token = enc.enc_verify_tree(zero - 1, pending[:, None].contiguous(), self.probabilities(logits), None,
                                                 self.uniform(self.batch, 1))
        self.commit(rows, path, count)
        return token

    def draft(self, pending):
        """A tree from the first layer: two branches at the root, then chains.
        Parents, depths, tokens, and the distribution after each node that its
        children were drawn from."""
        B, T = self.batch, self.nodes
        parents = torch.tensor([-1, 0, 0] + list(range(1, T - 2)), dtype=torch.int32)[:T]
        depth = torch.zeros(T, dtype=torch.int32)
        allowed = torch.eye(T, dtype=torch.bool)
        for i in range(1, T):
            depth[i] = depth[parents[i]] + 1
            allowed[i] |= allowed[parents[i]]
        words = (allowed.to(torch.int64) << torch.arange(T)).sum(1)     # T <= 64: one word a node
        dev = lambda t: t.to("cuda").repeat(B, *[1] * t.dim())  # noqa: E731
        self.tree = dev(parents), dev(depth), dev(words)[..., None].contiguous()
        tokens = torch.zeros(B, T, dtype=torch.int32, device="cuda")
        tokens[:, 0] = pending
        q = torch.zeros(B, T, self.model.vocab, device="cuda")
        for level in range(int(depth.max())):
            n = int((depth <= level).sum())
            logits, _ = self.forward(tokens[:, :n].contiguous(), self.tree[1][:, :n].contiguous(),
                                     self.tree[2][:, :n].contiguous(), 1)
            q[:, :n] = self.probabilities(logits)
            for i in range(n, int((depth <= level + 1).sum())):
                tokens[:, i] = torch.multinomial(q[:, int(parents[i])], 1, generator=self.rng)[:, 0].to(torch.int32)
        return tokens, q

    def step(self, pending):
        """Draft, run, verify, commit. Returns (next pending token, tokens of the
        accepted nodes [B, T], how many)."""
        tokens, q = self.draft(pending)
        parents, depth, words = self.tree
        logits, rows = self.forward(tokens, depth, words, self.model.layers)
        path, count, token = enc.enc_verify_tree(parents, tokens, self.probabilities(logits), q,
                                                 self.uniform(self.batch, self.nodes))
        self.commit(rows, path, count)
        return token, tokens.gather(1, path.clamp_min(0).long()), count


def generate(decoder, prompt, n, speculate=True):
    """At least n tokens after the prompt for each sequence, and the steps taken."""
    pending = decoder.prefill(prompt)
    out = [[] for _ in range(decoder.batch)]
    steps = 0
    while min(map(len, out)) < n:
        steps += 1
        if speculate:
            pending, kept, count = decoder.step(pending)
            for b, (row, c) in enumerate(zip(kept.tolist(), count.tolist())):
                out[b] += row[1:c]                  # node 0 was the pending token
        else:
            pending = decoder.plain_step(pending)
        for b, t in enumerate(pending.tolist()):
            out[b].append(t)
        if int(decoder.cache.status):               # nothing was appended: what followed would miss these rows
            raise RuntimeError("the cache refused the step's rows: %d" % int(decoder.cache.status))
    return [o[:n] for o in out], steps


def main():
    model = Model()
    prompt = torch.randint(0, model.vocab, (2, 40), dtype=torch.int32, generator=torch.Generator().manual_seed(1)).cuda()
    for temperature in (0.0, 1.0):
        _, plain_steps = generate(Decoder(model, 2, temperature=temperature), prompt, 64, speculate=False)
        decoder = Decoder(model, 2, temperature=temperature)
        _, steps = generate(decoder, prompt, 64)
        assert int(decoder.cache.status) == 0
        print("temperature %g: 64 tokens a sequence in %d steps, without drafts %d" % (temperature, steps, plain_steps))


if __name__ == "__main__":
    main()
