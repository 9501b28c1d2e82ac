"""Cases that measure what decoding several continuations of a prompt adds to a step.

Three operators run around the fused decompress-GEMMs of such a step:

- ``norm``: the norm after a block, its gate, the residual sum and the norm before the next block, in one pass over
  the GEMM's rows;
- ``attention``: sequences of a batch that were forked from the same prompt read its cached rows once for all of them;
  how many they share is either known to the program or found on the device in the cache's table;
- ``sample``: temperature, top-k, top-p and min-p on the logits, and the next token drawn from given random numbers or
  the filtered probabilities handed on to verification.

Sizes are those of the 8B-shaped layer that the benchmark uses (rows of 4096, 32 query heads, 8 KV heads of 128, a
vocabulary of 128256) and generic ones around it.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token between two GEMMs: fp32 rows in, fp32 residual stream, bf16 rows for the next GEMM
        norm_case("norm.one_token", tokens=1, width=4096, y="fp32", h="fp32", out="bf16"),
        # 24 sequences of 33 nodes, norms on both sides of the block, one gate for each sequence, weights around 0
        norm_case("norm.batch", tokens=24 * 33, width=2560, y="bf16", h="bf16", out="bf16", post=True, gate=24,
                  offset=True),
        # a prompt of 8192 tokens, norms on both sides, a gate for each channel
        norm_case("norm.prompt", tokens=8192, width=4096, y="fp32", h="fp32", out="bf16", post=True, gate=1),
        # rows of an odd length, a gate for each token
        norm_case("norm.odd", tokens=515, width=1537, y="fp16", h="fp32", out="fp16", post=True, gate=515),
        # 4 continuations of a prompt of 1021 tokens: the smallest call of a decoding loop
        attention_case("attention.few", groups=1, members=4, t=1, hq=32, hkv=8, d=128, prefix=1021, tail=37, page=16),
        # 64 continuations of a prompt of 8192 tokens, each with up to 512 tokens of its own
        attention_case("attention.samples", groups=1, members=64, t=1, hq=32, hkv=8, d=128, prefix=8192, tail=512,
                       page=16, find=True),
        # 6 prompts of up to 4099 tokens with up to 12 continuations each and trees of 8 nodes, heads of 64, fp16
        attention_case("attention.trees", groups=6, members=12, t=8, hq=16, hkv=4, d=64, prefix=4099, tail=300, page=64,
                       kind="tree", dt="fp16", ragged=True, find=True),
        # 16 questions about a document of 131072 tokens
        attention_case("attention.document", groups=1, members=16, t=1, hq=32, hkv=8, d=128, prefix=131072, tail=1000,
                       page=64, lse=True),
        # the next token of one sequence
        sample_case("sample.one_row", rows=1, vocab=128256, dt="fp32", filters="tkpm"),
        # 64 sequences with settings of their own, 16-bit logits with many ties
        sample_case("sample.batch", rows=64, vocab=128256, dt="bf16", filters="tkpm"),
        # the target's probabilities after each of 6 nodes of 16 sequences, for verification
        sample_case("sample.probabilities", rows=16 * 6, vocab=32003, dt="fp32", filters="tp", every=6, probs="fp32",
                    token=False),
        # a large batch, temperature and top-p
        sample_case("sample.large", rows=256, vocab=128256, dt="fp32", filters="tp"),
    ]


def norm_case(name, tokens, width, y, h, out, post=False, gate=0, offset=False):
    """gate: rows of gates (0: none), each for tokens / gate tokens in turn."""
    return dict(name=name, op="norm", tokens=tokens, width=width, y=y, h=h, out=out, post=post, gate=gate, offset=offset)


def attention_case(name, groups, members, t, hq, hkv, d, prefix, tail, page, kind="chain", dt="bf16", ragged=False,
                   find=False, lse=False):
    return dict(name=name, op="attention", groups=groups, members=members, t=t, hq=hq, hkv=hkv, d=d, prefix=prefix,
                tail=tail, page=page, kind=kind, dt=dt, ragged=ragged, find=find, lse=lse)


def sample_case(name, rows, vocab, dt, filters, every=1, probs="", token=True):
    """filters: t(emperature), k, p and m(in-p); every: rows that share one setting."""
    return dict(name=name, op="sample", rows=rows, vocab=vocab, dt=dt, filters=filters, every=every, probs=probs,
                token=token)


def log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "attention", "attention", "sample", "sample"])
    if op == "norm":
        width = rng.choice([log_uniform(rng, 64, 16384), 8 * log_uniform(rng, 8, 2048)])
        tokens = log_uniform(rng, 1, max(1, min(8192, 8192 * 4096 // width)))
        gate = rng.choice([0, 1, tokens, next(n for n in (6, 5, 4, 3, 2, 1) if tokens % n == 0)])
        case = norm_case("", tokens, width, rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                         rng.choice(["fp32", "fp32", "bf16", "fp16"]), rng.choice(["bf16", "fp16"]),
                         rng.random() < 0.5, gate, rng.random() < 0.3)
    elif op == "attention":
        d = rng.choice([64, 96, 128, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 7])
        t = rng.choice([1, 1, 1, 2, 5, 8, 33])
        members = rng.choice([2, 3, 4, 7, 16, 40, 64])
        prefix = log_uniform(rng, 16, 65536)
        tail = log_uniform(rng, 1, 1024)
        room = min((7 << 30) // (t * hq), (2 << 30) // hkv) // (d * members)   # as much work and data as the largest listed case
        tail = min(tail, max(1, room // 2))
        prefix = min(prefix, max(16, room - tail))
        most = max(1, min(8, room // (prefix + tail), (256 << 20) // (members * (prefix + tail) * hkv * d)))
        case = attention_case("", rng.randint(1, most), members, t, hq, hkv, d, prefix, tail,
                              rng.choice([8, 16, 20, 64, 128]), rng.choice(["chain", "tree"]), rng.choice(["bf16", "fp16"]),
                              rng.random() < 0.6, rng.random() < 0.5, rng.random() < 0.3)
    else:
        vocab = log_uniform(rng, 1000, 150000)
        rows = log_uniform(rng, 1, max(1, min(512, 256 * 128256 // vocab)))
        probs = rng.choice(["", "", "fp32", "bf16"])
        if probs:
            rows = max(1, rows // 2)
        case = sample_case("", rows, vocab, rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                           rng.choice(["", "t", "tk", "tp", "tkp", "tm", "tkpm", "kpm"]),
                           next(n for n in rng.sample([1, 2, 3, 4], 4) if rows % n == 0), probs,
                           not probs or rng.random() < 0.5)
    del case["name"]
    return case


def work(case):
    if case["op"] == "norm":
        n = case["tokens"] * case["width"]
        moved = n * (SIZE[case["y"]] + 2 * SIZE[case["h"]] + SIZE[case["out"]]) + 2 * case["gate"] * case["width"]
        return {"bytes": moved + (4 if case["post"] else 2) * case["width"], "flops": 9 * n}
    if case["op"] == "attention":
        sizes, prefixes, tails = shape_of(case)
        t, hq, hkv, d = (case[k] for k in ("t", "hq", "hkv", "d"))
        # a prompt's keys and values once for its continuations, everybody's own ones, q and the result
        keys = sum(prefixes) + sum(tails) + sum(sizes) * t
        seen = sum(n * p for n, p in zip(sizes, prefixes)) + sum(tails) + sum(sizes) * t
        return {"bytes": 2 * (2 * keys * hkv * d + 2 * sum(sizes) * t * hq * d), "flops": 4 * t * hq * d * seen}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * (SIZE[case["dt"]] + SIZE.get(case["probs"], 0)), "flops": 8 * n}


# ------------------------------------------------------------------ inputs
def spread(n, low, high, salt):
    """n whole numbers over [low, high], the same for a case whatever the seed, so that work() knows them."""
    return [low + (i * 2654435761 + salt * 40503 + 12345) % 1000003 % (high - low + 1) for i in range(n)]


def shape_of(case):
    """Continuations and prompt length of each group, and every sequence's own cached tokens."""
    groups, members, prefix = case["groups"], case["members"], case["prefix"]
    sizes, prefixes = [members] * groups, [prefix] * groups
    if case["ragged"]:
        sizes, prefixes = spread(groups, 1, members, prefix), spread(groups, 0, prefix, members)
        sizes[0], prefixes[0] = members, prefix
    tails = spread(sum(sizes), 0, case["tail"], case["t"])
    return sizes, prefixes, tails


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    state = {"norm": prepare_norm, "attention": prepare_attention, "sample": prepare_sample}[case["op"]](case, seed)
    state["case"] = case
    return state


def prepare_norm(case, seed):
    g = generator(seed)
    n, width = case["tokens"], case["width"]
    normal = lambda *shape: torch.randn(shape, device="cuda", generator=g)  # noqa: E731
    weight = lambda: ((0.0 if case["offset"] else 1.0) + 0.1 * normal(width)).to(torch.bfloat16)  # noqa: E731
    return dict(y=(1.7 * normal(n, width)).to(DT[case["y"]]), h=(4.0 * normal(n, width)).to(DT[case["h"]]),
                gate=(0.5 * normal(case["gate"], width)).to(torch.bfloat16) if case["gate"] else None,
                w_post=weight() if case["post"] else None, w_pre=weight(), h_scale=1.0,
                y_scale=0.25 if case["gate"] else 1.0, eps=1e-6)


def prepare_attention(case, seed):
    g = generator(seed)
    cpu = torch.Generator().manual_seed(seed)
    t, hq, hkv, d, page = (case[k] for k in ("t", "hq", "hkv", "d", "page"))
    dt = DT[case["dt"]]
    sizes, prefixes, tails = shape_of(case)
    b = sum(sizes)
    need = 3
    for n, p in zip(sizes, prefixes):
        need += p // page
    at = 0
    for n, p in zip(sizes, prefixes):
        for i in range(n):
            need += -(-(p % page + tails[at + i]) // page)
        at += n
    lens = [p + tails[i] for i, p in enumerate(p for n, p in zip(sizes, prefixes) for _ in range(n))]
    order = torch.randperm(need, generator=cpu).to(torch.int32)
    table = torch.full((b, max(1, -(-max(lens) // page))), -1, dtype=torch.int32)
    data = torch.empty((2, need, page, hkv, d), dtype=dt, device="cuda").normal_(generator=g)
    used = seq = 0
    copies = []
    for n, p in zip(sizes, prefixes):
        full = p // page                                   # a prompt's whole pages are shared
        shared = order[used:used + full]
        used += full
        first = None
        for i in range(n):
            own_pages = -(-(p % page + tails[seq]) // page)
            table[seq, :full] = shared
            table[seq, full:full + own_pages] = order[used:used + own_pages]
            if p % page:                                   # its last rows were copied when they were written behind
                if first is None:
                    first = int(order[used])
                else:
                    copies.append((first, int(order[used]), p % page))
            used += own_pages
            seq += 1
    for source, goal, rows in copies:
        data[:, goal, :rows] = data[:, source, :rows]
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + n)
    normal = lambda *shape: torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)  # noqa: E731
    node = torch.arange(t)
    allowed = torch.eye(t, dtype=torch.bool).repeat(b, 1, 1)
    if case["kind"] == "chain":
        allowed |= node[:, None] >= node
    else:
        for i in range(1, t):
            up = torch.randint(0, i, (b,), generator=cpu)
            allowed[:, i] |= allowed[torch.arange(b), up]
    words = -(-t // 64)
    bits = torch.zeros(b, t, words * 64, dtype=torch.int64)
    bits[:, :, :t] = allowed
    mask = (bits.view(b, t, words, 64) << torch.arange(64)).sum(-1)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(q=normal(b, t, hq, d), k_new=normal(b, t, hkv, d), v_new=normal(b, t, hkv, d), data=data,
                table=table.cuda(), lens=ints(lens), refs=torch.ones(need, dtype=torch.int32, device="cuda"),
                seqs=torch.arange(b, dtype=torch.int32, device="cuda"), starts=ints(starts), prefix=ints(prefixes),
                mask=mask.cuda(), scale=1.0 / math.sqrt(d))


def prepare_sample(case, seed):
    g = generator(seed)
    rows, vocab, n = case["rows"], case["vocab"], case["rows"] // case["every"]
    logits = torch.empty(rows, vocab, device="cuda")
    for r in range(0, rows, 64):                           # some distributions are sharper than others
        part = logits[r:r + 64]
        part.normal_(generator=g).mul_(1.5 + 2.5 * torch.rand(part.shape[0], 1, device="cuda", generator=g))
    state = dict(logits=logits.to(DT[case["dt"]]), u=torch.rand(rows, device="cuda", generator=g))
    pick = lambda *values: torch.tensor(values, device="cuda")[  # noqa: E731
        torch.randint(0, len(values), (n,), device="cuda", generator=g)]
    has = case["filters"]
    state["temperature"] = pick(0.0, 0.3, 0.6, 0.7, 0.8, 1.0, 1.0, 1.2, 1.5) if "t" in has else None
    state["top_k"] = pick(0, 1, 10, 20, 50, 50, 200, 1000).to(torch.int32) if "k" in has else None
    state["top_p"] = pick(1.0, 0.5, 0.8, 0.9, 0.9, 0.95, 0.99) if "p" in has else None
    state["min_p"] = pick(0.0, 0.01, 0.05, 0.1, 0.2) if "m" in has else None
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return OWN[state["case"]["op"]](state)
    return PLAIN[state["case"]["op"]](state)


def own_norm(s):
    from lossless_weight_compression_amd import enc
    case = s["case"]
    h, x = enc.enc_block_norm(s["h"], s["y"], gate=s["gate"], w_post=s["w_post"], w_pre=s["w_pre"],
                              post_norm=case["post"], h_scale=s["h_scale"], y_scale=s["y_scale"], eps=s["eps"],
                              unit_offset=case["offset"], out_dtype=DT[case["out"]])
    return {"h": h, "x": x}


def own_attention(s):
    from lossless_weight_compression_amd import enc
    case, data = s["case"], s["data"]
    if "ws" not in s:  # kept from step to step, as a serving loop does
        s["cache"] = enc.Cache(data, s["table"], s["lens"], s["refs"])
        s["ws"] = enc.prefix_attention_workspace(s["q"], s["k_new"], s["table"], data[0], s["starts"])
    shared = enc.enc_cache_shared(s["cache"], s["seqs"], s["starts"]) if case["find"] else s["prefix"]
    out, lse = enc.enc_prefix_attention(s["q"], s["k_new"], s["v_new"], data[0], data[1], s["table"], s["lens"],
                                        s["starts"], shared, mask=s["mask"], scale=s["scale"], return_lse=case["lse"],
                                        ws=s["ws"])
    outputs = {"out": out}
    if case["lse"]:
        outputs["lse"] = lse
    if case["find"]:
        outputs["shared"] = shared
    return outputs


def own_sample(s):
    from lossless_weight_compression_amd import enc
    case = s["case"]
    if "ws" not in s:
        s["ws"] = enc.sample_workspace(s["logits"])
    token, probs = enc.enc_sample(s["logits"], s["u"] if case["token"] else None, temperature=s["temperature"],
                                  top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"], return_probs=bool(case["probs"]),
                                  probs_dtype=DT.get(case["probs"]), ws=s["ws"])
    outputs = {}
    if case["token"]:
        outputs["token"] = token
    if case["probs"]:
        outputs["probs"] = probs
    return outputs


OWN = {"norm": own_norm, "attention": own_attention, "sample": own_sample}


def plain_norm(s):
    case = s["case"]
    offset = 1.0 if case["offset"] else 0.0
    z, h = s["y"].float(), s["h"].float()
    if case["post"]:
        z = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + s["eps"]) * (s["w_post"].float() + offset)
    if s["gate"] is not None:
        n, width = z.shape
        z = (z.view(s["gate"].shape[0], -1, width) * s["gate"].float()[:, None]).view(n, width)
    h = s["h_scale"] * h + s["y_scale"] * z
    x = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + s["eps"]) * (s["w_pre"].float() + offset)
    return {"h": h.to(s["h"].dtype), "x": x.to(DT[case["out"]])}


def plain_attention(s):
    case, table, lens, data = s["case"], s["table"], s["lens"], s["data"]
    b, t, hq, d = s["q"].shape
    page, hkv = data.shape[2:4]
    group, most = hq // hkv, table.shape[1] * page
    node = torch.arange(t, device=table.device)
    outs, lses = [], []
    step = max(1, (1 << 29) // (most * hkv * d))           # sequences at a time, for the copies' sake
    for first in range(0, b, step):
        part = slice(first, first + step)
        rows = table[part].clamp_min(0).long()
        n = rows.shape[0]
        k = torch.cat([data[0][rows].view(n, most, hkv, d), s["k_new"][part]], 1).transpose(1, 2).float()
        v = torch.cat([data[1][rows].view(n, most, hkv, d), s["v_new"][part]], 1).transpose(1, 2).float()
        q = s["q"][part].float().view(n, t, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, t * group, d)
        cached = torch.arange(most, device=q.device) < lens[part][:, None]
        tree = (s["mask"][part][:, :, node // 64] >> (node % 64)) & 1 != 0
        seen = torch.cat([cached[:, None].expand(n, t, most), tree], 2).repeat_interleave(group, 1)[:, None]
        scores = (torch.matmul(q, k.transpose(2, 3)) * s["scale"]).masked_fill_(~seen, -math.inf)
        top = scores.amax(-1, keepdim=True)
        weights = scores.sub_(top).exp_()
        total = weights.sum(-1, keepdim=True)
        out = torch.matmul(weights, v) / total
        outs.append(out.view(n, hkv, t, group, d).permute(0, 2, 1, 3, 4).reshape(n, t, hq, d).to(s["q"].dtype))
        lses.append((top + total.log()).view(n, hkv, t, group).permute(0, 2, 1, 3).reshape(n, t, hq))
    outputs = {"out": torch.cat(outs)}
    if case["lse"]:
        outputs["lse"] = torch.cat(lses)
    if case["find"]:
        shared, at = [], 0
        for n in shape_of(case)[0]:                        # leading table entries that all of a group have alike
            rows = table[at:at + n]
            alike = ((rows == rows[:1]) & (rows >= 0)).all(0).int().cumprod(0).sum() * page
            shared.append(torch.minimum(alike, lens[at:at + n].amin()))
            at += n
        outputs["shared"] = torch.stack(shared).int()
    return outputs


def settings(s, name, otherwise):
    """A setting's value for each row, in 64 bits."""
    rows = s["logits"].shape[0]
    if s[name] is None:
        return torch.full((rows, 1), otherwise, device="cuda", dtype=torch.float64)
    return s[name].double().repeat_interleave(s["case"]["every"])[:, None]


def plain_sample(s):
    case = s["case"]
    logits = s["logits"].double()                          # borders between tokens are finer than 32 bits
    rows, vocab = logits.shape
    temperature = settings(s, "temperature", 1.0)
    x = logits / torch.where(temperature > 0, temperature, 1.0)
    e = (x - x.amax(-1, keepdim=True)).exp()
    weights, order = torch.sort(e, dim=-1, descending=True, stable=True)
    rank = torch.arange(vocab, device="cuda")
    top_k = settings(s, "top_k", 0.0)
    keep = (rank < torch.where((top_k > 0) & (temperature > 0), top_k, float(vocab))) & (
        (rank < 1) | (temperature > 0))
    weights = torch.where(keep, weights, 0.0)
    top_p = settings(s, "top_p", 1.0)
    before = weights.cumsum(-1) - weights
    total = weights.sum(-1, keepdim=True)
    keep &= (before < top_p * total) | (top_p >= 1) | (rank < 1)
    keep &= (weights >= settings(s, "min_p", 0.0)) | (rank < 1)
    kept = torch.zeros_like(e).scatter_(-1, order, torch.where(keep, weights, 0.0))
    outputs = {}
    if case["token"]:
        run_sum = kept.cumsum(-1)
        goal = s["u"].double()[:, None] * run_sum[:, -1:]
        outputs["token"] = (run_sum <= goal).sum(-1).int()
    if case["probs"]:
        outputs["probs"] = (kept / kept.sum(-1, keepdim=True)).to(DT[case["probs"]])
    return outputs


PLAIN = {"norm": plain_norm, "attention": plain_attention, "sample": plain_sample}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": exact_norm, "attention": exact_attention, "sample": exact_sample}[case["op"]](case, s)


def exact_norm(case, s):
    def normed(x, w):
        size = (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt()
        return x / size * (w.double() + (1 if case["offset"] else 0))

    z = s["y"].double()
    if case["post"]:
        z = normed(z, s["w_post"])
    if s["gate"] is not None:
        every = case["tokens"] // case["gate"]
        z = z * s["gate"].double()[torch.arange(case["tokens"], device="cuda") // every]
    h = s["h"].double() * s["h_scale"] + z * s["y_scale"]
    return {"h": h, "x": normed(h, s["w_pre"])}


def exact_attention(case, s):
    b, t, hq, d = s["q"].shape
    page, hkv = s["data"].shape[2:4]
    if b * hkv * (case["prefix"] + case["tail"]) * d > 1 << 32:
        return None
    out = torch.zeros(b, t, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(b, t, hq, dtype=torch.float64, device="cuda")
    lens, mask = s["lens"].tolist(), s["mask"].cpu()
    for i in range(b):
        n = lens[i]
        used = s["table"][i, :-(-n // page)].long()
        allowed = torch.tensor([[int(mask[i, r, j // 64]) >> (j % 64) & 1 for j in range(t)] for r in range(t)]).cuda()
        for h in range(hkv):
            k = torch.cat([s["data"][0, used, :, h].reshape(-1, d)[:n], s["k_new"][i, :, h]]).double()
            v = torch.cat([s["data"][1, used, :, h].reshape(-1, d)[:n], s["v_new"][i, :, h]]).double()
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            x = torch.matmul(s["q"][i, :, heads].double(), k.T) * s["scale"]
            x[..., n:] = torch.where(allowed[:, None] == 0, -math.inf, x[..., n:])
            lse[i, :, heads] = torch.logsumexp(x, -1)
            out[i, :, heads] = torch.matmul((x - lse[i, :, heads, None]).exp(), v)
    outputs = {"out": out}
    if case["lse"]:
        outputs["lse"] = lse
    if case["find"]:
        outputs["shared"] = None                           # a whole number
    return outputs


def exact_sample(case, s):
    rows, vocab = s["logits"].shape
    tokens, probs = [], torch.zeros(rows, vocab, dtype=torch.float64, device="cuda") if case["probs"] else None
    get = lambda name, r, otherwise: (  # noqa: E731
        otherwise if s[name] is None else float(s[name][r // case["every"]]))
    for r in range(rows):
        row = s["logits"][r].double()
        heat, k = get("temperature", r, 1.0), int(get("top_k", r, 0))
        values, index = torch.sort(row, dim=0, descending=True, stable=True)
        if heat <= 0:
            values, index = values[:1], index[:1]
        elif k > 0:
            values, index = values[:k], index[:k]
        p = torch.softmax(values / (heat if heat > 0 else 1.0), 0)
        share, least = get("top_p", r, 1.0), get("min_p", r, 0.0)
        if share < 1:
            n = int(torch.searchsorted(p.cumsum(0), torch.tensor([share], dtype=p.dtype, device="cuda"))) + 1
            p, index = p[:n], index[:n]
        n = max(1, int((p >= least * p[0]).sum()))
        p, index = p[:n] / p[:n].sum(), index[:n]
        if case["probs"]:
            probs[r, index] = p
        if case["token"]:
            index, at = index.sort()
            run_sum = p[at].cumsum(0)
            place = torch.searchsorted(run_sum, s["u"][r].double().view(1) * run_sum[-1], right=True)
            tokens.append(index[place.clamp_max(len(index) - 1)])
    outputs = {}
    if case["token"]:
        outputs["token"] = torch.cat(tokens)
    if case["probs"]:
        outputs["probs"] = probs
    return outputs
