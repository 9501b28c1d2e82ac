"""Cases that measure the operators of one speculative decoding step.

Four operators run between a step's fused decompress-GEMMs and after its last one:

- ``rope``: RMS norms of each query and key head, the rotary position embedding,
  and the conversion of the GEMM's fp32 rows to the cache's type, in one pass;
- ``attention``: a tree of drafted tokens against a paged cache and itself;
- ``verify``: drafted tokens accepted or rejected against the target's
  probabilities from given random numbers, and the next token drawn;
- ``cache``: accepted rows compacted into the cache's pages, pages shared by
  forks, copied when written, and freed.

Sizes are those of the 8B-shaped layer that the benchmark uses (32 query heads,
8 KV heads of 128, a vocabulary of 128256, 32 layers) and generic ones around it.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token of one sequence: the smallest call of a decoding loop
        rope_case("rope.one_token", tokens=1, hq=32, hkv=8, d=128, rot=128, src="fp32", dst="bf16"),
        # 24 sequences with 33-node trees, heads of 64 in one packed bf16 projection, adjacent pairs, half rotated
        rope_case("rope.tree_batch", tokens=24 * 33, hq=16, hkv=4, d=64, rot=32, src="bf16", dst="bf16",
                  packed=True, adjacent=True),
        # a prompt of 8192 tokens
        rope_case("rope.prompt", tokens=8192, hq=32, hkv=8, d=128, rot=128, src="fp32", dst="bf16"),
        # one new token of one sequence with a short history
        attention_case("attention.one_token", b=1, t=1, hq=32, hkv=8, d=128, length=1021, page=16, kind="chain"),
        # 8 sequences with 33-node trees over about 4000 tokens each, heads of 64, fp16
        attention_case("attention.tree", b=8, t=33, hq=16, hkv=4, d=64, length=4099, page=64, kind="tree", dt="fp16",
                       ragged=True, lse=True),
        # a long history: 64-node tree over 131072 tokens, one sequence
        attention_case("attention.long", b=1, t=64, hq=32, hkv=8, d=128, length=131072, page=128, kind="tree"),
        # a full batch: 64 sequences of up to 8192 tokens, chains of 8
        attention_case("attention.batch", b=64, t=8, hq=32, hkv=8, d=128, length=8192, page=16, kind="chain",
                       ragged=True),
        # one sequence, a chain of 5 drafts after the pending token
        verify_case("verify.chain", b=1, t=6, vocab=128256, width=1, dt="fp32"),
        # 32 sequences, 16-node trees with up to 3 candidates a node
        verify_case("verify.tree", b=32, t=16, vocab=128256, width=3, dt="fp32"),
        # one sequence commits what an 8-node tree had accepted, all 32 layers
        cache_case("cache.commit_one", kind="commit", b=1, t=8, planes=64, row=2048, length=1021, page=16),
        # 64 sequences commit from 32-node trees, 8 layers
        cache_case("cache.commit_batch", kind="commit", b=64, t=32, planes=16, row=2048, length=300, page=16),
        # one prompt of 8191 tokens shared by 16 continuations, each of which then writes on its own
        cache_case("cache.branch", kind="branch", b=16, t=8, planes=16, row=2048, length=8191, page=64),
    ]


def rope_case(name, tokens, hq, hkv, d, rot, src, dst, packed=False, adjacent=False):
    return dict(name=name, op="rope", tokens=tokens, hq=hq, hkv=hkv, d=d, rot=rot, src=src, dst=dst, packed=packed,
                adjacent=adjacent)


def attention_case(name, b, t, hq, hkv, d, length, page, kind, dt="bf16", ragged=False, lse=False):
    return dict(name=name, op="attention", b=b, t=t, hq=hq, hkv=hkv, d=d, length=length, page=page, kind=kind, dt=dt,
                ragged=ragged, lse=lse)


def verify_case(name, b, t, vocab, width, dt, point=False):
    return dict(name=name, op="verify", b=b, t=t, vocab=vocab, width=width, dt=dt, point=point)


def cache_case(name, kind, b, t, planes, row, length, page):
    return dict(name=name, op="cache", kind=kind, b=b, t=t, planes=planes, row=row, length=length, page=page)


def log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rope", "attention", "attention", "verify", "cache"])
    if op == "rope":
        d = rng.choice([64, 80, 96, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 7])
        tokens = log_uniform(rng, 1, max(1, min(8192, 8192 * 48 * 128 // ((hq + 2 * hkv) * d))))
        case = rope_case("", tokens, hq, hkv, d, rng.choice([d, d // 2]), rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                         rng.choice(["bf16", "fp16"]), rng.random() < 0.5, rng.random() < 0.3)
    elif op == "attention":
        d = rng.choice([64, 96, 128, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 7])
        t = rng.choice([1, 2, 5, 8, 16, 33, 64, 100])
        length = log_uniform(rng, 16, 65536)
        most = max(1, min(64, (128 << 20) // (length * hkv * d), (256 << 20) // (length * hq * t)))
        case = attention_case("", log_uniform(rng, 1, most), t, hq, hkv, d, length, rng.choice([8, 16, 20, 64, 128]),
                              rng.choice(["chain", "tree"]), rng.choice(["bf16", "fp16"]), rng.random() < 0.6,
                              rng.random() < 0.3)
    elif op == "verify":
        vocab = log_uniform(rng, 1000, 130000)
        t = rng.choice([2, 4, 6, 9, 16, 24])
        b = log_uniform(rng, 1, max(1, min(48, 32 * 16 * 128256 // (t * vocab))))
        case = verify_case("", b, t, vocab, rng.choice([1, 1, 2, 3]), rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                           rng.random() < 0.3)
    else:
        kind = rng.choice(["commit", "branch"])
        planes = rng.choice([2, 8, 16, 64])
        row = rng.choice([256, 1024, 2048])
        length = log_uniform(rng, 1, 2000)
        b = log_uniform(rng, 1, max(1, min(64, (512 << 20) // (planes * row * (length + 64)))))
        case = cache_case("", kind, b, rng.choice([1, 4, 8, 17, 32]), planes, row, length, rng.choice([8, 16, 48, 64]))
    del case["name"]
    return case


def work(case):
    op = case["op"]
    if op == "rope":
        values = case["tokens"] * (case["hq"] + 2 * case["hkv"]) * case["d"]
        table = case["tokens"] * case["rot"] * 4
        return {"bytes": values * (SIZE[case["src"]] + SIZE[case["dst"]]) + table + 4 * case["tokens"], "flops": 8 * values}
    if op == "attention":
        keys = sum(history(case)) + case["b"] * case["t"]  # each key and value once, q and o once
        b, t, hq, hkv, d = (case[k] for k in ("b", "t", "hq", "hkv", "d"))
        return {"bytes": 2 * (2 * keys * hkv * d + 2 * b * t * hq * d), "flops": 4 * t * hq * d * keys}
    if op == "verify":
        # per sequence the row that the next token is drawn from, and what was taken off it: at a walk's end one
        # rejection is the rule, and a target row and a draft row are read
        rows = case["b"] * (1 if case["point"] else 2)
        return {"bytes": rows * case["vocab"] * SIZE[case["dt"]], "flops": 4 * rows * case["vocab"]}
    # each accepted row read and written once in every plane; a forked page's filled rows copied once; tables
    rows = sum(accepted_counts(case))
    if case["kind"] == "branch":
        rows += case["b"] * (case["length"] % case["page"])
    entries = case["b"] * -(-(case["length"] + case["t"]) // case["page"])
    return {"bytes": 2 * rows * case["planes"] * case["row"] + 8 * entries, "flops": rows}


# ------------------------------------------------------------------ inputs
def spread(n, low, high, salt):
    """n whole numbers over [low, high], the same for a case whatever the seed, so that work() knows them."""
    return [low + (i * 2654435761 + salt * 40503 + 12345) % 1000003 % (high - low + 1) for i in range(n)]


def history(case):
    """Cached tokens of each sequence: ragged batches hold everything from nothing to the full length."""
    if not case["ragged"]:
        return [case["length"]] * case["b"]
    lens = spread(case["b"], 0, case["length"], case["t"])
    lens[0] = case["length"]
    return lens


def accepted_counts(case):
    return spread(case["b"], 1, case["t"], case["length"])


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def random_tree(b, t, width, seed):
    """Parents of b trees of t nodes, node 0 the root, at most `width` children a node, parents before children."""
    g = torch.Generator()
    g.manual_seed(seed)
    parents = torch.full((b, t), -1, dtype=torch.int32)
    for s in range(b):
        room = [0] * max(width - int(torch.randint(0, width, (1,), generator=g)), 1)
        picks = torch.rand(t, generator=g).tolist()
        for i in range(1, t):
            parents[s, i] = room.pop(int(picks[i] * min(len(room), width)))
            room += [i] * (1 + int(picks[i] * 7919) % width)
    return parents


def ancestors(parents):
    """allowed[b, i, j]: node j is node i or one of its ancestors."""
    b, t = parents.shape
    allowed = torch.eye(t, dtype=torch.bool).repeat(b, 1, 1)
    for i in range(1, t):
        allowed[:, i] |= allowed[torch.arange(b), parents[:, i].long()]
    return allowed


def words_of(allowed):
    """The masks as 64-bit words, bit j % 64 of word j / 64 for node j."""
    b, t, _ = allowed.shape
    words = -(-t // 64)
    bits = torch.zeros(b, t, words * 64, dtype=torch.int64)
    bits[:, :, :t] = allowed
    return (bits.view(b, t, words, 64) << torch.arange(64)).sum(-1)


def prepare(case, seed):
    state = {"rope": prepare_rope, "attention": prepare_attention, "verify": prepare_verify,
             "cache": prepare_cache}[case["op"]](case, seed)
    state["case"] = case
    return state


def prepare_rope(case, seed):
    g = generator(seed)
    n, hq, hkv, d, rot = (case[k] for k in ("tokens", "hq", "hkv", "d", "rot"))
    x = torch.randn(n, hq + 2 * hkv, d, device="cuda", generator=g).to(DT[case["src"]])
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if not case["packed"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    limit = max(2 * n, 4096)
    inv = 500000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    angle = torch.arange(limit, dtype=torch.float64)[:, None] * inv
    table = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
    return dict(q=q, k=k, v=v, positions=torch.randint(0, limit, (n,), device="cuda", generator=g, dtype=torch.int32),
                table=table, qw=(1 + 0.1 * torch.randn(d, device="cuda", generator=g)).to(torch.bfloat16),
                kw=(1 + 0.1 * torch.randn(d, device="cuda", generator=g)).to(torch.bfloat16), eps=1e-6)


def prepare_attention(case, seed):
    g = generator(seed)
    b, t, hq, hkv, d, page = (case[k] for k in ("b", "t", "hq", "hkv", "d", "page"))
    dt = DT[case["dt"]]
    lens = history(case)
    most = -(-max(lens) // page)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((b, max(most, 1)), -1, dtype=torch.int32)
    at = 0
    for s in range(b):
        table[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
    normal = lambda *shape: torch.empty(shape, dtype=dt, device="cuda").normal_(generator=g)  # noqa: E731
    if case["kind"] == "chain":
        allowed = torch.ones(t, t, dtype=torch.bool).tril().repeat(b, 1, 1)
    else:
        allowed = ancestors(random_tree(b, t, 3, seed))
    return dict(q=normal(b, t, hq, d), k_new=normal(b, t, hkv, d), v_new=normal(b, t, hkv, d),
                k_cache=normal(pages, page, hkv, d), v_cache=normal(pages, page, hkv, d), table=table.cuda(),
                lens=torch.tensor(lens, dtype=torch.int32).cuda(), mask=words_of(allowed).cuda(),
                scale=1.0 / math.sqrt(d), lse=case["lse"])


def prepare_verify(case, seed):
    g = generator(seed)
    b, t, vocab = case["b"], case["t"], case["vocab"]
    dt = DT[case["dt"]]
    if case["width"] == 1:
        parents = (torch.arange(t, dtype=torch.int32) - 1).repeat(b, 1)
    else:
        parents = random_tree(b, t, case["width"], seed)
    parents = parents.cuda()
    logits = torch.randn(b, t, vocab, device="cuda", generator=g) * 3.0
    target = torch.softmax(logits, -1).to(dt)
    draft = torch.softmax(logits + 0.7 * torch.randn(b, t, vocab, device="cuda", generator=g), -1).to(dt)
    del logits
    # each node's token is drawn from the draft's probabilities after its parent
    up = parents.clamp_min(0).long()
    draws = torch.multinomial(draft.float().view(b * t, vocab), case["width"], replacement=True, generator=g)
    index = torch.arange(t, device="cuda")
    earlier = ((parents[:, :, None] == parents[:, None, :]) & (index[:, None] > index)).sum(-1)
    rank = torch.minimum(earlier, torch.tensor(case["width"] - 1, device="cuda"))
    tokens = draws.view(b, t, -1)[torch.arange(b, device="cuda")[:, None], up, rank].to(torch.int32)
    u = torch.rand(b, t, device="cuda", generator=g)
    return dict(parents=parents, tokens=tokens, target=target, draft=None if case["point"] else draft, u=u)


def prepare_cache(case, seed):
    g = generator(seed)
    b, t, planes, row, length, page = (case[k] for k in ("b", "t", "planes", "row", "length", "page"))
    entries = -(-(length + t) // page) + 1
    filled = -(-length // page)
    holders = b if case["kind"] == "commit" else 1
    pages = holders * filled + b * (2 + -(-t // page)) + 5
    cpu = torch.Generator().manual_seed(seed)
    order = torch.randperm(pages, generator=cpu).to(torch.int32)
    table = torch.full((holders if case["kind"] == "commit" else 1 + b, entries), -1, dtype=torch.int32)
    table[:holders, :filled] = order[:holders * filled].view(holders, filled)
    lens = torch.zeros(table.shape[0], dtype=torch.int32)
    lens[:holders] = length
    refs = torch.zeros(pages, dtype=torch.int32)
    refs[order[:holders * filled].long()] = 1
    half = lambda *shape: torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # noqa: E731
    counts = accepted_counts(case)
    path = torch.full((b, t), -1, dtype=torch.int32)
    for s in range(b):
        kept = torch.randperm(t - 1, generator=cpu)[:counts[s] - 1] + 1
        path[s, 0] = 0
        path[s, 1:counts[s]] = kept.sort().values.to(torch.int32)
    writers = torch.arange(b, dtype=torch.int32) + (0 if case["kind"] == "commit" else 1)
    return dict(data=half(planes, pages, page, row // 2), table=table.cuda(), lens=lens.cuda(), refs=refs.cuda(),
                draft=half(planes, b, t, row // 2), path=path.cuda(),
                count=torch.tensor(counts, dtype=torch.int32).cuda(), seqs=writers.cuda(),
                base=torch.full((b,), length, dtype=torch.int32, device="cuda"),
                parent=torch.zeros(b, dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return OWN[state["case"]["op"]](state)
    return PLAIN[state["case"]["op"]](state)


def own_rope(s):
    from lossless_weight_compression_amd import enc
    q, k, v = enc.enc_qk_norm_rope(s["q"], s["k"], s["v"], s["positions"], s["table"], s["qw"], s["kw"], eps=s["eps"],
                                   adjacent=s["case"]["adjacent"], out_dtype=DT[s["case"]["dst"]])
    return {"q": q, "k": k, "v": v}


def own_attention(s):
    from lossless_weight_compression_amd import enc
    if "ws" not in s:  # kept from step to step, as a serving loop does
        s["ws"] = enc.tree_attention_workspace(s["q"], s["k_new"], s["table"], s["k_cache"])
    out, lse = enc.enc_tree_attention(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                      mask=s["mask"], scale=s["scale"], return_lse=s["lse"], ws=s["ws"])
    return {"out": out, "lse": lse} if s["lse"] else {"out": out}


def own_verify(s):
    from lossless_weight_compression_amd import enc
    if "ws" not in s:
        s["ws"] = enc.verify_tree_workspace(s["tokens"], s["target"])
    path, count, token = enc.enc_verify_tree(s["parents"], s["tokens"], s["target"], s["draft"], s["u"], ws=s["ws"])
    return {"path": path, "count": count, "token": token}


def own_cache(s):
    from lossless_weight_compression_amd import enc
    if "cache" not in s:
        s["cache"] = enc.Cache(s["data"], s["table"], s["lens"], s["refs"])
        s["ws"] = enc.cache_workspace(s["cache"], s["path"])
    if s["case"]["kind"] == "commit":
        enc.enc_cache_truncate(s["cache"], s["seqs"], s["base"])
    else:
        enc.enc_cache_fork(s["cache"], s["parent"], s["seqs"])
    enc.enc_cache_commit(s["cache"], s["seqs"], s["draft"], s["path"], s["count"], ws=s["ws"])
    return {"data": s["data"], "table": s["table"], "lens": s["lens"], "refs": s["refs"]}


OWN = {"rope": own_rope, "attention": own_attention, "verify": own_verify, "cache": own_cache}


def plain_rope(s):
    case, rot = s["case"], s["case"]["rot"]
    half = rot // 2
    row = s["table"][s["positions"].long()]
    cos, sin = row[:, None, :half], row[:, None, half:]

    def one(x, w):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * w.float()
        if case["adjacent"]:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:rot]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([turned, x[..., rot:]], -1).to(DT[case["dst"]])

    return {"q": one(s["q"], s["qw"]), "k": one(s["k"], s["kw"]), "v": s["v"].float().to(DT[case["dst"]])}


def plain_attention(s):
    b, t, hq, d = s["q"].shape
    page, hkv = s["k_cache"].shape[1:3]
    group, most = hq // hkv, s["table"].shape[1] * page
    table = s["table"].clamp_min(0).long()
    # [b, hkv, keys, d]: the cached rows, then the tree's
    k = torch.cat([s["k_cache"][table].view(b, most, hkv, d), s["k_new"]], 1).transpose(1, 2).float()
    v = torch.cat([s["v_cache"][table].view(b, most, hkv, d), s["v_new"]], 1).transpose(1, 2).float()
    q = s["q"].float().view(b, t, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, t * group, d)
    cached = torch.arange(most, device=q.device) < s["lens"][:, None]
    node = torch.arange(t, device=q.device)
    tree = (s["mask"][:, :, node // 64] >> (node % 64)) & 1 != 0
    seen = torch.cat([cached[:, None].expand(b, t, most), tree], 2)
    seen = seen.repeat_interleave(group, 1)[:, None]
    scores = (torch.matmul(q, k.transpose(2, 3)) * s["scale"]).masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_min(-3e38)
    weights = scores.sub_(top).exp_()
    total = weights.sum(-1, keepdim=True)
    out = torch.matmul(weights, v) / total
    out = out.view(b, hkv, t, group, d).permute(0, 2, 1, 3, 4).reshape(b, t, hq, d).to(s["q"].dtype)
    if not s["lse"]:
        return {"out": out}
    lse = (top + total.log()).view(b, hkv, t, group).permute(0, 2, 1, 3).reshape(b, t, hq)
    return {"out": out, "lse": lse}


def mass(x):
    """Probabilities as whole numbers of 2^-40, so that their sums are exact in any order."""
    return torch.round(x * 2.0 ** 40).to(torch.int64)


def plain_verify(s):
    parents, tokens, u = s["parents"].long(), s["tokens"].long(), s["u"]
    b, t = tokens.shape
    width = s["case"]["width"]
    index = torch.arange(t, device=u.device)
    rest = s["target"].float().clamp(0.0, 1.0)
    earlier = ((parents[:, :, None] == parents[:, None, :]) & (index[:, None] > index)).sum(-1)
    child = torch.full((b, t * width + 1), -1, device=u.device, dtype=torch.int64)
    place = torch.where(parents >= 0, parents.clamp_min(0) * width + earlier.clamp_max(width - 1), t * width)
    child = child.scatter(1, place, index.expand(b, t))[:, :-1].view(b, t, width)
    taken = torch.full_like(tokens, -1)
    left = rest  # what the next token is drawn from, up to a factor
    for j in range(width):  # all nodes at once: the j-th child of each
        c = child[:, :, j]
        x = tokens.gather(1, c.clamp_min(0))[..., None]
        live = (c >= 0) & (taken < 0)
        if s["draft"] is None:
            q = torch.zeros_like(rest).scatter_(2, x, 1.0)
        else:
            q = s["draft"].float().clamp(0.0, 1.0)
        ok = live & (u.gather(1, c.clamp_min(0)) * q.gather(2, x)[..., 0] < rest.gather(2, x)[..., 0])
        taken = torch.where(ok, c, taken)
        over = (rest - q).clamp_min(0.0)
        total = mass(over).sum(-1)
        use = (live & ~ok & (total > 0))[..., None]
        left = torch.where(use, over, left)
        rest = torch.where(use, over / (total.float() * 2.0 ** -40)[..., None], rest)
    # a node is on the path if it and every node above it was taken
    on = (taken.gather(1, parents.clamp_min(0)) == index) | (index == 0)
    up = parents.clamp_min(0)
    for _ in range(max(1, (t - 1).bit_length())):
        on, up = on & on.gather(1, up), up.gather(1, up)
    count = on.sum(1)
    path = torch.where(on, index, t).sort(1).values
    end = path.gather(1, count[:, None] - 1)
    path = torch.where(index < count[:, None], path, -1)
    run_sum = mass(left[torch.arange(b, device=u.device), end[:, 0]]).cumsum(1)
    total = run_sum[:, -1:]
    point = (u[:, :1].clamp(0.0, 1.0 - 2.0 ** -24) * 2.0 ** 24).long()
    goal = (total >> 24) * point + (((total & (2 ** 24 - 1)) * point) >> 24)
    token = torch.where(total > 0, (run_sum <= goal).sum(1, keepdim=True), -1)[:, 0]
    return {"path": path.int(), "count": count.int(), "token": token.int()}


def plain_cache(s):
    data, table, lens, refs, seqs = s["data"], s["table"], s["lens"], s["refs"], s["seqs"].long()
    planes, pages, page, row = data.shape
    b, t = s["path"].shape
    entry = torch.arange(table.shape[1], device=table.device)
    one = torch.ones((), dtype=torch.int32, device=table.device)

    def count_pages(entries, sign):
        refs.index_add_(0, entries.clamp_min(0).view(-1).long(), (entries >= 0).view(-1).int() * sign)

    if s["case"]["kind"] == "commit":  # back to the committed length
        lens[seqs] = torch.minimum(lens[seqs], s["base"])
        gone = entry >= ((lens[seqs] + page - 1) // page)[:, None]
        old = table[seqs]
        count_pages(torch.where(gone, old, -1), -1)
        table[seqs] = torch.where(gone, -1, old)
    else:  # the children let go of what they held and share the parent's pages
        old, new = table[seqs], table[s["parent"].long()]
        count_pages(old, -1)
        count_pages(new, 1)
        table[seqs] = new
        lens[seqs] = lens[s["parent"].long()]

    length, count = lens[seqs].long(), s["count"].long()
    slots = torch.arange(-(-t // page) + 1, device=table.device)
    at = length[:, None] // page + slots
    at_in = at.clamp_max(table.shape[1] - 1)
    old = table[seqs[:, None], at_in].long()
    touched = (at * page < (length + count)[:, None]) & (at < table.shape[1])
    shared = (old >= 0) & (refs[old.clamp_min(0)] > 1)
    want = touched & ((old < 0) | shared)
    rank = want.view(-1).cumsum(0)
    free = torch.searchsorted((refs == 0).cumsum(0), rank).view(b, -1)
    new = torch.where(want, free, old)
    write = touched.view(-1)
    table[seqs[:, None].expand_as(at)[touched], at_in[touched]] = new[touched].int()
    count_pages(torch.where(want & shared, old, -1), -1)
    refs.index_put_((new[want],), one)
    flat = data.view(planes, pages * page, row)
    within = torch.arange(page, device=table.device)
    copied = (want & shared)[:, 0, None] & (within < (length % page)[:, None])
    source, goal = (old[:, :1] * page + within)[copied], (new[:, :1] * page + within)[copied]
    flat[:, goal] = flat[:, source]
    step = torch.arange(t, device=table.device)
    taken = step < count[:, None]
    position = length[:, None] + step
    goal = new.gather(1, position // page - length[:, None] // page) * page + position % page
    source = torch.arange(b, device=table.device)[:, None] * t + s["path"].long()
    flat[:, goal[taken]] = s["draft"].view(planes, b * t, row)[:, source[taken]]
    lens[seqs] += s["count"]
    return {"data": data, "table": table, "lens": lens, "refs": refs}


PLAIN = {"rope": plain_rope, "attention": plain_attention, "verify": plain_verify, "cache": plain_cache}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return exact_rope(case, s)
    if case["op"] == "attention":
        return exact_attention(s)
    return None  # whole numbers and copies


def exact_rope(case, s):
    rot = case["rot"]
    outputs = {}
    for name in ("q", "k"):
        x = s[name].double()
        y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt() * s[name + "w"].double()
        pair = torch.arange(rot // 2, device=x.device)
        first, second = (2 * pair, 2 * pair + 1) if case["adjacent"] else (pair, pair + rot // 2)
        z = torch.complex(y[..., first], y[..., second])
        turn = s["table"].double()[s["positions"].long()]
        z = z * torch.complex(turn[:, :rot // 2], turn[:, rot // 2:])[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        outputs[name] = y
    outputs["v"] = s["v"].double()
    return outputs


def exact_attention(s):
    b, t, hq, d = s["q"].shape
    page, hkv = s["k_cache"].shape[1:3]
    out = torch.zeros(b, t, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(b, t, hq, dtype=torch.float64, device="cuda")
    lens, mask = s["lens"].tolist(), s["mask"].cpu()
    for i in range(b):
        n = lens[i]
        used = s["table"][i, :-(-n // page)].long()
        allowed = torch.tensor([[int(mask[i, r, j // 64]) >> (j % 64) & 1 for j in range(t)] for r in range(t)]).cuda()
        for h in range(hkv):
            k = torch.cat([s["k_cache"][used, :, h].reshape(-1, d)[:n], s["k_new"][i, :, h]]).double()
            v = torch.cat([s["v_cache"][used, :, h].reshape(-1, d)[:n], s["v_new"][i, :, h]]).double()
            for e in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                x = s["q"][i, :, e].double() @ k.T * s["scale"]
                x[:, n:][allowed == 0] = -math.inf
                lse[i, :, e] = torch.logsumexp(x, -1)
                out[i, :, e] = (x - lse[i, :, e, None]).exp() @ v
    return {"out": out, "lse": lse} if s["lse"] else {"out": out}
