"""Plain implementations of the decoding-step operators, in 64 bits (and, where
the definition fixes the arithmetic, in exactly that arithmetic). Nothing here
is shared with the library."""
import math

import numpy as np


# ------------------------------------------------------------------ head norms, rotation
def norm_rope(x, w, table, positions, eps, adjacent, norm=True):
    """x [tokens, heads, dim] float64 -> the same, normed and rotated; also the
    magnitudes that the rounding of the two products of each value scales with."""
    x = x.astype(np.float64)
    y = x
    if norm:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if w is not None:
        y = y * w.astype(np.float64)
    size = np.abs(y)
    y, size = y.copy(), size.copy()
    if table is not None:
        rot = table.shape[1]
        half = rot // 2
        for t, p in enumerate(positions):
            if not 0 <= p < table.shape[0]:
                y[t] = np.nan
                continue
            for i in range(half):
                c, s = float(table[p, i]), float(table[p, half + i])
                a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
                u, v = y[t, :, a].copy(), y[t, :, b].copy()
                y[t, :, a], y[t, :, b] = u * c - v * s, v * c + u * s
                size[t, :, a], size[t, :, b] = (abs(u * c) + abs(v * s)), (abs(v * c) + abs(u * s))
    return y, size


# ------------------------------------------------------------------ attention
def tree_attention(q, k_new, v_new, k_cache, v_cache, table, lens, seen, scale, seqs=None, nodes=None):
    """All float64. seen [batch, nodes, nodes] bool. Sums run over the keys a row
    sees and nothing else. Returns out, lse and sum_j p_j |v_j|."""
    B, T, H, D = q.shape
    G = k_new.shape[2]
    page = k_cache.shape[1]
    out, size = np.zeros((B, T, H, D)), np.zeros((B, T, H, D))
    lse = np.full((B, T, H), -np.inf)
    for b in range(B):
        s = b if seqs is None else int(seqs[b])
        n = int(lens[s]) if 0 <= s < len(lens) else 0
        n = max(0, min(n, table.shape[1] * page))
        live = T if nodes is None else max(0, min(int(nodes[b]), T))
        idx = [(int(table[s, j // page]), j % page) for j in range(n)]
        pg, rw = np.array([i[0] for i in idx], int), np.array([i[1] for i in idx], int)
        for h in range(H):
            g = h // (H // G)
            kc = k_cache[pg, rw, g] if n else np.zeros((0, D))
            vc = v_cache[pg, rw, g] if n else np.zeros((0, D))
            for i in range(live):
                cols = [j for j in range(live) if seen[b, i, j]]
                k = np.concatenate([kc, k_new[b, cols, g]])
                v = np.concatenate([vc, v_new[b, cols, g]])
                if len(k) == 0:
                    continue
                with np.errstate(invalid="ignore", over="ignore"):
                    x = (k @ q[b, i, h]) * scale
                    top = x.max()
                    p = np.exp(x - top)
                    total = p.sum()
                    out[b, i, h] = (p[:, None] * v).sum(0) / total
                    size[b, i, h] = (p[:, None] * np.abs(v)).sum(0) / total
                    lse[b, i, h] = top + math.log(total) if total == total and total > 0 else np.nan
    return out, lse, size


def mask_words(seen):
    """bool [batch, nodes, nodes] -> int64 words."""
    B, T, _ = seen.shape
    W = -(-T // 64)
    words = np.zeros((B, T, W), np.uint64)
    for j in range(T):
        words[:, :, j // 64] |= seen[:, :, j].astype(np.uint64) << np.uint64(j % 64)
    return words.view(np.int64)


def ancestors(parents):
    B, T = parents.shape
    seen = np.zeros((B, T, T), bool)
    for b in range(B):
        for i in range(T):
            j = i
            while True:
                seen[b, i, j] = True
                if j == 0 or not 0 <= parents[b, j] < j:
                    break
                j = parents[b, j]
    return seen


# ------------------------------------------------------------------ verification
def _mass(x):
    return np.rint(x.astype(np.float64) * 2.0 ** 40).astype(np.int64)   # exact product; ties to even


def verify(parents, tokens, target, draft, u, nodes=None):
    """The definition, one sequence and node at a time; float32 steps, whole sums."""
    f = np.float32
    B, T = tokens.shape
    V = target.shape[2]
    path, count, token = np.full((B, T), -1, np.int32), np.zeros(B, np.int32), np.full(B, -1, np.int32)

    def clean(row):
        row = row.astype(f)
        return np.where(row > 0, np.minimum(row, f(1)), f(0)).astype(f)

    for b in range(B):
        live = T if nodes is None else max(0, min(int(nodes[b]), T))
        if live == 0:
            continue
        cur, walked, last = 0, [0], 0
        r = clean(target[b, 0])
        left = r
        while True:
            kids = [i for i in range(last + 1, live) if parents[b, i] == cur]
            if not kids:
                break
            c = kids[0]
            last = c
            x = int(tokens[b, c])
            if not 0 <= x < V:
                continue
            if draft is None:
                q = np.zeros(V, f)
                q[x] = 1
            else:
                q = clean(draft[b, cur])
            if f(u[b, c]) * q[x] < r[x]:
                cur = c
                walked.append(c)
                r = clean(target[b, c])
                left = r
                continue
            over = np.maximum(r - q, f(0)).astype(f)
            total = int(_mass(over).sum())
            if total:
                left = over
                r = (over / f(f(total) * f(2.0 ** -40))).astype(f)
        path[b, :len(walked)] = walked
        count[b] = len(walked)
        m = _mass(left)
        total = int(m.sum())
        if total:
            u0 = float(u[b, 0])
            point = int(min(max(u0, 0.0), 1 - 2.0 ** -24) * 2 ** 24) if u0 == u0 else 0
            goal = total * point >> 24
            token[b] = int(np.searchsorted(np.cumsum(m), goal, side="right"))
    return path, count, token


# ------------------------------------------------------------------ pages
class Pages:
    """The cache as plain lists: what each call must leave behind."""

    def __init__(self, data, table, lens, refs):
        self.data, self.table, self.lens, self.refs = data.copy(), table.copy(), lens.copy(), refs.copy()

    def commit(self, seqs, draft, path, count):
        P, page = self.data.shape[0], self.data.shape[2]
        S, M = self.table.shape
        T = path.shape[1]
        errors, plans, need = [], [], 0
        for b, s in enumerate(seqs):
            n = int(count[b])
            if not 0 <= s < S:
                errors.append(-1)
                continue
            if not 0 <= n <= T:
                errors.append(-2)
                continue
            if any(not 0 <= path[b, j] < T for j in range(n)):
                errors.append(-2)
            length = int(self.lens[s])
            if not 0 <= length <= M * page:
                errors.append(-4)
                continue
            if length + n > M * page:
                errors.append(-3)
                continue
            fresh, leave = [], None
            for p in sorted({t // page for t in range(length, length + n)}):
                e = int(self.table[s, p])
                if p == length // page and length % page:
                    if not 0 <= e < len(self.refs):
                        errors.append(-4)
                    elif self.refs[e] > 1:
                        leave = e
                        fresh.append(p)
                else:
                    if e != -1:
                        errors.append(-4)
                    fresh.append(p)
            plans.append((b, int(s), length, n, fresh, leave))
            need += len(fresh)
        if errors:
            return min(errors)
        free = [g for g in range(len(self.refs)) if self.refs[g] == 0]
        if need > len(free):
            return need - len(free)
        for b, s, length, n, fresh, leave in plans:
            for p in fresh:
                g = free.pop(0)
                if leave is not None and p == length // page:
                    self.refs[leave] -= 1
                    self.data[:, g, :length % page] = self.data[:, leave, :length % page]
                self.table[s, p] = g
                self.refs[g] = 1
            for j in range(n):
                t = length + j
                self.data[:, self.table[s, t // page], t % page] = draft[:, b, path[b, j]]
            self.lens[s] = length + n
        return 0

    def fork(self, src, dst):
        S = len(self.lens)
        for s, d in zip(src, dst):
            if not (0 <= s < S and 0 <= d < S) or s == d:
                continue
            for e in self.table[d]:
                if e >= 0:
                    self.refs[e] -= 1
            for e in self.table[s]:
                if e >= 0:
                    self.refs[e] += 1
            self.table[d] = self.table[s]
            self.lens[d] = self.lens[s]

    def truncate(self, seqs, lens):
        page = self.data.shape[2]
        for s, n in zip(seqs, lens):
            if not 0 <= s < len(self.lens):
                continue
            keep = max(0, min(int(self.lens[s]), int(n)))
            for p in range(-(-keep // page), self.table.shape[1]):
                e = self.table[s, p]
                if e >= 0:
                    self.refs[e] -= 1
                    self.table[s, p] = -1
            self.lens[s] = keep
