"""fp64 oracle of the calls around a tree of drafts (layout, attention, the walk), of
sampling with cuts, and of the cache's pages: test infrastructure only.

Sources: "Attention Drift", section 2 (the target scores the drafted tokens in one pass and
the longest valid prefix is kept: here of every line of a tree), and "P-EAGLE: parallel
speculative decoding in vLLM", KV cache and CUDA graphs (a paged cache addressed by slots).
"""

from __future__ import annotations

import numpy as np


def lines(parent):
    """Of each node: the node and its ancestors.  A parent that is no earlier node is none."""
    out = []
    for j, p in enumerate(parent):
        out.append((out[p] if 0 <= p < j else []) + [j])
    return out


def pack(bits, words):
    """[n][m] truths -> [n][words] uint32 as int32."""
    w = np.zeros((len(bits), words), np.uint32)
    for j, row in enumerate(bits):
        for i in np.flatnonzero(row):
            if i < 32 * words:
                w[j, i // 32] |= np.uint32(1 << (i % 32))
    return w.view(np.int32)


def unpack(words):
    """[n][words] int32 -> [n][32 words] truths."""
    w = np.ascontiguousarray(words).view(np.uint32)
    return (w[:, :, None] >> np.arange(32, dtype=np.uint32) & 1).astype(bool).reshape(len(w), -1)


def tree_layout(qsl, seq_len, parent, table, num_blocks, bs, words):
    """(mask, pos, slot) of all rows; those of no request are -7."""
    T = len(parent)
    mask, pos, slot = np.full((T, words), -7, np.int32), np.full(T, -7, np.int64), np.full(T, -7, np.int64)
    for r in range(len(seq_len)):
        lo, hi = int(qsl[r]), int(qsl[r + 1])
        n = hi - lo
        ctx = int(seq_len[r]) - n
        of = lines(parent[lo:hi])
        for j in range(n):
            bits = np.zeros((1, 32 * words), bool)
            if j < 32 * words:
                bits[0, of[j]] = True
            mask[lo + j] = pack(bits, words)[0]
            pos[lo + j] = ctx + (len(of[j]) - 1 if j < 32 * words else 0)
            t = ctx + j
            blk = table[r][t // bs] if 0 <= t < table.shape[1] * bs else -1
            slot[lo + j] = blk * bs + t % bs if 0 <= blk < num_blocks and j < 32 * words else -1
    return mask, pos, slot


def tree_attention(qsl, seq_len, q, k_cache, v_cache, table, mask, sink=None):
    """(out, spread) as oracle.pe_paged.chunk_attention, the rows' own keys by their masks."""
    q = np.asarray(q, dtype=np.float64)
    T, H, hd = q.shape
    nb, G, bs, _ = k_cache.shape
    out, spread = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    for r in range(len(seq_len)):
        lo, hi = int(qsl[r]), int(qsl[r + 1])
        n, L = hi - lo, int(seq_len[r])
        if n == 0:
            continue
        out[lo:hi], spread[lo:hi] = 0.0, 0.0
        t = np.arange(max(L, 0))
        blk = table[r][t // bs]
        t = t[(blk >= 0) & (blk < nb)]
        if len(t) == 0:
            continue
        blk = table[r][t // bs]
        bits = unpack(mask[lo:hi])
        node = t - (L - n)
        see = np.ones((n, len(t)), bool)
        own = node >= 0
        see[:, own] = np.where(node[own] < bits.shape[1], bits[:, np.minimum(node[own], bits.shape[1] - 1)], False)
        for h in range(H):
            g = h // (H // G)
            K, V = k_cache[blk, g, t % bs], v_cache[blk, g, t % bs]
            any_row = see.any(0)  # what no row sees may hold anything
            s = np.where(see, q[lo:hi, h] @ np.where(any_row[:, None], K, 0.0).T / np.sqrt(hd), -np.inf)
            for j in range(n):
                x = s[j, see[j]]
                if len(x) == 0:
                    continue
                top = max(x.max(), float(sink[h]) if sink is not None else -np.inf)
                w = np.exp(x - top)
                w /= w.sum() + (np.exp(float(sink[h]) - top) if sink is not None else 0.0)
                out[lo + j, h] = w @ V[see[j]]
                spread[lo + j, h] = w @ np.abs(V[see[j]])
    return out, spread


def tree_accept(qsl, parent, tok, target):
    """(accepted, path, bonus); the path of rows of no request is -7."""
    B = len(qsl) - 1
    acc, bonus, path = np.zeros(B, np.int32), np.full(B, -1, np.int32), np.full(len(tok), -7, np.int32)
    for r in range(B):
        lo, hi = int(qsl[r]), int(qsl[r + 1])
        n = hi - lo
        if n == 0:
            continue
        up = [p if 0 <= p < j else -1 for j, p in enumerate(parent[lo:hi])]
        walk = [0]
        while True:
            want = target[lo + walk[-1]]
            kids = [j for j in range(n) if up[j] == walk[-1] and tok[lo + j] == want >= 0]
            if not kids:
                break
            walk.append(kids[0])
        acc[r], bonus[r] = len(walk) - 1, target[lo + walk[-1]]
        path[lo:hi] = walk + [-1] * (n - len(walk))
    return acc, path, bonus


def compact(qsl, seq_len, accepted, path, table, k_cache, v_cache):
    """Caches [layers][blocks][G][bs][hd] after the accepted nodes have moved."""
    k, v = k_cache.copy(), v_cache.copy()
    nb, bs = k.shape[1], k.shape[3]
    for r in range(len(seq_len)):
        lo, hi = int(qsl[r]), int(qsl[r + 1])
        n = hi - lo
        ctx = int(seq_len[r]) - n
        a = min(max(int(accepted[r]), 0), max(n - 1, 0))
        way = [0] + [int(x) for x in path[lo + 1:lo + 1 + a]]
        if any(y <= x or y >= n for x, y in zip(way, way[1:])):
            continue

        def place(t):
            blk = table[r][t // bs] if 0 <= t < table.shape[1] * bs else -1
            return (int(blk), t % bs) if 0 <= blk < nb else None

        for d in range(1, a + 1):
            f, t = place(ctx + way[d]), place(ctx + d)
            if f and t:
                for c in (k, v):
                    c[:, t[0], :, t[1]] = c[:, f[0], :, f[1]]
    return k, v


class Pool:
    """The pool's calls, entry by entry: table [rows][max_blocks], refs [num_blocks]."""

    def __init__(self, table, refs, bs):
        self.table, self.refs, self.bs, self.refused = table.copy(), refs.copy(), bs, False

    def _entries(self, length):
        e = -(-length // self.bs)
        return None if length < 0 or e > self.table.shape[1] else e

    def _hand_out(self, needs):
        """Pages of each entry: None where it is refused."""
        free = [int(i) for i in np.flatnonzero(self.refs == 0)]
        at, out = 0, []
        for need in needs:
            if need is None:
                out.append(None)
                continue
            out.append(free[at:at + need] if at + need <= len(free) or need == 0 else None)
            at += need
        self.refused |= any(x is None for x in out)
        return out

    def reserve(self, rows, lengths):
        needs = []
        for row, length in zip(rows, lengths):
            e = self._entries(length)
            ok = 0 <= row < len(self.table) and list(rows).count(row) == 1 and e is not None
            needs.append(int((self.table[row, :e] < 0).sum()) if ok else None)
        for row, length, pages in zip(rows, lengths, self._hand_out(needs)):
            if pages:
                at = np.flatnonzero(self.table[row, :self._entries(length)] < 0)
                self.table[row, at] = pages
                self.refs[pages] = 1

    def fork(self, parents, children, lengths, caches=()):
        needs = []
        nb = len(self.refs)
        for p, c, length in zip(parents, children, lengths):
            e = self._entries(length)
            rows = len(self.table)
            ok = 0 <= p < rows and 0 <= c < rows and e is not None and list(children).count(c) == 1 \
                and c not in list(parents) and (self.table[c] < 0).all() \
                and all(0 <= x < nb and self.refs[x] > 0 for x in self.table[p, :e])
            needs.append(int(length % self.bs != 0) if ok else None)
        for p, c, length, pages in zip(parents, children, lengths, self._hand_out(needs)):
            if pages is None:
                continue
            full, part = divmod(length, self.bs)
            self.table[c, :full] = self.table[p, :full]
            np.add.at(self.refs, self.table[p, :full], 1)
            if part:
                self.table[c, full], self.refs[pages[0]] = pages[0], 1
                for x in caches:
                    x[:, pages[0], :, :part] = x[:, self.table[p, full], :, :part]

    def free(self, rows):
        for row in rows:
            if not 0 <= row < len(self.table):
                self.refused = True
                continue
            for page in self.table[row]:
                if 0 <= page < len(self.refs):
                    if self.refs[page] > 0:
                        self.refs[page] -= 1
                    else:
                        self.refused = True
            self.table[row] = -1


FP32_MAX = float(np.finfo(np.float32).max)


def _sample_row(x, temp, k, p, min_p, g):
    """(token, lead) of one row: the score's lead over the next kept token's."""
    V = len(x)
    if temp == 0:
        return int(np.argmax(x)), np.inf  # (numpy's argmax takes the first NaN)
    top = x.max()
    if not np.isfinite(top):
        return -1, np.inf
    order = np.lexsort((np.arange(V), -x))
    w = np.exp((x[order] - top) / temp)
    m = k if 0 < k < V else V
    keep = np.arange(V) < m
    before = np.concatenate([[0.0], np.cumsum(w[:m])[:-1], np.full(V - m, np.inf)])
    if p < 1:
        keep &= (before < p * w[:m].sum()) | (np.arange(V) == 0)
    if min_p > 0:
        keep &= (w >= min_p) | (np.arange(V) == 0)
    keep &= ~np.isneginf(x[order])
    with np.errstate(invalid="ignore"):
        s = np.where(keep, (x[order] - top) / temp + np.where(keep, g[order].astype(np.float64), 0.0), -np.inf)
    s[np.isnan(s) | (s < -FP32_MAX)] = -np.inf
    if np.isneginf(s).all():
        return -1, np.inf
    best = s.max()
    tok = int(order[s == best].min())
    rest = s[order != tok]
    with np.errstate(invalid="ignore"):
        lead = best - rest.max() if len(rest) else np.inf
    return tok, 0.0 if np.isnan(lead) else lead


def sample(qsl, logits, temperature, top_k, top_p, min_p, gumbel):
    """(token, clear): of each row; -7 for rows of no request.  clear: the answer stays the same
    if the bounds of the weights move by 2e-5 of their size, and the winning score is ahead by 1e-4."""
    logits = np.asarray(logits, dtype=np.float64)
    T = len(logits)
    token, clear = np.full(T, -7, np.int64), np.ones(T, bool)
    for r in range(len(qsl) - 1):
        t = 1.0 if temperature is None else float(temperature[r])
        t = min(max(t, 1e-30), 1e30) if t > 0 else 0.0
        k = 0 if top_k is None else int(top_k[r])
        p = 1.0 if top_p is None else float(top_p[r])
        m = 0.0 if min_p is None else float(min_p[r])
        p, m = 1.0 if np.isnan(p) else p, 0.0 if np.isnan(m) else m
        for row in range(int(qsl[r]), int(qsl[r + 1])):
            tok, lead = _sample_row(logits[row], t, k, p, m, gumbel[row])
            token[row] = tok
            near = [_sample_row(logits[row], t, k, min(p * f, 1.0) if p < 1 else p, m * g, gumbel[row])[0]
                    for f in (1 - 2e-5, 1 + 2e-5) for g in (1 - 2e-5, 1 + 2e-5)] if p < 1 or 0 < m < 1 else []
            clear[row] = lead > 1e-4 and all(x == tok for x in near)
    return token, clear


def _sample_holds(x, temp, k, p, min_p, g, tok):
    """Whether a row's token may stand: it may be kept if the bounds of the weights move by 2e-5 of their size,
    and no token that is kept wherever they lie has a score ahead of its by more than the fp32 forms of the two are
    off: 1e-6 of their terms (a quotient and a sum, up to ten rescalings of a running score, 2^-24 each)."""
    V = len(x)
    top = x.max()
    if temp == 0 or not np.isfinite(top):
        return tok == _sample_row(x, temp, k, p, min_p, g)[0]
    order = np.lexsort((np.arange(V), -x))
    w = np.exp((x[order] - top) / temp)
    first = np.arange(V) == 0
    m = k if 0 < k < V else V
    before = np.concatenate([[0.0], np.cumsum(w[:m])[:-1], np.full(V - m, np.inf)])

    def kept(by):
        keep = (np.arange(V) < m) & ~np.isneginf(x[order])
        if p < 1:
            keep &= (before < p * by * w[:m].sum()) | first
        if min_p > 0:
            keep &= (w >= (min_p / by if min_p <= 1 else min_p)) | first
        return keep

    with np.errstate(invalid="ignore"):
        term, noise = (x[order] - top) / temp, g[order].astype(np.float64)
        score = np.where(np.isneginf(term) | np.isnan(noise), -np.inf, term + noise)
        score[score < -FP32_MAX] = -np.inf
        sure = x[order] - top > -FP32_MAX
        off = np.where(np.isfinite(score), 1e-6 * (np.abs(term) + np.abs(noise)), 0.0)
    low = np.where(kept(1 - 2e-5) & sure, score - off, -np.inf)
    if tok == -1:
        return bool(np.isneginf(low).all())
    if not 0 <= tok < V:
        return False
    at = int(np.flatnonzero(order == tok)[0])
    if not kept(1 + 2e-5)[at] or np.isneginf(score[at]):
        return False
    return bool(score[at] + off[at] >= low.max())


def sample_holds(qsl, logits, temperature, top_k, top_p, min_p, gumbel, token):
    """Of each row of a request: whether its token is one of those that the formulas allow (_sample_holds).
    Rows of no request: whether it is -7."""
    logits = np.asarray(logits, dtype=np.float64)
    ok = np.asarray(token) == -7
    for r in range(len(qsl) - 1):
        t = 1.0 if temperature is None else float(temperature[r])
        t = min(max(t, 1e-30), 1e30) if t > 0 else 0.0
        k = 0 if top_k is None else int(top_k[r])
        p = 1.0 if top_p is None else float(top_p[r])
        m = 0.0 if min_p is None else float(min_p[r])
        p, m = 1.0 if np.isnan(p) else p, 0.0 if np.isnan(m) else m
        for row in range(int(qsl[r]), int(qsl[r + 1])):
            ok[row] = _sample_holds(logits[row], t, k, p, m, gumbel[row], int(token[row]))
    return ok
