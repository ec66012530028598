"""fp64 oracle of the paged attention calls and of verification by sampling: test
infrastructure only.

Sources: "P-EAGLE: parallel speculative decoding in vLLM", KV cache and CUDA
graphs (a paged cache addressed by slots, rejected rows at slot -1), and
"Attention Drift", section 2 (rejection sampling of the drafts against the
target's own distribution, the longest valid prefix accepted) and section 3 (the
per-head sink logit).
"""

from __future__ import annotations

import numpy as np


def norm_rotate(x, gain, pos, theta, eps):
    """x [T][heads][hd] fp64: optional RMS norm over hd, then the rotation of the
    pairs (i, i + hd/2) by pos * theta^(-2i/hd)."""
    x = np.asarray(x, dtype=np.float64)
    hd = x.shape[-1]
    if gain is not None:
        x = x * gain / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    half = hd // 2
    ang = np.asarray(pos, dtype=np.longdouble)[:, None] * \
        np.longdouble(theta) ** (-2 * np.arange(half, dtype=np.longdouble) / hd)
    z = (x[..., :half] + 1j * x[..., half:]) * \
        (np.cos(ang) + 1j * np.sin(ang)).astype(np.complex128)[:, None, :]
    return np.concatenate([z.real, z.imag], -1)


def qkv_append(qkv, H, G, gamma_q, gamma_k, pos, slot, k_cache, v_cache, theta=10000.0, eps=1e-6):
    """(q, k_cache, v_cache) after the call, all fp64; caches [blocks][G][bs][hd]."""
    T = len(pos)
    x = np.asarray(qkv, dtype=np.float64).reshape(T, H + 2 * G, -1)
    q = norm_rotate(x[:, :H], gamma_q, pos, theta, eps)
    k = norm_rotate(x[:, H:H + G], gamma_k, pos, theta, eps)
    kc, vc = np.array(k_cache, dtype=np.float64), np.array(v_cache, dtype=np.float64)
    nb, _, bs, _ = kc.shape
    for t in range(T):
        if 0 <= slot[t] < nb * bs:
            kc[slot[t] // bs, :, slot[t] % bs] = k[t]
            vc[slot[t] // bs, :, slot[t] % bs] = x[t, H + G:]
    return q, kc, vc


def chunk_attention(qsl, seq_len, q, k_cache, v_cache, table, sink=None):
    """(out, spread): out [T][H][hd] fp64, and sum_t p_t |v_t| of each output, which
    bounds what a relative error of the weights does to it.  Rows of no request
    stay NaN.  A key in an invalid block does not exist; a row that sees no key
    gives zeros."""
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
        blk = table[r][t // bs]
        for h in range(H):
            g = h // (H // G)
            K, V = k_cache[blk, g, t % bs], v_cache[blk, g, t % bs]
            s = q[lo:hi, h] @ K.T / np.sqrt(hd)
            s[t[None, :] > L - n + np.arange(n)[:, None]] = -np.inf
            if len(t) == 0:
                continue
            top = s.max(-1)
            if sink is not None:
                top = np.maximum(top, float(sink[h]))
            live = np.isfinite(s).any(-1)
            top = np.where(live, top, 0.0)
            w = np.exp(s - top[:, None])
            den = w.sum(-1) + (np.exp(float(sink[h]) - top) if sink is not None else 0.0)
            w /= np.where(live, den, 1.0)[:, None]
            # a key that no row sees may hold anything: its weight is 0, it does not enter
            see = w > 0
            Vf = np.where(see.any(0)[:, None], V, 0.0)
            out[lo:hi, h] = w @ Vf
            spread[lo:hi, h] = w @ np.abs(Vf)
    return out, spread


def verify_sampled(qsl, tok, logits, temperature, u, gumbel):
    """(accepted, bonus, p, margin) of each request; p [T] is the target's
    probability of each draft (1 for row 0 of a request), margin[r] how far the
    request is from another answer: the least |u - p| over the drafts it looks at
    and the lead of the winning score."""
    B = len(qsl) - 1
    logits = np.asarray(logits, dtype=np.float64)
    V = logits.shape[1]
    acc, bonus = np.zeros(B, np.int64), np.full(B, -1, np.int64)
    p, margin = np.full(len(tok), np.nan), np.full(B, np.inf)
    for r in range(B):
        lo, hi = int(qsl[r]), int(qsl[r + 1])
        n, temp = hi - lo, float(temperature[r])
        temp = min(max(temp, 1e-30), 1e30) if temp > 0 else temp
        if n == 0:
            continue
        p[lo] = 1.0
        rows = []
        for j in range(n):
            x = logits[lo + j]
            top = x.max()
            if temp == 0:
                d = np.zeros(V)
                d[int(np.argmax(x))] = 1.0
            elif np.isfinite(top):
                d = np.exp((x - top) / temp)
                d /= d.sum()
            else:
                d = None
            rows.append(d)
        for j in range(1, n):
            v = int(tok[lo + j])
            p[lo + j] = 0.0 if rows[j - 1] is None or not 0 <= v < V else rows[j - 1][v]
        a = 0
        while a < n - 1:
            m = p[lo + a + 1]
            if temp > 0:
                margin[r] = min(margin[r], abs(float(u[lo + a + 1]) - m))
            if not (m == 1.0 if temp == 0 else float(u[lo + a + 1]) < m):
                break
            a += 1
        acc[r] = a
        if temp == 0:
            bonus[r] = int(np.argmax(logits[lo + a]))
        elif rows[a] is not None:
            with np.errstate(invalid="ignore"):
                s = logits[lo + a] / temp + np.asarray(gumbel[r], dtype=np.float64)
            s[np.isneginf(logits[lo + a])] = -np.inf
            if a < n - 1 and 0 <= tok[lo + a + 1] < V:
                s[int(tok[lo + a + 1])] = -np.inf
            if np.isneginf(s).all():
                continue
            bonus[r] = int(np.argmax(s))
            rest = np.delete(s, bonus[r])
            if len(rest):
                margin[r] = min(margin[r], s[bonus[r]] - rest.max())
    return acc, bonus, p, margin
