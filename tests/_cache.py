"""The cache ops' definitions in numpy, 64 bits, one sample and head at a time (see include/fr.h)."""
from __future__ import annotations

import numpy as np


def sees(words, N):
    """[N][N] truth values from one sample's mask words (None: a sequence)."""
    if words is None:
        return np.tril(np.ones((N, N), bool))
    return np.array([[bool((int(words[i][j // 32]) >> (j % 32)) & 1) for j in range(N)] for i in range(N)])


def words_of(seen):
    """Mask words [N][ceil(N/32)] (uint32) of [N][N] truth values."""
    N = len(seen)
    out = np.zeros((N, -(-N // 32)), np.uint32)
    for i in range(N):
        for j in np.flatnonzero(seen[i]):
            out[i, j // 32] |= np.uint32(1 << (int(j) % 32))
    return out


def attend(q, k, v, lens, words):
    """q [B][Hq][N][dh], k, v [B][Hkv][S][dh]: o, its tolerance's sums, lse and score sizes; padded samples stay 0."""
    B, Hq, N, dh = q.shape
    g = Hq // k.shape[1]
    o, pv = np.zeros((B, N, Hq, dh)), np.zeros((B, N, Hq, dh))
    lse, size = np.zeros((B, Hq, N)), np.zeros((B, Hq, N))
    for b, n0 in enumerate(lens):
        if n0 < 0:
            continue
        seen = sees(None if words is None else words[b], N)
        for h in range(Hq):
            kk, vv = k[b, h // g, :n0 + N], v[b, h // g, :n0 + N]
            vis = np.concatenate([np.ones((N, n0), bool), seen], axis=1)
            s = np.where(vis, q[b, h] @ kk.T / np.sqrt(dh), -np.inf)
            m = s.max(axis=1)
            some = m > -np.inf
            e = np.exp(s - np.where(some, m, 0.0)[:, None])
            l = e.sum(axis=1)
            p = e / np.where(some, l, 1.0)[:, None]
            o[b, :, h], pv[b, :, h] = p @ vv, p @ np.abs(vv)
            with np.errstate(divide="ignore"):
                lse[b, h] = np.where(some, m + np.log(l), -np.inf)
            size[b, h] = np.where(vis, np.abs(q[b, h]) @ np.abs(kk).T, 0.0).max(axis=1) / np.sqrt(dh)
    return o, pv, lse, size


def weigh(q, k, lse, lens, words, use, acc):
    """acc after the call, and the weights added."""
    B, Hq, N, dh = q.shape
    Hkv = k.shape[1]
    g = Hq // Hkv
    acc, w = acc.astype(np.float64).copy(), np.zeros(acc.shape)
    for b, n0 in enumerate(lens):
        if n0 < 0:
            continue
        seen = sees(None if words is None else words[b], N)
        counts = np.array([use is None or bool((int(use[b][i // 32]) >> (i % 32)) & 1) for i in range(N)])
        for h in range(Hq):
            vis = np.concatenate([np.ones((N, n0), bool), seen], axis=1) & (counts & (lse[b, h] > -np.inf))[:, None]
            x = q[b, h] @ k[b, h // g, :n0 + N].T / np.sqrt(dh) - np.where(lse[b, h] > -np.inf, lse[b, h], 0.0)[:, None]
            w[b, h // g, :n0 + N] += np.exp(np.where(vis, x, -np.inf)).sum(axis=0)
        acc[b, :, :n0] += w[b, :, :n0]
        acc[b, :, n0:n0 + N] = w[b, :, n0:n0 + N]
    return acc, w


def evict_one(acc, pos, keep, recent):
    """Old slot of each kept slot of one (sample, head): [min(len, keep)]."""
    n = len(acc)
    if n <= keep:
        return np.arange(n)
    protected = pos.astype(np.int64) > int(pos.max()) - recent
    rank = [(0 if protected[s] else 1, 0.0 if protected[s] else (np.inf if np.isnan(acc[s]) else -float(acc[s])),
             1 if np.isnan(acc[s]) and not protected[s] else 0, s) for s in range(n)]
    best = sorted(r[3] for r in sorted(rank)[:keep])
    src = np.arange(keep)
    src[sorted(set(range(keep)) - set(best))] = [s for s in best if s >= keep]
    return src
