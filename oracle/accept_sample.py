"""Sampled acceptance of speculative draft trees, in 64 bits -- TEST
INFRASTRUCTURE (the oracle of the library's sampled accept step and of the
compaction after it; only tests/ may use it; it shares no code with the CUDA
path).

Each request's nodes carry the target model's logits; p_v = softmax(logits[v]
/ T).  From the root, node v's children are tried in index order: child c,
token x, drawn from q = draft_probs[v], is accepted iff u[c] q(x) < r(x); a
rejection replaces r by max(r - q, 0), normalised (speculative sampling,
Leviathan et al. 2023, with one residual per rejected sibling as in SpecInfer,
Miao et al. 2024).  Without draft_probs q is 1 at the token.  When no child is
accepted the bonus token is argmax_x r(x) / noise(x) (r without mass: p).
T = 0: one-hot at the first argmax.

The residuals are iterated as the definition has them, and `margin` says how
far every decision was from its border, relative to the size of what was
compared: a rounding below it cannot change the answer.
"""
from __future__ import annotations

import numpy as np


def softmax64(row, t):
    row = np.asarray(row, dtype=np.float64)
    if t == 0:
        p = np.zeros_like(row)
        p[int(np.argmax(row))] = 1.0
        return p
    m = row.max()
    if m == -np.inf:
        return np.zeros_like(row)
    e = np.exp((row - m) / t)
    return e / e.sum()


def accept_sampled(logits, qo_indptr, tokens, parents, u, noise, temperature=None, draft_probs=None):
    """Returns (accept_len [B], paths: list of int arrays, bonus [B], logprobs
    [total], margin)."""
    logits = np.asarray(logits)
    V = logits.shape[1]
    B = len(qo_indptr) - 1
    total = logits.shape[0]
    acc, bonus, paths = np.zeros(B, np.int64), np.full(B, -1, np.int64), []
    logp, margin = np.zeros(total), np.inf
    for b in range(B):
        o, n = int(qo_indptr[b]), int(qo_indptr[b + 1] - qo_indptr[b])
        if n == 0:
            paths.append(np.zeros(0, np.int64))
            continue
        t = 1.0 if temperature is None else float(temperature[b])
        v, path = 0, []
        while True:
            path.append(v)
            p = softmax64(logits[o + v], t)
            dead = not p.any()
            r, nxt = p.copy(), -1
            A, Bn = 0.0, 1.0            # r = max(p - A q, 0) / Bn, kept for the margin alone
            q = None if draft_probs is None else np.asarray(draft_probs[o + v], np.float64)
            for c in range(v + 1, n):
                if int(parents[o + c]) != v or dead:
                    continue
                x = int(tokens[o + c])
                if not 0 <= x < V:
                    rx, qx = 0.0, 1.0 if q is None else 0.0
                else:
                    rx, qx = r[x], 1.0 if q is None else q[x]
                if t == 0:
                    ok = rx > 0 if q is None else p[x] > 0 if 0 <= x < V else False
                else:
                    ok = float(u[o + c]) * qx < rx
                    size = (p[x] if 0 <= x < V else 0.0) + (1.0 + A) * qx
                    if size > 0:
                        margin = min(margin, abs(float(u[o + c]) * qx - rx) * Bn / size)
                if ok:
                    nxt = c
                    break
                if t == 0:
                    continue
                if q is None:
                    left = r.copy()
                    if 0 <= x < V:
                        left[x] = 0.0
                else:
                    left = np.maximum(r - q, 0.0)
                mass = left.sum()
                A += Bn
                Bn *= mass
                r = left / mass if mass > 0 else left
            if nxt >= 0:
                logp[o + len(path) - 1] = 0.0 if t == 0 else np.log(p[int(tokens[o + nxt])])
                v = nxt
                continue
            if not dead:
                w = r if r.any() else p
                key = np.where(w > 0, w / np.maximum(np.asarray(noise[b], np.float64), 1e-300), -1.0)
                bonus[b] = int(np.argmax(key))
                logp[o + len(path) - 1] = 0.0 if t == 0 else np.log(p[bonus[b]])
                if t != 0 and V > 1:
                    # the two best candidates against what each was computed from
                    two = np.argsort(-key, kind="stable")[:2]
                    size = sum((p[i] + (0.0 if q is None else A * q[i])) / max(float(noise[b][i]), 1e-300) for i in two)
                    gap = (key[two[0]] - max(key[two[1]], 0.0)) * (Bn if w is r and q is not None else 1.0)
                    if key[two[0]] != key[two[1]]:   # equal candidates: the lower index, no rounding involved
                        margin = min(margin, gap / size if size > 0 else np.inf)
            break
        acc[b] = len(path)
        paths.append(np.array(path, np.int64))
    return acc, paths, bonus, logp, margin


def compact_rows(qo_indptr, kv_indptr, last_page_len, page_size, kv_indices, accept_len, path):
    """[(source (page, slot), destination (page, slot))] in order, and the new
    kv length of each request: node path[k]'s row moves to position prefix + k."""
    moves, new_len = [], []
    for b in range(len(accept_len)):
        o, n = int(qo_indptr[b]), int(qo_indptr[b + 1] - qo_indptr[b])
        k0, npg = int(kv_indptr[b]), int(kv_indptr[b + 1] - kv_indptr[b])
        kv_len = (npg - 1) * page_size + int(last_page_len[b]) if npg else 0
        pre = kv_len - n
        for k in range(int(accept_len[b])):
            s, d = pre + int(path[o + k]), pre + k
            if s != d:
                moves.append(((int(kv_indices[k0 + s // page_size]), s % page_size),
                              (int(kv_indices[k0 + d // page_size]), d % page_size)))
        new_len.append(pre + int(accept_len[b]))
    return moves, np.array(new_len, np.int64)
