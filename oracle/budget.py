"""A budgeted cache in double precision: norm and rotation of new heads, the
attention weight that each cached key receives, and the eviction by it, written
from their definitions (include/verify_attn.h) in numpy."""
import numpy as np


def prepare_heads(x, weight, offset, eps, positions, freq, rot, interleaved):
    """x [total, heads, d] float64: each head divided by its root mean square and
    weighted (weight None: as it is), then its first `rot` elements rotated at
    positions * freq (positions None: not).  Returns the result and, element by
    element, the sum of the magnitudes that were added to make it."""
    y = x.astype(np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * (weight.astype(np.float64) + offset)
    size = np.abs(y)
    if positions is None or rot == 0:
        return y, size
    angle = positions.astype(np.float64)[:, None] * freq[None]
    cos, sin = np.cos(angle)[:, None], np.sin(angle)[:, None]
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    out = y.copy()
    out[..., a] = y[..., a] * cos - y[..., b] * sin
    out[..., b] = y[..., a] * sin + y[..., b] * cos
    both = np.abs(y[..., a]) + np.abs(y[..., b])
    size[..., a], size[..., b] = both, both
    return out, size


def slots_of(kv_indptr, kv_indices, last, page_size, b):
    """(pages, slots) of request b's keys in position order."""
    pages = kv_indices[kv_indptr[b]:kv_indptr[b + 1]]
    n = (len(pages) - 1) * page_size + int(last[b]) if len(pages) else 0
    j = np.arange(n)
    return pages[j // page_size], j % page_size


def visible(n, kv_len, mask=None, offset=0, full=False):
    """[n, kv_len]: which keys the n query tokens see."""
    v = np.ones((n, kv_len), bool)
    if mask is None:
        v[:, kv_len - n:] = np.tril(np.ones((n, n), bool))
        return v
    width = kv_len if full else n
    e = offset + np.arange(n * width)
    bits = ((mask[e // 8] >> (e % 8)) & 1).astype(bool).reshape(n, width)
    v[:, kv_len - width:] = bits
    return v


def key_weights(q, k, lse, seen, scale, path=None):
    """One request: q [n, h_q, d], k [m, h_kv, d] (scaled), lse [n, h_q], seen [n,
    m].  Weights received [m', h_kv] -- m' = m, or the prefix and the path --
    and a bound of what fp32 may lose of each."""
    n, hq, d = q.shape
    m, h = k.shape[:2]
    G = hq // h
    q4 = q.astype(np.float64).reshape(n, h, G, d)
    k = k.astype(np.float64)
    s = np.einsum("nhgd,mhd->nhgm", q4, k) * scale
    sizes = np.einsum("nhgd,mhd->nhgm", np.abs(q4), np.abs(k)) * scale
    l = lse.astype(np.float64).reshape(n, h, G, 1)
    on = seen[:, None, None, :] & (l != -np.inf)
    if path is not None:
        keep = np.zeros(n, bool)
        keep[path] = True
        on = on & keep[:, None, None, None]
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.where(on, np.exp(s - np.where(l == -np.inf, 0, l)), 0.0)
        # a product of two bf16 numbers is exact in fp32; d of them added up, in
        # any order and with truncation, lose d steps of 2^-23 of the sum of their
        # magnitudes; log2(e) times logit and lse round once each, their difference
        # and the product's constant once more; 2^x is good to 2 steps
        rel = d * 2.0 ** -23 * sizes + 4 * 2.0 ** -24 * (np.abs(np.where(on, s, 0)) + np.abs(np.where(on, l, 0))) + 2.0 ** -22
        loss = np.where(on, e * rel, 0.0)
    w, loss = e.sum((0, 2)).T, loss.sum((0, 2)).T
    loss = loss + (n * G + 4) * 2.0 ** -24 * w
    if path is not None:
        rows = np.concatenate([np.arange(m - n), m - n + np.asarray(path, int)])
        w, loss = w[rows], loss[rows]
    return w, loss


def survivors(w, keep, sinks, recent):
    """Positions that stay of one request, layer and KV head, ascending."""
    n = len(w)
    keep = min(keep, n)
    first = min(sinks, keep)
    tail = min(recent, keep - first)
    mid = sorted(range(first, n - tail), key=lambda j: (-np.inf if np.isnan(w[j]) else 0, -float(w[j]) if w[j] == w[j] else 0, j))
    return sorted(list(range(first)) + mid[:keep - first - tail] + list(range(n - tail, n)))
