"""fp64 definitions of the decode-loop operators: tokens written into a paged
cache at positions of several axes, one new token attending a paged sequence
with its attention weights added up, and eviction by those weights.  Test
infrastructure, like the rest of this package; arrays are numpy, caches
[blocks][block_size][heads][dim], weights [blocks][weight_heads][block_size].
"""

from __future__ import annotations

import numpy as np

from .pic_oracle import attention_decode, rotate, rotate_rows


def rotate_axes(rows, pos, freq_axis, theta, pairing, rope_offset, rope_dim):
    """Rows [heads][dim] with frequency f turned by pos[freq_axis[f]] * theta[f]."""
    theta = np.asarray(theta, dtype=np.float64)
    # the angle of frequency f is 1 * (pos theta)_f: one rotation by delta 1 of scaled frequencies
    scaled = np.array([float(pos[a]) for a in freq_axis]) * theta
    out = np.asarray(rows, dtype=np.float64).copy()
    sl = slice(rope_offset, rope_offset + rope_dim)
    out[..., sl] = rotate(out[..., sl], 1, scaled, pairing)
    return out


def slot_row(table, slot, block_size):
    return int(table[slot // block_size]), slot % block_size


def write_tokens(q, k, v, positions, freq_axis, theta, pairing, rope_offset, rope_dim, req, slot, tables, block_size,
                 k_cache, v_cache, weights=None):
    """Returns (q_out, k_cache, v_cache, weights) as new arrays; positions [axes][tokens]."""
    q_out = None if q is None else np.stack(
        [rotate_axes(q[i], positions[:, i], freq_axis, theta, pairing, rope_offset, rope_dim) for i in range(len(q))])
    k_cache = k_cache.copy()
    v_cache = None if v_cache is None else v_cache.copy()
    weights = None if weights is None else weights.copy()
    for i in range(len(slot)):
        if slot[i] < 0:
            continue
        b, row = slot_row(tables[req[i]], int(slot[i]), block_size)
        k_cache[b, row] = rotate_axes(k[i], positions[:, i], freq_axis, theta, pairing, rope_offset, rope_dim)
        if v is not None:
            v_cache[b, row] = v[i]
        if weights is not None:
            weights[b, :, row] = 0.0
    return q_out, k_cache, v_cache, weights


def attend_paged(q, k_cache, v_cache, tables, lens, block_size, scale, weights=None):
    """q [n_req][Hq][D].  Returns (out, lse, weights); an empty sequence gives
    out 0, lse -inf.  MLA: v_cache is the latent slice of k_cache."""
    n_req, hq, _ = q.shape
    out = np.zeros((n_req, hq, v_cache.shape[-1]))
    lse = np.full((n_req, hq), -np.inf)
    weights = None if weights is None else weights.astype(np.float64).copy()
    for r in range(n_req):
        if lens[r] == 0:
            continue
        at = [slot_row(tables[r], s, block_size) for s in range(lens[r])]
        keys = np.stack([k_cache[b, i] for b, i in at])
        vals = np.stack([v_cache[b, i] for b, i in at])
        out[r], lse[r] = attention_decode(q[r], keys, vals, scale)
        if weights is not None:
            group = hq // keys.shape[1]
            share = hq // weights.shape[1]   # query heads of a weight head
            for g in range(hq):
                p = np.exp(scale * (keys[:, g // group] @ q[r, g]) - lse[r, g])
                for t, (b, i) in enumerate(at):
                    weights[b, g // share, i] += p[t]
    return out, lse, weights


def kept_slots(w, length, budget, n_first, n_recent):
    """Slots that stay, ascending: the first n_first, the last n_recent, and of
    the others the heaviest (equal weights: the lower slot; NaN lowest)."""
    if length <= budget:
        return list(range(length))
    middle = list(range(n_first, length - n_recent))
    order = sorted(middle, key=lambda s: (-np.inf if np.isnan(w[s]) else float(w[s])), reverse=True)
    # sorted() with reverse keeps equal keys in their order; NaN must come after -inf too
    order = [s for s in order if not np.isnan(w[s])] + [s for s in middle if np.isnan(w[s])]
    take = order[:budget - n_first - n_recent]
    return sorted(list(range(n_first)) + list(range(length - n_recent, length)) + take)


def evict_tokens(k_cache, v_cache, weights, tables, lens, block_size, budget, n_first, n_recent, renumber, theta, pairing,
                 rope_offset, rope_dim):
    """One layer.  Returns (k_cache, v_cache, weights, kept [n_req][weight_heads][budget], lens)."""
    k_new, v_new, w_new = k_cache.copy(), None if v_cache is None else v_cache.copy(), weights.copy()
    heads, wh = k_cache.shape[2], weights.shape[1]
    kept = np.full((len(lens), wh, budget), -1, dtype=np.int32)
    for r, n in enumerate(lens):
        at = [slot_row(tables[r], s, block_size) for s in range(n)]
        for h in range(wh):
            stay = kept_slots([weights[b, h, i] for b, i in at], n, budget, n_first, n_recent)
            kept[r, h, :len(stay)] = stay
            kv = range(heads) if wh == 1 else [h]
            for j, s in enumerate(stay):
                (b, i), (sb, si) = at[j], at[s]
                w_new[b, h, i] = weights[sb, h, si]
                for x in kv:
                    row = k_cache[sb, si, x]
                    if renumber and j != s:
                        row = rotate_rows(row, j - s, theta, pairing, rope_offset, rope_dim)
                    k_new[b, i, x] = row
                    if v_cache is not None:
                        v_new[b, i, x] = v_cache[sb, si, x]
    return k_new, v_new, w_new, kept, np.minimum(lens, budget)
