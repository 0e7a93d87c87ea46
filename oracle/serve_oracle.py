"""fp64 definitions of a serving step's operators: blocks and slots from request
lengths, head norms before the rotation, attention of any number of new tokens
per request (with a window and first tokens that stay visible), and of requests
that share a prefix.  Test infrastructure, like the rest of this package.
"""

from __future__ import annotations

import numpy as np

from .decode_oracle import rotate_axes, slot_row

BAD_BLOCK, CAPACITY, BAD_LENGTH = 0x1, 0x10, 0x40


def map_tokens(lens, grow, tables, free, n_free, block_size, n_tokens, shift=None):
    """One serving step, request by request.  Returns (new_lens, tables, free,
    new_n_free, indptr, req, slot, pos, status) of plain lists and arrays."""
    tables, free = np.array(tables), list(free)
    blocks, limit, status = len(free), tables.shape[1] * block_size, 0
    up = lambda n: -(-n // block_size)  # noqa: E731
    if not 0 <= n_free <= blocks:
        n_free, status = 0, status | BAD_LENGTH
    legal = [0 <= n <= limit and 0 <= n + g <= limit for n, g in zip(lens, grow)]
    refused = [not x for x in legal]
    if not all(legal):
        status |= BAD_LENGTH
    pile, back = n_free, 0
    for r, (n, g) in enumerate(zip(lens, grow)):
        if legal[r] and g < 0 and up(n) > up(n + g):
            back += up(n) - up(n + g)
            if n_free + back > blocks:
                refused[r], status = True, status | CAPACITY
                continue
            for b in range(up(n + g), up(n)):
                block = int(tables[r][b])
                if not 0 <= block < blocks:
                    status |= BAD_BLOCK
                free[pile] = block
                pile += 1
    top, asked, ends, req, slot = pile, 0, [0], [], []
    for r, (n, g) in enumerate(zip(lens, grow)):
        ends.append(ends[-1] + max(0, g))
        need = up(n + g) - up(n) if legal[r] and g > 0 else 0
        asked += need
        if g > 0 and ends[-1] > n_tokens or need > 0 and asked > pile:
            status |= CAPACITY
            refused[r] = True
        if not refused[r]:
            for b in range(up(n), up(n) + need):
                top -= 1
                if not 0 <= free[top] < blocks:
                    status |= BAD_BLOCK
                tables[r][b] = free[top]
            if need:
                # what refused requests asked for stays on the pile, and none behind them gets any
                assert top == pile - asked
        for j in range(max(0, min(g, n_tokens - len(req)))):
            req.append(r)
            slot.append(-1 if refused[r] else n + j)
    new_lens = [n if refused[r] else n + g for r, (n, g) in enumerate(zip(lens, grow))]
    pad = n_tokens - len(req)
    req, slot = req + [0] * pad, slot + [-1] * pad
    pos = [0 if s < 0 else s + (0 if shift is None else shift[r]) for r, s in zip(req, slot)]
    return new_lens, tables, free, top, [min(e, n_tokens) for e in ends], req, slot, pos, status


def head_norm(x, weight, eps, offset=0.0):
    """x [..., dims] / sqrt(mean(x^2) + eps) * (offset + weight)"""
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (offset + np.asarray(weight, dtype=np.float64))


def sees(slot, t, window, n_first):
    """Whether a token at `slot` sees slots t."""
    t = np.asarray(t)
    if slot < 0:
        return np.zeros(t.shape, bool)
    near = t > slot - window if window else np.ones(t.shape, bool)
    return (t <= slot) & (near | (t < n_first))


def attend_rows(q, k, v, seen, scale):
    """q [Hq][D]; k [Hk][T][D], v [Hk][T][Dv]; seen [T].  Returns (out, lse)."""
    hq, group = len(q), len(q) // len(k)
    out, lse = np.zeros((hq, v.shape[-1])), np.full(hq, -np.inf)
    if not seen.any():
        return out, lse
    for h in range(hq):
        x = scale * (k[h // group][seen] @ q[h])
        top = x.max()
        e = np.exp(x - top)
        out[h], lse[h] = e @ v[h // group][seen] / e.sum(), top + np.log(e.sum())
    return out, lse


def gather(cache, table, slots, block_size):
    """Rows [heads][T][dim] of slots of one request."""
    at = [slot_row(table, int(s), block_size) for s in slots]
    rows = cache[[a for a, _ in at], [b for _, b in at]]
    return rows.transpose(1, 0, 2)


def attend_tokens(q, k_cache, v_cache, tables, indptr, slot, block_size, scale, window=0, n_first=0):
    """Returns (out, lse) of the rows of all requests; NaN where a row is of none."""
    out, lse = np.full(q.shape, np.nan), np.full(q.shape[:2], np.nan)
    for r in range(len(indptr) - 1):
        for i in range(indptr[r], indptr[r + 1]):
            t = np.arange(slot[i] + 1)
            t = t[sees(slot[i], t, window, n_first)]
            k, v = gather(k_cache, tables[r], t, block_size), gather(v_cache, tables[r], t, block_size)
            out[i], lse[i] = attend_rows(q[i], k, v, np.ones(len(t), bool), scale)
    return out, lse


def attend_shared(q, k_cache, v_cache, prefix_table, prefix_len, tables, lens, block_size, scale):
    out, lse = np.zeros(q.shape), np.zeros(q.shape[:2])
    for r in range(len(q)):
        head, tail = np.arange(min(prefix_len, lens[r])), np.arange(prefix_len, max(prefix_len, lens[r]))
        k, v = (np.concatenate([gather(c, prefix_table, head, block_size), gather(c, tables[r], tail, block_size)], 1)
                for c in (k_cache, v_cache))
        out[r], lse[r] = attend_rows(q[r], k, v, np.ones(k.shape[1], bool), scale)
    return out, lse


def write_normed(q, k, q_norm, k_norm, eps, offset, positions, freq_axis, theta, pairing, rope_offset, rope_dim):
    """Turned rows of q and k, normalised first (k's latent for rope_offset > 0)."""
    def norm(x, w):
        x = np.asarray(x, dtype=np.float64).copy()
        if w is not None:
            part = x[..., :rope_offset] if rope_offset else x
            part[...] = head_norm(part, w, eps, offset)
        return x
    turn = lambda x: np.stack([rotate_axes(x[i], positions[:, i], freq_axis, theta, pairing, rope_offset, rope_dim)  # noqa: E731
                               for i in range(len(x))])
    return turn(norm(q, q_norm)), turn(norm(k, k_norm))
