"""Oracle: the step over a paged KV cache (test infrastructure).

A paged cache holds slot s of request b in row ``s % page`` of page
``table[b, s // page]``. The steps over it are those of the contiguous cache
(`attention.py`, `commit.py`) on the gathered slots; added are the norms and
rotation that produce the new tokens' queries and keys, and the book-keeping
of the pages. Everything in fp64 or integers, one request after another.
"""
from __future__ import annotations

import numpy as np

from .attention import tree_attention
from .heads import bf16_to_f64


def gather(pool, row, n):
    """[Hkv, n, dh]: the first n slots of one request, whose table row is `row`."""
    _, hkv, page, dh = pool.shape
    out = np.zeros((hkv, n, dh), dtype=pool.dtype)
    for s in range(n):
        out[:, s] = pool[row[s // page], :, s % page]
    return out


def tree_attention_paged(q, k_pages, v_pages, table, prefix_len, parent, scale=None):
    """out[b, t, h, :] fp64; requests with prefix_len -1 are idle: zeros."""
    B, T, Hq, dh = q.shape
    out = np.zeros((B, T, Hq, dh))
    for b in range(B):
        P = int(prefix_len[b])
        if P < 0:
            continue
        k = gather(k_pages, table[b], P + T)[None]
        v = gather(v_pages, table[b], P + T)[None]
        out[b] = tree_attention(q[b:b + 1], k, v, [P], parent, scale)[0]
    return out


def norm_rotate(x, w, pos, inv_freq, eps, interleaved):
    """x [..., dh] fp64 (one position): RMS norm with weight w (None: none), then
    each pair turned by pos * inv_freq."""
    y = np.array(x, dtype=np.float64)
    if w is not None:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps) * w
    out = y.copy()
    half = len(inv_freq)
    for f in range(half):
        i, j = (2 * f, 2 * f + 1) if interleaved else (f, f + half)
        a = float(pos) * float(inv_freq[f])
        out[..., i] = y[..., i] * np.cos(a) - y[..., j] * np.sin(a)
        out[..., j] = y[..., j] * np.cos(a) + y[..., i] * np.sin(a)
    return out


def qk_rope_append(q, k, v, pos, inv_freq, table, prefix_len, pool_shape, q_norm=None, k_norm=None, eps=1e-6,
                   interleaved=False, n_new=None):
    """q_out [B, T, Hq, dh] fp64 (NaN where the call writes nothing) and the
    written pool rows: {(page, row): (k [Hkv, dh] fp64, v bits [Hkv, dh])}."""
    B, T, Hq, dh = q.shape
    pages, _, page, _ = pool_shape
    out = np.full((B, T, Hq, dh), np.nan)
    written = {}
    qw = None if q_norm is None else bf16_to_f64(q_norm)
    kw = None if k_norm is None else bf16_to_f64(k_norm)
    for b in range(B):
        P = int(prefix_len[b])
        if P == -1:
            continue
        for t in range(T if n_new is None else min(T, int(n_new[b]))):
            out[b, t] = norm_rotate(bf16_to_f64(q[b, t]), qw, pos[b, t], inv_freq, eps, interleaved)
            s = P + t
            if P < 0 or s >= table.shape[1] * page:
                continue
            pg = int(table[b, s // page])
            if 0 <= pg < pages:
                written[(pg, s % page)] = (norm_rotate(bf16_to_f64(k[b, t]), kw, pos[b, t], inv_freq, eps, interleaved),
                                           v[b, t])
    return out, written


def tree_commit_paged(k_pages, v_pages, table, prefix_len, accept_len, path, bonus, T):
    """Pools [layers, pages, Hkv, page, dh]; returns copies and the next step's inputs. A request
    with an accepted node in no page of the pool stays as it is."""
    k, v = k_pages.copy(), v_pages.copy()
    page = k.shape[3]
    newp, root, row = [], [], []
    for b in range(len(prefix_len)):
        P, L = int(prefix_len[b]), int(accept_len[b])
        if P == -1:
            newp.append(-1), root.append(-1), row.append(-1)
            continue
        slots = [P + int(path[b, i]) for i in range(L + 1)] + list(range(P, P + L + 1))
        if not all(0 <= table[b, s // page] < k.shape[1] for s in slots):
            newp.append(P), root.append(int(bonus[b])), row.append(-1)
            continue
        for i in range(L + 1):
            s, d = P + int(path[b, i]), P + i
            sp, dp = table[b, s // page], table[b, d // page]
            k[:, dp, :, d % page] = k_pages[:, sp, :, s % page]
            v[:, dp, :, d % page] = v_pages[:, sp, :, s % page]
        newp.append(P + L + 1), root.append(int(bonus[b])), row.append(b * T + int(path[b, L]))
    return k, v, np.array(newp), np.array(root), np.array(row)


def pages_resize(table, n_pages, refcount, length, page, extra=0):
    """Copies of the three arrays after the call, and whether the pool ran short."""
    table, n_pages, ref = table.copy(), n_pages.copy(), refcount.copy()
    B, width = table.shape
    want = [0 if length[b] < 0 else -(-(int(length[b]) + extra) // page) for b in range(B)]
    ok = [want[b] <= width and 0 <= n_pages[b] <= width for b in range(B)]
    for b in range(B):
        if ok[b]:
            while n_pages[b] > want[b]:
                n_pages[b] -= 1
                ref[table[b, n_pages[b]]] -= 1
                table[b, n_pages[b]] = -1
    free = [p for p in range(len(ref)) if ref[p] == 0]
    left, short = len(free), False
    for b in range(B):
        need = max(0, want[b] - int(n_pages[b])) if ok[b] else 0
        left -= need
        if need and left < 0:
            short = True
        elif need:
            for _ in range(need):
                pg = free.pop(0)
                table[b, n_pages[b]] = pg
                ref[pg] = 1
                n_pages[b] += 1
    return table, n_pages, ref, short


def pages_fork(k_pages, v_pages, table, n_pages, refcount, src, dst, length):
    """Copies of the pools (bit patterns), table, counts and lengths after the call."""
    k, v = k_pages.copy(), v_pages.copy()
    table, n_pages, ref, length = table.copy(), n_pages.copy(), refcount.copy(), length.copy()
    page = k.shape[3]
    jobs = []
    for i in range(len(src)):
        n = int(length[src[i]]) if src[i] != -1 else -1
        if n > 0 and n % page and not 0 <= table[src[i], n // page] < len(ref):
            continue                                    # no page to copy from
        if src[i] != -1 and dst[i] not in [s for s in src if s != -1] and dst[i] not in [d for _, d in jobs]:
            jobs.append((int(src[i]), int(dst[i])))
    for _, d in jobs:
        for p in range(n_pages[d]):
            ref[table[d, p]] -= 1
        table[d, :] = -1
        n_pages[d] = 0
    for s, d in jobs:
        n = int(length[s])
        full, rows = (n // page, n % page) if n > 0 else (0, 0)
        length[d] = n if n >= 0 else -1
        fresh = -1
        if rows:
            free = [p for p in range(len(ref)) if ref[p] == 0]
            if not free:
                length[d] = -1
                continue
            fresh = free[0]
            ref[fresh] = 1
            for pool, old in ((k, k_pages), (v, v_pages)):
                pool[:, fresh, :, :rows] = old[:, table[s, full], :, :rows]
        for p in range(full):
            table[d, p] = table[s, p]
            ref[table[s, p]] += 1
        if rows:
            table[d, full] = fresh
        n_pages[d] = full + (1 if rows else 0)
    return k, v, table, n_pages, ref, length
