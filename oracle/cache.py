"""Plain numpy reference of the 8-bit key/value cache (float64, one token at a time
where order matters).  A pool is a dict of arrays with the layouts of include/hstu.h:
k_codes [N, H, 64, d], v_codes [N, H, d, 64], k_scale, v_scale [N, H], timestamps,
positions, weights [N, 64]."""

from __future__ import annotations

import math

import numpy as np

from . import fp8

PAGE = 64


VALUES = fp8.e4m3_decode(np.arange(256, dtype=np.uint8)).astype(np.float64)


def encode(x):
    """Codes of finite x (exact in float32), saturated at 448."""
    return fp8.e4m3_encode(np.asarray(x, np.float32)).astype(np.uint8)


def scale_of(amax):
    """The smallest 2^e, e >= -126, with amax <= 448 * 2^e; 0 for 0, NaN if not finite."""
    amax = float(amax)
    if not math.isfinite(amax):
        return math.nan
    if amax == 0.0:
        return 0.0
    e = -126
    m, x = math.frexp(amax)
    e = max(e, x - 10)
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def new_pool(pages, heads, d):
    return dict(k_codes=np.zeros((pages, heads, PAGE, d), np.uint8), v_codes=np.zeros((pages, heads, d, PAGE), np.uint8),
                k_scale=np.zeros((pages, heads), np.float32), v_scale=np.zeros((pages, heads), np.float32),
                timestamps=np.zeros((pages, PAGE), np.int64), positions=np.zeros((pages, PAGE), np.int32),
                weights=np.zeros((pages, PAGE), np.float32))


def _block(pool, name, page, h):
    """Codes of a block as [64, d]."""
    c = pool[name + "_codes"][page, h]
    return c if name == "k" else c.T


def tokens(pool, name, table, length, h):
    """Values [length, d] of a sequence's cached keys or values of head h."""
    d = pool["k_codes"].shape[3]
    out = np.zeros((length, d))
    for j0 in range(0, length, PAGE):
        page = table[j0 // PAGE]
        n = min(PAGE, length - j0)
        out[j0:j0 + n] = VALUES[_block(pool, name, page, h)[:n]] * float(pool[name + "_scale"][page, h])
    return out


def append(pool, k, v, table, lens, seq_pos, offsets, ts, num_targets):
    """Appends in place; returns (new_lens, new_pos)."""
    B, H = len(lens), pool["k_scale"].shape[1]
    pos = lens if seq_pos is None else seq_pos
    new_lens, new_pos = lens.copy(), pos.copy()
    for b in range(B):
        n = int(offsets[b + 1] - offsets[b]) - (0 if num_targets is None else int(num_targets[b]))
        i = 0
        while i < n:
            at = int(lens[b]) + i
            page, slot = table[b, at // PAGE], at % PAGE
            m = min(PAGE - slot, n - i)
            rows = slice(int(offsets[b]) + i, int(offsets[b]) + i + m)
            for name, x in (("k", k), ("v", v)):
                for h in range(H):
                    y = x[rows, h].astype(np.float64)
                    scale = scale_of(np.max(np.abs(y)))
                    codes = _block(pool, name, page, h)
                    old = float(pool[name + "_scale"][page, h]) if slot else 0.0
                    if math.isnan(old) or math.isnan(scale):
                        scale = math.nan
                    else:
                        scale = max(scale, old)
                    r = 1.0 / scale if scale > 0 else 0.0
                    if slot:
                        codes[:slot] = encode(VALUES[codes[:slot]] * (old if old == old else 0.0) * r)
                    codes[slot:slot + m] = encode(np.where(np.isfinite(y), y, 0.0) * r)
                    pool[name + "_scale"][page, h] = scale
            pool["timestamps"][page, slot:slot + m] = ts[rows]
            pool["positions"][page, slot:slot + m] = int(pos[b]) + i + np.arange(m)
            pool["weights"][page, slot:slot + m] = 0.0
            i += m
        new_lens[b] += max(n, 0)
        new_pos[b] += max(n, 0)
    return new_lens, new_pos


def attn(pool, q, table, lens, seq_pos, offsets, ts, num_targets, rab_pos, rab_time, inv_n, pos_lo, pos_hi,
         own=False, addend=None):
    """(out [T, H, d], weights [N, 64], terms): terms has what error bounds are made of,
    per output the roots of the sums over the cached tokens of (P v)^2, (h v)^2, (m v)^2 and
    (x v)^2, where h = |s| / 2, m = sum |q k| + |bias|, x = max |q| sum |k|, all times
    inv_n; per cached token the same without v."""
    T, H, d = q.shape
    pos = lens if seq_pos is None else seq_pos
    rab_pos = np.broadcast_to(rab_pos.astype(np.float64), (H, rab_pos.shape[-1]))
    rab_time = np.broadcast_to(rab_time.astype(np.float64), (H, rab_time.shape[-1]))
    nb = rab_time.shape[1]
    out = np.zeros((T, H, d)) if addend is None else addend.astype(np.float64).copy()
    w = pool["weights"].astype(np.float64).copy()
    t_out = {x: np.zeros((T, H, d)) for x in "Phmx"}
    t_w = {x: np.zeros(w.shape) for x in "Phmx"}
    for b in range(len(lens)):
        s0, n, L = int(offsets[b]), int(offsets[b + 1] - offsets[b]), int(lens[b])
        if n == 0 or L == 0:
            continue
        hist = n - (0 if num_targets is None else int(num_targets[b]))
        i = np.arange(n)
        pi = int(pos[b]) + (i if own else np.minimum(i, hist))
        j = np.arange(L)
        page, slot = np.asarray(table[b])[j // PAGE], j % PAGE
        pj, tj = pool["positions"][page, slot].astype(np.int64), pool["timestamps"][page, slot]
        dp = np.clip(pi[:, None] - pj[None, :], pos_lo, pos_hi) - pos_lo
        dt = np.maximum(ts[s0:s0 + n][:, None] - tj[None, :], 0) + 1
        bucket = np.minimum(np.frompyfunc(lambda x: int(x).bit_length() - 1, 1, 1)(dt).astype(np.int64), nb - 1)
        for h in range(H):
            kk, vv = tokens(pool, "k", table[b], L, h), tokens(pool, "v", table[b], L, h)
            qq = q[s0:s0 + n, h].astype(np.float64)
            bias = rab_pos[h][dp] + rab_time[h][bucket]
            s = qq @ kk.T + bias
            m = np.abs(qq) @ np.abs(kk).T + np.abs(rab_pos[h][dp]) + np.abs(rab_time[h][bucket])
            big = np.abs(qq).max(1)[:, None] * np.abs(kk).sum(1)[None, :]
            P = s / (1.0 + np.exp(-s)) * inv_n
            out[s0:s0 + n, h] += P @ vv
            w[page, slot] += np.abs(P).sum(0)
            for x, a in (("P", P), ("h", 0.5 * np.abs(s) * inv_n), ("m", m * inv_n), ("x", big * inv_n)):
                t_out[x][s0:s0 + n, h] = np.sqrt((a * a) @ (vv * vv))
                t_w[x][page, slot] += (a * a).sum(0)
    return out, w, dict(out=t_out, w={x: np.sqrt(a) for x, a in t_w.items()})


def kept_tokens(weights, length, keep, first, recent):
    """Indices that an eviction of a sequence with these token weights keeps, in order."""
    if length <= keep:
        return list(range(length))
    late = min(keep, recent)
    early = min(keep - late, first, length - late)
    rest = range(early, length - late)
    key = [(-math.inf if math.isnan(weights[j]) else float(weights[j])) for j in range(length)]
    # NaN sorts below every number, -inf included
    rest = sorted(rest, key=lambda j: (bool(math.isnan(weights[j])), -key[j], j))[:keep - late - early]
    return sorted(list(range(early)) + rest + list(range(length - late, length)))


def evict(pool, table, lens, new_pages, keep, first, recent):
    """Evicts in place; returns (new_table, new_lens, kept)."""
    B = len(lens)
    H = pool["k_scale"].shape[1]
    new_table, new_lens = table.copy(), lens.copy()
    kept = np.full((B, keep), -1, np.int32)
    for b in range(B):
        L = int(lens[b])
        j = np.arange(L)
        w = pool["weights"][np.asarray(table[b])[j // PAGE], j % PAGE]
        idx = np.array(kept_tokens(w, L, keep, first, recent), np.int64)
        kept[b, :len(idx)] = idx
        new_lens[b] = len(idx)
        if L <= keep:
            continue
        new_table[b] = new_pages[b]
        for j0 in range(0, keep, PAGE):
            part = idx[j0:j0 + PAGE]
            m, to = len(part), new_pages[b, j0 // PAGE]
            page, slot = np.asarray(table[b])[part // PAGE], part % PAGE
            for name in ("timestamps", "positions", "weights"):
                pool[name][to, :m] = pool[name][page, slot]
            for name in ("k", "v"):
                for h in range(H):
                    x = np.stack([VALUES[_block(pool, name, p, h)[t]] * float(pool[name + "_scale"][p, h])
                                  for p, t in zip(page, slot)])
                    scale = scale_of(np.max(np.abs(x)))
                    codes = _block(pool, name, to, h)
                    codes[:m] = encode(np.where(np.isfinite(x), x, 0.0) * (1.0 / scale if scale > 0 else 0.0))
                    pool[name + "_scale"][to, h] = scale
    return new_table, new_lens, kept
