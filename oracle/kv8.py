"""The 8-bit per-head cache and the page operators, in 64 bits and plain loops.

Written from the definitions in include/nvfp4mla.h; shares no code with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

from oracle.codec import e4m3_decode, e4m3_encode

PAGE, BLOCK = 64, 16


def page_bytes(kv_heads: int, head_dim: int) -> int:
    n = kv_heads * (2 * PAGE * head_dim + 8)
    return (n + 127) // 128 * 128


def parts(cache: np.ndarray, kv_heads: int, head_dim: int):
    """Views of a cache [P, page bytes]: codes [P, 2, Hk, 64, D] and scale bytes [P, Hk, 2, 4]."""
    n = kv_heads * PAGE * head_dim
    codes = cache[:, :2 * n].reshape(cache.shape[0], 2, kv_heads, PAGE, head_dim)
    scales = cache[:, 2 * n:2 * n + 8 * kv_heads].reshape(cache.shape[0], kv_heads, 2, 4)
    assert np.shares_memory(codes, cache) and np.shares_memory(scales, cache)
    return codes, scales


def scale_byte(amax: float) -> int:
    """The smallest byte e, 1 <= e <= 253, with amax <= 448 * 2^(e - 127)."""
    e = 1
    while e < 253 and amax > 448.0 * math.ldexp(1.0, e - 127):
        e += 1
    return e


def append(cache, k, v, cu_tokens, seq_lens, page_table, kv_heads: int, head_dim: int) -> list:
    """Writes k, v (float64 [N, Hk, D]) into cache, in place. Returns [bad pages, bad requests]."""
    codes, scales = parts(cache, kv_heads, head_dim)
    bad_pages = bad_requests = 0
    for b in range(len(seq_lens)):
        c0, c1, length = int(cu_tokens[b]), int(cu_tokens[b + 1]), int(seq_lens[b])
        first = length - (c1 - c0)
        if c0 < 0 or c1 < c0 or c1 > len(k) or (first < 0 and c1 > c0):
            bad_requests += 1
            continue
        at = first
        while at < length:
            end = min(length, at // BLOCK * BLOCK + BLOCK)
            col = at // PAGE
            page = int(page_table[b][col]) if col < page_table.shape[1] else -1
            if not 0 <= page < len(cache):
                bad_pages += 1
                at = end
                continue
            lo, block = at % PAGE, at % PAGE // BLOCK
            for which, x in enumerate((k, v)):
                for h in range(kv_heads):
                    new = x[c0 + at - first:c0 + end - first, h]
                    fine = np.abs(new[np.isfinite(new)])
                    e = scale_byte(float(fine.max()) if fine.size else 0.0)
                    if lo % BLOCK:
                        before = int(scales[page, h, which, block])
                        if before > e:
                            e = before
                        old = codes[page, which, h, block * BLOCK:lo]
                        nan = (old & 0x7F) == 0x7F
                        less = e4m3_encode(np.where(nan, 0.0, e4m3_decode(old)) * 2.0 ** (before - e))
                        codes[page, which, h, block * BLOCK:lo] = np.where(nan, old, less)
                    nan = np.isnan(new)
                    got = e4m3_encode(np.where(nan, 0.0, np.clip(new, -1e300, 1e300)) * 2.0 ** (127 - e))
                    codes[page, which, h, lo:lo + end - at] = np.where(nan, 0x7F | (np.signbit(new) * 0x80), got)
                    scales[page, h, which, block] = e
            at = end
    return [bad_pages, bad_requests]


def rows(cache, page_row, length: int, kv_heads: int, head_dim: int):
    """Keys and values float64 [Hk, length, D] of one request, and which positions have a page."""
    codes, scales = parts(cache, kv_heads, head_dim)
    k = np.zeros((kv_heads, length, head_dim))
    v = np.zeros_like(k)
    have = np.zeros(length, bool)
    for t0 in range(0, length, PAGE):
        col = t0 // PAGE
        page = int(page_row[col]) if col < len(page_row) else -1
        n = min(PAGE, length - t0)
        if not 0 <= page < len(cache):
            continue
        have[t0:t0 + n] = True
        for which, x in ((0, k), (1, v)):
            s = np.repeat(2.0 ** (scales[page, :, which].astype(np.float64) - 127), BLOCK, axis=1)
            x[:, t0:t0 + n] = (e4m3_decode(codes[page, which]) * s[..., None])[:, :n]
    return k, v, have


def value_scales(cache, page_row, length: int, kv_heads: int, head_dim: int):
    """The values' scales float64 [Hk, length] (1 where there is no page)."""
    _, scales = parts(cache, kv_heads, head_dim)
    s = np.ones((kv_heads, length))
    for t in range(0, length, BLOCK):
        page = int(page_row[t // PAGE]) if t // PAGE < len(page_row) else -1
        if 0 <= page < len(cache):
            s[:, t:t + BLOCK] = 2.0 ** (scales[page, :, 1, t % PAGE // BLOCK].astype(np.float64) - 127)[:, None]
    return s


def decode(q, cache, page_table, seq_lens, kv_heads: int, scale: float, window: int = 0):
    """out float64 [B, Q, H, D] and lse [B, Q, H] for q float64 [B, Q, H, D], and what rounding bounds
    are made of: mass = sum_t p_t |v_t| [B, Q, H, D], reach = max_t scale * sum_d |q_d k_td| [B, Q, H],
    and spread = max_t (p_t s_t) * sum_t |code_t| [B, Q, H, D], s_t and code_t a value's scale and code."""
    B, Q, H, D = q.shape
    mass, reach, spread = np.zeros(q.shape), np.zeros(q.shape[:3]), np.zeros(q.shape)
    out = np.zeros(q.shape)
    lse = np.full(q.shape[:3], -np.inf)
    for b in range(B):
        length = max(0, int(seq_lens[b]))
        k, v, have = rows(cache, page_table[b], length, kv_heads, D)
        s = value_scales(cache, page_table[b], length, kv_heads, D)
        for j in range(Q):
            p = length - Q + j
            t = np.arange(length)
            ok = have & (t <= p) & ((t > p - window) if window else True)
            if not ok.any():
                continue
            for h in range(H):
                g = h // (H // kv_heads)
                with np.errstate(invalid="ignore"):
                    z = scale * (k[g][ok] @ q[b, j, h])
                    m = z.max()
                    e = np.exp(z - m)
                    out[b, j, h] = (e[:, None] * v[g][ok]).sum(0) / e.sum()
                    lse[b, j, h] = m + np.log(e.sum())
                    mass[b, j, h] = (e[:, None] * np.abs(v[g][ok])).sum(0) / e.sum()
                    reach[b, j, h] = scale * (np.abs(k[g][ok]) @ np.abs(q[b, j, h])).max()
                    spread[b, j, h] = (e * s[g][ok]).max() / e.sum() * (np.abs(v[g][ok]) / s[g][ok][:, None]).sum(0)
    return out, lse, mass, reach, spread


# ------------------------------------------------------------------ pages
def lowest_free(refs, n: int) -> list:
    return [int(p) for p in np.flatnonzero(np.asarray(refs) == 0)[:n]]


def copy(cache, src, dst) -> int:
    """cache [layers, P, bytes], in place; returns the bad pairs."""
    before, bad = cache.copy(), 0
    for s, d in zip(src, dst):
        if s == -1 or d == -1:
            continue
        if not (0 <= s < cache.shape[1] and 0 <= d < cache.shape[1]):
            bad += 1
            continue
        cache[:, d] = before[:, s]
    return bad


def free(table, lens, refs, seqs) -> None:
    for s in seqs:
        if not 0 <= s < len(lens):
            continue
        for i, p in enumerate(table[s]):
            if 0 <= p < len(refs) and refs[p] > 0:
                refs[p] -= 1
            table[s, i] = -1
        lens[s] = 0


def fork(cache, table, lens, refs, src, dst) -> list:
    """cache [layers, P, bytes], in place; returns new_pages."""
    lens0, named, pairs = lens.copy(), set(), []
    for s, d in zip(src, dst):
        ok = 0 <= s < len(lens) and 0 <= d < len(lens) and s != d
        n = int(lens0[s]) if ok else 0
        if ok and (n < 0 or -(-n // PAGE) > table.shape[1]):
            ok = False
        if ok and n % PAGE and not 0 <= table[s, n // PAGE] < len(refs):
            ok = False
        if ok and (lens0[d] != 0 or d in named):
            ok = False
        if ok:
            named.add(d)
        pairs.append((s, d, n, ok))
    pages = lowest_free(refs, len(pairs))
    new, taken = [], 0
    for s, d, n, ok in pairs:
        if not ok:
            new.append(-2)
            continue
        fresh = -1
        if n % PAGE:
            taken += 1
            if taken > len(pages):
                new.append(-2)
                continue
            fresh = pages[taken - 1]
            refs[fresh] = 1
            cache[:, fresh] = cache[:, table[s, n // PAGE]]
        for i in range(table.shape[1]):
            p = -1
            if i < n // PAGE and 0 <= table[s, i] < len(refs):
                p = table[s, i]
                refs[p] += 1
            elif i == n // PAGE and fresh >= 0:
                p = fresh
            table[d, i] = p
        lens[d] = n
        new.append(fresh)
    return new


def extend(table, lens, refs, add) -> list:
    pages, at, granted = lowest_free(refs, len(refs)), 0, []
    for s in range(len(lens)):
        have, want = -(-int(lens[s]) // PAGE), -(-(int(lens[s]) + int(add[s])) // PAGE)
        if lens[s] < 0 or add[s] < 0 or (add[s] > 0 and want > table.shape[1]):
            granted.append(0)
            continue
        if want - have > len(pages) - at:
            granted.append(0)
            continue
        for i in range(want - have):
            table[s, have + i] = pages[at + i]
            refs[pages[at + i]] = 1
        at += max(0, want - have)
        lens[s] += add[s]
        granted.append(1)
    return granted


def compact(cache, table, refs):
    """cache [layers, P, bytes], in place; returns (remap, number of pages in use)."""
    live = [int(p) for p in np.flatnonzero(refs > 0)]
    n = len(live)
    holes = [p for p in range(n) if refs[p] <= 0]
    remap = np.full(len(refs), -1, np.int32)
    for p in live:
        remap[p] = p
    for p, to in zip([p for p in live if p >= n], holes):
        remap[p] = to
        cache[:, to] = cache[:, p]
        refs[to], refs[p] = refs[p], 0
    for s in range(table.shape[0]):
        for i in range(table.shape[1]):
            p = table[s, i]
            if p != -1:
                table[s, i] = remap[p] if 0 <= p < len(refs) else -1
    return remap, n
