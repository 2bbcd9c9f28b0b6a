"""The speculative step over the 8-bit per-head cache, in 64 bits and plain loops.

Written from the definitions in include/nvfp4mla.h; shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

from oracle import kv8
from oracle.codec import e4m3_decode, e4m3_encode

PAGE, BLOCK = kv8.PAGE, kv8.BLOCK


def places(cu_tokens, seq_lens, n: int) -> np.ndarray:
    """Each token's place in its sequence, -1 where it belongs to none."""
    at = np.full(n, -1, np.int64)
    for b in range(len(seq_lens)):
        c0, c1 = int(cu_tokens[b]), int(cu_tokens[b + 1])
        if 0 <= c0 <= c1 <= n and int(seq_lens[b]) >= c1 - c0:
            at[c0:c1] = int(seq_lens[b]) - (c1 - c0) + np.arange(c1 - c0)
    return at


def rotate(x, weight, eps, cos_sin, positions, sections, interleaved: bool):
    """x float64 [N, heads, D] normalised (weight [D] or None) and turned; positions [axes][N], sections [axes].
    Returns the result and, for every element, a bound on what its two products add up to in size."""
    x = np.array(x, np.float64)
    if weight is not None:
        with np.errstate(invalid="ignore", divide="ignore"):
            x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    half = cos_sin.shape[1] // 2
    y, size = x.copy(), np.abs(x)
    axis = np.repeat(np.arange(len(sections)), sections)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        for t in range(x.shape[0]):
            p = int(positions[axis[i]][t])
            c, s = cos_sin[p, [i, half + i]].astype(np.float64) if 0 <= p < len(cos_sin) else (np.nan, np.nan)
            with np.errstate(invalid="ignore"):
                y[t, :, a], y[t, :, b] = x[t, :, a] * c - x[t, :, b] * s, x[t, :, b] * c + x[t, :, a] * s
                size[t, :, a] = np.abs(x[t, :, a] * c) + np.abs(x[t, :, b] * s)
                size[t, :, b] = np.abs(x[t, :, b] * c) + np.abs(x[t, :, a] * s)
    return y, size


def bits(mask: int, Q: int) -> list:
    return [i for i in range(Q) if (int(mask) >> i) & 1]


def decode_tree(q, cache, page_table, seq_lens, masks, kv_heads: int, scale: float, window: int = 0):
    """As kv8.decode, for trees: masks [B, Q] of unsigned numbers. A sixth result: span = max_t scale * max_d |q_d| *
    sum_d |k_td|."""
    B, Q, H, D = q.shape
    out, mass, spread = (np.zeros(q.shape) for _ in range(3))
    lse, reach, span = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3]), np.zeros(q.shape[:3])
    for b in range(B):
        length = max(0, int(seq_lens[b]))
        base = length - Q
        k, v, have = kv8.rows(cache, page_table[b], length, kv_heads, D)
        s = kv8.value_scales(cache, page_table[b], length, kv_heads, D)
        for j in range(Q):
            if int(masks[b, j]) == 0:
                continue
            nodes = bits(masks[b, j], Q)
            place = base + max(1, len(nodes)) - 1
            ok = np.zeros(length, bool)
            ok[max(0, place - window + 1) if window else 0:max(0, base)] = True
            for i in nodes:
                if base + i >= 0:
                    ok[base + i] = True
            ok &= have
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
                    span[b, j, h] = scale * np.abs(q[b, j, h]).max() * np.abs(k[g][ok]).sum(1).max()
                    spread[b, j, h] = (e * s[g][ok]).max() / e.sum() * (np.abs(v[g][ok]) / s[g][ok][:, None]).sum(0)
    return out, lse, mass, reach, spread, span


def softmax(x, t: float):
    """Probabilities of a row of logits at a temperature above 0; zeros where the row has none."""
    x = np.where(np.isnan(x), -np.inf, np.asarray(x, np.float64))
    m = x.max()
    if m == -np.inf:
        return np.zeros(len(x))
    with np.errstate(invalid="ignore"):
        e = np.where(x == m, 1.0, np.where(x == -np.inf, 0.0, np.exp((x - m) / t)))
    return e / e.sum()


def verify(logits, drafts, parents, uniforms, temperatures=None, draft_probs=None):
    """(tokens, path, accepted, bad, nearest): nearest is how close the closest decision or draw of a request came to
    falling otherwise, as a share of the probability."""
    B, Q, V = logits.shape
    tokens, path = np.full((B, Q), -1, np.int32), np.full((B, Q), -1, np.int32)
    accepted, nearest, bad = np.zeros(B, np.int32), np.full(B, np.inf), 0
    for b in range(B):
        t = 1.0 if temperatures is None else float(temperatures[b])
        u = [max(0.0, float(x)) if x < 1 else np.inf for x in uniforms[b]]
        node = [j == 0 or (0 <= parents[b, j] < j and 0 <= drafts[b, j] < V) for j in range(Q)]
        bad += sum(1 for j in range(1, Q) if parents[b, j] != -1 and not node[j])
        at, n = 0, 0
        while True:
            row = np.asarray(logits[b, at], np.float64)
            children = [j for j in range(at + 1, Q) if node[j] and parents[b, j] == at]
            took, word = None, -1
            if not t > 0:
                clean = np.where(np.isnan(row), -np.inf, row)
                word = int(clean.argmax()) if clean.max() > -np.inf else -1
                took = next((j for j in children if drafts[b, j] == word), None)
            else:
                p = softmax(row, t)
                r, s = p.copy(), 1.0
                for j in children:
                    x = int(drafts[b, j])
                    if draft_probs is None:
                        q = np.zeros(V)
                        q[x] = 1.0
                    else:
                        q = np.asarray(draft_probs[b, at], np.float64)
                    with np.errstate(invalid="ignore"):
                        nearest[b] = min(nearest[b], abs(u[j] * q[x] * s - r[x]) if u[j] < np.inf else np.inf)
                        if u[j] * q[x] * s < r[x]:
                            took = j
                            break
                        r = np.fmax(r - s * q, 0.0)
                    s = r.sum()
                if took is None and p.sum() > 0:
                    r = r if r.sum() > 0 else p
                    run = r.cumsum()
                    with np.errstate(invalid="ignore"):
                        past = np.flatnonzero((r > 0) & (run > u[0] * run[-1]))
                    word = int(past[0]) if len(past) else int(np.flatnonzero(r > 0)[-1])
                    if u[0] < 1:
                        nearest[b] = min(nearest[b], np.abs(run - u[0] * run[-1])[r > 0].min() / run[-1])
            if took is None:
                tokens[b, n] = word
                bad += word < 0
                break
            tokens[b, n], path[b, n] = drafts[b, took], took
            n, at = n + 1, took
        accepted[b] = n
    return tokens, path, accepted, bad, nearest


def keep(caches, page_table, seq_lens, path, accepted, kv_heads: int, head_dim: int):
    """caches [layers, P, bytes], in place. Returns (new lengths, bad pages, bad requests)."""
    Q = path.shape[1]
    new, bad_pages, bad = [], 0, 0
    for b in range(len(seq_lens)):
        length, n = int(seq_lens[b]), int(accepted[b])
        base = length - Q
        nodes = [int(x) for x in path[b, :max(0, n)]]
        if n >= 0 and (base < 0 or n >= Q or any(y <= x for x, y in zip([0] + nodes, nodes)) or any(x >= Q for x in nodes)):
            bad += 1
            new.append(length)
            continue
        new.append(length if n < 0 else base + 1 + n)
        if n <= 0:
            continue

        def page_of(t):
            p = int(page_table[b][t // PAGE]) if t // PAGE < page_table.shape[1] else -1
            return p if 0 <= p < caches.shape[1] else -1
        before = caches.copy()
        for t0 in range((base + 1) // BLOCK * BLOCK, base + n + 1, BLOCK):
            src = {t: base + nodes[t - base - 1] if t > base else t for t in range(t0, min(t0 + BLOCK, base + n + 1))}
            if all(t == s for t, s in src.items()):
                continue
            if page_of(t0) < 0:
                bad_pages += 1
                continue
            bad_pages += sum(1 for s in src.values() if page_of(s) < 0)
            src = {t: s for t, s in src.items() if page_of(s) >= 0}
            if not src:
                continue
            for layer in range(len(caches)):
                codes0, scales0 = kv8.parts(before[layer], kv_heads, head_dim)
                codes, scales = kv8.parts(caches[layer], kv_heads, head_dim)
                for which in range(2):
                    for h in range(kv_heads):
                        byte = {t: int(scales0[page_of(s), h, which, s % PAGE // BLOCK]) for t, s in src.items()}
                        top = max(byte.values())
                        for t, s in src.items():
                            old = codes0[page_of(s), which, h, s % PAGE]
                            nan = (old & 0x7F) == 0x7F
                            less = e4m3_encode(np.where(nan, 0.0, e4m3_decode(old)) * 2.0 ** (byte[t] - top))
                            codes[page_of(t), which, h, t % PAGE] = np.where(nan, old, less)
                        scales[page_of(t0), h, which, t0 % PAGE // BLOCK] = top
    return np.array(new, np.int32), bad_pages, bad


def trim(table, lens, refs, new_lens) -> int:
    """In place; returns how many were refused."""
    bad = 0
    for s in range(len(lens)):
        now = int(new_lens[s])
        if now < 0 or now > int(lens[s]):
            bad += 1
            continue
        for i in range(-(-now // PAGE), min(-(-int(lens[s]) // PAGE), table.shape[1])):
            p = int(table[s, i])
            if 0 <= p < len(refs) and refs[p] > 0:
                refs[p] -= 1
            table[s, i] = -1
        lens[s] = now
    return bad
