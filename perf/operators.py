"""The 8-bit paged cache's operators, as cases to be timed and compared.

Five kinds of case: `decode` (attention of a step's new tokens over the cache), `append` (new keys
and values into the cache), `turnover` (the sequences that end give their pages back, others are
forked, all grow), `compact` (the live pages move to the front) and `copy` (pages moved by a list).
Where `own` is false, `run` computes them with elementary torch operations; where it is true, it
makes the framework's calls.

The cache: uint8 [pages, page bytes]. A page holds 64 tokens of every key/value head: the keys' E4M3
codes [heads, 64, D], the values' [heads, 64, D], then for every head four scale bytes for its keys
and four for its values, one for each 16 tokens (a byte e stands for 2^(e - 127)), padded to a
multiple of 128 bytes.
"""
import math

import numpy as np
import torch

own = False

PAGE, BLOCK = 64, 16
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one chat turn on an idle server: nothing to hide latency behind
        dict(name="decode 1 short", kind="decode", B=1, Q=1, H=32, KV=8, D=128, lo=1000, hi=1000, window=0, dtype="bf16"),
        # one long document: the whole card works for eight key/value heads
        dict(name="decode 1 long", kind="decode", B=1, Q=1, H=64, KV=8, D=128, lo=131001, hi=131001, window=0, dtype="bf16"),
        # a speculative-verify step of small heads in a sliding-window layer, four draft tokens a request
        dict(name="decode verify 4 window", kind="decode", B=32, Q=4, H=32, KV=8, D=64, lo=900, hi=9000, window=4096, dtype="fp16"),
        # a full batch of long agent contexts: the largest read
        dict(name="decode 16 long", kind="decode", B=16, Q=1, H=64, KV=8, D=128, lo=20000, hi=90000, window=0, dtype="bf16"),
        # the same step's write: one token a request, most blocks part full
        dict(name="append 64 x 1", kind="append", B=64, KV=8, D=128, n_lo=1, n_hi=1, before=5000, dtype="bf16"),
        # prompts of a prefill batch, ragged, after an odd number of cached tokens
        dict(name="append prompts", kind="append", B=12, KV=8, D=128, n_lo=300, n_hi=9000, before=77, dtype="bf16"),
        # a serving step's bookkeeping: a few requests end, a few are forked, every live one grows by a token
        dict(name="turnover 64", kind="turnover", S=64, pages=4096, page_bytes=32896, layers=1, mean=1500, ended=4, forks=4, add=1),
        # best-of-8 sampling from 32 prompts over four layers' caches
        dict(name="turnover best-of-8", kind="turnover", S=320, pages=12000, page_bytes=8448, layers=4, mean=2500, ended=16, forks=224, add=1),
        # a small pool after a burst: few pages in the way
        dict(name="compact 1000", kind="compact", S=32, pages=1000, page_bytes=22528, live=0.5, mean=900),
        # a large pool half empty: hundreds of megabytes move
        dict(name="compact 40000", kind="compact", S=400, pages=40000, page_bytes=22528, live=0.6, mean=3500),
        # eight pages of a forked request
        dict(name="copy 8", kind="copy", pages=2000, page_bytes=22528, n=8),
        # a batch of requests moved to another part of the pool, 8-bit pages of eight heads
        dict(name="copy 3001", kind="copy", pages=8000, page_bytes=131200, n=3001),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["decode", "decode", "decode", "append", "append", "turnover", "compact", "copy"])
    if kind == "decode":
        KV, D = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128])
        Q, G = rng.choice([1, 1, 2, 3, 5, 8]), rng.choice([1, 2, 4, 5, 8, 16])
        B = _log(rng, 1, 128)
        most = max(200, min(130000, 600000 * 8 * 128 // (B * KV * D), 20000000 // (B * Q * G * KV)))
        hi = _log(rng, 20, most)
        return dict(kind=kind, B=B, Q=Q, H=KV * G, KV=KV, D=D, lo=rng.randint(0, hi), hi=hi, window=rng.choice([0, 0, rng.randint(1, hi)]), dtype=rng.choice(["bf16", "fp16"]))
    if kind == "append":
        KV, D, B = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128]), _log(rng, 1, 256)
        n = _log(rng, 1, max(1, 60000 * 8 * 128 // (B * KV * D) // 8))
        return dict(kind=kind, B=B, KV=KV, D=D, n_lo=rng.randint(0, n), n_hi=n, before=_log(rng, 1, 4000), dtype=rng.choice(["bf16", "fp16"]))
    if kind == "turnover":
        S, mean = _log(rng, 8, 400), _log(rng, 20, 3000)
        return dict(kind=kind, S=S, pages=2 * S * (2 * mean // PAGE + 3), page_bytes=128 * _log(rng, 10, 100), layers=rng.randint(1, 4), mean=mean, ended=rng.randint(0, S // 4), forks=rng.randint(1, S // 2), add=rng.randint(0, 70))
    if kind == "compact":
        S, mean = _log(rng, 4, 400), _log(rng, 64, 1500)
        return dict(kind=kind, S=S, pages=2 * S * (2 * mean // PAGE + 3), page_bytes=128 * _log(rng, 10, 150), live=rng.uniform(0.2, 0.9), mean=mean)
    pages = _log(rng, 20, 8000)
    return dict(kind=kind, pages=pages, page_bytes=16 * _log(rng, 40, 8000), n=_log(rng, 1, max(1, pages * 3 // 8)))


def page_bytes(KV, D):
    return -(-(KV * (2 * PAGE * D + 8)) // 128) * 128


def _spread(n, lo, hi):
    """n lengths from lo to hi, the same for every seed: a step's lengths are part of the case."""
    if n == 1 or lo == hi:
        return np.full(n, hi, np.int32)
    x = np.random.RandomState(n * 7919 + hi).uniform(size=n)
    x[0], x[-1] = 0.0, 1.0
    return np.round(np.exp(np.log(lo + 1) + x * (np.log(hi + 1) - np.log(lo + 1))) - 1).astype(np.int32)


def _tables(lens, pages, g):
    """Page tables [sequences, widest] for lens, pages drawn without replacement."""
    need = torch.from_numpy(-(-lens.astype(np.int64) // PAGE))
    width = max(1, int(need.max()))
    used = torch.arange(width)[None, :] < need[:, None]
    perm = torch.randperm(pages, generator=g)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    table[used] = perm[: int(need.sum())].to(torch.int32)
    return table


def _parts(cache, KV, D):
    """The pages' code bytes of keys and values [pages, KV, 64, D] and their scale bytes [pages, KV, 4], as views."""
    n = KV * PAGE * D
    k = cache[:, :n].unflatten(1, (KV, PAGE, D))
    v = cache[:, n:2 * n].unflatten(1, (KV, PAGE, D))
    s = cache[:, 2 * n:2 * n + 8 * KV].unflatten(1, (KV, 2, 4))
    return k, v, s[:, :, 0], s[:, :, 1]


def _pow2(byte):
    """2^(byte - 127) in 32 bits, exactly, for bytes of 1 to 254."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _random_pages(pages, KV, D, gen):
    """A cache in use: codes of normal values with a few large ones, scales that differ by block."""
    cache = torch.zeros((pages, page_bytes(KV, D)), dtype=torch.uint8, device=DEV)
    k, v, ks, vs = _parts(cache, KV, D)
    for at in range(0, pages, 4096):
        for x in (k, v):
            y = x[at:at + 4096]
            r = torch.randn(y.shape, device=DEV, generator=gen, dtype=torch.float32).mul_(90.0)
            y.copy_(r.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    ks.copy_(torch.randint(119, 122, ks.shape, device=DEV, generator=gen, dtype=torch.uint8))
    vs.copy_(torch.randint(118, 123, vs.shape, device=DEV, generator=gen, dtype=torch.uint8))
    return cache


def _append_counts(case):
    return _spread(case["B"], case["n_lo"], case["n_hi"]), _spread(case["B"], case["before"] // 3, case["before"])


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    kind = case["kind"]
    if kind == "decode":
        lens = _spread(case["B"], case["lo"], case["hi"])
        pages = max(1, int((-(-lens.astype(np.int64) // PAGE)).sum()))
        q = torch.randn((case["B"], case["Q"], case["H"], case["D"]), device=DEV, generator=gen).to(DTYPES[case["dtype"]])
        return dict(case=case, q=q, cache=_random_pages(pages, case["KV"], case["D"], gen), table=_tables(lens, pages, g).to(DEV),
                    lens=torch.from_numpy(lens).to(DEV), scale=case["D"] ** -0.5, out=torch.empty_like(q),
                    lse=torch.empty(q.shape[:3], dtype=torch.float32, device=DEV))
    if kind == "append":
        new, old = _append_counts(case)
        lens = new + old
        pages = int((-(-lens.astype(np.int64) // PAGE)).sum()) + 3
        n = int(new.sum())
        kv = torch.randn((2, n, case["KV"], case["D"]), device=DEV, generator=gen)
        kv *= torch.exp(0.5 * torch.randn((2, 1, case["KV"], case["D"]), device=DEV, generator=gen))
        kv *= torch.where(torch.rand((2, n, case["KV"], 1), device=DEV, generator=gen) < 0.01, 20.0, 1.0)
        kv = kv.to(DTYPES[case["dtype"]])
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        return dict(case=case, k=kv[0], v=kv[1], cu=torch.from_numpy(cu).to(DEV), lens=torch.from_numpy(lens).to(DEV),
                    table=_tables(lens, pages, g).to(DEV), cache=_random_pages(pages, case["KV"], case["D"], gen))
    if kind == "copy":
        cache = torch.randint(0, 256, (case["pages"], case["page_bytes"]), device=DEV, generator=gen, dtype=torch.uint8)
        perm = torch.randperm(case["pages"], generator=g).to(torch.int32).to(DEV)
        return dict(case=case, cache=cache, src=perm[:case["n"]].clone(), dst=perm[case["n"]:2 * case["n"]].clone())
    pages = case["pages"]
    if kind == "compact":
        S = case["S"]
        most = int(case["live"] * pages)
        lens = np.minimum(_spread(S, case["mean"] // 2, case["mean"] * 2), max(1, most // S) * PAGE)
        cache = torch.randint(0, 256, (pages, case["page_bytes"]), device=DEV, generator=gen, dtype=torch.uint8)
        table = _tables(lens, pages, g).to(DEV)
        rc = torch.zeros(pages, dtype=torch.int32, device=DEV)
        rc.index_add_(0, table.clamp(min=0).flatten(), (table >= 0).to(torch.int32).flatten())
        return dict(case=case, cache=cache, table0=table, rc0=rc, table=table.clone(), rc=rc.clone())
    S, F, E = case["S"], case["forks"], case["ended"]
    # the last sequences are empty: the forks' places are theirs and, first, those of the ended ones
    live = max(1, S - max(0, F - E))
    lens = np.zeros(S, np.int32)
    lens[:live] = _spread(live, case["mean"] // 2, case["mean"] * 2)
    order = torch.randperm(live, generator=g)
    ended = order[:min(E, live - 1)]
    stay = order[len(ended):]
    places = torch.cat([ended, torch.arange(live, S)])[:F]
    src = stay[torch.randint(0, len(stay), (len(places),), generator=g)]
    add = np.zeros(S, np.int32)
    add[stay.numpy()] = case["add"]
    add[places.numpy()] = case["add"]
    t = _tables(lens, pages, g)
    width = t.shape[1] + -(-case["add"] // PAGE) + 1
    table = torch.full((S, width), -1, dtype=torch.int32)
    table[:, :t.shape[1]] = t
    table = table.to(DEV)
    rc = torch.zeros(pages, dtype=torch.int32, device=DEV)
    rc.index_add_(0, table.clamp(min=0).flatten(), (table >= 0).to(torch.int32).flatten())
    cache = torch.randint(0, 256, (case["layers"], pages, case["page_bytes"]), device=DEV, generator=gen, dtype=torch.uint8)
    i32 = lambda x: x.to(torch.int32).to(DEV)  # noqa: E731
    lens = torch.from_numpy(lens).to(DEV)
    return dict(case=case, cache=cache, table0=table, rc0=rc, lens0=lens, table=table.clone(), rc=rc.clone(), lens=lens.clone(),
                ended=i32(ended), src=i32(src), dst=i32(places), add=torch.from_numpy(add).to(DEV))


# ------------------------------------------------------------------ decode
def _attend(q, cache, table, lens, KV, scale, window, dtype):
    """softmax(scale q k + mask) v over the cached tokens, and its log-sum-exp, in `dtype`."""
    B, Q, H, D = q.shape
    k, v, ks, vs = (x[table.clamp(min=0).long()] for x in _parts(cache, KV, D))  # [B, P, KV, ...]
    P = table.shape[1]

    def wide(x, s):
        x = x.view(torch.float8_e4m3fn).to(dtype).unflatten(3, (4, BLOCK)) * _pow2(s).to(dtype)[..., None, None]
        return x.flatten(3, 4).transpose(1, 2).flatten(2, 3)  # [B, KV, P * 64, D]

    k, v = wide(k, ks), wide(v, vs)
    t = torch.arange(P * PAGE, device=q.device)
    at = lens[:, None] - Q + torch.arange(Q, device=q.device)  # [B, Q]: the query's own place
    ok = (t <= at[:, :, None]) & ((t > at[:, :, None] - window) if window else True)
    z = torch.einsum("bqhgd,bhtd->bhgqt", q.to(dtype).unflatten(2, (KV, H // KV)), k) * scale
    z = z.masked_fill(~ok[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True).clamp(min=torch.finfo(dtype).min)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    out = torch.einsum("bhgqt,bhtd->bqhgd", e / total.clamp(min=torch.finfo(dtype).tiny), v)
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2)  # an empty row: log 0
    return out.flatten(2, 3), lse.flatten(2, 3)


def _decode(s):
    c = s["case"]
    out, lse = _attend(s["q"], s["cache"], s["table"], s["lens"], c["KV"], s["scale"], c["window"], torch.float32)
    return out.to(s["q"].dtype), lse.contiguous()


# ------------------------------------------------------------------ append
def _scales(amax, before):
    """The smallest power of two that takes amax to at most 448, as a byte, and no less than the block's byte before."""
    m, e = torch.frexp(amax.double() / 448)  # amax / 448 = m 2^e, m in [0.5, 1)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(amax > 0, e, -126).clamp(-126, 126) + 127
    return torch.maximum(e, before).to(torch.int32)


def _append(s):
    """Blocks of 16 tokens of every sequence, padded: the tokens before the new ones, the new ones, and what is behind them."""
    c = s["case"]
    KV, D, B = c["KV"], c["D"], c["B"]
    table, lens, cu = s["table"], s["lens"].long(), s["cu"].long()
    new = cu[1:] - cu[:-1]
    first = lens - new
    N = s["k"].shape[0]
    if N == 0:
        return _append_out(s)
    # every touched block, as (sequence, block): the new tokens' own, each once
    tok = torch.arange(N, device=DEV)
    b = torch.searchsorted(cu, tok, right=True) - 1
    pos = first[b] + tok - cu[b]
    opens = (tok == cu[b]) | (pos % BLOCK == 0)
    at = torch.nonzero(opens).flatten()
    b, block = b[at], pos[at] // BLOCK
    pos = block[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)  # [blocks, 16]
    is_new = (pos >= first[b][:, None]) & (pos < lens[b][:, None])
    is_old = pos < first[b][:, None]
    row = (cu[b][:, None] + pos - first[b][:, None]).clamp(0, N - 1)
    page = table[b, block * BLOCK // PAGE].long()
    quarter = block % (PAGE // BLOCK)
    rows = quarter[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)
    for x, codes, scales in ((s["k"], *_parts(s["cache"], KV, D)[0::2]), (s["v"], *_parts(s["cache"], KV, D)[1::2])):
        x = x[row].to(torch.float32).transpose(1, 2)  # [blocks, KV, 16, D]
        keep = codes[page[:, None], :, rows].transpose(1, 2).contiguous()
        before = scales[page, :, quarter].to(torch.int32)
        fine = is_new[:, None, :, None] & torch.isfinite(x)
        held = torch.where(is_old.any(1)[:, None], before, 0)
        after = _scales(torch.where(fine, x.abs(), 0.0).amax((2, 3)), held)
        fresh = (x * _pow2(254 - after)[..., None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        less = torch.where(is_old.any(1)[:, None], after - before, 0)  # the block's first scale counts from here on
        old = (keep.view(torch.float8_e4m3fn).to(torch.float32) * _pow2(127 - less.clamp(max=126))[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        got = torch.where(is_new[:, None, :, None], fresh, torch.where(is_old[:, None, :, None], old, keep))
        codes[page[:, None], :, rows] = got.transpose(1, 2)
        scales[page, :, quarter] = after.to(torch.uint8)
    return _append_out(s)


def _append_out(s):
    k, v, ks, vs = _parts(s["cache"], s["case"]["KV"], s["case"]["D"])
    return dict(k=k.view(torch.float8_e4m3fn), v=v.view(torch.float8_e4m3fn), k_scales=ks, v_scales=vs)


# ------------------------------------------------------------------ pages
def _lowest_free(rc, n):
    return torch.sort((rc != 0).to(torch.int8), stable=True).indices[:n].to(torch.int32)


def _free(table, lens, rc, seqs):
    rows = table[seqs.long()]
    rc.index_add_(0, rows.clamp(min=0).flatten(), -(rows >= 0).to(torch.int32).flatten())
    table[seqs.long()] = -1
    lens[seqs.long()] = 0


def _fork(cache, table, lens, rc, src, dst):
    src, dst = src.long(), dst.long()
    n = lens[src]
    part = n % PAGE > 0
    fresh = _lowest_free(rc, len(src))[(torch.cumsum(part, 0) - 1).clamp(min=0)]
    rows = table[src]
    last = (n // PAGE).clamp(max=table.shape[1] - 1).long()
    is_last = (torch.arange(table.shape[1], device=DEV) == last[:, None]) & part[:, None]
    shared = (rows >= 0) & ~is_last
    rc.index_add_(0, rows.clamp(min=0).flatten(), shared.to(torch.int32).flatten())
    rc.index_add_(0, fresh, part.to(torch.int32))
    table[dst] = torch.where(is_last, fresh[:, None], rows)
    lens[dst] = n
    at = torch.nonzero(part).flatten()
    old = rows.gather(1, last[:, None])[:, 0]
    cache[:, fresh[at].long()] = cache[:, old[at].long()]
    return torch.where(part, fresh, -1)


def _extend(table, lens, rc, add):
    have, want = (lens + PAGE - 1) // PAGE, (lens + add + PAGE - 1) // PAGE
    need = want - have
    col = torch.arange(table.shape[1], device=DEV)
    is_new = (col >= have[:, None]) & (col < want[:, None])
    rank = (torch.cumsum(need, 0) - need)[:, None] + col - have[:, None]
    fresh = _lowest_free(rc, rc.shape[0])[rank.clamp(0, rc.shape[0] - 1)]
    rc.index_add_(0, torch.where(is_new, fresh, 0).flatten(), is_new.to(torch.int32).flatten())
    table.copy_(torch.where(is_new, fresh, table))
    lens.add_(add)


def _compact(cache, table, rc):
    live = rc > 0
    n = live.sum()
    page = torch.arange(rc.shape[0], device=DEV)
    move, hole = live & (page >= n), ~live & (page < n)
    src, dst = torch.nonzero(move).flatten(), torch.nonzero(hole).flatten()
    remap = torch.where(live, page, -1)
    remap[src] = dst
    cache[dst] = cache[src]
    rc[dst] = rc[src]
    rc[src] = 0
    table.copy_(torch.where(table >= 0, remap[table.clamp(min=0).long()].to(torch.int32), -1))
    return remap.to(torch.int32), n.to(torch.int32).reshape(1)


def run(s):
    kind = s["case"]["kind"]
    if own:
        import nvfp4_compressed_sparse_gb300 as m
    if kind == "decode":
        if not own:
            return _decode(s)
        c = s["case"]
        if "workspace" not in s:  # kept by a program from step to step
            s["workspace"] = torch.empty(m.kv8_decode_workspace_size(c["B"], c["Q"], c["H"], c["KV"], c["D"]), dtype=torch.uint8, device=DEV)
        return m.kv8_decode(s["q"], s["cache"], s["table"], s["lens"], c["KV"], s["scale"], window=c["window"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
    if kind == "append":
        if not own:
            return _append(s)
        m.kv8_append(s["k"], s["v"], s["cu"], s["lens"], s["table"], s["cache"])
        return _append_out(s)
    if kind == "copy":
        if own:
            m.kv_pages_copy(s["cache"], s["src"], s["dst"])
        else:
            s["cache"][s["dst"].long()] = s["cache"][s["src"].long()]
        return s["cache"]
    # the tables are put back first, so that every pass finds the step's start
    table, rc = s["table"].copy_(s["table0"]), s["rc"].copy_(s["rc0"])
    if kind == "compact":
        remap, live = m.kv_pages_compact(s["cache"], table, rc) if own else _compact(s["cache"], table, rc)
        return dict(cache=s["cache"], table=table, rc=rc, remap=remap, live=live)
    lens = s["lens"].copy_(s["lens0"])
    if own:
        m.kv_pages_free(table, lens, rc, s["ended"])
        fresh = m.kv_pages_fork(s["cache"], table, lens, rc, s["src"], s["dst"], layered=True)
        m.kv_pages_extend(table, lens, rc, s["add"])
    else:
        _free(table, lens, rc, s["ended"])
        fresh = _fork(s["cache"], table, lens, rc, s["src"], s["dst"])
        _extend(table, lens, rc, s["add"])
    return dict(cache=s["cache"], table=table, lens=lens, rc=rc, fresh=fresh)


def work(case):
    kind = case["kind"]
    if kind == "decode":
        lens = _spread(case["B"], case["lo"], case["hi"]).astype(np.int64)
        Q, H, KV, D, w = case["Q"], case["H"], case["KV"], case["D"], case["window"]
        at = lens[:, None] - Q + np.arange(Q)
        seen = np.maximum(at + 1, 0)
        seen = np.minimum(seen, w) if w else seen
        read = lens - np.maximum(0, lens - Q + 1 - w) if w else lens
        return dict(bytes=float(read.sum()) * KV * (2 * D + 0.5) + lens.size * Q * H * (4 * D + 4) + 4.0 * float((-(-read // PAGE)).sum()),
                    flops=4.0 * float(seen.sum()) * H * D)
    if kind == "append":
        new, _ = _append_counts(case)
        n = float(new.sum()) * case["KV"] * case["D"] * 2
        return dict(bytes=3 * n + 4.0 * (4 * case["B"]) + 1, flops=2 * n)
    if kind == "copy":
        return dict(bytes=2.0 * case["n"] * case["page_bytes"] + 8 * case["n"], flops=0)
    if kind == "compact":
        s_pages = np.minimum(-(-_spread(case["S"], case["mean"] // 2, case["mean"] * 2).astype(np.int64) // PAGE), max(1, int(case["live"] * case["pages"]) // case["S"]))
        live = int(s_pages.sum())
        moved = live * (1 - live / case["pages"])  # a live page lies behind the live ones' number as often as a free one before it
        return dict(bytes=2.0 * moved * case["page_bytes"] + 12.0 * case["pages"] + 8.0 * live, flops=0)
    S, F, E = case["S"], case["forks"], case["ended"]
    rows = case["mean"] * 1.1 / PAGE
    return dict(bytes=2.0 * F * case["layers"] * case["page_bytes"] + 4.0 * case["pages"] + 4.0 * rows * (2 * E + 3 * F) + 16.0 * S, flops=0)


# ------------------------------------------------------------------ 64 bits, written apart
def exact(case, seed):
    if case["kind"] == "decode":
        return _exact_decode(prepare(case, seed))
    if case["kind"] == "append":
        return _exact_append(prepare(case, seed))
    return None


def _value(byte):
    """E4M3 bytes as 64-bit numbers, from the format: sign, four bits of exponent, three of mantissa."""
    i = torch.arange(256, dtype=torch.float64)
    e, m = torch.div(i % 128, 8, rounding_mode="floor"), i % 8
    table = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e - 10))
    table = torch.where(i >= 128, -table, table)
    table[127] = table[255] = math.nan
    return table.to(byte.device)[byte.long()]


def _exact_decode(s):
    c = s["case"]
    KV, D, Q, G = c["KV"], c["D"], c["Q"], c["H"] // c["KV"]
    table, lens = s["table"].cpu(), s["lens"].cpu().tolist()
    out = torch.zeros((c["B"], Q, c["H"], D), dtype=torch.float64, device=DEV)
    lse = torch.full((c["B"], Q, c["H"]), -math.inf, dtype=torch.float64, device=DEV)
    n = KV * PAGE * D
    for b, L in enumerate(lens):
        if L == 0:
            continue
        raw = s["cache"][table[b, :-(-L // PAGE)].long().to(DEV)]
        sc = torch.exp2(raw[:, 2 * n:2 * n + 8 * KV].reshape(-1, KV, 2, 4).double() - 127).repeat_interleave(BLOCK, 3)
        for h in range(KV):
            k = (_value(raw[:, h * PAGE * D:(h + 1) * PAGE * D].reshape(-1, PAGE, D)) * sc[:, h, 0, :, None]).reshape(-1, D)[:L]
            v = (_value(raw[:, n + h * PAGE * D:n + (h + 1) * PAGE * D].reshape(-1, PAGE, D)) * sc[:, h, 1, :, None]).reshape(-1, D)[:L]
            for j in range(Q):
                end = L - Q + j + 1
                start = max(0, end - c["window"]) if c["window"] else 0
                if end <= 0:
                    continue
                z = s["q"][b, j, h * G:(h + 1) * G].double() @ k[start:end].T * s["scale"]
                lse[b, j, h * G:(h + 1) * G] = torch.logsumexp(z, 1)
                out[b, j, h * G:(h + 1) * G] = torch.softmax(z, 1) @ v[start:end]
    return out, lse


def _nearest(x):
    """The E4M3 number nearest to x (64-bit), ties to the even mantissa, at most 448 in size."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    unit = torch.exp2(e - 3)
    return (torch.round(x / unit) * unit).clamp(-448, 448)


def _exact_append(s):
    c = s["case"]
    KV, D = c["KV"], c["D"]
    n, cu, lens = KV * PAGE * D, s["cu"].cpu().tolist(), s["lens"].cpu().tolist()
    if sum(-(-(b - a) // BLOCK) + 1 for a, b in zip(cu, cu[1:])) > 6000:
        return None
    raw, table = s["cache"], s["table"].cpu()
    answer = []
    for which, x in ((0, s["k"]), (1, s["v"])):
        codes = _value(raw[:, which * n:(which + 1) * n]).reshape(-1, KV, PAGE, D)
        scale = raw[:, 2 * n:2 * n + 8 * KV].reshape(-1, KV, 2, 4)[:, :, which].to(torch.int64).clone()
        for b, L in enumerate(lens):
            start = L - (cu[b + 1] - cu[b])
            at = start
            while at < L:
                end = min(L, at // BLOCK * BLOCK + BLOCK)
                page, lo, quarter = int(table[b, at // PAGE]), at % PAGE, at % PAGE // BLOCK
                y = x[cu[b] + at - start:cu[b] + end - start].double().transpose(0, 1)
                top = y.abs().amax((1, 2))
                e = torch.where(top > 0, torch.ceil(torch.log2(top / 448)), -126.0)
                e = torch.where(top > 448 * torch.exp2(e), e + 1, torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e))
                e = e.clamp(-126, 126).long() + 127
                if lo % BLOCK:
                    old = scale[page, :, quarter]
                    e = torch.maximum(e, old)
                    part = codes[page, :, quarter * BLOCK:lo]
                    codes[page, :, quarter * BLOCK:lo] = _nearest(part * torch.exp2((old - e).double())[:, None, None])
                codes[page, :, lo:lo + end - at] = _nearest(y * torch.exp2(127.0 - e)[:, None, None])
                scale[page, :, quarter] = e
                at = end
        answer.append((codes, scale))
    return dict(k=answer[0][0], v=answer[1][0], k_scales=answer[0][1], v_scales=answer[1][1])
