"""A speculative step over the 8-bit per-head cache, as cases to be timed and compared.

Four kinds of case: `rope` (queries and keys normalised and rotated, keys and values into the cache),
`tree` (attention of a tree of drafted tokens over the cache), `verify` (which drafts the target's
distribution accepts, and the token after them) and `accept` (the accepted drafts' keys and values
move up, the sequences give back what lies behind them). Where `own` is false, `run` computes them with
elementary torch operations; where it is true, it makes the framework's calls.

The cache: uint8 [pages, page bytes]. A page holds 64 tokens of every key/value head: the keys' E4M3
codes [heads, 64, D], the values' [heads, 64, D], then for every head four scale bytes for its keys
and four for its values, one for each 16 tokens (a byte e stands for 2^(e - 127)), padded to a
multiple of 128 bytes.

A tree: Q nodes a request, at its sequence's last Q places. Node 0 is the newest token that is certain,
the others are drafts; a node's parent has a smaller number (-1: no node, padding). Bit i of a node's
mask: it attends to node i (itself and its ancestors; 0 for padding).
"""
import math

import numpy as np
import torch

own = False

PAGE, BLOCK = 64, 16
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # a decode step of a full batch, one token a request: norms of each head, whole heads rotated
        dict(name="rope 64 x 1", kind="rope", B=64, H=32, KV=8, D=128, n_lo=1, n_hi=1, before=5000, rot=128, inter=False, norm=True, axes=1, tree=False, dtype="bf16"),
        # a verify step: trees of 32 drafts, whose places in the text are not their places in the cache
        dict(name="rope trees", kind="rope", B=16, H=64, KV=8, D=64, n_lo=32, n_hi=32, before=3000, rot=32, inter=True, norm=False, axes=1, tree=True, dtype="fp16"),
        # prompts with images: places of time, height and width, ragged, after an odd number of cached tokens
        dict(name="rope prompts", kind="rope", B=12, H=32, KV=8, D=128, n_lo=300, n_hi=9000, before=77, rot=128, inter=False, norm=True, axes=3, tree=False, dtype="bf16"),
        # one chat turn with a small tree: nothing to hide latency behind
        dict(name="tree 1 short", kind="tree", B=1, Q=8, H=32, KV=8, D=128, lo=1000, hi=1000, window=0, dtype="bf16"),
        # one long document, a tree of 16
        dict(name="tree 1 long", kind="tree", B=1, Q=16, H=64, KV=8, D=128, lo=131001, hi=131001, window=0, dtype="bf16"),
        # a batch of chats, trees of 32
        dict(name="tree 16 x 32", kind="tree", B=16, Q=32, H=32, KV=8, D=128, lo=2000, hi=16000, window=0, dtype="bf16"),
        # the largest trees in a sliding-window layer of small heads
        dict(name="tree 64 window", kind="tree", B=24, Q=64, H=32, KV=4, D=64, lo=900, hi=9000, window=4096, dtype="fp16"),
        # one request, four drafts in a row with the draft model's distributions
        dict(name="verify 1 chain", kind="verify", B=1, Q=5, V=32000, drafts=True, width=1, dtype="fp32"),
        # a batch of them over a large vocabulary
        dict(name="verify 64 chains", kind="verify", B=64, Q=5, V=128000, drafts=True, width=1, dtype="bf16"),
        # trees of a draft head's likeliest tokens, an odd vocabulary
        dict(name="verify 16 trees", kind="verify", B=16, Q=32, V=100003, drafts=False, width=4, dtype="bf16"),
        # the end of such a step in eight layers
        dict(name="accept 16 trees", kind="accept", B=16, Q=32, KV=8, D=128, layers=8, before=600, dtype="bf16"),
        # a large batch of small trees, four layers of small heads
        dict(name="accept 128", kind="accept", B=128, Q=12, KV=4, D=64, layers=4, before=900, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    kind = rng.choice(["rope", "rope", "tree", "tree", "tree", "verify", "verify", "accept"])
    KV, D = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128])
    if kind == "rope":
        B, G, tree = _log(rng, 1, 256), rng.choice([1, 2, 4, 5, 8]), rng.random() < 0.3
        n = rng.randint(1, 64) if tree else _log(rng, 1, 30000)
        n = max(1, min(n, 60000 * 1024 // (B * KV * (G + 2) * D) // 3))
        return dict(kind=kind, B=B, H=KV * G, KV=KV, D=D, n_lo=n if tree else rng.randint(0, n), n_hi=n, before=_log(rng, 1, 4000), rot=rng.choice([D, D, D // 2, 16, 48]), inter=rng.random() < 0.4,
                    norm=rng.random() < 0.6, axes=rng.choice([1, 1, 2, 3]), tree=tree, dtype=rng.choice(["bf16", "fp16"]))
    if kind == "tree":
        Q, G, B = _log(rng, 1, 64), rng.choice([1, 2, 4, 5, 8, 16]), _log(rng, 1, 64)
        most = max(2 * Q, min(130000, 600000 * 1024 // (B * KV * D), 250000000 // (B * Q * G * KV)))
        hi = _log(rng, Q, most)
        return dict(kind=kind, B=B, Q=Q, H=KV * G, KV=KV, D=D, lo=rng.randint(Q, hi), hi=hi, window=rng.choice([0, 0, rng.randint(Q, 2 * hi)]), dtype=rng.choice(["bf16", "fp16"]))
    if kind == "verify":
        drafts = rng.random() < 0.5
        V, Q = _log(rng, 500, 200000), _log(rng, 1, 16 if drafts else 64)
        return dict(kind=kind, B=_log(rng, 1, max(1, min(128, 50000000 // (Q * V)))), Q=Q, V=V, drafts=drafts, width=rng.choice([1, 1, 2, 3]) if drafts else rng.choice([1, 2, 4, 8]), dtype=rng.choice(["bf16", "fp16", "fp32"]))
    Q, layers = rng.randint(2, 64), rng.randint(1, 8)
    B = _log(rng, 1, 128)
    return dict(kind=kind, B=B, Q=Q, KV=KV, D=D, layers=layers, before=_log(rng, 20, max(20, min(2000, 500000 * 1024 // (B * KV * D * layers) // 2))), dtype="bf16")


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


def _trees(B, Q, width, r):
    """Parents [B, Q] of trees whose nodes come level by level, the first few children of each; every fourth request's tree is smaller."""
    parents = np.full((B, Q), -1, np.int32)
    for b in range(B):
        n = Q if b % 4 else max(1, Q - r.randint(0, Q // 4 + 1))
        at, kids = 0, 0
        for j in range(1, n):
            while kids >= (width if at == 0 else 1 + r.randint(0, width)):
                at, kids = at + 1, 0
            if at >= j:
                at = j - 1
            parents[b, j] = at
            kids += 1
    return parents


def _masks(parents):
    masks = np.zeros(parents.shape, np.uint64)
    masks[:, 0] = 1
    rows = np.arange(len(parents))
    for j in range(1, parents.shape[1]):
        up = parents[:, j]
        masks[:, j] = np.where(up >= 0, masks[rows, np.maximum(up, 0)] | np.uint64(1 << j), np.uint64(0))
    return masks.view(np.int64)


def _parts(cache, KV, D):
    """The pages' code bytes of keys and values [..., pages, KV, 64, D] and their scale bytes [..., pages, KV, 4], as views."""
    n = KV * PAGE * D
    k = cache[..., :n].unflatten(-1, (KV, PAGE, D))
    v = cache[..., n:2 * n].unflatten(-1, (KV, PAGE, D))
    s = cache[..., 2 * n:2 * n + 8 * KV].unflatten(-1, (KV, 2, 4))
    return k, v, s[..., 0, :], s[..., 1, :]


def _pow2(byte):
    """2^(byte - 127) in 32 bits, exactly, for bytes of 1 to 254."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _random_pages(pages, KV, D, gen, layers=1):
    """A cache in use: codes of normal values with a few large ones, scales that differ by block."""
    cache = torch.zeros((layers * pages, page_bytes(KV, D)), dtype=torch.uint8, device=DEV)
    k, v, ks, vs = _parts(cache, KV, D)
    for at in range(0, layers * pages, 4096):
        for x in (k, v):
            y = x[at:at + 4096]
            r = torch.randn(y.shape, device=DEV, generator=gen, dtype=torch.float32).mul_(90.0)
            y.copy_(r.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
    ks.copy_(torch.randint(119, 122, ks.shape, device=DEV, generator=gen, dtype=torch.uint8))
    vs.copy_(torch.randint(118, 123, vs.shape, device=DEV, generator=gen, dtype=torch.uint8))
    return cache.view(layers, pages, -1) if layers > 1 else cache


def _rope_counts(case):
    return _spread(case["B"], case["n_lo"], case["n_hi"]), _spread(case["B"], case["before"] // 3, case["before"])


def _sections(case):
    """How many of the pairs go by each axis."""
    pairs, axes = case["rot"] // 2, case["axes"]
    rest = [pairs // (axes + 1)] * (axes - 1)
    return [pairs - sum(rest)] + rest


def _accept_plan(case):
    """Lengths, parents and the accepted paths [B, Q] of an `accept` case: part of the case, as lengths are."""
    B, Q = case["B"], case["Q"]
    r = np.random.RandomState(B * 7919 + Q)
    lens = _spread(B, case["before"] // 3, case["before"]) + Q
    parents = _trees(B, Q, 3, r)
    path, count = np.full((B, Q), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        at = 0
        for j in range(1, Q):
            if parents[b, j] == at and r.uniform() < 0.6:
                path[b, count[b]] = at = j
                count[b] += 1
    return lens.astype(np.int32), path, count


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    kind, B = case["kind"], case["B"]
    r = np.random.RandomState(seed % (1 << 31))
    if kind == "verify":
        return _prepare_verify(case, gen, r)
    KV, D, dtype = case["KV"], case["D"], DTYPES[case["dtype"]]
    if kind == "accept":
        lens, path, count = _accept_plan(case)
        pages = int((-(-lens.astype(np.int64) // PAGE)).sum()) + 3
        table = _tables(lens, pages, g).to(DEV)
        rc = torch.zeros(pages, dtype=torch.int32, device=DEV)
        rc.index_add_(0, table.clamp(min=0).flatten(), (table >= 0).to(torch.int32).flatten())
        lens = torch.from_numpy(lens).to(DEV)
        cache = _random_pages(pages, KV, D, gen, case["layers"]).view(case["layers"], pages, -1)
        return dict(case=case, cache=cache, table0=table, rc0=rc, lens0=lens, table=table.clone(), rc=rc.clone(), lens=lens.clone(),
                    path=torch.from_numpy(path).to(DEV), count=torch.from_numpy(count).to(DEV))
    if kind == "tree":
        lens = _spread(B, case["lo"], case["hi"])
        pages = max(1, int((-(-lens.astype(np.int64) // PAGE)).sum()))
        q = torch.randn((B, case["Q"], case["H"], D), device=DEV, generator=gen).to(dtype)
        masks = torch.from_numpy(_masks(_trees(B, case["Q"], 4, r))).to(DEV)
        return dict(case=case, q=q, masks=masks, cache=_random_pages(pages, KV, D, gen), table=_tables(lens, pages, g).to(DEV), lens=torch.from_numpy(lens).to(DEV),
                    scale=D ** -0.5, out=torch.empty_like(q), lse=torch.empty(q.shape[:3], dtype=torch.float32, device=DEV))
    new, old = _rope_counts(case)
    lens = new + old
    pages = int((-(-lens.astype(np.int64) // PAGE)).sum()) + 3
    n, H = int(new.sum()), case["H"]
    qkv = torch.randn((n, H + 2 * KV, D), device=DEV, generator=gen)      # a fused projection's rows
    qkv *= torch.exp(0.5 * torch.randn((1, H + 2 * KV, D), device=DEV, generator=gen))
    qkv *= torch.where(torch.rand((n, H + 2 * KV, 1), device=DEV, generator=gen) < 0.01, 20.0, 1.0)
    qkv = qkv.to(dtype)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    span = int(lens.max()) + 64
    half = case["rot"] // 2
    angle = torch.arange(span, dtype=torch.float64)[:, None] * 1e4 ** (-torch.arange(half, dtype=torch.float64) / half)
    positions = None
    if case["tree"]:
        bits = np.unpackbits(_masks(_trees(B, case["n_hi"], 4, r)).view(np.uint8).reshape(B, case["n_hi"], 8), axis=2)
        positions = np.repeat(old, new) + np.maximum(bits.sum(2, dtype=np.int32), 1).reshape(-1) - 1
        positions = np.stack([positions] * case["axes"]) if case["axes"] > 1 else positions
    elif case["axes"] > 1:
        first = np.repeat(old - cu[:-1], new) + np.arange(n)
        positions = np.stack([first] + [r.randint(0, 64, n) for _ in range(case["axes"] - 1)])
    weight = lambda: (1 + 0.2 * torch.randn(D, device=DEV, generator=gen)).to(dtype) if case["norm"] else None  # noqa: E731
    return dict(case=case, q=qkv[:, :H], k=qkv[:, H:H + KV], v=qkv[:, H + KV:], cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float().to(DEV),
                positions=None if positions is None else torch.from_numpy(np.ascontiguousarray(positions, np.int32)).to(DEV), q_weight=weight(), k_weight=weight(), eps=1e-6,
                cu=torch.from_numpy(cu).to(DEV), lens=torch.from_numpy(lens).to(DEV), table=_tables(lens, pages, g).to(DEV), cache=_random_pages(pages, KV, D, gen),
                q_out=torch.empty((n, H, D), dtype=dtype, device=DEV))


def _prepare_verify(case, gen, r):
    """Logits with a few likely tokens a row; drafts from a model that is near the target."""
    B, Q, V = case["B"], case["Q"], case["V"]
    logits = torch.randn((B, Q, V), device=DEV, generator=gen).mul_(1.5)
    likely = torch.randint(0, V, (B, Q, 24), device=DEV, generator=gen)
    logits.scatter_(2, likely, 9.0 + 5.0 * torch.rand((B, Q, 24), device=DEV, generator=gen))
    draft = logits + 0.7 * torch.randn((B, Q, V), device=DEV, generator=gen)
    parents = np.full((B, Q), -1, np.int32)
    parents[:, 1:] = np.arange(Q - 1)
    if case["width"] > 1:
        parents = _trees(B, Q, case["width"], r)
    rank = np.zeros((B, Q), np.int64)
    for j in range(2, Q):
        rank[:, j] = (parents[:, 1:j] == parents[:, j:j + 1]).sum(1)
    up = torch.from_numpy(np.maximum(parents, 0)).long().to(DEV)
    probs = None
    if case["drafts"]:
        draft = draft - draft.logsumexp(-1, keepdim=True)
        tokens = torch.empty((B, Q), dtype=torch.int64, device=DEV)
        for j in range(Q):  # each child drawn from its parent's distribution
            row = draft[torch.arange(B, device=DEV), up[:, j]]
            tokens[:, j] = (row - torch.log(-torch.log(torch.rand((B, V), device=DEV, generator=gen).clamp(1e-20, 1 - 1e-7)))).argmax(-1)
        probs = draft.exp_()
    else:
        best = draft.topk(int(rank.max()) + 1, -1).indices
        tokens = best[torch.arange(B, device=DEV)[:, None], up, torch.from_numpy(rank).to(DEV)]
    temperatures = torch.rand(B, device=DEV, generator=gen) * 0.6 + 0.6
    temperatures[3::4] = 0.0
    return dict(case=case, logits=logits.to(DTYPES[case["dtype"]]), drafts=tokens.to(torch.int32), parents=torch.from_numpy(parents).to(DEV), probs=probs, temperatures=temperatures,
                uniforms=torch.rand((B, Q), device=DEV, generator=gen), tokens=torch.empty((B, Q), dtype=torch.int32, device=DEV),
                path=torch.empty((B, Q), dtype=torch.int32, device=DEV), accepted=torch.empty(B, dtype=torch.int32, device=DEV))


# ------------------------------------------------------------------ rope
def _rotated(x, weight, cos, sin, rot, inter, eps):
    """x [N, heads, D] normalised and rotated, in cos's type; cos, sin [N, rot / 2]."""
    x = x.to(cos.dtype)
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight.to(cos.dtype)
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    cos, sin = cos[:, None], sin[:, None]
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _angles(s, dtype):
    """cos and sin [N, rot / 2] of every new token."""
    c = s["case"]
    half, N = c["rot"] // 2, s["q"].shape[0]
    at = s["positions"]
    if at is None:
        cu = s["cu"].long()
        b = torch.searchsorted(cu, torch.arange(N, device=DEV), right=True) - 1
        at = s["lens"].long()[b] - cu[b + 1] + torch.arange(N, device=DEV)
    at = at.long().reshape(-1, N)
    ends = torch.tensor(_sections(c), device=DEV).cumsum(0)
    axis = torch.searchsorted(ends, torch.arange(half, device=DEV), right=True).clamp(max=at.shape[0] - 1)
    rows = s["cos_sin"][at.T[:, axis], torch.arange(half, device=DEV)], s["cos_sin"][at.T[:, axis], half + torch.arange(half, device=DEV)]
    return rows[0].to(dtype), rows[1].to(dtype)


def _scales(amax, before):
    """The smallest power of two that takes amax to at most 448, as a byte, and no less than the block's byte before."""
    m, e = torch.frexp(amax.double() / 448)  # amax / 448 = m 2^e, m in [0.5, 1)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(amax > 0, e, -126).clamp(-126, 126) + 127
    return torch.maximum(e, before).to(torch.int32)


def _rope(s):
    """The new tokens' rows, then blocks of 16 tokens: the tokens before the new ones, the new ones, and what is behind them."""
    c = s["case"]
    KV, D = c["KV"], c["D"]
    table, lens, cu = s["table"], s["lens"].long(), s["cu"].long()
    N = s["k"].shape[0]
    if N == 0:
        return _rope_out(s, s["q_out"])
    cos, sin = _angles(s, torch.float32)
    q = _rotated(s["q"], s["q_weight"], cos, sin, c["rot"], c["inter"], s["eps"]).to(s["q"].dtype)
    keys = _rotated(s["k"], s["k_weight"], cos, sin, c["rot"], c["inter"], s["eps"])
    first = lens - (cu[1:] - cu[:-1])
    tok = torch.arange(N, device=DEV)
    b = torch.searchsorted(cu, tok, right=True) - 1
    pos = first[b] + tok - cu[b]
    at = torch.nonzero((tok == cu[b]) | (pos % BLOCK == 0)).flatten()  # every touched block once, as (sequence, block)
    b, block = b[at], pos[at] // BLOCK
    pos = block[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)  # [blocks, 16]
    is_new = (pos >= first[b][:, None]) & (pos < lens[b][:, None])
    is_old = pos < first[b][:, None]
    row = (cu[b][:, None] + pos - first[b][:, None]).clamp(0, N - 1)
    page = table[b, block * BLOCK // PAGE].long()
    quarter = block % (PAGE // BLOCK)
    rows = quarter[:, None] * BLOCK + torch.arange(BLOCK, device=DEV)
    for x, codes, scales in ((keys, *_parts(s["cache"], KV, D)[0::2]), (s["v"].float(), *_parts(s["cache"], KV, D)[1::2])):
        x = x[row].transpose(1, 2)  # [blocks, KV, 16, D]
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
    return _rope_out(s, q)


def _rope_out(s, q):
    k, v, ks, vs = _parts(s["cache"], s["case"]["KV"], s["case"]["D"])
    return dict(q=q, k=k.view(torch.float8_e4m3fn), v=v.view(torch.float8_e4m3fn), k_scales=ks.view(torch.float8_e8m0fnu), v_scales=vs.view(torch.float8_e8m0fnu))


# ------------------------------------------------------------------ tree
def _tree(s):
    """softmax(scale q k + mask) v over the cached tokens, and its log-sum-exp."""
    c = s["case"]
    q, table, KV, Q = s["q"].float(), s["table"], c["KV"], c["Q"]
    k, v, ks, vs = (x[table.clamp(min=0).long()] for x in _parts(s["cache"], KV, c["D"]))  # [B, P, KV, ...]

    def wide(x, e):
        x = x.view(torch.float8_e4m3fn).float().unflatten(3, (4, BLOCK)) * _pow2(e)[..., None, None]
        return x.flatten(3, 4).transpose(1, 2).flatten(2, 3)  # [B, KV, P * 64, D]

    k, v = wide(k, ks), wide(v, vs)
    t = torch.arange(table.shape[1] * PAGE, device=DEV)
    base, masks = s["lens"].long() - Q, s["masks"]
    bits = (masks[:, :, None] >> torch.arange(Q, device=DEV)) & 1
    place = base[:, None] + bits.sum(-1) - 1
    draft = t - base[:, None]  # [B, T]
    is_draft = (draft >= 0) & (draft < Q)
    listed_ = bits.gather(2, draft.clamp(0, Q - 1)[:, None].expand(-1, Q, -1)) > 0
    before = t < base[:, None, None]
    if c["window"]:
        before = before & (t > place[:, :, None] - c["window"])
    ok = (before | (is_draft[:, None] & listed_)) & (masks != 0)[:, :, None]  # [B, Q, T]
    z = torch.einsum("bqhgd,bhtd->bhgqt", q.unflatten(2, (KV, c["H"] // KV)), k) * s["scale"]
    z = z.masked_fill(~ok[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    out = torch.einsum("bhgqt,bhtd->bqhgd", e / total.clamp(min=torch.finfo(torch.float32).tiny), v)
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2)  # an empty row: log 0
    return out.flatten(2, 3).to(s["q"].dtype), lse.flatten(2, 3).contiguous()


# ------------------------------------------------------------------ verify
def _verify(s):
    """The walk through all trees at once, node by node: parents come before their children."""
    logits, parents, drafts, u, probs = s["logits"].float(), s["parents"].long(), s["drafts"].long(), s["uniforms"].double(), s["probs"]
    B, Q, V = logits.shape
    greedy = s["temperatures"] == 0
    t = torch.where(greedy, 1.0, s["temperatures"])
    best = logits.argmax(-1)
    e = torch.exp((logits - logits.amax(-1, keepdim=True)) / t[:, None, None])
    p = e / e.sum(-1, keepdim=True, dtype=torch.float64).float()
    b = torch.arange(B, device=DEV)
    at = torch.zeros(B, dtype=torch.int64, device=DEV)
    count, left = at.clone(), torch.ones(B, dtype=torch.float64, device=DEV)
    rest = p[:, 0].clone()
    path = torch.full((B, Q), -1, dtype=torch.int64, device=DEV)
    for j in range(1, Q):
        x = drafts[:, j]
        child = parents[:, j] == at
        have = rest[b, x]
        qx = 1.0 if probs is None else probs[b, at, x].double()
        yes = child & torch.where(greedy, best[b, at] == x, u[:, j] * qx * left < have.double())
        no = child & ~yes
        if probs is None:
            rest[b, x] = torch.where(no, 0.0, have)
            left = torch.where(no, left - have.double(), left)
        else:
            less = (rest - left.float()[:, None] * probs[b, at]).clamp(min=0)
            rest = torch.where(no[:, None], less, rest)
            left = torch.where(no, less.sum(-1, dtype=torch.float64), left)
        path[b, count] = torch.where(yes, j, path[b, count])
        count += yes
        at = torch.where(yes, j, at)
        left = torch.where(yes, 1.0, left)
        rest = torch.where(yes[:, None], p[:, j], rest)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, p[b, at])  # nothing left: from the target's own
    run_ = rest.double().cumsum(-1)
    last = V - 1 - (rest.flip(-1) > 0).to(torch.int8).argmax(-1)
    x = torch.minimum((run_ <= u[:, :1] * run_[:, -1:]).sum(-1), last)
    x = torch.where(greedy, best[b, at], x)
    tokens = torch.where(path >= 0, drafts.gather(1, path.clamp(min=0)), -1)
    tokens[b, count] = x
    return dict(tokens=tokens.to(torch.int32), path=path.to(torch.int32), accepted=count.to(torch.int32))


# ------------------------------------------------------------------ accept
def _keep(cache, table, lens, path, count, KV, D):
    """Accepted nodes move up; returns the new lengths. Blocks of 16 places from the one of base + 1 on."""
    B, Q = path.shape
    base, count = lens.long() - Q, count.long()
    W = -(-(Q + BLOCK) // BLOCK) * BLOCK
    pos = ((base + 1) // BLOCK * BLOCK)[:, None] + torch.arange(W, device=DEV)  # [B, W]
    i = pos - base[:, None]
    lives = i <= count[:, None]
    src = torch.where((i >= 1) & lives, base[:, None] + path.long().gather(1, (i - 1).clamp(0, Q - 1)), pos)
    moved = (src != pos).unflatten(1, (-1, BLOCK)).any(2)  # [B, blocks]
    write = torch.nonzero((lives.unflatten(1, (-1, BLOCK)) & moved[:, :, None]).flatten(1))
    b, w = write[:, 0], write[:, 1]
    width = table.shape[1]
    page = lambda p: table[b, (p // PAGE).clamp(0, width - 1)].long()  # noqa: E731
    src, pos = src[b, w], pos[b, w]
    sp, dp, sr, dr = page(src), page(pos), src % PAGE, pos % PAGE
    which = torch.unique(b * W + w // BLOCK * BLOCK, return_inverse=True)[1]
    for codes, scales in (_parts(cache, KV, D)[0::2], _parts(cache, KV, D)[1::2]):
        byte = scales[:, sp, :, sr // BLOCK].to(torch.int32)  # [layers, rows, KV], or with the rows first
        old = codes[:, sp, :, sr]
        top = torch.zeros((B * W,) + byte.shape[1:], dtype=torch.int32, device=DEV)
        top = top.index_reduce(0, which, byte, "amax")[which]
        less = old.view(torch.float8_e4m3fn).float() * _pow2(127 - (top - byte).clamp(max=126))[..., None]
        codes[:, dp, :, dr] = less.to(torch.float8_e4m3fn).view(torch.uint8)
        scales[:, dp, :, dr // BLOCK] = top.to(torch.uint8)
    return (base + 1 + count).to(torch.int32)


def _trim(table, lens, rc, new):
    gone = (torch.arange(table.shape[1], device=DEV) >= ((new + PAGE - 1) // PAGE)[:, None]) & (table >= 0)
    rc.index_add_(0, torch.where(gone, table, 0).flatten(), -gone.to(torch.int32).flatten())
    table.masked_fill_(gone, -1)
    lens.copy_(new)


def run(s):
    c = s["case"]
    kind = c["kind"]
    if own:
        import nvfp4_compressed_sparse_gb300 as m
    if kind == "rope":
        if not own:
            return _rope(s)
        q = m.kv8_append_rope(s["q"], s["k"], s["v"], s["cos_sin"], s["cu"], s["lens"], s["table"], s["cache"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"],
                              positions=s["positions"], sections=_sections(c) if c["axes"] > 1 else None, interleaved=c["inter"], q_out=s["q_out"])
        return _rope_out(s, q)
    if kind == "tree":
        if not own:
            return _tree(s)
        if "workspace" not in s:  # kept by a program from step to step
            s["workspace"] = torch.empty(m.kv8_decode_tree_workspace_size(c["B"], c["Q"], c["H"], c["KV"], c["D"]), dtype=torch.uint8, device=DEV)
        return m.kv8_decode_tree(s["q"], s["cache"], s["table"], s["lens"], s["masks"], c["KV"], s["scale"], window=c["window"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
    if kind == "verify":
        if not own:
            return _verify(s)
        if "workspace" not in s:
            s["workspace"] = torch.empty(m.spec_verify_workspace_size(c["B"], c["Q"], c["V"]), dtype=torch.uint8, device=DEV)
        tokens, path, accepted = m.spec_verify(s["logits"], s["drafts"], s["parents"], s["uniforms"], temperatures=s["temperatures"], draft_probs=s["probs"], tokens=s["tokens"], path=s["path"],
                                               accepted=s["accepted"], workspace=s["workspace"])
        return dict(tokens=tokens, path=path, accepted=accepted)
    # the tables are put back first, so that every pass finds the step's end
    table, rc, lens = s["table"].copy_(s["table0"]), s["rc"].copy_(s["rc0"]), s["lens"].copy_(s["lens0"])
    if own:
        new = m.kv8_keep(s["cache"], table, lens, s["path"], s["count"], c["KV"], c["D"], layered=True)
        m.kv_pages_trim(table, lens, rc, new)
    else:
        new = _keep(s["cache"], table, lens, s["path"], s["count"], c["KV"], c["D"])
        _trim(table, lens, rc, new)
    k, v, ks, vs = _parts(s["cache"], c["KV"], c["D"])
    return dict(k=k.view(torch.float8_e4m3fn), v=v.view(torch.float8_e4m3fn), k_scales=ks, v_scales=vs, table=table, lens=lens, rc=rc, new=new)


def work(case):
    kind, B = case["kind"], case["B"]
    if kind == "verify":
        size = 4 if case["dtype"] == "fp32" else 2
        rows = B * case["Q"]
        return dict(bytes=float(rows) * case["V"] * size + (4.0 * B * case["V"] if case["drafts"] else 0) + 24.0 * rows, flops=4.0 * rows * case["V"])
    KV, D = case["KV"], case["D"]
    if kind == "rope":
        n = float(_rope_counts(case)[0].sum())
        return dict(bytes=n * D * (4 * case["H"] + 6 * KV) + n * 4 * (case["rot"] + (case["axes"] if case["tree"] or case["axes"] > 1 else 0)), flops=n * D * (8.0 * case["H"] + 10.0 * KV))
    if kind == "tree":
        Q, H, w = case["Q"], case["H"], case["window"]
        lens = _spread(B, case["lo"], case["hi"]).astype(np.int64)
        read = np.minimum(lens, w + Q) if w else lens
        return dict(bytes=float(read.sum()) * KV * (2 * D + 0.5) + B * Q * H * (4.0 * D + 4) + 8.0 * B * Q, flops=4.0 * float(read.sum()) * Q * H * D)
    lens, path, count = _accept_plan(case)
    moved = float((path[:, :] > np.arange(1, case["Q"] + 1)).sum())
    return dict(bytes=4.0 * moved * D * KV * case["layers"] + 8.0 * B * case["Q"], flops=2 * moved * D * KV * case["layers"])


# ------------------------------------------------------------------ 64 bits, written apart
def exact(case, seed):
    if case["kind"] == "rope":
        return _exact_rope(prepare(case, seed))
    if case["kind"] == "tree":
        return _exact_tree(prepare(case, seed))
    if case["kind"] == "verify":
        return _exact_verify(prepare(case, seed))
    return None  # codes that move: bytes, and not idempotent


def _value(byte):
    """E4M3 bytes as 64-bit numbers, from the format: sign, four bits of exponent, three of mantissa."""
    i = torch.arange(256, dtype=torch.float64)
    e, m = torch.div(i % 128, 8, rounding_mode="floor"), i % 8
    table = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e - 10))
    table = torch.where(i >= 128, -table, table)
    table[127] = table[255] = math.nan
    return table.to(byte.device)[byte.long()]


def _exact_tree(s):
    c = s["case"]
    KV, D, Q, G = c["KV"], c["D"], c["Q"], c["H"] // c["KV"]
    table, lens, masks = s["table"].cpu(), s["lens"].cpu().tolist(), s["masks"].cpu().numpy().view(np.uint64)
    out = torch.zeros((c["B"], Q, c["H"], D), dtype=torch.float64, device=DEV)
    lse = torch.full((c["B"], Q, c["H"]), -math.inf, dtype=torch.float64, device=DEV)
    n = KV * PAGE * D
    for b, L in enumerate(lens):
        raw = s["cache"][table[b, :-(-L // PAGE)].long().to(DEV)]
        sc = torch.exp2(raw[:, 2 * n:2 * n + 8 * KV].reshape(-1, KV, 2, 4).double() - 127).repeat_interleave(BLOCK, 3)
        seen = np.zeros((Q, L), bool)
        for j in range(Q):
            nodes = [i for i in range(Q) if int(masks[b, j]) >> i & 1]
            if nodes:
                end = L - Q
                seen[j, max(0, end + len(nodes) - c["window"]) if c["window"] else 0:end] = True
                seen[j, [end + i for i in nodes]] = True
        some = torch.from_numpy(seen.any(1)).to(DEV)
        seen = torch.from_numpy(seen).to(DEV)
        for h in range(KV):
            k = (_value(raw[:, h * PAGE * D:(h + 1) * PAGE * D].reshape(-1, PAGE, D)) * sc[:, h, 0, :, None]).reshape(-1, D)[:L]
            v = (_value(raw[:, n + h * PAGE * D:n + (h + 1) * PAGE * D].reshape(-1, PAGE, D)) * sc[:, h, 1, :, None]).reshape(-1, D)[:L]
            for i in range(h * G, (h + 1) * G):
                z = (s["q"][b, :, i].double() @ k.T * s["scale"])[some].masked_fill(~seen[some], -math.inf)
                lse[b, some, i] = torch.logsumexp(z, 1)
                out[b, some, i] = torch.softmax(z, 1) @ v
    return out, lse


def _nearest(x):
    """The E4M3 number nearest to x (64-bit), ties to the even mantissa, at most 448 in size."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    unit = torch.exp2(e - 3)
    return (torch.round(x / unit) * unit).clamp(-448, 448)


def _exact_rope(s):
    c = s["case"]
    KV, D, rot = c["KV"], c["D"], c["rot"]
    n, cu, lens = KV * PAGE * D, s["cu"].cpu().tolist(), s["lens"].cpu().tolist()
    if sum(-(-(b - a) // BLOCK) + 1 for a, b in zip(cu, cu[1:])) > 6000:
        return None
    N = s["q"].shape[0]
    where = [[L - (cu[b + 1] - cu[b]) + i for b, L in enumerate(lens) for i in range(cu[b + 1] - cu[b])]] if s["positions"] is None else s["positions"].cpu().reshape(-1, N).tolist()
    axis = [a for a, many in enumerate(_sections(c)) for _ in range(many)]
    sheet = s["cos_sin"].double()
    at = torch.tensor(where, device=DEV, dtype=torch.int64).reshape(len(where), N)

    def turned(x, w):
        x = x.double().clone()
        if w is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + s["eps"]) * w.double()
        y = x.clone()
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if c["inter"] else (i, i + rot // 2)
            spot = at[min(axis[i], len(where) - 1)]
            co, si = sheet[spot, i][:, None], sheet[spot, rot // 2 + i][:, None]
            y[:, :, a], y[:, :, b] = x[:, :, a] * co - x[:, :, b] * si, x[:, :, a] * si + x[:, :, b] * co
        return y

    raw, table = s["cache"], s["table"].cpu()
    answer = []
    for which, x in ((0, turned(s["k"], s["k_weight"])), (1, s["v"].double())):
        codes = _value(raw[:, which * n:(which + 1) * n]).reshape(-1, KV, PAGE, D)
        scale = raw[:, 2 * n:2 * n + 8 * KV].reshape(-1, KV, 2, 4)[:, :, which].to(torch.int64).clone()
        for b, L in enumerate(lens):
            start = L - (cu[b + 1] - cu[b])
            spot = start
            while spot < L:
                end = min(L, spot // BLOCK * BLOCK + BLOCK)
                page, lo, quarter = int(table[b, spot // PAGE]), spot % PAGE, spot % PAGE // BLOCK
                y = x[cu[b] + spot - start:cu[b] + end - start].transpose(0, 1)
                top = y.abs().amax((1, 2))
                e = torch.where(top > 0, torch.ceil(torch.log2(top / 448)), -126.0)
                e = torch.where(top > 448 * torch.exp2(e), e + 1, torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e))
                e = e.clamp(-126, 126).long() + 127
                if lo % BLOCK:
                    old = scale[page, :, quarter]
                    e = torch.maximum(e, old)
                    part = codes[page, :, quarter * BLOCK:lo]
                    codes[page, :, quarter * BLOCK:lo] = _nearest(part * torch.exp2((old - e).double())[:, None, None])
                codes[page, :, lo:lo + end - spot] = _nearest(y * torch.exp2(127.0 - e)[:, None, None])
                scale[page, :, quarter] = e
                spot = end
        answer.append((codes, torch.exp2(scale.double() - 127)))
    return dict(q=turned(s["q"], s["q_weight"]), k=answer[0][0], v=answer[1][0], k_scales=answer[0][1], v_scales=answer[1][1])


def _exact_verify(s):
    c = s["case"]
    B, Q, V = c["B"], c["Q"], c["V"]
    if B * Q > 600:
        return None
    parents, drafts, u, hot = (s[k].cpu().numpy() for k in ("parents", "drafts", "uniforms", "temperatures"))
    tokens, path = np.full((B, Q), -1, np.int32), np.full((B, Q), -1, np.int32)
    accepted = np.zeros(B, np.int32)
    for b in range(B):
        at = 0
        while True:
            row = s["logits"][b, at].double()
            if hot[b] == 0:
                word = int(torch.nonzero(row == row.max())[0])
                took = next((j for j in range(at + 1, Q) if parents[b, j] == at and drafts[b, j] == word), None)
            else:
                whole = torch.softmax(row / float(hot[b]), 0)
                p, left, took = whole.clone(), 1.0, None
                for j in range(at + 1, Q):
                    if parents[b, j] != at:
                        continue
                    x = int(drafts[b, j])
                    q = torch.zeros(V, dtype=torch.float64, device=DEV) if s["probs"] is None else s["probs"][b, at].double()
                    if s["probs"] is None:
                        q[x] = 1.0
                    if float(u[b, j]) * float(q[x]) * left < float(p[x]):
                        took = j
                        break
                    if s["probs"] is None:
                        p[x] = 0.0
                    else:
                        p = (p - left * q).clamp(min=0)
                    left = float(p.sum())
                if took is None:
                    p = p if left > 0 else whole
                    run_ = p.cumsum(0)
                    word = int(torch.searchsorted(run_, run_[-1] * float(u[b, 0]), right=True))
                    word = min(word, int(torch.nonzero(p)[-1]))
            if took is None:
                tokens[b, accepted[b]] = word
                break
            path[b, accepted[b]], tokens[b, accepted[b]] = took, drafts[b, took]
            accepted[b] += 1
            at = took
    return dict(tokens=tokens, path=path, accepted=accepted)
