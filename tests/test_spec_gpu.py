"""The speculative step's calls against the 64-bit oracle: tables and moved bytes equal, decisions equal, the rest within rounding."""
import numpy as np
import pytest
import torch

import nvfp4_compressed_sparse_gb300 as m
from oracle import kv8, spec
from tests.kv8_util import DTYPES, Case, dev, f64

pytestmark = pytest.mark.gpu


def tree(rng, Q, width=3, nodes=None):
    """Parents [Q] and masks [Q] (unsigned) of a random tree; -1 and 0 from `nodes` on."""
    parents, masks = np.full(Q, -1, np.int32), np.zeros(Q, np.uint64)
    masks[0] = 1
    for j in range(1, Q if nodes is None else nodes):
        parents[j] = rng.integers(max(0, j - 2 * width), j)
        masks[j] = masks[parents[j]] | np.uint64(1 << j)
    return parents, masks


def trees(rng, B, Q, width=3):
    both = [tree(rng, Q, width, Q if b % 3 else rng.integers(1, Q + 1)) for b in range(B)]
    return np.stack([p for p, _ in both]), np.stack([k for _, k in both])


# ------------------------------------------------------------------ append with norms and rotation
class Rope:
    def __init__(self, old, new, H, Hk, D, dtype, rot, norm=True, axes=1, positions=False, seed=0, spread=2.0):
        self.rng = rng = np.random.default_rng(seed)
        old, new = np.asarray(old), np.asarray(new)
        self.lens, self.cu = (old + new).astype(np.int32), np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.H, self.Hk, self.D, self.rot, self.dtype, self.eps = H, Hk, D, rot, DTYPES[dtype], 1e-5
        need = -(-self.lens // 64)
        self.table = np.full((len(old), max(1, need.max())), -1, np.int32)
        perm, at = rng.permutation(int(need.sum()) + 2), 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.cache = rng.integers(0, 256, (int(need.sum()) + 2, kv8.page_bytes(Hk, D)), dtype=np.uint8)
        before = [self.values(int(old.sum()), Hk, spread) for _ in range(2)]
        kv8.append(self.cache, f64(before[0]), f64(before[1]), np.concatenate([[0], np.cumsum(old)]), old, self.table, Hk, D)
        n = self.n = int(new.sum())
        self.q, self.k, self.v = self.values(n, H, spread), self.values(n, Hk, spread), self.values(n, Hk, spread)
        self.weights = [torch.from_numpy(1 + 0.3 * rng.standard_normal(D)).to(self.dtype) if norm else None for _ in range(2)]
        span = int(self.lens.max()) + 40
        angle = np.arange(span)[:, None] * 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
        self.sheet = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
        self.sections, self.positions = [rot // 2], None
        if axes > 1 or positions:
            cut = np.sort(rng.integers(0, rot // 2 + 1, axes - 1))
            self.sections = [int(x) for x in np.diff(np.concatenate([[0], cut, [rot // 2]]))]
            self.positions = rng.integers(0, span, (axes, n)).astype(np.int32)

    def values(self, n, heads, spread):
        x = self.rng.standard_normal((n, heads, self.D)) * np.exp2(np.round(spread * self.rng.standard_normal((n, heads, 1))))
        return torch.from_numpy(x).to(self.dtype)

    def run(self, inter=False, q=None, k=None, v=None, **kw):
        d = dev(self.cache, torch.uint8)
        put = lambda x: None if x is None else x.to("cuda")  # noqa: E731
        at = self.positions
        if at is not None:
            at = dev(at if len(at) > 1 else at[0])
        out = m.kv8_append_rope(put(self.q) if q is None else q, put(self.k) if k is None else k, put(self.v) if v is None else v,
                                put(torch.from_numpy(self.sheet)), dev(self.cu), dev(self.lens), dev(self.table), d,
                                q_weight=put(self.weights[0]), k_weight=put(self.weights[1]), eps=self.eps, positions=at,
                                sections=self.sections if len(self.sections) > 1 else None, interleaved=inter, **kw)
        torch.cuda.synchronize()
        return out, d.cpu().numpy()

    def turned(self, inter):
        at = self.positions if self.positions is not None else spec.places(self.cu, self.lens, self.n)[None]
        w = [None if x is None else f64(x) for x in self.weights]
        return [spec.rotate(f64(x), y, self.eps, self.sheet, at, self.sections, inter) for x, y in ((self.q, w[0]), (self.k, w[1]))]

    def check(self, out, cache, inter):
        """In fp32 a normalised value is off by at most D / 2 + 8 half steps (the sum of D squares, whose root halves it; the root,
        its inverse and two products), each of the two products of a turn by one more, their sum by one: (D / 2 + 11) 2^-24
        of the products' sizes added. A query is then rounded once to its type, a key once to its code."""
        (q, q_size), (k, k_size) = self.turned(inter)
        off = (self.D / 2 + 11) * 2.0 ** -24
        half = torch.finfo(out.dtype).eps / 2
        tiny = torch.finfo(out.dtype).smallest_normal * half
        got, nan = f64(out), np.isnan(q)
        assert np.array_equal(np.isnan(got), nan)
        assert np.all((np.abs(got - q) <= half * np.abs(q) + (1 + half) * off * q_size + tiny)[~nan])
        # keys: under the smallest scale for them (one that fp32 may see on the other side of a border is allowed), each
        # code within half a step; everything else of the cache as kv8_append leaves it
        want, fed = self.cache.copy(), np.where(np.isnan(k), np.nan, k)
        kv8.append(want, fed, f64(self.v), self.cu, self.lens, self.table, self.Hk, self.D)
        (c0, s0), (c1, s1) = kv8.parts(cache, self.Hk, self.D), kv8.parts(want, self.Hk, self.D)
        assert np.array_equal(c0[:, 1], c1[:, 1]) and np.array_equal(s0[:, :, 1], s1[:, :, 1])
        seen = np.zeros(c0[:, 0].shape[:3], bool)
        at = spec.places(self.cu, self.lens, self.n)
        for b in range(len(self.lens)):
            for t in range(self.cu[b], self.cu[b + 1]):
                page, r = self.table[b, at[t] // 64], at[t] % 64
                s = 2.0 ** (s0[page, :, 0, r // 16].astype(np.float64) - 127)[:, None]
                code = c0[page, 0, :, r]
                bad = np.isnan(k[t])
                assert np.all(code[bad] == 0x7F)
                y = np.where(bad, 0, kv8.e4m3_decode(np.where(bad, 0, code).astype(np.uint8))) * s
                x = np.clip(np.where(bad, 0, k[t]), -448 * s, 448 * s)
                tol = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s) * (1 + 2.0 ** -8) + off * np.where(bad, 0, k_size[t])
                assert np.all(np.abs(y - x) <= tol)
                seen[page, :, r] = True
        same = s0[:, :, 0] == s1[:, :, 0]                # [pages, heads, blocks]
        assert np.all(np.abs(s0[:, :, 0].astype(int) - s1[:, :, 0].astype(int)) <= 1) and (~same).mean() < 0.02
        rows = np.repeat(same, 16, axis=2) & ~seen
        assert np.array_equal(c0[:, 0][rows], c1[:, 0][rows])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("H,Hk,D,rot", [(4, 2, 128, 128), (3, 1, 128, 48), (6, 3, 64, 64), (1, 1, 64, 16), (40, 8, 64, 32)])
def test_rope_matches_the_oracle(H, Hk, D, rot, inter, dtype):
    for norm, axes, positions in ((True, 1, False), (False, 3, True), (True, 1, True), (True, 4, True)):
        c = Rope([0, 15, 16, 40, 5, 63], [1, 1, 20, 33, 0, 2], H, Hk, D, dtype, rot, norm, axes, positions, seed=H + rot)
        c.check(*c.run(inter), inter)


@pytest.mark.parametrize("old,new", [([0], [1]), ([0] * 70, [1] * 70), ([9] * 40, [1, 2, 3, 0] * 10), ([130], [300])])
def test_rope_lengths(old, new):
    c = Rope(old, new, 5, 1, 128, "bf16", 128, seed=len(old))
    c.check(*c.run(), False)


def test_rope_with_a_table_of_ones_appends_as_kv8_append_does():
    """No norm, and angles of zero: the bytes are kv8_append's, and the queries stay."""
    for dtype in ("bf16", "fp16"):
        c = Rope([3, 0, 0, 20], [40, 16, 16, 50], 4, 2, 64, dtype, 64, norm=False, seed=4)
        c.sheet[:, :32], c.sheet[:, 32:] = 1, 0
        c.k[1, 0, :4] = torch.tensor([float("inf"), -float("inf"), 0.0, -0.0])
        c.sheet[:, 32] = 0
        out, cache = c.run()
        d = dev(c.cache, torch.uint8)
        finite = torch.isfinite(c.k).all(-1)
        m.kv8_append(c.k.to("cuda"), c.v.to("cuda"), dev(c.cu), dev(c.lens), dev(c.table), d)
        assert torch.equal(out.cpu(), c.q)
        a, b = (kv8.parts(x, 2, 64) for x in (cache, d.cpu().numpy()))
        assert np.array_equal(a[1], b[1]) and not finite.all()
        page, r = c.table[0, 0], 3 + 1                   # the row with infinities: their partners become NaN (inf x 0)
        a[0][page, 0, 0, r] = b[0][page, 0, 0, r] = 0
        assert np.array_equal(a[0], b[0])


def test_rope_strides_and_in_place():
    """Slices of a fused projection, queries turned where they lie, keys of one row for all heads, positions with a stride."""
    c = Rope([2, 70], [33, 7], 8, 4, 128, "bf16", 64, axes=2, positions=True, seed=6)
    fused = torch.from_numpy(c.rng.standard_normal((40, 16, 128))).to(torch.bfloat16).to("cuda")
    c.q, c.k, c.v = (x.cpu().clone() for x in (fused[:, :8], fused[:, 8:12], fused[:, 12:]))
    rest = fused[:, 8:].clone()
    out, cache = c.run(q=fused[:, :8], k=fused[:, 8:12], v=fused[:, 12:], q_out=fused[:, :8])
    assert out.data_ptr() == fused.data_ptr() and torch.equal(fused[:, 8:], rest)
    c.check(out, cache, False)
    one = torch.from_numpy(c.rng.standard_normal((40, 1, 128))).to(torch.bfloat16).to("cuda").expand(40, 4, 128)
    c.k = one.cpu().clone()
    wide = torch.empty((40, 8, 2, 128), dtype=torch.bfloat16, device="cuda")
    out, cache = c.run(k=one, q_out=wide[:, :, 1])
    c.check(out, cache, False)


def test_rope_leaves_out_and_counts_bad_data():
    old, new = [10, 0, 5, 64, 3, 60], [20, 8, 3, 70, 4, 30]
    c = Rope(old, new, 2, 2, 128, "fp16", 128, positions=True, seed=7)
    c.lens[1] = 5                      # eight new tokens would begin at -3
    c.table[2, 0] = -1
    c.table[3, 2] = len(c.cache)       # positions 128 .. 133
    c.positions[0, [3, 30, 100]] = [-1, len(c.sheet), 1 << 30]
    status = dev(np.zeros(4))
    q_out = torch.full((c.n, 2, 128), 7.0, dtype=torch.float16, device="cuda")
    out, cache = c.run(dev_status=status, q_out=q_out)
    want = c.cache.copy()
    (q, _), (k, _) = c.turned(False)
    bad = kv8.append(want, k, f64(c.v), c.cu, c.lens, c.table, 2, 128)
    assert status.tolist() == [3, bad[0], 0, bad[1]] and bad == [2, 1]
    rows = np.arange(c.n)
    left_out = (rows >= c.cu[1]) & (rows < c.cu[2])
    assert np.all(f64(out)[left_out] == 7) and np.all(np.isnan(f64(out)[[3, 30, 100]]))
    fine = ~left_out & ~np.isin(rows, [3, 30, 100])
    assert np.allclose(f64(out)[fine], q[fine], rtol=2.0 ** -10, atol=1e-4)
    codes = kv8.parts(cache, 2, 128)[0]
    assert np.all(codes[c.table[0, 0], 0, :, 10 + 3] == 0x7F)
    untouched = np.setdiff1d(np.arange(len(c.cache)), c.table[(c.table >= 0) & (c.table < len(c.cache))])
    assert np.array_equal(cache[untouched], c.cache[untouched])


def test_rope_leaves_rows_of_no_request_alone():
    """A padded batch: tokens before the first request, behind the last one, and of requests without new tokens."""
    c = Rope([5, 7, 0, 64], [3, 0, 20, 2], 3, 1, 64, "bf16", 64, seed=9)
    pad = lambda x: torch.cat([x[:2], x, x[:7]])  # noqa: E731
    c.q, c.k, c.v = pad(c.q), pad(c.k), pad(c.v)
    c.cu, c.n = c.cu + 2, c.n + 9
    q_out = torch.full((c.n, 3, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out, cache = c.run(q_out=q_out)
    assert np.all(f64(out)[:2] == 7) and np.all(f64(out)[-7:] == 7)
    (q, _), _ = c.turned(False)
    c.n, c.cu = c.n - 9, c.cu - 2
    c.q, c.k, c.v = c.q[2:-7], c.k[2:-7], c.v[2:-7]
    c.check(out[2:-7], cache, False)
    assert not np.array_equal(cache, c.cache) and q.shape == out.shape


def test_rope_refuses_rows_that_overlap():
    """Results of all heads, or tokens, in one place; the queries' own memory in another order. Axes of one entry have any stride."""
    c = Rope([2], [6], 6, 2, 128, "bf16", 128, seed=11)
    q = c.q.to("cuda")
    room = torch.zeros((6, 6, 128), dtype=torch.bfloat16, device="cuda")
    for out in (room[:, :1].expand(6, 6, 128), room[:1].expand(6, 6, 128), room.view(-1).as_strided((6, 6, 128), (64, 768, 1)), q.transpose(0, 1)):
        with pytest.raises(m.NvFp4MlaError):
            c.run(q=q, q_out=out)
    assert torch.equal(q.cpu(), c.q) and not room.any()
    out, cache = c.run(q=q, q_out=room.transpose(0, 1))
    c.check(out, cache, False)
    one = Rope([2], [1], 6, 2, 128, "bf16", 128, seed=12)
    out, cache = one.run(q_out=room.view(-1).as_strided((1, 6, 128), (8, 128, 1)))
    one.check(out, cache, False)


def test_rope_table_at_any_word():
    """Cosines and sines that do not begin at 16 bytes, and axes that part within four pairs."""
    c = Rope([2, 70], [33, 7], 8, 4, 128, "bf16", 96, axes=3, positions=True, seed=10)
    c.sections = [3, 10, 35]
    want = c.run()
    c.check(*want, False)
    room = torch.zeros(c.sheet.size + 3, device="cuda")
    sheet = room[3:].view(*c.sheet.shape)
    sheet.copy_(torch.from_numpy(c.sheet))
    d = dev(c.cache, torch.uint8)
    out = m.kv8_append_rope(*(x.to("cuda") for x in (c.q, c.k, c.v)), sheet, dev(c.cu), dev(c.lens), dev(c.table), d, q_weight=c.weights[0].to("cuda"),
                            k_weight=c.weights[1].to("cuda"), eps=c.eps, positions=dev(c.positions), sections=c.sections)
    assert torch.equal(out, want[0]) and np.array_equal(d.cpu().numpy(), want[1])


def test_rope_special_values():
    """Zeros, infinities, NaN and the largest numbers in queries and keys, with and without norms."""
    for norm in (False, True):
        c = Rope([0, 5], [20, 13], 2, 1, 64, "bf16", 32, norm=norm, seed=8)
        big = torch.finfo(torch.bfloat16).max
        for x in (c.q, c.k):
            x[1] = 0
            x[2, 0, 40] = float("nan")          # behind the turned dims
            x[3, 0, 3] = float("inf")
            x[4, 0, :] = 1e-20
        if not norm:
            c.k[6, 0, 50] = big
        with np.errstate(over="ignore"):
            (q, _), (k, _) = c.turned(False)
        out, cache = c.run()
        assert np.array_equal(np.isnan(f64(out)), np.isnan(q)) and np.all(f64(out)[1] == 0)
        codes, scales = kv8.parts(cache, 1, 64)
        page = c.table[0, 0]
        for t in range(7):
            assert np.array_equal((codes[page, 0, 0, t] & 0x7F) == 0x7F, np.isnan(k[t, 0]))
        if not norm:
            assert scales[page, 0, 0, 0] == kv8.scale_byte(float(big)) and (codes[page, 0, 0, 3, 3] & 0x7F) == 0x7E


# ------------------------------------------------------------------ tree attention
def check_tree(out, lse, ref, adds, what=""):
    """Outputs against the oracle's.

    A score is a sum of D products in fp32, off by at most (D + 8) 2^-24 of reach; a query's elements are held to 2^-17 of the row's
    largest: 2^-17 of span. A weight is off by that, by the exponential's 2^-21, and by its rounding to fp16: half a step, 2^-12, or,
    below 2^-14, half of 2^-24. The reference of a column's products is a power of two of which the largest product is more than
    half, and what is at the reference is held as 2^9: so the largest is held above 2^8, of which 2^-25 is less than 2^-33. The sum
    that divides is one of unrounded weights; both sums are made of `adds` additions in 32 bits, each off by at most a step of what
    it has reached. The output is rounded once to its type; one that the type does not hold becomes an infinity."""
    r_out, r_lse, mass, reach, spread, span = ref
    dz = (r_out.shape[-1] + 8) * 2.0 ** -24 * reach + 2.0 ** -17 * span
    dw = 2 * (dz + 2.0 ** -21) + 2.0 ** -12 + adds * 2.0 ** -23
    half = torch.finfo(out.dtype).eps / 2
    tiny = torch.finfo(out.dtype).smallest_normal * half
    got, got_lse = f64(out), f64(lse)
    nan = np.isnan(r_out)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN in other places"
    tol = half * np.abs(r_out) + (1 + half) * (dw[..., None] * mass + 2.0 ** -33 * spread) + tiny
    most = torch.finfo(out.dtype).max * (1 + half)           # what is nearer to it than to the largest number
    with np.errstate(invalid="ignore"):
        got = np.where((got == np.copysign(np.inf, r_out)) & (np.abs(r_out) + tol >= most), r_out, got)
        assert not np.any((np.abs(r_out) - tol > most) & (got != r_out)), f"{what}: not an infinity"
    worst = np.nanmax(np.where(nan, 0, np.abs(got - r_out) / tol)) if got.size else 0
    assert worst <= 1, f"{what}: out off by {worst:.2f} of the bound"
    assert np.array_equal(np.isnan(got_lse), np.isnan(r_lse)), f"{what}: NaN lse in other places"
    empty = np.isneginf(r_lse)
    assert np.array_equal(np.isneginf(got_lse), empty), f"{what}: empty rows differ"
    fine = ~empty & ~np.isnan(r_lse)
    tol = (dz + 2.0 ** -21 + adds * 2.0 ** -23 + 2.0 ** -22 * np.maximum(1, np.abs(np.where(fine, r_lse, 0))))[fine]
    assert np.all(np.abs(got_lse[fine] - r_lse[fine]) <= tol), f"{what}: lse"


def run_tree(c, masks, window=0, cache=None, q=None, **kw):
    return m.kv8_decode_tree(c.q if q is None else q, dev(c.cache if cache is None else cache, torch.uint8), dev(c.table), dev(c.lens),
                             dev(masks.view(np.int64), torch.int64), c.Hk, c.scale, window=window, **kw)


def tree_reference(c, masks, window=0, cache=None, q=None):
    return spec.decode_tree(f64(c.q if q is None else q), c.cache if cache is None else cache, c.table, c.lens, masks, c.Hk, c.scale, window)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("Hk,G,D,Q", [(1, 1, 128, 1), (2, 4, 128, 8), (1, 8, 64, 33), (2, 5, 64, 64), (1, 16, 128, 64), (3, 2, 64, 7), (1, 128, 128, 3)])
def test_tree_matches_the_oracle(Hk, G, D, Q, dtype):
    rng = np.random.default_rng(Q + G)
    lens = [Q, Q + 1, Q + 15, Q + 63, 64, 128, 129 + Q, 500, 700][:9 if Q * G < 200 else 6]
    lens = [max(x, Q) for x in lens]
    c = Case(lens, Hk, D, dtype, Q, G, seed=Q)
    _, masks = trees(rng, len(lens), Q)
    check_tree(*run_tree(c, masks), tree_reference(c, masks), 1500)


@pytest.mark.parametrize("D", [64, 128])
def test_tree_windows(D):
    rng = np.random.default_rng(1)
    c = Case([20, 64, 300, 470, 1000], 2, D, "bf16", 20, 3, seed=2)
    _, masks = trees(rng, 5, 20)
    for window in (20, 64, 100, 257, 999, 5000):
        check_tree(*run_tree(c, masks, window), tree_reference(c, masks, window), 2500, f"window {window}")


def test_tree_of_a_chain_is_kv8_decode():
    """Each node the child of the one before: what kv8_decode gives, within both bounds."""
    c = Case([4, 100, 517], 2, 128, "bf16", 4, 4, seed=3)
    masks = np.repeat(np.array([[1, 3, 7, 15]], np.uint64), 3, 0)
    for window in (0, 100):
        ref = tree_reference(c, masks, window)
        want = c.reference(window)
        assert all(np.array_equal(a, b) for a, b in zip(ref[:2], want[:2]))
        check_tree(*run_tree(c, masks, window), ref, 1500)


@pytest.mark.parametrize("D", [64, 128])
def test_tree_weights_just_above_a_power_of_two(D):
    """Keys that are all alike, so that all weights of a column round the same way and nothing averages out. Half a step of an fp16 is
    2^-11 of a weight just above a power of two; that and, as small as the rest of check_tree's bound is here, little else is what
    an output may be off by beside its own rounding. Some come to more than 2^-12 would allow: the bound is not too wide."""
    Hk, Q, n = 1, 64, 200
    k, v = np.zeros((n, Hk, D)), np.tile(1 + np.arange(D) % 8 / 8, (n, Hk, 1))
    k[:, :, 0] = 1
    cache, table, lens = np.zeros((4, kv8.page_bytes(Hk, D)), np.uint8), np.arange(4, dtype=np.int32)[None], np.array([n], np.int32)
    kv8.append(cache, k, v, [0, n], lens, table, Hk, D)
    q = torch.zeros((1, Q, 2, D), dtype=torch.float16)
    q[..., 0] = 1 + torch.arange(2 * Q).view(1, Q, 2) / 1024
    masks = (np.uint64(1) << np.arange(Q, dtype=np.uint64))[None]
    half, beyond = 2.0 ** -11, False
    for s in (0.0, 3e-4, 6.7e-4, 6.9e-4):                # weights of 2^(8 + s + c / 1024), c = 0 .. 127
        scale = float(np.log(2) * (1 + s))
        out, lse = m.kv8_decode_tree(q.to("cuda"), dev(cache, torch.uint8), dev(table), dev(lens), dev(masks.view(np.int64), torch.int64), Hk, scale)
        r, _, mass, reach, _, span = spec.decode_tree(f64(q), cache, table, lens, masks, Hk, scale)
        dz = (D + 8) * 2.0 ** -24 * reach + 2.0 ** -17 * span
        rest = (2 * (dz + 2.0 ** -21) + n * 2.0 ** -23)[..., None]
        off = np.abs(f64(out) - r)
        assert np.all(off <= half * np.abs(r) + (1 + half) * (2.0 ** -11 + rest) * mass)
        beyond |= bool(np.any(off > half * np.abs(r) + (1 + half) * (2.0 ** -12 + rest) * mass))
        assert np.all(np.isfinite(f64(lse)))
    assert beyond


def test_tree_masks_of_any_kind():
    """No node, only bits behind Q, only others' bits, sequences shorter than the tree and empty ones."""
    rng = np.random.default_rng(5)
    c = Case([0, 3, 9, 40, 200], 1, 64, "fp16", 9, 2, seed=5)
    masks = rng.integers(0, 1 << 9, (5, 9)).astype(np.uint64)
    masks[:, 2] = 0
    masks[:, 5] = 1 << 20
    masks[:, 7] = 1 << 3
    masks[3] = 0
    for window in (0, 30):
        check_tree(*run_tree(c, masks, window), tree_reference(c, masks, window), 1000)


def test_tree_nan_reaches_those_that_attend_to_it():
    """NaN codes in keys and values: of the text, of drafts that some nodes attend to, of padding that none does, and behind the end."""
    rng = np.random.default_rng(6)
    for D in (64, 128):
        c = Case([150, 170], 1, D, "bf16", 12, 2, seed=6)
        _, masks = trees(rng, 2, 12)
        masks[:, 9:] = 0
        for where, which in (((0, 20), 0), ((0, 60), 1), ((1, 170 - 12 + 3), 0), ((1, 170 - 12 + 4), 1), ((0, 150 - 12 + 7), 1), ((0, 149), 0), ((1, 169), 1)):
            cache = c.cache.copy()
            b, t = where
            kv8.parts(cache, 1, D)[0][c.table[b, t // 64], which, 0, t % 64, [0, 5, D - 1]] = [0x7F, 0xFF, 0x7F]
            check_tree(*run_tree(c, masks, cache=cache), tree_reference(c, masks, cache=cache), 500, f"{where} {which}")


def test_tree_queries_with_nan_and_infinities():
    c = Case([90, 200], 1, 128, "fp16", 6, 3, seed=7)
    _, masks = trees(np.random.default_rng(7), 2, 6)
    masks[:] = np.maximum(masks, 1)
    q = c.q.clone()
    q[0, 1, 2, 5], q[1, 4, 0, 100], q[1, 0, 1] = float("inf"), float("nan"), 0.0
    got, lse = run_tree(c, masks, q=q)
    want = f64(q)
    want[0, 1, 2] = want[1, 4, 0] = np.nan
    check_tree(got, lse, tree_reference(c, masks, q=torch.from_numpy(want).to(torch.float16)), 500)


def test_tree_wide_scores_and_scales():
    """Scores of hundreds, and value blocks whose scales lie far apart: weights far below the largest count by their scale."""
    for dtype, D in (("bf16", 128), ("fp16", 64)):
        rng = np.random.default_rng(8)
        c = Case([400, 260], 1, D, dtype, 5, 4, seed=8)
        scales = kv8.parts(c.cache, 1, D)[1]
        scales[:, :, 1] = rng.integers(100, 150, scales[:, :, 1].shape)
        scales[:, :, 0] += rng.integers(0, 4, scales[:, :, 0].shape).astype(np.uint8)
        _, masks = trees(rng, 2, 5)
        check_tree(*run_tree(c, masks), tree_reference(c, masks), 1000)
        scales[:, :, 1] = rng.choice([30, 127, 200], scales[:, :, 1].shape)
        q = c.q * 0.01
        check_tree(*run_tree(c, masks, q=q), tree_reference(c, masks, q=q), 1000)


def test_tree_blocks_that_hold_anything():
    """Codes and scale bytes of every value where nothing is attended to (behind the end, before the window), and blocks with the
    smallest scale byte, 0, among those that are attended to in part."""
    for D, window in ((64, 0), (128, 40)):
        rng = np.random.default_rng(17)
        c = Case([70, 200, 131, 64 + 16], 2, D, "bf16", 12, 3, seed=17)
        _, masks = trees(rng, 4, 12)
        codes, scales = kv8.parts(c.cache, 2, D)
        for b, n in enumerate(c.lens):
            first = max(0, n - 12 + 1 - window) if window else 0
            for t in range(c.table.shape[1] * 64):
                page = c.table[b, t // 64]
                if page < 0 or first <= t < n:
                    continue
                codes[page, :, :, t % 64] = rng.integers(0, 256, codes[page, :, :, 0].shape)
                if t % 16 == 0 and (t >= n or t + 16 <= first):
                    scales[page, :, :, t % 64 // 16] = rng.choice([0, 1, 120, 254, 255], scales[page, :, :, 0].shape)
            t = n - 1
            scales[c.table[b, t // 64], 0, 0, t % 64 // 16] = 0
            scales[c.table[b, t // 64], 1, 1, t % 64 // 16] = 0
        check_tree(*run_tree(c, masks, window), tree_reference(c, masks, window), 500, f"{D}")


def test_tree_bad_pages_are_left_out_and_counted():
    c = Case([64 * 5 + 3, 64 * 4, 100], 2, 64, "bf16", 6, 2, seed=9)
    _, masks = trees(np.random.default_rng(9), 3, 6)
    c.table[0, 1], c.table[0, 3], c.table[1, 3] = -1, len(c.cache), -7
    status = dev(np.zeros(4))
    check_tree(*run_tree(c, masks, dev_status=status), tree_reference(c, masks), 1000)
    assert status.tolist() == [0, 3, 0, 0]
    c.lens[2] = 64 * 9                                   # longer than the table's row: six columns
    status.zero_()
    check_tree(*run_tree(c, masks, dev_status=status), tree_reference(c, masks), 1000)
    assert status.tolist()[1] == 3 + (9 - 2)             # four entries of the row are -1, three columns are behind it


@pytest.mark.parametrize("ctas", [1, 2, 3, 7, 40])
def test_tree_cut_in_any_way(ctas):
    """The work over few CTAs, whose parts of a request are joined."""
    c = Case([30, 900, 2000, 16, 131], 2, 64, "bf16", 16, 4, seed=10)
    _, masks = trees(np.random.default_rng(10), 5, 16)
    ref = tree_reference(c, masks)
    check_tree(*run_tree(c, masks, max_ctas=ctas), ref, 4000)


def test_tree_strided_queries_other_stream_and_graph():
    c = Case([70, 300], 2, 128, "bf16", 10, 2, seed=11)
    _, masks = trees(np.random.default_rng(11), 2, 10)
    ref = tree_reference(c, masks)
    fused = torch.zeros((2, 10, 9, 128), dtype=torch.bfloat16, device="cuda")
    fused[:, :, 3:7] = c.q
    check_tree(*run_tree(c, masks, q=fused[:, :, 3:7]), ref, 1000)
    heads_first = c.q.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
    check_tree(*run_tree(c, masks, q=heads_first), ref, 1000)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run_tree(c, masks, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check_tree(*got, ref, 1000)
    ws = torch.randint(0, 256, (m.kv8_decode_tree_workspace_size(2, 10, 4, 2, 128),), dtype=torch.uint8, device="cuda")
    args = dev(c.cache, torch.uint8), dev(c.table), dev(c.lens), dev(masks.view(np.int64), torch.int64)
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:3], device="cuda")
    run = lambda: m.kv8_decode_tree(c.q, *args, 2, c.scale, out=out, lse=lse, workspace=ws)  # noqa: E731
    run()
    graphs = []
    for _ in range(2):                                   # two graphs that share a workspace, in order
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for g in graphs + graphs[::-1]:
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        check_tree(out, lse, ref, 1000)


def test_tree_results_are_the_same_on_every_run():
    c = Case([3000, 700, 64], 2, 128, "bf16", 24, 4, seed=12)
    _, masks = trees(np.random.default_rng(12), 3, 24)
    a = run_tree(c, masks)
    for _ in range(5):
        b = run_tree(c, masks)
        assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("Hk,G,D,Q", [(1, 128, 64, 64), (256, 1, 64, 2), (256, 2, 128, 1)])
def test_tree_largest_sizes(Hk, G, D, Q):
    """64 column tiles of one head; as many heads as a page may have."""
    rng = np.random.default_rng(13)
    c = Case([Q + 1, 70 + Q], Hk, D, "bf16", Q, G, seed=13)
    _, masks = trees(rng, 2, Q)
    check_tree(*run_tree(c, masks), tree_reference(c, masks), 500)


def test_tree_waits_are_bounded_and_the_next_calls_are_right():
    """A step whose tiles never come (a testing flag) gives up after its limit, says so, and leaves workspace
    and device fit for the next step, a replay of a captured one over the same workspace included."""
    c = Case([3000, 200], 2, 64, "bf16", 6, 2, seed=14)
    _, masks = trees(np.random.default_rng(14), 2, 6)
    ref = tree_reference(c, masks)
    ws = torch.zeros(m.kv8_decode_tree_workspace_size(2, 6, 4, 2, 64), dtype=torch.uint8, device="cuda")
    args = (c.q, dev(c.cache, torch.uint8), dev(c.table), dev(c.lens), dev(masks.view(np.int64), torch.int64), 2, c.scale)
    out, lse = m.kv8_decode_tree(*args, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.kv8_decode_tree(*args, out=out, lse=lse, workspace=ws)
    status = dev(np.zeros(4))
    m.kv8_decode_tree(*args, workspace=ws, dev_status=status, test_timeout=True)
    torch.cuda.synchronize()
    assert status[2] > 0 and status[[0, 1, 3]].tolist() == [0, 0, 0]
    for _ in range(2):
        out.fill_(7)
        g.replay()
        check_tree(out, lse, ref, 1500)
    check_tree(*m.kv8_decode_tree(*args, workspace=ws), ref, 1500)


def test_tree_two_calls_at_once():
    """On two streams, each with its own workspace: what each gives alone."""
    cases = [Case([2500, 300, 64], 2, 128, "bf16", 12, 4, seed=15), Case([900, 1800], 1, 64, "fp16", 30, 4, seed=16)]
    masks = [trees(np.random.default_rng(i), len(c.lens), c.q.shape[1])[1] for i, c in enumerate(cases)]
    args = [(c.q, dev(c.cache, torch.uint8), dev(c.table), dev(c.lens), dev(k.view(np.int64), torch.int64), c.Hk, c.scale) for c, k in zip(cases, masks)]
    want = [m.kv8_decode_tree(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    for _ in range(10):
        got = [m.kv8_decode_tree(*a, stream=s) for a, s in zip(args, streams)]
        torch.cuda.synchronize()
        for (x, y), (w, z) in zip(got, want):
            assert torch.equal(x.view(torch.int16), w.view(torch.int16)) and torch.equal(y, z)


# ------------------------------------------------------------------ verification
def verify_case(rng, B, Q, V, dtype, probs, width=2, chain=False):
    logits = rng.standard_normal((B, Q, V)) * 1.5
    for _ in range(6):
        logits[np.arange(B)[:, None], np.arange(Q)[None], rng.integers(0, V, (B, Q))] += 5 * rng.random((B, Q))
    logits = torch.from_numpy(logits).to(dtype)
    parents = np.tile(np.arange(-1, Q - 1, dtype=np.int32), (B, 1)) if chain else trees(rng, B, Q, width)[0]
    near = f64(logits) + 0.7 * rng.standard_normal((B, Q, V))
    e = np.exp(near - near.max(-1, keepdims=True))
    e /= e.sum(-1, keepdims=True)
    drafts = np.zeros((B, Q), np.int32)
    for b in range(B):
        for j in range(Q):
            row = e[b, max(0, parents[b, j])]
            drafts[b, j] = rng.choice(V, p=row) if probs else np.argsort(-row)[rng.integers(0, min(V, 4))]
    hot = np.where(rng.random(B) < 0.25, 0, rng.uniform(0.4, 1.5, B)).astype(np.float32)
    return dict(logits=logits, drafts=drafts, parents=parents, uniforms=rng.random((B, Q)).astype(np.float32), temperatures=hot,
                draft_probs=e.astype(np.float32) if probs else None)


def run_verify(c, **kw):
    args = {k: None if x is None else (x if isinstance(x, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(x))).to("cuda") for k, x in c.items()}
    status = dev(np.zeros(4))
    tokens, path, accepted = m.spec_verify(**args, dev_status=status, **kw)
    return tokens.cpu().numpy(), path.cpu().numpy(), accepted.cpu().numpy(), status.tolist()


def check_verify(c, **kw):
    """Equal, but for requests that come within 2^-20 of deciding otherwise: the fp32 exponentials' error, 2^-22 each, and their
    sums' with it (a derived bound: a probability is a quotient of two such)."""
    got = run_verify(c, **kw)
    with np.errstate(over="ignore"):
        want = spec.verify(f64(c["logits"]), *(c[k] for k in ("drafts", "parents", "uniforms", "temperatures", "draft_probs")))
    sure = want[4] > 2.0 ** -20
    assert sure.mean() >= 0.9
    for a, b in zip(got[:3], want[:3]):
        assert np.array_equal(a[sure], b[sure])
    assert got[3] == [want[3], 0, 0, 0]
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("B,Q,V", [(1, 1, 7), (3, 5, 1), (9, 6, 1000), (5, 12, 1025), (4, 33, 3001), (2, 64, 5000), (70, 2, 2047)])
def test_verify_matches_the_oracle(B, Q, V, probs, dtype):
    rng = np.random.default_rng(B * Q + V)
    for chain in (True, False):
        check_verify(verify_case(rng, B, Q, V, {**DTYPES, "fp32": torch.float32}[dtype], probs, chain=chain))


def test_verify_many_siblings():
    """A node with 63 children, most of them refused, some the same token twice."""
    rng = np.random.default_rng(20)
    for probs in (False, True):
        c = verify_case(rng, 12, 64, 400, torch.float32, probs)
        c["parents"][:, 1:] = 0
        c["drafts"][:, 1:] = rng.integers(0, 400, (12, 63))
        c["drafts"][:, 30] = c["drafts"][:, 3]
        c["temperatures"][:] = 1
        check_verify(c)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_verify_row_alignments(dtype):
    """Rows that begin at every offset inside of 16 bytes, between others' values that may not be read."""
    rng = np.random.default_rng(21)
    for V, stride in ((1030, 1033), (2048, 2049), (5, 7), (1023, 1031)):
        c = verify_case(rng, 5, 8, V, dtype, True)
        rows = torch.full((5 * 8 * stride + 8,), float("nan"), dtype=dtype, device="cuda")
        probs = torch.full((5 * 8 * stride + 8,), 1e9, dtype=torch.float32, device="cuda")
        a, p = (x[3:3 + 40 * stride].view(5, 8, stride)[:, :, :V] for x in (rows, probs))
        a.copy_(c["logits"])
        p.copy_(torch.from_numpy(c["draft_probs"]))
        want = run_verify(c)
        got = run_verify({**c, "logits": a, "draft_probs": p})
        assert all(np.array_equal(x, y) for x, y in zip(got, want))
        check_verify(c)


def test_verify_special_logits():
    """-inf, +inf and NaN logits, rows of nothing but -inf, ties of the largest."""
    rng = np.random.default_rng(22)
    for probs in (False, True):
        c = verify_case(rng, 10, 4, 2100, torch.float32, probs, chain=True)
        c["temperatures"][:] = [1, 1, 1, 0, 0, 0, 1, 0, 0.5, 1]
        x = c["logits"]
        x[0, 0, 100:] = -float("inf")
        x[1, :, ::3] = float("nan")
        x[2, 0, [5, 9, 2000]] = float("inf")
        x[3, 0, [7, 1500]] = 50.0                        # a tie: the smaller
        x[4, 0] = -float("inf")
        x[5, 0] = float("nan")
        x[6, 0] = -float("inf")
        x[7, 0, 3] = float("inf")
        c["drafts"][3, 1], c["drafts"][2, 1] = 7, 9
        got = check_verify(c)
        assert got[0][3, 0] == 7 and got[2][3] >= 1 and got[0][4, 0] == got[0][5, 0] == got[0][6, 0] == -1 and got[3][0] == 3


def test_verify_uniforms_at_the_ends():
    rng = np.random.default_rng(23)
    c = verify_case(rng, 6, 3, 1500, torch.float32, False, chain=True)
    c["temperatures"][:] = 1
    c["logits"][:, :, 1400:] = -float("inf")
    c["drafts"][:, 1:] = 1450                            # no probability: refused even by 0
    c["uniforms"][:, 1:] = [[0, 0]] * 6
    c["uniforms"][:, 0] = [0, -1, 1, 2, float("nan"), 1 - 2.0 ** -24]
    got = run_verify(c)
    assert np.all(got[2] == 0) and list(got[0][:2, 0]) == [0, 0] and np.all(got[0][2:5, 0] == 1399)
    c["drafts"][:, 1:] = 3
    c["uniforms"][:, 1] = [0, -5, 1, 3, float("nan"), 0]
    assert list(np.minimum(run_verify(c)[2], 1)) == [1, 1, 0, 0, 0, 1]


def test_verify_uniforms_of_one_and_more_refuse():
    """Whatever the probabilities are, and what is left then is not below 0."""
    rng = np.random.default_rng(27)
    for probs in (False, True):
        c = verify_case(rng, 6, 4, 300, torch.float32, probs)
        c["parents"][:] = [-1, 0, 0, 0]
        c["temperatures"][:] = 1
        c["logits"][:, 0, 200:] = -float("inf")
        c["drafts"][:, 1:] = [[3, 5, 250]] * 6               # 250: no probability
        c["logits"][:, 0, [3, 5]] = 30.0                     # what is left behind them is near 0
        c["uniforms"][:, 1:] = [[1, 2, 0.5], [float("nan"), 7, 0.9], [1, 1, 1], [float("inf"), 1, 0], [1.5, 1.5, 0.25], [2, 2, 0.75]]
        if probs:
            c["draft_probs"][:, 0, 3] = 1e-6                 # far less than the target's
        got = run_verify(c)
        assert np.all(got[2] == 0) and np.all(got[0][:, 0] < 200)


@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_verify_siblings_of_tokens_far_below(dtype, probs):
    """Drafts whose logit is the type's lowest number have no probability, and their refusal takes nothing from what is left for
    the siblings behind them."""
    rng = np.random.default_rng(70)
    dt = {**DTYPES, "fp32": torch.float32}[dtype]
    c = verify_case(rng, 12, 6, 600, dt, probs)
    c["parents"][:] = [-1, 0, 0, 0, 0, 0]
    c["logits"][:, 0, 400:] = torch.finfo(dt).min
    likely = np.argsort(-f64(c["logits"])[:, 0], axis=1)
    c["drafts"][:, [1, 4]] = rng.integers(400, 600, (12, 2))
    c["drafts"][:, [2, 3, 5]] = likely[:, [2, 3, 1]]
    c["temperatures"][:] = np.repeat([0.6, 1, 1.4], 4)
    c["uniforms"][:, 1:] = rng.uniform(0.6, 0.99, (12, 5))
    if probs:
        np.put_along_axis(c["draft_probs"][:, 0], c["drafts"][:, 1:], np.float32(0.05), 1)
    got = check_verify(c)
    assert np.all(got[2] <= 1) and not np.isin(got[1][:, 0], [1, 4]).any() and (got[2] == 0).any()


def test_verify_siblings_beside_infinite_distances():
    """A finite draft beside logits of +inf, and one beside two equal largest at a temperature next to 0: refused, with all left for
    the next."""
    rng = np.random.default_rng(71)
    for probs in (False, True):
        c = verify_case(rng, 12, 5, 700, torch.float32, probs)
        c["parents"][:] = [-1, 0, 0, 0, 0]
        c["temperatures"][:] = [1, 0.7, 1e-30, 1, 1e-40, 1e-38] * 2
        c["logits"][[0, 1, 3, 6, 7, 9], 0, 5] = c["logits"][[0, 1, 3, 6, 7, 9], 0, 9] = c["logits"][[0, 1, 3, 6, 7, 9], 0, 300] = float("inf")
        c["logits"][:, 0, 5] = c["logits"][:, 0, 9] = c["logits"][:, 0].max(-1).values.clamp(min=40.0)
        c["drafts"][:, 1:] = [3, 9, 40, 5]
        c["uniforms"][:, 1:] = np.column_stack([rng.uniform(0.1, 0.9, 12), rng.uniform(0.7, 0.99, 12), rng.uniform(0.1, 0.9, 12), rng.uniform(0.1, 0.4, 12)])
        if probs:
            c["draft_probs"][:, 0] = 0
            c["draft_probs"][:, 0, [3, 9, 40, 5]] = 0.25
        got = check_verify(c)
        assert not np.isin(got[1][:, 0], [1, 3]).any()
        if not probs:
            assert not (got[1][:, 0] == 2).any()             # u of 0.7 and more, where half or a third is its own


def test_verify_temperatures_at_the_ends():
    """An infinite one: all that are not -inf are equally likely; a tiny one: the largest is all there is."""
    rng = np.random.default_rng(28)
    for probs in (False, True):
        c = verify_case(rng, 6, 5, 1300, torch.float32, probs, chain=True)
        c["logits"][:, :, 900:] = -float("inf")
        c["temperatures"][:] = [float("inf"), 3e38, 1e30, 1e-40, 1e-30, float("inf")]
        c["drafts"][3:5, 1:] = f64(c["logits"]).argmax(-1)[3:5, :-1]
        got = check_verify(c)
        assert np.all(got[2][3:5] == 4)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_verify_large_temperatures_over_the_whole_range(dtype):
    """Logits at the type's lowest number at temperatures of its size: as likely as softmax(logits / T) says, at an infinite one as
    all others. (A rate is off by two of fp32's smallest steps, an exponent by 2 x 2^-149 x 2^128, a weight by 2^-20.5 of itself and
    so a share, p (1 - p) of that, by less than 2^-22: within check_verify's bound.)"""
    rng = np.random.default_rng(72)
    dt = {**DTYPES, "fp32": torch.float32}[dtype]
    for probs in (False, True):
        for V in (40, 1300):
            c = verify_case(rng, 10, 4, V, dt, probs)
            c["parents"][:] = [-1, 0, 0, 1]
            c["logits"][:, :, 1::2] = torch.finfo(dt).min
            c["logits"][:, :, 2::5] = -float("inf")
            c["temperatures"][:] = [float("inf"), 3.4e38, 3e38, 2e38, 1e38, 5e37, 2e37, 1e37, 1e36, 1e31]
            check_verify(c)
            c["uniforms"][:, 1:] = 1                         # every child refused: draws
            got = check_verify(c)
            assert np.all(got[2] == 0)
            c["uniforms"][:, 0] = 0.999                      # (a draw from the far end of what is left)
            got = check_verify(c)
            assert np.all(got[0][:3, 0] > V // 2)


def test_verify_refuses_results_over_inputs():
    c = verify_case(np.random.default_rng(29), 2, 3, 50, torch.float32, False)
    logits, drafts, parents, u = (torch.as_tensor(c[k]).to("cuda") for k in ("logits", "drafts", "parents", "uniforms"))
    both = torch.zeros((2, 2, 3), dtype=torch.int32, device="cuda")
    for kw in (dict(tokens=drafts), dict(path=parents), dict(tokens=u.view(torch.int32)), dict(accepted=drafts[0, :2]),
               dict(tokens=both[0], path=both[0]), dict(path=both[1], accepted=both[1, 0, 1:])):
        with pytest.raises(m.NvFp4MlaError):
            m.spec_verify(logits, drafts, parents, u, **kw)
    m.spec_verify(logits, drafts, parents, u, tokens=both[0], path=both[1])


def test_verify_leaves_out_and_counts_bad_drafts():
    rng = np.random.default_rng(24)
    c = verify_case(rng, 4, 6, 500, torch.float32, False, chain=True)
    c["temperatures"][:] = 0
    best = f64(c["logits"]).argmax(-1)
    c["drafts"][:, 1:] = best[:, :-1]                    # every draft right
    c["parents"][0, 3], c["drafts"][1, 2], c["drafts"][2, 1], c["parents"][3, 5] = 3, 500, -1, -2
    got = run_verify(c)
    assert list(got[2]) == [2, 1, 0, 4] and got[3] == [4, 0, 0, 0]
    check_verify(c)


def test_verify_draws_what_the_target_would():
    """20,000 requests of one distribution over 6 tokens, a tree of drafts drawn from another: the first token's frequencies are
    the target's within five standard deviations, with and without the drafts' distributions."""
    rng = np.random.default_rng(25)
    B, Q, V = 20000, 4, 6
    row, q = rng.standard_normal(V), rng.dirichlet(np.ones(V)).astype(np.float32)
    p = spec.softmax(row, 1.0)
    for probs in (False, True):
        c = dict(logits=torch.from_numpy(np.tile(row, (B, Q, 1))).float(), parents=np.tile(np.array([-1, 0, 0, 0], np.int32), (B, 1)),
                 drafts=(rng.choice(V, (B, Q), p=q / q.sum(dtype=np.float64)) if probs else np.tile([0, 4, 2, 4], (B, 1))).astype(np.int32),
                 uniforms=rng.random((B, Q)).astype(np.float32), draft_probs=np.tile(q, (B, Q, 1)) if probs else None)
        first = run_verify(c)[0][:, 0]
        share = np.bincount(first, minlength=V) / B
        assert np.all(np.abs(share - p) <= 5 * np.sqrt(p * (1 - p) / B))


def test_verify_other_stream_and_graph():
    rng = np.random.default_rng(26)
    c = verify_case(rng, 8, 5, 3000, torch.bfloat16, True, chain=True)
    want = run_verify(c)
    args = {k: (x if isinstance(x, torch.Tensor) else torch.from_numpy(x)).to("cuda") for k, x in c.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = m.spec_verify(**args, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, want))
    ws = torch.empty(m.spec_verify_workspace_size(8, 5, 3000), dtype=torch.uint8, device="cuda")
    outs = dict(tokens=torch.empty_like(got[0]), path=torch.empty_like(got[1]), accepted=torch.empty_like(got[2]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.spec_verify(**args, **outs, workspace=ws)
    for _ in range(3):
        for x in outs.values():
            x.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(outs.values(), want))


# ------------------------------------------------------------------ the accepted drafts' places
def keep_case(rng, lens, Q, Hk, D, layers=1):
    lens = np.asarray(lens, np.int32)
    need = -(-lens // 64)
    table = np.full((len(lens), max(1, need.max()) + 1), -1, np.int32)
    perm, at = rng.permutation(int(need.sum()) + 2), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    caches = rng.integers(0, 256, (layers, int(need.sum()) + 2, kv8.page_bytes(Hk, D)), dtype=np.uint8)
    for c in caches:
        kv8.parts(c, Hk, D)[1][:] = rng.integers(118, 131, kv8.parts(c, Hk, D)[1].shape)
    path, count = np.full((len(lens), Q), -1, np.int32), np.zeros(len(lens), np.int32)
    for b in range(len(lens)):
        nodes = np.sort(rng.choice(np.arange(1, Q), rng.integers(0, Q), replace=False)) if Q > 1 else []
        if b % 4 == 1:
            nodes = np.arange(1, rng.integers(1, Q + 1))     # a chain from the start: nothing moves
        path[b, :len(nodes)], count[b] = nodes, len(nodes)
    return caches, table, lens, path, count


@pytest.mark.parametrize("Q", [1, 2, 9, 33, 64])
@pytest.mark.parametrize("Hk,D,layers", [(1, 64, 1), (3, 128, 2), (8, 64, 3)])
def test_keep_bytes(Q, Hk, D, layers):
    rng = np.random.default_rng(Q * Hk)
    for start in (0, 1, 15, 16, 40, 63):
        caches, table, lens, path, count = keep_case(rng, Q + start + np.array([0, 1, 5, 47, 64, 100, 12]), Q, Hk, D, layers)
        d = dev(caches, torch.uint8)
        status = dev(np.zeros(4))
        new = m.kv8_keep(d if layers > 1 else d[0], dev(table), dev(lens), dev(path), dev(count), Hk, D, layered=layers > 1, dev_status=status)
        want = caches.copy()
        lens_want, bad_pages, bad = spec.keep(want, table, lens, path, count, Hk, D)
        assert np.array_equal(d.cpu().numpy(), want)
        assert new.tolist() == lens_want.tolist() and bad == bad_pages == 0 and status.tolist() == [0] * 4


def test_keep_leaves_out_and_counts_bad_data():
    rng = np.random.default_rng(30)
    caches, table, lens, path, count = keep_case(rng, [100, 100, 100, 100, 8, 130, 100, 131], 10, 2, 64)
    path[:], count[:] = -1, 3
    path[:, :3] = [2, 5, 9]
    path[0, 1] = 2                     # twice the same
    path[1, 2] = 10                    # no node
    count[2] = 10                      # more than there are drafts
    count[3] = -1                      # left out
    #                                  # request 4 is shorter than its tree
    table[5, 2] = -1                   # positions 128, 129: node 9 cannot be read
    path[6, 0] = 0
    table[7, 1] = len(caches[0])       # positions 64 .. 127, where nodes 5 and 6 lie (base 121), and all would go
    d, status = dev(caches, torch.uint8), dev(np.zeros(4))
    new = m.kv8_keep(d[0], dev(table), dev(lens), dev(path), dev(count), 2, 64, dev_status=status)
    want = caches.copy()
    lens_want, bad_pages, bad = spec.keep(want, table, lens, path, count, 2, 64)
    assert np.array_equal(d.cpu().numpy(), want) and new.tolist() == lens_want.tolist()
    assert bad == 5 and bad_pages >= 2 and status.tolist() == [0, bad_pages, 0, bad]


def test_keep_leaves_a_block_whose_drafts_have_no_page():
    """Two drafts on a page that is none, for a block that gets nothing else: its scale bytes, too, stay."""
    rng = np.random.default_rng(32)
    caches, table, lens, path, count = keep_case(rng, [67], 20, 1, 128)
    path[:], count[:] = -1, 2
    path[0, :2] = [17, 18]             # positions 64 and 65, to 48 and 49
    table[0, 1] = -1
    d, status = dev(caches, torch.uint8), dev(np.zeros(4))
    new = m.kv8_keep(d[0], dev(table), dev(lens), dev(path), dev(count), 1, 128, dev_status=status)
    assert np.array_equal(d.cpu().numpy(), caches) and new.tolist() == [50] and status.tolist() == [0, 2, 0, 0]
    want = caches.copy()
    assert spec.keep(want, table, lens, path, count, 1, 128)[1:] == (2, 0) and np.array_equal(want, caches)


def test_keep_refuses_new_lengths_over_inputs():
    rng = np.random.default_rng(33)
    caches, table, lens, path, count = keep_case(rng, [100, 130], 10, 2, 64)
    d, t, n, p, a = dev(caches, torch.uint8), dev(table), dev(lens), dev(path), dev(count)
    for new in (n, a, p[0, :2], p[1, 8:]):
        with pytest.raises(m.NvFp4MlaError):
            m.kv8_keep(d[0], t, n, p, a, 2, 64, new_lens=new)
    assert np.array_equal(d.cpu().numpy(), caches)


def test_trim():
    rng = np.random.default_rng(31)
    lens = np.array([0, 1, 64, 65, 200, 640, 300, 128, 5000], np.int32)
    need = -(-lens // 64)
    table = np.full((9, 80), -1, np.int32)
    perm, at = rng.permutation(int(need.sum()) + 5).astype(np.int32), 0
    for s, n in enumerate(need):
        table[s, :n] = perm[at:at + n]
        at += n
    table[7, 0] = table[6, 0]          # a shared page
    refs = np.bincount(table[table >= 0], minlength=len(perm)).astype(np.int32)
    new = np.array([0, 0, 64, 64, 201, 63, -1, 0, 70], np.int32)
    dt, dl, dr, status = dev(table), dev(lens), dev(refs), dev(np.zeros(4))
    m.kv_pages_trim(dt, dl, dr, dev(new), dev_status=status)
    bad = spec.trim(table, lens, refs, new)
    assert np.array_equal(dt.cpu().numpy(), table) and np.array_equal(dl.cpu().numpy(), lens) and np.array_equal(dr.cpu().numpy(), refs)
    assert bad == 2 and status.tolist() == [0, 0, 0, 2]
    m.kv_pages_trim(dt, dl, dr, dl, dev_status=status)      # to the present lengths: nothing
    assert np.array_equal(dt.cpu().numpy(), table) and status.tolist() == [0, 0, 0, 2]


def test_trim_refuses_new_lengths_over_the_state():
    """But seq_lens itself, which cuts nothing."""
    room = torch.full((5,), 70, dtype=torch.int32, device="cuda")
    table = torch.tensor([[0, 1], [2, 3], [4, 5], [6, 7]], dtype=torch.int32, device="cuda")
    refs = torch.ones(16, dtype=torch.int32, device="cuda")
    lens = room[:4]
    for new in (room[1:], table.view(-1)[2:6], refs[8:12]):
        with pytest.raises(m.NvFp4MlaError):
            m.kv_pages_trim(table, lens, refs, new)
    m.kv_pages_trim(table, lens, refs, lens)
    assert room.tolist() == [70] * 5 and table.view(-1).tolist() == list(range(8)) and refs.tolist() == [1] * 16
    m.kv_pages_trim(table, lens, refs, dev([64, 70, 1, 0]))
    assert lens.tolist() == [64, 70, 1, 0] and table.tolist() == [[0, -1], [2, 3], [4, -1], [-1, -1]]


def test_rope_keep_and_trim_on_another_stream():
    """What they take for their results, they take on that stream; what they give is what the current stream's call gives."""
    c = Rope([0, 15, 40], [3, 20, 33], 4, 2, 64, "bf16", 32, positions=True, seed=73)
    rng = np.random.default_rng(73)
    caches, table, lens, path, count = keep_case(rng, [70, 150, 90, 33], 12, 2, 64, layers=2)
    refs = np.bincount(table[table >= 0], minlength=caches.shape[1]).astype(np.int32)
    put = lambda x: x.to("cuda")  # noqa: E731

    def step(stream):
        rope, keep = dev(c.cache, torch.uint8), dev(caches, torch.uint8)
        args = (put(c.q), put(c.k), put(c.v), put(torch.from_numpy(c.sheet)), dev(c.cu), dev(c.lens), dev(c.table))
        weights = dict(q_weight=put(c.weights[0]), k_weight=put(c.weights[1]), eps=c.eps, positions=dev(c.positions[0]))
        dt, dl, dr, dp, da = dev(table), dev(lens), dev(refs), dev(path), dev(count)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        q = m.kv8_append_rope(*args, rope, **weights, stream=stream)
        new = m.kv8_keep(keep, dt, dl, dp, da, 2, 64, stream=stream, layered=True)
        m.kv_pages_trim(dt, dl, dr, new, stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        return q.clone(), rope, new.clone(), keep, dt, dl, dr

    want = step(None)
    c.check(want[0], want[1].cpu().numpy(), False)
    side = torch.cuda.Stream()
    for _ in range(5):
        for a, b in zip(step(side), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ------------------------------------------------------------------ together
def test_speculative_steps():
    """Several steps as a server makes them: room, rotated drafts, attention, verification, the accepted ones kept. Tables as the
    oracle's throughout, and the attention over the cache as it stands."""
    rng = np.random.default_rng(40)
    Hk, G, D, Q, V, layers, pages = 2, 4, 64, 9, 700, 2, 40
    H, B = Hk * G, 4
    table, lens, refs = np.full((B, 8), -1, np.int32), np.zeros(B, np.int32), np.zeros(pages, np.int32)
    dt, dl, dr = dev(table), dev(lens), dev(refs)
    cache = torch.zeros((layers, pages, m.kv8_page_bytes(Hk, D)), dtype=torch.uint8, device="cuda")
    angle = np.arange(600)[:, None] * 10000.0 ** (-np.arange(D // 2) / (D // 2))
    sheet = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1)).float().to("cuda")
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")

    def rows(n, heads):
        return torch.from_numpy(rng.standard_normal((n, heads, D))).to(torch.bfloat16).to("cuda")

    add = np.array([100, 63, 1, 130], np.int32)
    m.kv_pages_extend(dt, dl, dr, dev(add))
    kv8.extend(table, lens, refs, add)
    n = int(add.sum())
    for layer in range(layers):
        m.kv8_append_rope(rows(n, H), rows(n, Hk), rows(n, Hk), sheet, dev(np.concatenate([[0], np.cumsum(add)])), dl, dt, cache[layer], q_weight=w, k_weight=w)
    for step in range(6):
        parents, masks = trees(rng, B, Q)
        depth = np.array([[max(1, len(spec.bits(x, Q))) - 1 for x in row] for row in masks])
        at = (lens[:, None] + depth).astype(np.int32)
        m.kv_pages_extend(dt, dl, dr, dev(np.full(B, Q)))
        kv8.extend(table, lens, refs, np.full(B, Q))
        for layer in range(layers):
            q = m.kv8_append_rope(rows(B * Q, H), rows(B * Q, Hk), rows(B * Q, Hk), sheet, dev(np.arange(B + 1) * Q), dl, dt, cache[layer],
                                  q_weight=w, k_weight=w, positions=dev(at.reshape(-1))).view(B, Q, H, D)
            out, lse = m.kv8_decode_tree(q, cache[layer], dt, dl, dev(masks.view(np.int64), torch.int64), Hk, D ** -0.5)
            ref = spec.decode_tree(f64(q), cache[layer].cpu().numpy(), table, lens, masks, Hk, D ** -0.5)
            check_tree(out, lse, ref, 1000, f"step {step}")
        c = verify_case(rng, B, Q, V, torch.float32, False)
        c["parents"] = parents
        tokens, path, accepted = m.spec_verify(c["logits"].to("cuda"), *(torch.from_numpy(c[k]).to("cuda") for k in ("drafts", "parents", "uniforms", "temperatures")))
        want = spec.verify(f64(c["logits"]), c["drafts"], parents, c["uniforms"], c["temperatures"])
        assert np.array_equal(path.cpu().numpy(), want[1]) and np.array_equal(tokens.cpu().numpy(), want[0])
        before = cache.cpu().numpy()
        new = m.kv8_keep(cache, dt, dl, path, accepted, Hk, D, layered=True)
        m.kv_pages_trim(dt, dl, dr, new)
        new_want, _, _ = spec.keep(before, table, lens, want[1], want[2], Hk, D)
        spec.trim(table, lens, refs, new_want)
        assert np.array_equal(cache.cpu().numpy(), before)
        for a, b in ((dt, table), (dl, lens), (dr, refs)):
            assert np.array_equal(a.cpu().numpy(), b)


def step_args(rng, B, Q, Hk, G, D, V, old, pages, layers=1, first=0):
    """What a step needs, on the device, with sequences of `old` tokens whose pages begin at number `first`."""
    H, lens = Hk * G, np.asarray(old, np.int32)
    table, refs, at = np.full((B, 8), -1, np.int32), np.zeros(pages, np.int32), first
    for b, n in enumerate(-(-lens // 64)):
        table[b, :n] = np.arange(at, at + n)
        refs[at:at + n] = 1
        at += n
    refs[:first] = 1
    small = rng.integers(0, 0x78, (layers, at - first, m.kv8_page_bytes(Hk, D)), dtype=np.uint8)
    for x in small:
        kv8.parts(x, Hk, D)[1][:] = rng.integers(118, 131, kv8.parts(x, Hk, D)[1].shape)
    cache = torch.zeros((layers, pages, small.shape[2]), dtype=torch.uint8, device="cuda")
    cache[:, first:at] = torch.from_numpy(small).to("cuda")
    parents, masks = trees(rng, B, Q)
    depth = np.array([[max(1, len(spec.bits(x, Q))) - 1 for x in row] for row in masks])
    angle = np.arange(600)[:, None] * 10000.0 ** (-np.arange(D // 2) / (D // 2))
    rows = lambda heads: torch.from_numpy(rng.standard_normal((B * Q, heads, D))).to(torch.bfloat16).to("cuda")  # noqa: E731
    c = verify_case(rng, B, Q, V, torch.float32, True)
    put = lambda x: torch.as_tensor(x).to("cuda")  # noqa: E731
    return dict(cache=cache, table=dev(table), lens=dev(lens), refs=dev(refs), q=rows(H), k=rows(Hk), v=rows(Hk), cu=dev(np.arange(B + 1) * Q),
                add=dev(np.full(B, Q)), at=dev((lens[:, None] + depth).reshape(-1)), masks=dev(masks.view(np.int64), torch.int64),
                parents=dev(parents), sheet=put(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)), logits=put(c["logits"]),
                drafts=dev(c["drafts"]), uniforms=put(c["uniforms"]), temperatures=put(c["temperatures"]), probs=put(c["draft_probs"]),
                q_out=torch.zeros((B * Q, H, D), dtype=torch.bfloat16, device="cuda"),
                out=torch.zeros((layers, B, Q, H, D), dtype=torch.bfloat16, device="cuda"), lse=torch.zeros((layers, B, Q, H), device="cuda"),
                tokens=torch.zeros((B, Q), dtype=torch.int32, device="cuda"), path=torch.zeros((B, Q), dtype=torch.int32, device="cuda"),
                accepted=torch.zeros(B, dtype=torch.int32, device="cuda"), new=torch.zeros(B, dtype=torch.int32, device="cuda"),
                ws=torch.empty(m.kv8_decode_tree_workspace_size(B, Q, H, Hk, D), dtype=torch.uint8, device="cuda"),
                ws2=torch.empty(m.spec_verify_workspace_size(B, Q, V), dtype=torch.uint8, device="cuda"))


def run_step(a, Hk):
    layers, B, Q, H, D = a["out"].shape
    m.kv_pages_extend(a["table"], a["lens"], a["refs"], a["add"])
    for i in range(layers):
        m.kv8_append_rope(a["q"], a["k"], a["v"], a["sheet"], a["cu"], a["lens"], a["table"], a["cache"][i], positions=a["at"], q_out=a["q_out"])
        m.kv8_decode_tree(a["q_out"].view(B, Q, H, D), a["cache"][i], a["table"], a["lens"], a["masks"], Hk, D ** -0.5, out=a["out"][i], lse=a["lse"][i],
                          workspace=a["ws"])
    m.spec_verify(a["logits"], a["drafts"], a["parents"], a["uniforms"], a["temperatures"], a["probs"], tokens=a["tokens"], path=a["path"],
                  accepted=a["accepted"], workspace=a["ws2"])
    m.kv8_keep(a["cache"], a["table"], a["lens"], a["path"], a["accepted"], Hk, D, new_lens=a["new"], layered=True)
    m.kv_pages_trim(a["table"], a["lens"], a["refs"], a["new"])


def test_a_captured_step_replays():
    """A whole step in one graph, replayed over other tables, tokens and logits: what the calls do one by one."""
    one, two = (step_args(np.random.default_rng(50 + i), 5, 14, 2, 3, 128, 1200, [60 + i, 3, 128 - i, 200, 1], 60, layers=2) for i in range(2))
    start = {k: x.clone() for k, x in one.items()}
    run_step(one, 2)                   # (loads the kernels)
    for k, x in one.items():
        x.copy_(start[k])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run_step(one, 2)
    for source in (start, {k: x.clone() for k, x in two.items()}, start):
        for k in one:
            one[k].copy_(source[k])
            two[k].copy_(source[k])
        g.replay()
        run_step(two, 2)
        torch.cuda.synchronize()
        for k in one:
            if k not in ("ws", "ws2"):
                assert torch.equal(one[k].view(torch.uint8), two[k].view(torch.uint8)), k


def test_a_step_far_into_a_large_pool():
    """Pages whose bytes lie beyond 2^32: the results of the same step in a small pool."""
    big = step_args(np.random.default_rng(60), 3, 20, 8, 2, 128, 500, [50, 100, 200], 34000, first=33900)
    small = step_args(np.random.default_rng(60), 3, 20, 8, 2, 128, 500, [50, 100, 200], 100, first=0)
    assert big["cache"].stride(1) * 33900 > 1 << 32
    run_step(big, 8)
    run_step(small, 8)
    torch.cuda.synchronize()
    for k in ("q_out", "out", "lse", "tokens", "path", "accepted", "lens"):
        assert torch.equal(big[k].view(torch.uint8), small[k].view(torch.uint8)), k
    assert torch.equal(torch.where(big["table"] >= 0, big["table"] - 33900, -1), small["table"])
    assert torch.equal(big["cache"][:, 33900:], small["cache"])


def test_steps_of_no_requests():
    """B = 0, N = 0: nothing is enqueued, and nothing refused."""
    e = lambda *n, t=torch.int32: torch.zeros(n, dtype=t, device="cuda")  # noqa: E731
    bf, cache = torch.bfloat16, torch.zeros((3, m.kv8_page_bytes(2, 64)), dtype=torch.uint8, device="cuda")
    x = e(0, 2, 64, t=bf)
    assert m.kv8_append_rope(e(0, 4, 64, t=bf), x, x, e(10, 64, t=torch.float32), e(1), e(0), e(0, 2), cache).shape == (0, 4, 64)
    assert m.kv8_append_rope(e(0, 4, 64, t=bf), x, x, e(10, 64, t=torch.float32), e(3), e(2), e(2, 2), cache).shape == (0, 4, 64)
    assert m.kv8_decode_tree(e(0, 5, 4, 64, t=bf), cache, e(0, 2), e(0), e(0, 5, t=torch.int64), 2, 0.1)[0].shape == (0, 5, 4, 64)
    assert m.spec_verify(e(0, 5, 9, t=torch.float32), e(0, 5), e(0, 5), e(0, 5, t=torch.float32))[0].shape == (0, 5)
    assert m.kv8_keep(cache, e(0, 2), e(0), e(0, 5), e(0), 2, 64).shape == (0,)
