"""kv8_append and kv8_decode against the 64-bit oracle: bytes equal, attention within rounding."""
import numpy as np
import pytest
import torch

import nvfp4_compressed_sparse_gb300 as m
from oracle import kv8
from tests.kv8_util import DTYPES, Case, check, check_small_weights, dev, f64

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ append
def _append_case(rng, old, new, Hk, D, dtype, spare=2, width=None):
    """State after `old` tokens a request, written by the oracle over random bytes, and `new` more to append."""
    total = np.asarray(old) + np.asarray(new)
    need = -(-total // 64)
    table = np.full((len(old), width or max(1, need.max())), -1, np.int32)
    perm, at = rng.permutation(int(need.sum()) + spare), 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    cache = rng.integers(0, 256, (int(need.sum()) + spare, kv8.page_bytes(Hk, D)), dtype=np.uint8)

    def values(n):
        x = rng.standard_normal((n, Hk, D)) * np.exp2(rng.integers(-6, 7, (n, Hk, 1)))
        return torch.from_numpy(x).to(DTYPES[dtype])

    cu = np.concatenate([[0], np.cumsum(old)])
    kv8.append(cache, f64(values(cu[-1])), f64(values(cu[-1])), cu, np.asarray(old), table, Hk, D)
    n = int(np.sum(new))
    return cache, table, total.astype(np.int32), np.concatenate([[0], np.cumsum(new)]).astype(np.int32), values(n), values(n)


def _append(cache, k, v, cu, lens, table, **kw):
    d = dev(cache, torch.uint8)
    m.kv8_append(k.to("cuda"), v.to("cuda"), dev(cu), dev(lens), dev(table), d, **kw)
    torch.cuda.synchronize()
    return d.cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("Hk,D", [(1, 64), (3, 64), (2, 128), (8, 128)])
@pytest.mark.parametrize("old,new", [([0], [1]), ([0, 15, 16, 17, 63, 64, 65], [1] * 7), ([5, 0, 100, 31], [0, 64, 37, 130]),
                                     ([1, 2, 3], [0, 0, 1]), ([7] * 40, [1, 2, 3, 0] * 10)])
def test_append_bytes(old, new, Hk, D, dtype):
    rng = np.random.default_rng(len(old) * 100 + Hk + D)
    cache, table, lens, cu, k, v = _append_case(rng, old, new, Hk, D, dtype)
    got = _append(cache, k, v, cu, lens, table)
    want = cache.copy()
    assert kv8.append(want, f64(k), f64(v), cu, lens, table, Hk, D) == [0, 0]
    assert np.array_equal(got, want)


def test_append_one_token_at_a_time_ends_as_the_oracle_does():
    """96 steps: scales grow inside blocks, whose earlier codes are rounded again."""
    rng = np.random.default_rng(3)
    cache, table, lens, _, _, _ = _append_case(rng, [0, 9], [96, 96], 2, 64, "bf16")
    d, want = dev(cache, torch.uint8), cache.copy()
    for i in range(96):
        x = rng.standard_normal((2, 2, 2, 64)) * 2.0 ** (i % 16 - 8)
        k, v = (torch.from_numpy(y).to(torch.bfloat16) for y in x)
        at = np.array([i + 1, 10 + i], np.int32)
        m.kv8_append(k.to("cuda"), v.to("cuda"), dev([0, 1, 2]), dev(at), dev(table), d)
        kv8.append(want, f64(k), f64(v), [0, 1, 2], at, table, 2, 64)
    assert np.array_equal(d.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_special_values(dtype):
    """Zeros, both infinities, NaN of both signs, the smallest and largest numbers, and every power of two around 448."""
    rng = np.random.default_rng(4)
    cache, table, lens, cu, k, v = _append_case(rng, [3, 0, 0, 20], [40, 16, 16, 50], 2, 64, dtype)
    fin = torch.finfo(DTYPES[dtype])
    k[1, 0, :8] = torch.tensor([float("inf"), -float("inf"), float("nan"), -0.0, fin.tiny, -fin.tiny, fin.max, fin.min])
    v[2, 1, :6] = torch.tensor([float("inf"), -float("inf"), 0.0, fin.smallest_normal / 4, -fin.smallest_normal / 8, 1.0])
    bits = k.view(torch.int16)
    bits[5, 1, 3] = -1                     # a NaN with its sign set
    k[40:56] = 0                           # a block of zeros
    v[40:56] = 0
    v[40, 0, 0] = float("nan")             # no finite value but zeros
    k[56:72] = torch.where(torch.rand(16, 2, 64, generator=torch.Generator().manual_seed(1)) < 0.5, 448.0, 1.75)
    k[72:, 0] = 2.0 ** torch.randint(-8, 15, (50, 64)).to(k.dtype)
    got = _append(cache, k, v, cu, lens, table)
    want = cache.copy()
    kv8.append(want, f64(k), f64(v), cu, lens, table, 2, 64)
    nan = np.isnan(f64(k))                 # f64 loses a NaN's sign on some machines: the codes' magnitudes are compared there
    assert nan.any()
    a, b = kv8.parts(got, 2, 64), kv8.parts(want, 2, 64)
    assert np.array_equal(a[1], b[1])
    differ = a[0] != b[0]
    assert np.all((a[0][differ] & 0x7F) == 0x7F) and np.all((b[0][differ] & 0x7F) == 0x7F)
    page = table[0][0]
    assert a[0][page, 0, 1, 3 + 5, 3] == 0xFF


def test_append_scale_is_the_smallest_for_every_largest_value():
    """Every positive finite fp16, and bf16 of every exponent, as a block's largest value."""
    for dtype, bits in (("fp16", np.arange(1, 0x7C00)), ("bf16", np.arange(1, 0x7F80))):
        x = torch.from_numpy(bits.astype(np.int16)).view(DTYPES[dtype])
        n = len(x)
        k = torch.zeros((n * 16, 1, 64), dtype=DTYPES[dtype])
        k[::16, 0, 7] = x
        pages = -(-n * 16 // 64)
        table = np.arange(pages, dtype=np.int32)[None]
        cache = np.zeros((pages, kv8.page_bytes(1, 64)), np.uint8)
        got = _append(cache, k, k, np.array([0, n * 16]), np.array([n * 16]), table)
        scales = kv8.parts(got, 1, 64)[1][:, 0, 0].reshape(-1)[:n].astype(np.float64)
        s, a = 2.0 ** (scales - 127), f64(x)
        assert np.all(a <= 448 * s) and np.all((a > 224 * s) | (scales == 1))


def test_append_strides():
    """k and v as slices of a fused projection, and one key row for all heads (stride 0)."""
    rng = np.random.default_rng(6)
    cache, table, lens, cu, _, _ = _append_case(rng, [2, 70], [33, 7], 4, 128, "bf16")
    fused = torch.from_numpy(rng.standard_normal((40, 12, 128))).to(torch.bfloat16).to("cuda")
    k, v = fused[:, 4:8], fused[:, 8:]
    for a, b in ((k, v), (fused[:, 2:3].expand(40, 4, 128), v), (fused.transpose(0, 1)[:4, :, :].transpose(0, 1), v)):
        d = dev(cache, torch.uint8)
        m.kv8_append(a, b, dev(cu), dev(lens), dev(table), d)
        want = cache.copy()
        kv8.append(want, f64(a), f64(b), cu, lens, table, 4, 128)
        assert np.array_equal(d.cpu().numpy(), want)


def test_append_leaves_out_and_counts_bad_data():
    rng = np.random.default_rng(7)
    old, new = [10, 0, 5, 64, 3, 60], [20, 8, 3, 70, 4, 30]
    cache, table, lens, cu, k, v = _append_case(rng, old, new, 2, 128, "fp16")
    lens[1] = 5                      # eight new tokens would begin at -3
    table[2, 0] = -1
    table[3, 2] = len(cache)         # the second half of request 3's tokens: positions 128 .. 133
    table[5, 1:] = -1                # request 5's first four new tokens fit, the others do not
    status = dev(np.zeros(4))
    got = _append(cache, k, v, cu, lens, table, dev_status=status)
    want = cache.copy()
    bad = kv8.append(want, f64(k), f64(v), cu, lens, table, 2, 128)
    assert np.array_equal(got, want)
    assert status.tolist() == [0, bad[0], 0, bad[1]] and bad[1] == 1


def test_append_table_narrower_than_the_positions_and_tokens_behind_k():
    rng = np.random.default_rng(8)
    cache, table, lens, cu, k, v = _append_case(rng, [60, 1], [80, 20], 1, 64, "bf16")
    status = dev(np.zeros(4))
    got = _append(cache, k[:90], v[:90], cu, lens, table[:, :2].copy(), dev_status=status)
    want = cache.copy()
    bad = kv8.append(want, f64(k[:90]), f64(v[:90]), cu, lens, table[:, :2], 1, 64)
    assert np.array_equal(got, want) and bad == [1, 1] and status.tolist() == [0, 1, 0, 1]


def test_append_of_nothing():
    d = torch.full((2, m.kv8_page_bytes(1, 64)), 7, dtype=torch.uint8, device="cuda")
    k = torch.zeros((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    m.kv8_append(k, k, dev([0, 0]), dev([5]), dev([[0]]), d)
    m.kv8_append(k, k, dev([0]), dev(np.zeros(0)), dev(np.zeros((0, 1))), d)
    assert bool((d == 7).all())


def test_decode_of_no_requests():
    """A step that has none is as good as any, as it is for kv8_append; what it is given is checked all the same."""
    cache = torch.zeros((2, m.kv8_page_bytes(2, 64)), dtype=torch.uint8, device="cuda")
    q, table, lens = torch.zeros((0, 3, 4, 64), dtype=torch.float16, device="cuda"), dev(np.zeros((0, 5))), dev(np.zeros(0))
    out, lse = m.kv8_decode(q, cache, table, lens, 2, 0.125)
    assert out.shape == (0, 3, 4, 64) and out.dtype == torch.float16 and lse.shape == (0, 3, 4) and lse.dtype == torch.float32
    for bad in (dict(page_table=dev(np.zeros((1, 5)))), dict(cache=cache[:, 1:]), dict(window=-1)):
        with pytest.raises(ValueError):
            m.kv8_decode(**(dict(q=q, cache=cache, page_table=table, seq_lens=lens, kv_heads=2, softmax_scale=0.125) | bad))


# ------------------------------------------------------------------ decode
LENS = [1, 0, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 300, 1000]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hk,G,Q", [(1, 1, 1), (2, 4, 1), (1, 8, 1), (3, 5, 2), (2, 8, 2), (1, 16, 3), (2, 3, 16), (1, 33, 1), (1, 128, 1)])
def test_decode(Hk, G, Q, D, dtype):
    c = Case(LENS, Hk, D, dtype, Q=Q, G=G, seed=G + Q)
    check(*c.run(), c.reference())


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 128, 200, 5000])
@pytest.mark.parametrize("Q", [1, 5])
def test_decode_window(window, Q):
    c = Case(LENS, 2, 64, "bf16", Q=Q, G=2, seed=window)
    check(*c.run(window), c.reference(window))


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 128, 200, 5000])
@pytest.mark.parametrize("Q,G,dtype", [(1, 4, "bf16"), (5, 3, "fp16"), (4, 8, "bf16")])
def test_decode_window_at_128_dims(window, Q, G, dtype):
    c = Case(LENS, 2, 128, dtype, Q=Q, G=G, seed=window)
    check(*c.run(window), c.reference(window))


def test_decode_rows_that_masks_leave_empty():
    """More new tokens than cached ones, lengths of zero and below: out 0, lse -inf."""
    c = Case([0, 1, 3, 7, 8, 64], 2, 128, Q=8, G=2)
    c.lens[0] = 0
    out, lse = c.run()
    check(out, lse, c.reference())
    assert torch.isneginf(lse[1, :7]).all() and not out[1, :7].any()
    lens = c.lens.copy()
    c.lens = np.array([-5, -2147483648, 3, 7, 8, 64], np.int32)
    out2, lse2 = c.run()
    assert torch.isneginf(lse2[:2]).all() and not out2[:2].any()
    c.lens = lens
    assert torch.equal(out2[2:], out[2:])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[40000], [9000, 70, 25000, 1]])
def test_decode_long(lens, D):
    c = Case(lens, 1, D, "fp16", Q=2, G=4, seed=len(lens))
    check(*c.run(), c.reference())


@pytest.mark.parametrize("max_ctas", [1, 2, 3, 7, 40])
def test_decode_any_split_gives_the_same_within_rounding(max_ctas):
    c = Case([700, 1, 0, 1300, 129, 128, 4000, 64], 2, 64, "bf16", Q=2, G=3, seed=5)
    check(*c.run(max_ctas=max_ctas), c.reference())


@pytest.mark.parametrize("D,Hk,G", [(64, 1, 2), (64, 2, 12), (128, 1, 4), (128, 3, 16)])
@pytest.mark.parametrize("max_ctas", [0, 1, 3])
def test_decode_many_requests_of_a_tile_or_two(D, Hk, G, max_ctas):
    """Units of one tile leave one stream of tiles without work for many units in a row."""
    lens = np.random.default_rng(D + G).choice([0, 1, 5, 100, 128, 129, 200, 256, 257, 300, 640], 90, p=[.1, .1, .1, .3, .1, .05, .05, .05, .05, .05, .05])
    c = Case(lens, Hk, D, "fp16", G=G, seed=G)
    check(*c.run(max_ctas=max_ctas), c.reference())


@pytest.mark.parametrize("D,Hk,G,Q,dtype", [(64, 2, 2, 1, "bf16"), (64, 3, 12, 1, "fp16"), (128, 8, 4, 2, "bf16"), (128, 2, 16, 3, "fp16"),
                                            (64, 4, 5, 4, "bf16"), (128, 1, 1, 1, "fp16")])
@pytest.mark.parametrize("max_ctas", [0, 2, 7])
def test_decode_of_short_requests_only(D, Hk, G, Q, dtype, max_ctas):
    """Every unit has a tile or two: the streams take units in turn."""
    top = 256 if D == 128 else 512
    lens = np.random.default_rng(D + G + Q).choice([0, 1, 7, 64, top // 2 - 1, top // 2, top // 2 + 1, top - 1, top], 170)
    c = Case(lens, Hk, D, dtype, G=G, Q=Q, seed=G)
    check(*c.run(max_ctas=max_ctas), c.reference())


@pytest.mark.parametrize("D,G", [(64, 4), (64, 16), (128, 4), (128, 16)])
def test_decode_of_short_requests_with_nan_and_windows(D, G):
    """As above, with NaN in values that some queries attend to, a window, and pages that are none."""
    lens = np.random.default_rng(D + G).integers(1, 256, 120)
    c = Case(lens, 2, D, "bf16", G=G, Q=3, seed=G)
    codes, _ = kv8.parts(c.cache, 2, D)
    for b in range(0, 120, 7):
        t = int(lens[b]) - 1 - b % 3                        # the newest positions: some queries see them
        if t >= 0:
            codes[c.table[b, t // 64], 1, b % 2, t % 64, b % D] = 0x7F
    c.table[3::11, 0] = -1
    for window in (0, 70):
        check(*c.run(window, max_ctas=5), c.reference(window))


def test_decode_scales_far_apart():
    """Blocks whose scales differ by up to 2^60, keys and values apart; and a block of zeros."""
    c = Case([300, 1200], 2, 128, "bf16", Q=2, G=4, seed=9)
    codes, scales = kv8.parts(c.cache, 2, 128)
    used = scales != 0xFF
    scales[:, :, 1][used[:, :, 1]] = c.rng.integers(97, 157, used[:, :, 1].sum())
    scales[:, :, 0][used[:, :, 0]] = c.rng.integers(100, 121, used[:, :, 0].sum())
    codes[c.table[1, 3], :, :, 16:32] = 0
    scales[c.table[1, 3], :, :, 1] = 1
    check(*c.run(), c.reference())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_decode_one_weight_over_many_small_ones(dtype):
    """One key that outweighs each of 20,000 others by e^9 to e^14, whose values all have one sign."""
    for gap in (9.0, 11.0, 14.0):
        c = Case([20000], 1, 64, dtype, G=2, seed=1)
        codes, scales = kv8.parts(c.cache, 1, 64)
        q = torch.zeros((1, 1, 2, 64), dtype=DTYPES[dtype], device="cuda")
        q[..., 0] = 1.0
        c.q, c.scale = q, gap
        t = np.arange(20000)
        page, row = c.table[0][t // 64], t % 64
        codes[page, 0, 0, row] = 0
        codes[page, 1, 0, row] = 0x38 + c.rng.integers(0, 8, (20000, 64))     # 1 .. 1.875
        scales[page, 0, :, row // 16] = 127
        at = 12345
        codes[page[at], 0, 0, row[at], 0] = 0x38                              # the one key: 1
        codes[page[at], 1, 0, row[at]] = 0xB8                                 # its value: -1
        check(*c.run(), c.reference())


@pytest.mark.parametrize("low,high", [(252, 253), (1, 2), (1, 253), (190, 253)])
@pytest.mark.parametrize("D,G,Q", [(128, 4, 1), (64, 3, 1), (128, 4, 4), (64, 8, 2)])
@pytest.mark.parametrize("max_ctas", [0, 1, 5])
def test_decode_values_at_the_ends_of_the_range(low, high, D, G, Q, max_ctas):
    """Block scales of values from 2^-126 to 2^126, with scores that rise by 2^-50 to 2^50 from block to block."""
    c = Case([1000, 130, 40, 5], 2, D, "bf16", Q=Q, G=G, seed=low + G)
    codes, scales = kv8.parts(c.cache, 2, D)
    used = scales[:, :, 1] != 0xFF
    scales[:, :, 1][used] = c.rng.integers(low, high + 1, used.sum())
    codes[:, 1] = np.where(codes[:, 1] == 0xFF, 0xFF, codes[:, 1] & 0xBF)     # values below 2
    c.scale *= 4
    check(*c.run(max_ctas=max_ctas), c.reference())


@pytest.mark.parametrize("log2_step", [13, 25, 29])
@pytest.mark.parametrize("D,Q", [(128, 1), (64, 4)])
def test_decode_of_scores_that_rise_slowly(D, Q, log2_step):
    """Every 128 tokens the weights are 2^log2_step times those before: the sum's reference, which is raised by factors
    of more than 2^60, lies far below the largest, and the values are near fp32's end."""
    c = Case([1500, 257], 1, D, "bf16", Q=Q, G=4, seed=2)
    codes, scales = kv8.parts(c.cache, 1, D)
    c.q = torch.zeros((2, Q, 4, D), dtype=torch.bfloat16, device="cuda")
    c.q[..., 0] = 1.0
    c.scale = log2_step * float(np.log(2))
    for b, n in enumerate(c.lens):
        t = np.arange(n)
        page, row = c.table[b, t // 64], t % 64
        codes[page, 0, 0, row] = 0
        codes[page, 0, 0, row, 0] = kv8.e4m3_encode(t // 128.0)
        scales[page, 0, 0, row // 16] = 127
        codes[page, 1, 0, row] = 0x38 + c.rng.integers(0, 8, (n, D))
        scales[page, 0, 1, row // 16] = 253
    for ctas in (0, 1, 3):
        check(*c.run(max_ctas=ctas), c.reference())


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("D,Q,G", [(64, 1, 2), (128, 2, 8)])
def test_decode_of_large_scores_that_are_all_equal(sign, D, Q, G):
    """Scores of +-2^106: the result is the mean of the values, and lse the score."""
    c = Case([700, 3], 1, D, "bf16", Q=Q, G=G, seed=7)
    codes, scales = kv8.parts(c.cache, 1, D)
    codes[:, 0] = 0
    codes[:, 0, :, :, 5] = 0x38
    scales[:, :, 0] = 127 + 50
    c.q = torch.zeros(c.q.shape, dtype=torch.bfloat16, device="cuda")
    c.q[..., 5] = sign * 2.0 ** 56
    c.scale = 1.0
    out, lse = c.run()
    v = kv8.rows(c.cache, c.table[0], 700, 1, D)[1][0]
    half, steps = 2.0 ** -8, 2.0 ** -14
    for j in range(Q):
        seen = v[:700 - Q + 1 + j]
        want, mass = seen.mean(0), np.abs(seen).mean(0)
        assert np.all(np.abs(f64(out[0, j]) - want) <= half * np.abs(want) + (1 + half) * steps * mass)
    assert np.all(np.abs(f64(lse) - sign * 2.0 ** 106) <= 2.0 ** (106 - 21))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,log2_scale,at", [(10007, 10, 0), (100003, 10, 50000), (100003, 0, 77), (131000, 0, 130999), (131000, 6, 9)])
def test_decode_one_key_as_heavy_as_all_others_together(n, log2_scale, at, D, dtype):
    """One weight that equals the sum of n - 1 equal others, whose value has a block scale 2^log2_scale times theirs and
    is 0 in all dims but one: in those the result is the others' share alone. On one CTA, so that nothing is split."""
    c = Case([n], 1, D, dtype, G=2, seed=n)
    codes, scales = kv8.parts(c.cache, 1, D)
    c.q = torch.zeros((1, 1, 2, D), dtype=DTYPES[dtype], device="cuda")
    c.q[..., 0] = 1.0
    c.scale = float(np.log(n - 1))
    t = np.arange(n)
    page, row = c.table[0][t // 64], t % 64
    codes[page, 0, 0, row] = 0
    codes[page, 1, 0, row] = 0x38 + c.rng.integers(0, 8, (n, D))              # 1 .. 1.875
    scales[page, 0, :, row // 16] = 127
    block = at // 16 * 16 + np.arange(16)
    block = block[block < n]
    codes[page[block], 1, 0, row[block]] = 0                                  # (the scale is its whole block's)
    scales[page[at], 0, 1, row[at] // 16] = 127 + log2_scale
    codes[page[at], 0, 0, row[at], 0] = 0x38
    codes[page[at], 1, 0, row[at], D - 1] = 0xB8                              # -1
    out, lse = c.run(max_ctas=1)
    ref = c.reference()
    check_small_weights(out, ref, n / 64)                                     # two streams, 32 tokens an addition
    check(out, lse, ref)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,G,Q", [(128, 4, 1), (64, 3, 2), (128, 4, 4), (64, 16, 1), (128, 11, 3)])
@pytest.mark.parametrize("max_ctas", [0, 1, 4])
def test_decode_within_the_bound_of_what_weights_lose(D, G, Q, dtype, max_ctas):
    """Scores and block scales of a wide spread, cut into units of one and of several CTAs."""
    c = Case([3000, 700, 129, 1], 2, D, dtype, Q=Q, G=G, seed=D + G)
    _, scales = kv8.parts(c.cache, 2, D)
    used = scales[:, :, 1] != 0xFF
    low, high = (112, 138) if dtype == "bf16" else (112, 131)
    scales[:, :, 1][used] = c.rng.integers(low, high, used.sum())
    c.scale *= 2
    check_small_weights(c.run(max_ctas=max_ctas)[0], c.reference(), 3000 / 32)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_decode_a_key_far_above_a_million_others(dtype):
    """The others' weights are e^-15.9 of the one key's, and all their sum is an eighth of it."""
    n = 1 << 20
    c = Case([n], 1, 64, dtype, G=1, seed=3)
    codes, scales = kv8.parts(c.cache, 1, 64)
    c.q = torch.zeros((1, 1, 1, 64), dtype=DTYPES[dtype], device="cuda")
    c.q[..., 0] = 1.0
    c.scale = 15.9
    codes[:] = 0
    scales[:] = 127
    codes[:, 1] = 0x38 + c.rng.integers(0, 8, codes[:, 1].shape)
    codes[c.table[0, 700], 0, 0, 5, 0] = 0x38
    codes[c.table[0, 700], 1, 0, 5] = 0
    out, _ = c.run(max_ctas=1)
    check_small_weights(out, c.reference(), n / 64)


def test_decode_nan_reaches_only_who_attends_to_it():
    c = Case([200, 130], 2, 128, "bf16", Q=4, G=2, seed=11)
    codes, _ = kv8.parts(c.cache, 2, 128)
    codes[c.table[0, 3], 1, 0, 198 - 192, 5] = 0x7F      # a value of position 198: queries 2 and 3 of request 0
    codes[c.table[1, 0], 1, 1, 10, 127] = 0xFF           # a value of position 10: all queries of request 1 without a window
    codes[c.table[1, 1], 0, 0, 127 - 64, 0] = 0x7F       # a key of position 127: queries 1 to 3 of request 1
    for window in (0, 3, 120):
        check(*c.run(window), c.reference(window))


@pytest.mark.parametrize("D,Hk,G,Q,dtype", [(128, 3, 8, 2, "bf16"), (64, 2, 4, 4, "fp16"), (128, 1, 16, 2, "fp16")])
@pytest.mark.parametrize("max_ctas", [1, 3])
def test_decode_nan_of_some_columns_in_one_unit_after_the_other(D, Hk, G, Q, dtype, max_ctas):
    """More than eight columns (two warpgroups a stream), units of a tile or two, and in every unit a NaN in values
    that the later queries alone attend to: what one unit notes of it is gone, and only that, when the next begins."""
    lens = np.random.default_rng(G).integers(Q, 2 * (128 if D == 128 else 256), 150)
    c = Case(lens, Hk, D, dtype, G=G, Q=Q, seed=G)
    codes, _ = kv8.parts(c.cache, Hk, D)
    for b in range(150):
        t = int(lens[b]) - 1                                # the newest position: the last query's
        codes[c.table[b, t // 64], 1, :, t % 64, b % D] = 0x7F
        if b % 3 == 0:
            codes[c.table[b, (t - 1) // 64], 1, 0, (t - 1) % 64, (b + 17) % D] = 0xFF
    ref = c.reference()
    assert np.isnan(ref[0][:, -1]).any() and not np.isnan(ref[0][1::3, 0]).any()
    for _ in range(5):
        check(*c.run(max_ctas=max_ctas), ref)


def test_decode_non_finite_queries():
    c = Case([200, 64, 0], 1, 64, "fp16", Q=2, G=2, seed=12)
    c.q[0, 0, 0, 3] = float("inf")
    c.q[0, 1, 1, 4] = float("nan")
    c.q[1, 0, 1, 9] = -float("inf")
    c.q[2, 0, 0, 0] = float("nan")           # no position: 0
    out, lse = c.run()
    for b, j, h in ((0, 0, 0), (0, 1, 1), (1, 0, 1)):
        assert torch.isnan(out[b, j, h]).all() and torch.isnan(lse[b, j, h])
    ref = [x.copy() for x in c.reference()]
    for b, j, h in ((0, 0, 0), (0, 1, 1), (1, 0, 1)):
        ref[0][b, j, h] = ref[1][b, j, h] = np.nan
        ref[2][b, j, h] = ref[3][b, j, h] = ref[4][b, j, h] = 0
    check(out, lse, ref)


def test_decode_large_and_small_queries():
    c = Case([500], 2, 64, "bf16", Q=1, G=3, seed=13)
    c.q[0, 0, 0] *= 2.0 ** -120
    c.q[0, 0, 1] = 0
    c.q[0, 0, 2] *= 2.0 ** 6
    c.q[0, 0, 3] *= torch.exp2(torch.arange(64, device="cuda") - 40.0)
    check(*c.run(), c.reference())


def test_decode_leaves_out_and_counts_bad_pages():
    c = Case([500, 300, 70], 2, 64, Q=2, G=2, seed=14)
    c.table[0, 2] = -1
    c.table[0, 5] = len(c.cache)
    c.table[1, 0] = -7
    c.table[2] = -1
    status = dev(np.zeros(4))
    out, lse = c.run(dev_status=status)
    check(out, lse, c.reference())
    assert status.tolist() == [0, 5, 0, 0]
    c.lens = np.array([5000, 300, 70], np.int32)      # 79 pages, 8 of them in the table
    status.zero_()
    check(*c.run(dev_status=status), c.reference())
    assert status.tolist() == [0, 5 + 71, 0, 0]


def test_decode_strided_q():
    c = Case([100, 77, 300], 2, 64, Q=3, G=2, seed=15)
    fused = torch.randn((3, 3, 12, 64), device="cuda").to(torch.bfloat16)
    for q in (fused[:, :, 4:8], fused[:, :, 3:4].expand(3, 3, 4, 64)):
        check(*c.run(q=q), c.reference(q=q))


def test_decode_offsets_beyond_32_bits():
    """Pages at the end of a cache of 6.3 GB."""
    c = Case([300, 129], 8, 128, G=1, seed=16)
    pages = 48000
    cache = torch.zeros((pages, m.kv8_page_bytes(8, 128)), dtype=torch.uint8, device="cuda")
    moved = np.where(c.table >= 0, pages - 1 - 4000 * c.table, -1)
    for a, b in zip(c.table.ravel(), moved.ravel()):
        if a >= 0:
            cache[int(b)] = dev(c.cache[a], torch.uint8)
    out, lse = m.kv8_decode(c.q, cache, dev(moved), dev(c.lens), 8, c.scale)
    check(out, lse, c.reference())
    k, v = c.k[:1].to("cuda"), c.v[:1].to("cuda")
    m.kv8_append(k, v, dev([0, 1]), dev([301]), dev(moved[:1]), cache)
    want = c.cache.copy()
    kv8.append(want, f64(k), f64(v), [0, 1], [301], c.table[:1], 8, 128)
    last = int(c.table[0, 4])
    assert np.array_equal(cache[int(moved[0, 4])].cpu().numpy(), want[last])


def test_decode_graphs_that_share_a_workspace():
    """Two captured steps of different sizes over one workspace, replayed in turn with new inputs."""
    cases = [Case([900, 40, 3000], 2, 64, Q=2, G=2, seed=17), Case([5000], 4, 128, G=3, seed=18)]
    need = max(m.kv8_decode_workspace_size(len(c.lens), c.Q, c.H, c.Hk, c.D) for c in cases)
    ws = torch.randint(0, 256, (need,), dtype=torch.uint8, device="cuda")
    graphs = []
    for c in cases:
        args = [c.q.clone(), dev(c.cache, torch.uint8), dev(c.table), dev(c.lens)]
        out, lse = m.kv8_decode(*args, c.Hk, c.scale, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.kv8_decode(*args, c.Hk, c.scale, out=out, lse=lse, workspace=ws)
        graphs.append((c, g, args, out, lse))
    for turn in range(3):
        for c, g, args, out, lse in graphs:
            q = torch.randn(c.q.shape, device="cuda").to(c.q.dtype)
            args[0].copy_(q)
            out.fill_(7)
            lse.fill_(7)
            g.replay()
            torch.cuda.synchronize()
            check(out, lse, c.reference(q=q), f"turn {turn}")


def test_decode_on_two_streams_at_once():
    cases = [Case([3000, 200], 2, 64, G=2, seed=s) for s in (19, 20)]
    streams = [torch.cuda.Stream() for _ in cases]
    args = [(c.q, dev(c.cache, torch.uint8), dev(c.table), dev(c.lens), c.Hk, c.scale) for c in cases]
    torch.cuda.synchronize()
    results = []
    for _ in range(20):
        for c, a, s in zip(cases, args, streams):
            with torch.cuda.stream(s):
                results.append((c, m.kv8_decode(*a)))
    torch.cuda.synchronize()
    refs = {id(c): c.reference() for c in cases}
    for c, (out, lse) in results:
        check(out, lse, refs[id(c)])


def test_decode_repeats_bit_for_bit():
    c = Case([9000, 70, 2500, 1], 2, 128, Q=2, G=4, seed=21)
    first = c.run()
    for _ in range(10):
        again = c.run()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_decode_waits_are_bounded_and_the_next_calls_are_right():
    """A step whose tiles never come (a testing flag) gives up after its limit, says so, and leaves workspace
    and device fit for the next step, a replay of a captured one over the same workspace included."""
    c = Case([3000, 200], 2, 64, Q=2, G=2, seed=22)
    ws = torch.zeros(m.kv8_decode_workspace_size(2, 2, 4, 2, 64), dtype=torch.uint8, device="cuda")
    args = (c.q, dev(c.cache, torch.uint8), dev(c.table), dev(c.lens), 2, c.scale)
    out, lse = m.kv8_decode(*args, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.kv8_decode(*args, out=out, lse=lse, workspace=ws)
    status = dev(np.zeros(4))
    m.kv8_decode(*args, workspace=ws, dev_status=status, test_timeout=True)
    torch.cuda.synchronize()
    assert status[2] > 0 and status[[0, 1, 3]].tolist() == [0, 0, 0]
    for _ in range(2):
        out.fill_(7)
        g.replay()
        check(out, lse, c.reference())
    check(*m.kv8_decode(*args, workspace=ws), c.reference())


def test_decode_on_a_stream_of_its_own_keeps_what_it_took():
    """out, lse and workspace taken by the call itself, on the current stream, while the step waits on another:
    what is taken from the allocator next must not be theirs."""
    c = Case([2000, 900], 2, 128, Q=1, G=4, seed=23)
    args = (c.q, dev(c.cache, torch.uint8), dev(c.table), dev(c.lens), 2, c.scale)
    want = m.kv8_decode(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    x = torch.randn((4096, 4096), device="cuda")
    size = m.kv8_decode_workspace_size(2, 1, 8, 2, 128)
    for _ in range(3):
        with torch.cuda.stream(s):
            for _ in range(20):
                x = x @ x * 1e-3            # some milliseconds before the step
        out, lse = m.kv8_decode(*args, stream=s)
        for _ in range(8):
            torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        s.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_decode_of_expanded_and_one_entry_axes():
    """Axes of one entry may have any stride; a batch axis that repeats one query row (stride 0)."""
    c = Case([100, 77], 1, 64, Q=1, G=1, seed=24)
    wide = torch.randn((2, 1, 1, 100), device="cuda").to(torch.bfloat16)
    q = wide.as_strided((2, 1, 1, 64), (0, 7, 13, 1))
    check(*c.run(q=q), c.reference(q=q))


def test_refusals():
    c = Case([100, 30], 2, 64, "bf16", G=2, seed=30)
    cache, table, lens, short = dev(c.cache, torch.uint8), dev(c.table), dev(c.lens), dev(np.zeros(3))
    k, cu = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda"), dev([0, 1, 2])
    ws = torch.empty(2 * m.kv8_decode_workspace_size(2, 1, 4, 2, 64), dtype=torch.uint8, device="cuda")
    before = cache.clone()
    odd = torch.zeros(2, 2, 65, dtype=torch.bfloat16, device="cuda")[:, :, :64]      # strides that are no multiples of 8
    decodes = [dict(window=-1), dict(window=1 << 31), dict(window=(1 << 32) + 5), dict(dev_status=short), dict(workspace=ws[::2]),
               dict(workspace=ws[:256]), dict(workspace=ws[4:]), dict(q=c.q.cpu()), dict(q=c.q.float()), dict(q=c.q[..., ::2]),
               dict(q=c.q[:1]), dict(out=torch.empty_like(c.q).half()), dict(lse=torch.empty(2, 1, 3, device="cuda"))]
    calls = [lambda kw=kw: m.kv8_decode(kw.pop("q", c.q), cache, table, lens, 2, c.scale, **kw) for kw in decodes]
    calls += [lambda: m.kv8_decode(c.q, cache, table, lens, 2, 0.0), lambda: m.kv8_decode(c.q, cache, table, lens, 3, c.scale),
              lambda: m.kv8_decode(c.q, cache[:, :-1], table, lens, 2, c.scale),
              lambda: m.kv8_append(k, k, cu, lens, table, cache, dev_status=short), lambda: m.kv8_append(odd, k, cu, lens, table, cache),
              lambda: m.kv8_append(k, k.half(), cu, lens, table, cache), lambda: m.kv8_append(k, k[:1], cu, lens, table, cache),
              lambda: m.kv8_append(k, k, cu[:2], lens, table, cache), lambda: m.kv8_append(k, k, cu, lens, table, cache.cpu()),
              lambda: m.kv8_append(k[:, :1], k[:, :1], cu, lens, table, cache)]
    for i, call in enumerate(calls):
        with pytest.raises((ValueError, TypeError, m.NvFp4MlaError)):
            call()
            pytest.fail(f"call {i} was not refused")
    torch.cuda.synchronize()
    assert torch.equal(cache, before)
    check(*c.run(), c.reference())
