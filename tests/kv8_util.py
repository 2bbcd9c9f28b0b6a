"""Helpers of the 8-bit cache's and the page operators' GPU tests."""
import numpy as np
import torch

import nvfp4_compressed_sparse_gb300 as m
from oracle import kv8

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dtype)


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


class Case:
    """A cache filled by the oracle, over bytes that no kernel may read: 0xFF wherever no token is."""

    def __init__(self, lens, Hk, D, dtype="bf16", Q=1, G=1, seed=0, spare=3, garbage=0xFF, spread=1.0):
        self.rng = np.random.default_rng(seed)
        self.Hk, self.D, self.Q, self.H, self.dtype = Hk, D, Q, Hk * G, DTYPES[dtype]
        self.lens = np.asarray(lens, np.int32)
        need = [-(-max(0, int(n)) // 64) for n in lens]
        pages = sum(need) + spare
        perm = self.rng.permutation(pages)
        self.table = np.full((len(lens), max(1, max(need))), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.cache = np.full((pages, kv8.page_bytes(Hk, D)), garbage, np.uint8)
        tokens = int(np.maximum(self.lens, 0).sum())
        shape = (tokens, Hk, D)
        self.k = self.values(shape, spread)
        self.v = self.values(shape, spread)
        cu = np.concatenate([[0], np.cumsum(np.maximum(self.lens, 0))])
        assert kv8.append(self.cache, f64(self.k), f64(self.v), cu, np.maximum(self.lens, 0), self.table, Hk, D) == [0, 0]
        self.q = self.values((len(lens), Q, self.H, D), spread).to("cuda")
        self.scale = D ** -0.5

    def values(self, shape, spread=1.0):
        x = self.rng.standard_normal(shape) * np.exp(0.5 * self.rng.standard_normal(shape[1:]))
        x *= np.exp2(np.round(spread * self.rng.standard_normal((shape[0],) + (1,) * (len(shape) - 1))))
        return torch.from_numpy(x).to(self.dtype)

    def reference(self, window=0, cache=None, q=None):
        return kv8.decode(f64(self.q if q is None else q), self.cache if cache is None else cache, self.table, self.lens,
                          self.Hk, self.scale, window)

    def run(self, window=0, q=None, **kw):
        return m.kv8_decode(self.q if q is None else q, dev(self.cache, torch.uint8), dev(self.table), dev(self.lens),
                            self.Hk, self.scale, window=window, **kw)


def check(out, lse, ref, what=""):
    """Outputs against the oracle's.

    A score is a sum of D products in fp32, off by at most (D + 8) 2^-24 of reach (each of its D additions, and
    the scalings, by half a step of 2^-24). A weight is off by that, by the exponential's 2^-21, and by its own
    rounding to at least 16 bits (2^-16); the quotient of two such sums by twice as much. The output is then
    rounded once to its type: half a step.

    The 16 bits hold for weights (times their value's scale) that are not far below the largest one. A weight x is
    held as four E4M3 parts, each a sixteenth of the one before, in units in which the largest is 16 to 256: below
    2^-6 a part has steps of 2^-9, so the last part's are 2^-9 / 16^3 = 2^-21, half of that is 2^-22, and that is
    at most 2^-26 of the largest. So a code is added with a weight that is off by 2^-26 of the largest: 2^-26 spread.
    """
    r_out, r_lse, mass, reach, spread = ref
    D = r_out.shape[-1]
    dz = (D + 8) * 2.0 ** -24 * reach
    dw = dz + 2.0 ** -21 + 2.0 ** -16
    half = torch.finfo(out.dtype).eps / 2
    tiny = torch.finfo(out.dtype).smallest_normal * half
    got, got_lse = f64(out), f64(lse)
    nan = np.isnan(r_out)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN in other places"
    tol = half * np.abs(r_out) + (1 + half) * (2 * dw[..., None] * mass + 2.0 ** -26 * spread) + tiny
    worst = np.nanmax(np.where(nan, 0, np.abs(got - r_out) / tol)) if got.size else 0
    assert worst <= 1, f"{what}: out off by {worst:.2f} of the bound"
    assert np.array_equal(np.isnan(got_lse), np.isnan(r_lse)), f"{what}: NaN lse in other places"
    empty = np.isneginf(r_lse)
    assert np.array_equal(np.isneginf(got_lse), empty), f"{what}: empty rows differ"
    fine = ~empty & ~np.isnan(r_lse)
    tol = (dw + 2.0 ** -22 * np.maximum(1, np.abs(np.where(fine, r_lse, 0))))[fine]
    assert np.all(np.abs(got_lse[fine] - r_lse[fine]) <= tol), f"{what}: lse"


def check_small_weights(out, ref, adds, what=""):
    """Outputs against the oracle's, with what weights far below the largest one may lose.

    A weight is held as four E5M2 parts, each a sixteenth of the one before, with the largest at 2^11 to 2^15. A part
    has three bits: it leaves at most 2^-3 of the power of two below its value, which is itself at least the power of
    two above what is left, so that the next ones leave 2^-4 each: 2^-3-4-4-4 = 2^-15. Below 2^-14 a part has steps of
    2^-16, so the last one leaves 2^-17 / 16^3 = 2^-29, 2^-40 of the largest weight times its value's scale. The sum
    is made of `adds` additions in 32 bits, each off by at most a step (2^-23) of what it has reached. Scores and
    exponentials as in check(); the sum that divides is of unrounded weights. (check() was derived for four E4M3 parts:
    it has 2^-16 twice, as if the divisor were rounded too, which covers 2^-15 once, and 2^-26 of spread.)"""
    r_out, _, mass, reach, spread = ref
    dz = (r_out.shape[-1] + 8) * 2.0 ** -24 * reach
    dw = 2 * (dz + 2.0 ** -21) + 2.0 ** -15 + adds * 2.0 ** -23
    half = torch.finfo(out.dtype).eps / 2
    tiny = torch.finfo(out.dtype).smallest_normal * half
    tol = half * np.abs(r_out) + (1 + half) * (dw[..., None] * mass + 2.0 ** -40 * spread) + tiny
    worst = np.max(np.abs(f64(out) - r_out) / tol)
    assert worst <= 1, f"{what}: out off by {worst:.2f} of the bound"
