"""The page operators against plain loops: every table, count and byte equal; and a server's steps end to end."""
import numpy as np
import pytest
import torch

import nvfp4_compressed_sparse_gb300 as m
from oracle import kv8
from tests.kv8_util import Case, check, dev, f64

pytestmark = pytest.mark.gpu


class State:
    """A pool in use, on the device and as arrays for the oracle."""

    def __init__(self, lens, pages, page_bytes=256, layers=1, width=None, seed=0):
        rng = np.random.default_rng(seed)
        self.lens = np.asarray(lens, np.int32)
        need = -(-self.lens // 64)
        self.table = np.full((len(lens), width or max(1, int(need.max()) + 2)), -1, np.int32)
        perm, at = rng.permutation(pages), 0
        self.refs = np.zeros(pages, np.int32)
        for s, n in enumerate(need):
            self.table[s, :n] = perm[at:at + n]
            self.refs[perm[at:at + n]] += 1
            at += n
        self.cache = rng.integers(0, 256, (layers, pages, page_bytes), dtype=np.uint8)
        self.d_table, self.d_lens, self.d_refs = dev(self.table), dev(self.lens), dev(self.refs)
        self.d_cache = dev(self.cache, torch.uint8)
        self.status = dev(np.zeros(4))

    def same(self):
        assert np.array_equal(self.d_table.cpu().numpy(), self.table)
        assert np.array_equal(self.d_lens.cpu().numpy(), self.lens)
        assert np.array_equal(self.d_refs.cpu().numpy(), self.refs)
        assert np.array_equal(self.d_cache.cpu().numpy(), self.cache)
        held = np.bincount(self.table[self.table >= 0].ravel(), minlength=len(self.refs))
        assert np.array_equal(held, self.refs)

    def free(self, seqs):
        m.kv_pages_free(self.d_table, self.d_lens, self.d_refs, dev(seqs), dev_status=self.status)
        kv8.free(self.table, self.lens, self.refs, seqs)

    def fork(self, src, dst):
        new = m.kv_pages_fork(self.d_cache, self.d_table, self.d_lens, self.d_refs, dev(src), dev(dst), dev_status=self.status, layered=True)
        assert new.tolist() == kv8.fork(self.cache, self.table, self.lens, self.refs, src, dst)

    def extend(self, add):
        granted = dev(np.full(len(add), 9))
        m.kv_pages_extend(self.d_table, self.d_lens, self.d_refs, dev(add), granted=granted, dev_status=self.status)
        assert granted.tolist() == kv8.extend(self.table, self.lens, self.refs, add)

    def compact(self):
        remap, live = m.kv_pages_compact(self.d_cache, self.d_table, self.d_refs, dev_status=self.status, layered=True)
        want, n = kv8.compact(self.cache, self.table, self.refs)
        assert np.array_equal(remap.cpu().numpy(), want) and live.item() == n


@pytest.mark.parametrize("page_bytes,layers", [(16, 1), (4112, 2), (22528, 3), (131200, 1)])
@pytest.mark.parametrize("n", [0, 1, 7, 40])
def test_copy(page_bytes, layers, n):
    s = State([10], 100, page_bytes, layers, seed=n)
    perm = np.random.default_rng(n).permutation(100)
    src, dst = perm[:n], perm[n:2 * n]
    m.kv_pages_copy(s.d_cache, dev(src), dev(dst), layered=True)
    kv8.copy(s.cache, src, dst)
    s.same()


def test_copy_skips_and_counts():
    s = State([10], 10, seed=1)
    src, dst = [-1, 0, 1, 10, 2, -2, 3, 5, 2147483647], [4, -1, 6, 7, 11, 8, 9, 5, 0]
    m.kv_pages_copy(s.d_cache, dev(src), dev(dst), dev_status=s.status, layered=True)
    assert kv8.copy(s.cache, src, dst) == 4
    s.same()
    assert s.status.tolist() == [0, 4, 0, 0]


def test_copy_of_one_cache_of_the_other_kinds():
    """[P, 64, row bytes], as the packed MLA caches are held."""
    cache = torch.randint(0, 256, (9, 64, 352), dtype=torch.uint8, device="cuda")
    want = cache.clone()
    want[[1, 3]] = cache[[8, 0]]
    m.kv_pages_copy(cache, dev([8, 0]), dev([1, 3]))
    assert torch.equal(cache, want)


@pytest.mark.parametrize("seqs", [[], [0], [3, 1, 0, 2], [2, 2, 2], [-1, 1], [1, 4, -2, 3, 1]])
def test_free(seqs):
    s = State([100, 64, 1, 0], 20, width=3, seed=2)
    s.fork([0], [3])
    s.free(seqs)
    s.same()
    assert s.status.tolist() == [0, 0, 0, sum(x < -1 or x > 3 for x in seqs)]


def test_free_of_wide_rows_and_broken_entries():
    s = State([70000, 65], 1200, page_bytes=16, seed=3)
    lost = int(s.table[1, 1])                          # its entry goes, its count stays
    s.d_table[1, 1], s.table[1, 1] = 1200, 1200
    s.refs[s.table[1, 0]] = 0
    s.d_refs.copy_(dev(s.refs))
    m.kv_pages_free(s.d_table, s.d_lens, s.d_refs, dev([0, 1]), dev_status=s.status)
    assert torch.nonzero(s.d_refs).flatten().tolist() == [lost] and s.d_refs[lost] == 1
    assert bool((s.d_table == -1).all()) and not s.d_lens.any()
    assert s.status.tolist() == [0, 2, 0, 0]


@pytest.mark.parametrize("layers,page_bytes", [(1, 128), (3, 20000)])
@pytest.mark.parametrize("lens,src,dst", [
    ([100, 64, 1, 0, 0, 0, 0], [0, 1, 2], [3, 4, 5]),
    ([100, 64, 1, 0, 0, 0, 0], [0, 0, 0, 0], [6, 3, 5, 4]),
    ([100, 64, 1, 0, 0, 0, 0], [], []),
    ([100, 64, 1, 0, 0, 0, 0], [0, 1, 2, 0], [3, 3, 3, 4]),        # the same target again
    ([100, 64, 1, 0, 0, 0, 0], [0, 1, 7, -1, 5, 2], [1, 0, 3, 3, 5, 3]),   # targets in use, numbers that are none, itself
    ([100, 64, 1, 0, 0, 0, 0], [3, 0, 4], [4, 3, 5]),              # an empty source, which is a target too
    ([100, 64, 1, 0, 0, 0, 0], [0, 3, 3], [3, 4, 4]),
])
def test_fork(lens, src, dst, layers, page_bytes):
    s = State(lens, 12, page_bytes, layers, seed=4)
    s.fork(src, dst)
    s.same()


def test_fork_when_pages_run_out():
    s = State([100, 64, 1, 65, 0, 0, 0, 0, 0, 0], 8, seed=5)       # 6 in use
    s.fork([0, 1, 2, 3, 0, 1], [4, 5, 6, 7, 8, 9])
    s.same()
    assert s.lens.tolist() == [100, 64, 1, 65, 100, 64, 1, 0, 0, 64]
    assert s.status.tolist() == [0, 0, 0, 0]


def test_fork_of_many_pairs():
    rng = np.random.default_rng(6)
    lens = np.concatenate([rng.integers(0, 300, 4000), np.zeros(16000, np.int64)])
    s = State(lens, 40000, page_bytes=16, seed=6)
    src = rng.integers(0, 4000, 16384)
    dst = 4000 + rng.integers(0, 16000, 16384)                     # many named twice
    s.fork(src, dst)
    s.same()


@pytest.mark.parametrize("pages", [10, 300, 5001])
@pytest.mark.parametrize("seed", range(3))
def test_extend(pages, seed):
    rng = np.random.default_rng(seed)
    s = State([0, 1, 63, 64, 65, 0, 128], pages, width=40, seed=seed)
    for _ in range(6):
        s.extend(rng.integers(0, 2, 7) * rng.choice([1, 63, 64, 65, 1000], 7))
        s.same()


def test_extend_passes_over_what_does_not_fit():
    """A sequence that asks for more than there is left takes nothing from those behind it."""
    s = State([64] * 6, 16, width=40, seed=14)                         # 10 free
    s.extend([64 * 20, 64 * 3, 64 * 8, 64 * 7, 1, 0])
    assert s.lens.tolist() == [64, 256, 64, 512, 64, 64] and not (s.refs == 0).any()
    s.same()


@pytest.mark.parametrize("n,pages", [(5, 12), (33, 100), (1500, 3000), (16384, 30000), (16384, 16400)])
def test_extend_when_pages_run_out(n, pages):
    rng = np.random.default_rng(n)
    s = State(rng.integers(0, 65, n), pages, page_bytes=16, width=300, seed=n)
    for _ in range(3):
        s.extend(rng.integers(0, 2, n) * rng.choice([1, 60, 300, 2000, 17000], n, p=[.4, .3, .2, .05, .05]))
        s.same()
    assert (s.refs == 0).sum() < 5


def test_extend_refuses():
    s = State([10, 20, 30, 64, 0], 100, width=2, seed=7)
    s.d_lens[4], s.lens[4] = -3, -3
    s.extend([118, 109, -1, 64, 5])      # to 128 tokens, to 129 in a row of two pages, a negative add, to 128, a negative length
    assert s.lens.tolist() == [128, 20, 30, 128, -3] and s.status.tolist() == [0, 0, 0, 3]
    assert np.array_equal(s.d_lens.cpu().numpy(), s.lens) and np.array_equal(s.d_table.cpu().numpy(), s.table)


def test_extend_of_many_sequences_and_pages():
    rng = np.random.default_rng(8)
    s = State(rng.integers(0, 200, 16384), 150000, page_bytes=16, width=8, seed=8)
    s.free(rng.permutation(16384)[:5000])
    s.extend(rng.integers(0, 200, 16384))
    s.same()


def test_extend_of_needs_that_add_up_beyond_32_bits():
    """1,100 sequences in rows of 2^21 pages, of which all but two ask for a whole row: 2.3e9 pages."""
    n, width = 1100, 1 << 21
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    lens, refs, granted = dev(np.zeros(n)), dev(np.zeros(100)), dev(np.full(n, 9))
    refs[[0, 3]] = 1
    add = np.full(n, width * 64)
    add[[0, 1]] = 65, 1
    m.kv_pages_extend(table, lens, refs, dev(add), granted=granted)
    assert granted.tolist() == [1, 1] + [0] * (n - 2) and lens.tolist() == [65, 1] + [0] * (n - 2)
    assert torch.nonzero(refs).flatten().tolist() == [0, 1, 2, 3, 4]
    assert table[0, :3].tolist() == [1, 2, -1] and table[1, :2].tolist() == [4, -1]
    table[0, :2] = table[1, 0] = -1
    assert int(table.max()) == int(table.min()) == -1


@pytest.mark.parametrize("layers,page_bytes", [(1, 16), (2, 33008)])
@pytest.mark.parametrize("pages", [7, 129, 700])
def test_compact(pages, layers, page_bytes):
    rng = np.random.default_rng(pages)
    lens = rng.integers(0, 130, max(1, pages // 4))
    s = State(lens, pages, page_bytes, layers, seed=pages)
    s.free(rng.permutation(len(lens))[:len(lens) // 3])
    s.compact()
    s.same()
    s.compact()                                                    # nothing is left to move
    s.same()


@pytest.mark.parametrize("lens", [[0, 0], [640]])
def test_compact_of_an_empty_and_of_a_full_pool(lens):
    s = State(lens, 10, seed=9)
    s.compact()
    s.same()


def test_compact_counts_entries_that_name_no_page_in_use():
    s = State([64, 64, 64], 9, seed=10)
    free = int(np.flatnonzero(s.refs == 0)[0])
    s.d_table[1, 0] = free
    s.d_table[2, 1] = 9
    m.kv_pages_compact(s.d_cache, s.d_table, s.d_refs, dev_status=s.status, layered=True)
    assert s.d_table[1, 0] == -1 and s.d_table[2, 1] == -1
    assert s.status.tolist() == [0, 2, 0, 0]


def test_compact_of_a_large_pool():
    rng = np.random.default_rng(11)
    s = State(rng.integers(0, 2000, 3000), 200000, page_bytes=16, seed=11)
    s.free(rng.permutation(3000)[:1500])
    s.fork([int(np.flatnonzero(s.lens)[0])] * 5, np.flatnonzero(s.lens == 0)[:5])
    s.compact()
    s.same()


@pytest.mark.parametrize("lens,layers,page_bytes", [([64 * 900], 2, 33008), ([0, 64 * 300, 5, 64 * 700 + 1], 3, 16400), ([64 * 9000], 1, 16)])
def test_compact_of_more_chunks_than_blocks(lens, layers, page_bytes):
    # several items a copy block, whose layers and chunks differ; a table much shorter than the pool
    s = State(lens, 30000 if page_bytes == 16 else 2000, page_bytes, layers, seed=13)
    s.compact()
    s.same()


def test_page_numbers_up_to_the_largest():
    """A pool of 2^31 - 1 pages of 16 bytes (34 GB): its last pages are found, moved and given out like any others."""
    n = (1 << 31) - 1
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB")
    cache = torch.empty((n, 16), dtype=torch.uint8, device="cuda")
    refs = torch.zeros(n, dtype=torch.int32, device="cuda")
    held = [5, 7, n - 130, n - 129, n - 3, n - 1]
    for i, p in enumerate(held):
        refs[p] = 1
        cache[p] = i + 1
    table, lens = dev(np.array([held + [-1], [-1] * 7])), dev([6 * 64 - 1, 0])
    remap, live = m.kv_pages_compact(cache, table, refs)
    assert live.item() == 6 and table[0].tolist() == [5, 0, 1, 2, 3, 4, -1]
    assert [cache[int(p), 0].item() for p in table[0, :6]] == [1, 2, 3, 4, 5, 6]
    assert remap[torch.tensor([5, 6, 7, n - 130, n - 129, n - 3, n - 2, n - 1], device="cuda")].tolist() == [5, -1, 0, 1, 2, 3, -1, 4]
    assert torch.nonzero(refs[:100]).flatten().tolist() == [0, 1, 2, 3, 4, 5] and not refs[n - 200:].any()
    del remap
    refs.fill_(1)
    refs[n - 1] = refs[n - 2] = 0
    new = m.kv_pages_fork(cache, table, lens, refs, dev([0]), dev([1]))
    assert new.tolist() == [n - 2] and cache[n - 2, 0] == 6 and refs[n - 2] == 1
    granted = dev([9, 9])
    m.kv_pages_extend(table, lens, refs, dev([1, 2]), granted=granted)
    assert granted.tolist() == [1, 1] and table[1].tolist() == [5, 0, 1, 2, 3, n - 2, n - 1] and lens.tolist() == [384, 385]
    del cache, refs
    torch.cuda.empty_cache()


def test_a_captured_step_replays_on_the_state_it_finds():
    s = State([100, 64, 1, 0, 0, 0], 40, seed=12)
    ended, src, dst, add = dev([-1]), dev([0]), dev([3]), dev(np.ones(6))
    new = torch.empty(1, dtype=torch.int32, device="cuda")
    remap, live = torch.empty(40, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(m.kv_pages_compact_workspace_size(40), dtype=torch.uint8, device="cuda")

    def step():
        m.kv_pages_free(s.d_table, s.d_lens, s.d_refs, ended)
        m.kv_pages_fork(s.d_cache, s.d_table, s.d_lens, s.d_refs, src, dst, new_pages=new, layered=True)
        m.kv_pages_extend(s.d_table, s.d_lens, s.d_refs, add)
        m.kv_pages_compact(s.d_cache, s.d_table, s.d_refs, remap=remap, num_live=live, workspace=ws, layered=True)

    def oracle(e, a, b):
        kv8.free(s.table, s.lens, s.refs, [e])
        kv8.fork(s.cache, s.table, s.lens, s.refs, [a], [b])
        kv8.extend(s.table, s.lens, s.refs, [1] * 6)
        kv8.compact(s.cache, s.table, s.refs)

    step()
    oracle(-1, 0, 3)
    s.same()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for e, a, b in ((1, 0, 1), (3, 2, 3), (0, 2, 0), (2, 0, 2)):
        ended.fill_(e)
        src.fill_(a)
        dst.fill_(b)
        g.replay()
        oracle(e, a, b)
        s.same()


@pytest.mark.parametrize("call", ["decode", "fork", "compact"])
def test_what_a_call_takes_on_another_stream_is_free_there(call):
    """A call on an idle stream, while the current one still has to write memory that it gave back before: neither
    results nor workspace of the call are that memory. Everything that the call could take is given back beforehand."""
    c = Case([2000, 900], 2, 128, Q=1, G=4, seed=31)
    args = (c.q, dev(c.cache, torch.uint8), dev(c.table), dev(c.lens), 2, c.scale)
    size = m.kv8_decode_workspace_size(2, 1, 8, 2, 128)
    want = m.kv8_decode(*args)
    x = torch.randn((4096, 4096), device="cuda")
    s = torch.cuda.Stream()
    src, dst = dev([0, 1]), dev([3, 4])
    for turn in range(3):
        p = State([100, 64, 1, 0, 0], 300, 4096, 2, seed=turn)
        torch.cuda.synchronize()
        blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (c.q.numel() * 2, c.q.numel(), size, 8, 1200, 4, 512, 2048) for _ in range(4)]
        for _ in range(20):
            x = x @ x * 1e-3                # some milliseconds before the blocks are written
        for block in blocks:
            block.fill_(255)
        del blocks, block
        if call == "decode":
            got = m.kv8_decode(*args, stream=s)
        elif call == "fork":
            got = m.kv_pages_fork(p.d_cache, p.d_table, p.d_lens, p.d_refs, src, dst, layered=True, stream=s)
        else:
            got = m.kv_pages_compact(p.d_cache, p.d_table, p.d_refs, layered=True, stream=s)
        s.synchronize()
        torch.cuda.synchronize()
        if call == "decode":
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            continue
        if call == "fork":
            assert got.tolist() == kv8.fork(p.cache, p.table, p.lens, p.refs, [0, 1], [3, 4])
        else:
            remap, n = kv8.compact(p.cache, p.table, p.refs)
            assert np.array_equal(got[0].cpu().numpy(), remap) and got[1].item() == n
        p.same()


def test_refusals_leave_everything_as_it_was():
    s = State([100, 64, 0], 40, seed=20)
    seqs, short = dev([0]), dev(np.zeros(3))
    misaligned = torch.zeros(41, dtype=torch.int32, device="cuda")[1:]
    ws = torch.empty(2 * m.kv_pages_compact_workspace_size(40), dtype=torch.uint8, device="cuda")
    calls = [lambda: m.kv_pages_copy(s.d_cache, seqs, seqs, dev_status=short, layered=True),
             lambda: m.kv_pages_copy(s.d_cache, seqs, seqs[:0], layered=True),
             lambda: m.kv_pages_copy(s.d_cache[:, ::2], seqs, seqs, layered=True),
             lambda: m.kv_pages_free(s.d_table, s.d_lens, s.d_refs, seqs, dev_status=short),
             lambda: m.kv_pages_free(s.d_table, s.d_lens[:2], s.d_refs, seqs),
             lambda: m.kv_pages_free(s.d_table, s.d_lens, misaligned, seqs),
             lambda: m.kv_pages_free(s.d_table.cpu(), s.d_lens, s.d_refs, seqs),
             lambda: m.kv_pages_fork(s.d_cache, s.d_table, s.d_lens, s.d_refs, seqs, seqs, dev_status=short, layered=True),
             lambda: m.kv_pages_fork(s.d_cache, s.d_table, s.d_lens, s.d_refs[:20], seqs, seqs, layered=True),
             lambda: m.kv_pages_fork(s.d_cache, s.d_table, s.d_lens, s.d_refs, seqs, dev([0, 1]), layered=True),
             lambda: m.kv_pages_extend(s.d_table, s.d_lens, s.d_refs, dev([1, 1, 1]), dev_status=short),
             lambda: m.kv_pages_extend(s.d_table, s.d_lens, s.d_refs, dev([1, 1])),
             lambda: m.kv_pages_extend(s.d_table, s.d_lens, s.d_refs, dev([1, 1, 1]), granted=dev([0])),
             lambda: m.kv_pages_compact(s.d_cache, s.d_table, s.d_refs, dev_status=short, layered=True),
             lambda: m.kv_pages_compact(s.d_cache, s.d_table, s.d_refs, workspace=ws[::2], layered=True),
             lambda: m.kv_pages_compact(s.d_cache, s.d_table, s.d_refs, workspace=ws[:100], layered=True),
             lambda: m.kv_pages_compact(s.d_cache, s.d_table, s.d_refs, workspace=ws[1:], layered=True),
             lambda: m.kv_pages_compact(s.d_cache, s.d_table, s.d_refs, remap=dev([0]), layered=True)]
    for i, call in enumerate(calls):
        with pytest.raises((ValueError, TypeError, m.NvFp4MlaError)):
            call()
            pytest.fail(f"call {i} was not refused")
    torch.cuda.synchronize()
    s.same()


@pytest.mark.parametrize("D,dtype", [(64, torch.float16), (128, torch.bfloat16)])
def test_a_server_runs_on_the_operators_alone(D, dtype):
    """Prompts, decode steps, forks that share pages, endings and a compaction: after each, the attention over
    the pages is that over what every sequence wrote."""
    rng = np.random.default_rng(D)
    S, Hk, H, pages = 6, 2, 6, 64
    table = torch.full((S, 8), -1, dtype=torch.int32, device="cuda")
    lens, refs = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (S, pages))
    cache = torch.full((pages, m.kv8_page_bytes(Hk, D)), 0xFF, dtype=torch.uint8, device="cuda")
    status = dev(np.zeros(4))
    plain = np.full((S * 8, kv8.page_bytes(Hk, D)), 0xFF, np.uint8)   # the oracle's cache: eight pages a sequence, nothing shared
    rows = np.arange(S * 8, dtype=np.int32).reshape(S, 8)
    held = np.zeros(S, np.int32)

    def grow(add):
        nonlocal held
        n = int(np.sum(add))
        k, v = (torch.from_numpy(rng.standard_normal((n, Hk, D)) * 2.0 ** rng.integers(-3, 4)).to(dtype) for _ in range(2))
        cu = np.concatenate([[0], np.cumsum(add)]).astype(np.int32)
        m.kv_pages_extend(table, lens, refs, dev(add), dev_status=status)
        m.kv8_append(k.to("cuda"), v.to("cuda"), dev(cu), lens, table, cache, dev_status=status)
        held = (held + add).astype(np.int32)
        kv8.append(plain, f64(k), f64(v), cu, held, rows, Hk, D)

    def attend():
        q = torch.from_numpy(rng.standard_normal((S, 1, H, D))).to(dtype)
        out, lse = m.kv8_decode(q.to("cuda"), cache, table, lens, Hk, D ** -0.5, dev_status=status)
        check(out, lse, kv8.decode(f64(q), plain, rows, held, Hk, D ** -0.5))

    def fork(src, dst):
        m.kv_pages_fork(cache, table, lens, refs, dev(src), dev(dst), dev_status=status)
        for a, b in zip(src, dst):
            plain[rows[b]] = plain[rows[a]]
            held[b] = held[a]

    def free(seqs):
        m.kv_pages_free(table, lens, refs, dev(seqs), dev_status=status)
        held[list(seqs)] = 0

    grow([130, 0, 64, 7, 0, 0])
    attend()
    for _ in range(3):
        grow([1, 0, 1, 1, 0, 0])
        attend()
    fork([0, 0, 2], [1, 4, 5])
    for _ in range(20):
        grow([1] * 6)
    attend()
    free([0, 3])
    m.kv_pages_compact(cache, table, refs, dev_status=status)
    attend()
    fork([1], [3])
    grow([200, 1, 1, 40, 1, 1])
    attend()
    assert np.array_equal(lens.cpu().numpy(), held) and status.tolist() == [0, 0, 0, 0]
    free(range(S))
    assert not refs.any()
