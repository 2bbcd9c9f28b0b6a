"""Host-side checks of the 8-bit cache's and the page operators' entry points, and the binding's (CPU only)."""
import ctypes

import numpy as np
import pytest
import torch

import nvfp4_compressed_sparse_gb300 as m
from oracle import kv8

OK, INVALID, ALIGN, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4
A = 1 << 20     # a well aligned address that is nothing: every call is refused before it is used


@pytest.fixture(scope="module")
def lib():
    return m.load_library()


def P(x):
    return ctypes.c_void_p(x) if x else None


def test_page_bytes(lib):
    for hk in (1, 2, 3, 8, 256):
        for d in (64, 128):
            assert lib.kv8_page_bytes(hk, d) == kv8.page_bytes(hk, d)
    for hk, d in ((0, 64), (257, 64), (1, 32), (1, 96), (1, 256), (-1, 128)):
        assert lib.kv8_page_bytes(hk, d) == 0
        with pytest.raises(ValueError):
            m.kv8_page_bytes(hk, d)


def append(lib, k=A, kt=256, kh=128, v=A, vt=256, vh=128, dt=0, n=4, cu=A, sl=A, pt=A, mp=4, B=2, hk=2, d=128, cache=A, pages=5, st=0):
    return lib.kv8_append(P(k), kt, kh, P(v), vt, vh, dt, n, P(cu), P(sl), P(pt), mp, B, hk, d, P(cache), pages, P(st), None)


def test_append_checks(lib):
    for kw in (dict(n=-1), dict(B=-1), dict(mp=0), dict(pages=0), dict(pages=1 << 31), dict(hk=0), dict(hk=257), dict(d=96), dict(dt=2),
               dict(dt=-1), dict(kt=-8), dict(vh=-8), dict(k=0), dict(v=0), dict(cu=0), dict(sl=0), dict(pt=0), dict(cache=0), dict(n=1 << 31)):
        assert append(lib, **kw) == INVALID, kw
    for kw in (dict(k=A + 8), dict(v=A + 2), dict(cache=A + 64), dict(kt=257), dict(vt=4), dict(kh=129), dict(vh=2), dict(cu=A + 2),
               dict(sl=A + 1), dict(pt=A + 3), dict(st=A + 2)):
        assert append(lib, **kw) == ALIGN, kw
    assert append(lib, n=0) == OK and append(lib, B=0) == OK
    assert append(lib) == INVALID                       # addresses that are no device memory
    host = np.zeros(1 << 16, np.uint8)
    at = (host.ctypes.data + 255) // 256 * 256
    assert append(lib, k=at, v=at, cu=at, sl=at, pt=at, cache=at) == INVALID and not host.any()


def decode(lib, q=A, qt=512, qh=128, dt=0, cache=A, pages=5, pt=A, mp=4, sl=A, B=2, Q=1, H=4, hk=2, d=128, scale=0.1, w=0, out=A, lse=A,
           ws=A, wb=1 << 40, st=0, flags=0):
    return lib.kv8_decode(P(q), qt, qh, dt, P(cache), pages, P(pt), mp, P(sl), B, Q, H, hk, d, scale, w, P(out), P(lse), P(ws), wb, P(st),
                          flags, None)


def test_decode_checks(lib):
    for kw in (dict(B=0), dict(Q=0), dict(Q=17), dict(H=0), dict(H=5), dict(H=258), dict(hk=0), dict(d=192), dict(dt=3), dict(pages=0),
               dict(pages=(1 << 31) - 1), dict(mp=0), dict(w=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(qt=-8), dict(qh=-8), dict(q=0), dict(cache=0), dict(pt=0), dict(sl=0), dict(out=0), dict(lse=0)):
        assert decode(lib, **kw) == INVALID, kw
    for kw in (dict(q=A + 8), dict(out=A + 4), dict(cache=A + 16), dict(qt=4), dict(qh=100), dict(pt=A + 1), dict(sl=A + 2), dict(lse=A + 2),
               dict(st=A + 1)):
        assert decode(lib, **kw) == ALIGN, kw


def test_decode_workspace_size(lib):
    assert lib.kv8_decode_workspace_size(2, 1, 8, 2, 128, 152) > 0
    # the partial results are the schedule's, not the batch's
    assert lib.kv8_decode_workspace_size(1, 1, 8, 2, 128, 152) == lib.kv8_decode_workspace_size(4096, 1, 8, 2, 128, 152)
    for bad in ((0, 1, 8, 2, 128), (1, 0, 8, 2, 128), (1, 17, 8, 2, 128), (1, 1, 7, 2, 128), (1, 1, 8, 2, 100), (1, 1, 8, 0, 128), (1, 1, 258, 2, 64)):
        assert lib.kv8_decode_workspace_size(*bad, 152) == 0


def test_page_operator_checks(lib):
    def copy(cache=A, layers=1, stride=0, pages=4, each=64, src=A, dst=A, n=2, st=0):
        return lib.kv_pages_copy(P(cache), layers, stride, pages, each, P(src), P(dst), n, P(st), None)
    for kw in (dict(cache=0), dict(layers=0), dict(layers=2, stride=255), dict(pages=0), dict(each=0), dict(n=-1), dict(each=1 << 62, pages=4)):
        assert copy(**kw) == INVALID, kw
    for kw in (dict(cache=A + 8), dict(each=24), dict(layers=2, stride=264)):
        assert copy(**kw) == ALIGN, kw
    assert copy() == INVALID

    def state(f, pt=A, mp=4, sl=A, S=3, rc=A, pages=4, x=A, n=2, st=0):
        if f == "free":
            return lib.kv_pages_free(P(pt), mp, P(sl), S, P(rc), pages, P(x), n, P(st), None)
        return lib.kv_pages_extend(P(pt), mp, P(sl), S, P(rc), pages, P(x), None, P(st), None)
    for f in ("free", "extend"):
        for kw in (dict(pt=0), dict(mp=0), dict(sl=0), dict(S=0), dict(rc=0), dict(pages=0)):
            assert state(f, **kw) == INVALID, (f, kw)
        for kw in (dict(pt=A + 2), dict(sl=A + 1), dict(rc=A + 4), dict(st=A + 2)):
            assert state(f, **kw) == ALIGN, (f, kw)
        assert state(f) == INVALID
    assert state("free", n=-1) == INVALID
    assert state("extend", S=16385) == INVALID

    def fork(n=2, **kw):
        a = dict(cache=A, layers=1, stride=0, pages=4, each=64, pt=A, mp=4, sl=A, S=3, rc=A, src=A, dst=A, new=A) | kw
        return lib.kv_pages_fork(P(a["cache"]), a["layers"], a["stride"], a["pages"], a["each"], P(a["pt"]), a["mp"], P(a["sl"]), a["S"],
                                 P(a["rc"]), P(a["src"]), P(a["dst"]), n, P(a["new"]), None, None)
    assert fork(n=-1) == INVALID and fork(n=16385) == INVALID and fork(cache=0) == INVALID and fork() == INVALID
    assert fork(cache=A + 8) == ALIGN

    def compact(wb=1 << 30, **kw):
        a = dict(cache=A, pages=4, each=64, pt=A, mp=4, S=3, rc=A, remap=A, live=A, ws=A) | kw
        return lib.kv_pages_compact(P(a["cache"]), 1, 0, a["pages"], a["each"], P(a["pt"]), a["mp"], a["S"], P(a["rc"]), P(a["remap"]),
                                    P(a["live"]), P(a["ws"]), wb, None, None)
    assert compact(cache=0) == INVALID and compact() == INVALID and compact(each=8) == INVALID and compact(cache=A + 4) == ALIGN
    assert lib.kv_pages_compact_workspace_size(0) == 0 and lib.kv_pages_compact_workspace_size(1 << 31) == 0
    for n in (1, 2, 3, 1001):
        assert lib.kv_pages_compact_workspace_size(n) >= 4 * (2 * (n // 2) + 1)


def test_binding_refuses_before_the_library():
    cpu = torch.zeros
    k = cpu((3, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        m.kv8_append(k.float(), k.float(), None, None, None, None)
    with pytest.raises(ValueError):
        m.kv8_append(k, k, None, None, None, None)              # not on the device
    with pytest.raises(TypeError):
        m.kv8_decode(k.float()[None], None, None, None, 2, 1.0)
    with pytest.raises(ValueError):
        m.kv8_decode(k[None], None, None, None, 2, 1.0)
    c, i = cpu((4, 64), dtype=torch.uint8), cpu(3, dtype=torch.int32)
    for call in (lambda: m.kv_pages_copy(c, i, i), lambda: m.kv_pages_free(i[None], i, i, i), lambda: m.kv_pages_extend(i[None], i, i, i),
                 lambda: m.kv_pages_fork(c, i[None], i, i, i, i), lambda: m.kv_pages_compact(c, i[None], i)):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ the oracle itself
def test_oracle_append_then_decode_is_plain_attention_of_the_rounded_rows():
    rng = np.random.default_rng(0)
    Hk, D, n = 2, 64, 50
    k, v = rng.standard_normal((2, n, Hk, D))
    cache = np.zeros((2, kv8.page_bytes(Hk, D)), np.uint8)
    assert kv8.append(cache, k, v, [0, n], [n], np.array([[1, 0]]), Hk, D) == [0, 0]
    kk, vv, have = kv8.rows(cache, [1, 0], n, Hk, D)
    assert have.all()
    assert np.abs(kk - k.transpose(1, 0, 2)).max() <= 2.0 ** -4 * np.abs(k).max()
    assert np.all(np.abs(vv - v.transpose(1, 0, 2)) <= 2.0 ** -4 * np.abs(v.transpose(1, 0, 2)) + 2.0 ** -9 * np.abs(v).max() / 224)
    q = rng.standard_normal((1, 1, 4, D))
    out, lse, mass, reach, spread = kv8.decode(q, cache, np.array([[1, 0]]), [n], Hk, 0.125)
    z = np.einsum("hd,hnd->hn", q[0, 0], kk.repeat(2, 0)) * 0.125
    p = np.exp(z) / np.exp(z).sum(1, keepdims=True)
    assert np.allclose(out[0, 0], np.einsum("hn,hnd->hd", p, vv.repeat(2, 0)), atol=1e-12)
    assert np.allclose(lse[0, 0], np.log(np.exp(z).sum(1)), atol=1e-12)
    assert (mass >= np.abs(out) - 1e-12).all() and (reach[0, 0] >= np.abs(z).max(1) - 1e-12).all()
    assert (spread >= mass - 1e-12).all()


def test_oracle_scale_byte():
    assert kv8.scale_byte(0.0) == 1 and kv8.scale_byte(448.0) == 127 and kv8.scale_byte(448.1) == 128
    assert kv8.scale_byte(224.0) == 126 and kv8.scale_byte(2.0 ** 127 * 1.99) == 247


def test_oracle_pages():
    table = np.full((4, 3), -1, np.int32)
    lens, refs = np.zeros(4, np.int32), np.zeros(8, np.int32)
    cache = np.arange(8, dtype=np.uint8)[None, :, None].repeat(16, 2)
    assert kv8.extend(table, lens, refs, [70, 64, 0, 0]) == [1] * 4
    assert table[0].tolist() == [0, 1, -1] and table[1].tolist() == [2, -1, -1]
    assert kv8.fork(cache, table, lens, refs, [0, 1], [2, 3]) == [3, -1]
    assert table[2].tolist() == [0, 3, -1] and refs.tolist() == [2, 1, 2, 1, 0, 0, 0, 0] and cache[0, 3, 0] == 1
    kv8.free(table, lens, refs, [0])
    remap, n = kv8.compact(cache, table, refs)
    assert n == 3 and remap.tolist() == [0, -1, 2, 1, -1, -1, -1, -1] and table[2].tolist() == [0, 1, -1]
