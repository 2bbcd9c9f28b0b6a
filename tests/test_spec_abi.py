"""Host-side checks of the speculative step's entry points and the binding's, and the oracle's own properties (CPU only)."""
import ctypes

import numpy as np
import pytest
import torch

import nvfp4_compressed_sparse_gb300 as m
from oracle import kv8, spec

OK, INVALID, ALIGN, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4
A = 1 << 20     # a well aligned address that is nothing: every call is refused before it is used


@pytest.fixture(scope="module")
def lib():
    return m.load_library()


def P(x):
    return ctypes.c_void_p(x) if x else None


def rope(lib, q=A, qt=512, qh=128, k=A, kt=256, kh=128, v=A, vt=256, vh=128, dt=0, n=4, cu=A, sl=A, pt=A, mp=4, B=2, H=4, hk=2, d=128,
         qw=0, kw=0, eps=1e-6, cs=A, positions=100, rot=128, inter=0, at=0, step=0, sections=None, axes=1, out=A, ot=512, oh=128, cache=A,
         pages=5, st=0):
    parts = (ctypes.c_int32 * len(sections))(*sections) if sections is not None else None
    return lib.kv8_append_rope(P(q), qt, qh, P(k), kt, kh, P(v), vt, vh, dt, n, P(cu), P(sl), P(pt), mp, B, H, hk, d, P(qw), P(kw), eps,
                               P(cs), positions, rot, inter, P(at), step, parts, axes, P(out), ot, oh, P(cache), pages, P(st), None)


def test_rope_checks(lib):
    for kw in (dict(n=-1), dict(B=-1), dict(mp=0), dict(pages=0), dict(H=0), dict(H=1 << 20), dict(hk=0), dict(d=96), dict(dt=2), dict(dt=-1),
               dict(qt=-8), dict(oh=-8), dict(vt=-8), dict(step=-1), dict(q=0), dict(k=0), dict(v=0), dict(out=0), dict(cs=0), dict(cu=0),
               dict(sl=0), dict(pt=0), dict(cache=0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(positions=0),
               dict(positions=1 << 31), dict(rot=0), dict(rot=8), dict(rot=24), dict(rot=144), dict(d=64, rot=128), dict(axes=0), dict(axes=5),
               dict(axes=2, sections=[32, 32]), dict(axes=2, at=A), dict(axes=2, at=A, sections=[32, 31]), dict(axes=2, at=A, sections=[65, -1]),
               dict(axes=3, at=A, sections=[1 << 30, 1 << 30, 1 << 30])):
        assert rope(lib, **kw) == INVALID, kw
    for kw in (dict(q=A + 8), dict(out=A + 8), dict(k=A + 8), dict(qw=A + 8), dict(kw=A + 4), dict(cache=A + 64), dict(qt=4), dict(oh=12),
               dict(cs=A + 2), dict(at=A + 2), dict(cu=A + 2), dict(st=A + 1)):
        assert rope(lib, **kw) == ALIGN, kw
    assert rope(lib, n=0) == OK and rope(lib, B=0) == OK
    assert rope(lib, axes=3, at=A, sections=[0, 64, 0]) == INVALID     # addresses that are no device memory


def tree(lib, q=A, qt=512, qh=128, dt=0, cache=A, pages=5, pt=A, mp=4, sl=A, masks=A, B=2, Q=8, H=4, hk=2, d=128, scale=0.1, w=0, out=A,
         lse=A, ws=A, wb=1 << 40, st=0):
    return lib.kv8_decode_tree(P(q), qt, qh, dt, P(cache), pages, P(pt), mp, P(sl), P(masks), B, Q, H, hk, d, scale, w, P(out), P(lse), P(ws),
                               wb, P(st), 0, None)


def test_tree_checks(lib):
    for kw in (dict(B=0), dict(Q=0), dict(Q=65), dict(H=0), dict(H=5), dict(H=258), dict(hk=0), dict(d=192), dict(dt=2), dict(pages=0), dict(mp=0),
               dict(w=-1), dict(scale=0.0), dict(scale=float("nan")), dict(qt=-8), dict(q=0), dict(cache=0), dict(pt=0), dict(sl=0), dict(masks=0),
               dict(out=0), dict(lse=0)):
        assert tree(lib, **kw) == INVALID, kw
    for kw in (dict(q=A + 8), dict(out=A + 4), dict(cache=A + 16), dict(qt=4), dict(qh=100), dict(masks=A + 4), dict(lse=A + 2), dict(st=A + 1)):
        assert tree(lib, **kw) == ALIGN, kw
    assert tree(lib, w=7) == UNSUPPORTED                # a window that could leave out drafts
    size = lib.kv8_decode_tree_workspace_size
    assert size(2, 8, 8, 2, 128, 152) > 0 and size(1, 64, 256, 2, 64, 152) > 0
    for bad in ((0, 1, 8, 2, 128), (1, 65, 8, 2, 128), (1, 1, 7, 2, 128), (1, 1, 8, 2, 100), (1, 1, 258, 2, 64)):
        assert size(*bad, 152) == 0


def verify(lib, logits=A, ls=100, dt=2, probs=0, ps=100, drafts=A, parents=A, u=A, t=0, B=2, Q=5, V=100, tokens=A, path=A, acc=A, ws=A,
           wb=1 << 40, st=0):
    return lib.spec_verify(P(logits), ls, dt, P(probs), ps, P(drafts), P(parents), P(u), P(t), B, Q, V, P(tokens), P(path), P(acc), P(ws), wb,
                           P(st), None)


def test_verify_checks(lib):
    for kw in (dict(B=0), dict(Q=0), dict(Q=65), dict(V=0), dict(V=(1 << 24) + 1), dict(dt=3), dict(dt=-1), dict(ls=-1), dict(ps=-1), dict(logits=0),
               dict(drafts=0), dict(parents=0), dict(u=0), dict(tokens=0), dict(path=0), dict(acc=0)):
        assert verify(lib, **kw) == INVALID, kw
    for kw in (dict(logits=A + 2), dict(logits=A + 1, dt=0), dict(probs=A + 2), dict(drafts=A + 1), dict(u=A + 2), dict(t=A + 2), dict(ws=A + 128),
               dict(acc=A + 2), dict(st=A + 2)):
        assert verify(lib, **kw) == ALIGN, kw
    need = lib.spec_verify_workspace_size(2, 5, 100)
    assert verify(lib, ws=0) == WORKSPACE and verify(lib, wb=need - 1) == WORKSPACE and verify(lib, wb=need) == INVALID
    assert lib.spec_verify_workspace_size(2, 65, 100) == lib.spec_verify_workspace_size(0, 5, 100) == 0
    assert verify(lib, B=(1 << 28), Q=1, V=1, wb=1 << 60) == UNSUPPORTED     # a cluster of eight each
    assert verify(lib, logits=A + 2, dt=1) == INVALID   # two-byte logits may begin there: addresses that are no device memory


def keep(lib, cache=A, layers=1, stride=0, pages=5, pt=A, mp=4, sl=A, path=A, acc=A, B=2, Q=8, hk=2, d=128, new=A, st=0):
    return lib.kv8_keep(P(cache), layers, stride, pages, P(pt), mp, P(sl), P(path), P(acc), B, Q, hk, d, P(new), P(st), None)


def test_keep_and_trim_checks(lib):
    each = lib.kv8_page_bytes(2, 128)
    for kw in (dict(cache=0), dict(layers=0), dict(layers=2, stride=5 * each - 16), dict(pages=0), dict(pt=0), dict(mp=0), dict(sl=0), dict(path=0),
               dict(acc=0), dict(B=-1), dict(Q=0), dict(Q=65), dict(hk=0), dict(d=32), dict(new=0)):
        assert keep(lib, **kw) == INVALID, kw
    for kw in (dict(cache=A + 64), dict(layers=2, stride=5 * each + 8), dict(pt=A + 2), dict(path=A + 1), dict(acc=A + 2), dict(new=A + 2), dict(st=A + 3)):
        assert keep(lib, **kw) == ALIGN, kw
    assert keep(lib, B=0) == OK and keep(lib) == INVALID

    def trim(pt=A, mp=4, sl=A, seqs=3, rc=A, pages=9, new=A, st=0):
        return lib.kv_pages_trim(P(pt), mp, P(sl), seqs, P(rc), pages, P(new), P(st), None)
    for kw in (dict(pt=0), dict(mp=0), dict(sl=0), dict(seqs=0), dict(rc=0), dict(pages=0), dict(new=0)):
        assert trim(**kw) == INVALID, kw
    for kw in (dict(pt=A + 2), dict(rc=A + 4), dict(new=A + 1), dict(st=A + 2)):
        assert trim(**kw) == ALIGN, kw
    assert trim() == INVALID


def test_binding_refuses():
    """Shapes, types and strides that the binding can see, before anything touches a device."""
    bf = torch.bfloat16
    q, k = torch.zeros((4, 4, 64), dtype=bf), torch.zeros((4, 2, 64), dtype=bf)
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    cache = torch.zeros((3, m.kv8_page_bytes(2, 64)), dtype=torch.uint8)
    sheet = torch.zeros((10, 64))
    with pytest.raises((TypeError, ValueError)):        # tensors on the CPU
        m.kv8_append_rope(q, k, k, sheet, i32(2), i32(1), i32(1, 2), cache)
    with pytest.raises(TypeError):
        m.kv8_append_rope(q.float(), k, k, sheet, i32(2), i32(1), i32(1, 2), cache)
    with pytest.raises((TypeError, ValueError)):
        m.kv8_decode_tree(q[None], cache, i32(1, 2), i32(1), torch.zeros((1, 4), dtype=torch.int64), 2, 0.1)
    with pytest.raises(TypeError):
        m.spec_verify(torch.zeros((1, 2, 9), dtype=torch.float64), i32(1, 2), i32(1, 2), torch.zeros((1, 2)))
    with pytest.raises((TypeError, ValueError)):
        m.spec_verify(torch.zeros((1, 2, 9)), i32(1, 2), i32(1, 2), torch.zeros((1, 2)))
    with pytest.raises((TypeError, ValueError)):
        m.kv8_keep(cache, i32(1, 2), i32(1), i32(1, 4), i32(1), 2, 64)
    with pytest.raises((TypeError, ValueError)):
        m.kv_pages_trim(i32(1, 2), i32(1), i32(8), i32(1))


# ------------------------------------------------------------------ the oracle
def test_oracle_walk_draws_from_the_target():
    """Any tree, with and without the drafts' distributions: the first token's frequencies over 40,000 walks are the target's."""
    rng = np.random.default_rng(1)
    V, B = 4, 40000
    row, q = rng.standard_normal(V), rng.dirichlet(np.ones(V))
    p = spec.softmax(row, 0.8)
    for probs in (False, True):
        drafts = rng.choice(V, (B, 3), p=q) if probs else np.tile([0, 2, 1], (B, 1))
        got = spec.verify(np.tile(row, (B, 3, 1)), drafts, np.tile([-1, 0, 0], (B, 1)), rng.random((B, 3)), np.full(B, 0.8),
                          np.tile(q, (B, 3, 1)) if probs else None)[0][:, 0]
        share = np.bincount(got, minlength=V) / B
        assert np.all(np.abs(share - p) <= 5 * np.sqrt(p * (1 - p) / B))


def test_oracle_tree_of_a_chain_is_its_decode():
    rng = np.random.default_rng(2)
    cache = np.zeros((4, kv8.page_bytes(2, 64)), np.uint8)
    table = np.array([[2, 0], [1, -1]], np.int32)
    lens = np.array([100, 40])
    kv8.append(cache, rng.standard_normal((140, 2, 64)), rng.standard_normal((140, 2, 64)), [0, 100, 140], lens, table, 2, 64)
    q = rng.standard_normal((2, 3, 4, 64))
    masks = np.tile(np.array([1, 3, 7], np.uint64), (2, 1))
    for window in (0, 3, 50):
        a, b = spec.decode_tree(q, cache, table, lens, masks, 2, 0.1, window), kv8.decode(q, cache, table, lens, 2, 0.1, window)
        assert all(np.array_equal(x, y) for x, y in zip(a[:5], b))


def test_oracle_rotation_keeps_products():
    """A rotation by the same angle leaves a query's product with a key; by different ones it depends on their difference."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((2, 1, 64))
    angle = np.arange(50)[:, None] * 100.0 ** (-np.arange(32) / 32)
    sheet = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    for inter in (False, True):
        got = []
        for a, b in ((0, 0), (7, 7), (3, 10), (20, 27)):
            y = spec.rotate(x, None, 0, sheet, [[a, b]], [32], inter)[0]
            got.append(float(y[0, 0] @ y[1, 0]))
        assert np.isclose(got[0], got[1], rtol=1e-12) and np.isclose(got[2], got[3], rtol=1e-12)
