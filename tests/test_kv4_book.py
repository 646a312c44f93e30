"""The page book of the 4-bit KV cache (host only) and the refusals of its
calls that need no GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def g():
    from nvfp4_gated_deltanet_gb300 import build
    build.build()
    import nvfp4_gated_deltanet_gb300 as pkg
    return pkg


def consistent(book):
    held = [0] * book.num_pages
    for pages, n in book.seqs.values():
        assert len(pages) == -(-n // book.page_tokens) and len(set(pages)) == len(pages)
        for p in pages:
            held[p] += 1
    assert held == book.holders
    assert sorted(book._free) == [p for p in range(book.num_pages) if not held[p]]


def test_growth_fork_and_copy_on_write(g):
    b = g.KV4Book(8, 16)
    s = b.new()
    assert b.extend([s], [17]) == [] and b.pages(s) == [0, 1] and b.length(s) == 17
    t, u = b.fork(s), b.fork(s)
    consistent(b)
    assert b.free_pages == 6 and b.pages(t) == [0, 1]
    # all three grow at once: two leave the shared last page, the last one keeps it
    assert b.extend([s, t, u], [1, 1, 1]) == [(1, 2), (1, 3)]
    assert (b.pages(s), b.pages(t), b.pages(u)) == ([0, 2], [0, 3], [0, 1])
    consistent(b)
    b.truncate(t, 16)
    assert b.pages(t) == [0]
    assert b.extend([t], [1]) == []  # a full shared page is not copied
    b.truncate(t, 3)
    assert b.extend([t], [2]) == [(0, 3)]  # growing inside a shared page copies it
    assert b.extend([t], [0]) == []
    consistent(b)
    b.free(s)
    b.free(t)
    consistent(b)
    assert b.pages(u) == [0, 1]


def test_running_out_changes_nothing(g):
    b = g.KV4Book(3, 16)
    s, t = b.new(), b.new()
    b.extend([s, t], [16, 20])
    before = (b.holders[:], {k: [v[0][:], v[1]] for k, v in b.seqs.items()})
    with pytest.raises(MemoryError):
        b.extend([t, s], [3, 1])
    assert (b.holders, b.seqs) == before
    for bad in ([-1, 0], [1]):
        with pytest.raises(ValueError):
            b.extend([s, t], bad)
    with pytest.raises(ValueError):
        b.extend([s, s], [0, 0])
    with pytest.raises(ValueError):
        b.truncate(s, 17)
    consistent(b)


@pytest.mark.parametrize("seed", range(6))
def test_random_use_and_compaction(g, seed):
    import random
    rng = random.Random(seed)
    b = g.KV4Book(37, 16)
    b.new()
    for _ in range(300):
        ids = list(b.seqs)
        op = rng.choice(["new", "extend", "extend", "fork", "free", "truncate", "compact"])
        s = rng.choice(ids) if ids else None
        if op == "new" or s is None:
            b.new()
        elif op == "extend":
            some = rng.sample(ids, rng.randint(1, min(4, len(ids))))
            try:
                copies = b.extend(some, [rng.randint(0, 40) for _ in some])
                assert len({d for _, d in copies}) == len(copies)
                assert not {d for _, d in copies} & {x for x, _ in copies}
            except MemoryError:
                b.free(s)
        elif op == "fork" and len(ids) < 12:
            b.fork(s)
        elif op == "free":
            b.free(s)
        elif op == "truncate":
            b.truncate(s, rng.randint(0, b.length(s)))
        elif op == "compact":
            live = {p for p in range(b.num_pages) if b.holders[p]}
            old = {k: v[0][:] for k, v in b.seqs.items()}
            to = b.compact()
            assert {to[p] for p in live} == set(range(len(live)))
            assert all(to[p] == -1 for p in range(b.num_pages) if p not in live)
            assert all(to[p] == p for p in live if p < len(live))
            moved = [p for p in sorted(live) if p >= len(live)]
            assert [to[p] for p in moved] == sorted(to[p] for p in moved)
            assert all(v[0] == [to[p] for p in old[k]] for k, v in b.seqs.items())
        consistent(b)


GOOD = 0x10000  # never dereferenced: every call below fails its checks first


def cache(g, **kw):
    f = dict(pages=GOOD, num_pages=4, page_tokens=16, n_kv_heads=2, head_dim=128, k_scale=1.0, v_scale=1.0)
    f.update(kw)
    return ctypes.byref(g.Kv4CacheStruct(**f))


def batch(g, **kw):
    f = dict(kv_len=GOOD, block_table=GOOD, q_start=None, B=2, max_pages=2, T=2)
    f.update(kw)
    return ctypes.byref(g.Kv4BatchStruct(**f))


BAD = [("cache", dict(head_dim=96), 2), ("cache", dict(page_tokens=24), 2), ("cache", dict(page_tokens=512), 2),
       ("cache", dict(num_pages=0), 2), ("cache", dict(n_kv_heads=0), 2), ("cache", dict(k_scale=float("nan")), 4),
       ("cache", dict(v_scale=float("inf")), 4), ("cache", dict(k_scale=0.0), 5), ("cache", dict(v_scale=-1.0), 5),
       ("cache", dict(pages=None), 1), ("cache", dict(pages=GOOD + 8), 3), ("batch", dict(kv_len=None), 1),
       ("batch", dict(block_table=None), 1), ("batch", dict(block_table=GOOD + 2), 3), ("batch", dict(B=-1), 2),
       ("batch", dict(T=-1), 2), ("batch", dict(B=0), 2), ("batch", dict(T=3), 2), ("batch", dict(max_pages=0), 2),
       ("batch", dict(max_pages=2 ** 28), 7)]


@pytest.mark.parametrize("which,change,status", BAD)
def test_refusals_of_cache_and_batch(g, which, change, status):
    L = g.lib()
    c = cache(g, **(change if which == "cache" else {}))
    b = batch(g, **(change if which == "batch" else {}))
    big = 1 << 40
    assert L.kv4_append(c, b, GOOD, 256, GOOD, 256, None, None) == status
    assert L.kv4_read(c, b, GOOD, GOOD, None, None) == status
    assert L.kv4_decode(c, b, GOOD, 512, 4, 1.0, GOOD, GOOD, GOOD, big, None, None) == status
    assert L.kv4_prefill(c, b, 64, GOOD, 512, 4, 1.0, GOOD, GOOD, GOOD, big, None, None) == status


def test_refusals_of_the_calls(g):
    L, c, b = g.lib(), cache(g), batch(g)
    big = 1 << 40
    assert L.kv4_append(None, b, GOOD, 256, GOOD, 256, None, None) == 1
    assert L.kv4_append(c, None, GOOD, 256, GOOD, 256, None, None) == 1
    assert L.kv4_append(c, b, None, 256, GOOD, 256, None, None) == 1
    assert L.kv4_append(c, b, GOOD, 256, GOOD + 2, 256, None, None) == 3
    assert L.kv4_append(c, b, GOOD, 260, GOOD, 256, None, None) == 2    # not a multiple of 8
    assert L.kv4_append(c, b, GOOD, 256, GOOD, 128, None, None) == 2    # rows overlap
    assert L.kv4_read(c, b, GOOD, None, None, None) == 1
    assert L.kv4_read(c, b, GOOD + 4, GOOD, None, None) == 3

    def dec(q=GOOD, stride=512, hq=4, sm=1.0, out=GOOD, lse=GOOD, b=b):
        return L.kv4_decode(c, b, q, stride, hq, sm, out, lse, GOOD, big, None, None)

    def pre(q=GOOD, stride=512, hq=4, sm=1.0, out=GOOD, lse=GOOD, b=b):
        return L.kv4_prefill(c, b, 64, q, stride, hq, sm, out, lse, GOOD, big, None, None)

    for f in (dec, pre):
        assert f(q=None) == 1 and f(out=None) == 1
        assert f(q=GOOD + 2) == 3 and f(out=GOOD + 8) == 3 and f(lse=GOOD + 2) == 3
        assert f(hq=3) == 2 and f(hq=0) == 2 and f(hq=130, stride=130 * 128) == 2
        assert f(stride=504) == 2 and f(stride=516) == 2
        assert f(sm=float("nan")) == 4 and f(sm=0.0) == 5 and f(sm=-1.0) == 5
        assert f(b=batch(g, T=0)) == 0                                  # nothing to do
    assert dec(b=batch(g, q_start=GOOD)) == 2                           # decode rows are even
    assert L.kv4_prefill(c, b, -1, GOOD, 512, 4, 1.0, GOOD, None, GOOD, big, None, None) == 2
    for q_start in (None, GOOD):
        need = L.kv4_prefill_workspace(c, batch(g, q_start=q_start), 64, 4)
        if need:
            assert L.kv4_prefill(c, batch(g, q_start=q_start), 64, GOOD, 512, 4, 1.0, GOOD, None, GOOD, need - 1, None,
                                 None) == 2
    need = L.kv4_decode_workspace(c, b, 4)
    if need:
        assert L.kv4_decode(c, b, GOOD, 512, 4, 1.0, GOOD, None, GOOD, need - 1, None, None) == 2

    def copy(pages=GOOD, layers=2, stride=4096, num=4, size=1024, src=GOOD, dst=GOOD, n=3):
        return L.kv4_copy_pages(pages, layers, stride, num, size, src, dst, n, None, None)

    assert copy(pages=None) == 1 and copy(src=None) == 1 and copy(dst=None) == 1
    assert copy(pages=GOOD + 8) == 3 and copy(src=GOOD + 2) == 3
    assert copy(layers=0) == 2 and copy(size=24) == 2 and copy(n=-1) == 2 and copy(stride=4080) == 2
    assert copy(num=1 << 20, size=1 << 30, layers=1) == 7
    assert copy(n=0, src=None, dst=None) == 0

    def compact(num=4, rows=2, cols=2, table=GOOD, out=GOOD, pmap=GOOD, live=GOOD, ws=GOOD, nb=big, size=1024):
        return L.kv4_compact(GOOD, 1, 0, num, size, table, rows, cols, out, pmap, live, ws, nb, None, None)

    assert compact(table=None) == 1 and compact(out=None) == 1 and compact(pmap=None) == 1 and compact(live=None) == 1
    assert compact(ws=None) == 1 and compact(num=(1 << 20) + 1) == 2 and compact(rows=-1) == 2
    assert compact(nb=L.kv4_compact_workspace(4) - 1) == 2
    assert compact(table=GOOD + 2) == 3 and compact(ws=GOOD + 8) == 3
    assert compact(rows=1 << 16, cols=1 << 16) == 7


def test_python_refusals(g):
    import torch
    pages = torch.zeros(4, 2, 1, 18 * 128, dtype=torch.uint8)
    t = torch.zeros(2, 2, dtype=torch.int32)
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    n = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        g.kv4_decode(q, pages, t, n, 1.0, 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        g.kv4_append(q[:, :2], q[:, :2], pages, t, n, 1.0, 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        g.kv4_copy_pages(pages, n, n)
    with pytest.raises(ValueError, match="CUDA"):
        g.kv4_compact(pages, t)


@pytest.mark.parametrize("d", [64, 128])
def test_reference_forms_agree(d):
    """The tensor forms of the float64 reference equal the ones written token by token."""
    import numpy as np
    import torch
    import kv4_ref as ref
    rng = np.random.RandomState(d)
    pages = rng.randint(0, 256, (5, 2, 2, 18 * d)).astype(np.uint8)
    pages[..., 16 * d:] %= 120                       # finite positive scales
    row = np.array([3, 0, 4, 1], np.int32)
    for n, new in ((0, 2), (1, 3), (77, 5), (128, 1)):
        K, V = ref.cached(pages, row, n, d, 0.017, 0.013)
        Kt, Vt = ref.cached_torch(torch.from_numpy(pages), torch.from_numpy(row), n, d, 0.017, 0.013)
        assert np.array_equal(K, Kt.numpy()) and np.array_equal(V, Vt.numpy())
        q = rng.randn(new, 6, d) * 0.05
        for a, b in zip(ref.attention(q, K, V, 0.1), ref.attention_torch(torch.from_numpy(q), Kt, Vt, 0.1)):
            np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-12)


def test_every_layout_place_is_used_once():
    import numpy as np
    import kv4_ref as ref
    for d in (64, 128):
        at = np.concatenate([np.concatenate(ref.places(t, d)) for t in range(16)])
        assert np.array_equal(np.sort(at), np.arange(18 * d))
