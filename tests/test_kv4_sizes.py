"""The largest sizes of shared decode, scores and eviction: what a kernel's 31-bit places
could not count is refused on the host (nothing here reaches a device)."""
import ctypes

import pytest

pytest.importorskip("torch")
GOOD = 0x10000  # an address that no call reads
OVERFLOW = 7
MOST = 2 ** 31 - 1 - 2 ** 15


@pytest.fixture(scope="module")
def g():
    from nvfp4_gated_deltanet_gb300 import build
    build.build()
    import nvfp4_gated_deltanet_gb300 as pkg
    return pkg


def structs(g, max_pages=1, tokens=32, page=16):
    return (g.Kv4CacheStruct(pages=GOOD, num_pages=8, page_tokens=page, n_kv_heads=1, head_dim=64, k_scale=1.0, v_scale=1.0),
            g.Kv4BatchStruct(kv_len=GOOD, block_table=GOOD, q_start=None, B=1, max_pages=max_pages, T=1, zero_padding=0),
            g.Kv4ScoresStruct(in_=GOOD, out=GOOD, slots=None, n_slots=1, tokens=tokens),
            g.Kv4SharedStruct(group_start=GOOD, shared_len=GOOD, groups=1, max_shared=16))


@pytest.mark.parametrize("page", [16, 256])
def test_tables_of_nearly_two_to_the_31_tokens(g, page):
    L, ref = g.lib(), ctypes.byref
    c, b, s, h = structs(g, max_pages=MOST // page + 1, tokens=2 ** 31 - 1, page=page)
    assert L.kv4_score(ref(c), ref(b), GOOD, 64, 1, 1.0, GOOD, ref(s), None, GOOD, 1 << 40, None, None) == OVERFLOW
    assert L.kv4_decode_shared(ref(c), ref(b), ref(h), GOOD, 64, 1, 1.0, GOOD, None, GOOD, 1 << 60, None, None) == OVERFLOW
    assert L.kv4_decode_shared_workspace(ref(c), ref(b), ref(h), 1) == 0
    evict = lambda s, most: L.kv4_evict(ref(c), 1, 0, ref(b), GOOD, 0, ref(s), 0, GOOD, 2, GOOD, most, GOOD, None, None)
    assert evict(s, 16) == OVERFLOW


def test_kept_places_of_nearly_two_to_the_31(g):
    L, ref = g.lib(), ctypes.byref
    c, b, s, _ = structs(g)
    for most in (MOST + 1, 2 ** 31 - 1):
        assert L.kv4_evict(ref(c), 1, 0, ref(b), GOOD, 0, ref(s), 0, GOOD, 2, GOOD, most, GOOD, None, None) == OVERFLOW
