"""The workspaces of the 4-bit KV cache's attention calls: their sizes, and
what is refused (host only: every call fails its checks before it launches)."""
import pytest

from test_kv4_book import GOOD, batch, cache


@pytest.fixture(scope="module")
def g():
    from nvfp4_gated_deltanet_gb300 import build
    build.build()
    import nvfp4_gated_deltanet_gb300 as pkg
    return pkg


@pytest.mark.parametrize("hq", [0, -4, 3, 130])
def test_no_workspace_for_heads_that_the_calls_refuse(g, hq):
    L, c, b = g.lib(), cache(g), batch(g, max_pages=4096)
    assert L.kv4_decode_workspace(c, b, 4) > 0 and L.kv4_prefill_workspace(c, b, 64, 4) > 0
    assert L.kv4_decode_workspace(c, b, hq) == 0 and L.kv4_prefill_workspace(c, b, 64, hq) == 0
    stride = 128 * max(hq, 8)
    assert L.kv4_decode(c, b, GOOD, stride, hq, 1.0, GOOD, None, GOOD, 1 << 40, None, None) == 2
    assert L.kv4_prefill(c, b, 64, GOOD, stride, hq, 1.0, GOOD, None, GOOD, 1 << 40, None, None) == 2


@pytest.mark.parametrize("head_dim,hq,T", [(128, 4, 2), (64, 32, 8), (128, 128, 2)])
def test_decode_refuses_a_workspace_that_is_too_small(g, head_dim, hq, T):
    L, c, b = g.lib(), cache(g, head_dim=head_dim), batch(g, max_pages=4096, T=T)
    need = L.kv4_decode_workspace(c, b, hq)
    assert need > 0
    for have in (0, need - 1):
        assert L.kv4_decode(c, b, GOOD, head_dim * hq, hq, 1.0, GOOD, None, GOOD, have, None, None) == 2
    assert L.kv4_decode(c, b, GOOD, head_dim * hq, hq, 1.0, GOOD, None, None, need, None, None) == 1
    assert L.kv4_decode(c, b, GOOD, head_dim * hq, hq, 1.0, GOOD, None, GOOD + 8, need, None, None) == 3
    need = L.kv4_prefill_workspace(c, batch(g, max_pages=4096, T=T, q_start=GOOD), 1000, hq)
    assert need > 0
    for have in (0, need - 1):
        assert L.kv4_prefill(c, batch(g, max_pages=4096, T=T, q_start=GOOD), 1000, GOOD, head_dim * hq, hq, 1.0, GOOD, None,
                             GOOD, have, None, None) == 2
