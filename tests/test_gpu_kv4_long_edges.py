"""Shared decode, scores and eviction of the 4-bit KV cache where calls meet: streams,
launches that overlap, rows and members that count for nothing."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if torch.cuda.is_available():
    from kv4_inputs import KS, VS, attention, close, ints, prefixed, queries, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import nvfp4_gated_deltanet_gb300 as pkg
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return pkg


def rows(T, heads, d, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(T, heads, d, generator=gen, device="cuda").bfloat16()


def test_kept_places_dropped_while_the_current_stream_reads_them(g):
    """What an eviction on another stream returned is read on the current one and dropped: the other stream's next
    tensors do not overwrite it meanwhile."""
    c = g.KV4Cache(600, 16, 2, 64, KS, VS, score_slots=6, score_tokens=600)
    seqs = [c.new() for _ in range(6)]
    batch = c.grow(seqs, 600)
    c.append(0, rows(3600, 2, 64, 1), rows(3600, 2, 64, 2), batch)
    q = queries(3600, 4, 64, 3)
    c.score(0, q, c.prefill(0, q, batch, return_lse=True)[1], batch)
    big = torch.randn(4096, 4096, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, most = [], []
    for s in seqs:
        side.wait_stream(torch.cuda.current_stream())
        kept = c.evict([s], 256, recent=16, stream=side)[1]
        torch.cuda.current_stream().wait_stream(side)
        for _ in range(10):
            big @ big
        got.append(kept + 0)
        most.append(kept.shape)
        del kept
        with torch.cuda.stream(side):
            torch.full(most[-1], -7, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert c.check() == 0
    for x in got:
        assert (x[..., 240:] == torch.arange(584, 600, device="cuda")).all() and (x >= 0).all() and (x.diff(dim=-1) > 0).all()
