"""Which tokens KV4Cache takes to have a score, layer by layer, without a GPU: what it
hands to kv4_score, and when it refuses to evict."""
import contextlib
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def made(monkeypatch):
    """make(**kw): a cache on the CPU, and its device calls written down instead of made."""
    from nvfp4_gated_deltanet_gb300 import build
    build.build()
    import nvfp4_gated_deltanet_gb300 as g
    from nvfp4_gated_deltanet_gb300 import kv4

    def make(n_layers=2, **kw):
        c = g.KV4Cache(64, 16, 2, 64, 1.0, 1.0, n_layers=n_layers, device="cpu", **{**dict(score_slots=3, score_tokens=200), **kw})
        monkeypatch.setattr(c, "_dev", lambda rows: torch.tensor(rows, dtype=torch.int32))
        calls = []
        for name in ("kv4_score", "kv4_copy_pages"):
            monkeypatch.setattr(kv4, name, lambda *a, name=name, **k: calls.append((name, a, k)))

        def evict(*a, **k):
            calls.append(("kv4_evict", a, k))
            return torch.zeros(n_layers, a[2].shape[0], 2, k["max_keep"], dtype=torch.int32), None

        monkeypatch.setattr(kv4, "kv4_evict", evict)
        return c, calls

    return make


def rows(n):
    return torch.zeros(n, 4, 64, dtype=torch.bfloat16), torch.zeros(n, 4)


def test_evict_wants_every_layer_scored(made):
    c, calls = made(n_layers=3)
    a = c.new()
    batch = c.grow([a], 50)
    for layers in ((), (0,), (-1, 0)):                  # one layer at least has none
        for l in layers:
            c.score(l, *rows(50), batch)
        with pytest.raises(ValueError, match="no score"):
            c.evict([a], 20, recent=4)
    c.score(1, *rows(50), batch)
    assert c.evict([a], 20, recent=4)[0] == [a]
    # a step that a layer did not score: as long as it lies within what is kept anyway
    batch = c.grow([a], 3)
    c.score(0, *rows(3), batch)
    c.score(2, *rows(3), batch)
    with pytest.raises(ValueError, match="3 tokens have no score"):
        c.evict([a], 10, recent=2)
    assert c.evict([a], 10, recent=3)[0] == [a]


def test_a_used_slot_counts_for_nothing(made):
    c, _ = made(score_slots=1)
    a = c.new()
    batch = c.grow([a], 50)
    for l in range(2):
        c.score(l, *rows(50), batch)
    c.free(a)
    b = c.new()
    batch = c.grow([b], 50)
    c.score(0, *rows(50), batch)
    with pytest.raises(ValueError, match="no score"):
        c.evict([b], 20)


def test_a_score_that_fails_counts_for_nothing(made, monkeypatch):
    from nvfp4_gated_deltanet_gb300 import kv4
    c, _ = made()
    a = c.new()
    batch = c.grow([a], 50)
    c.score(0, *rows(50), batch)

    def fails(*a, **k):
        raise RuntimeError("launch")

    with monkeypatch.context() as m:
        m.setattr(kv4, "kv4_score", fails)
        with pytest.raises(RuntimeError):
            c.score(1, *rows(50), batch)
    with pytest.raises(ValueError, match="no score"):
        c.evict([a], 20)
    c.score(1, *rows(50), batch)
    c.evict([a], 20)


def test_each_layer_goes_on_from_its_own(made):
    """Forks, truncation and eviction keep each layer's count."""
    c, calls = made()
    a = c.new()
    batch = c.grow([a], 50)
    c.score(0, *rows(50), batch)
    c.score(1, *rows(50), batch)
    batch = c.grow([a], 6)
    c.score(1, *rows(6), batch)                         # layer 0: 50 of 56
    f = c.fork(a)

    def scored(seq, layer):
        batch = c.batch([seq], [1])
        c.score(layer, *rows(1), batch)
        given = calls[-1][2]["scored"]
        return (batch.kv_len if given is None else given).tolist()

    assert c.evict([f], 30, recent=8)[0] == [f]         # the newest 8 with layer 0's six among them
    batch = c.grow([f], 1)
    for l, n in ((0, 24), (1, 30)):
        c.score(l, *rows(1), batch)
        assert calls[-1][2]["scored"].tolist() == [n]
    c.truncate(a, 53)
    assert scored(a, 1) == [53] and scored(a, 0) == [50]
    assert scored(a, 0) == [53]


def test_scored_twice_adds_twice(made):
    """The same batch again (a prompt's other window) goes on from what the first call left; so does a batch that
    was made before another one was scored."""
    c, calls = made(n_layers=1)
    a, b = c.new(), c.new()
    c.score(0, *rows(60), c.grow([a, b], [50, 10]))
    first = c.grow([a, b], [4, 1])
    second = c.grow([b, a], [1, 2])
    q, lse = rows(5)
    c.score(0, q, lse, first)
    assert calls[-1][2]["scored"] is first.scored and first.scored.tolist() == [50, 10]
    c.score(0, q[:3], lse[:3], first, q_start=torch.tensor([0, 2, 3], dtype=torch.int32))
    assert calls[-1][2]["scored"] is None               # all of its tokens have a score by now
    c.score(0, *rows(3), second)
    assert second.scored.tolist() == [10, 50] and calls[-1][2]["scored"].tolist() == [11, 54]
    c.score(0, q, lse, first)                           # an older one: nothing is forgotten
    assert calls[-1][2]["scored"] is None
    assert c.grow([a, b], 1).scored.tolist() == [56, 12]


def test_a_batch_of_a_freed_sequence_is_refused(made):
    """Its slot may be another sequence's by now."""
    c, calls = made(score_slots=2)
    a, b = c.new(), c.new()
    batch = c.grow([a, b], 5)
    c.free(b)
    c.new()
    n = len(calls)
    with pytest.raises(KeyError):
        c.score(0, *rows(10), batch)
    assert len(calls) == n


def test_evict_on_a_stream_returns_memory_of_the_current_one_too(made, monkeypatch):
    """The call itself gets the stream, so that it records its outputs on the stream that is current for the caller;
    the tables are made on the call's stream."""
    from nvfp4_gated_deltanet_gb300 import kv4
    c, calls = made(n_layers=1)
    a = c.new()
    c.score(0, *rows(50), c.grow([a], 50))
    side, inside, made_on = SimpleNamespace(), [], []

    @contextlib.contextmanager
    def on(stream):
        inside.append(stream)
        yield
        inside.pop()

    dev, evict = c._dev, kv4.kv4_evict
    monkeypatch.setattr(c, "_on", on)
    monkeypatch.setattr(c, "_dev", lambda x: made_on.append(inside[-1]) or dev(x))
    monkeypatch.setattr(kv4, "kv4_evict", lambda *x, **k: (calls.append(list(inside)), evict(*x, **k))[1])
    c.evict([a], 20, stream=side)
    assert calls[-2] == [] and calls[-1][2]["stream"] is side and set(map(id, made_on)) == {id(side)}


def test_sums_that_go_elsewhere_are_no_scores_of_the_cache(made):
    c, calls = made(n_layers=1)
    a = c.new()
    batch = c.grow([a], 50)
    c.score(0, *rows(50), batch, out=torch.zeros(3, 2, 200))
    with pytest.raises(ValueError, match="no score"):
        c.evict([a], 20)
    c.score(0, *rows(50), batch)
    assert calls[-1][2]["scored"].tolist() == [0]
    c.evict([a], 20)
