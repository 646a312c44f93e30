"""Shared prefixes, scores and eviction of the 4-bit KV cache without a GPU: what the
book decides, what the calls refuse before they touch a device, what KV4Cache hands on."""
import ctypes
import random

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def g():
    from nvfp4_gated_deltanet_gb300 import build
    build.build()
    import nvfp4_gated_deltanet_gb300 as pkg
    return pkg


def common(a, b):
    n = 0
    while n < min(len(a), len(b)) and a[n] == b[n]:
        n += 1
    return n


def test_groups_of_forks(g):
    b = g.KV4Book(200, 16)
    a = b.new()
    b.extend([a], [100])                          # 6 whole pages and a part
    x, y = b.fork(a), b.fork(a)
    b.extend([a, x, y], [5, 20, 1])               # two of them copy the part, the last keeps it
    lone = b.new()
    b.extend([lone], [40])
    z = b.fork(lone)
    assert b.groups([a, x, y, lone, z]) == ([0, 3, 5], [96, 48])
    assert b.groups([a, lone, x]) == ([0, 1, 2, 3], [0, 0, 0])
    assert b.groups([a]) == ([0, 1], [0])
    assert b.groups([]) == ([0], [])


@pytest.mark.parametrize("seed", range(5))
def test_groups_share_what_they_say(g, seed):
    """Every member of a group has its shared pages; nobody is left alone who shares pages with a neighbour."""
    rng = random.Random(seed)
    b = g.KV4Book(4000, 16)
    seqs = []
    for _ in range(12):
        if seqs and rng.random() < 0.7:
            s = b.fork(rng.choice(seqs))
            b.truncate(s, rng.randint(0, b.length(s)))
        else:
            s = b.new()
        b.extend([s], [rng.randint(0, 200)])
        seqs.append(s)
    start, shared = b.groups(seqs)
    assert start[0] == 0 and start[-1] == len(seqs) and sorted(set(start)) == start
    for i, S in enumerate(shared):
        members = seqs[start[i]:start[i + 1]]
        for s in members:
            assert b.pages(s)[:S // 16] == b.pages(members[0])[:S // 16] and len(b.pages(s)) >= S // 16
    for i in range(1, len(seqs)):
        if start.count(i) and common(b.pages(seqs[i - 1]), b.pages(seqs[i])):
            assert len(seqs[start[start.index(i) - 1]:i]) > 1


def state(book):
    return book.holders[:], book._free[:], {k: (v[0][:], v[1]) for k, v in book.seqs.items()}


def test_exchange_release_restore(g):
    b = g.KV4Book(20, 16)
    a, c = b.new(), b.new()
    b.extend([a, c], [100, 50])
    f = b.fork(a)
    before = state(b)
    with pytest.raises(MemoryError):
        b.exchange([a, c], [100, 50 + 16])
    assert state(b) == before
    old = b.exchange([a, c], [40, 0])
    assert b.length(a) == 40 and len(b.pages(a)) == 3 and b.pages(c) == [] and not set(b.pages(a)) & set(old[0][0])
    b.restore([a, c], old)
    assert state(b) == before
    old = b.exchange([a, c], [40, 0])
    b.release(old)
    assert b.pages(f) == old[0][0] and b.free_pages == 20 - 7 - 3      # the fork still holds the old pages
    b.free(f), b.free(a), b.free(c)
    assert b.free_pages == 20 and not any(b.holders)


def fake(g, monkeypatch, **kw):
    """A cache on the CPU whose device calls are written down instead."""
    from nvfp4_gated_deltanet_gb300 import kv4
    c = g.KV4Cache(64, 16, 2, 64, 1.0, 1.0, n_layers=2, device="cpu", **kw)
    monkeypatch.setattr(c, "_dev", lambda rows: torch.tensor(rows, dtype=torch.int32))
    calls = []
    for name in ("kv4_score", "kv4_decode_shared", "kv4_copy_pages"):
        monkeypatch.setattr(kv4, name, lambda *a, name=name, **k: calls.append((name, a, k)))

    def evict(*a, **k):
        calls.append(("kv4_evict", a, k))
        return torch.zeros(2, a[2].shape[0], 2, k["max_keep"], dtype=torch.int32), None

    monkeypatch.setattr(kv4, "kv4_evict", evict)
    return c, calls


def test_cache_scores_and_evicts(g, monkeypatch):
    c, calls = fake(g, monkeypatch, score_slots=3, score_tokens=200)
    a, b = c.new(), c.new()
    q, lse = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 4)
    batch = c.grow([a, b], [50, 30])
    assert batch.scored.tolist() == [0, 0] and len(set(batch.slots.tolist())) == 2
    with pytest.raises(ValueError, match="rows"):
        c.score(0, q, lse, batch)                                     # 2 rows of 80
    c.score(0, q, lse, batch, q_start=torch.tensor([0, 1, 2], dtype=torch.int32))
    c.score(1, q, lse, batch, q_start=torch.tensor([0, 1, 2], dtype=torch.int32))
    batch = c.grow([b, a], 1)
    assert batch.scored.tolist() == [30, 50]
    c.score(0, q, lse, batch)
    name, args, kw = calls[-1]
    assert kw["q_start"] is None and kw["scored"] is batch.scored and args[6] == 1.0
    c.score(1, q[:, None], lse[:, None], batch)
    assert calls[-1][2]["q_start"] is None
    with pytest.raises(ValueError, match="rows"):
        c.score(1, q[:1, None], lse[:1, None], batch)
    batch = c.batch([a, b], [2, 2])
    c.score(0, torch.zeros(4, 4, 64, dtype=torch.bfloat16), torch.zeros(4, 4), batch)
    assert calls[-1][1][0].shape == (2, 2, 4, 64) and calls[-1][1][1].shape == (2, 2, 4)
    batch = c.batch([a, b], [2, 1])
    c.score(0, torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 4), batch)
    assert calls[-1][2]["q_start"] is batch.q_start
    n = len(calls)
    c.score(0, q[:0], lse[:0], c.batch([a, b], [0, 0]))               # no rows: nothing to add
    assert len(calls) == n
    batch = c.grow([a, b], [3, 0])                                    # three that are not scored
    with pytest.raises(ValueError, match="no score"):
        c.evict([a, b], 20, recent=2)
    before = c.book.pages(a)
    cut, kept = c.evict([a, b], [20, 100], recent=4)
    assert cut == [a] and kept.shape == (2, 1, 2, 20) and c.book.length(a) == 20 and c.book.length(b) == 31
    name, args, kw = calls[-1]
    assert args[1].tolist() == [before] and args[2].tolist() == [54] and args[3].tolist() == [20] and args[4] == 4
    assert args[6].tolist() == [c.book.pages(a)] and not set(before) & set(c.book.pages(a))
    assert c.grow([a], 1).scored.tolist() == [17]                     # the three newest have none still
    assert c.evict([b], 31)[0] == [] and len(calls) == 6 + 1
    c.truncate(b, 10)
    f = c.fork(b)
    assert c.grow([b, f], 0).scored.tolist() == [10, 10]
    with pytest.raises(MemoryError, match="slot"):
        c.new()
    with pytest.raises(MemoryError, match="slot"):
        c.fork(a)
    assert len(c.book.seqs) == 3
    c.free(f)
    c.new()
    with pytest.raises(MemoryError, match="holds"):
        c.grow([a], 200)
    assert c.book.length(a) == 21


def test_fork_copies_scores(g, monkeypatch):
    c, _ = fake(g, monkeypatch, score_slots=2, score_tokens=20)
    a = c.new()
    c.scores[:, c._slot[a]] = torch.rand(2, 2, 20)
    f = c.fork(a)
    assert torch.equal(c.scores[:, c._slot[f]], c.scores[:, c._slot[a]]) and c._slot[a] != c._slot[f]


def test_evict_that_fails_leaves_the_book(g, monkeypatch):
    from nvfp4_gated_deltanet_gb300 import kv4
    c, calls = fake(g, monkeypatch, score_slots=2, score_tokens=1000)
    a, b = c.new(), c.new()
    c.grow([a, b], [600, 300])                                        # 57 of 64 pages
    c._scored.update({a: 600, b: 300})
    before = state(c.book)
    with pytest.raises(MemoryError):
        c.evict([a, b], 200)                                          # 26 new pages
    assert state(c.book) == before

    def fails(*a, **k):
        raise RuntimeError("launch")

    monkeypatch.setattr(kv4, "kv4_evict", fails)
    with pytest.raises(RuntimeError, match="launch"):
        c.evict([a, b], 48)
    assert state(c.book) == before and c._scored == {a: 600, b: 300}
    for bad in (dict(keep=-1), dict(keep=[1]), dict(keep=5, recent=-1)):
        with pytest.raises(ValueError):
            c.evict([a, b], **bad)
    with pytest.raises(ValueError):
        c.evict([a, a], 5)


def test_cache_without_scores_or_groups_refuses(g, monkeypatch):
    c, calls = fake(g, monkeypatch)
    a = c.new()
    batch = c.grow([a], 1)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="score_slots"):
        c.score(0, q, None, batch)
    with pytest.raises(ValueError, match="score_slots"):
        c.evict([a], 5)
    with pytest.raises(ValueError, match="share"):
        c.decode_shared(0, q, batch)
    f = c.fork(a)
    batch = c.grow([a, f], 2, share=True)
    with pytest.raises(ValueError, match="rows"):
        c.decode_shared(0, q, batch)
    c.decode_shared(1, torch.zeros(2, 2, 4, 64, dtype=torch.bfloat16), batch)
    assert calls[-1][0] == "kv4_decode_shared" and calls[-1][2]["max_shared"] == 0


def test_shares_where_that_pays(g, monkeypatch):
    """share="auto": long prefixes of many, none of few or of short ones; where nothing is left, decode."""
    from nvfp4_gated_deltanet_gb300 import kv4
    c = g.KV4Cache(6000, 16, 8, 128, 1.0, 1.0, device="cpu")
    monkeypatch.setattr(c, "_dev", lambda rows: torch.tensor(rows, dtype=torch.int32))
    calls = []
    for name in ("kv4_decode", "kv4_decode_shared", "kv4_copy_pages"):
        monkeypatch.setattr(kv4, name, lambda *a, name=name, **k: calls.append((name, k)))
    a, b = c.new(), c.new()
    c.grow([a, b], [32768, 8192])
    few, many = [c.fork(a) for _ in range(4)], [c.fork(b) for _ in range(20)]
    ask = lambda seqs, **kw: c.decode_shared(0, torch.zeros(len(seqs), 1, 8, 128, dtype=torch.bfloat16), c.batch(seqs, [1] * len(seqs), **kw))
    ask(few, share="auto")
    assert calls[-1][0] == "kv4_decode"
    ask(few, share=True)
    assert calls[-1][0] == "kv4_decode_shared" and calls[-1][1]["max_shared"] == 32768
    ask(many[:8], share="auto")
    assert calls[-1][0] == "kv4_decode"
    ask(many, share="auto")
    assert calls[-1][0] == "kv4_decode_shared" and calls[-1][1]["max_shared"] == 8192
    batch = c.batch(few[:2] + many, [1] * 22, share="auto")           # of two that share 32768 tokens each reads its own
    assert batch.shared_len.tolist() == [0, 8192] and batch.group_start.tolist() == [0, 2, 22] and not batch.plain
    batch = c.batch(few + many, [1] * 24, share="auto")
    assert batch.shared_len.tolist() == [32768, 8192]
    assert c.batch([], [], share="auto").plain
    held = state(c.book)
    with pytest.raises(ValueError, match="share"):
        c.grow(few, 1, share="always")
    assert state(c.book) == held


GOOD = 0x10000  # an address that no call reads: each of these is refused first


def structs(g, **kw):
    c = dict(pages=GOOD, num_pages=8, page_tokens=16, n_kv_heads=2, head_dim=64, k_scale=1.0, v_scale=1.0)
    b = dict(kv_len=GOOD, block_table=GOOD, q_start=None, B=2, max_pages=2, T=2, zero_padding=0)
    s = dict(in_=GOOD, out=GOOD, slots=None, n_slots=2, tokens=32)
    h = dict(group_start=GOOD, shared_len=GOOD, groups=1, max_shared=16)
    for k, v in kw.items():
        [d for d in (c, b, s, h) if k in d][0][k] = v
    return g.Kv4CacheStruct(**c), g.Kv4BatchStruct(**b), g.Kv4ScoresStruct(**s), g.Kv4SharedStruct(**h)


def refs(*x):
    return [None if y is None else ctypes.byref(y) for y in x]


def test_decode_shared_refusals(g):
    L = g.lib()

    def call(q=GOOD, stride=4 * 64, hq=4, sm=1.0, out=GOOD, ws=GOOD, n=1 << 30, no_groups=False, **kw):
        c, b, _, h = structs(g, **kw)
        return L.kv4_decode_shared(*refs(c, b, None if no_groups else h), q, stride, hq, sm, out, None, ws, n, None, None)

    assert call(no_groups=True) == 1 and call(group_start=None) == 1 and call(shared_len=None) == 1
    assert call(ws=None) == 1 and call(q=None) == 1 and call(out=None) == 1
    assert call(groups=-1) == 2 and call(max_shared=-1) == 2 and call(q_start=GOOD) == 2 and call(hq=3) == 2
    assert call(stride=4 * 64 + 4) == 2 and call(n=16) == 2 and call(T=3) == 2 and call(head_dim=96) == 2
    assert call(group_start=GOOD + 2) == 3 and call(ws=GOOD + 8) == 3 and call(q=GOOD + 2) == 3
    assert call(sm=float("nan")) == 4 and call(sm=0.0) == 5 and call(v_scale=-1.0) == 5
    assert call(T=0, B=0) == 0 and call(groups=2 ** 31 - 8) == 7
    c, b, _, h = structs(g)
    need = L.kv4_decode_shared_workspace(*refs(c, b, h), 4)
    assert need > 0 and call(n=need - 1) == 2
    for kw in (dict(q_start=GOOD), dict(groups=-1), dict(T=0), dict(page_tokens=8)):
        c, b, _, h = structs(g, **kw)
        assert L.kv4_decode_shared_workspace(*refs(c, b, h), 4) == 0


def test_score_refusals(g):
    L = g.lib()

    def call(q=GOOD, stride=4 * 64, hq=4, sm=1.0, lse=GOOD, scored=None, no_scores=False, **kw):
        c, b, s, _ = structs(g, **kw)
        return L.kv4_score(*refs(c, b), q, stride, hq, sm, lse, *refs(None if no_scores else s), scored, GOOD, 1 << 40, None,
                           None)

    assert call(no_scores=True) == 1 and call(q=None) == 1 and call(lse=None) == 1 and call(in_=None) == 1
    assert call(out=None) == 1 and call(kv_len=None) == 1 and call(kv_len=None, T=0) == 1
    assert call(hq=3) == 2 and call(hq=130) == 2 and call(stride=8) == 2 and call(n_slots=-1) == 2 and call(tokens=-1) == 2
    assert call(out=GOOD + 4 * 2 * 2 * 32 - 4) == 2 and call(out=GOOD - 4) == 2          # overlaps in part
    assert call(lse=GOOD + 2) == 3 and call(slots=GOOD + 1) == 3 and call(scored=GOOD + 2) == 3 and call(in_=GOOD + 2) == 3
    assert call(sm=float("inf")) == 4 and call(sm=-1.0) == 5 and call(k_scale=0.0) == 5
    assert call(n_slots=2 ** 31 - 1, tokens=2 ** 31 - 1) == 7
    assert call(B=0, T=0) == 0 and call(n_slots=0) == 0
    assert call(max_pages=2 ** 20, B=2 ** 20, T=2 ** 20) == 7


def test_evict_refusals(g):
    L = g.lib()
    page = 2 * 18 * 64

    def call(layers=1, stride=0, keep=GOOD, recent=0, score_stride=0, table=GOOD, cols=2, kept=GOOD, most=32, n=GOOD, **kw):
        c, b, s, _ = structs(g, **kw)
        return L.kv4_evict(*refs(c), layers, stride, *refs(b), keep, recent, *refs(s), score_stride, table, cols, kept, most,
                           n, None, None)

    assert call(keep=None) == 1 and call(n=None) == 1 and call(kept=None) == 1 and call(table=None) == 1
    assert call(pages=None) == 1 and call(in_=None) == 1
    assert call(layers=0) == 2 and call(recent=-1) == 2 and call(cols=-1) == 2 and call(most=-1) == 2
    assert call(layers=2, stride=8 * page - 16, score_stride=128) == 2 and call(layers=2, stride=8 * page + 8, score_stride=128) == 2
    assert call(layers=2, stride=8 * page, score_stride=127) == 2 and call(out=GOOD + 256) == 2
    assert call(keep=GOOD + 2) == 3 and call(pages=GOOD + 8) == 3 and call(kept=GOOD + 3) == 3
    assert call(num_pages=2 ** 31 - 1, page_tokens=256, n_kv_heads=1024) == 7
    assert call(most=2 ** 31 - 1, B=2 ** 10) == 7 and call(most=16, B=2 ** 27) == 7
    assert call(B=0, T=0) == 0


def on(device, *shape, dtype=torch.int32):
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        return torch.empty(*shape, dtype=dtype, device=device)


def calls(g):
    bf, fl, u8, i4 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
    pages, table, lens, status = ((4, 2, 1, 18 * 128), u8), ((2, 2), i4), ((2,), i4), ((1,), i4)
    q, lse, rows = ((2, 4, 128), bf), ((2, 4), fl), ((2, 2, 32), fl)
    common = dict(pages=pages, block_table=table, kv_len=lens, dev_status=status)
    return [
        (g.kv4_decode_shared, dict(common, q=q, group_start=lens, shared_len=status, out=q, lse=lse, workspace=((4096,), u8)),
         dict(k_scale=1.0, v_scale=1.0)),
        (g.kv4_score, dict(common, q=q, lse=lse, scores=rows, q_start=((3,), i4), slots=lens, scored=lens, out=rows,
                           workspace=((4096,), u8)), dict(k_scale=1.0)),
        (g.kv4_evict, dict(common, keep=lens, scores=rows, new_table=table, slots=lens, kept=((2, 2, 32), i4), new_len=lens,
                           scores_out=rows), dict(recent=0))]


@pytest.mark.parametrize("i", range(3))
def test_tensors_of_several_devices_are_refused(g, i):
    from types import SimpleNamespace
    if torch.cuda.device_count() == 1:
        pytest.skip("where there is one GPU, not even a stand-in can name a second")
    f, tensors, rest = calls(g)[i]
    for odd in tensors:
        for here, there in (("cuda:0", "cuda:1"), ("cuda:0", "cpu")):
            args = {k: on(there if k == odd else here, *shape, dtype=dt) for k, (shape, dt) in tensors.items()}
            with pytest.raises(ValueError, match="cuda:1|cpu|CUDA"):
                f(**args, **rest)
    args = {k: on("cuda:1", *shape, dtype=dt) for k, (shape, dt) in tensors.items()}
    with pytest.raises(ValueError, match="stream"):
        f(**args, **rest, stream=SimpleNamespace(cuda_stream=0, device_index=0))
