"""kv4_evict on the GPU: which tokens stay, where their bytes go and their scores,
against a plain choice on the host, exactly."""
import numpy as np
import pytest

import kv4_ref as ref

torch = pytest.importorskip("torch")
if torch.cuda.is_available():
    from kv4_inputs import KS, VS, ints, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import nvfp4_gated_deltanet_gb300 as pkg
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return pkg


def cache(lens, keeps, page, hkv, d, layers, seed=0, spare=2):
    """Pages of random bytes, shuffled tables of the sequences and of their new pages."""
    rng = np.random.RandomState(seed)
    need = [-(-n // page) for n in lens] + [-(-k // page) for k in keeps]
    ids = rng.permutation(sum(need) + spare).tolist()
    rows = [[ids.pop() for _ in range(n)] for n in need]

    def table(rows):
        cols = max([1] + [len(r) for r in rows])
        return ints([r + [-3] * (cols - len(r)) for r in rows])

    gen = torch.Generator(device="cuda").manual_seed(seed)
    pages = torch.randint(0, 256, (layers, sum(need) + spare, hkv, page // 16, 18 * d), generator=gen, dtype=torch.uint8,
                          device="cuda")
    return pages, table(rows[:len(lens)]), table(rows[len(lens):])


def choose(x, k, recent):
    """The kept places of scores x (numpy float32): sorted by falling score and then by age."""
    n = len(x)
    k = min(k, n)
    old = n - min(recent, k)
    order = sorted(range(old), key=lambda i: (-np.inf if np.isnan(x[i]) else x[i], -i), reverse=True)
    # NaN below minus infinity
    order = [i for i in order if not np.isnan(x[i])] + [i for i in order if np.isnan(x[i])]
    return sorted(order[:k - (n - old)]) + list(range(old, n))


def move(pages, old, new, kept, d, page):
    """pages (numpy, changed in place) of one layer and head: the kept tokens' bytes to their new places."""
    src = pages.copy()
    for i0 in range(0, len(kept), 16):
        cell = pages[new[i0 // page], i0 % page // 16]
        cell[:] = 0
        for i in range(i0, min(i0 + 16, len(kept))):
            t = kept[i]
            from_cell = src[old[t // page], t % page // 16]
            for a, b in zip(ref.places(t % 16, d), ref.places(i % 16, d)):
                cell[b] = from_cell[a]


def expect(pages, tab, new, scores, slots, lens, keeps, recent, page, d, most):
    pages, scores, tab, new = (t.cpu().numpy().copy() for t in (pages, scores, tab, new))
    L, hkv = pages.shape[0], pages.shape[2]
    kept = np.full((L, len(lens), hkv, most), -1, np.int32)
    for l in range(L):
        for b, n in enumerate(lens):
            for h in range(hkv):
                row = scores[l, slots[b], h]
                at = choose(row[:n], keeps[b], recent)
                kept[l, b, h, :len(at)] = at
                row[:len(at)] = row[at]
                row[len(at):n] = 0
                move(pages[l, :, h], tab[b], new[b], at, d, page)
    return pages, scores, kept


def random_scores(shape, seed, kind="weights"):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.exp(2.5 * torch.randn(shape, generator=gen, device="cuda") - 6)
    if kind == "ties":
        x = (4 * torch.rand(shape, generator=gen, device="cuda")).floor() * 0.25
    elif kind == "signs":                               # negative ones, both zeros, infinities and NaN among them
        x = torch.randn(shape, generator=gen, device="cuda")
        pick = (12 * torch.rand(shape, generator=gen, device="cuda")).floor()
        for i, v in enumerate((0.0, -0.0, float("inf"), float("-inf"), float("nan"), -float("nan"))):
            x = torch.where(pick == i, torch.full_like(x, v), x)
    elif kind == "equal":
        x = torch.full(shape, 0.5, device="cuda")
    return x


def bits(t):
    return t.view(torch.int32).cpu().numpy()


@pytest.mark.parametrize("hkv,d,page,layers,lens,keeps,recent", [
    (2, 128, 16, 2, [40, 1, 0, 300], [17, 1, 5, 100], 8),
    (1, 64, 64, 1, [1000], [333], 0),
    (3, 64, 32, 2, [100, 64, 33], [64, 64, 32], 1000),          # all that stays is recent
    (2, 128, 256, 1, [700, 255], [0, 16], 3),                   # nothing stays
    (4, 128, 64, 3, [513, 129], [512, 128], 64),                # all but one
    (1, 128, 128, 1, [9001], [4097], 1024),
    (8, 64, 16, 1, [77] * 9, [7] * 9, 2),
    (1, 64, 64, 1, [70000], [300], 10),                         # far more tokens than a CTA has threads
    (1, 64, 256, 1, [800000], [1000], 100),                     # more than a cluster's shared memory holds
    (1, 64, 256, 1, [700000, 200], [1000, 100], 100),           # the most that it holds, nearly
    (2, 64, 64, 5, [40000], [100], 7),                          # clusters of 4
    (2, 64, 64, 1, [30000, 17], [20011, 9], 5),
    (1, 64, 64, 1, [12000], [7], 0),
    (2, 64, 64, 40, [9000], [3], 1),                            # a CTA a row
])
@pytest.mark.parametrize("kind", ["weights", "ties"])
def test_evict(g, hkv, d, page, layers, lens, keeps, recent, kind):
    pages, tab, new = cache(lens, [min(k, n) for k, n in zip(keeps, lens)], page, hkv, d, layers, seed=len(lens))
    B, room = len(lens), max(lens) + 3
    slots = torch.randperm(B + 2, device="cuda")[:B].to(torch.int32)
    scores = random_scores((layers, B + 2, hkv, room), 3, kind)
    most = max(keeps)
    want_p, want_s, want_k = expect(pages, tab, new, scores, slots.tolist(), lens, keeps, recent, page, d, most)
    st = ints([0])
    args = (ints(lens), ints(keeps), recent)
    # scores to another tensor, whose other places stay
    p1, mark = pages.clone(), torch.full_like(scores, -5.0)
    kept, n = g.kv4_evict(p1, tab, *args, scores, new, max_keep=most, slots=slots, scores_out=mark, dev_status=st)
    assert np.array_equal(kept.cpu().numpy(), want_k) and n.tolist() == [min(a, b) for a, b in zip(lens, keeps)]
    assert np.array_equal(p1.cpu().numpy(), want_p)
    named = torch.zeros_like(scores, dtype=torch.bool)
    for b, m in enumerate(lens):
        named[:, slots[b], :, :m] = True
    assert np.array_equal(bits(mark[named]), bits(torch.from_numpy(want_s).cuda()[named])) and (mark[~named] == -5).all()
    # in place
    kept2, n2 = g.kv4_evict(pages, tab, *args, scores, new, max_keep=most, slots=slots, dev_status=st)
    assert torch.equal(kept, kept2) and torch.equal(n, n2) and torch.equal(pages, p1)
    assert np.array_equal(bits(scores), want_s.view(np.int32)) and st.item() == 0


@pytest.mark.parametrize("kind", ["signs", "equal"])
@pytest.mark.parametrize("n", [5, 33, 1024, 1025, 5000, 20001])
def test_order_of_scores(g, kind, n):
    """Ties to the older, the zeros equal, NaN below all; the scores keep their bits."""
    hkv, d, page = 2, 64, 64
    for k, recent in ((n // 3, 0), (n - 1, 1), (n // 2, n // 4), (1, 0)):
        pages, tab, new = cache([n], [max(k, 1)], page, hkv, d, 1, seed=n)
        scores = random_scores((1, 1, hkv, n), n, kind)
        want = expect(pages, tab, new, scores, [0], [n], [k], recent, page, d, max(k, 1))
        kept, _ = g.kv4_evict(pages, tab, ints([n]), ints([k]), recent, scores, new, max_keep=max(k, 1))
        assert np.array_equal(kept.cpu().numpy(), want[2])
        assert np.array_equal(pages.cpu().numpy(), want[0]) and np.array_equal(bits(scores), want[1].view(np.int32))


def test_one_layer_and_defaults(g):
    """Pages of four dimensions, no slots, max_keep from the new pages' room; given outputs."""
    pages, tab, new = cache([100, 60], [40, 20], 16, 2, 128, 1)
    scores = random_scores((1, 2, 2, 128), 1)
    want_p, want_s, want_k = expect(pages, tab, new, scores, [0, 1], [100, 60], [40, 20], 4, 16, 128, 48)
    kept, n = torch.empty(2, 2, 48, dtype=torch.int32, device="cuda"), ints([9, 9])
    got = g.kv4_evict(pages[0], tab, ints([100, 60]), ints([40, 20]), 4, scores[0], new, kept=kept, new_len=n)
    assert got[0].data_ptr() == kept.data_ptr() and got[1].data_ptr() == n.data_ptr()
    assert np.array_equal(kept.cpu().numpy(), want_k[0]) and n.tolist() == [40, 20]
    assert np.array_equal(pages.cpu().numpy(), want_p) and np.array_equal(bits(scores), want_s.view(np.int32))


def test_left_out_sequences(g):
    """Bad lengths, limits and slots: nothing of theirs changes, the others are right."""
    lens, keeps, page, hkv, d = [50, 60, 70, 80], [20, 20, 20, 20], 16, 2, 64
    pages, tab, new = cache(lens, keeps, page, hkv, d, 2)
    scores = random_scores((2, 6, hkv, 85), 2)
    good_p, good_s, good_k = expect(pages, tab, new, scores, [0, 1, 2, 3], lens, keeps, 2, page, d, 20)

    def run(lens=lens, keeps=keeps, slots=None, most=20):
        p, s, st = pages.clone(), scores.clone(), ints([0])
        kept, n = g.kv4_evict(p, tab, ints(lens), ints(keeps), 2, s, new, max_keep=most,
                              slots=None if slots is None else ints(slots), dev_status=st)
        return p, s, kept, n.tolist(), st.item()

    def left(got, out, flagged):
        p, s, kept, n, st = got
        assert st == (6 if flagged else 0)
        for b in range(4):
            own = new[b][new[b] >= 0].long()
            if b in out:
                assert n[b] == -1 and (kept[:, b] == -1).all() and torch.equal(p[:, own], pages[:, own])
                assert torch.equal(s[:, b], scores[:, b])
            else:
                assert n[b] == 20 and np.array_equal(kept[:, b].cpu().numpy(), good_k[:, b])
                assert np.array_equal(p[:, own].cpu().numpy(), good_p[:, own.cpu().numpy()])
                assert np.array_equal(bits(s[:, b]), good_s[:, b].view(np.int32))

    left(run(), [], False)
    left(run(slots=[0, -1, 2, 3]), [1], False)
    left(run(slots=[0, 6, 2, -2]), [1, 3], True)
    left(run(slots=[0, 5, 2, 5]), [1, 3], True)
    for bad in (-1, 81 + 16 * 5, 2 ** 31 - 1):
        left(run(lens=[50, bad, 70, 80]), [1], True)
    left(run(keeps=[20, 20, -1, 20]), [2], True)
    left(run(keeps=[20, 20, 21, 20]), [2], True)         # more than max_keep
    p, s, kept, n, st = run(keeps=[20, 20, 60, 20], most=60)
    left((p, s, kept[..., :20], n, st), [2], True)       # more than its new pages hold
    long = ints([50, 60, 70, 80])
    short = scores[..., :65].contiguous()                # 70 and 80 tokens do not fit the rows
    p, st = pages.clone(), ints([0])
    kept, n = g.kv4_evict(p, tab, long, ints(keeps), 2, short, new, max_keep=20, dev_status=st)
    assert n.tolist() == [20, 20, -1, -1] and st.item() == 6
    bad = new.clone()
    bad[0, 1] = 10 ** 6                                  # a new page that is none
    p, s, st = pages.clone(), scores.clone(), ints([0])
    g.kv4_evict(p, tab, long, ints(keeps), 2, s, bad, max_keep=20, dev_status=st)
    assert st.item() == 6
    for b in (1, 2, 3):
        own = new[b][new[b] >= 0].long()
        assert np.array_equal(p[:, own].cpu().numpy(), good_p[:, own.cpu().numpy()])


def test_captured_and_replayed(g):
    """In a graph, lengths and limits read at the replay; a given stream."""
    page, hkv, d = 16, 2, 64
    pages, tab, new = cache([200, 150], [64, 64], page, hkv, d, 2)
    scores = random_scores((2, 2, hkv, 200), 4)
    lens, keeps = ints([100, 100]), ints([10, 64])
    out = torch.zeros_like(scores)
    kept, n = torch.empty(2, 2, hkv, 64, dtype=torch.int32, device="cuda"), ints([0, 0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        g.kv4_evict(pages, tab, lens, keeps, 5, scores, new, kept=kept, new_len=n, max_keep=64, scores_out=out)
    lens.copy_(ints([200, 150]))
    keeps.copy_(ints([33, 48]))
    want = expect(pages, tab, new, scores, [0, 1], [200, 150], [33, 48], 5, page, d, 64)
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(kept.cpu().numpy(), want[2]) and n.tolist() == [33, 48]
    assert np.array_equal(pages.cpu().numpy(), want[0])
    side = pages.clone()
    s.wait_stream(torch.cuda.current_stream())
    k2, n2 = g.kv4_evict(side, tab, lens, keeps, 5, scores, new, max_keep=64, scores_out=out, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(k2, kept) and n2.tolist() == [33, 48] and torch.equal(side, pages)
