"""kv4_score on the GPU against sums of attention weights in float64, within
bounds derived from its roundings."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if torch.cuda.is_available():
    from kv4_inputs import KS, VS, ints, prefixed, queries, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import nvfp4_gated_deltanet_gb300 as pkg
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return pkg


def cached(g, lens, page, hkv, d, seed=0):
    pages, table, n, *_ = prefixed(g, [(0, lens)], page, hkv, d, seed)
    return pages, table, n


def attend(g, q, pages, table, n, counts):
    start = ints(np.concatenate([[0], np.cumsum(counts)]).tolist())
    return start, g.kv4_prefill(q, pages, table, n, start, KS, VS, return_lse=True)[1]


def check(out, before, slots, scored, lens, want, err):
    """Named rows: the sums; every other place: as before, bit for bit."""
    left = torch.ones_like(before, dtype=torch.bool)
    for b, m in enumerate(lens):
        s = slots[b]
        old = before[s, :, :m].double()
        if scored is not None:
            old[:, scored[b]:] = 0
        w = old + want[b]
        e = err[b] + 2.0 ** -23 * (old.abs() + want[b])
        over = (out[s, :, :m].double() - w).abs() / (e + 1e-300)
        assert m == 0 or over.max() <= 1, (b, over.max().item())
        left[s, :, :m] = False
    assert torch.equal(out[left], before[left])


@pytest.mark.parametrize("hq,hkv,d,page,r,lens", [
    (8, 2, 128, 64, 1, [1, 700, 64, 0, 33, 257]),       # a decode step, ragged
    (4, 4, 64, 16, 1, [300, 1, 16]),                    # no shared heads
    (16, 2, 128, 16, 3, [2, 40, 500, 3]),               # candidates; a sequence with fewer tokens than rows
    (16, 1, 64, 32, 5, [129, 31]),
    (64, 1, 128, 256, 1, [1000]),                       # 64 heads of one KV head
    (3, 1, 128, 128, 8, [513, 8]),
    (32, 8, 128, 64, 2, [2100, 4, 1025]),
])
@pytest.mark.parametrize("fresh", [False, True])
def test_step(g, hq, hkv, d, page, r, lens, fresh):
    pages, table, n = cached(g, lens, page, hkv, d, seed=hq + r)
    B = len(lens)
    q = queries(B * r, hq, d, seed=r)
    lse = g.kv4_decode(q.unflatten(0, (B, r)), pages, table, n, KS, VS, return_lse=True)[1]
    gen = torch.Generator(device="cuda").manual_seed(5)
    slots = torch.randperm(B + 3, generator=gen, device="cuda")[:B].to(torch.int32)
    before = torch.rand(B + 3, hkv, max(lens) + 5, generator=gen, device="cuda")
    scored = [max(0, m - r) for m in lens] if fresh else None
    if fresh:                                           # what lies there counts for nothing
        for b, m in enumerate(lens):
            before[slots[b], :, scored[b]:] = float("nan")
    status = ints([0])
    want, err = weights(pages, table, lens, [r] * B, q, lse.reshape(B * r, hq), hkv, d)
    args = dict(slots=slots, scored=None if scored is None else ints(scored), dev_status=status)
    out = before.clone()
    q4 = q.unflatten(0, (B, r))
    g.kv4_score(q4, lse, pages, table, n, out, KS, **args)
    clean = torch.nan_to_num(before, nan=7.0)
    check(torch.where(torch.isnan(before) & torch.isnan(out), 7.0, out), clean, slots.tolist(), scored, lens, want, err)
    # the same into another tensor, and from ragged rows
    other = before.clone()
    g.kv4_score(q4, lse, pages, table, n, before, KS, out=other, **args)
    assert torch.equal(other.nan_to_num(7.0), out.nan_to_num(7.0))
    other = before.clone()
    g.kv4_score(q, lse.reshape(B * r, hq), pages, table, n, other, KS, q_start=ints([r * b for b in range(B + 1)]), **args)
    check(torch.where(torch.isnan(before) & torch.isnan(other), 7.0, other), clean, slots.tolist(), scored, lens, want, err)
    assert status.item() == 0


@pytest.mark.parametrize("hq,hkv,d,page,counts,lens", [
    (8, 2, 128, 64, [64, 64, 10], [700, 64, 10]),       # windows of prompts, a whole short prompt
    (8, 8, 64, 16, [333], [333]),
    (6, 2, 128, 16, [0, 200, 1, 77], [40, 500, 129, 77]),   # no rows for a sequence with tokens
    (16, 1, 128, 128, [129, 3], [129, 1500]),
    (32, 4, 64, 32, [256, 1], [2000, 0]),
    (5, 1, 64, 64, [700, 650], [700, 3000]),
    (4, 1, 128, 64, [90], [60]),                        # more rows than tokens: the first see nothing
    (32, 8, 128, 64, [400], [1300]),
])
def test_prompt(g, hq, hkv, d, page, counts, lens):
    pages, table, n = cached(g, lens, page, hkv, d, seed=len(lens) + hq)
    T = sum(counts)
    q = queries(T + 3, hq, d, seed=T)                   # three padding rows, which add nothing
    start, lse = attend(g, q, pages, table, n, counts)
    lse[T:] = float("nan")
    B = len(lens)
    before = torch.rand(B, hkv, max(lens), device="cuda")
    scored = [m // 2 for m in lens]
    want, err = weights(pages, table, lens, counts, q[:T], lse[:T], hkv, d)
    status, out = ints([0]), before.clone()
    g.kv4_score(q, lse, pages, table, n, out, KS, q_start=start, scored=ints(scored), dev_status=status)
    check(out, before, list(range(B)), scored, lens, want, err)
    again = before.clone()
    g.kv4_score(q, lse, pages, table, n, again, KS, q_start=start, scored=ints(scored))
    assert torch.equal(again, out) and status.item() == 0


def test_weights_of_a_row_sum_to_one(g):
    """Over all tokens the weights of a row-head sum to 1: every scored row adds G per KV head. Each weight is off
    by its bound, and by as much and 2^-16 again for the lse that it is taken by."""
    hq, hkv, d, lens, r = 8, 2, 128, [777, 50], 2
    pages, table, n = cached(g, lens, 32, hkv, d)
    q = queries(4, hq, d, seed=9).unflatten(0, (2, 2))
    lse = g.kv4_decode(q, pages, table, n, KS, VS, return_lse=True)[1]
    scores = torch.zeros(2, hkv, 800, device="cuda")
    want, err = weights(pages, table, lens, [r, r], q.flatten(0, 1), lse.flatten(0, 1), hkv, d)
    tol = 2 * max((e / w).max().item() for e, w in zip(err, want)) + 2.0 ** -16
    for i in range(3):
        g.kv4_score(q, lse, pages, table, n, scores, KS)
        assert (scores.double().sum(-1) / (4 * r * (i + 1)) - 1).abs().max() <= tol


def test_strided_queries_and_other_scale(g):
    hq, hkv, d, lens = 8, 2, 64, [100, 37, 64]
    pages, table, n = cached(g, lens, 16, hkv, d)
    wide = queries(3, hq + 2 * hkv, d, seed=3)
    q = wide[:, :hq]
    assert not q.is_contiguous()
    lse = g.kv4_decode(q.contiguous(), pages, table, n, KS, VS, return_lse=True, sm_scale=0.3)[1]
    a, b = torch.zeros(2, 3, hkv, 100, device="cuda")
    g.kv4_score(q, lse, pages, table, n, a, KS, sm_scale=0.3)
    g.kv4_score(q.contiguous(), lse, pages, table, n, b, KS, sm_scale=0.3)
    want, err = weights(pages, table, lens, [1] * 3, q, lse, hkv, d, sm=float(np.float32(0.3)))
    assert torch.equal(a, b)
    for x, m, w, e in zip(a, lens, want, err):
        assert ((x[:, :m].double() - w).abs() <= e).all()


def test_left_out_sequences(g):
    """Slot -1, slots out of range or named twice, rows that are too short, bad lengths: nothing of theirs is
    written, the others are right, and all but slot -1 are flagged."""
    hq, hkv, d, lens = 4, 2, 64, [50, 60, 70, 80, 40, 90]
    pages, table, n = cached(g, lens, 16, hkv, d)
    q = queries(6, hq, d, seed=4)
    lse = g.kv4_decode(q, pages, table, n, KS, VS, return_lse=True)[1]
    good = torch.zeros(8, hkv, 100, device="cuda")
    g.kv4_score(q, lse, pages, table, n, good, KS)

    def run(slots, tokens=100, lengths=n):
        st, out = ints([0]), torch.zeros(8, hkv, tokens, device="cuda")
        g.kv4_score(q, lse, pages, table, lengths, out, KS, slots=None if slots is None else ints(slots), dev_status=st)
        return out, st.item()

    out, st = run([0, 1, -1, 3, 4, 5])
    assert st == 0 and not out[2].any() and torch.equal(out[[0, 1, 3, 4, 5]], good[[0, 1, 3, 4, 5]])
    for bad in (8, -2, 2 ** 31 - 1, -2 ** 31):
        out, st = run([0, 1, bad, 3, 4, 5])
        assert st == 6 and not out[[2, 6, 7]].any() and torch.equal(out[[0, 1, 3, 4, 5]], good[[0, 1, 3, 4, 5]])
    out, st = run([0, 7, 2, 7, 4, 5])
    assert st == 6 and not out[7].any() and torch.equal(out[[0, 2, 4, 5]], good[[0, 2, 4, 5]])
    out, st = run(None, tokens=75)                      # 80 and 90 tokens do not fit
    assert st == 6 and not out[[3, 5]].any() and torch.equal(out[[0, 1, 2, 4], :, :40], good[[0, 1, 2, 4], :, :40])
    for bad in (-1, 16 * table.shape[1] + 1, 2 ** 31 - 1):
        m = n.clone()
        m[1] = bad
        out, st = run(None, lengths=m)
        assert st == 6 and not out[1].any() and torch.equal(out[[0, 2, 3, 4, 5]], good[[0, 2, 3, 4, 5]])
    bad = table.clone()
    bad[2, 1] = 10 ** 6                                 # a page id under read tokens: flagged, the others right
    st, out = ints([0]), torch.zeros(8, hkv, 100, device="cuda")
    g.kv4_score(q, lse, pages, bad, n, out, KS, dev_status=st)
    assert st.item() == 6 and torch.equal(out[[0, 1, 3, 4, 5]], good[[0, 1, 3, 4, 5]])


def test_extreme_rows(g):
    """A row of zeros weighs all tokens alike; one that sees nothing (lse -infinity) adds nothing; large queries."""
    hq, hkv, d, lens = 2, 1, 128, [333]
    pages, table, n = cached(g, lens, 64, hkv, d)
    q = queries(1, hq, d, seed=1)
    q[0, 0] = 0
    q[0, 1] *= 200
    lse = g.kv4_decode(q, pages, table, n, KS, VS, return_lse=True)[1]
    out = torch.zeros(1, 1, 333, device="cuda")
    g.kv4_score(q, lse, pages, table, n, out, KS)
    want, err = weights(pages, table, lens, [1], q, lse, hkv, d)
    assert ((out[0].double() - want[0]).abs() <= err[0]).all()
    lse[0, 1] = float("-inf")
    out.zero_()
    g.kv4_score(q, lse, pages, table, n, out, KS)
    assert (out - 1 / 333).abs().max() < 2.0 ** -15 / 333  # the lse is good to 2^-16 and a little


def test_no_rows(g):
    """Nothing is added; tokens without a score get one of 0."""
    pages, table, n = cached(g, [70, 0, 33], 16, 2, 64)
    old = torch.rand(3, 2, 80, device="cuda")
    q, lse = torch.empty(0, 8, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 8, device="cuda")
    out, st = torch.full_like(old, 9.0), ints([0])
    g.kv4_score(q, lse, pages, table, n, old, KS, q_start=ints([0] * 4), scored=ints([50, 0, 0]), out=out, dev_status=st)
    want = torch.full_like(old, 9.0)
    want[0, :, :50], want[0, :, 50:70], want[2, :, :33] = old[0, :, :50], 0, 0
    assert torch.equal(out, want) and st.item() == 0


def test_captured_and_replayed_on_a_side_stream(g):
    """In a graph, on another stream; lengths that have grown since the capture are read anew."""
    hq, hkv, d, lens = 8, 2, 128, [300, 90]
    pages, table, n = cached(g, lens, 64, hkv, d)
    n.copy_(ints([290, 80]))
    q = queries(2, hq, d, seed=6)
    lse = torch.empty(2, hq, device="cuda")
    scores = torch.zeros(2, hkv, 320, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        g.kv4_decode(q, pages, table, n, KS, VS, lse=lse)
        g.kv4_score(q, lse, pages, table, n, scores, KS)
        n.add_(1)

    with torch.cuda.stream(s):
        step()
        torch.cuda.synchronize()
        n.copy_(ints([290, 80]))
        scores.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
        for _ in range(5):
            graph.replay()
    torch.cuda.synchronize()
    got = scores.clone()
    n.copy_(ints([290, 80]))
    scores.zero_()
    for _ in range(5):
        step()
    assert torch.equal(got, scores) and (got[0, :, 294:] == 0).all() and (got[0, :, 293] > 0).all()
