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


@pytest.mark.parametrize("hq,hkv,d,counts", [
    (4, 1, 64, [1, 1, 0]),                              # up to 8 rows, up to 16, and tiles
    (8, 2, 128, [2, 1, 1]),
    (8, 1, 64, [1, 1, 0]),
    (6, 1, 128, [2, 0, 0]),
    (8, 2, 128, [300, 40, 7]),
    (5, 1, 64, [130, 0, 90]),
])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_a_row_left_out_of_the_scores_may_hold_anything(g, hq, hkv, d, counts, what):
    """lse = -infinity: the row adds nothing, whatever its queries are."""
    lens = [700, 400, 129]
    pages, table, n, *_ = prefixed(g, [(0, lens)], 16, hkv, d, seed=hq)
    T = sum(counts)
    start = ints(np.concatenate([[0], np.cumsum(counts)]).tolist())
    q = queries(T, hq, d, seed=3)
    lse = g.kv4_prefill(q, pages, table, n, start, KS, VS, return_lse=True)[1]
    gen = torch.Generator(device="cuda").manual_seed(4)
    out_of = torch.rand(T, hq, generator=gen, device="cuda") < 0.3
    out_of[0, 0] = True
    lse[out_of] = float("-inf")
    bad = q.clone()
    bad[out_of] = what
    bad[out_of & (torch.rand(T, hq, generator=gen, device="cuda") < 0.5)] *= -1
    q[out_of] = 0
    a, b = torch.zeros(2, 3, hkv, 700, device="cuda")
    g.kv4_score(q, lse, pages, table, n, a, KS, q_start=start)
    g.kv4_score(bad, lse, pages, table, n, b, KS, q_start=start)
    assert torch.equal(a, b) and torch.isfinite(a).all()
    want, err = weights(pages, table, lens, counts, q, lse, hkv, d)
    for x, m, w, e in zip(a, lens, want, err):
        assert ((x[:, :m].double() - w).abs() <= e).all()


@pytest.mark.parametrize("hq,r", [(2, 1), (8, 2), (8, 40)])
@pytest.mark.parametrize("graph", [False, True])
def test_scores_of_tokens_written_right_before(g, graph, hq, r):
    """Scores right behind an append, and behind an eviction, whose kernels may still run when the score's begins:
    they see the new bytes in pages that earlier scores have read."""
    hkv, d, n, keep = 1, 128, 2000, 512
    pages, table, kv, *_ = prefixed(g, [(0, [n])], 64, hkv, d, seed=5, spare=8)
    used = set(table[0].tolist())
    new = ints([[p for p in range(pages.shape[0]) if p not in used][:8]])
    steps = 6
    ks, vs = rows(steps * n, hkv, d, 1).view(steps, n, hkv, d), rows(steps * n, hkv, d, 2).view(steps, n, hkv, d)
    q = queries(r, hq, d, 3)[None]
    lse = torch.full((1, r, hq), 5.0, device="cuda")
    rank = torch.rand(steps, 1, hkv, n, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda")
    sums, moved = torch.zeros(steps, 1, hkv, n, device="cuda"), torch.zeros(steps, 1, hkv, n, device="cuda")
    kept, count, limit = torch.zeros(1, hkv, keep, dtype=torch.int32, device="cuda"), ints([keep]), ints([keep])
    aside = torch.zeros_like(rank[0])

    def run(wait):
        for i in range(steps):
            g.kv4_append(ks[i], vs[i], pages, table, kv, KS, VS)
            wait()
            g.kv4_score(q, lse, pages, table, kv, sums[i], KS)
            wait()
            g.kv4_evict(pages, table, kv, limit, 8, rank[i], new, kept=kept, new_len=count, scores_out=aside)
            wait()
            g.kv4_score(q, lse, pages, new, limit, moved[i], KS)
            wait()

    run(torch.cuda.synchronize)
    want = sums.clone(), moved.clone()
    assert (want[0][1:] != want[0][:-1]).any(-1).all() and (want[1][1:] != want[1][:-1]).any(-1).all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step = lambda: run(lambda: None)
        if graph:
            G = torch.cuda.CUDAGraph()
            with torch.cuda.graph(G, stream=s):
                run(lambda: None)
            step = G.replay
        for _ in range(10):
            sums.zero_(), moved.zero_()
            step()
            torch.cuda.synchronize()
            assert torch.equal(sums, want[0]) and torch.equal(moved, want[1])


@pytest.mark.parametrize("groups,page,hq,hkv,d,r", [
    ([(64, [0, 80, 0])], 16, 8, 2, 64, 1),
    ([(5000, [5100, 0, 0, 0])], 64, 16, 2, 128, 2),
    ([(320, [0, 0, 400]), (128, [0, 130]), (64, [70])], 16, 4, 4, 64, 1),
])
def test_members_without_tokens_do_not_count(g, groups, page, hq, hkv, d, r):
    """A group with one member that has tokens, as a batch padded to a fixed size has it, reads for itself: bit for bit
    as without a group. (kv_len 0: padding.)"""
    pages, table, n, start, shared, lens = prefixed(g, groups, page, hkv, d, seed=len(groups))
    B = len(lens)
    q = queries(B * r, hq, d, 5).unflatten(0, (B, r))
    st = ints([0])
    out, lse = g.kv4_decode_shared(q, pages, table, n, start, shared, KS, VS, return_lse=True, dev_status=st)
    want, wlse = g.kv4_decode_shared(q, pages, table, n, ints([0]), ints([]), KS, VS, return_lse=True)
    close(out, lse, attention(pages, table, lens, [r] * B, q.flatten(0, 1), d), d)
    assert torch.equal(out, want) and torch.equal(lse, wlse) and st.item() == 0


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("d,hq,hkv", [(128, 16, 2), (64, 8, 4)])
def test_other_lengths_call_after_call_in_one_workspace(g, graph, d, hq, hkv):
    """Nothing of one call's plan, sums or pieces is read by the next one, which begins while it ends: batches of other
    lengths, tables and groups in turn, all in the same workspace and outputs."""
    pages, table, n, start, shared, lens = prefixed(g, [(4096, [4200, 5000, 4111, 4096]), (640, [700, 9000, 2000])], 64, hkv, d)
    q = queries(7, hq, d, 2)
    back = torch.tensor([3, 2, 1, 0, 6, 5, 4], device="cuda")
    batches = [(table, n, start, shared), (table[back].contiguous(), n[back].contiguous(), start, shared),
               (table, ints([4097, 0, 4096, 0, 640, 641, 650]), start, ints([4096, 64])),
               (table, ints([1, 5000, 70, 0, 0, 9000, 0]), ints([0, 1, 7]), ints([64, 0])),
               (table, n, start, ints([0, 0])), (table, ints([4096, 4200, 4111, 4000, 700, 8999, 1]), start, shared)]
    batches = [b for _ in range(4) for b in batches]
    ws = torch.full((1 << 23,), float("nan"), device="cuda")
    outs = [torch.zeros(7, hq, d, dtype=torch.bfloat16, device="cuda") for _ in batches]
    lses = [torch.zeros(7, hq, device="cuda") for _ in batches]

    def run(wait=lambda: None):
        for b, o, l in zip(batches, outs, lses):
            g.kv4_decode_shared(q, pages, *b, KS, VS, out=o, lse=l, workspace=ws)
            wait()

    def each_alone():
        ws.fill_(float("nan"))
        torch.cuda.synchronize()

    run(each_alone)
    want = [o.clone() for o in outs], [l.clone() for l in lses]
    for b, o, l in zip(batches[:6], *want):
        close(o, l, attention(pages, b[0], b[1].tolist(), [1] * 7, q, d), d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step = run
        if graph:
            G = torch.cuda.CUDAGraph()
            with torch.cuda.graph(G, stream=s):
                run()
            step = G.replay
        for _ in range(20):
            for o in outs:
                o.zero_()
            step()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(outs, want[0])) and all(torch.equal(x, y) for x, y in zip(lses, want[1]))
