"""Prompts, samples that share one, scores and eviction together, as KV4Cache is
used for long contexts."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if torch.cuda.is_available():
    from kv4_inputs import KS, VS, attention, close, ints, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import nvfp4_gated_deltanet_gb300 as pkg
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return pkg


# How far a row's weights may be from 1 in all: each is off by at most (d + 10) 2^-24 sum |q k| sm (sums here stay
# below 60) and as much again with the lse, which has 2^-16 of its own: 74 * 60 * 2^-23 + 2^-16 < 2^-10
ONE = 2.0 ** -10


def rows(T, heads, d, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(T, heads, d, generator=gen, device="cuda").bfloat16()


def held(g, c, layer, seq):
    """The values a sequence's pages hold: K and V [tokens][Hkv][d]."""
    b = c.batch([seq], [c.book.length(seq)])
    return g.kv4_read(c.layers[layer], b.block_table, b.kv_len, KS, VS, b.T, q_start=b.q_start)


@pytest.mark.parametrize("stream", [False, True])
def test_samples_of_a_long_prompt(g, stream):
    hq, hkv, d, L = 8, 2, 64, 2
    with torch.cuda.stream(torch.cuda.Stream() if stream else torch.cuda.current_stream()):
        c = g.KV4Cache(300, 16, hkv, d, KS, VS, n_layers=L, score_slots=6, score_tokens=700)
        a, other = c.new(), c.new()
        prompt = [530, 45]
        batch = c.grow([a, other], prompt)
        for l in range(L):
            c.append(l, rows(575, hkv, d, l), rows(575, hkv, d, 10 + l), batch)
            q = queries(575, hq, d, 20 + l)
            _, lse = c.prefill(l, q, batch, return_lse=True)
            # the prompt's last 32 rows score it
            pick = torch.cat([torch.arange(530 - 32, 530), torch.arange(575 - 32, 575)]).cuda()
            c.score(l, q[pick], lse[pick].contiguous(), batch, q_start=ints([0, 32, 64]))
        assert ((c.scores[:, c._slot[a]].double().sum(-1) / (32 * hq // hkv) - 1).abs() < ONE).all()
        seqs = [a] + [c.fork(a) for _ in range(3)] + [other]
        for step in range(5):
            batch = c.grow(seqs, 1, share=True)
            assert batch.group_start.tolist() == [0, 4, 5] and batch.shared_len.tolist() == [528, 0]
            for l in range(L):
                c.append(l, rows(5, hkv, d, 100 + step + 7 * l), rows(5, hkv, d, 200 + step + 7 * l), batch)
                q = queries(5, hq, d, 300 + step + 7 * l)
                out, lse = c.decode_shared(l, q, batch, return_lse=True)
                lens = batch.kv_len.tolist()
                close(out, lse, attention(c.layers[l], batch.block_table, lens, [1] * 5, q, d), d)
                before = c.scores[l].double().sum(-1)
                c.score(l, q, lse, batch)
                more = c.scores[l].double().sum(-1) - before
                used = [c._slot[s] for s in seqs]                # (differences of sums: four times the bound)
                assert ((more[used] / (hq // hkv) - 1).abs() < 4 * ONE).all() and not more[[i for i in range(6) if i not in used]].any()
        # the prompt's owner and a sample are cut, the others keep theirs
        was = {(l, s): held(g, c, l, s) for l in range(L) for s in seqs}
        scores = {s: c.scores[:, c._slot[s]].clone() for s in seqs}
        free = c.book.free_pages
        cut, kept = c.evict([a, seqs[2], other], 100, recent=20)
        assert cut == [a, seqs[2]] and kept.shape == (L, 2, hkv, 100) and c.check() == 0
        assert c.book.free_pages == free - 2 * 7 + 2            # each gave up its last page, the prompt's are still shared
        for l in range(L):
            for i, s in enumerate(cut):
                for h in range(hkv):
                    at = kept[l, i, h].long()
                    x = scores[s][l, h, :535].clone()
                    assert (at[80:] == torch.arange(515, 535, device="cuda")).all() and (at.diff() > 0).all()
                    assert x[at[:80]].min() >= np.partition(x[:515].cpu().numpy(), -80)[-80]
                    for now, old in zip(held(g, c, l, s), was[l, s]):
                        assert torch.equal(now[:, h], old[at, h])
                    row = c.scores[l, c._slot[s], h]
                    assert torch.equal(row[:100], x[at]) and not row[100:535].any()
            for s in (seqs[1], seqs[3], other):
                assert all(torch.equal(x, y) for x, y in zip(held(g, c, l, s), was[l, s]))
                assert torch.equal(c.scores[:, c._slot[s]], scores[s])
        # and go on, in a batch with the others
        c.free(seqs.pop(1))
        c.compact()
        batch = c.grow(seqs, 2, share=True)
        for l in range(L):
            c.append(l, rows(8, hkv, d, 400 + l), rows(8, hkv, d, 500 + l), batch)
            q = queries(8, hq, d, 600 + l)
            out, lse = c.decode_shared(l, q.unflatten(0, (4, 2)), batch, return_lse=True)
            close(out, lse, attention(c.layers[l], batch.block_table, batch.kv_len.tolist(), [2] * 4, q, d), d)
            c.score(l, q, lse.flatten(0, 1), batch)
        assert batch.kv_len.tolist() == [102, 102, 537, 52] and batch.scored.tolist() == [100, 100, 535, 50]
        assert c.check() == 0


@pytest.mark.parametrize("which", ["shared", "evict"])
def test_outputs_for_a_stream_are_no_memory_that_another_still_writes(g, which):
    """A call on another stream than the current one must not get blocks for its outputs that the current stream
    has freed and still writes."""
    from kv4_inputs import prefixed
    pages, table, n, start, shared, lens = prefixed(g, [(1024, [1100] * 64)], 16, 2, 128)
    q = queries(64, 16, 128, 1)
    new = ints([[pages.shape[0] - 1]])
    scores = torch.rand(1, 2, 1200, device="cuda")

    def call(stream=None):
        if which == "shared":
            return g.kv4_decode_shared(q, pages, table, n, start, shared, KS, VS, return_lse=True, stream=stream)
        return g.kv4_evict(pages, table[:1], n[:1], ints([16]), 2, scores, new, max_keep=4096, scores_out=torch.empty_like(scores),
                           stream=stream)

    want = [x.clone() for x in call()]
    big = torch.randn(4096, 4096, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        held = [torch.empty_like(x) for x in want]
        for _ in range(20):
            big @ big
        for x in held:
            x.fill_(7)
        at = {x.data_ptr() for x in held}
        del held, x
        got = call(side)
        assert not at & {x.data_ptr() for x in got}
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        del got


@pytest.mark.parametrize("graph", [False, True])
def test_order_among_streams_and_other_kernels(g, graph):
    """Each call sees what came before it in its stream and only that: its inputs are written by other kernels
    right before it, and overwritten right after."""
    from kv4_inputs import prefixed
    pages, table, n, start, shared, lens = prefixed(g, [(512, [600, 530, 700, 513])], 16, 2, 64)
    q = queries(4, 8, 64, 5)
    want, wlse = g.kv4_decode_shared(q, pages, table, n, start, shared, KS, VS, return_lse=True)
    score = torch.zeros(4, 2, 700, device="cuda")
    g.kv4_score(q, wlse, pages, table, n, score, KS)
    new = ints([[i] for i in range(pages.shape[0], pages.shape[0] + 4)])
    more = torch.cat([pages, torch.zeros_like(pages[:4])])
    kept, _ = g.kv4_evict(more, table, n, ints([16] * 4), 4, score, new, scores_out=torch.empty_like(score))
    p2, q2, l2, t2, s2 = more.clone(), torch.zeros_like(q), torch.zeros_like(wlse), torch.zeros_like(table), torch.zeros_like(score)
    out, lse, k2, n2 = torch.zeros_like(want), torch.zeros_like(wlse), torch.zeros_like(kept), ints([0] * 4)
    moved = torch.zeros_like(score)
    sixteen, len2 = ints([16] * 4), torch.zeros_like(n)

    def run():
        p2[:-4].copy_(pages)
        q2.copy_(q)
        t2.copy_(table)
        len2.copy_(n)
        g.kv4_decode_shared(q2, p2, t2, len2, start, shared, KS, VS, out=out, lse=lse)
        l2.copy_(lse)
        s2.zero_()
        g.kv4_score(q2, l2, p2, t2, len2, s2, KS)
        q2.zero_()
        l2.zero_()
        g.kv4_evict(p2, t2, len2, sixteen, 4, s2, new, kept=k2, new_len=n2, scores_out=moved)
        p2[:-4].fill_(0x7F)
        t2.fill_(-1)
        len2.zero_()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        if graph:
            run()
            G = torch.cuda.CUDAGraph()
            with torch.cuda.graph(G, stream=s):
                run()
            step = G.replay
        else:
            step = run
        for _ in range(20):
            out.zero_(), k2.zero_(), s2.zero_()
            step()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(lse, wlse) and torch.equal(s2, score) and torch.equal(k2, kept)
            assert torch.equal(p2[-4:], more[-4:])


@pytest.mark.parametrize("members,pays", [(3, False), (40, True)])
def test_shared_where_that_pays(g, members, pays):
    """share="auto" is either attention: the same results, whichever it takes."""
    hq, hkv, d = 16, 8, 128
    c = g.KV4Cache(600, 64, hkv, d, KS, VS)
    root = c.new()
    c.append(0, rows(8192, hkv, d, 1), rows(8192, hkv, d, 2), c.grow([root], 8192))
    seqs = [c.fork(root) for _ in range(members)]
    batch = c.grow(seqs, 1, share="auto")
    assert batch.plain != pays
    c.append(0, rows(members, hkv, d, 3), rows(members, hkv, d, 4), batch)
    q = queries(members, hq, d, 5)
    out, lse = c.decode_shared(0, q, batch, return_lse=True)
    close(out, lse, attention(c.layers[0], batch.block_table, [8193] * members, [1] * members, q, d), d)
    assert c.check() == 0
