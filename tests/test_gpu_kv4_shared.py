"""kv4_decode_shared on the GPU against attention in float64, within the bounds of
kv4_decode: whatever the groups are, the result is each sequence's own attention."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if torch.cuda.is_available():
    from kv4_inputs import KS, VS, attention, close, ints, prefixed, queries

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import nvfp4_gated_deltanet_gb300 as pkg
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return pkg


def run(g, groups, page, hq, hkv, d, r, seed=0, **kw):
    pages, table, n, start, shared, lens = prefixed(g, groups, page, hkv, d, seed)
    B = len(lens)
    q = queries(B * r, hq, d, seed)
    st = ints([0])
    out, lse = g.kv4_decode_shared(q.unflatten(0, (B, r)), pages, table, n, start, shared, KS, VS, return_lse=True,
                                   dev_status=st, **kw)
    close(out, lse, attention(pages, table, lens, [r] * B, q, d), d)
    assert st.item() == 0
    return pages, table, n, start, shared, q.unflatten(0, (B, r)), out, lse


@pytest.mark.parametrize("groups,page,hq,hkv,d,r", [
    ([(64, [65, 70, 64, 100])], 16, 8, 2, 128, 1),            # one of them has no token of its own
    ([(512, [520, 600, 513])], 64, 4, 4, 64, 1),
    ([(128, [130, 140]), (0, [40]), (256, [300, 257, 256])], 32, 8, 1, 128, 2),
    ([(100, [140, 120])], 16, 4, 2, 64, 3),                   # part of a page: each reads it for itself
    ([(200, [150, 90, 230])], 16, 4, 2, 128, 1),              # members shorter than what the group claims
    ([(64, [0, 80, 0, 90])], 16, 8, 2, 64, 1),                # padding rows, the first among them
    ([(64, [0, 0])], 16, 8, 2, 64, 1),                        # nothing but padding
    ([(64, [64, 64])], 64, 8, 2, 128, 4),                     # candidates inside the shared page: nothing is shared
    ([(1000, [1100] * 20)], 128, 16, 1, 128, 1),              # 320 rows per KV head
    ([(1000, [1000 + 7 * i for i in range(1, 70)])], 8 * 16, 8, 1, 64, 4),   # 2208 rows
    ([(300, [400] * 3)] * 7, 16, 6, 2, 128, 1),               # 3 heads per KV head, many groups
    ([(256, [300, 310])], 256, 64, 1, 64, 1),
    ([(5000, [5001, 5300])], 64, 8, 8, 128, 1),               # a long prefix for few rows
    ([(3001, [3100] * 9), (2000, [2500] * 30)], 16, 10, 2, 64, 1),
])
def test_shared(g, groups, page, hq, hkv, d, r):
    run(g, groups, page, hq, hkv, d, r, seed=len(groups) + r)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shared", [16, 48, 64, 112, 128, 144, 272, 1040])
def test_prefix_ends_anywhere_in_a_tile(g, shared, d):
    run(g, [(shared, [shared + 1 + i for i in range(5)])], 16, 8, 2, d, 1, seed=shared)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (5, 1), (14, 2), (48, 1), (64, 1)])
def test_heads_per_kv_head(g, hq, hkv):
    run(g, [(320, [330, 400, 340])], 16, hq, hkv, 128, 2, seed=hq)


def test_same_as_decode(g):
    """No groups, groups of one, nothing shared: kv4_decode's own result, up to the order of sums."""
    pages, table, n, start, shared, q, out, lse = run(g, [(640, [700, 900, 641])], 64, 8, 2, 128, 1)
    want, wl = g.kv4_decode(q, pages, table, n, KS, VS, return_lse=True)
    for st, sh in (([0], []), ([0, 1, 2, 3], [640] * 3), ([0, 3], [0]), ([1, 2], [640]), ([1, 1, 3], [5, 640]), ([0, 3], [640])):
        o, l = g.kv4_decode_shared(q, pages, table, n, ints(st), ints(sh), KS, VS, return_lse=True)
        assert (o.float() - want.float()).abs().max() <= 2.0 ** -8 * want.float().abs().max()
        assert (l - wl).abs().max() < 1e-5


def test_bad_groups_share_nothing_and_bounds_hold(g):
    pages, table, n, start, shared, q, out, lse = run(g, [(640, [700, 900, 641])], 64, 8, 2, 128, 1)
    want = attention(pages, table, n.tolist(), [1] * 3, q.flatten(0, 1), 128)
    for st, sh in (([0, 4], [640]), ([-1, 3], [640]), ([2, 1], [640]), ([0, 2, 1, 3], [640] * 3), ([0, 3], [-5]),
                   ([0, 2 ** 31 - 1], [640]), ([-2 ** 31, 3], [640])):
        status = ints([0])
        o, l = g.kv4_decode_shared(q, pages, table, n, ints(st), ints(sh), KS, VS, return_lse=True, dev_status=status)
        close(o, l, want, 128)
        assert status.item() == 6
    for sh, most in ((640, 639), (640, 0), (2 ** 31 - 1, None), (2 ** 31 - 1, 64)):    # no more than max_shared is shared
        status = ints([0])
        o, l = g.kv4_decode_shared(q, pages, table, n, start, ints([sh]), KS, VS, max_shared=most, return_lse=True,
                                   dev_status=status)
        close(o, l, want, 128)
        assert status.item() == 0


def test_bad_lengths_and_pages_are_flagged(g):
    pages, table, n, start, shared, q, out, lse = run(g, [(640, [700, 900, 641])], 64, 8, 2, 128, 1)
    for bad in (-1, 64 * table.shape[1] + 1, 2 ** 31 - 1):
        m, status = n.clone(), ints([0])
        m[1] = bad
        o, l = g.kv4_decode_shared(q, pages, table, m, start, shared, KS, VS, return_lse=True, dev_status=status)
        assert status.item() == 6 and torch.isinf(l[1]).all()
        want = attention(pages, table, [700, 0, 641], [1] * 3, q.flatten(0, 1), 128)
        close(o, l, want, 128)
    for row, col in ((0, 3), (1, 12)):
        t, status = table.clone(), ints([0])
        t[row, col] = 10 ** 6
        g.kv4_decode_shared(q, pages, t, n, start, shared, KS, VS, dev_status=status)
        assert status.item() == 6


def test_repeats_and_given_outputs(g):
    """Bit-identical from call to call, in given outputs and a workspace full of NaN, on a side stream."""
    pages, table, n, start, shared, q, out, lse = run(g, [(1024, [1100] * 9), (512, [700] * 5)], 64, 16, 2, 128, 2)
    for _ in range(3):
        o, l = g.kv4_decode_shared(q, pages, table, n, start, shared, KS, VS, return_lse=True)
        assert torch.equal(o, out) and torch.equal(l, lse)
    ws = torch.full((1 << 24,), float("nan"), device="cuda")
    o, l = torch.full_like(out, 3.0), torch.full_like(lse, 3.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = g.kv4_decode_shared(q, pages, table, n, start, shared, KS, VS, max_shared=1024, out=o, lse=l, workspace=ws, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert got.data_ptr() == o.data_ptr() and torch.equal(o, out) and torch.equal(l, lse)


def test_captured_lengths_grow(g):
    """One graph for all steps: lengths, and with them what is shared, are read at the replay."""
    pages, table, n, start, shared, q, out, lse = run(g, [(320, [350, 400, 330])], 64, 8, 2, 128, 1)
    full = n.clone()
    n.copy_(ints([300, 321, 330]))          # the first has not come to the end of the shared pages
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        o, l = g.kv4_decode_shared(q, pages, table, n, start, shared, KS, VS, return_lse=True)
    for lens in ([300, 321, 330], [350, 400, 330], [320, 320, 320], [0, 1, 330]):
        n.copy_(ints(lens))
        graph.replay()
        torch.cuda.synchronize()
        close(o, l, attention(pages, table, lens, [1] * 3, q.flatten(0, 1), 128), 128)
    n.copy_(full)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, out)


def test_two_calls_at_once(g):
    """On two streams, each with its own scratch."""
    a = run(g, [(2048, [2100] * 16)], 64, 16, 4, 128, 1, seed=1)
    b = run(g, [(1536, [1600] * 16)], 64, 16, 4, 128, 1, seed=2)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for x, st in ((a, s), (b, t)):
            got.append((x, g.kv4_decode_shared(x[5], *x[:5], KS, VS, stream=st)))
    torch.cuda.synchronize()
    for x, o in got:
        assert torch.equal(o, x[6])


def test_queries_of_extreme_size(g):
    """Rows of zeros, and rows so large that one key has all the weight."""
    pages, table, n, start, shared, lens = prefixed(g, [(640, [700, 900])], 64, 2, 128, 3)
    q = queries(2, 8, 128, 3)
    q[0, 0], q[0, 1], q[1, 3] = 0, q[0, 1] * 300, q[1, 3] * 2.0 ** -40
    out, lse = g.kv4_decode_shared(q, pages, table, n, start, shared, KS, VS, return_lse=True)
    close(out, lse, attention(pages, table, lens, [1, 1], q, 128), 128)


@pytest.mark.parametrize("d", [64, 128])
def test_maximum_that_moves(g, d):
    """Queries up to forty times as large: their maximum rises in several tiles of the prefix, in some rows of a warp only."""
    pages, table, n, start, shared, lens = prefixed(g, [(4000, [4100, 4001, 4200, 4030, 4007])], 32, 2, d, 8)
    q = queries(5, 16, d, 8)
    q *= torch.tensor([1, 4, 13, 40], device="cuda").repeat(4)[None, :, None]
    out, lse = g.kv4_decode_shared(q, pages, table, n, start, shared, KS, VS, return_lse=True)
    close(out, lse, attention(pages, table, lens, [1] * 5, q, d), d)
