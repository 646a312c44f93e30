"""kv4_score of steps by how many rows a sequence and KV head has: up to 8, up to 16 (two
blocks of query columns) and more (tiles), against float64 within the bounds of
kv4_inputs.weights."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if torch.cuda.is_available():
    from kv4_inputs import KS, VS, ints, prefixed, queries, weights
    from test_gpu_kv4_score import attend, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import nvfp4_gated_deltanet_gb300 as pkg
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return pkg


def score_step(g, pages, table, n, lens, q, hkv, d, r, seed):
    B = len(lens)
    q4 = q.unflatten(0, (B, r))
    lse = g.kv4_decode(q4, pages, table, n, KS, VS, return_lse=True)[1]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    before = torch.rand(B + 1, hkv, max(lens) + 3, generator=gen, device="cuda")
    slots, scored = list(range(B, 0, -1)), [max(0, m - r) for m in lens]
    status, out = ints([0]), before.clone()
    g.kv4_score(q4, lse, pages, table, n, out, KS, slots=ints(slots), scored=ints(scored), dev_status=status)
    want, err = weights(pages, table, lens, [r] * B, q, lse.flatten(0, 1), hkv, d)
    check(out, before, slots, scored, lens, want, err)
    assert status.item() == 0
    return lse, before, out


@pytest.mark.parametrize("hq,hkv,r", [
    (8, 1, 1), (4, 2, 4),                               # 8 rows
    (9, 1, 1), (3, 1, 3),                               # 9
    (12, 2, 2), (12, 1, 1),                             # 12
    (16, 1, 1), (8, 2, 4), (4, 4, 16), (5, 1, 3),       # 16 (and 15)
    (17, 1, 1), (34, 2, 1),                             # 17: the first that are tiles
])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_a_step(g, hq, hkv, r, d):
    """Candidates across a unit of 64 tokens' end and a tile's, sequences shorter than their rows, empty ones."""
    lens = [700, 64 + r // 2, 129, max(1, r - 1), 0, 64, 1, 1030]
    pages, table, n, *_ = prefixed(g, [(0, lens)], 16, hkv, d, seed=hq + r)
    B = len(lens)
    q = queries(B * r, hq, d, seed=hq)
    lse, before, out = score_step(g, pages, table, n, lens, q, hkv, d, r, seed=r)
    # the second block's rows count as the first's: heads in the other order give the same sums, up to their order
    back = torch.arange(hq - 1, -1, -1, device="cuda").view(hkv, hq // hkv).flip(0).flatten()
    other = before.clone()
    g.kv4_score(q.unflatten(0, (B, r))[:, :, back].contiguous(), lse[:, :, back].contiguous(), pages, table, n, other, KS,
                slots=ints(list(range(B, 0, -1))), scored=ints([max(0, m - r) for m in lens]))
    want, err = weights(pages, table, lens, [r] * B, q, lse.flatten(0, 1), hkv, d)
    check(other, before, list(range(B, 0, -1)), [max(0, m - r) for m in lens], lens, want, err)


@pytest.mark.parametrize("hq,hkv,counts", [
    (4, 1, [2, 0, 1, 1]),                               # T G = 16, one to eight rows each
    (3, 1, [1, 2, 0, 1]),                               # 12
    (16, 4, [0, 3, 0, 1]),                              # 16
    (9, 1, [0, 0, 1, 0]),                               # 9
    (1, 1, [13, 0, 0, 2]),                              # 15: 13 rows of one sequence
])
@pytest.mark.parametrize("d", [64, 128])
def test_ragged_rows(g, hq, hkv, counts, d):
    lens = [70, 515, 64, 2000]
    pages, table, n, *_ = prefixed(g, [(0, lens)], 32, hkv, d, seed=hq)
    T = sum(counts)
    q = queries(T, hq, d, seed=T)
    start, lse = attend(g, q, pages, table, n, counts)
    before = torch.rand(4, hkv, 2000, generator=torch.Generator(device="cuda").manual_seed(T), device="cuda")
    scored = [max(0, m - c) for m, c in zip(lens, counts)]
    status, out = ints([0]), before.clone()
    g.kv4_score(q, lse, pages, table, n, out, KS, q_start=start, scored=ints(scored), dev_status=status)
    want, err = weights(pages, table, lens, counts, q, lse, hkv, d)
    check(out, before, [0, 1, 2, 3], scored, lens, want, err)
    assert status.item() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("r", [1, 2])
def test_extreme_rows_of_the_second_block(g, d, r):
    """A row of zeros, large ones, tiny ones and one left out, among 9 to 16."""
    hq, lens = 16 // r, [333, 90]
    pages, table, n, *_ = prefixed(g, [(0, lens)], 64, 1, d, seed=2)
    q = queries(2 * r, hq, d, seed=1)
    q[:, hq - 1] = 0
    q[:, hq - 2] *= 200
    q[:, hq - 3] *= 2.0 ** -40
    lse = g.kv4_decode(q.unflatten(0, (2, r)), pages, table, n, KS, VS, return_lse=True)[1]
    lse[:, :, hq - 4] = float("-inf")
    out = torch.zeros(2, 1, 333, device="cuda")
    g.kv4_score(q.unflatten(0, (2, r)), lse, pages, table, n, out, KS)
    want, err = weights(pages, table, lens, [r, r], q, lse.flatten(0, 1), 1, d)
    for x, m, w, e in zip(out, lens, want, err):
        assert ((x[:, :m].double() - w).abs() <= e).all()
