"""Rows of a batch that hold no token, and what the 4-bit KV cache's calls do with them."""
import pytest

from test_gpu_kv4 import KS, VS, queries
from test_gpu_kv4 import setup as cached

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def g():
    import nvfp4_gated_deltanet_gb300 as pkg
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return pkg


# new rows and tokens of each sequence: fewer tokens than rows, none, as many, more; in and beyond a group of 16
@pytest.mark.parametrize("d,hkv", [(64, 3), (128, 8)])
@pytest.mark.parametrize("counts,lens", [([3, 4, 5], [2, 0, 5]), ([40, 17, 16], [1, 0, 16]), ([16, 33, 70], [15, 17, 100]),
                                         ([1, 1], [0, 0]), ([300], [0]), ([5] * 50, [3] * 50)])
def test_read_writes_zeros_where_a_row_has_no_token(g, counts, lens, d, hkv):
    pages, tab, n, *_ = cached(g, lens, 16, hkv, d)
    T = sum(counts)
    start = torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32, device="cuda")
    full = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    whole = g.kv4_read(pages, tab, n, KS, VS, sum(lens), q_start=full)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = (torch.full((T, hkv, d), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g.kv4_read(pages, tab, n, KS, VS, T, q_start=start, k=k, v=v, dev_status=st)
    for x, y in zip((k, v), whole):
        for b, (m, have) in enumerate(zip(counts, lens)):
            rows, left = x[start[b]:start[b + 1]], max(0, m - have)
            assert (rows[:left] == 0).all()
            assert torch.equal(rows[left:], y[full[b + 1] - (m - left):full[b + 1]])
    if len(set(counts)) == 1:                        # the same without row starts
        for x, y in zip(g.kv4_read(pages, tab, n, KS, VS, T, dev_status=st), (k, v)):
            assert torch.equal(x, y)
    assert st.item() == 0
