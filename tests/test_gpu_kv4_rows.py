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


def dirty(like):
    """Leave NaN in the memory that the next tensors of these sizes are made of."""
    held = [torch.full_like(x, float("nan")) for x in like for _ in range(3)]
    del held


@pytest.mark.parametrize("d,hkv,hq,pad", [(64, 2, 6, 1), (128, 8, 16, 37), (128, 1, 64, 700)])
def test_padding_rows(g, d, hkv, hq, pad):
    """Rows from q_start[B] on: zeros (lse -infinity) in outputs that a call makes, left alone in given ones."""
    counts, lens = [3, 40, 1], [20, 40, 0]
    pages, tab, n, *_ = cached(g, lens, 16, hkv, d)
    T = sum(counts)
    start = torch.tensor([0, 3, 43, 44], dtype=torch.int32, device="cuda")
    q = queries(T + pad, hq, d, 1)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def read(**kw):
        return g.kv4_read(pages, tab, n, KS, VS, T + pad, q_start=start, dev_status=st, **kw)

    def prefill(**kw):
        return g.kv4_prefill(q, pages, tab, n, start, KS, VS, return_lse=True, dev_status=st, **kw)

    for call, names, rest in ((read, ("k", "v"), (0.0, 0.0)), (prefill, ("out", "lse"), (0.0, -float("inf")))):
        want = [x.clone() for x in call()]
        for x, z in zip(want, rest):
            assert not x[:T].isnan().any() and (x[T:] == z).all()
        for _ in range(3):
            dirty(want)
            got = call()
            assert all(torch.equal(x, y) for x, y in zip(got, want))
            del got
        for mine in (names, names[:1], names[1:]):   # both given, one of the two
            given = {m: torch.full_like(want[names.index(m)], 7.0) for m in mine}
            dirty(want)
            for m, x, y, z in zip(names, call(**given), want, rest):
                assert torch.equal(x[:T], y[:T]) and (x[T:] == (7.0 if m in mine else z)).all()
    assert st.item() == 0


@pytest.mark.parametrize("rows", [[0, 4], [2, 1], [-1, 3], [0, -1], [4, 4], [0, 2 ** 31 - 1], [-2 ** 31, 0]])
def test_bad_row_starts_are_flagged_and_write_nothing(g, rows):
    """Row starts that do not ascend or leave the batch's three rows: GDN_E_RANGE from every call that takes them."""
    hkv, hq, d = 2, 8, 128
    x = torch.randn(3, hkv, d, device="cuda").bfloat16()
    q = queries(3, hq, d, 0)
    tab = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    n = torch.tensor([3], dtype=torch.int32, device="cuda")
    start = torch.tensor(rows, dtype=torch.int32, device="cuda")
    pages, st = g.kv4_new_pages(2, 16, hkv, d), torch.zeros(1, dtype=torch.int32, device="cuda")
    g.kv4_append(x, x, pages, tab, n, KS, VS, q_start=start, dev_status=st)
    assert st.item() == 6 and not pages.any()
    st.zero_()
    g.kv4_read(pages, tab, n, KS, VS, 3, q_start=start, dev_status=st)
    assert st.item() == 6
    st.zero_()
    g.kv4_prefill(q, pages, tab, n, start, KS, VS, dev_status=st)
    assert st.item() == 6 and not pages.any()


# whole-CTA teams and teams of four, cut items of 8, 16 and 32 rows
@pytest.mark.parametrize("B,n,r,hq,hkv,d", [(2, 9000, 1, 8, 2, 128), (90, 900, 1, 16, 2, 128), (5, 6000, 4, 16, 4, 64),
                                            (3, 5000, 8, 8, 2, 128)])
def test_decode_in_a_workspace_of_exactly_its_size(g, B, n, r, hq, hkv, d):
    """A caller's workspace, full of NaN, with bytes after it that stay: the result of the call's own."""
    import ctypes
    pages, tab, lens, *_ = cached(g, [n - 9 * b for b in range(B)], 64, hkv, d)
    q = queries(B * r, hq, d, r).reshape(B, r, hq, d)
    c = g.Kv4CacheStruct(pages.data_ptr(), pages.shape[0], 64, hkv, d, KS, VS)
    b = g.Kv4BatchStruct(lens.data_ptr(), tab.data_ptr(), None, B, tab.shape[1], B * r)
    need = g.lib().kv4_decode_workspace(ctypes.byref(c), ctypes.byref(b), hq)
    assert need > 0
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = g.kv4_decode(q, pages, tab, lens, KS, VS, return_lse=True)
    room = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        got = g.kv4_decode(q, pages, tab, lens, KS, VS, return_lse=True, workspace=room[:need], dev_status=st)
        assert all(torch.equal(x, y) for x, y in zip(got, want)) and (room[need:] == 0xFF).all() and st.item() == 0
    with pytest.raises(g.GdnError, match="GDN_E_SHAPE"):
        g.kv4_decode(q, pages, tab, lens, KS, VS, workspace=room[:need - 1])


@pytest.mark.parametrize("bad", [[0, 5, -1], [0, 5, 3], [0, 5, 99], [0, 5, 0], [0, 5, -2 ** 31]])
def test_a_bad_row_start_takes_no_rows_from_other_sequences(g, bad):
    """The first sequence's rows are as with good row starts, in outputs that the calls make."""
    hkv, hq, d, T = 2, 8, 128, 40
    pages, tab, n, *_ = cached(g, [30, 20], 16, hkv, d)
    q = queries(T, hq, d, 3)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def both(start):
        start = torch.tensor(start, dtype=torch.int32, device="cuda")
        return (*g.kv4_read(pages, tab, n, KS, VS, T, q_start=start, dev_status=st),
                *g.kv4_prefill(q, pages, tab, n, start, KS, VS, return_lse=True, dev_status=st))

    want = both([0, 5, 9])
    assert st.item() == 0
    for _ in range(20):
        got = both(bad)
        assert all(torch.equal(x[:5], y[:5]) for x, y in zip(got, want))
    assert st.item() == 6
