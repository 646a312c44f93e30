"""A wait of the 4-bit KV cache's kernels that runs out reports GDN_E_TIMEOUT and
leaves the context usable: with a budget of one SM cycle (tuning knob 12) they
give up on whatever is not there at once, wait for their copies in flight and
end. The next call, with the default budget, is right."""
import pytest

from test_gpu_kv4 import KS, VS, queries
from test_gpu_kv4 import setup as cached

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

GDN_E_TIMEOUT = 10


@pytest.fixture(scope="module")
def g():
    import nvfp4_gated_deltanet_gb300 as pkg
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return pkg


@pytest.fixture()
def short(g):
    """Set (True) and take back (False) a wait budget of one cycle."""
    def budget(on):
        assert g.lib().gdn_set_tuning(12, int(on)) == 0
    yield budget
    budget(False)


# sequences, tokens each, r, hq, hkv, d, page: whole CTAs and teams of four warps, all column blocks, items cut and
# whole; each warp goes through several tiles, and 90 MB or more, so that tiles are waited for
DECODE = [(1, 200000, 1, 16, 4, 128, 64), (200, 3000, 1, 16, 2, 128, 64), (24, 14000, 4, 16, 4, 64, 32),
          (8, 40000, 8, 8, 2, 128, 128), (90, 8000, 8, 8, 2, 64, 64), (60, 6000, 2, 32, 4, 128, 64), (160, 500, 1, 8, 8, 128, 64)]


@pytest.mark.parametrize("B,n,r,hq,hkv,d,page", DECODE)
def test_decode(g, short, B, n, r, hq, hkv, d, page):
    pages, tab, lens, *_ = cached(g, [n - 7 * (b % 5) for b in range(B)], page, hkv, d, seed=B)
    q = queries(B * r, hq, d, r).reshape(B, r, hq, d)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = g.kv4_decode(q, pages, tab, lens, KS, VS, return_lse=True, dev_status=st)
    assert st.item() == 0
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for _ in range(4):
        flush.fill_(1)                               # out of L2
        short(True)
        g.kv4_decode(q, pages, tab, lens, KS, VS, dev_status=st)
        assert st.item() == GDN_E_TIMEOUT
        short(False)
        st.zero_()
        got = g.kv4_decode(q, pages, tab, lens, KS, VS, return_lse=True, dev_status=st)
        assert st.item() == 0 and all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("lens,hkv,d", [([20000, 12001, 9, 33], 8, 128), ([700] * 40, 3, 64), ([1, 5], 1, 128)])
def test_append(g, short, lens, hkv, d):
    page = 32
    pages, tab, n, k, v, start = cached(g, lens, page, hkv, d, spare=4)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    unused = sorted(set(range(pages.shape[0])) - set(tab[tab >= 0].tolist()))
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for _ in range(4):
        again = torch.full_like(pages, 0x7F)
        flush.fill_(1)
        short(True)
        g.kv4_append(k, v, again, tab, n, KS, VS, q_start=start, dev_status=st)
        assert st.item() == GDN_E_TIMEOUT and (again[unused] == 0x7F).all()
        short(False)
        st.zero_()
        g.kv4_append(k, v, again, tab, n, KS, VS, q_start=start, dev_status=st)
        assert st.item() == 0 and torch.equal(again, pages)


@pytest.mark.parametrize("counts,lens,hq,hkv,d,page", [([2000, 900, 33], [6000, 900, 5000], 16, 4, 128, 64), ([700], [700], 8, 2, 64, 16),
                                                       ([3000, 3000], [9000, 3001], 32, 8, 64, 64), ([70] * 9, [3000] * 9, 8, 1, 128, 32)])
def test_prefill(g, short, counts, lens, hq, hkv, d, page):
    """With one cycle every role gives up at its first wait; with more of them in the middle of an item, or not at all."""
    pages, tab, n, *_ = cached(g, lens, page, hkv, d, seed=len(lens))
    T = sum(counts)
    q = queries(T, hq, d, T)
    start = torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(total_kv=sum(lens), return_lse=True, dev_status=st)
    want = g.kv4_prefill(q, pages, tab, n, start, KS, VS, **kw)
    assert st.item() == 0
    for budget in (1, 1, 300, 1000, 2000, 4000, 8000, 16000):
        short(budget)
        g.kv4_prefill(q, pages, tab, n, start, KS, VS, **kw)
        assert st.item() == GDN_E_TIMEOUT or (budget > 1 and st.item() == 0)
        short(0)
        st.zero_()
        got = g.kv4_prefill(q, pages, tab, n, start, KS, VS, **kw)
        assert st.item() == 0 and all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("B,n,r,hq,hkv,d,page", DECODE)
def test_decode_gives_up_midway(g, short, B, n, r, hq, hkv, d, page):
    pages, tab, lens, *_ = cached(g, [n - 7 * (b % 5) for b in range(B)], page, hkv, d, seed=B)
    q = queries(B * r, hq, d, r).reshape(B, r, hq, d)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = g.kv4_decode(q, pages, tab, lens, KS, VS, dev_status=st)
    for budget in (200, 600, 1500, 3000, 6000):
        short(budget)
        g.kv4_decode(q, pages, tab, lens, KS, VS, dev_status=st)
        assert st.item() in (0, GDN_E_TIMEOUT)
        short(0)
        st.zero_()
        assert torch.equal(g.kv4_decode(q, pages, tab, lens, KS, VS, dev_status=st), want) and st.item() == 0
