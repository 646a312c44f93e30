"""Waits of kv4_decode_shared's and kv4_score's kernels that run out report
GDN_E_TIMEOUT and leave the context usable: with a short budget (tuning knob 12)
they give up, wait for their copies in flight and end, and the next call is right."""
import pytest

torch = pytest.importorskip("torch")
if torch.cuda.is_available():
    from kv4_inputs import KS, VS, ints, prefixed, queries

pytestmark = pytest.mark.gpu
GDN_E_TIMEOUT = 10
BUDGETS = (1, 1, 300, 1000, 2000, 4000, 8000, 16000)


@pytest.fixture(scope="module")
def g():
    import nvfp4_gated_deltanet_gb300 as pkg
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return pkg


@pytest.fixture()
def short(g):
    def budget(cycles):
        assert g.lib().gdn_set_tuning(12, cycles) == 0
    yield budget
    budget(0)


def gives_up(short, call, out):
    """call(status) with short budgets and, each time after that, with the default one; out: its outputs."""
    st = ints([0])
    call(st)
    assert st.item() == 0
    want = [t.clone() for t in out]
    for budget in BUDGETS:
        short(budget)
        call(st)
        assert st.item() == GDN_E_TIMEOUT or (budget > 1 and st.item() == 0)
        short(0)
        st.zero_()
        call(st)
        assert st.item() == 0 and all(torch.equal(x, y) for x, y in zip(out, want))


@pytest.mark.parametrize("groups,page,hq,hkv,d,r", [([(9000, [9100] * 40)], 64, 8, 2, 128, 1),
                                                    ([(3000, [3500] * 9), (800, [900] * 3)], 16, 16, 4, 64, 2),
                                                    ([(640, [650, 700])] * 30, 32, 8, 4, 128, 1)])
def test_decode_shared(g, short, groups, page, hq, hkv, d, r):
    pages, table, n, start, shared, lens = prefixed(g, groups, page, hkv, d)
    B = len(lens)
    q = queries(B * r, hq, d, r).unflatten(0, (B, r))
    out, lse = torch.empty_like(q), torch.empty(B, r, hq, device="cuda")
    # scratch full of large numbers: what a kernel that gave up has not written may be anything
    ws = torch.full((1 << 27,), -1, dtype=torch.uint8, device="cuda")

    def call(st):
        ws.fill_(0x3C)
        g.kv4_decode_shared(q, pages, table, n, start, shared, KS, VS, out=out, lse=lse, workspace=ws, dev_status=st)

    gives_up(short, call, [out, lse])


@pytest.mark.parametrize("counts,lens,hq,hkv,d,page", [([900, 33], [5000, 700], 16, 4, 128, 64), ([700], [700], 8, 2, 64, 16),
                                                       ([64] * 5, [4000] * 5, 24, 2, 128, 32)])
def test_score(g, short, counts, lens, hq, hkv, d, page):
    pages, table, n, *_ = prefixed(g, [(0, lens)], page, hkv, d)
    q = queries(sum(counts), hq, d, 1)
    start = ints([sum(counts[:i]) for i in range(len(counts) + 1)])
    lse = g.kv4_prefill(q, pages, table, n, start, KS, VS, return_lse=True)[1]
    old = torch.rand(len(lens), hkv, max(lens), device="cuda")
    out = torch.zeros_like(old)

    def call(st):
        g.kv4_score(q, lse, pages, table, n, old, KS, q_start=start, out=out, dev_status=st)

    gives_up(short, call, [out])
