"""The 4-bit paged KV cache on the GPU against the float64 reference of
kv4_ref.py: the page layout and the quantiser bit for bit, attention within
bounds derived from its roundings, page moves byte for byte."""
import numpy as np
import pytest

import kv4_ref as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

KS, VS = 0.017, 0.013


@pytest.fixture(scope="module")
def g():
    import nvfp4_gated_deltanet_gb300 as pkg
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return pkg


def f64(t):
    return t.double().cpu().numpy()


def setup(g, lens, page, hkv, d, seed=0, spare=2):
    """Random cached tokens for sequences of the given lengths: pages full of
    NaN scales except where a token was appended, shuffled tables."""
    rng = np.random.RandomState(seed)
    need = [-(-n // page) for n in lens]
    num = sum(need) + spare
    ids = rng.permutation(num).astype(np.int32)
    cols = max([1] + need)
    table = np.full((len(lens), cols), -7, np.int32)  # entries that must not be read
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    pages = torch.full((num, hkv, page // 16, 18 * d), 0x7F, dtype=torch.uint8, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lens)
    k = (torch.randn(T, hkv, d, generator=gen, device="cuda") *
         torch.exp(0.5 * torch.randn(hkv, d, generator=gen, device="cuda"))).bfloat16()
    v = torch.randn(T, hkv, d, generator=gen, device="cuda").bfloat16()
    tab, n = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    start = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    g.kv4_append(k, v, pages, tab, n, KS, VS, q_start=start, dev_status=st)
    assert st.item() == 0
    return pages, tab, n, k, v, start


def queries(T, hq, d, seed, scale=1.5):
    gen = torch.Generator(device="cuda").manual_seed(1000 + seed)
    return (scale * torch.randn(T, hq, d, generator=gen, device="cuda")).bfloat16()


def want(pages, tab, lens, counts, q, d):
    """The reference's outputs and error sums of every row."""
    p, t, q = pages.cpu().numpy(), tab.cpu().numpy(), f64(q)
    parts, at = [], 0
    for b, (n, m) in enumerate(zip(counts, lens)):
        K, V = ref.cached(p, t[b], m, d, KS, VS)
        parts.append(ref.attention(q[at:at + n], K, V, float(np.float32(d ** -0.5))))
        at += n
    return [np.concatenate(x) for x in zip(*parts)]


def close(out, lse, w, d):
    eo, el = ref.bounds(w, d)
    out, lse = f64(out).reshape(w[0].shape), f64(lse).reshape(w[1].shape)
    assert np.isfinite(out).all()
    over = np.abs(out - w[0]) / eo
    assert over.max() <= 1, (over.max(), np.unravel_index(over.argmax(), over.shape))
    none = np.isinf(w[1])
    assert (lse[none] == -np.inf).all() and (out[none] == 0).all()
    over = np.abs(lse[~none] - w[1][~none]) / el[~none]
    assert none.all() or over.max() <= 1, over.max()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_append_layout_and_quantiser(g, d, page):
    """Every byte of an appended token lies where the layout says and equals
    nvfp4_quantize's; nothing else changes; reading back gives the values."""
    lens, hkv = [5, 33, 0, 16 * 9 + 1], 3
    pages, tab, n, k, v, start = setup(g, lens, page, hkv, d)
    T = sum(lens)
    got = pages.cpu().numpy()
    expect = np.full_like(got, 0x7F)
    rows = []
    for x, ts in ((k, KS), (v, VS)):
        c, s = g.nvfp4_quantize(x.reshape(T * hkv, d).contiguous(), ts)
        rows.append((c.cpu().numpy().reshape(T, hkv, -1), s.cpu().numpy().reshape(T, hkv, -1)))
    t = tab.cpu().numpy()
    at, vals = 0, [np.empty((T, hkv, d)), np.empty((T, hkv, d))]
    for b, m in enumerate(lens):
        for p in range(m):
            kc, vc, ks, vs = ref.places(p % 16, d)
            for h in range(hkv):
                cell = expect[t[b, p // page], h, p % page // 16]
                cell[kc], cell[ks] = rows[0][0][at, h], rows[0][1][at, h]
                cell[vc], cell[vs] = rows[1][0][at, h], rows[1][1][at, h]
                for i, ts in enumerate((KS, VS)):
                    vals[i][at, h] = ref.decode_row(rows[i][0][at, h], rows[i][1][at, h]) * float(np.float32(ts))
            at += 1
    assert np.array_equal(got, expect)
    rk, rv = g.kv4_read(pages, tab, n, KS, VS, T, q_start=start)
    for r, w in zip((rk, rv), vals):
        # one FP32 rounding by the tensor scale, one to BF16
        assert (np.abs(f64(r) - w) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(w)).all()
    assert np.array_equal(pages.cpu().numpy(), expect)


def test_append_strided_rows_padding_and_partial(g):
    """Rows as slices of fused projections, padding rows past q_start[B], new
    tokens after old ones, a token before the sequence's start."""
    d, hkv, page = 64, 2, 16
    pages, tab, n, k, v, start = setup(g, [20, 40], page, hkv, d)
    before = pages.clone()
    row = torch.randn(9, 5 * hkv, d, device="cuda").bfloat16()
    k2, v2 = row[:, hkv:2 * hkv], row[:, 3 * hkv:4 * hkv]
    start2 = torch.tensor([0, 3, 7], dtype=torch.int32, device="cuda")   # rows 7 and 8 are padding
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    g.kv4_append(k2, v2, pages, tab, n, KS, VS, q_start=start2, dev_status=st)
    rk, rv = g.kv4_read(pages, tab, n, KS, VS, 60, q_start=start)
    other, = (g.kv4_new_pages(7, page, hkv, d),)
    ids = torch.arange(7, dtype=torch.int32, device="cuda")[None]
    g.kv4_append(row[:7, hkv:2 * hkv].contiguous(), row[:7, 3 * hkv:4 * hkv].contiguous(), other, ids,
                 torch.tensor([7], dtype=torch.int32, device="cuda"), KS, VS)
    ok, ov = g.kv4_read(other, ids, torch.tensor([7], dtype=torch.int32, device="cuda"), KS, VS, 7)
    new = [17, 18, 19, 56, 57, 58, 59]
    assert torch.equal(rk[new], ok) and torch.equal(rv[new], ov)
    old = [i for i in range(60) if i not in new]
    bk, bv = g.kv4_read(before, tab, n, KS, VS, 60, q_start=start)
    assert torch.equal(rk[old], bk[old]) and torch.equal(rv[old], bv[old])
    # more new rows than tokens: the ones before the start are left out
    again = before.clone()
    g.kv4_append(k2[:6], v2[:6], again, tab, torch.tensor([2, 0], dtype=torch.int32, device="cuda"), KS, VS,
                 dev_status=st)
    rk, _ = g.kv4_read(again, tab, n, KS, VS, 60, q_start=start)
    assert torch.equal(rk[:2], ok[1:3]) and torch.equal(rk[2:], bk[2:])
    assert st.item() == 0


def test_append_flags_nonfinite_and_bad_tables(g):
    d, hkv, page = 128, 1, 16
    x = torch.randn(3, hkv, d, device="cuda").bfloat16()
    tab = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    three = torch.tensor([3], dtype=torch.int32, device="cuda")

    def run(k=x, tab=tab, n=three, start=None):
        pages, st = g.kv4_new_pages(2, page, hkv, d), torch.zeros(1, dtype=torch.int32, device="cuda")
        g.kv4_append(k, x, pages, tab, n, KS, VS, q_start=start, dev_status=st)
        return pages, st.item()

    bad = x.clone()
    bad[1, 0, 20], bad[2, 0, 100] = float("nan"), float("-inf")
    pages, st = run(bad)
    assert st == 4
    rk, _ = g.kv4_read(pages, tab, three, KS, VS, 3)
    gk, _ = g.kv4_read(run()[0], tab, three, KS, VS, 3)
    hit = torch.zeros(3, 1, d, dtype=torch.bool, device="cuda")
    hit[1, 0, 16:32], hit[2, 0, 96:112] = True, True
    assert (rk[hit] == 0).all() and torch.equal(rk[~hit], gk[~hit])
    for i in (-1, 2, 2 ** 31 - 1):
        pages, st = run(tab=torch.tensor([[i]], dtype=torch.int32, device="cuda"))
        assert st == 6 and not pages.any()
    for n in (-3, 17):
        pages, st = run(n=torch.tensor([n], dtype=torch.int32, device="cuda"))
        assert st == 6 and not pages.any()
    for s in ([0, 4], [2, 1], [-1, 3]):
        pages, st = run(start=torch.tensor(s, dtype=torch.int32, device="cuda"))
        assert st == 6 or not pages.any()


DECODE = [  # lens, r, hq, hkv, d, page
    ([1], 1, 1, 1, 64, 16), ([1], 1, 8, 1, 128, 16), ([2, 0, 17], 1, 4, 2, 128, 16), ([16, 15, 64, 65], 1, 6, 2, 64, 32),
    ([300], 1, 16, 2, 128, 64), ([700, 3, 129], 1, 8, 8, 64, 128), ([257, 64, 63], 1, 24, 2, 128, 256),
    ([3, 1, 0, 90], 4, 8, 2, 128, 16), ([100, 7], 8, 16, 1, 64, 64), ([129], 3, 5, 1, 128, 32), ([40, 200], 2, 64, 1, 64, 16),
    ([1500], 1, 2, 1, 128, 16)]


@pytest.mark.parametrize("lens,r,hq,hkv,d,page", DECODE)
def test_decode(g, lens, r, hq, hkv, d, page):
    pages, tab, n, *_ = setup(g, lens, page, hkv, d, seed=len(lens) + r)
    q = queries(len(lens) * r, hq, d, r).reshape(len(lens), r, hq, d)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = g.kv4_decode(q, pages, tab, n, KS, VS, return_lse=True, dev_status=st)
    assert st.item() == 0
    close(out, lse, want(pages, tab, lens, [r] * len(lens), q.flatten(0, 1), d), d)
    again = g.kv4_decode(q, pages, tab, n, KS, VS, return_lse=True)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


PREFILL = [  # (new, cached with them) per sequence, hq, hkv, d, page
    ([(1, 1)], 1, 1, 64, 16), ([(5, 5), (0, 9), (1, 30)], 4, 2, 128, 16), ([(130, 130)], 4, 1, 128, 32),
    ([(33, 200), (70, 70), (2, 129)], 8, 2, 64, 64), ([(9, 4), (3, 0), (20, 20)], 6, 2, 128, 16),
    ([(150, 290)], 12, 4, 64, 128), ([(40, 300)], 16, 1, 128, 256), ([(257, 257)], 2, 2, 128, 64),
    ([(17, 17)], 64, 1, 64, 16), ([(65, 128), (64, 64)], 5, 1, 128, 16)]


@pytest.mark.parametrize("seqs,hq,hkv,d,page", PREFILL)
def test_prefill(g, seqs, hq, hkv, d, page):
    counts, lens = [s[0] for s in seqs], [s[1] for s in seqs]
    pages, tab, n, *_ = setup(g, lens, page, hkv, d, seed=sum(counts))
    T = sum(counts)
    q = queries(T, hq, d, T)
    start = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = g.kv4_prefill(q, pages, tab, n, start, KS, VS, total_kv=sum(lens), return_lse=True, dev_status=st)
    assert st.item() == 0
    close(out, lse, want(pages, tab, lens, counts, q, d), d)
    again = g.kv4_prefill(q, pages, tab, n, start, KS, VS, return_lse=True)  # total_kv from the tables
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("d", [64, 128])
def test_extreme_scores(g, d):
    """Scores far apart (one key takes all, later keys larger than earlier ones
    and the other way round), equal ones, and large and tiny queries."""
    lens, hkv, hq = [400, 400, 400, 400, 400], 1, 2
    pages, tab, n, *_ = setup(g, lens, 16, hkv, d, seed=5)
    unit = torch.zeros(5, 400, hkv, d, device="cuda")
    unit[0, :, :, 0] = torch.linspace(0, 8, 400, device="cuda")[:, None]      # rising
    unit[1, :, :, 0] = torch.linspace(8, 0, 400, device="cuda")[:, None]      # falling
    unit[2, :, :, 0] = 1.0                                                    # equal
    unit[3, 200, :, 0] = 8.0                                                  # one
    unit[4] = torch.randn(400, hkv, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    k = unit.reshape(2000, hkv, d).bfloat16()
    v = torch.randn(2000, hkv, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4)).bfloat16()
    start = torch.arange(6, dtype=torch.int32, device="cuda") * 400
    g.kv4_append(k, v, pages, tab, n, KS, VS, q_start=start)
    for scale in (1.0, 60.0, 2.0 ** 20, 2.0 ** -40):
        q = torch.zeros(5, hq, d, device="cuda")
        q[:, 0, 0], q[:, 1, 0] = scale, -scale
        q[:, :, 1] = 0.37 * scale
        q = q.bfloat16()
        w = want(pages, tab, lens, [1] * 5, q, d)
        close(*g.kv4_decode(q, pages, tab, n, KS, VS, return_lse=True), w, d)
        one = torch.arange(6, dtype=torch.int32, device="cuda")
        close(*g.kv4_prefill(q, pages, tab, n, one, KS, VS, return_lse=True), w, d)


def test_nonfinite_queries_stay_in_their_rows(g):
    d, hq = 128, 8
    pages, tab, n, *_ = setup(g, [70, 90], 32, 2, d)
    q = queries(2, hq, d, 0)
    good = g.kv4_decode(q, pages, tab, n, KS, VS)
    q2 = q.clone()
    q2[0, 3, 5], q2[1, 6, 0] = float("nan"), float("inf")
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    goodp = g.kv4_prefill(q, pages, tab, n, start, KS, VS)
    for base, out in ((good, g.kv4_decode(q2, pages, tab, n, KS, VS)),
                      (goodp, g.kv4_prefill(q2, pages, tab, n, start, KS, VS))):
        hit = torch.zeros(2, hq, dtype=torch.bool, device="cuda")
        hit[0, 3] = hit[1, 6] = True
        assert out[hit].isnan().all() and torch.equal(out[~hit], base[~hit])


def test_strides_streams_outputs_and_graph(g):
    """q as a slice of fused rows, given outputs, a side stream, and a captured
    append + decode replayed on new tokens and lengths."""
    d, hq, hkv, page = 128, 8, 2, 16
    pages, tab, n, *_ = setup(g, [50, 59], page, hkv, d)
    rows = torch.randn(2, hq + 2 * hkv, d, device="cuda").bfloat16()
    q = rows[:, :hq]
    base = g.kv4_decode(q.contiguous(), pages, tab, n, KS, VS)
    out = torch.empty(2, hq, d, dtype=torch.bfloat16, device="cuda")
    assert g.kv4_decode(q, pages, tab, n, KS, VS, out=out) is out and torch.equal(out, base)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = g.kv4_decode(q, pages, tab, n, KS, VS, stream=side)
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    pre = g.kv4_prefill(q, pages, tab, n, start, KS, VS, stream=side)
    side.synchronize()
    assert torch.equal(other, base)
    assert (pre.float() - base.float()).abs().max() <= 2.0 ** -6 * base.float().abs().max()
    # captured: the lengths, tables and rows are read when the graph runs
    def step():
        g.kv4_append(rows[:, hq:hq + hkv], rows[:, hq + hkv:], pages, tab, n, KS, VS)
        return g.kv4_decode(q, pages, tab, n, KS, VS, out=out)
    saved = pages.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    pages.copy_(saved)
    for add in (1, 1, 1):
        rows.copy_(torch.randn_like(rows.float()).bfloat16())
        n += add
        graph.replay()
        got = out.clone()
        kept = pages.clone()
        assert torch.equal(step(), got) and torch.equal(pages, kept)


def test_bad_ids_are_flagged_and_confined(g):
    d, hq, hkv, page = 64, 4, 2, 16
    pages, tab, n, *_ = setup(g, [40, 40], page, hkv, d)
    q = queries(2, hq, d, 1)
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    dec = g.kv4_decode(q, pages, tab, n, KS, VS)
    pre = g.kv4_prefill(q, pages, tab, n, start, KS, VS)
    for change in ("table", "negative", "len", "neglen"):
        t, m = tab.clone(), n.clone()
        if change in ("table", "negative"):
            t[0, 1] = 10 ** 6 if change == "table" else -1
        else:
            m[0] = 49 if change == "len" else -2
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        assert torch.equal(g.kv4_decode(q, pages, t, m, KS, VS, dev_status=st)[1], dec[1]) and st.item() == 6
        st.zero_()
        out = g.kv4_prefill(q, pages, t, m, start, KS, VS, dev_status=st)
        assert torch.equal(out[1], pre[1]) and st.item() == 6
    st.zero_()
    g.kv4_prefill(q, pages, tab, n, start, KS, VS, total_kv=80, dev_status=st)
    assert st.item() == 0


@pytest.mark.parametrize("layers,page_bytes", [(1, (2, 1, 18 * 64)), (3, (3, 4, 18 * 128))])
def test_copy_pages(g, layers, page_bytes):
    num = 23
    gen = torch.Generator(device="cuda").manual_seed(1)
    pages = torch.randint(0, 256, (layers, num, *page_bytes), generator=gen, dtype=torch.uint8, device="cuda")
    ids = torch.randperm(num, generator=gen, device="cuda").to(torch.int32)
    src, dst = ids[:9].clone(), ids[9:18].clone()
    src[3] = src[2]                               # one page to two places
    w = pages.clone()
    w[:, dst.long()] = pages[:, src.long()]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    g.kv4_copy_pages(pages if layers > 1 else pages[0], src, dst, dev_status=st)
    assert torch.equal(pages, w) and st.item() == 0
    src[0], dst[1] = num, -1
    g.kv4_copy_pages(pages, src, dst, dev_status=st)
    assert torch.equal(pages, w) and st.item() == 6
    g.kv4_copy_pages(pages, src[:0], dst[:0])


@pytest.mark.parametrize("num,rows,cols,fill,seed", [(1, 1, 1, 1.0, 0), (7, 3, 4, 0.6, 1), (64, 2, 40, 1.0, 2), (33, 4, 9, 0.0, 3),
                                                     (1000, 20, 50, 0.4, 4), (70001, 64, 600, 0.5, 5)])
def test_compact(g, num, rows, cols, fill, seed):
    rng = np.random.RandomState(seed)
    n_live = int(round(num * fill))
    ids = rng.permutation(num)[:n_live]
    table = np.full(rows * cols, -1, np.int32)
    some = rng.permutation(rows * cols)[:n_live]
    table[some] = ids[:len(some)]
    if n_live:
        spare = np.setdiff1d(np.arange(rows * cols), some)[:5]
        table[spare] = ids[0]                     # a page with several holders
    table = table.reshape(rows, cols)
    live = np.unique(table[table >= 0])
    L = len(live)
    to = np.full(num, -1, np.int32)
    low = live[live < L]
    to[low] = low
    to[live[live >= L]] = np.setdiff1d(np.arange(L), low)
    pages = torch.randint(0, 256, (2, num, 1, 1, 144), dtype=torch.uint8, device="cuda")
    w = pages.clone()
    moved = np.flatnonzero(to >= 0)
    w[:, torch.from_numpy(to[moved]).long().cuda()] = pages[:, torch.from_numpy(moved).cuda()]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tab = torch.from_numpy(table).cuda()
    for _ in range(2):                            # the same tables again give the same result
        t2, m, k = g.kv4_compact(pages, tab, dev_status=st)
        assert k.item() == L and np.array_equal(m.cpu().numpy(), to)
        assert np.array_equal(t2.cpu().numpy(), np.where(table >= 0, to[table], -1))
        assert torch.equal(pages, w)
    assert st.item() == 0
    tab[0, 0] = num
    t2, _, _ = g.kv4_compact(pages.clone(), tab, dev_status=st)
    assert st.item() == 6 and t2[0, 0].item() == -1


def test_cache_in_use(g):
    """A cache of two layers: a prompt, a fork, both continued, one freed, the
    rest compacted: every step's attention equals a fresh cache's of the same tokens."""
    hq, hkv, d, page = 4, 2, 64, 16
    c = g.KV4Cache(30, page, hkv, d, KS, VS, n_layers=2)
    toks = {}
    gen = torch.Generator(device="cuda").manual_seed(9)

    def rand(n, h):
        return torch.randn(n, h, d, generator=gen, device="cuda").bfloat16()

    def step(seqs, counts, decode):
        batch = c.grow(seqs, counts)
        for layer in range(2):
            k, v = rand(sum(counts), hkv), rand(sum(counts), hkv)
            q = rand(sum(counts), hq)
            at = 0
            for s, n in zip(seqs, counts):
                old = toks[s][layer]
                toks[s][layer] = (torch.cat([old[0], k[at:at + n]]), torch.cat([old[1], v[at:at + n]]))
                at += n
            c.append(layer, k, v, batch)
            if decode:
                out = c.decode(layer, q.reshape(len(seqs), -1, hq, d), batch).flatten(0, 1)
            else:
                out = c.prefill(layer, q, batch)
            at = 0
            for s, n in zip(seqs, counts):
                fk, fv = toks[s][layer]
                m = fk.shape[0]
                cols = -(-m // page)
                fresh = g.kv4_new_pages(cols, page, hkv, d)
                tab = torch.arange(cols, dtype=torch.int32, device="cuda")[None]
                ln = torch.tensor([m], dtype=torch.int32, device="cuda")
                g.kv4_append(fk, fv, fresh, tab, ln, KS, VS)
                w = want(fresh, tab, [m], [n], q[at:at + n], d)
                eo, _ = ref.bounds(w, d)
                assert (np.abs(f64(out[at:at + n]) - w[0]) <= eo).all()
                at += n

    a, b = c.new(), c.new()
    for s in (a, b):
        toks[s] = [(torch.empty(0, hkv, d, device="cuda", dtype=torch.bfloat16),) * 2 for _ in range(2)]
    step([a, b], [37, 20], False)
    f = c.fork(a)
    toks[f] = list(toks[a])
    step([a, f, b], [1, 1, 1], True)
    step([f, a], [3, 3], True)
    c.free(a)
    del toks[a]
    n = c.compact()
    assert n == len(set(c.book.pages(b) + c.book.pages(f))) and max(c.book.pages(b) + c.book.pages(f)) == n - 1
    step([b, f], [2, 2], True)
    step([f], [25], False)
    assert c.check() == 0


def want_fast(pages, tab, lens, counts, q, d):
    parts, at = [], 0
    for b, (n, m) in enumerate(zip(counts, lens)):
        need = -(-m // (16 * pages.shape[2]))
        K, V = ref.cached_torch(pages, tab[b, :need], m, d, KS, VS)
        parts.append(ref.attention_torch(q[at:at + n].double(), K, V, float(np.float32(d ** -0.5))))
        at += n
    return [np.concatenate(x) for x in zip(*parts)]


# sequences, tokens at most, r, hq, hkv, d, page: runs that cut items, in both team sizes and all column blocks
SPLIT = [(40, 1500, 1, 8, 8, 128, 64), (160, 700, 1, 4, 1, 128, 16), (30, 1200, 2, 48, 8, 128, 32), (6, 3000, 5, 16, 2, 128, 64),
         (50, 900, 1, 16, 4, 64, 16), (45, 800, 3, 32, 8, 64, 64), (40, 600, 8, 24, 4, 64, 128), (3, 9000, 1, 4, 2, 64, 256),
         (2, 20000, 1, 16, 1, 128, 128), (1, 30000, 8, 64, 1, 128, 64), (1, 12000, 2, 64, 2, 64, 32), (200, 130, 1, 8, 2, 128, 16)]


@pytest.mark.parametrize("B,most,r,hq,hkv,d,page", SPLIT)
def test_decode_split_over_runs(g, B, most, r, hq, hkv, d, page):
    rng = np.random.RandomState(B + r)
    lens = [most] + [int(x) for x in np.exp(rng.uniform(0, np.log(most), B - 1))]
    if B > 4:
        lens[2] = 0
    pages, tab, n, *_ = setup(g, lens, page, hkv, d, seed=B)
    q = queries(B * r, hq, d, B).reshape(B, r, hq, d)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = g.kv4_decode(q, pages, tab, n, KS, VS, return_lse=True, dev_status=st)
    close(out, lse, want_fast(pages, tab, lens, [r] * B, q.flatten(0, 1), d), d)
    again = g.kv4_decode(q, pages, tab, n, KS, VS, return_lse=True, dev_status=st)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1]) and st.item() == 0


# (new, cached) of the longest, sequences, hq, hkv, d, page: more items than CTAs, rows of several sequences, long caches
MANY = [(1200, 1200, 4, 32, 8, 128, 64), (300, 5000, 3, 16, 4, 64, 32), (64, 900, 40, 8, 8, 128, 16), (700, 701, 7, 12, 2, 64, 128),
        (1, 3000, 50, 40, 8, 128, 64), (500, 2500, 2, 56, 8, 128, 256)]


@pytest.mark.parametrize("new,total,B,hq,hkv,d,page", MANY)
def test_prefill_many_items(g, new, total, B, hq, hkv, d, page):
    rng = np.random.RandomState(new)
    counts = [new] + [int(x) for x in rng.randint(0, new + 1, B - 1)]
    lens = [total] + [c + int(rng.randint(0, total - new + 1)) for c in counts[1:]]
    pages, tab, n, *_ = setup(g, lens, page, hkv, d, seed=B)
    T = sum(counts)
    q = queries(T + 3, hq, d, T)                     # three padding rows, left alone
    start = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((T + 3, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 3, hq), 7.0, device="cuda")
    g.kv4_prefill(q, pages, tab, n, start, KS, VS, total_kv=sum(lens), out=out, lse=lse, dev_status=st)
    close(out[:T], lse[:T], want_fast(pages, tab, lens, counts, q, d), d)
    assert (out[T:] == 7).all() and (lse[T:] == 7).all()
    again = g.kv4_prefill(q[:T].contiguous(), pages, tab, n, start, KS, VS, return_lse=True, dev_status=st)
    assert torch.equal(out[:T], again[0]) and torch.equal(lse[:T], again[1]) and st.item() == 0


def test_a_rows_result_depends_on_no_other_row(g):
    """The same queries beside others give the same bits (the maxima and the rescaling are decided row by row)."""
    d, hq, hkv, page = 128, 8, 2, 16
    lens = [600, 600]
    pages, tab, n, *_ = setup(g, lens, page, hkv, d)
    start = torch.tensor([0, 70, 140], dtype=torch.int32, device="cuda")
    q = queries(140, hq, d, 1)
    other = q.clone()
    other[:, ::2] *= 40
    a, b = (g.kv4_prefill(x, pages, tab, n, start, KS, VS) for x in (q, other))
    assert torch.equal(a[:, 1::2], b[:, 1::2]) and not torch.equal(a, b)
    a, b = (g.kv4_decode(x[[69, 139]], pages, tab, n, KS, VS) for x in (q, other))
    assert torch.equal(a[:, 1::2], b[:, 1::2]) and not torch.equal(a, b)


def test_offsets_past_32_bits(g):
    """A cache of 4.7 GB: its last pages lie past 2^32 bytes."""
    d, hkv, hq, page, num = 128, 8, 16, 256, 16000
    pages = g.kv4_new_pages(num, page, hkv, d)
    assert pages.numel() > 2 ** 32
    T = 300
    gen = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(T, hkv, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    tab = torch.tensor([[num - 1, num - 3]], dtype=torch.int32, device="cuda")
    n = torch.tensor([T], dtype=torch.int32, device="cuda")
    g.kv4_append(k, v, pages, tab, n, KS, VS)
    small = g.kv4_new_pages(2, page, hkv, d)
    stab = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    g.kv4_append(k, v, small, stab, n, KS, VS)
    assert torch.equal(pages[[num - 1, num - 3]], small)
    for x, y in zip(g.kv4_read(pages, tab, n, KS, VS, T), g.kv4_read(small, stab, n, KS, VS, T)):
        assert torch.equal(x, y)
    q = queries(5, hq, d, 3)
    start = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    assert torch.equal(g.kv4_decode(q[None], pages, tab, n, KS, VS), g.kv4_decode(q[None], small, stab, n, KS, VS))
    assert torch.equal(g.kv4_prefill(q, pages, tab, n, start, KS, VS), g.kv4_prefill(q, small, stab, n, start, KS, VS))
    g.kv4_copy_pages(pages, torch.tensor([num - 1], dtype=torch.int32, device="cuda"),
                     torch.tensor([num - 2], dtype=torch.int32, device="cuda"))
    assert torch.equal(pages[num - 2], small[0])
    t2, m, live = g.kv4_compact(pages, tab)
    # in ascending order: num - 3 to page 0, num - 1 to page 1
    assert t2.tolist() == [[1, 0]] and live.item() == 2 and torch.equal(pages[[1, 0]], small)


def test_prefill_workspace_too_small_is_flagged(g):
    """total_kv below the real sum: GDN_E_RANGE, nothing out of bounds, the sequences that fit are right."""
    d, hq, hkv, page = 64, 4, 2, 16
    pages, tab, n, *_ = setup(g, [200, 900], page, hkv, d)
    q = queries(2, hq, d, 1)
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    good = g.kv4_prefill(q, pages, tab, n, start, KS, VS)
    out = g.kv4_prefill(q, pages, tab, n, start, KS, VS, total_kv=200, dev_status=st)
    assert st.item() == 6 and torch.equal(out[0], good[0])


def test_python_refusals_on_the_gpu(g):
    d, hq, hkv, page = 64, 4, 2, 16
    pages, tab, n, k, v, start = setup(g, [20, 20], page, hkv, d)
    q = queries(2, hq, d, 0)
    one = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    bad = [(ValueError, lambda: g.kv4_decode(q.float(), pages, tab, n, KS, VS)),
           (ValueError, lambda: g.kv4_decode(q[..., ::2], pages, tab, n, KS, VS)),
           (ValueError, lambda: g.kv4_decode(q.transpose(0, 1), pages, tab, n, KS, VS)),
           (ValueError, lambda: g.kv4_decode(q[:1], pages, tab, n, KS, VS)),
           (ValueError, lambda: g.kv4_decode(q, pages, tab.long(), n, KS, VS)),
           (ValueError, lambda: g.kv4_decode(q, pages, tab, n[:1], KS, VS)),
           (ValueError, lambda: g.kv4_decode(q, pages.transpose(0, 1), tab, n, KS, VS)),
           (ValueError, lambda: g.kv4_decode(q, pages, tab, n, KS, VS, out=torch.empty(2, hq, d, device="cuda"))),
           (ValueError, lambda: g.kv4_decode(q, pages, tab, n, KS, VS, lse=torch.empty(2, hq + 1, device="cuda"))),
           (g.GdnError, lambda: g.kv4_decode(q[:, :3], pages, tab, n, KS, VS)),
           (g.GdnError, lambda: g.kv4_decode(q, pages, tab, n, 0.0, VS)),
           (g.GdnError, lambda: g.kv4_decode(q, pages, tab, n, KS, VS, sm_scale=-1.0)),
           (ValueError, lambda: g.kv4_prefill(q, pages, tab, n, one[:2], KS, VS)),
           (g.GdnError, lambda: g.kv4_prefill(q, pages, tab, n, one, KS, VS, total_kv=-1)),
           (g.GdnError, lambda: g.kv4_prefill(q, pages, tab, n, one, KS, VS, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))),
           (ValueError, lambda: g.kv4_append(k, v[1:], pages, tab, n, KS, VS, q_start=start)),
           (ValueError, lambda: g.kv4_append(k.float(), v, pages, tab, n, KS, VS, q_start=start)),
           (ValueError, lambda: g.kv4_copy_pages(pages, one, one[:2])),
           (ValueError, lambda: g.kv4_copy_pages(pages[:, :1], one, one)),
           (ValueError, lambda: g.kv4_compact(pages, tab, page_map=one)),
           (TypeError, lambda: g.kv4_decode(q, pages, tab, n, "x", VS))]
    for kind, f in bad:
        with pytest.raises(kind):
            f()
    odd = torch.zeros(2 * hq * d + 8, dtype=torch.bfloat16, device="cuda")[1:1 + 2 * hq * d].reshape(2, hq, d)
    with pytest.raises(g.GdnError, match="GDN_E_ALIGN"):
        g.kv4_decode(odd, pages, tab, n, KS, VS)
    with pytest.raises(g.GdnError, match="GDN_E_SHAPE"):    # rows 4 elements off a multiple of 8 apart
        g.kv4_decode(torch.zeros(2, hq * d + 4, dtype=torch.bfloat16, device="cuda")[:, :hq * d].view(2, hq, d), pages, tab, n, KS, VS)


def test_a_side_stream_throughout(g):
    """A cache used on a side stream only, its outputs dropped and reallocated
    on the current one meanwhile: the results are those of the current stream."""
    hq, hkv, d = 8, 2, 128
    gen = torch.Generator(device="cuda").manual_seed(4)
    rows = [torch.randn(300, hq + 2 * hkv, d, generator=gen, device="cuda").bfloat16() for _ in range(3)]
    want = []
    side = torch.cuda.Stream()
    for stream in (None, side):
        c = g.KV4Cache(64, 16, hkv, d, KS, VS)
        a, b = c.new(), c.new()
        torch.cuda.synchronize()
        outs = []
        for k, x in enumerate(rows):
            if k == 1:
                f = c.fork(a)
            seqs = [a, b] if k == 0 else [a, f, b]
            counts = [200, 100] if k == 0 else [100, 100, 100]
            batch = c.grow(seqs, counts, stream=stream)
            c.append(0, x[:, hq:hq + hkv], x[:, hq + hkv:], batch, stream=stream)
            out = c.prefill(0, x[:, :hq], batch, stream=stream)
            if stream is not None:
                side.synchronize()
            outs.append(out.clone())
            for _ in range(4):
                c.prefill(0, x[:, :hq], batch, stream=stream)            # dropped at once
                torch.full((300, hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
            if k == 1:
                c.free(b)
                b = c.new()
                c.compact(stream=stream)
        torch.cuda.synchronize()
        assert c.check() == 0
        if stream is None:
            want = outs
        else:
            assert all(torch.equal(x, y) for x, y in zip(outs, want))


@pytest.mark.parametrize("graph", [False, True])
def test_order_among_streams_and_other_kernels(g, graph):
    """Inputs written on another stream (an event between) and by copies, fills
    and kernels of other libraries just before a call, and overwritten just after
    it: every call sees what came before it in its stream."""
    hkv, d, T = 4, 128, 512
    gen = torch.Generator(device="cuda").manual_seed(8)
    src = torch.randn(2, T, hkv, d, generator=gen, device="cuda").bfloat16()
    q = torch.randn(1, 1, 8, d, generator=gen, device="cuda").bfloat16()
    table = torch.randperm(T // 16, generator=gen, device="cuda").int().view(1, -1)
    full = torch.tensor([T], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    big = torch.randn(4096, 4096, generator=gen, device="cuda").bfloat16()

    def fresh():
        return g.kv4_new_pages(T // 16, 16, hkv, d)

    want_pages = fresh()
    g.kv4_append(src[0], src[1], want_pages, table, full, KS, VS, q_start=start)
    want = [*g.kv4_read(want_pages, table, full, KS, VS, T, q_start=start), g.kv4_decode(q, want_pages, table, full, KS, VS)]
    pages, rows, lens, tab = fresh(), torch.zeros_like(src), torch.zeros_like(full), torch.zeros_like(table)
    spare = fresh()
    got = [torch.zeros_like(x) for x in want]
    side = torch.cuda.Stream()

    def go():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            for _ in range(4):
                big @ big
            rows.copy_(src)
        lens.copy_(full)
        tab.copy_(table)
        g.kv4_append(src[1], src[0], spare, tab, lens, KS, VS, q_start=start)
        here.wait_stream(side)
        g.kv4_append(rows[0], rows[1], pages, tab, lens, KS, VS, q_start=start)
        rows.zero_()
        g.kv4_read(pages, tab, lens, KS, VS, T, q_start=start, k=got[0], v=got[1])
        g.kv4_decode(q, pages, tab, lens, KS, VS, out=got[2])
        lens.zero_()
        tab.zero_()
        pages.zero_()

    if graph:
        run = torch.cuda.Stream()
        run.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(run):
            go()
        torch.cuda.current_stream().wait_stream(run)
        cuda_graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cuda_graph):
            go()
    for _ in range(10):
        for x in got:
            x.zero_()
        cuda_graph.replay() if graph else go()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


# one long sequence among short ones: an item of many runs' pieces beside whole ones, more items than the join has
# CTAs, one item over all runs, 8-, 16- and 32-row items in both team sizes
SKEW = [(160, 12000, 5, 1, 8, 8, 64, 16), (20, 30000, 40, 1, 32, 8, 128, 64), (3, 40000, 7, 4, 16, 2, 64, 32),
        (1, 60000, 0, 1, 8, 1, 128, 128), (40, 20000, 3, 4, 32, 4, 64, 16), (2, 20000, 1000, 7, 24, 2, 128, 16)]


@pytest.mark.parametrize("B,long,short,r,hq,hkv,d,page", SKEW)
def test_decode_one_long_among_short(g, B, long, short, r, hq, hkv, d, page):
    lens = [short + b % 3 for b in range(B)]
    lens[B // 3] = long
    pages, tab, n, *_ = setup(g, lens, page, hkv, d, seed=B)
    q = queries(B * r, hq, d, B + 1).reshape(B, r, hq, d)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = g.kv4_decode(q, pages, tab, n, KS, VS, return_lse=True, dev_status=st)
    close(out, lse, want_fast(pages, tab, lens, [r] * B, q.flatten(0, 1), d), d)
    again = g.kv4_decode(q, pages, tab, n, KS, VS, return_lse=True, dev_status=st)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1]) and st.item() == 0
