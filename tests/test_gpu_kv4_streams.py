"""The 4-bit KV cache's calls on a stream that is not the current one."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

KS, VS = 0.017, 0.013


@pytest.fixture(scope="module")
def g():
    import nvfp4_gated_deltanet_gb300 as pkg
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return pkg


@pytest.mark.parametrize("which", ["read", "decode", "prefill", "compact"])
def test_outputs_for_a_stream_are_no_memory_that_another_still_writes(g, which):
    """The current stream frees tensors of the outputs' sizes while its kernels
    have yet to write them. A call on another stream, which waits for none of
    that, must not get those blocks for its outputs."""
    hkv, hq, d, T = 2, 8, 128, 4096
    gen = torch.Generator(device="cuda").manual_seed(6)
    k, v = (torch.randn(T, hkv, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(T, hq, d, generator=gen, device="cuda").bfloat16()
    pages = g.kv4_new_pages(T // 16 + 64, 16, hkv, d)
    table = torch.randperm(T // 16 + 64, generator=gen, device="cuda")[:T // 16].int().view(1, -1)
    n = torch.tensor([T], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    g.kv4_append(k, v, pages, table, n, KS, VS, q_start=start)

    def call(stream=None):
        if which == "read":
            return g.kv4_read(pages, table, n, KS, VS, T, q_start=start, stream=stream)
        if which == "decode":
            return g.kv4_decode(q[None], pages, table, n, KS, VS, return_lse=True, stream=stream)
        if which == "prefill":
            return g.kv4_prefill(q, pages, table, n, start, KS, VS, return_lse=True, stream=stream)
        return g.kv4_compact(pages, table, stream=stream)    # again with the same tables: the same result

    want = [x.clone() for x in call()]
    big = torch.randn(4096, 4096, generator=gen, device="cuda").bfloat16()
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


def test_an_output_dropped_while_the_current_stream_reads_it(g):
    """An output of a call on another stream is read on the current one and
    dropped: the other stream's next outputs do not overwrite it meanwhile."""
    hkv, hq, d = 2, 8, 128
    gen = torch.Generator(device="cuda").manual_seed(7)
    pages = g.kv4_new_pages(64, 16, hkv, d)
    table = torch.arange(64, dtype=torch.int32, device="cuda").view(1, -1)
    n = torch.tensor([1024], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(1024, hkv, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    g.kv4_append(k, v, pages, table, n, KS, VS)
    qs = torch.randn(6, 1, 64, hq, d, generator=gen, device="cuda").bfloat16()
    want = [g.kv4_decode(q, pages, table, n, KS, VS) for q in qs]
    big = torch.randn(4096, 4096, generator=gen, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    kept = []
    for q in qs:
        out = g.kv4_decode(q, pages, table, n, KS, VS, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        for _ in range(10):
            big @ big
        kept.append(out + 0)
        del out
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(kept, want))


def test_outputs_for_a_stream_within_a_capture(g):
    """A captured fork: a call on the side stream allocates its output, the
    capturing stream reads it; replays give the eager results."""
    hkv, hq, d = 2, 8, 128
    gen = torch.Generator(device="cuda").manual_seed(8)
    pages = g.kv4_new_pages(64, 16, hkv, d)
    table = torch.arange(64, dtype=torch.int32, device="cuda").view(1, -1)
    n = torch.tensor([1024], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(1024, hkv, d, generator=gen, device="cuda").bfloat16() for _ in range(2))
    g.kv4_append(k, v, pages, table, n, KS, VS)
    q = torch.randn(64, hq, d, generator=gen, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    held = torch.zeros_like(q)

    def go():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        one = g.kv4_decode(held[None], pages, table, n, KS, VS, stream=side)
        two = g.kv4_prefill(held, pages, table, n, start, KS, VS, stream=side)
        here.wait_stream(side)
        both = one[0].float() + two.float()
        del one, two
        return both, torch.full_like(both, 3.0)

    graph = torch.cuda.CUDAGraph()
    go()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got, _ = go()
    for scale in (1.0, 0.25):
        held.copy_(q * scale)
        graph.replay()
        first = got.clone()
        assert torch.equal(first, go()[0])
        torch.cuda.synchronize()


@pytest.mark.parametrize("own", [False, True])
def test_check_sees_what_other_streams_have_yet_to_flag(g, own):
    """An append on a side stream, behind milliseconds of other work there, names a
    page that does not exist: check() (of all streams, or of that one) tells."""
    c = g.KV4Cache(8, 16, 2, 64, KS, VS)
    big = torch.randn(8192, 8192, device="cuda").bfloat16()
    k = torch.randn(3, 2, 64, device="cuda").bfloat16()
    seq = c.new()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    batch = c.grow([seq], 3, stream=side)
    with torch.cuda.stream(side):
        batch.block_table.fill_(99)
        for _ in range(50):
            big @ big
    c.append(0, k, k, batch, stream=side)
    assert c.check(side if own else None) == 6
    assert c.check() == 0
    batch = c.grow([seq], 3, stream=side)
    c.append(0, k, k, batch, stream=side)
    assert c.check(side) == 0


@pytest.mark.parametrize("graph", [False, True])
def test_order_of_prefill_copies_and_compaction(g, graph):
    """Queries, lengths, row starts, tables, page ids and pages written just
    before a call (on another stream, by copies and fills, by the calls
    themselves) and overwritten just after it: prefill, page copies and
    compaction see what came before them in their stream, and only that."""
    hkv, hq, d, T, new = 4, 16, 128, 1500, 700
    num = 2 * (T // 16 + 1)
    gen = torch.Generator(device="cuda").manual_seed(9)
    src = torch.randn(2, T, hkv, d, generator=gen, device="cuda").bfloat16()
    queries = torch.randn(new, hq, d, generator=gen, device="cuda").bfloat16()
    table = torch.randperm(num, generator=gen, device="cuda")[:T // 16 + 1].int().view(1, -1)
    full = torch.tensor([T], dtype=torch.int32, device="cuda")
    rows, all_rows = (torch.tensor([0, m], dtype=torch.int32, device="cuda") for m in (new, T))
    free = torch.tensor([p for p in range(num) if p not in set(table[0].tolist())][:20], dtype=torch.int32, device="cuda")
    some = table[0, :20].contiguous()
    big = torch.randn(4096, 4096, generator=gen, device="cuda").bfloat16()
    start = g.kv4_new_pages(num, 16, hkv, d)
    g.kv4_append(src[0], src[1], start, table, full, KS, VS, q_start=all_rows)

    q, lens, at, tab = torch.zeros_like(queries), torch.zeros_like(full), torch.zeros_like(rows), torch.zeros_like(table)
    ids, to, pages = torch.zeros_like(some), torch.zeros_like(free), torch.zeros_like(start)
    out, lse = torch.zeros_like(queries), torch.zeros(new, hq, device="cuda")
    last, last_lse = torch.zeros_like(out), torch.zeros_like(lse)
    tables, where, live = torch.zeros_like(table), torch.zeros(num, dtype=torch.int32, device="cuda"), torch.zeros_like(full)
    got = [out, lse, last, last_lse, tables, where, live]
    moved = torch.zeros_like(start)
    side = torch.cuda.Stream()

    def go(sync=lambda: None):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            for _ in range(4):
                big @ big
            q.copy_(queries)
            pages.copy_(start)
        for x, y in ((lens, full), (at, rows), (tab, table), (ids, some), (to, free)):
            x.copy_(y)
        here.wait_stream(side)
        sync()
        g.kv4_prefill(q, pages, tab, lens, at, KS, VS, total_kv=T, out=out, lse=lse)
        sync()
        q.zero_()
        at.zero_()
        g.kv4_copy_pages(pages, ids, to)
        sync()
        ids.fill_(3)
        tab[0, :20].copy_(to)                        # the copies in place of the pages they were made of
        to.fill_(5)
        g.kv4_compact(pages, tab, tables_out=tables, page_map=where, n_live=live)
        sync()
        tab.zero_()
        q.copy_(queries)
        at.copy_(rows)
        g.kv4_prefill(q, pages, tables, lens, at, KS, VS, total_kv=T, out=last, lse=last_lse)
        sync()
        moved.copy_(pages)
        for x in (q, lens, at, pages):
            x.zero_()

    go(torch.cuda.synchronize)                       # each call alone on the device
    torch.cuda.synchronize()
    want = [x.clone() for x in (*got, moved)]
    assert torch.equal(out, last) and torch.equal(lse, last_lse) and live.item() == T // 16 + 1
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
        for x in (*got, moved):
            x.zero_()
        cuda_graph.replay() if graph else go()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip((*got, moved), want))
