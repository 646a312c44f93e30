"""What the 4-bit KV cache's Python calls refuse before they touch a device
(no GPU: tensors without data that name a CUDA device stand in for real ones)."""
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def g():
    from nvfp4_gated_deltanet_gb300 import build
    build.build()
    import nvfp4_gated_deltanet_gb300 as pkg
    return pkg


def on(device, *shape, dtype=torch.int32):
    """A tensor of `device` without data: reading its address raises RuntimeError, no call gets past that."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        return torch.empty(*shape, dtype=dtype, device=device)


def calls(g):
    """Every call: its function, and its tensors by argument name."""
    bf, fl, u8 = torch.bfloat16, torch.float32, torch.uint8
    pages, table, lens = ((4, 2, 1, 18 * 128), u8), ((2, 2), torch.int32), ((2,), torch.int32)
    starts, status = ((3,), torch.int32), ((1,), torch.int32)
    kv, q, lse = ((2, 2, 128), bf), ((2, 4, 128), bf), ((2, 4), fl)
    common = dict(pages=pages, block_table=table, kv_len=lens, dev_status=status)
    scales = dict(k_scale=1.0, v_scale=1.0)
    return [
        (g.kv4_append, dict(common, k=kv, v=kv, q_start=starts), scales),
        (g.kv4_read, dict(common, q_start=starts, k=kv, v=kv), dict(scales, rows=2)),
        (g.kv4_decode, dict(common, q=q, out=q, lse=lse, workspace=((4096,), u8)), scales),
        (g.kv4_prefill, dict(common, q=q, q_start=starts, out=q, lse=lse, workspace=((4096,), u8)), scales),
        (g.kv4_copy_pages, dict(pages=pages, src=lens, dst=lens, dev_status=status), {}),
        (g.kv4_compact, dict(pages=pages, block_table=table, tables_out=table, page_map=((4,), torch.int32),
                             n_live=((1,), torch.int32), workspace=((4096,), u8), dev_status=status), {})]


@pytest.mark.parametrize("i", range(6))
def test_tensors_of_several_devices_are_refused(g, i):
    if torch.cuda.device_count() == 1:
        pytest.skip("where there is one GPU, not even a stand-in can name a second")
    f, tensors, rest = calls(g)[i]
    for odd in tensors:
        args = {k: on("cuda:1" if k == odd else "cuda:0", *shape, dtype=dt) for k, (shape, dt) in tensors.items()}
        with pytest.raises(ValueError, match="cuda:1"):
            f(**args, **rest)
    args = {k: on("cuda:1", *shape, dtype=dt) for k, (shape, dt) in tensors.items()}
    with pytest.raises(ValueError, match="stream"):
        f(**args, **rest, stream=SimpleNamespace(cuda_stream=0, device_index=0))
    for odd in tensors:                              # a host tensor among them
        args = {k: torch.zeros(*shape, dtype=dt) if k == odd else on("cuda:0", *shape, dtype=dt)
                for k, (shape, dt) in tensors.items()}
        with pytest.raises(ValueError, match="cpu|CUDA"):
            f(**args, **rest)


def test_check_waits_for_the_device_before_it_reads(g, monkeypatch):
    """A status that a call on some stream has yet to set is not missed."""
    c = g.KV4Cache(4, 16, 2, 64, 1.0, 1.0, device="cpu")
    late, waits = [6], []

    def wait(device=None):
        waits.append(device)
        if late:
            c.status.fill_(late.pop())

    monkeypatch.setattr(torch.cuda, "synchronize", wait)
    assert c.check() == 6 and waits[0] == c.device
    assert c.check() == 0 and c.status.item() == 0


def test_decode_refuses_other_rows_than_the_batch_has(g, monkeypatch):
    """Candidates of another number than the batch was grown by would be masked at the wrong tokens."""
    c = g.KV4Cache(16, 16, 2, 64, 1.0, 1.0, device="cpu")
    monkeypatch.setattr(c, "_dev", lambda rows: torch.tensor(rows, dtype=torch.int32))
    a, b = c.new(), c.new()

    def q(*shape):
        return torch.zeros(*shape, 4, 64, dtype=torch.bfloat16)

    def grow(tokens):
        c.book.extend([a, b], tokens)
        return c.batch([a, b], tokens)

    for batch, fit, bad in ((grow([3, 3]), [q(2, 3)], [q(2), q(2, 1), q(2, 4), q(1, 6), q(3, 2)]),
                            (grow([1, 1]), [q(2), q(2, 1)], [q(2, 2), q(1), q(1, 2)]),
                            (grow([3, 1]), [], [q(2), q(2, 2), q(4), q(1, 4)]),
                            (g.KV4Batch(torch.zeros(2, 1), torch.zeros(2), torch.zeros(3), 4, 4), [q(2, 2)], [q(2), q(4)])):
        for x in bad:
            with pytest.raises(ValueError, match="rows"):
                c.decode(0, x, batch)
        for x in fit:                                # goes on to the checks of the call itself
            with pytest.raises(ValueError, match="CUDA"):
                c.decode(0, x, batch)


def test_a_return_lse_without_a_truth_value_raises_its_error(g):
    """Not a result with an error set, which Python reports as a SystemError of the next call."""
    pages, table, n = torch.zeros(4, 2, 1, 18 * 64, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2).int()
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    for both in (torch.ones(2), torch.zeros(3)):
        with pytest.raises(RuntimeError, match="Boolean value"):
            g.kv4_decode(q, pages, table, n, 1.0, 1.0, return_lse=both)
        with pytest.raises(RuntimeError, match="Boolean value"):
            g.kv4_prefill(q, pages, table, n, None, 1.0, 1.0, return_lse=both)


@pytest.mark.parametrize("page", [0, 8, 17, 24, 40, 100, 250, -16])
def test_pages_that_are_no_whole_groups_are_refused(g, page):
    """24 tokens a page would be 16 on the device, and the book's pages others than the kernels'."""
    with pytest.raises(ValueError, match="page_tokens"):
        g.kv4_new_pages(4, page, 2, 64, device="cpu")
    with pytest.raises(ValueError, match="page_tokens"):
        g.KV4Cache(4, page, 2, 64, 1.0, 1.0, device="cpu")


def state(book):
    return book.holders[:], book._free[:], {k: (v[0][:], v[1]) for k, v in book.seqs.items()}


def test_growth_that_fails_on_the_device_leaves_the_book(g, monkeypatch):
    """No memory for the tables: the sequences are not longer, and shared pages not given up for copies nobody made."""
    c = g.KV4Cache(16, 16, 2, 64, 1.0, 1.0, device="cpu")
    a, b = c.new(), c.new()
    c.book.extend([a, b], [40, 16])
    f = c.fork(a)
    before = state(c.book)

    def full(rows):
        raise torch.cuda.OutOfMemoryError("no memory")

    monkeypatch.setattr(c, "_dev", full)
    for seqs, tokens in (([a, f, b], [1, 20, 1]), ([b], 30), ([f], [0]), ([a, b], 3)):
        with pytest.raises(torch.cuda.OutOfMemoryError):
            c.grow(seqs, tokens)
        assert state(c.book) == before


@pytest.mark.parametrize("seed", range(4))
def test_retract_takes_an_extend_back(g, seed):
    import random
    rng = random.Random(seed)
    b = g.KV4Book(60, 16)
    for _ in range(400):
        ids = list(b.seqs)
        op = rng.choice(["new", "extend", "extend", "extend", "fork", "free", "truncate", "compact"])
        if op == "new" or not ids:
            b.new()
        elif op == "extend":
            some = rng.sample(ids, rng.randint(1, min(5, len(ids))))
            tokens = [rng.randint(0, 40) for _ in some]
            before = state(b)
            try:
                copies = b.extend(some, tokens)
            except MemoryError:
                b.free(some[0])
                continue
            after = state(b)
            b.retract(some, tokens, copies)
            assert state(b) == before
            assert b.extend(some, tokens) == copies and state(b) == after
        elif op == "fork" and len(ids) < 12:
            b.fork(rng.choice(ids))
        elif op == "free":
            b.free(rng.choice(ids))
        elif op == "truncate":
            s = rng.choice(ids)
            b.truncate(s, rng.randint(0, b.length(s)))
        elif op == "compact":
            b.compact()
