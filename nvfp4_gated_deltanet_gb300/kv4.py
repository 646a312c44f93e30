"""The paged KV cache in 4 bits: its calls, and the book of who holds which page.

The functions marshal the kv4_* entry points of ``include/gdn.h`` (layout,
errors and numerics are described there). ``pages`` is a uint8 CUDA tensor
[num_pages][Hkv][page_tokens / 16][18 * d], or [layers][num_pages]... for the
calls that take all layers at once; its shape gives page_tokens, Hkv and d. A
call runs on the pages' device, where its other tensors must be, and on that
device's current stream unless one is given. Outputs it makes on a given stream
are that stream's memory, kept until the current stream is done with them too;
its inputs are the caller's to keep until the given stream has read them.

    pages = kv4_new_pages(num_pages, page_tokens, n_kv_heads, head_dim)
    kv4_append(k, v, pages, table, kv_len, k_scale, v_scale)
    out = kv4_decode(q, pages, table, kv_len, k_scale, v_scale)

``KV4Book`` decides on the host which page goes where (allocation, forks that
share pages, copy on write, compaction); ``KV4Cache`` joins a book with the
pages of all layers.
"""
from __future__ import annotations

import contextlib
import importlib

import torch

from . import lib

__all__ = ["kv4_new_pages", "kv4_append", "kv4_read", "kv4_decode", "kv4_prefill", "kv4_copy_pages", "kv4_compact",
           "KV4Book", "KV4Batch", "KV4Cache"]

_module = None


def _native():
    """The native binding; raises if it or the library was not built."""
    global _module
    if _module is None:
        lib()
        try:
            _module = importlib.import_module("._kv4", __package__)
        except ImportError as e:
            raise RuntimeError(f"the _kv4 binding is missing ({e}): build it with {__package__}.build.build()") from e
    return _module


def kv4_new_pages(num_pages, page_tokens, n_kv_heads, head_dim, n_layers=None, device="cuda"):
    """Zeroed pages [num_pages][Hkv][page_tokens / 16][18 d], with a leading [n_layers] when given."""
    if page_tokens < 16 or page_tokens % 16:         # the pages would hold fewer tokens than the caller counts
        raise ValueError(f"page_tokens: expected a multiple of 16, not {page_tokens}")
    shape = (num_pages, n_kv_heads, page_tokens // 16, 18 * head_dim)
    return torch.zeros(shape if n_layers is None else (n_layers, *shape), dtype=torch.uint8, device=device)


def kv4_append(k, v, pages, block_table, kv_len, k_scale, v_scale, q_start=None, dev_status=None, stream=None):
    """Quantise the new rows k and v [T][Hkv][d] (BF16, a row's heads together,
    rows evenly spaced) into their sequences' pages; kv_len counts them already."""
    _native().append(k, v, pages, block_table, kv_len, k_scale, v_scale, q_start, dev_status, stream)


def kv4_read(pages, block_table, kv_len, k_scale, v_scale, rows, q_start=None, k=None, v=None, dev_status=None,
             stream=None):
    """(k, v) [rows][Hkv][d] BF16: the values that the pages hold for the
    batch's new rows, zeros in rows that hold no token. Padding rows (from
    q_start[B] on) of a given k or v are left alone."""
    return _native().read(pages, block_table, kv_len, k_scale, v_scale, rows, q_start, k, v, dev_status, stream)


def kv4_decode(q, pages, block_table, kv_len, k_scale, v_scale, sm_scale=None, out=None, lse=None, return_lse=False,
               workspace=None, dev_status=None, stream=None):
    """Attention of the batch's newest tokens: q [B][Hq][d] (one token per
    sequence) or [B][r][Hq][d] (r candidates) -> out of q's shape, BF16; with
    return_lse also the rows' log-sum-exp, FP32. sm_scale: d^-1/2 by default."""
    return _native().decode(q, pages, block_table, kv_len, k_scale, v_scale, sm_scale, out, lse, return_lse, workspace,
                            dev_status, stream)


def kv4_prefill(q, pages, block_table, kv_len, q_start, k_scale, v_scale, total_kv=None, sm_scale=None, out=None,
                lse=None, return_lse=False, workspace=None, dev_status=None, stream=None):
    """Causal attention of ragged prompt chunks: q [T][Hq][d], sequence b's rows
    [q_start[b], q_start[b + 1]) being its newest tokens. total_kv: an upper
    bound of kv_len's sum (default: what the tables can hold). Padding rows
    (from q_start[B] on) get zeros and lse = -infinity; in a given out or lse
    they are left alone."""
    return _native().prefill(q, pages, block_table, kv_len, q_start, k_scale, v_scale, total_kv, sm_scale, out, lse,
                             return_lse, workspace, dev_status, stream)


def kv4_copy_pages(pages, src, dst, dev_status=None, stream=None):
    """Copy pages src[i] -> dst[i] (int32 CUDA tensors) in every layer."""
    _native().copy_pages(pages, src, dst, dev_status, stream)


def kv4_compact(pages, block_table, tables_out=None, page_map=None, n_live=None, workspace=None, dev_status=None,
                stream=None):
    """Move the live pages (those that block_table names) to the front in every
    layer. Returns (the tables with the new ids, every page's new id or -1, the
    number of live pages [1]), all int32."""
    return _native().compact(pages, block_table, tables_out, page_map, n_live, workspace, dev_status, stream)


class KV4Book:
    """Which sequence holds which pages (host only). Pages are counted by their
    holders; a fork shares them all, and a sequence that grows into a page that
    it shares gets a copy of its own first."""

    def __init__(self, num_pages: int, page_tokens: int):
        self.num_pages, self.page_tokens = num_pages, page_tokens
        self.holders = [0] * num_pages
        self._free = list(range(num_pages - 1, -1, -1))  # the lowest id is handed out first
        self.seqs = {}                                   # id -> [pages, tokens]
        self._next = 0

    @property
    def free_pages(self) -> int:
        return len(self._free)

    def length(self, seq: int) -> int:
        return self.seqs[seq][1]

    def pages(self, seq: int) -> list:
        return list(self.seqs[seq][0])

    def new(self) -> int:
        self._next += 1
        self.seqs[self._next - 1] = [[], 0]
        return self._next - 1

    def extend(self, seqs, tokens) -> list:
        """Room for tokens[i] more tokens of sequence seqs[i]; returns the
        (src, dst) page copies to make before they are written. Changes nothing
        when the pages run out."""
        if len(tokens) != len(seqs) or len(set(seqs)) != len(seqs) or any(n < 0 for n in tokens):
            raise ValueError("one number of tokens, zero or more, for each of distinct sequences")
        left, plan, want = {}, [], 0  # left: holders of a shared last page that have not yet left it
        for s, add in zip(seqs, tokens):
            pages, n = self.seqs[s]
            need = -(-(n + add) // self.page_tokens) - len(pages)
            shared = False
            if add > 0 and n % self.page_tokens != 0:
                last = pages[-1]
                shared = left.setdefault(last, self.holders[last]) > 1
                left[last] -= shared
            plan.append((s, add, need, shared))
            want += need + shared
        if want > len(self._free):
            raise MemoryError(f"{want} pages wanted, {len(self._free)} free")
        copies = []
        for s, add, need, shared in plan:
            pages = self.seqs[s][0]
            if shared:
                mine = self._take()
                copies.append((pages[-1], mine))
                self.holders[pages[-1]] -= 1
                pages[-1] = mine
            pages += [self._take() for _ in range(need)]
            self.seqs[s][1] += add
        return copies

    def retract(self, seqs, tokens, copies):
        """Take back the extend that was the book's last change; its copies need not have been made."""
        source = {dst: src for src, dst in copies}
        for s, add in zip(reversed(seqs), reversed(tokens)):
            entry = self.seqs[s]
            pages, n = entry[0], entry[1] - add
            while len(pages) > -(-n // self.page_tokens):
                self._drop(pages.pop())
            if pages and pages[-1] in source:
                mine, pages[-1] = pages[-1], source[pages[-1]]
                self.holders[pages[-1]] += 1
                self._drop(mine)
            entry[1] = n

    def fork(self, seq: int) -> int:
        pages, n = self.seqs[seq]
        for p in pages:
            self.holders[p] += 1
        child = self.new()
        self.seqs[child] = [list(pages), n]
        return child

    def truncate(self, seq: int, tokens: int):
        """Drop the tokens from `tokens` on (rejected candidates) and the pages that only they needed."""
        pages, n = self.seqs[seq]
        if not 0 <= tokens <= n:
            raise ValueError("a sequence is cut to at most its length")
        keep = -(-tokens // self.page_tokens)
        for p in pages[keep:]:
            self._drop(p)
        self.seqs[seq] = [pages[:keep], tokens]

    def free(self, seq: int):
        for p in self.seqs.pop(seq)[0]:
            self._drop(p)

    def compact(self) -> list:
        """kv4_compact's plan: every page's new id (-1: free), applied to the book."""
        live = [p for p in range(self.num_pages) if self.holders[p]]
        L = len(live)
        holes = iter([p for p in range(L) if not self.holders[p]])
        to = [-1] * self.num_pages
        for p in live:
            to[p] = p if p < L else next(holes)
        held = [0] * self.num_pages
        for p in live:
            held[to[p]] = self.holders[p]
        self.holders = held
        self._free = list(range(self.num_pages - 1, L - 1, -1))
        for s in self.seqs.values():
            s[0] = [to[p] for p in s[0]]
        return to

    def _take(self) -> int:
        p = self._free.pop()
        self.holders[p] = 1
        return p

    def _drop(self, p: int):
        self.holders[p] -= 1
        if self.holders[p] == 0:
            self._free.append(p)


class KV4Batch:
    """A batch's device tables: block_table [B][cols], kv_len [B], q_start
    [B + 1] (int32), and on the host its rows T, its cached tokens total_kv and
    the rows of each sequence, None where they differ (by default T / B)."""

    def __init__(self, block_table, kv_len, q_start, T, total_kv, rows="even"):
        self.block_table, self.kv_len, self.q_start, self.T, self.total_kv = block_table, kv_len, q_start, T, total_kv
        B = kv_len.shape[0]
        self.rows = rows if rows != "even" else T // B if B and T % B == 0 else None


class KV4Cache:
    """The pages of n_layers attention layers, their tensor scales and the book
    of their sequences. A step: batch = cache.grow(seqs, new_tokens), then per
    layer append, and decode or prefill."""

    def __init__(self, num_pages, page_tokens, n_kv_heads, head_dim, k_scale, v_scale, n_layers=1, device="cuda"):
        self.book = KV4Book(num_pages, page_tokens)
        self.layers = kv4_new_pages(num_pages, page_tokens, n_kv_heads, head_dim, n_layers, device)
        self.scales = [(float(k_scale), float(v_scale))] * n_layers
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.device = self.layers.device

    def new(self) -> int:
        return self.book.new()

    def free(self, seq: int):
        self.book.free(seq)

    def fork(self, seq: int) -> int:
        """A new sequence with the same tokens; no page is copied until one of the two grows."""
        return self.book.fork(seq)

    def truncate(self, seq: int, tokens: int):
        self.book.truncate(seq, tokens)

    def _dev(self, rows):
        return torch.tensor(rows, dtype=torch.int32).pin_memory().to(self.device, non_blocking=True)

    @staticmethod
    def _on(stream):
        """Tables are uploaded, used and freed in the order of one stream."""
        return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)

    def grow(self, seqs, tokens, stream=None) -> KV4Batch:
        """Room for tokens[i] (or `tokens` each) new tokens of every sequence,
        the copies of shared pages made, and the batch of the new rows; all on
        `stream` (default: the current one), where the batch is to be used.
        Where one of these fails, the book is as before."""
        seqs = list(seqs)
        tokens = [tokens] * len(seqs) if isinstance(tokens, int) else list(tokens)
        pairs = self.book.extend(seqs, tokens)
        try:
            with self._on(stream):
                if pairs:
                    src, dst = self._dev([p[0] for p in pairs]), self._dev([p[1] for p in pairs])
                    kv4_copy_pages(self.layers, src, dst, dev_status=self.status)
                return self.batch(seqs, tokens)
        except BaseException:
            self.book.retract(seqs, tokens, pairs)
            raise

    def batch(self, seqs, tokens) -> KV4Batch:
        """The tables of the sequences as they are, their newest tokens[i] as the rows."""
        pages = [self.book.pages(s) for s in seqs]
        cols = max([1] + [len(p) for p in pages])
        lens = [self.book.length(s) for s in seqs]
        at = [0]
        for n in tokens:
            at.append(at[-1] + n)
        rows = tokens[0] if len(set(tokens)) == 1 else None
        return KV4Batch(self._dev([p + [-1] * (cols - len(p)) for p in pages]), self._dev(lens), self._dev(at), at[-1],
                        sum(lens), rows)

    def append(self, layer, k, v, batch, stream=None):
        kv4_append(k, v, self.layers[layer], batch.block_table, batch.kv_len, *self.scales[layer],
                   q_start=batch.q_start, dev_status=self.status, stream=stream)

    def decode(self, layer, q, batch, **kw):
        """q [B][Hq][d] or [B][r][Hq][d]: as many rows per sequence as the batch
        has (a row's place in its sequence, and so what it sees, follows from that)."""
        if q.dim() in (3, 4):
            B, r = q.shape[0], q.shape[1] if q.dim() == 4 else 1
            if B != batch.kv_len.shape[0] or r != batch.rows:
                has = "different numbers of rows" if batch.rows is None else f"{batch.rows} rows each"
                raise ValueError(f"q: {B} sequences of {r} rows, but the batch has {batch.kv_len.shape[0]} with {has}")
        return kv4_decode(q, self.layers[layer], batch.block_table, batch.kv_len, *self.scales[layer],
                          dev_status=self.status, **kw)

    def prefill(self, layer, q, batch, **kw):
        return kv4_prefill(q, self.layers[layer], batch.block_table, batch.kv_len, batch.q_start, *self.scales[layer],
                           total_kv=batch.total_kv, dev_status=self.status, **kw)

    def compact(self, stream=None) -> int:
        """Move the live pages to the front of every layer; returns their number. Earlier batches are void."""
        seqs = list(self.book.seqs)
        pages = [self.book.pages(s) for s in seqs]
        cols = max([1] + [len(p) for p in pages])
        with self._on(stream):
            table = self._dev([p + [-1] * (cols - len(p)) for p in pages] or [[-1]])
            kv4_compact(self.layers, table, dev_status=self.status)
        self.book.compact()
        return self.book.num_pages - self.book.free_pages

    def check(self, stream=None) -> int:
        """Wait for `stream` (default: for every stream of the device), return
        the sticky status of what ran there and clear it; what is launched
        after that sets it anew."""
        wait = stream.synchronize if stream is not None else lambda: torch.cuda.synchronize(self.device)
        wait()
        with self._on(stream):
            st = int(self.status.item())
            if st:
                self.status.zero_()
        if st:
            wait()
        return st
