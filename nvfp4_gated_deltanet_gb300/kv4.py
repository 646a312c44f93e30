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

__all__ = ["kv4_new_pages", "kv4_append", "kv4_read", "kv4_decode", "kv4_decode_shared", "kv4_prefill", "kv4_score",
           "kv4_evict", "kv4_copy_pages", "kv4_compact", "KV4Book", "KV4Batch", "KV4Cache"]

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


def kv4_decode_shared(q, pages, block_table, kv_len, group_start, shared_len, k_scale, v_scale, max_shared=None,
                      sm_scale=None, out=None, lse=None, return_lse=False, workspace=None, dev_status=None, stream=None):
    """kv4_decode of sequences that share a prefix: sequences [group_start[g],
    group_start[g + 1]) hold the same first shared_len[g] tokens, of which whole
    pages are read once for all of them. max_shared: an upper bound of shared_len
    (default: what the tables can hold)."""
    return _native().decode_shared(q, pages, block_table, kv_len, group_start, shared_len, k_scale, v_scale, max_shared,
                                   sm_scale, out, lse, return_lse, workspace, dev_status, stream)


def kv4_prefill(q, pages, block_table, kv_len, q_start, k_scale, v_scale, total_kv=None, sm_scale=None, out=None,
                lse=None, return_lse=False, workspace=None, dev_status=None, stream=None):
    """Causal attention of ragged prompt chunks: q [T][Hq][d], sequence b's rows
    [q_start[b], q_start[b + 1]) being its newest tokens. total_kv: an upper
    bound of kv_len's sum (default: what the tables can hold). Padding rows
    (from q_start[B] on) get zeros and lse = -infinity; in a given out or lse
    they are left alone."""
    return _native().prefill(q, pages, block_table, kv_len, q_start, k_scale, v_scale, total_kv, sm_scale, out, lse,
                             return_lse, workspace, dev_status, stream)


def kv4_score(q, lse, pages, block_table, kv_len, scores, k_scale, q_start=None, slots=None, scored=None, out=None,
              sm_scale=None, workspace=None, dev_status=None, stream=None):
    """Add the attention weights exp(sm_scale q k - lse) that the rows q gave to
    each cached token, summed over rows and query heads, to the sequences' rows of
    scores FP32 [slots][Hkv][tokens] (sequence b's: slots[b], or b). q and lse as
    kv4_decode takes and returns them, or ragged with q_start as kv4_prefill;
    scored [B]: how many tokens of each sequence have a score, the others' begin
    at 0 (default: all have). out: where the sums go (default: scores itself)."""
    _native().score(q, lse, pages, block_table, kv_len, scores, k_scale, q_start, slots, scored, out, sm_scale, workspace,
                    dev_status, stream)


def kv4_evict(pages, block_table, kv_len, keep, recent, scores, new_table, max_keep=None, slots=None, kept=None,
              new_len=None, scores_out=None, dev_status=None, stream=None):
    """Keep min(keep[b], kv_len[b]) tokens of each sequence and KV head: the newest
    `recent` and, of the others, those of the highest scores (of equal ones the
    older). They move in order to the pages of new_table, their scores with them
    (to scores_out: default scores itself). Returns (kept [B][Hkv][max_keep], the
    places they had, -1 past the last; new_len [B]), int32; with pages and scores
    of all layers, [layers][num_pages]... and [layers][slots]..., kept has a
    leading [layers]. max_keep: an upper bound of keep (default: what the new
    pages can hold)."""
    return _native().evict(pages, block_table, kv_len, keep, recent, scores, new_table, max_keep, slots, kept, new_len,
                           scores_out, dev_status, stream)


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

    def exchange(self, seqs, tokens) -> list:
        """Give distinct sequences seqs[i] new pages for tokens[i] tokens; returns
        what they held, for release or restore. Changes nothing when the pages run out."""
        want = sum(-(-n // self.page_tokens) for n in tokens)
        if want > len(self._free):
            raise MemoryError(f"{want} pages wanted, {len(self._free)} free")
        old = [self.seqs[s] for s in seqs]
        for s, n in zip(seqs, tokens):
            self.seqs[s] = [[self._take() for _ in range(-(-n // self.page_tokens))], n]
        return old

    def release(self, old):
        """Drop the pages that sequences held before an exchange."""
        for pages, _ in old:
            for p in pages:
                self._drop(p)

    def restore(self, seqs, old):
        """Take back the exchange that was the book's last change."""
        for s, entry in zip(reversed(seqs), reversed(old)):
            for p in reversed(self.seqs[s][0]):
                self._drop(p)
            self.seqs[s] = entry

    def groups(self, seqs):
        """Neighbours among seqs that share leading pages, as kv4_decode_shared takes
        them: where each group begins (and len(seqs)), and its shared tokens. A
        sequence joins the group before it where that saves more page reads."""
        def common(a, b):  # sequences that share a page share all before it
            lo, hi = 0, min(len(a), len(b))
            while lo < hi:
                mid = (lo + hi) // 2
                if a[mid] == b[mid]:
                    lo = mid + 1
                else:
                    hi = mid
            return lo

        start, shared = [], []
        pages, n = [self.seqs[s][0] for s in seqs], len(seqs)
        for i in range(n):
            if start:
                members = i - start[-1]
                both = common(pages[i - 1], pages[i])
                if members > 1:
                    both = min(both, shared[-1])
                if members * both > (members - 1) * shared[-1]:
                    shared[-1] = both
                    continue
            start.append(i)
            shared.append(0)
        return start + [n], [p * self.page_tokens for p in shared]

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
    the rows of each sequence, None where they differ (by default T / B). With
    shared prefixes: group_start, shared_len and on the host max_shared, or plain; of a cache
    with scores: slots and scored, and on the host the sequences, their lengths and what scored holds."""

    def __init__(self, block_table, kv_len, q_start, T, total_kv, rows="even"):
        self.block_table, self.kv_len, self.q_start, self.T, self.total_kv = block_table, kv_len, q_start, T, total_kv
        B = kv_len.shape[0]
        self.rows = rows if rows != "even" else T // B if B and T % B == 0 else None
        self.group_start = self.shared_len = self.max_shared = None
        self.plain = False                               # decode_shared is decode: nothing is worth sharing
        self.slots = self.scored = self.seqs = self.lens = self.counts = None


class KV4Cache:
    """The pages of n_layers attention layers, their tensor scales and the book
    of their sequences. A step: batch = cache.grow(seqs, new_tokens), then per
    layer append, and decode or prefill.

    With score_slots and score_tokens the cache also keeps what attention weight
    each token got, for up to score_slots sequences of up to score_tokens tokens
    (4 bytes per token, KV head and layer): score after decode or prefill, in
    every layer and for the same batches, and evict from time to time."""

    def __init__(self, num_pages, page_tokens, n_kv_heads, head_dim, k_scale, v_scale, n_layers=1, device="cuda",
                 score_slots=0, score_tokens=0):
        self.book = KV4Book(num_pages, page_tokens)
        self.layers = kv4_new_pages(num_pages, page_tokens, n_kv_heads, head_dim, n_layers, device)
        self.scales = [(float(k_scale), float(v_scale))] * n_layers
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.device = self.layers.device
        self.scores = None
        if score_slots:
            self.scores = torch.zeros(n_layers, score_slots, n_kv_heads, score_tokens, device=device)
        # _scored: the tokens of a sequence that have a score in every layer; _ahead: {layer: tokens} of the
        # layers that have come further
        self._free_slots, self._slot, self._scored, self._ahead = list(range(score_slots - 1, -1, -1)), {}, {}, {}

    def _needs_scores(self):
        if self.scores is None:
            raise ValueError("the cache was made without score_slots")

    def _slot_for(self, make, scored, ahead):
        """The sequence that `make` adds to the book, with a slot where the cache has scores."""
        if self.scores is None:
            return make()
        if not self._free_slots:
            raise MemoryError("no score slot is free")
        seq = make()
        self._slot[seq], self._scored[seq], self._ahead[seq] = self._free_slots.pop(), scored, dict(ahead)
        return seq

    def new(self) -> int:
        return self._slot_for(self.book.new, 0, {})

    def free(self, seq: int):
        self.book.free(seq)
        if self.scores is not None:
            self._free_slots.append(self._slot.pop(seq))
            del self._scored[seq], self._ahead[seq]

    def fork(self, seq: int, stream=None) -> int:
        """A new sequence with the same tokens; no page is copied until one of the
        two grows (its scores are, on `stream`)."""
        child = self._slot_for(lambda: self.book.fork(seq), self._scored.get(seq, 0), self._ahead.get(seq, {}))
        if self.scores is not None:
            with self._on(stream):
                self.scores[:, self._slot[child]].copy_(self.scores[:, self._slot[seq]])
        return child

    def truncate(self, seq: int, tokens: int):
        self.book.truncate(seq, tokens)
        if self.scores is not None:
            self._recount(seq, lambda n: min(n, tokens))

    def _count(self, seq, layer):
        """How many of a sequence's tokens have a score in the layer."""
        return self._ahead[seq].get(layer, self._scored[seq])

    def _recount(self, seq, f):
        """f of every layer's count."""
        self._scored[seq] = f(self._scored[seq])
        self._ahead[seq] = {layer: f(n) for layer, n in self._ahead[seq].items()}

    def _dev(self, rows):
        return torch.tensor(rows, dtype=torch.int32).pin_memory().to(self.device, non_blocking=True)

    @staticmethod
    def _on(stream):
        """Tables are uploaded, used and freed in the order of one stream."""
        return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)

    def grow(self, seqs, tokens, stream=None, share=False) -> KV4Batch:
        """Room for tokens[i] (or `tokens` each) new tokens of every sequence,
        the copies of shared pages made, and the batch of the new rows; all on
        `stream` (default: the current one), where the batch is to be used.
        share: with the tables that decode_shared needs; sequences that share
        pages have to be neighbours in seqs. share="auto": only what is long enough
        and shared by enough of them is read once, and where nothing is,
        decode_shared is decode. Where one of these fails, the book is as before."""
        seqs = list(seqs)
        tokens = [tokens] * len(seqs) if isinstance(tokens, int) else list(tokens)
        pairs = self.book.extend(seqs, tokens)
        try:
            with self._on(stream):
                if pairs:
                    src, dst = self._dev([p[0] for p in pairs]), self._dev([p[1] for p in pairs])
                    kv4_copy_pages(self.layers, src, dst, dev_status=self.status)
                return self.batch(seqs, tokens, share)
        except BaseException:
            self.book.retract(seqs, tokens, pairs)
            raise

    def batch(self, seqs, tokens, share=False) -> KV4Batch:
        """The tables of the sequences as they are, their newest tokens[i] as the rows."""
        if share not in (False, True, "auto"):
            raise ValueError(f"share: True, False or \"auto\", not {share!r}")
        if self.scores is not None and max([0] + [self.book.length(s) for s in seqs]) > self.scores.shape[3]:
            raise MemoryError(f"a row of scores holds {self.scores.shape[3]} tokens")
        pages = [self.book.pages(s) for s in seqs]
        cols = max([1] + [len(p) for p in pages])
        lens = [self.book.length(s) for s in seqs]
        at = [0]
        for n in tokens:
            at.append(at[-1] + n)
        rows = tokens[0] if len(set(tokens)) == 1 else None
        batch = KV4Batch(self._dev([p + [-1] * (cols - len(p)) for p in pages]), self._dev(lens), self._dev(at), at[-1],
                         sum(lens), rows)
        if share:
            start, shared = self.book.groups(seqs)
            if share == "auto":
                shared = self._paying(start, shared)
                batch.plain = not any(shared)
            batch.group_start, batch.shared_len, batch.max_shared = self._dev(start), self._dev(shared), max([0] + shared)
        if self.scores is not None:
            batch.seqs, batch.lens, batch.counts = list(seqs), lens, [self._scored[s] for s in seqs]
            batch.slots, batch.scored = self._dev([self._slot[s] for s in seqs]), self._dev(batch.counts)
        return batch

    def _paying(self, start, shared):
        """The groups' shared tokens where reading them once is the faster way, 0 elsewhere.

        In us per token and KV head: read by decode 2.2e-5 a member (d = 128; 1.4e-5 at
        64), read once for all 6.2e-5, up to 256 rows; and 13 us a call for its other
        launches. Decode and decode_shared, 32 query heads on 8 of d = 128: 8 sequences on
        8192 tokens 21.0 and 27.0 us, 16 33.8 and 30.2; on 32768 tokens 4 31.4 and 41.0, 8
        54.6 and 41.7. 16 on 4 of 64, 32768 tokens: 8 21.1 and 29.8, 16 34.4 and 29.4."""
        heads, each = self.layers.shape[2], 2.2e-5 if self.layers.shape[4] == 18 * 128 else 1.4e-5
        gain = [S * heads * ((b - a) * each - 6.2e-5) for S, a, b in zip(shared, start, start[1:])]
        pays = sum(max(x, 0.0) for x in gain) > 13.0
        return [S if pays and x > 0.0 else 0 for S, x in zip(shared, gain)]

    def append(self, layer, k, v, batch, stream=None):
        kv4_append(k, v, self.layers[layer], batch.block_table, batch.kv_len, *self.scales[layer],
                   q_start=batch.q_start, dev_status=self.status, stream=stream)

    @staticmethod
    def _same_rows(q, batch):
        if q.dim() in (3, 4):
            B, r = q.shape[0], q.shape[1] if q.dim() == 4 else 1
            if B != batch.kv_len.shape[0] or r != batch.rows:
                has = "different numbers of rows" if batch.rows is None else f"{batch.rows} rows each"
                raise ValueError(f"q: {B} sequences of {r} rows, but the batch has {batch.kv_len.shape[0]} with {has}")

    def decode(self, layer, q, batch, **kw):
        """q [B][Hq][d] or [B][r][Hq][d]: as many rows per sequence as the batch
        has (a row's place in its sequence, and so what it sees, follows from that)."""
        self._same_rows(q, batch)
        return kv4_decode(q, self.layers[layer], batch.block_table, batch.kv_len, *self.scales[layer],
                          dev_status=self.status, **kw)

    def decode_shared(self, layer, q, batch, **kw):
        """decode, the pages that neighbours of the batch share read once (a batch of grow(..., share=True), or "auto")."""
        self._same_rows(q, batch)
        if batch.plain:
            return self.decode(layer, q, batch, **kw)
        if batch.group_start is None:
            raise ValueError("the batch was made without share=True")
        return kv4_decode_shared(q, self.layers[layer], batch.block_table, batch.kv_len, batch.group_start,
                                 batch.shared_len, *self.scales[layer], max_shared=batch.max_shared,
                                 dev_status=self.status, **kw)

    def prefill(self, layer, q, batch, **kw):
        return kv4_prefill(q, self.layers[layer], batch.block_table, batch.kv_len, batch.q_start, *self.scales[layer],
                           total_kv=batch.total_kv, dev_status=self.status, **kw)

    def score(self, layer, q, lse, batch, q_start=None, **kw):
        """Add the weights of the batch's rows to its sequences' scores, by the
        queries and the log-sum-exp of decode, decode_shared or prefill. q_start
        [B + 1]: q holds only these of the newest rows (a prompt's window). A batch
        is scored in every layer; again in one, it adds to what it has there. With
        out (a tensor as kv4_score's) the cache's own scores stay as they are."""
        self._needs_scores()
        if batch.T == 0:
            return
        if q.dim() == 4:
            self._same_rows(q, batch)
        elif q_start is None:
            if q.dim() == 3 and q.shape[0] != batch.T:
                raise ValueError(f"q: {q.shape[0]} rows, but the batch has {batch.T}")
            if batch.rows is None:
                q_start = batch.q_start
            elif batch.rows != 1:                        # as many rows each: a batch of candidates
                q, lse = (x.unflatten(0, (-1, batch.rows)) for x in (q, lse))
        at = range(len(self.layers))[layer]              # -1 is the last one
        counts, scored = [self._count(s, at) for s in batch.seqs], batch.scored
        if counts != batch.counts:                       # the layer has come further than that, or all layers have
            if all(x >= n for x, n in zip(counts, batch.lens)):
                scored = None
            else:
                with self._on(kw.get("stream")):
                    scored = self._dev(counts)
        kv4_score(q, lse, self.layers[layer], batch.block_table, batch.kv_len, self.scores[layer], self.scales[layer][0],
                  q_start=q_start, slots=batch.slots, scored=scored, dev_status=self.status, **kw)
        if kw.get("out") is not None:                    # the sums went elsewhere
            return
        for s, n, x in zip(batch.seqs, batch.lens, counts):
            ahead = self._ahead[s]
            ahead[at] = max(x, min(n, self.book.length(s)))
            if len(ahead) == len(self.layers):
                self._scored[s] = low = min(ahead.values())
                self._ahead[s] = {i: y for i, y in ahead.items() if y > low}

    def evict(self, seqs, keep, recent=0, stream=None):
        """Cut each of the sequences that is longer to keep[i] (or `keep`) tokens per
        layer and KV head: the newest `recent`, and of the others those that got the
        most attention weight; tokens that some layer has not scored have to be among
        the newest (ValueError). Returns the sequences that were cut and the places
        their kept tokens had, int32 [layers][cut][Hkv][most], -1 past the last. From
        then on a cached token's place is not its position in the text, and differs
        between heads. The cut sequences get new pages, the old ones are free after
        the call (MemoryError when there are not enough; the book is then as before):
        evict a few sequences at a time where pages are short. Earlier batches are void."""
        self._needs_scores()
        seqs = list(seqs)
        keep = [keep] * len(seqs) if isinstance(keep, int) else list(keep)
        if len(keep) != len(seqs) or len(set(seqs)) != len(seqs) or recent < 0 or any(k < 0 for k in keep):
            raise ValueError("one number of tokens, zero or more, for each of distinct sequences")
        cut = [(s, k) for s, k in zip(seqs, keep) if self.book.length(s) > k]
        news = [self.book.length(s) - self._scored[s] for s, _ in cut]  # the newest tokens, which some layer has not scored
        for (s, k), n in zip(cut, news):
            if n > min(recent, k):
                raise ValueError(f"sequence {s}: {n} tokens have no score in some layer")
        seqs, keep = [s for s, _ in cut], [k for _, k in cut]
        most = max([0] + keep)
        if not seqs:
            heads = self.layers.shape[2]
            return [], torch.empty(len(self.layers), 0, heads, 0, dtype=torch.int32, device=self.device)

        def table():
            pages = [self.book.pages(s) for s in seqs]
            cols = max([1] + [len(p) for p in pages])
            return self._dev([p + [-1] * (cols - len(p)) for p in pages])

        with self._on(stream):
            before, lens = table(), self._dev([self.book.length(s) for s in seqs])
            slots, keeps = self._dev([self._slot[s] for s in seqs]), self._dev(keep)
        old = self.book.exchange(seqs, keep)
        try:
            with self._on(stream):
                after = table()
            # (not within: what it returns is kept until the current stream is done with it too)
            kept, _ = kv4_evict(self.layers, before, lens, keeps, recent, self.scores, after, max_keep=most, slots=slots,
                                dev_status=self.status, stream=stream)
        except BaseException:
            self.book.restore(seqs, old)
            raise
        self.book.release(old)
        for s, k, (_, n) in zip(seqs, keep, old):
            self._recount(s, lambda x: k - (n - x))      # what had no score is among the newest still
        return seqs, kept

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
