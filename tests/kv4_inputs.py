"""Cached sequences for the tests of the 4-bit KV cache's attention over shared
prefixes, scores and eviction: pages, tables and the float64 reference over them."""
import numpy as np
import torch

import kv4_ref as ref

KS, VS = 0.017, 0.013


def ints(x, device="cuda"):
    return torch.tensor(x, dtype=torch.int32, device=device)


def queries(T, hq, d, seed, scale=1.5):
    gen = torch.Generator(device="cuda").manual_seed(1000 + seed)
    return (scale * torch.randn(T, hq, d, generator=gen, device="cuda")).bfloat16()


def fill(g, pages, rows, seed):
    """Random tokens appended to the sequences rows = [(page ids, tokens)]; all else stays NaN scales."""
    num, hkv, groups, width = pages.shape
    d = width // 18
    lens = [n for _, n in rows]
    cols = max([1] + [len(p) for p, _ in rows])
    table = ints([list(p) + [-7] * (cols - len(p)) for p, _ in rows])
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lens)
    k = (torch.randn(T, hkv, d, generator=gen, device="cuda") *
         torch.exp(0.5 * torch.randn(hkv, d, generator=gen, device="cuda"))).bfloat16()
    v = torch.randn(T, hkv, d, generator=gen, device="cuda").bfloat16()
    st = ints([0])
    g.kv4_append(k, v, pages, table, ints(lens), KS, VS, q_start=ints(np.concatenate([[0], np.cumsum(lens)]).tolist()),
                 dev_status=st)
    assert st.item() == 0


def prefixed(g, groups, page, hkv, d, seed=0, spare=2):
    """groups: [(shared tokens, [each member's tokens, shared ones among them])]. A
    member with fewer tokens than the group shares holds the front of them. Returns
    pages, table, kv_len, group_start, shared_len and the lengths on the host."""
    rng = np.random.RandomState(seed)
    need = [-(-S // page) for S, _ in groups] + [-(-max(0, n - S // page * page) // page) for S, ns in groups for n in ns]
    ids = rng.permutation(sum(need) + spare).tolist()
    pages = torch.full((len(ids), hkv, page // 16, 18 * d), 0x7F, dtype=torch.uint8, device="cuda")
    take = lambda n: [ids.pop() for _ in range(n)]
    rows, tables, lens, start = [], [], [], [0]
    for S, ns in groups:
        whole = S // page * page            # what lies on shared pages; the rest of S each member holds for itself
        front = take(whole // page)
        rows.append((front, whole))
        for n in ns:
            own = take(-(-max(0, n - whole) // page))
            if n > whole:
                rows.append((own, n - whole))
            tables.append(front[:-(-min(n, whole) // page)] + own)
            lens.append(n)
        start.append(start[-1] + len(ns))
    fill(g, pages, rows, seed)
    cols = max([1] + [len(t) for t in tables])
    table = ints([t + [-7] * (cols - len(t)) for t in tables])
    return pages, table, ints(lens), ints(start), ints([S for S, _ in groups]), lens


def attention(pages, table, lens, counts, q, d):
    """kv4_ref's five results of every row."""
    parts, at = [], 0
    for b, (n, m) in enumerate(zip(counts, lens)):
        page = pages.shape[2] * 16
        K, V = ref.cached_torch(pages, table[b, : -(-m // page)], m, d, KS, VS)
        parts.append(ref.attention_torch(q[at: at + n].double(), K, V, float(np.float32(d ** -0.5))))
        at += n
    return [np.concatenate(x) for x in zip(*parts)]


def close(out, lse, want, d):
    eo, el = ref.bounds(want, d)
    out, lse = (t.double().cpu().numpy().reshape(w.shape) for t, w in ((out, want[0]), (lse, want[1])))
    assert np.isfinite(out).all()
    over = np.abs(out - want[0]) / eo
    assert over.size == 0 or over.max() <= 1, (over.max(), np.unravel_index(over.argmax(), over.shape))
    none = np.isinf(want[1])
    assert (lse[none] == -np.inf).all() and (out[none] == 0).all()
    over = np.abs(lse[~none] - want[1][~none]) / el[~none]
    assert none.all() or over.max() <= 1, over.max()


def weights(pages, table, lens, counts, q, lse, hkv, d, sm=None):
    """Per sequence the float64 sums [Hkv][m] of exp(z - lse) over the rows that see a token, and bounds of
    what FP32 may be off.

    z is a sum of d exact products (at most d + 4 roundings of 2^-24 of sum |q_i k_i| sm) times two scales
    and a power of two; its difference from the lse, in bits, is rounded once (2^-24 of its magnitude) and
    2^x is good to 2^-22: the weight of a row is off by at most ez relatively, and by 2^-126 where it
    underflows. The sum of N such weights is rounded N times, adding the old score once more."""
    out, err, at = [], [], 0
    for b, (n, m) in enumerate(zip(counts, lens)):
        page = pages.shape[2] * 16
        K, _ = ref.cached_torch(pages, table[b, : -(-m // page)], m, d, KS, VS)
        G = q.shape[1] // hkv
        x = q[at: at + n].double().reshape(n, hkv, G, d).permute(1, 0, 2, 3).reshape(hkv, n * G, d)
        L = lse[at: at + n].double().reshape(n, hkv, G).permute(1, 0, 2).reshape(hkv, n * G, 1)
        sm = float(np.float32(d ** -0.5)) if sm is None else sm
        see = torch.arange(m, device=q.device)[None] <= (m - n + torch.arange(n, device=q.device)).repeat_interleave(G)[:, None]
        see = see & ~torch.isinf(L)
        z = x @ K.transpose(1, 2) * sm - torch.where(torch.isinf(L), torch.zeros_like(L), L)
        p = torch.where(see, torch.exp(z), torch.zeros_like(z))
        big = x.abs() @ K.abs().transpose(1, 2) * sm
        ez = (d + 10) * 2.0 ** -24 * big + 2.0 ** -23 * z.abs() + 2.0 ** -22
        out.append(p.sum(1))
        err.append((p * torch.expm1(ez)).sum(1) + (n * G + 2) * 2.0 ** -24 * p.sum(1) + n * G * 2.0 ** -126)
        at += n
    return out, err

