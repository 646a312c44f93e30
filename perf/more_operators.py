"""Operators for long 4-bit KV caches, as they are timed: a prefix that a batch
shares, and the eviction of what attention does not look at.

Three operators beside those of the paged cache: kv4_decode_shared (attention of
the newest tokens of sequences that share a prefix, the prefix read once for all
of them), kv4_score (what weight attention gives to each cached token, summed
over query rows and heads and added to what it had) and kv4_evict (the tokens of
the highest scores and the newest ones are kept, per KV head; they move to new
pages, in order, with their scores).

One page holds page_tokens tokens of every KV head; pages is uint8
[num_pages][Hkv][page_tokens / 16][18 d]. A group of 16 tokens of one head is
18 d bytes: 8 d of K codes, 8 d of V codes (E2M1, element 2i in the low nibble
of byte i), d of K scales and d of V scales (E4M3, one per 16 elements). Scores
are FP32 [slots][Hkv][tokens], a row for each sequence and KV head.
"""
import math
import random

import numpy as np
import torch

own = False

K_SCALE, V_SCALE = 0.017, 0.013


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a few samples of one short prompt, a token each: latency only
        {"name": "shared few", "op": "shared", "B": 4, "r": 1, "groups": 1, "shared": 512, "tail": 61, "mix": 3,
         "hq": 16, "hkv": 2, "d": 128, "page": 16},
        # a served batch behind one system prompt, everybody's own turn ragged
        {"name": "shared batch of 64", "op": "shared", "B": 64, "r": 1, "groups": 1, "shared": 8192, "tail": 1000,
         "mix": 4, "hq": 32, "hkv": 8, "d": 128, "page": 64},
        # many questions about one long document: the prefix is a matrix product
        {"name": "shared document", "op": "shared", "B": 128, "r": 1, "groups": 1, "shared": 65536, "tail": 301,
         "mix": 5, "hq": 32, "hkv": 4, "d": 128, "page": 128},
        # five prompts of other lengths, several sequences behind each, four candidate tokens to check per sequence
        {"name": "shared five prefixes", "op": "shared", "B": 37, "r": 4, "groups": 5, "shared": 6016, "tail": 777,
         "mix": 6, "hq": 16, "hkv": 4, "d": 64, "page": 32},
        # the scores of one short conversation after a step: latency only
        {"name": "score one short", "op": "score", "B": 1, "q": 1, "kv": 131, "mix": 0, "hq": 16, "hkv": 2, "d": 128,
         "page": 16, "fresh": False},
        # a served batch's scores after a decode step, ragged
        {"name": "score batch of 64", "op": "score", "B": 64, "q": 1, "kv": 8190, "mix": 7, "hq": 32, "hkv": 8,
         "d": 128, "page": 64, "fresh": False},
        # prompts scored by their last 64 rows, before the rest of them is evicted
        {"name": "score prompt windows", "op": "score", "B": 4, "q": 64, "kv": 16001, "mix": 8, "hq": 32, "hkv": 8,
         "d": 128, "page": 64, "fresh": True, "window": True},
        # prompt chunks scored by all their rows, over cached prefixes
        {"name": "score prompt chunks", "op": "score", "B": 2, "q": 4096, "kv": 8100, "mix": 4, "hq": 32, "hkv": 8,
         "d": 128, "page": 64, "fresh": True},
        # one short conversation in two layers: latency only
        {"name": "evict one short", "op": "evict", "B": 1, "kv": 301, "keep": 130, "recent": 32, "layers": 2, "mix": 0,
         "hkv": 2, "d": 64, "page": 16},
        # a served batch cut to a quarter in a few layers
        {"name": "evict batch of 16", "op": "evict", "B": 16, "kv": 8190, "keep": 2048, "recent": 256, "layers": 4,
         "mix": 9, "hkv": 8, "d": 128, "page": 64},
        # one long context: few rows, long ones
        {"name": "evict one long", "op": "evict", "B": 1, "kv": 200001, "keep": 20000, "recent": 1024, "layers": 1,
         "mix": 0, "hkv": 4, "d": 128, "page": 128},
        # many short sequences in all layers, some of them below the limit
        {"name": "evict many short", "op": "evict", "B": 48, "kv": 1501, "keep": 601, "recent": 77, "layers": 12,
         "mix": 11, "hkv": 2, "d": 128, "page": 32},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "score", "score", "score", "evict", "evict"])
    d, page, mix = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128]), 1 + rng.randrange(1000)
    hkv = rng.choice([1, 2, 4, 8])
    hq = min(64, hkv * rng.choice([1, 2, 3, 4, 6, 8, 8, 16]))
    if op == "shared":
        B, r = _log(rng, 2, 128), rng.choice([1, 1, 1, 2, 3, 4])
        S = _log(rng, page, min(60000, (200 << 20) // (B * r * hq)))
        return {"op": op, "B": B, "r": r, "groups": rng.choice([1, 1, 1, 2, 3, min(B, 6)]),
                "shared": max(1, S // page) * page, "tail": r + _log(rng, 1, min(2000, 120000 // B)), "mix": mix, "hq": hq,
                "hkv": hkv, "d": d, "page": page}
    if op == "score":
        if rng.random() < 0.5:                               # after a decode step, or the check of a few candidates
            B, q = _log(rng, 1, 96), rng.choice([1, 1, 1, 2, 3, 4, 5, 8])
            kv = _log(rng, 1, min(200000, 500000 // (B * min(hkv, 4))))
            return {"op": op, "B": B, "q": q, "kv": kv, "mix": mix, "hq": hq, "hkv": hkv, "d": d, "page": page,
                    "fresh": rng.random() < 0.3}
        B = _log(rng, 1, 6)
        hq = min(hq, 32)
        if rng.random() < 0.5:                               # windows of prompts
            return {"op": op, "B": B, "q": _log(rng, 1, 200), "kv": _log(rng, 200, 30000 // B), "mix": mix, "hq": hq,
                    "hkv": hkv, "d": d, "page": page, "fresh": True, "window": True}
        q = _log(rng, 1, 4000 // B)
        return {"op": op, "B": B, "q": q, "kv": q + rng.choice([0, _log(rng, 1, 4500 // B)]), "mix": mix, "hq": hq,
                "hkv": hkv, "d": d, "page": page, "fresh": rng.random() < 0.5}
    B, layers = _log(rng, 1, 48), rng.randint(1, 8)
    kv = _log(rng, 20, min(100000, 1000000 // (B * layers * hkv)))
    keep = max(1, int(kv * rng.choice([0.1, 0.25, 0.5, 0.9])))
    return {"op": op, "B": B, "kv": kv, "keep": keep, "recent": rng.choice([0, 1, keep // 8, keep // 2, keep]),
            "layers": layers, "mix": mix, "hkv": hkv, "d": d, "page": page}


def _groups(case):
    """The first sequence of each group (and B), each group's shared tokens (whole pages) and each
    sequence's tokens, by the case alone."""
    rng = random.Random(case["mix"])
    B, n = case["B"], min(case["groups"], case["B"])
    start = [0] + sorted(rng.sample(range(1, B), n - 1)) + [B]
    page = case["page"]
    shared = [case["shared"]] + [max(1, int(case["shared"] * rng.uniform(0.2, 1.0)) // page) * page for _ in range(n - 1)]
    r = case["r"]
    tails = [case["tail"]] + [rng.randint(r, case["tail"]) for _ in range(B - 1)]
    kvs = [shared[g] + tails[b] for g in range(n) for b in range(start[g], start[g + 1])]
    return start, shared, kvs


def _lens(case):
    """(query rows, cached tokens) of each sequence, by the case alone."""
    B, kv, mix, q = case["B"], case["kv"], case["mix"], case.get("q", 1)
    if mix == 0 or B == 1:
        return [q] * B, [kv] * B
    rng = random.Random(mix)
    kvs = [kv] + [max(1, int(kv * rng.uniform(0.05, 1.0))) for _ in range(B - 1)]
    if q <= 8:
        return [q] * B, kvs
    if case.get("window"):
        return [min(q, n) for n in kvs], kvs
    qs = [q] + [max(1, int(q * rng.uniform(0.1, 1.0))) for _ in range(B - 1)]
    return qs, [max(a, b) for a, b in zip(qs, kvs)]


def work(case):
    d, hkv = case["d"], case["hkv"]
    half = hkv * (d // 2 + d // 16)                          # 4-bit bytes of one token's K
    if case["op"] == "shared":
        start, shared, kvs = _groups(case)
        r = case["r"]
        alone = sum(kvs) - sum(shared[g] * (start[g + 1] - start[g]) for g in range(len(shared)))
        pairs = sum(sum(n - r + i + 1 for i in range(r)) for n in kvs)
        return {"bytes": 2 * half * (sum(shared) + alone) + case["B"] * r * case["hq"] * (4 * d + 4),
                "flops": 4 * d * pairs * case["hq"]}
    qs, kvs = _lens(case)
    if case["op"] == "score":
        pairs = sum(sum(max(0, kv - q + i + 1) for i in range(q)) for q, kv in zip(qs, kvs))
        entry = 4 if case["fresh"] else 8                    # a score is written, and read where it is added to
        return {"bytes": sum(kvs) * (half + entry * hkv) + sum(qs) * case["hq"] * (2 * d + 4),
                "flops": 2 * d * pairs * case["hq"]}
    kept = sum(min(case["keep"], n) for n in kvs)
    # scores read, kept tokens' K and V read and written, their places and all new scores written
    return {"bytes": case["layers"] * (hkv * 8 * sum(kvs) + kept * (4 * half + 4 * hkv)), "flops": 0}


# ---------------------------------------------------------------- the page layout, plainly
def _v_bytes(d, dev):
    """[16][d/2]: where byte i of token t's V codes lies in a group's V block. Token t is row
    rho(t) = t3 t0 t2 t1 (bits); for d = 128 the two 32-byte halves swap in rows with bit 1 set."""
    t = torch.arange(16, device=dev)[:, None]
    i = torch.arange(d // 2, device=dev)[None, :]
    rho = (t & 8) | ((t & 1) << 2) | ((t >> 1) & 3)
    swap = ((rho >> 1) & 1) if d == 128 else torch.zeros_like(rho)
    return rho * (d // 2) + ((i >> 5) ^ swap) * 32 + (i & 31)


def _v_scales(d, dev):
    """[16][d/16]: where the scale of token t, block b lies in a group's V scales."""
    t = torch.arange(16, device=dev)[:, None]
    b = torch.arange(d // 16, device=dev)[None, :]
    return b * 16 + ((t >> 1) & 3) * 4 + ((t & 1) | ((t >> 3) << 1))


def _token_bytes(d, dev):
    """[16][9 d / 8]: the bytes of a group that belong to token t: K codes, V codes, K scales, V scales."""
    t = torch.arange(16, device=dev)[:, None]
    return torch.cat([t * (d // 2) + torch.arange(d // 2, device=dev), 8 * d + _v_bytes(d, dev),
                      16 * d + t * (d // 16) + torch.arange(d // 16, device=dev), 17 * d + _v_scales(d, dev)], dim=1)


def _quantise(x, ts):
    """x FP32 [..., d] -> (codes uint8 [..., d/2], E4M3 scale bytes uint8 [..., d/16])."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    one = torch.ones((), device=x.device)
    t = torch.full((), ts, device=x.device)
    s8 = (b.abs().amax(-1) * (one / (6.0 * t))).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = s8.float()
    r = torch.where(s > 0, one / (s * t), torch.zeros_like(s))
    y = (b * r[..., None]).abs()
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    code = code + 8 * (torch.signbit(b) & (s > 0)[..., None]).to(torch.uint8)
    code = code.reshape(*x.shape[:-1], x.shape[-1] // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), s8.view(torch.uint8)


def _values(codes, scales):
    """codes [..., d/2], scale bytes [..., d/16] -> E2M1 x E4M3, FP32 [..., d] (exact)."""
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    lut = torch.cat([lut, -lut])
    byte = torch.arange(256, device=codes.device)
    v = torch.stack([lut[byte & 15], lut[byte >> 4]], dim=1)[codes.long()]
    v = v.reshape(*codes.shape[:-1], codes.shape[-1] // 8, 16)
    v = v * scales.view(torch.float8_e4m3fn).float()[..., None]
    return v.reshape(*codes.shape[:-1], 2 * codes.shape[-1])


def _cached(pages, table, d, with_v=True):
    """K (and V) of the pages that the table's rows name, FP32 [rows][Hkv][cols x page_tokens][d]."""
    g = pages[table.long().clamp(min=0)]                          # [rows][cols][Hkv][groups][18 d]
    g = g.permute(0, 2, 1, 3, 4).reshape(table.shape[0], pages.shape[1], -1, 18 * d)
    shape = (table.shape[0], pages.shape[1], -1, d)
    kc, ks = g[..., : 8 * d].reshape(*g.shape[:3], 16, d // 2), g[..., 16 * d: 17 * d].reshape(*g.shape[:3], 16, d // 16)
    k = _values(kc, ks.contiguous()).reshape(shape)
    if not with_v:
        return k, None
    vc, vs = g[..., 8 * d: 16 * d][..., _v_bytes(d, g.device)], g[..., 17 * d:][..., _v_scales(d, g.device)]
    return k, _values(vc, vs.contiguous()).reshape(shape)


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _token_pages(g, num, hkv, page, d):
    """Pages of cached tokens: keys with a few strong channels, as projections give them, quantised."""
    pages = torch.empty(num, hkv, page // 16, 18 * d, dtype=torch.uint8, device="cuda")
    gain = torch.exp(0.5 * torch.randn(hkv, 1, 1, d, generator=g, device="cuda"))
    places = _token_bytes(d, "cuda").reshape(-1)
    step = max(1, (1 << 27) // (hkv * page * d))
    for at in range(0, num, step):
        n = min(step, num - at)
        k = (torch.randn(n, hkv, page // 16, 16, d, generator=g, device="cuda") * gain).to(torch.bfloat16)
        v = torch.randn(n, hkv, page // 16, 16, d, generator=g, device="cuda").to(torch.bfloat16)
        (kc, ks), (vc, vs) = _quantise(k.float(), K_SCALE), _quantise(v.float(), V_SCALE)
        pages[at: at + n, :, :, places] = torch.cat([kc, vc, ks, vs], dim=-1).flatten(-2)
    return pages


def _own_pages(ids, needs):
    """A table [len(needs)][max(needs)] of the next ids, -1 where a row has fewer."""
    table = torch.full((len(needs), max([1] + needs)), -1, dtype=torch.int32)
    ids = ids.cpu()
    at = 0
    for b, n in enumerate(needs):
        table[b, :n] = ids[at: at + n]
        at += n
    return table


def prepare(case, seed):
    g = _gen(seed)
    d, hkv, page, B = case["d"], case["hkv"], case["page"], case["B"]
    s = {"op": case["op"], "page": page, "d": d, "B": B}
    if case["op"] == "shared":
        start, shared, kvs = _groups(case)
        tails = [kvs[b] - shared[k] for k in range(len(shared)) for b in range(start[k], start[k + 1])]
        need = [n // page for n in shared] + [-(-n // page) for n in tails]
        num = sum(need) + 3
        rows = _own_pages(torch.randperm(num, generator=g, device="cuda").to(torch.int32), need)
        cols = max(-(-n // page) for n in kvs)
        table = torch.full((B, cols), -1, dtype=torch.int32)
        for k, n in enumerate(shared):
            for b in range(start[k], start[k + 1]):
                both = torch.cat([rows[k, : n // page], rows[len(shared) + b, : -(-tails[b] // page)]])
                table[b, : len(both)] = both
        s.update(table=table.cuda(), kv_len=_ints(kvs), group_start=_ints(start), shared_len=_ints(shared),
                 most=max(shared), tail=max(tails), members=max(b - a for a, b in zip(start, start[1:])))
        s["pages"] = _token_pages(g, num, hkv, page, d)
        s["q"] = (1.5 * torch.randn(B, case["r"], case["hq"], d, generator=g, device="cuda")).to(torch.bfloat16)
        return s
    qs, kvs = _lens(case)
    need = [-(-n // page) for n in kvs]
    slots = B + 2
    s["slots"] = torch.randperm(slots, generator=g, device="cuda")[:B].to(torch.int32)
    s["kv_len"] = _ints(kvs)
    room = -(-max(kvs) // 64) * 64 + 64
    if case["op"] == "score":
        num = sum(need) + 3
        s["table"] = _own_pages(torch.randperm(num, generator=g, device="cuda").to(torch.int32), need).cuda()
        s["pages"] = _token_pages(g, num, hkv, page, d)
        T = sum(qs)
        s.update(T=T, most=max(qs), q_start=_ints(np.concatenate([[0], np.cumsum(qs)])))
        s["q"] = (1.5 * torch.randn(T, case["hq"], d, generator=g, device="cuda")).to(torch.bfloat16)
        s["lse"] = _row_lse(s)
        if case["q"] <= 8:                                             # every sequence has the same rows
            s["q"], s["lse"] = s["q"].unflatten(0, (B, -1)), s["lse"].unflatten(0, (B, -1))
        s["scores"] = torch.rand(slots, hkv, room, generator=g, device="cuda") * 0.01
        s["scored"] = _ints([0] * B) if case["fresh"] else None        # tokens from here on have no score yet
        s["out"] = torch.zeros_like(s["scores"])
        return s
    keeps = [min(case["keep"], n) for n in kvs]
    more = [-(-n // page) for n in keeps]
    num = sum(need) + sum(more) + 3
    ids = torch.randperm(num, generator=g, device="cuda").to(torch.int32)
    s["table"], s["new_table"] = _own_pages(ids, need).cuda(), _own_pages(ids[sum(need):], more).cuda()
    s["pages"] = torch.randint(0, 256, (case["layers"], num, hkv, page // 16, 18 * d), generator=g, dtype=torch.uint8,
                               device="cuda")
    # sums of attention weights: a few tokens have most of them, many have next to none, some exactly none
    x = torch.exp(2.5 * torch.randn(case["layers"], slots, hkv, room, generator=g, device="cuda") - 6.0)
    s["scores"] = torch.where(x < 1e-4, torch.zeros_like(x), x)
    s.update(keep=_ints(keeps), most=max(keeps), recent=case["recent"], out=torch.zeros_like(x))
    return s


# ---------------------------------------------------------------- one pass
def _run_own(s):
    import nvfp4_gated_deltanet_gb300 as gdn
    if s["op"] == "shared":
        return gdn.kv4_decode_shared(s["q"], s["pages"], s["table"], s["kv_len"], s["group_start"], s["shared_len"],
                                     K_SCALE, V_SCALE, max_shared=s["most"], return_lse=True)
    if s["op"] == "score":
        same = s["q"].dim() == 4
        gdn.kv4_score(s["q"], s["lse"], s["pages"], s["table"], s["kv_len"], s["scores"], K_SCALE,
                      q_start=None if same else s["q_start"], slots=s["slots"], scored=s["scored"], out=s["out"])
        return s["out"]
    kept, new_len = gdn.kv4_evict(s["pages"], s["table"], s["kv_len"], s["keep"], s["recent"], s["scores"],
                                  s["new_table"], max_keep=s["most"], slots=s["slots"], scores_out=s["out"])
    return kept, new_len, s["out"], s["pages"]


def _safe(top):
    return torch.where(top == -math.inf, torch.zeros_like(top), top)


def _run_shared(s):
    """softmax(q K^T) V over the group's shared tokens and each sequence's own, joined in one softmax."""
    d, B, page, pages, kv_len = s["d"], s["B"], s["page"], s["pages"], s["kv_len"].long()
    r, hq, hkv, dev = s["q"].shape[1], s["q"].shape[2], pages.shape[1], pages.device
    first, shared = s["group_start"].long(), s["shared_len"].long()
    G = hq // hkv
    b = torch.arange(B, device=dev)
    g = torch.searchsorted(first[1:], b, right=True)                   # each sequence's group, and place in it
    m = b - first[g]
    member = (first[:-1, None] + torch.arange(s["members"], device=dev)).clamp(max=B - 1)
    q = s["q"].float().reshape(B, r, hkv, G, d).permute(0, 2, 1, 3, 4)  # [B][Hkv][r][G][d]
    c = K_SCALE / math.sqrt(d)
    # the shared tokens, all members' rows at once: [groups][Hkv][members][r G][S]
    k, v0 = _cached(pages, s["table"][first[:-1], : s["most"] // page], d)
    x = q[member].transpose(1, 2).reshape(len(shared), hkv, -1, d)
    z0 = torch.matmul(x, k.transpose(-1, -2)).mul_(c)
    z0.masked_fill_((torch.arange(s["most"], device=dev) >= shared[:, None])[:, None, None], -math.inf)
    z0 = z0.reshape(len(shared), hkv, s["members"], r * G, -1)
    # each sequence's own: [B][Hkv][r G][tail]
    col = shared[g][:, None] // page + torch.arange(-(-s["tail"] // page), device=dev)
    k, v1 = _cached(pages, s["table"].gather(1, col.clamp(max=s["table"].shape[1] - 1)), d)
    z1 = torch.matmul(q.reshape(B, hkv, r * G, d), k.transpose(-1, -2)).mul_(c)
    pos = shared[g][:, None] + torch.arange(k.shape[2], device=dev)
    last = (kv_len[:, None] - r + torch.arange(r, device=dev)).repeat_interleave(G, dim=1)
    z1.masked_fill_((pos[:, None] > last[..., None])[:, None], -math.inf)
    v1 = torch.where((pos < kv_len[:, None])[:, None, :, None], v1, torch.zeros((), device=dev))
    # one maximum and one sum for both
    top = _safe(torch.maximum(z0.amax(-1).transpose(1, 2)[g, m], z1.amax(-1)))
    z1 = z1.sub_(top[..., None]).exp_()
    z0 = z0.sub_(top[member].transpose(1, 2)[..., None]).exp_()
    total = z0.sum(-1).transpose(1, 2)[g, m] + z1.sum(-1)
    o = torch.matmul(z0.flatten(2, 3), v0).reshape(len(shared), hkv, s["members"], r * G, d).transpose(1, 2)[g, m]
    o = (o + torch.matmul(z1, v1)).mul_(V_SCALE) / total[..., None]
    o = o.reshape(B, hkv, r, G, d).permute(0, 2, 1, 3, 4).reshape(B, r, hq, d)
    lse = (top + total.log()).reshape(B, hkv, r, G).permute(0, 2, 1, 3).reshape(B, r, hq)
    return o.to(torch.bfloat16), lse


def _products(s):
    """sm q_i . k_j [B][Hkv][rows G][n] of every (padded) row and key, -inf where a row does not see a key."""
    d, kv_len, qs = s["d"], s["kv_len"].long(), s["q_start"].long()
    k = _cached(s["pages"], s["table"], d, with_v=False)[0]
    B, hkv, n, _ = k.shape
    q = s["q"].reshape(s["T"], -1, d)
    G = q.shape[1] // hkv
    count = qs[1:] - qs[:-1]
    i = torch.arange(s["most"], device=q.device)
    at = (qs[:-1, None] + i).clamp(max=s["T"] - 1)                     # [B][most]
    x = q[at].float().reshape(B, -1, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, -1, d)
    z = torch.matmul(x, k.transpose(-1, -2)).mul_(K_SCALE / math.sqrt(d))
    last = kv_len[:, None] - count[:, None] + i                        # padded rows see nothing
    last = torch.where(i < count[:, None], last, -torch.ones_like(last)).repeat_interleave(G, dim=1)
    z.masked_fill_((torch.arange(n, device=q.device) > last[..., None])[:, None], -math.inf)
    return z


def _row_lse(s):
    """The logarithm of each row's sum, as the attention call before gave it: FP32 [T][Hq]."""
    z = _products(s)
    B, hkv, _, n = z.shape
    top = _safe(z.amax(-1, keepdim=True))
    lse = (top + z.sub_(top).exp_().sum(-1, keepdim=True).log()).reshape(B, hkv, s["most"], -1)
    lse = lse.transpose(1, 2).reshape(B, s["most"], -1)
    row, qs = torch.arange(s["T"], device=z.device), s["q_start"].long()
    b = torch.searchsorted(qs[1:], row, right=True)
    return lse[b, row - qs[b]]


def _run_score(s):
    """scores + sum over rows and the KV head's query heads of exp(z - lse), tokens without a score from 0."""
    kv_len, qs = s["kv_len"].long(), s["q_start"].long()
    z = _products(s)
    B, hkv, _, n = z.shape
    lse = s["lse"].reshape(s["T"], hkv, -1)
    at = (qs[:-1, None] + torch.arange(s["most"], device=z.device)).clamp(max=s["T"] - 1)
    lse = lse[at].transpose(1, 2).reshape(B, hkv, -1)                  # [B][Hkv][rows G]
    w = z.sub_(_safe(lse)[..., None]).exp_().sum(2)
    slots = s["slots"].long()
    old = s["scores"][slots]
    room = old.shape[-1]
    pos = torch.arange(room, device=z.device)
    if s["scored"] is not None:
        old = torch.where((pos < s["scored"][:, None])[:, None], old, torch.zeros_like(old))
    w = torch.nn.functional.pad(w, (0, max(0, room - n)))[..., :room]
    s["out"][slots] = torch.where((pos < kv_len[:, None])[:, None], old + w, s["out"][slots])
    return s["out"]


def _run_evict(s):
    """The newest `recent` tokens and the best of the others, `keep` in all, in order, into the new pages."""
    kv_len, keep, slots, dev = s["kv_len"].long(), s["keep"].long(), s["slots"].long(), s["pages"].device
    scores, d, page = s["scores"][:, slots], s["d"], s["page"]          # [L][B][Hkv][room]
    L, B, hkv, room = scores.shape
    pos = torch.arange(room, device=dev)
    inside = pos < kv_len[:, None]
    recent = keep.clamp(max=s["recent"])
    newest = inside & (pos >= (kv_len - recent)[:, None])
    key = torch.where(newest[:, None], math.inf, torch.where(inside[:, None], scores, -math.inf))
    order = key.sort(dim=-1, descending=True, stable=True).indices[..., : s["most"]]
    order = torch.where(pos[: s["most"]] < keep[:, None, None], order, room).sort(dim=-1).values
    have = order < room
    kept = torch.where(have, order, -1).to(torch.int32)
    src = torch.where(have, order, 0)
    moved = torch.where(have, scores.gather(-1, src), torch.zeros((), device=dev))
    out = torch.zeros_like(scores)
    out[..., : s["most"]] = moved
    s["out"][:, slots] = torch.where(inside[:, None], out, s["out"][:, slots])
    # the tokens' bytes, whole groups of 16: what no token fills of the last one becomes zeros
    width = -(-s["most"] // 16) * 16
    src, have = (torch.nn.functional.pad(x, (0, width - s["most"])) for x in (src, have))
    place = _token_bytes(d, dev)
    l, b, h = (torch.arange(n, device=dev).reshape(shape) for n, shape in ((L, (-1, 1, 1, 1)), (B, (1, -1, 1, 1)),
                                                                          (hkv, (1, 1, -1, 1))))
    at = s["table"].long()[b, src // page].clamp(min=0)
    cell = s["pages"][l[..., None], at[..., None], h[..., None], (src % page // 16)[..., None], place[src % 16]]
    cell = torch.where(have[..., None], cell, torch.zeros_like(cell))
    to = torch.arange(width, device=dev).expand(L, B, hkv, width)
    writes = to // 16 * 16 < keep[:, None, None]
    l, b, h = (x.expand(L, B, hkv, width)[writes] for x in (l, b, h))
    to, cell = to[writes], cell[writes]
    at = s["new_table"].long()[b, to // page]
    s["pages"][l[:, None], at[:, None], h[:, None], (to % page // 16)[:, None], place[to % 16]] = cell
    return kept, torch.minimum(keep, kv_len).to(torch.int32), s["out"], s["pages"]


def run(state):
    if own:
        return _run_own(state)
    return {"shared": _run_shared, "score": _run_score, "evict": _run_evict}[state["op"]](state)


# ---------------------------------------------------------------- the definition, in 64 bits
def _exact_head(cells, d, which):
    """FP64 [n][d] of one head's K (0) or V (1) from its groups' bytes, uint8 [n/16][18 d]."""
    n = cells.shape[0]
    grid = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=cells.device) / 2
    out = torch.empty(n, 16, d, dtype=torch.float64, device=cells.device)
    for t in range(16):
        row = t
        if which:
            row = 8 * (t // 8) + 4 * (t % 2) + (t % 8) // 2
        code = cells[:, (8 * d if which else 0) + row * d // 2:][:, : d // 2].long()
        if which and d == 128 and row // 2 % 2:
            code = torch.cat([code[:, 32:], code[:, :32]], dim=1)
        nib = torch.stack([code % 16, code // 16], dim=2).reshape(n, d)
        val = grid[nib % 8] * (1 - 2 * (nib // 8))
        for b in range(d // 16):
            at = 17 * d + 16 * b + 4 * (t % 8 // 2) + t % 2 + 2 * (t // 8) if which else 16 * d + t * (d // 16) + b
            byte = cells[:, at].long()
            e, man = byte // 8 % 16, (byte % 8).double()
            sc = torch.where(e > 0, (8 + man) * 2.0 ** (e.double() - 10), man * 2.0 ** -9)
            out[:, t, 16 * b: 16 * b + 16] = val[:, 16 * b: 16 * b + 16] * sc[:, None]
    return out.reshape(n * 16, d)


def exact(case, seed):
    s = prepare(case, seed)
    d, hkv, dev = case["d"], case["hkv"], "cuda"
    if case["op"] == "evict":
        return _exact_evict(case, s)
    ks, vs = float(np.float32(K_SCALE)), float(np.float32(V_SCALE))
    hq = case["hq"]
    G = hq // hkv
    if case["op"] == "shared":
        kvs, r = s["kv_len"].tolist(), case["r"]
        out = torch.zeros(case["B"], r, hq, d, dtype=torch.float64, device=dev)
        lse = torch.zeros(case["B"], r, hq, dtype=torch.float64, device=dev)
        start, shared = s["group_start"].tolist(), s["shared_len"].tolist()
        for h in range(hkv):
            for k, S in enumerate(shared):
                cells = s["pages"][s["table"][start[k], : S // case["page"]].long()][:, h].reshape(-1, 18 * d)
                K0, V0 = _exact_head(cells, d, 0), _exact_head(cells, d, 1)
                for b in range(start[k], start[k + 1]):
                    n = kvs[b]
                    cols = s["table"][b, S // case["page"]: -(-n // case["page"])].long()
                    cells = s["pages"][cols][:, h].reshape(-1, 18 * d)
                    K = torch.cat([K0, _exact_head(cells, d, 0)])[:n]
                    V = torch.cat([V0, _exact_head(cells, d, 1)])[:n]
                    q = s["q"][b, :, h * G: h * G + G].double()
                    z = q @ K.T * (ks / math.sqrt(d))                  # [r][G][n]
                    for i in range(r):
                        z[i, :, n - r + i + 1:] = -math.inf
                    top = z.max(-1, keepdim=True).values
                    p = torch.exp(z - top)
                    out[b, :, h * G: h * G + G] = p @ V / p.sum(-1, keepdim=True) * vs
                    lse[b, :, h * G: h * G + G] = (top + torch.log(p.sum(-1, keepdim=True)))[..., 0]
        return out, lse
    qs, kvs = _lens(case)
    got = torch.zeros(s["out"].shape, dtype=torch.float64, device=dev)
    q, lse = s["q"].reshape(-1, hq, d), s["lse"].reshape(-1, hq).double()
    at = 0
    for b, (n, m) in enumerate(zip(qs, kvs)):
        used = s["pages"][s["table"][b, : -(-m // case["page"])].long()]
        for h in range(hkv):
            K = _exact_head(used[:, h].reshape(-1, 18 * d), d, 0)[:m]
            total = torch.zeros(m, dtype=torch.float64, device=dev)
            for lo in range(0, n, 512):
                hi = min(n, lo + 512)
                z = q[at + lo: at + hi, h * G: h * G + G].double().reshape(-1, d) @ K.T * (ks / math.sqrt(d))
                p = torch.exp(z - lse[at + lo: at + hi, h * G: h * G + G].reshape(-1, 1))
                last = m - n + torch.arange(lo, hi, device=dev).repeat_interleave(G)
                p[torch.arange(m, device=dev)[None] > last[:, None]] = 0.0
                total += p.sum(0)
            slot = int(s["slots"][b])
            if not case["fresh"]:
                total += s["scores"][slot, h, :m].double()
            got[slot, h, :m] = total
        at += n
    return got


def _exact_evict(case, s):
    """Places, lengths and moved scores, a row at a time; the pages' bytes are no computed numbers."""
    _, kvs = _lens(case)
    scores = s["scores"].cpu().numpy().astype(np.float64)
    keep, slots = s["keep"].tolist(), s["slots"].tolist()
    kept = np.full((case["layers"], case["B"], case["hkv"], s["most"]), -1, np.int64)
    out = np.zeros(scores.shape)
    for b, n in enumerate(kvs):
        old = n - min(case["recent"], keep[b])                         # the tokens that have to compete
        for l in range(case["layers"]):
            for h in range(case["hkv"]):
                x = scores[l, slots[b], h, :n]
                best = np.lexsort((np.arange(old), -x[:old]))[: keep[b] - (n - old)]
                at = np.sort(np.concatenate([best, np.arange(old, n)]))
                kept[l, b, h, : len(at)] = at
                out[l, slots[b], h, : len(at)] = x[at]
    new = np.minimum(keep, kvs)
    return torch.from_numpy(kept).int(), torch.from_numpy(new).int(), torch.from_numpy(out), None
