"""The 4-bit KV cache and its attention in float64, from the layout and the
formulas alone (numpy, one head and one token at a time)."""
import math

import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def e4m3(byte):
    e, m = byte >> 3 & 15, byte & 7
    if e == 15 and m == 7:
        return math.nan
    v = (1 + m / 8) * 2.0 ** (e - 7) if e else m / 8 * 2.0 ** -6
    return -v if byte & 128 else v


E4M3 = np.array([e4m3(b) for b in range(256)])


def v_row(t):
    return (t & 8) | ((t & 1) << 2) | ((t >> 1) & 3)


def places(t, d):
    """Byte offsets within a group of token t: K codes, V codes, K scales, V scales."""
    i = np.arange(d // 2)
    r = v_row(t)
    swap = (r >> 1 & 1) << 5 if d == 128 else 0
    b = np.arange(d // 16)
    return (t * (d // 2) + i, 8 * d + r * (d // 2) + (i ^ swap), 16 * d + t * (d // 16) + b,
            17 * d + 16 * b + 4 * (t >> 1 & 3) + ((t & 1) | (t >> 3) << 1))


def decode_row(codes, scales):
    nib = np.stack([codes & 15, codes >> 4], 1).reshape(-1)
    val = E2M1[nib & 7] * np.where(nib & 8, -1.0, 1.0)
    return val * np.repeat(E4M3[scales], 16)


def cached(pages, table_row, n, d, ks, vs):
    """float64 K, V [Hkv][n][d] of a sequence's first n tokens (pages: numpy uint8)."""
    H, groups = pages.shape[1], pages.shape[2]
    K, V = np.empty((H, n, d)), np.empty((H, n, d))
    for p in range(n):
        page, off = table_row[p // (16 * groups)], p % (16 * groups)
        kc, vc, ksc, vsc = places(off % 16, d)
        for h in range(H):
            cell = pages[page, h, off // 16]
            K[h, p] = decode_row(cell[kc], cell[ksc]) * float(np.float32(ks))
            V[h, p] = decode_row(cell[vc], cell[vsc]) * float(np.float32(vs))
    return K, V


def places_all(d):
    """places() of the 16 tokens as index arrays [16][d / 2] and [16][d / 16]."""
    return [np.stack(x) for x in zip(*(places(t, d) for t in range(16)))]


def cached_torch(pages, table_row, n, d, ks, vs):
    """cached() by tensor indexing (torch, any device): float64 K, V [Hkv][n][d]."""
    import torch
    dev = pages.device
    cells = pages[table_row.long()]                                 # [pages][Hkv][groups][18 d]
    cells = cells.permute(1, 0, 2, 3).reshape(pages.shape[1], -1, 18 * d)
    val = torch.tensor(np.concatenate([E2M1, -E2M1]), device=dev)
    scl = torch.tensor(E4M3, device=dev)
    kc, vc, ksc, vsc = (torch.from_numpy(x).to(dev) for x in places_all(d))
    out = []
    for c, s, ts in ((kc, ksc, ks), (vc, vsc, vs)):
        code = cells[..., c].long()
        x = torch.stack([val[code & 15], val[code >> 4]], -1).reshape(*code.shape[:-1], d)
        x = x * scl[cells[..., s].long()].repeat_interleave(16, -1) * float(np.float32(ts))
        out.append(x.reshape(pages.shape[1], -1, d)[:, :n])
    return out


def attention_torch(q, K, V, sm):
    """attention() by tensor products (float64 torch): the same five results as numpy arrays."""
    import torch
    n, Hq, d = q.shape
    H, m, _ = K.shape
    G = Hq // H
    x = q.reshape(n, H, G, d).permute(1, 0, 2, 3).reshape(H, n * G, d)
    see = torch.arange(m, device=q.device)[None] <= (m - n + torch.arange(n, device=q.device)).repeat_interleave(G)[:, None]
    z = torch.where(see, x @ K.transpose(1, 2) * sm, -math.inf)
    top = z.amax(-1, keepdim=True) if m else torch.full((H, n * G, 1), -math.inf, dtype=z.dtype, device=z.device)
    safe = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(z - safe)
    total = p.sum(-1, keepdim=True)
    lse = (safe + torch.log(total))[..., 0]
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    big = torch.where(see, x.abs() @ K.abs().transpose(1, 2) * sm, 0.0).amax(-1) if m else torch.zeros_like(lse)
    seen_v = torch.cumsum(V.abs(), 1) if m else V
    last = (m - n + torch.arange(n, device=q.device)).repeat_interleave(G).clamp(min=0)
    flat = (p.amax(-1, keepdim=True) * seen_v[:, last] if m else torch.zeros_like(x))
    back = lambda t: t.reshape(H, n, G, *t.shape[2:]).transpose(0, 1).reshape(n, Hq, *t.shape[2:]).cpu().numpy()
    return back(p @ V), back(lse), back(big), back(p @ V.abs()), back(flat)


def attention(q, K, V, sm):
    """q [n][Hq][d] float64 (the sequence's newest tokens) against K, V [Hkv][m][d].
    Returns out, lse, and the sums the error bounds are made of: the largest
    sum_i |q_i k_i| sm over the keys a row sees, sum_j p_j |v_j|, and
    p_max sum_j |v_j|."""
    n, Hq, d = q.shape
    H, m, _ = K.shape
    out, lse = np.zeros((n, Hq, d)), np.full((n, Hq), -math.inf)
    big, mass, flat = np.zeros((n, Hq)), np.zeros((n, Hq, d)), np.zeros((n, Hq, d))
    for i in range(n):
        see = m - n + i + 1
        if see <= 0:
            continue
        for h in range(Hq):
            k, v = K[h // (Hq // H), :see], V[h // (Hq // H), :see]
            z = k @ q[i, h] * sm
            top = z.max()
            p = np.exp(z - top)
            lse[i, h] = top + math.log(p.sum())
            p /= p.sum()
            out[i, h] = p @ v
            mass[i, h] = p @ np.abs(v)
            flat[i, h] = p.max() * np.abs(v).sum(0)
            big[i, h] = (np.abs(k) @ np.abs(q[i, h])).max() * sm
    return out, lse, big, mass, flat


def bounds(ref, d):
    """Elementwise error bounds of the BF16 output and the FP32 lse.

    A score is a sum of d exact products in FP32 (each of its at most d + 4
    roundings at most 2^-24 of sum |q_i k_i|) times the scales (2 roundings),
    and 2^x and the lse's logarithm are good to a few 2^-22. The weight of a
    key is then off by at most ez relatively, is rounded to FP16 (2^-11; the
    sum of the weights is taken before it), and P V and the sum are FP32 sums
    of n positive-weighted terms in blocks (2^-16 covers n / 16 + 64 steps of
    the lengths tested). FP16 is fixed point at its lower end, with steps of
    2^-24: the weights are scaled by at least 2^6 over the largest, so one that
    is far below it is off by up to 2^-31 of the largest instead. The output is
    rounded to BF16 (2^-8, at most 2^-134 near zero)."""
    out, lse, big, mass, flat = ref
    ez = (d + 8) * 2.0 ** -24 * big + 2.0 ** -20
    rel = 2 * ez[..., None] + 2.0 ** -11 + 2.0 ** -15
    err = rel * mass + 2.0 ** -31 * flat
    return 2.0 ** -8 * (np.abs(out) + err) + err + 1e-38, ez + 2.0 ** -16 + 2.0 ** -23 * np.abs(np.where(np.isfinite(lse), lse, 0))
