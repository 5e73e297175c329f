"""Plain fp64 definitions of the serving operators on CPU tensors, for the tests."""
import math

import torch


def rotate(x, positions, inv_freq, interleaved, mscale=1.0, inverse=False):
    """x [..., H, d] with one position per leading entry [...]; m R x, or m R^T x."""
    rot = 2 * inv_freq.shape[0]
    a = positions.double().unsqueeze(-1) * inv_freq.double()
    cos, sin = (torch.cos(a) * mscale).unsqueeze(-2), (torch.sin(a) * mscale).unsqueeze(-2)
    if inverse:
        sin = -sin
    x = x.double()
    y = x.clone()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y[..., first] = x[..., first] * cos - x[..., second] * sin
    y[..., second] = x[..., second] * cos + x[..., first] * sin
    return y


def e4m3_value(code):
    """Value of an e4m3 code (int), from its fields."""
    sign = -1.0 if code & 0x80 else 1.0
    e, m = (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return math.nan
    return sign * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))


E4M3 = torch.tensor([e4m3_value(c) for c in range(256)], dtype=torch.float64)


def quantise_row(x):
    """(codes, byte) of one row of floats, from the definition: the smallest exponent e in
    [-127, 120] with max|finite x| <= 448 * 2^e, codes to the nearest value, ties to even."""
    x = [float(t) for t in x]
    amax = max([abs(t) for t in x if math.isfinite(t)] or [0.0])
    e = -127
    while e < 120 and amax > 448.0 * 2.0 ** e:
        e += 1
    positive = E4M3[:127]                      # codes 0 .. 126 in rising order, 126 = 448
    codes = []
    for t in x:
        if math.isnan(t):
            codes.append(0x7f)
            continue
        y = min(abs(t) * 2.0 ** -e if math.isfinite(t) else 448.0, 448.0)
        dist = (positive - y).abs()
        best = dist.min()
        near = [c for c in range(127) if dist[c] == best]
        c = near[0] if len(near) == 1 else [n for n in near if n % 2 == 0][0]
        codes.append(c | (0x80 if math.copysign(1.0, t) < 0 else 0))
    return codes, e + 127


def widened(codes_u8, scale_u8):
    """codes [..., d] uint8 and scale bytes [...] -> fp64 values."""
    return E4M3[codes_u8.long()] * torch.exp2(scale_u8.double() - 127).unsqueeze(-1)


def gathered(cache, table_row, L):
    """Positions [0, L) of a sequence from fp64 pages [P, H, page, d] -> [H, L, d]."""
    page = cache.shape[2]
    ids = table_row[: -(-L // page)].long() if L > 0 else table_row[:0].long()
    x = cache[ids]
    return x.transpose(0, 1).reshape(cache.shape[1], -1, cache.shape[3])[:, :L]


def attend(q, k_cache, v_cache, table, cu_q, kv_len, scale, causal=True, window=None):
    """(o, lse, wabs) in fp64 for packed q [T, Hq, d]; wabs = sum_j w_j |v_j|, which bounds what
    rounding P can do.  Rows behind the last sequence are NaN."""
    T, Hq, d = q.shape
    G = Hq // k_cache.shape[1]
    o = torch.full((T, Hq, d), math.nan, dtype=torch.float64)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64)
    wabs = torch.full((T, Hq, d), math.nan, dtype=torch.float64)
    for b in range(len(kv_len)):
        L = max(0, int(kv_len[b]))
        k, v = gathered(k_cache, table[b], L), gathered(v_cache, table[b], L)
        key = torch.arange(L)
        for t in range(int(cu_q[b]), int(cu_q[b + 1])):
            pos = L - int(cu_q[b + 1]) + t
            seen = key <= pos if causal else key >= 0
            if window is not None and window >= 0:
                seen = seen & (key >= pos - window)
            if not bool(seen.any()):
                o[t], lse[t], wabs[t] = 0.0, -math.inf, 0.0
                continue
            ks, vs = k[:, seen].repeat_interleave(G, 0), v[:, seen].repeat_interleave(G, 0)
            s = torch.einsum("hd,hkd->hk", q[t].double(), ks) * scale
            w = torch.softmax(s, -1)
            o[t] = torch.einsum("hk,hkd->hd", w, vs)
            wabs[t] = torch.einsum("hk,hkd->hd", w, vs.abs())
            lse[t] = torch.logsumexp(s, -1)
    return o, lse, wabs
