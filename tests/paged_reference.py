"""Plain 64-bit forms of the operators of a cache in pages, and the bounds the GPU tests hold the kernels to."""
import math

import torch

from tests.tree_reference import BF, TERMS, U

E4M3 = torch.float8_e4m3fn


def code_values():
    """The value of each e4m3 code, from its bits."""
    out = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out.append(math.nan if c & 127 == 127 else -x if c & 128 else x)
    return torch.tensor(out, dtype=torch.float64)


def power(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def exponents(x):
    """The byte of each block of 32 of the float64 rows x: the smallest e in [-100, 7] with max|x| <= 448 * 2^e, + 127."""
    y = x.unflatten(-1, (-1, 32))
    most = y.abs().amax(-1)
    finite = torch.isfinite(y).all(-1)
    e = torch.full(most.shape, 7, dtype=torch.int64, device=x.device)
    for k in range(6, -101, -1):
        e[most <= 448.0 * 2.0 ** k] = k
    return torch.where(finite, e + 127, 255)


def quantise(x):
    """(codes E4M3, bytes) of float64 rows: the nearest code, ties to the even one."""
    s = exponents(x)
    y = x.unflatten(-1, (-1, 32)) / power(torch.where(s == 255, 127, s) - 127)[..., None]
    y = torch.where(torch.isfinite(y), y, 0.0).clamp(-448.0, 448.0)
    y = torch.where((s == 255)[..., None], 0.0, y)
    table = code_values().to(x.device)
    pos = table[:127]  # rising
    a = y.abs()
    hi = torch.searchsorted(pos, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - pos[lo], pos[hi] - a
    code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = torch.where(torch.signbit(y), code + 128, code)
    return code.to(torch.uint8).flatten(-2).view(E4M3), s.to(torch.uint8)


def values(codes, scales):
    """The float64 values of 8-bit rows."""
    x = code_values().to(codes.device)[codes.view(torch.uint8).long()]
    f = torch.where(scales == 255, torch.nan, power(scales.long() - 127))
    return x * f.repeat_interleave(32, -1)


def rows_of(pool, table, n):
    """Rows [0, n) of a sequence in a layer's float64 pool [pages][Hkv][ps][hd], as [Hkv][n][hd]; zeros on pages outside."""
    P, Hkv, ps, hd = pool.shape
    out = []
    for i in range(-(-n // ps)):
        p = int(table[i])
        out.append(pool[p] if 0 <= p < P else torch.zeros(Hkv, ps, hd, dtype=pool.dtype, device=pool.device))
    return torch.cat(out, 1)[:, :n] if out else pool.new_zeros(Hkv, 0, hd)


def attention(q, k, v, table, starts, lengths, scale, window, sinks):
    """(out, bound) in float64 [n][Hq][hd] for float64 pools k, v; tokens outside every sequence are NaN in both. The
    bound is that of tree_reference.attention, whose terms hold here as they do there."""
    f32 = q.dtype == torch.float32
    N, Hq, hd = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    out = torch.full((N, Hq, hd), math.nan, dtype=torch.float64, device=q.device)
    tol = torch.full_like(out, math.nan)
    for b in range(len(lengths)):
        lo, hi = (max(0, min(int(x), N)) for x in (starts[b], starts[b + 1]))
        n = hi - lo
        if n <= 0:
            continue
        L = max(0, min(int(lengths[b]), table.shape[1] * k.shape[2]))
        kk, vv = rows_of(k, table[b], L), rows_of(v, table[b], L)
        p = torch.arange(L - n, L, device=q.device)[:, None]
        j = torch.arange(L, device=q.device)[None]
        seen = j <= p
        if window:
            seen = seen & ((j > p - window) | (j < sinks))
        count = seen.sum(1).clamp(min=1)[None, :, None, None]
        for h in range(Hkv):
            qh = q[lo:hi, h * G:(h + 1) * G].double()
            on = seen[:, None, :]
            ks, vs = torch.nan_to_num(kk[h], 0.0, 0.0, 0.0), vv[h]
            s = torch.where(on, scale * qh @ kk[h].T, -math.inf) if L else qh.new_zeros(n, G, 0)
            w = torch.softmax(s, -1) if L else s
            w = torch.where(on, w, 0.0)
            w = torch.where(seen.any(1)[:, None, None], w, 0.0)
            if bool(torch.isfinite(vs).all()):
                o, a = w @ vs, w @ vs.abs()
            else:  # (what a token does not see must not count: row by row)
                o = torch.stack([w[t][:, seen[t]] @ vs[seen[t]] for t in range(n)])
                a = torch.stack([w[t][:, seen[t]] @ vs[seen[t]].abs() for t in range(n)])
            d = scale * (qh.abs() @ ks.abs().T) * ((TERMS + U if f32 else 0.0) + 3 * hd * U)
            d = torch.where(on, d, 0.0).amax(-1, keepdim=True) if L else qh.new_zeros(n, G, 1)
            big = torch.where(on & torch.isfinite(s), s, 0.0).abs().amax() if L else 0.0
            rel = 2 * (d + 2 * U * big) + (TERMS if f32 else 2.0 ** -16) + 2.0 ** -20 + (3 * count[0] / 16 + 80) * 2.0 ** -23
            out[lo:hi, h * G:(h + 1) * G] = o
            tol[lo:hi, h * G:(h + 1) * G] = a * rel + (0.0 if f32 else BF) * (o.abs() + a * rel) + 1e-30
    return out, tol
