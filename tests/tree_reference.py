"""Plain 64-bit forms of the drafted-tree operators, and the error bounds the
GPU tests hold the kernels to (derived in the functions' comments).

u = 2^-24 is half a step of fp32, 2^-8 half a step of bf16, relative to the
value."""
import math

import torch

U = 2.0 ** -24
BF = 2.0 ** -8
TERMS = 2.0 ** -24  # what three bf16 terms leave of a value: half a step of the third (2^-8 of a rest of a rest)


def rope(qkv, Hq, Hkv, hd, positions, inv_freq, q_norm, k_norm, eps, mscale, interleaved):
    """(rotated q, rotated k, v) in float64, and for each of q, k the bound's scale |a| + |b|."""
    n, half = qkv.shape[0], inv_freq.shape[0]
    x = qkv.double().reshape(n, Hq + 2 * Hkv, hd)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    ang = positions.double()[:, None] * inv_freq.double()[None]
    c, s = ang.cos()[:, None] * mscale, ang.sin()[:, None] * mscale

    def turn(y, gain):
        if gain is not None:
            y = y / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt() * gain.double()
        i = torch.arange(half, device=y.device)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        out, mag = y.clone(), y.abs()
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        mag[..., a] = mag[..., b] = (y[..., a].abs() + y[..., b].abs()) * mscale
        return out, mag

    return turn(q, q_norm), turn(k, k_norm), v


# The norm: a sum of squares over 4 + log2(32) adds and a product (9 u, halved
# by the root), the reciprocal root within two steps (4 u) and eps (1 u), two
# products (2 u): 12 u. The angle: the fraction of a turn rounded to fp32 (3.2 u
# of a radian), sine and cosine within 2 u, times mscale (1 u), a product and an
# add (2 u): 8.2 u.
# A position below 2^17 adds 2^17 * 2^-53 turns: nothing. Rounded up to 24 u.
ROPE_TOL = 24 * U


def attention(q, k, v, lengths, masks, counts, slots, scale):
    """(out, bound) in float64 [B][T][Hq][hd]; rows of nodes behind counts[b] are NaN.

    With p the normalised weights and A = sum p |v| the kernel's error is at most A times
      2 d    the scores' error d (the larger of the row's) moves every weight by at most e^(2d) - 1;
             d = scale sum |q k| (e_q + 3 hd u): e_q = TERMS + u for fp32 queries, scaled before they are split (0 for
             bf16), fp32 sums of 3 hd terms; and the scaled difference from the maximum rounded: u (|s| + |m|) <= 2 u
             max|s|
      e_p    the weights' own rounding: TERMS (fp32) or BF (bf16), and exp2 within 2^-20
      (3 n/16 + 80) 2^-23   the running sums of weights and products over the n rows, 16 rows and a term at a time,
             tens of rescalings and joins, one step each (a tensor core's sum may cut instead of rounding)
    plus the rounding of a bf16 result."""
    f32 = q.dtype == torch.float32
    B, T, Hq, hd = q.shape
    Hkv, G = k.shape[1], Hq // k.shape[1]
    out = torch.full((B, T, Hq, hd), float("nan"), dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for b in range(B):
        n, c = int(lengths[b]), T if counts is None else int(counts[b])
        if c == 0:
            continue
        sl = b if slots is None else int(slots[b])
        words = [w & ((1 << 64) - 1) for w in masks[b].tolist()]
        seen = torch.ones(c, n + c, dtype=torch.bool)
        seen[:, n:] = torch.tensor([[bool((words[t] >> j) & 1) for j in range(c)] for t in range(c)])
        seen = seen.to(q.device)
        for h in range(Hkv):
            kk, vv = k[sl, h, :n + c].double(), v[sl, h, :n + c].double()
            for t in range(c):
                on = seen[t].nonzero()[:, 0]
                if not len(on):
                    out[b, t, h * G:(h + 1) * G] = 0
                    continue
                qt, kt, vt = q[b, t, h * G:(h + 1) * G].double(), kk[on], vv[on]
                s = scale * qt @ kt.T
                p = torch.softmax(s, -1)
                a = p @ vt.abs()
                d = scale * (qt.abs() @ kt.abs().T) * ((TERMS + U if f32 else 0.0) + 3 * hd * U) + 2 * U * s.abs().amax()
                rel = 2 * d.amax(-1, keepdim=True) + (TERMS if f32 else BF) + 2.0 ** -20
                rel = rel + (3 * len(on) / 16 + 80) * 2.0 ** -23
                o = p @ vt
                out[b, t, h * G:(h + 1) * G] = o
                tol[b, t, h * G:(h + 1) * G] = a * rel + (0.0 if f32 else BF) * (o.abs() + a * rel) + 1e-30
    return out, tol


def random_parents(n, gen, roots=1):
    p = [-1] * n
    for t in range(roots, n):
        p[t] = t - 1 - int(torch.randint(0, min(t, 8), (1,), generator=gen))
    return p


def mask_words(parents):
    w = []
    for t, p in enumerate(parents):
        w.append((w[p] if p >= 0 else 0) | (1 << t))
    return w


def signed(w):
    return w - (1 << 64) if w >= (1 << 63) else w


def compact(x, starts, nodes, counts):
    new = x.clone()
    for b in range(x.shape[1]):
        for i in range(int(counts[b])):
            src, dst = int(starts[b]) + int(nodes[b][i]), int(starts[b]) + i
            if int(nodes[b][i]) >= 0 and src < x.shape[3] and dst < x.shape[3]:
                new[:, b, :, dst] = x[:, b, :, src]
    return new


def reorder(x, sources, lengths):
    new = x.clone()
    for b in range(x.shape[1]):
        s, n = int(sources[b]), max(0, min(int(lengths[b]), x.shape[3]))
        if 0 <= s < x.shape[1]:
            new[:, b, :, :n] = x[:, s, :, :n]
    return new
