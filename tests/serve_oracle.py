"""Plain 64-bit forms of the serving operators (numpy, one row at a time where
that is the definition), written from their formulas, and the error bounds the
kernels are held to. Shared by the GPU tests; checked against hand-worked
values and closed forms in test_serve_oracle_cpu.py.

Bounds. u is half a unit in the last place of the output's type relative to
its value (2^-11 fp16, 2^-8 bf16, 2^-24 fp32); tiny is half its smallest step.
"""
from __future__ import annotations

import numpy as np

U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}


# ---- rotation and cache --------------------------------------------------------
def turns_of(inv_freq):
    """inv_freq / 2 pi as fractions of a turn in units of 2^-64 (Python integers
    from the exact value of the double)."""
    from fractions import Fraction
    out = []
    for f in np.asarray(inv_freq, dtype=np.float64) / (2 * np.pi):
        v = Fraction(float(f)) % 1
        out.append(round(v * 2 ** 64) % 2 ** 64)
    return out


def rotate(x, positions, inv_freq, interleaved):
    """x (T, H, D) in 64 bits with its first 2 len(inv_freq) elements rotated."""
    y = np.array(x, dtype=np.float64)
    n = len(inv_freq)
    if n == 0:
        return y
    a = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(inv_freq)[None]
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    i0 = np.arange(0, 2 * n, 2) if interleaved else np.arange(n)
    i1 = i0 + 1 if interleaved else i0 + n
    x0, x1 = y[..., i0].copy(), y[..., i1].copy()
    y[..., i0] = x0 * c - x1 * s
    y[..., i1] = x1 * c + x0 * s
    return y


def rotate_bound(x, y, n, interleaved, t):
    """|error| allowed: one rounding of the result; the angle is known to 2^-25
    of half a turn (pi 2^-25 < 1e-7 rad), sine and cosine to 4 ulp (2^-22), and
    the products and sum to 2^-23: under 1e-6 (|x0| + |x1|) together."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    b = U[t] * np.abs(y) + TINY[t]
    if n:
        i0 = np.arange(0, 2 * n, 2) if interleaved else np.arange(n)
        i1 = i0 + 1 if interleaved else i0 + n
        both = 1e-6 * (x[..., i0] + x[..., i1])
        b[..., i0] += both
        b[..., i1] += both
    return b


def place(k_cache, v_cache, k, v, slots):
    """k, v (T, H, D) into k_cache [P][H][ps][D] and v_cache [P][H][ps/8][D][8]."""
    P, _, ps, _ = k_cache.shape
    for t, s in enumerate(slots):
        if 0 <= s < P * ps:
            k_cache[s // ps, :, s % ps] = k[t]
            v_cache[s // ps, :, (s % ps) // 8, :, s % 8] = v[t]


def tokens_of(k_cache, v_cache, ids, n):
    """The first n tokens of the pages ids: K and V as (H, n, D)."""
    P, H, ps, D = k_cache.shape
    k = np.zeros((H, n, D))
    v = np.zeros((H, n, D))
    for j in range(n):
        p, o = ids[j // ps], j % ps
        k[:, j] = k_cache[p, :, o]
        v[:, j] = v_cache[p, :, o // 8, :, o % 8]
    return k, v


# ---- attention -----------------------------------------------------------------
def attention(q, k_cache, v_cache, pages, lens, prefix_pages, prefix_len, q_start, scale, t):
    """(out, lse, bound of out, bound of lse), all (T, Hq[, D]).

    Bound: a logit's error is at most (D + 2) 2^-23 scale sum |q_i k_i| (fp32
    sums in any order; the factor log2(e) and the product with it included),
    S its largest value over the row's keys. A weight is off by that twice (its
    own and the reference's), by 2^-21 from exp2 and the rescalings, and by its
    rounding u; the output is rounded once more.
    """
    T, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    G = Hq // Hkv
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    bo, bl = np.full((T, Hq, D), TINY[t]), np.zeros((T, Hq))
    pk, pv = tokens_of(k_cache, v_cache, prefix_pages, prefix_len)
    for b in range(len(lens)):
        sk, sv = tokens_of(k_cache, v_cache, pages[b], lens[b])
        n = q_start[b + 1] - q_start[b]
        for i in range(n):
            seen = max(0, lens[b] - n + i + 1)
            k = np.concatenate((pk, sk[:, :seen]), 1)
            v = np.concatenate((pv, sv[:, :seen]), 1)
            if k.shape[1] == 0:
                continue
            for h in range(Hq):
                r, hk = q_start[b] + i, h // G
                z = scale * (k[hk] @ q[r, h])
                S = scale * (np.abs(k[hk]) @ np.abs(q[r, h])).max() * (D + 2) * 2.0 ** -23
                m = z.max()
                p = np.exp(z - m)
                out[r, h] = p @ v[hk] / p.sum()
                lse[r, h] = m + np.log(p.sum())
                a = p @ np.abs(v[hk]) / p.sum()
                bo[r, h] += (2 * S + 2.0 ** -21 + U[t]) * a + U[t] * np.abs(out[r, h])
                # weights below 2^-39 of the largest are lost in fp16
                bo[r, h] += len(z) * 2.0 ** -39 * np.abs(v[hk]).max()
                bl[r, h] = S + 2.0 ** -20 + 2.0 ** -22 * abs(lse[r, h])
    return out, lse, bo, bl


# ---- 8-bit floats --------------------------------------------------------------
def e4m3_value(code):
    """Value of an e4m3 code: sign, 4 exponent bits (bias 7), 3 fraction bits;
    no infinities, 0x7F and 0xFF are NaN."""
    s, e, f = code >> 7, (code >> 3) & 15, code & 7
    if e == 15 and f == 7:
        return float("nan")
    v = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
    return -v if s else v


E4M3 = np.array([e4m3_value(c) for c in range(256)])


def e4m3_round(x):
    """x (float64, |x| <= 448 (1 + 2^-20)) to the nearest e4m3 value, ties to even."""
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    # log2 may round up just below a power of two
    e = np.where(np.abs(x) < 2.0 ** e, e - 1, e)
    e = np.maximum(e, -6)
    step = 2.0 ** (e - 3)
    return np.clip(np.rint(x / step) * step, -448.0, 448.0)


def quantize(x):
    """x (M, K) fp32 values -> (code values (M, K), scales (blocks, M) fp32)."""
    x = np.asarray(x, dtype=np.float32)
    M, K = x.shape
    blocks = -(-K // 128)
    vals, scales = np.zeros((M, K)), np.zeros((blocks, M), dtype=np.float32)
    for b in range(blocks):
        g = x[:, 128 * b:128 * b + 128]
        s = np.maximum(np.abs(g).max(1) / np.float32(448.0), np.float32(2.0 ** -126))
        scales[b] = s
        vals[:, 128 * b:128 * b + 128] = e4m3_round((g / s[:, None]).astype(np.float64))
    return vals, scales


def f8_product(w, ws, x, xs):
    """w (N, K), x (M, K) code values; the scaled product (M, N) in 64 bits."""
    (N, K), M = w.shape, x.shape[0]
    kb = np.arange(K) // 128
    W = w * ws.astype(np.float64)[np.arange(N) // 128][:, kb]
    X = x * xs.astype(np.float64)[kb].T
    return X @ W.T
