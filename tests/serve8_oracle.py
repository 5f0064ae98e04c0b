"""Plain 64-bit forms of the serving operators in fewer bits (numpy), written
from their formulas, and the error bounds the kernels are held to. Shared by the
GPU tests; checked against hand-worked values in test_serve8_oracle_cpu.py.

u is half a step of a type relative to its value (serve_oracle.U); e4m3 2^-4 of
the value, and 2^-10 of the scale below 2^-6 of it."""
from __future__ import annotations

import numpy as np

from serve_oracle import E4M3, TINY, U, e4m3_round, rotate

E_MIN, E_MAX = -60, {"f16": 7, "bf16": 60}
NP16 = {"f16": np.float16}


def to_type(x, t):
    """float64 rounded to the 16-bit type (as float64)."""
    if t == "f16":
        with np.errstate(over="ignore"):
            return x.astype(np.float16).astype(np.float64)
    x = x.astype(np.float32)
    b = x.view(np.uint32)
    r = ((b + 0x7fff + ((b >> 16) & 1)) & np.uint32(0xffff0000)).view(np.float32)
    return np.where(np.isfinite(x), r, x).astype(np.float64)


# ---- norm and append -----------------------------------------------------------
def norm(x, w, eps):
    """x / sqrt(mean(x^2) + eps) * w over the last axis; w None: x."""
    x = np.asarray(x, dtype=np.float64)
    if w is None:
        return x
    with np.errstate(invalid="ignore", divide="ignore"):
        return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w


def norm_rotate(x, w, eps, pos, inv, inter):
    """The value, and the error that fp32 may make of it: of the norm, at most 22
    additions to half effect, the root, the quotient and two products, 15 2^-24 <
    2^-20 of each element; of the rotation 1e-6 of both elements of a pair (as in
    serve_oracle.rotate_bound)."""
    y = norm(x, w, eps)
    z = rotate(y, pos, inv, inter)
    a, n = np.abs(y), len(inv)
    e = (2.0 ** -20 * a) if w is not None else np.zeros_like(a)
    if n:
        i0 = np.arange(0, 2 * n, 2) if inter else np.arange(n)
        i1 = i0 + 1 if inter else i0 + n
        both = (1e-6 + (2.0 ** -20 if w is not None else 0)) * (a[..., i0] + a[..., i1])
        e[..., i0], e[..., i1] = both, both
    return z, e


def exponent(top, t):
    """Least e with top <= 448 2^e, within the bounds of the type."""
    top = np.asarray(top, dtype=np.float64)
    m, e = np.frexp(top)  # top = m 2^e, m in [0.5, 1)
    e = np.where(m > 0.875, e - 8, e - 9)
    return np.where(top > 0, e, E_MIN).clip(E_MIN, E_MAX[t])


def quant(x, t):
    """x (.., D) to (code values, exponents); infinities and NaN become NaN."""
    x = np.where(np.isfinite(x), x, np.nan).astype(np.float64)
    with np.errstate(all="ignore"):
        top = np.nan_to_num(np.abs(x), nan=0.0).max(-1)
    e = exponent(top, t)
    y = np.clip(x * np.exp2(-e.astype(np.float64))[..., None], -448, 448)
    return np.where(np.isnan(y), np.nan, e4m3_round(np.nan_to_num(y))), e


def held_bound(y, err, e, t):
    """|error| allowed of a value held with exponent e: half a step of its code,
    and what it was off by before."""
    lim = 448.0 * np.exp2(e.astype(np.float64))[..., None]
    over = np.maximum(np.abs(y) - lim, 0)
    return np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * lim / 448.0) + over + 1.0625 * err


# ---- cache ---------------------------------------------------------------------
def place(k_codes, v_codes, k_scales, v_scales, k, v, ke, ve, slots):
    """Values and exponents of tokens into [P][H][ps][D], [P][H][ps/8][D][8] and
    [P][H][ps]."""
    P, _, ps, _ = k_codes.shape
    for t, s in enumerate(slots):
        if 0 <= s < P * ps:
            p, o = s // ps, s % ps
            k_codes[p, :, o], k_scales[p, :, o] = k[t], ke[t]
            v_codes[p, :, o // 8, :, o % 8], v_scales[p, :, o] = v[t], ve[t]


def tokens_of(k_codes, v_codes, k_scales, v_scales, ids, n):
    """The first n tokens of the pages ids: K and V values (H, n, D), and V's
    exponents (H, n). Codes are values, scales bytes."""
    P, H, ps, D = k_codes.shape
    k, v, ve = np.zeros((H, n, D)), np.zeros((H, n, D)), np.zeros((H, n))
    for j in range(n):
        p, o = ids[j // ps], j % ps
        p = p if 0 <= p < P else 0
        ke = k_scales[p, :, o].astype(np.float64) - 127
        ve[:, j] = v_scales[p, :, o].astype(np.float64) - 127
        k[:, j] = k_codes[p, :, o] * np.exp2(ke)[:, None]
        v[:, j] = v_codes[p, :, o // 8, :, o % 8] * np.exp2(ve[:, j])[:, None]
    return k, v, ve


# ---- attention -----------------------------------------------------------------
def attention(q, cache, pages, lens, prefix_pages, prefix_len, q_start, scale, t):
    """(out, lse, bound of out, bound of lse), all (T, Hq[, D]). cache: code
    values and scale bytes, as for tokens_of.

    Bound, as in serve_oracle.attention: a logit's error S, twice; 2^-21 for exp2
    and the rescalings; the weight's rounding u; the output's rounding u. Beside
    these, E: adding V's exponent rounds the logit (in units of log2) at the size
    of the sum, and so does the difference to the reference, 2^-24 of each and of
    the reference's own. Small weights w = p 2^e are lost, each times a code of at
    most 448: the largest is held at 2^6 or more in fp16 (2^14, and a reference up
    to 2^8 above it), whose steps end at 2^-24, so that a weight is off by 2^-25 /
    2^6 = 2^-31 of the largest; at 2^-8 or more in bf16, where exp2 ends at the
    least normal number, 2^-126, so that 2^-118 of the largest vanishes. In fp16 a
    value of V below 2^-14 may enter in steps of 2^-24, off by 2^-25, and so their
    mean."""
    T, Hq, D = q.shape
    Hkv = cache[0].shape[1]
    G = Hq // Hkv
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    bo, bl = np.full((T, Hq, D), TINY[t]), np.zeros((T, Hq))
    pk, pv, pe = tokens_of(*cache, prefix_pages, prefix_len)
    pk = to_type(pk, t)
    for b in range(len(lens)):
        sk, sv, se = tokens_of(*cache, pages[b], lens[b])
        sk = to_type(sk, t)
        n = q_start[b + 1] - q_start[b]
        for i in range(n):
            seen = max(0, lens[b] - n + i + 1)
            k = np.concatenate((pk, sk[:, :seen]), 1)
            v = np.concatenate((pv, sv[:, :seen]), 1)
            e = np.concatenate((pe, se[:, :seen]), 1)
            if k.shape[1] == 0:
                continue
            for h in range(Hq):
                r, hk = q_start[b] + i, h // G
                z = scale * (k[hk] @ q[r, h])
                S = abs(scale) * (np.abs(k[hk]) @ np.abs(q[r, h])).max() * (D + 2) * 2.0 ** -23
                y = z / np.log(2) + e[hk]
                E = 2.0 ** -23 * (2 * np.abs(y).max() + 64)
                m = z.max()
                p = np.exp(z - m)
                total = p.sum()
                out[r, h] = p @ v[hk] / total
                lse[r, h] = m + np.log(total)
                a = p @ np.abs(v[hk]) / total
                bo[r, h] += (2 * S + 2 * E + 2.0 ** -21 + U[t]) * a + U[t] * np.abs(out[r, h])
                w = np.exp2(y - y.max())
                lost = 2.0 ** -31 if t == "f16" else 2.0 ** -118
                if t == "f16":
                    bo[r, h] += 2.0 ** -25
                bo[r, h] += len(z) * lost * 448 * np.exp2(y.max() - m / np.log(2)) / total
                S = S + E
                bl[r, h] = S + 2.0 ** -20 + 2.0 ** -22 * abs(lse[r, h]) + len(z) * 2.0 ** -118 / w.sum()
    return out, lse, bo, bl


# ---- microscaled 4-bit floats ----------------------------------------------------
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1 = np.concatenate((E2M1, -E2M1))


def mx_quant(x):
    """x (M, K) -> (codes (M, K) 0..15, scale bytes (M, K / 32))."""
    x = np.asarray(x, dtype=np.float64)
    M, K = x.shape
    g = x.reshape(M, K // 32, 32)
    odd = ~np.isfinite(g).all(-1)
    g = np.where(odd[..., None], 0.0, g)
    _, e = np.frexp(np.abs(g).max(-1))  # largest in [2^(e-1), 2^e)
    e = np.where(np.abs(g).max(-1) > 0, e - 3, -127).clip(min=-127)
    a = np.abs(g) * np.exp2(-e.astype(np.float64))[..., None]
    mag = E2M1[:8]
    mid = (mag[1:] + mag[:-1]) / 2
    lo = (a[..., None] > mid).sum(-1)  # ties go to the even code
    hi = (a[..., None] >= mid).sum(-1)
    c = np.where(lo % 2 == 0, lo, hi)
    c = c + 8 * np.signbit(g)
    return c.reshape(M, K).astype(np.uint8), np.where(odd, 255, e + 127).astype(np.uint8)


def mx_pack(c):
    return (c[:, 0::2] | c[:, 1::2] << 4).astype(np.uint8)


def mx_values(c, s):
    """Values (M, K) of codes and scale bytes."""
    v = E2M1[c] * np.exp2(s.astype(np.float64) - 127).repeat(32, 1)
    return np.where(s.repeat(32, 1) == 255, np.nan, v)
