"""serve8_oracle.attention for many rows: the same formula and bounds in 64 bits
by products of whole matrices (torch, on any device). Checked against it in
test_serve8_dense_cpu.py."""
import numpy as np
import torch

from serve8_oracle import TINY, U, to_type


def tokens_of(cache, ids, n):
    """serve8_oracle.tokens_of in one step."""
    k_codes, v_codes, k_scales, v_scales = cache
    P, _, ps, _ = k_codes.shape
    j = np.arange(n)
    p, o = np.asarray(ids, dtype=np.int64)[j // ps] if n else j, j % ps
    p = np.where((p >= 0) & (p < P), p, 0)
    k, v = k_codes[p, :, o], v_codes[p, :, o // 8, :, o % 8]  # (n, H, D)
    ke, ve = (s[p, :, o].astype(np.float64) - 127 for s in (k_scales, v_scales))
    return (k * np.exp2(ke)[..., None]).transpose(1, 0, 2), (v * np.exp2(ve)[..., None]).transpose(1, 0, 2), ve.T


def attention(q, cache, pages, lens, prefix_pages, prefix_len, q_start, scale, t, device="cpu"):
    T, Hq, D = q.shape
    Hkv = cache[0].shape[1]
    G = Hq // Hkv
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)  # noqa: E731
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    bo, bl = np.full((T, Hq, D), TINY[t]), np.zeros((T, Hq))
    pre = tokens_of(cache, prefix_pages, prefix_len)
    for b in range(len(lens)):
        r0, n = int(q_start[b]), int(q_start[b + 1] - q_start[b])
        if n == 0 or prefix_len + lens[b] == 0:
            continue
        k, v, e = (np.concatenate(x, 1) for x in zip(pre, tokens_of(cache, pages[b], lens[b])))
        k = to_type(k, t)
        tok = torch.arange(n, device=device).repeat_interleave(G)
        key = torch.arange(k.shape[1], device=device)
        hidden = key[None] >= prefix_len + (lens[b] - n + 1 + tok).clamp(min=0)[:, None]
        seen = (~hidden).sum(-1).double()
        some = seen > 0
        for h in range(Hkv):
            Q = up(q[r0:r0 + n, h * G:(h + 1) * G].reshape(n * G, D))
            K, V, ev = up(k[h]), up(v[h]), up(e[h])
            kt = K.t().contiguous()
            z = scale * (Q @ kt)
            S = (abs(scale) * (Q.abs() @ kt.abs())).masked_fill(hidden, 0).amax(-1) * (D + 2) * 2.0 ** -23
            y = (z / np.log(2) + ev).masked_fill(hidden, -torch.inf)
            top = y.amax(-1)
            E = 2.0 ** -23 * (2 * y.abs().masked_fill(hidden, 0).amax(-1) + 64)
            w = torch.exp2(y - top[:, None]).sum(-1)
            z = z.masked_fill(hidden, -torch.inf)
            m = z.amax(-1)
            p = torch.exp(z - m[:, None])
            total = p.sum(-1)
            o, l = p @ V / total[:, None], m + torch.log(total)
            a = p @ V.abs() / total[:, None]
            of = (2 * S + 2 * E + 2.0 ** -21 + U[t])[:, None] * a + U[t] * o.abs()
            lost = 2.0 ** -31 if t == "f16" else 2.0 ** -118
            of += (seen * lost * 448 * torch.exp2(top - m / np.log(2)) / total)[:, None]
            if t == "f16":
                of += 2.0 ** -25
            lf = S + E + 2.0 ** -20 + 2.0 ** -22 * l.abs() + seen * 2.0 ** -118 / w
            at = (slice(r0, r0 + n), slice(h * G, (h + 1) * G))
            none = ~some
            for dst, x, empty in ((out, o, 0.0), (lse, l, -np.inf)):
                x[none] = empty
                dst[at] = x.cpu().numpy().reshape(dst[at].shape)
            for dst, x in ((bo, of), (bl, lf)):
                x[none] = 0.0
                dst[at] += x.cpu().numpy().reshape(dst[at].shape)
    return out, lse, bo, bl
