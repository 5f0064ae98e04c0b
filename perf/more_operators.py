"""Timing cases of the serving operators in fewer bits: norms and rotation of
queries and keys with the append to a 16-bit or 8-bit paged cache, reading the
8-bit cache back, attention over it, and microscaled 4-bit products with the
quantization of their activations.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits) or, with ``own`` set, through the library's entry points; ``exact``
computes it in 64 bits from its definition. What is held in 8 bits goes to
``exact`` before its rounding, as 16-bit outputs do.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda:0"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn
E8 = torch.float8_e8m0fnu
F8_MAX = 448.0
E_MIN, E_MAX = -60, {"f16": 7, "bf16": 60}  # exponents of the 8-bit cache's scales
EPS = 1e-6


# ---- cases ------------------------------------------------------------------
def listed():
    return [
        # one token of one conversation enters its 8-bit cache: launch latency
        {"name": "append_1", "op": "append", "tokens": 1, "hq": 32, "hkv": 8, "d": 128, "page": 16,
         "pages": 64, "rot": 128, "inter": False, "run": "decode", "in": "f16", "type": "f16",
         "bits": 8, "norm": True},
        # a decode step of a 203-sequence batch straight from the fp32 GEMVs into a
        # 16-bit cache, some slots padded; adjacent pairs over part of the head
        {"name": "append_203", "op": "append", "tokens": 203, "hq": 40, "hkv": 8, "d": 128,
         "page": 32, "pages": 512, "rot": 64, "inter": True, "run": "decode", "in": "f32",
         "type": "f16", "bits": 16, "norm": True},
        # a long prompt's prefill into an 8-bit cache, starting inside a page
        {"name": "append_16381", "op": "append", "tokens": 16381, "hq": 64, "hkv": 8, "d": 128,
         "page": 64, "pages": 320, "rot": 128, "inter": False, "run": "prefill", "in": "bf16",
         "type": "bf16", "bits": 8, "norm": True},
        # one short conversation leaves the cache: latency
        {"name": "read_1x611", "op": "read", "batch": 1, "hkv": 8, "d": 128, "page": 16, "len": 611,
         "type": "f16"},
        # a batch of conversations of all lengths is handed on
        {"name": "read_24x8209", "op": "read", "batch": 24, "hkv": 8, "d": 128, "page": 64,
         "len": 8209, "type": "bf16"},
        # two conversations, short caches, no shared prefix: latency
        {"name": "attn_2x97", "op": "attn", "batch": 2, "hq": 32, "hkv": 8, "d": 128, "page": 16,
         "prefix": 0, "suffix": 97, "new": 1, "ragged": False, "type": "f16"},
        # ordinary paged decode over long caches, ragged lengths and padded
        # (empty) batch entries
        {"name": "attn_24x8209", "op": "attn", "batch": 24, "hq": 32, "hkv": 8, "d": 128,
         "page": 32, "prefix": 0, "suffix": 8209, "new": 1, "ragged": True, "type": "f16"},
        # many conversations behind one long system prompt
        {"name": "attn_96x32801", "op": "attn", "batch": 96, "hq": 64, "hkv": 8, "d": 128,
         "page": 64, "prefix": 32801, "suffix": 701, "new": 1, "ragged": True, "type": "bf16"},
        # chunks of new prompts behind a shared document, 64-wide heads
        {"name": "attn_6x8200_new", "op": "attn", "batch": 6, "hq": 32, "hkv": 4, "d": 64,
         "page": 16, "prefix": 8200, "suffix": 531, "new": 301, "ragged": True, "type": "f16"},
        # one token through a large feed-forward weight: quantized, then multiplied
        {"name": "mx_1x28672x8192", "op": "mx", "m": 1, "n": 28672, "k": 8192, "type": "f16"},
        # a decode batch through an odd-sized projection
        {"name": "mx_45x4127x4128", "op": "mx", "m": 45, "n": 4127, "k": 4128, "type": "f32"},
        # prefill through a feed-forward weight
        {"name": "mx_4096x14336x4096", "op": "mx", "m": 4096, "n": 14336, "k": 4096,
         "type": "bf16"},
    ]


def _log_int(rng, lo, hi):
    """Spread over the logarithm; odd above 500."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n | 1 if n > 500 else n


def draw(rng: random.Random):
    op = rng.choice(["append", "append", "read", "attn", "attn", "mx", "mx"])
    t16 = rng.choice(["f16", "bf16"])
    if op == "append":
        hkv = rng.choice([1, 2, 4, 8, 32])
        hq = hkv * rng.choice([1, 2, 4, 7, 8]) if hkv < 32 else 32
        d = rng.choice([64, 96, 128, 256])
        page = rng.choice([8, 16, 32, 64, 128])
        tokens = min(_log_int(rng, 1, 12000), 16381 * 64 * 128 // ((hq + 2 * hkv) * d))
        pages = -(-tokens // page) + rng.randint(1, 40) + (256 if tokens < 512 else 0)
        return {"op": op, "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "page": page,
                "pages": pages, "rot": rng.choice([d, d, d // 2]), "inter": rng.random() < 0.5,
                "run": "prefill" if tokens >= 512 else "decode",
                "in": rng.choice(["f32", t16]), "type": t16, "bits": rng.choice([8, 8, 16]),
                "norm": rng.random() < 0.7}
    if op == "read":
        batch, length = _log_int(rng, 1, 64), _log_int(rng, 1, 8000)
        hkv, d = rng.choice([1, 2, 4, 8, 32]), rng.choice([64, 96, 128, 256])
        while batch * length * hkv * d > 24 * 8209 * 8 * 128:
            batch, length = max(1, batch // 2), length if batch > 1 else length // 2
        return {"op": op, "batch": batch, "hkv": hkv, "d": d,
                "page": rng.choice([8, 16, 32, 64, 128]), "len": length,
                "type": rng.choice([t16, t16, "f32"])}
    if op == "attn":
        hkv = rng.choice([1, 2, 4, 8, 8])
        hq = hkv * rng.choice([1, 2, 4, 7, 8])
        d = rng.choice([64, 96, 128, 128, 256])
        new = rng.choice([1, 1, 1, 4, _log_int(rng, 2, 256)])
        batch = max(1, min(_log_int(rng, 1, 96), 2048 // new))
        prefix = rng.choice([0, _log_int(rng, 1, 16000)])
        suffix = new + _log_int(rng, 1, 8000)
        # no more work than the largest listed cases
        while batch * new * hq * d * (prefix + suffix) > 2.0e11 and batch > 1:
            batch = batch // 2
        return {"op": op, "batch": batch, "hq": hq, "hkv": hkv, "d": d,
                "page": rng.choice([8, 16, 32, 64, 128]), "prefix": prefix, "suffix": suffix,
                "new": new, "ragged": rng.random() < 0.7, "type": t16}
    n = rng.choice([1024, 4096, 12288, rng.randint(100, 7000) * 2 + 1])
    k = rng.choice([1024, 2048, 4096, 32 * (2 * rng.randint(4, 63) + 1)])
    return {"op": op, "m": _log_int(rng, 1, 4000), "n": n, "k": k,
            "type": rng.choice(["f16", "bf16", "f32"])}


# ---- inputs -----------------------------------------------------------------
def _turns(rot, base=10000.0):
    """inv_freq / 2 pi as 64-bit fractions of a turn (two's complement in int64)."""
    f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot) / (2 * math.pi)
    v = [int(round(float(x) * 2.0 ** 64)) % 2 ** 64 for x in f]
    return np.array([x - 2 ** 64 if x >= 2 ** 63 else x for x in v], dtype=np.int64)


def _up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _codes8(shape, g):
    """e4m3 codes as a cache holds them: most of the range used, no NaN."""
    x = torch.randn(shape, device=DEV, generator=g, dtype=torch.float16)
    return x.mul_(F8_MAX / 4).clamp_(-F8_MAX, F8_MAX).to(F8)


def _scales8(shape, g):
    """Scales near 2^-7 that differ from token to token."""
    e = torch.randint(-8, -5, shape, device=DEV, generator=g)
    return (e + 127).to(torch.uint8).view(E8)


def _cache(P, hkv, ps, d, g):
    return {"k_cache": _codes8((P, hkv, ps, d), g), "v_cache": _codes8((P, hkv, ps // 8, d, 8), g),
            "k_scales": _scales8((P, hkv, ps), g), "v_scales": _scales8((P, hkv, ps), g)}


def _prepare_append(case, seed, g):
    T, hq, hkv, d, ps, P = (case[k] for k in ("tokens", "hq", "hkv", "d", "page", "pages"))
    r = np.random.default_rng(seed)
    it, ct = TYPES[case["in"]], TYPES[case["type"]]
    # q, k and v are slices of one projection's rows
    qkv = torch.randn(T, hq + 2 * hkv, d, device=DEV, generator=g).to(it)
    if case["run"] == "prefill":  # one sequence, consecutive, pages in any order
        first = int(r.integers(0, ps))
        tok = np.arange(T) + first
        order = r.permutation(P)[: -(-(T + first) // ps)]
        slots = order[tok // ps].astype(np.int64) * ps + tok % ps
        pos = tok + int(r.integers(0, 30000))
    else:  # one token of each of T sequences
        slots = r.permutation(P * ps)[:T].astype(np.int64)
        slots[np.arange(T) % 16 == 9] = -1
        pos = r.integers(0, 120000, T)
    weight = lambda: 1 + 0.2 * torch.randn(d, device=DEV, generator=g)  # noqa: E731
    s = {"case": case, "q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "v": qkv[:, hq + hkv:],
         "pos": _up(pos.astype(np.int32)), "slots": _up(slots), "turns": _up(_turns(case["rot"])),
         "q_norm": weight() if case["norm"] else None, "k_norm": weight() if case["norm"] else None,
         "q_out": torch.empty(T, hq, d, device=DEV, dtype=ct)}
    if case["bits"] == 8:
        return s | _cache(P, hkv, ps, d, g)
    return s | {"k_cache": torch.randn(P, hkv, ps, d, device=DEV, generator=g).to(ct),
                "v_cache": torch.randn(P, hkv, ps // 8, d, 8, device=DEV, generator=g).to(ct)}


def _read_lens(case):
    """Lengths of the conversations that are read: one full, the others spread."""
    return [max(1, round(case["len"] * (1.0 if b == 0 else (b * 0.6180339887) % 1.0)))
            for b in range(case["batch"])]


def _prepare_read(case, seed, g):
    B, hkv, d, ps = (case[k] for k in ("batch", "hkv", "d", "page"))
    r = np.random.default_rng(seed)
    lens = np.array(_read_lens(case))[r.permutation(B)]
    mp = -(-int(lens.max()) // ps)
    P = int((-(-lens // ps)).sum()) + 7
    ids = r.permutation(P).astype(np.int32)
    table = np.zeros((B, mp), dtype=np.int32)
    at = 0
    for b in range(B):
        n = -(-int(lens[b]) // ps)
        table[b, :n] = ids[at:at + n]
        at += n
    start = np.concatenate([[0], np.cumsum(lens)])
    row = np.repeat(np.arange(B), lens)
    return {"case": case, "pages": _up(table), "start": _up(start.astype(np.int32)),
            "tokens": int(start[-1]), "seq": _up(row), "tok": _up(np.arange(start[-1]) - start[row]),
            **_cache(P, hkv, ps, d, g)}


def _lens(case):
    """Cache and new-token counts of each sequence, the same for every seed:
    spread over (0, suffix], one at the full length, every ninth entry of a
    ragged batch of one-token steps padded (empty)."""
    n, lens, news = case["batch"], [], []
    for b in range(n):
        u = 1.0 if b == 0 or not case["ragged"] else (b * 0.6180339887) % 1.0
        new = max(1, int(round(case["new"] * (0.5 + 0.5 * u))))
        s = new + int((case["suffix"] - new) * u)
        if case["ragged"] and case["new"] == 1 and b % 9 == 5:
            s = 0
        lens.append(s)
        news.append(new)
    return lens, news


def _prepare_attn(case, seed, g):
    B, hq, hkv, d, ps = (case[k] for k in ("batch", "hq", "hkv", "d", "page"))
    r = np.random.default_rng(seed)
    lens, news = _lens(case)
    order = r.permutation(B)
    lens, news = np.array(lens)[order], np.array(news)[order]
    mp = max(1, -(-int(lens.max()) // ps))
    pp = -(-case["prefix"] // ps)
    P = int((-(-lens // ps)).sum()) + pp + 7
    ids = r.permutation(P).astype(np.int32)
    table = np.zeros((B, mp), dtype=np.int32)
    at = pp
    for b in range(B):
        n = -(-int(lens[b]) // ps)
        table[b, :n] = ids[at:at + n]
        at += n
    start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    T = int(start[-1])
    q = (1.5 * torch.randn(T, hq, d, device=DEV, generator=g)).to(TYPES[case["type"]])
    row = np.repeat(np.arange(B), news)
    return {"case": case, "q": q, "pages": _up(table), "lens": _up(lens.astype(np.int32)),
            "prefix_pages": _up(ids[:pp]) if pp else None,
            "start": _up(start) if case["new"] > 1 else None,
            # the host's view of the same batch
            "seq": _up(row), "tok": _up(np.arange(T) - start[row]), "news": _up(news),
            "most": int(news.max()), "rows": int(lens.max()), **_cache(P, hkv, ps, d, g)}


def _prepare_mx(case, seed, g):
    m, n, k = case["m"], case["n"], case["k"]
    # a weight's codes (low nibble first) follow a bell curve; scales differ by block
    x = torch.randn(n, k, device=DEV, generator=g, dtype=torch.float16).mul_(1.8)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV, dtype=torch.float16)
    c = torch.bucketize(x.abs(), edges, out_int32=True).to(torch.uint8)
    c.add_(x.lt(0), alpha=8)
    e = torch.randint(-1, 2, (n, k // 32), device=DEV, generator=g) - round(math.log2(k) / 2)
    a = torch.randn(m, k, device=DEV, generator=g)
    # a few channels are far larger than the others, as in trained models
    a *= torch.exp(0.8 * torch.randn(k, device=DEV, generator=g))
    return {"case": case, "x": a.to(TYPES[case["type"]]), "w": c[:, 0::2] + 16 * c[:, 1::2],
            "ws": (e + 127).to(torch.uint8).view(E8)}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return {"append": _prepare_append, "read": _prepare_read, "attn": _prepare_attn,
            "mx": _prepare_mx}[case["op"]](case, int(seed), g)


# ---- plain forms ------------------------------------------------------------
def _rotate(x, c, s, rot, inter):
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _norm(x, w):
    x = x.float()
    return x if w is None else x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def _quant8(x, t):
    """x (.., D) to e4m3 codes and the exponent of their scale."""
    m, e = torch.frexp(x.abs().amax(-1))  # m 2^e, m in [0.5, 1): 448 is 0.875 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(m > 0, e, E_MIN).clamp(E_MIN, E_MAX[t])
    return torch.ldexp(x, -e[..., None]).clamp(-F8_MAX, F8_MAX).to(F8), e


def _plain_append(s):
    case = s["case"]
    ps, t = case["page"], case["type"]
    phase = s["pos"].long()[:, None] * s["turns"][None]  # wraps: whole turns drop out
    angle = (phase >> 32).float() * (2 * math.pi / 2.0 ** 32)
    c, n = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    s["q_out"].copy_(_rotate(_norm(s["q"], s["q_norm"]), c, n, case["rot"], case["inter"]))
    keep = s["slots"] >= 0
    slot = s["slots"][keep]
    k = _rotate(_norm(s["k"], s["k_norm"]), c, n, case["rot"], case["inter"])[keep]
    v = s["v"][keep]
    page, off = slot // ps, slot % ps
    if case["bits"] == 16:
        s["k_cache"][page, :, off] = k.to(TYPES[t])
        s["v_cache"][page, :, off // 8, :, off % 8] = v.to(TYPES[t])
        return s["q_out"], s["k_cache"], s["v_cache"]
    (k, ke), (v, ve) = _quant8(k, t), _quant8(v.float(), t)
    u8 = torch.uint8
    s["k_cache"].view(u8)[page, :, off] = k.view(u8)
    s["v_cache"].view(u8)[page, :, off // 8, :, off % 8] = v.view(u8)
    s["k_scales"].view(u8)[page, :, off] = (ke + 127).to(u8)
    s["v_scales"].view(u8)[page, :, off] = (ve + 127).to(u8)
    return s["q_out"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]


def _gather(s, name, ids):
    """Keys ("k") or values ("v") of pages of any shape: (shape, Hkv, tokens, D)
    in 32 bits."""
    ids = ids.long()
    x = s[name + "_cache"].view(torch.uint8)[ids].view(F8).float()
    if name == "v":  # [.., Hkv, ps/8, D, 8] -> [.., Hkv, ps, D]
        x = x.transpose(-1, -2).flatten(-3, -2)
    e = s[name + "_scales"].view(torch.uint8)[ids].int() - 127
    return torch.ldexp(x, e[..., None])


def _plain_read(s):
    case = s["case"]
    ps = case["page"]
    page = s["pages"][s["seq"], s["tok"] // ps].long()
    off = s["tok"] % ps
    u8 = torch.uint8
    k = s["k_cache"].view(u8)[page, :, off].view(F8).float()
    v = s["v_cache"].view(u8)[page, :, off // 8, :, off % 8].view(F8).float()
    ke = s["k_scales"].view(u8)[page, :, off].int() - 127
    ve = s["v_scales"].view(u8)[page, :, off].int() - 127
    t = TYPES[case["type"]]
    return torch.ldexp(k, ke[..., None]).to(t), torch.ldexp(v, ve[..., None]).to(t)


def _plain_attn(s):
    case = s["case"]
    B, hq, hkv, d, ps = (case[k] for k in ("batch", "hq", "hkv", "d", "page"))
    G, L, N = hq // hkv, case["prefix"], s["most"]
    q = torch.zeros(B, N, hq, d, device=DEV)
    q[s["seq"], s["tok"]] = s["q"].float()
    q = q.view(B, N, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, N * G, d) / math.sqrt(d)
    mp = s["pages"].shape[1]
    # each sequence's own keys: [B, hkv, mp * ps, d]
    k = _gather(s, "k", s["pages"]).transpose(1, 2).flatten(2, 3)
    v = _gather(s, "v", s["pages"]).transpose(1, 2).flatten(2, 3)
    z = torch.matmul(q, k.transpose(-1, -2))
    key = torch.arange(mp * ps, device=DEV)
    tok = torch.arange(N, device=DEV)
    seen = key[None, None] <= (s["lens"] - s["news"])[:, None, None] + tok[None, :, None]
    seen = seen & (key < s["lens"][:, None, None])
    z = z.view(B, hkv, N, G, -1).masked_fill(~seen[:, None, :, None], -math.inf).flatten(2, 3)
    m = z.amax(-1)
    if L:
        kp = _gather(s, "k", s["prefix_pages"]).transpose(0, 1).flatten(1, 2)[:, :L]
        vp = _gather(s, "v", s["prefix_pages"]).transpose(0, 1).flatten(1, 2)[:, :L]
        qp = q.transpose(0, 1).reshape(hkv, B * N * G, d)
        zp = torch.matmul(qp, kp.transpose(-1, -2))
        m = torch.maximum(m, zp.amax(-1).view(hkv, B, N * G).transpose(0, 1))
    low = m.masked_fill(m == -math.inf, 0.0)[..., None]
    p = torch.exp(z - low)
    total, o = p.sum(-1), torch.matmul(p, v)
    if L:
        pp = torch.exp(zp - low.transpose(0, 1).reshape(hkv, B * N * G, 1))
        total = total + pp.sum(-1).view(hkv, B, N * G).transpose(0, 1)
        o = o + torch.matmul(pp, vp).view(hkv, B, N * G, d).transpose(0, 1)
    o = o / total.clamp_min(1e-37)[..., None]
    lse = torch.log(total) + low[..., 0]
    back = lambda x: x.view(B, hkv, N, G, -1).permute(0, 2, 1, 3, 4).reshape(B, N, hq, -1)[s["seq"], s["tok"]]  # noqa: E731
    return back(o).to(TYPES[case["type"]]), back(lse)[..., 0].contiguous()


E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _plain_mx(s):
    m, k = s["x"].shape
    x = s["x"].float().view(m, k // 32, 32)
    _, e = torch.frexp(x.abs().amax(-1, keepdim=True))  # the largest is in [2^(e-1), 2^e)
    e = (e - 3).clamp(min=-127)
    a = torch.ldexp(x, -e)
    # steps of 0.5 below 2, of 1 below 4, of 2 up to 6
    step = torch.where(a.abs() < 2, 0.5, torch.where(a.abs() < 4, 1.0, 2.0))
    a = torch.ldexp((torch.round(a / step) * step).clamp(-6, 6), e).view(m, k)
    table = torch.tensor(E2M1 + [-v for v in E2M1], device=DEV)
    w = torch.stack((table[(s["w"] & 15).int()], table[(s["w"] >> 4).int()]), -1)
    n = w.shape[0]
    we = s["ws"].view(torch.uint8).int() - 127
    w = torch.ldexp(w.view(n, k // 32, 32), we[..., None]).view(n, k)
    return torch.matmul(a, w.t()).to(TYPES[s["case"]["type"]])


# ---- the library's entry points ---------------------------------------------
def _own(s):
    import block_quantized_matmul_amd as bq
    case = s["case"]
    if case["op"] == "append":
        held = case["bits"] == 8
        bq.lqmm_kv_append_norm(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["k_cache"],
                               s["v_cache"], k_scales=s["k_scales"] if held else None,
                               v_scales=s["v_scales"] if held else None, q_norm=s["q_norm"],
                               k_norm=s["k_norm"], eps=EPS, rope_turns=s["turns"],
                               interleaved=case["inter"], q_out=s["q_out"])
        return (s["q_out"], s["k_cache"], s["v_cache"]) + (
            (s["k_scales"], s["v_scales"]) if held else ())
    if case["op"] == "read":
        return bq.lqmm_kv_read_f8(s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                                  s["pages"], s["start"], s["tokens"], dtype=TYPES[case["type"]])
    if case["op"] == "attn":
        return bq.lqmm_attn_prefix_f8(s["q"], s["k_cache"], s["v_cache"], s["k_scales"],
                                      s["v_scales"], s["pages"], s["lens"],
                                      prefix_pages=s["prefix_pages"], prefix_len=case["prefix"],
                                      q_start=s["start"], max_q=s["most"], return_lse=True)
    codes, scales = bq.lqmm_quant_mxfp4(s["x"])
    return bq.lqmm_gemm_mxfp4(s["w"], s["ws"], codes, scales, out_dtype=TYPES[case["type"]])


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "read": _plain_read, "attn": _plain_attn,
            "mx": _plain_mx}[state["case"]["op"]](state)


# ---- 64 bits ----------------------------------------------------------------
def _two(scales):
    """Values of e8m0 scales in 64 bits."""
    return torch.exp2(scales.view(torch.uint8).double() - 127)


def _exact_append(s):
    case = s["case"]
    rot, ps, half, t = case["rot"], case["page"], case["rot"] // 2, case["type"]
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    ang = s["pos"].double()[:, None] * freq[None]
    unit = torch.polar(torch.ones_like(ang), ang)[:, None]

    def turn(x, w):
        y = x.double().clone()
        if w is not None:
            y = y * torch.rsqrt((y * y).sum(-1, keepdim=True) / case["d"] + EPS) * w.double()
        if case["inter"]:
            z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], half, 2).contiguous()) * unit
            y[..., :rot] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :half], y[..., half:rot]) * unit
            y[..., :half], y[..., half:rot] = z.real, z.imag
        return y

    q, k, v = turn(s["q"], s["q_norm"]), turn(s["k"], s["k_norm"]), s["v"].double()
    at = torch.nonzero(s["slots"] >= 0)[:, 0]
    slot = s["slots"][at]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    scales = []
    if case["bits"] == 8:
        for i, x in enumerate((k, v)):
            top = x.abs().max(-1).values.clamp(min=1e-300)
            sc = torch.exp2(torch.ceil(torch.log2(top / F8_MAX)).clamp(E_MIN, E_MAX[t]))
            x /= sc[..., None]
            all_sc = _two(s["v_scales" if i else "k_scales"])
            for h in range(case["hkv"]):
                all_sc[slot // ps, h, slot % ps] = sc[at, h]
            scales.append(all_sc)
    for h in range(case["hkv"]):
        kc[slot // ps, h, slot % ps] = k[at, h]
        vc[slot // ps, h, (slot % ps) // 8, :, slot % 8] = v[at, h]
    return (q, kc, vc, *scales)


def _dense(s, ids):
    """K and V of a list of pages in 64 bits, (Hkv, tokens, D) each."""
    ids = ids.long()
    u8 = torch.uint8
    P, hkv, ps, d = s["k_cache"].shape
    n = ids.numel() * ps
    ks, vs = (_two(s[x])[ids].transpose(0, 1).reshape(hkv, n, 1) for x in ("k_scales", "v_scales"))
    k = s["k_cache"].view(u8)[ids].view(F8).double().permute(1, 0, 2, 3).reshape(hkv, n, d)
    v = s["v_cache"].view(u8)[ids].view(F8).double().permute(1, 0, 2, 4, 3).reshape(hkv, n, d)
    return k * ks, v * vs


def _exact_read(s):
    ks, vs = [], []
    start = s["start"].tolist()
    for b in range(s["case"]["batch"]):
        k, v = _dense(s, s["pages"][b])
        n = start[b + 1] - start[b]
        ks.append(k[:, :n].transpose(0, 1))
        vs.append(v[:, :n].transpose(0, 1))
    return torch.cat(ks), torch.cat(vs)


def _exact_attn(s):
    case = s["case"]
    hq, hkv, d, L = (case[k] for k in ("hq", "hkv", "d", "prefix"))
    G = hq // hkv
    if L:
        pk, pv = (x[:, :L].contiguous() for x in _dense(s, s["prefix_pages"]))
    lens, news = s["lens"].tolist(), s["news"].tolist()
    outs, lses, t0 = [], [], 0
    for b, (ln, nw) in enumerate(zip(lens, news)):
        k, v = (x[:, :ln] for x in _dense(s, s["pages"][b]))
        if L:
            k, v = torch.cat((pk, k), 1), torch.cat((pv, v), 1)
        kt = k.transpose(1, 2).contiguous()
        # rows in pieces, so that the logits of a long prefix stay small
        for i0 in range(0, nw, 64):
            n = min(64, nw - i0)
            x = s["q"][t0 + i0:t0 + i0 + n].double().view(n, hkv, G, d).transpose(0, 1).reshape(hkv, n * G, d)
            z = torch.matmul(x, kt) / math.sqrt(d)
            if ln:
                last = ln - nw + i0 + torch.arange(n, device=DEV).repeat_interleave(G)
                z[:, :, L:].masked_fill_(torch.arange(ln, device=DEV)[None] > last[:, None], -math.inf)
            if z.shape[-1]:
                lse = torch.logsumexp(z, -1)
                p = torch.exp(z - lse[..., None].masked_fill(torch.isinf(lse)[..., None], 0.0))
                o = torch.matmul(p, v)
            else:
                lse, o = torch.full_like(x[..., 0], -math.inf), torch.zeros_like(x)
            outs.append(o.view(hkv, n, G, d).transpose(0, 1).reshape(n, hq, d))
            lses.append(lse.view(hkv, n, G).transpose(0, 1).reshape(n, hq))
        t0 += nw
    return torch.cat(outs), torch.cat(lses)


def _exact_mx(s):
    (m, k), n = s["x"].shape, s["w"].shape[0]
    grid = torch.tensor(E2M1, device=DEV, dtype=torch.float64)
    between = (grid[1:] + grid[:-1]) / 2  # ties go to the even code
    y = torch.zeros(m, n, device=DEV, dtype=torch.float64)
    for b in range(k // 32):
        x = s["x"][:, 32 * b:32 * b + 32].double()
        sc = torch.exp2((torch.floor(torch.log2(x.abs().max(1).values.clamp(min=1e-300))) - 2).clamp(min=-127))
        a = (x / sc[:, None])
        lo, hi = (torch.bucketize(a.abs(), between, right=right) for right in (False, True))
        a = torch.sign(a) * grid[torch.where(lo % 2 == 0, lo, hi)] * sc[:, None]
        c = s["w"][:, 16 * b:16 * b + 16].long()
        c = torch.stack((c & 15, c >> 4), -1).view(n, 32)
        w = grid[c % 8] * (1 - 2 * (c // 8)) * _two(s["ws"][:, b:b + 1])
        y += torch.matmul(a, w.t().contiguous())
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attn": _exact_attn,
            "mx": _exact_mx}[case["op"]](s)


# ---- bytes and operations ---------------------------------------------------
def work(case):
    size = {"f16": 2, "bf16": 2, "f32": 4}
    e = size[case["type"]]
    if case["op"] == "append":
        T, hq, hkv, d = (case[k] for k in ("tokens", "hq", "hkv", "d"))
        kept = T if case["run"] == "prefill" else sum(t % 16 != 9 for t in range(T))
        held = d + 1 if case["bits"] == 8 else d * e  # bytes of a head's vector in the cache
        return {"bytes": (hq * T + 2 * hkv * kept) * d * size[case["in"]] + hq * T * d * e
                + 2 * hkv * kept * held + T * 12 + case["rot"] * 4 + (8 * d if case["norm"] else 0),
                "flops": T * (hq + hkv) * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    if case["op"] == "read":
        lens = _read_lens(case)
        T, heads, d = sum(lens), case["hkv"], case["d"]
        pages = sum(-(-n // case["page"]) for n in lens)
        return {"bytes": 2 * T * heads * (d + 1 + d * e) + 4 * pages + 4 * (case["batch"] + 1),
                "flops": 2 * T * heads * d}
    if case["op"] == "attn":
        lens, news = _lens(case)
        T, row = sum(news), case["hkv"] * (case["d"] + 1)
        pages = sum(-(-n // case["page"]) for n in [*lens, case["prefix"]])
        pairs = T * case["prefix"]
        for n, w in zip(lens, news):  # token i of a sequence sees n - w + i + 1 keys
            pairs += sum(max(0, n - w + i + 1) for i in range(w))
        return {"bytes": 2 * row * (sum(lens) + case["prefix"]) + T * case["hq"] * (2 * case["d"] * e + 4)
                + 4 * pages + 8 * case["batch"],
                "flops": 4 * pairs * case["hq"] * case["d"]}
    m, n, k = case["m"], case["n"], case["k"]
    return {"bytes": n * k // 2 + n * k // 32 + m * k * e + m * n * e, "flops": 2 * m * n * k}
