"""Timing cases of the serving operators around the block-quantized products:
appending rotated keys and values to a paged cache, attention over that cache
for a batch that shares a prefix, and the 8-bit float product with a scale for
each block of 128 with the quantization of its activations.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits) or, with ``own`` set, through the library's entry points; ``exact``
computes it in 64 bits from its definition.
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
F8_MAX = 448.0
TINY = 2.0 ** -126


# ---- cases ------------------------------------------------------------------
def listed():
    return [
        # one token of one conversation enters its cache: launch latency
        {"name": "append_1", "op": "append", "tokens": 1, "hq": 32, "hkv": 8, "d": 128, "page": 16,
         "pages": 64, "rot": 128, "inter": False, "run": "decode", "in": "f16", "type": "f16"},
        # a decode step of a 200-sequence batch straight from the fp32 GEMVs,
        # some slots padded; rotation of adjacent pairs over part of the head
        {"name": "append_203", "op": "append", "tokens": 203, "hq": 32, "hkv": 32, "d": 128,
         "page": 32, "pages": 512, "rot": 64, "inter": True, "run": "decode", "in": "f32",
         "type": "f16"},
        # a long prompt's prefill, starting inside a page
        {"name": "append_16381", "op": "append", "tokens": 16381, "hq": 64, "hkv": 8, "d": 128,
         "page": 64, "pages": 320, "rot": 128, "inter": False, "run": "prefill", "in": "bf16",
         "type": "bf16"},
        # two conversations, short caches, no shared prefix: latency
        {"name": "attn_2x97", "op": "attn", "batch": 2, "hq": 32, "hkv": 8, "d": 128, "page": 16,
         "prefix": 0, "suffix": 97, "new": 1, "ragged": False, "type": "f16"},
        # ordinary paged decode, one key head per query head, ragged lengths
        # and padded (empty) batch entries
        {"name": "attn_24x4111", "op": "attn", "batch": 24, "hq": 32, "hkv": 32, "d": 128,
         "page": 32, "prefix": 0, "suffix": 4111, "new": 1, "ragged": True, "type": "f16"},
        # many conversations behind one long system prompt
        {"name": "attn_96x32801", "op": "attn", "batch": 96, "hq": 64, "hkv": 8, "d": 128,
         "page": 64, "prefix": 32801, "suffix": 701, "new": 1, "ragged": True, "type": "bf16"},
        # chunks of new prompts behind a shared document, 64-wide heads
        {"name": "attn_6x8200_new", "op": "attn", "batch": 6, "hq": 32, "hkv": 4, "d": 64,
         "page": 16, "prefix": 8200, "suffix": 531, "new": 301, "ragged": True, "type": "f16"},
        # activations of one decode step
        {"name": "quant_3x4096", "op": "quant", "m": 3, "k": 4096, "type": "f16"},
        # activations of a prefill chunk, the last group of a row cut short
        {"name": "quant_4099x11024", "op": "quant", "m": 4099, "k": 11024, "type": "bf16"},
        # one token through a large feed-forward weight
        {"name": "gemm_1x28672x8192", "op": "gemm", "m": 1, "n": 28672, "k": 8192, "type": "f16"},
        # a decode batch through an odd-sized projection
        {"name": "gemm_45x4127x4112", "op": "gemm", "m": 45, "n": 4127, "k": 4112, "type": "f32"},
        # prefill through a feed-forward weight
        {"name": "gemm_4096x14336x4096", "op": "gemm", "m": 4096, "n": 14336, "k": 4096,
         "type": "bf16"},
    ]


def _log_int(rng, lo, hi):
    """Spread over the logarithm; odd above 500."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n | 1 if n > 500 else n


def draw(rng: random.Random):
    op = rng.choice(["append", "attn", "attn", "quant", "gemm", "gemm"])
    t16 = rng.choice(["f16", "bf16"])
    if op == "append":
        hkv = rng.choice([1, 2, 4, 8, 32])
        hq = hkv * rng.choice([1, 2, 4, 7, 8]) if hkv < 32 else 32
        d = rng.choice([64, 128, 256])
        page = rng.choice([8, 16, 32, 64, 128])
        tokens = min(_log_int(rng, 1, 12000), 16381 * 64 * 128 // ((hq + 2 * hkv) * d))
        pages = -(-tokens // page) + rng.randint(1, 40) + (256 if tokens < 512 else 0)
        return {"op": op, "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "page": page,
                "pages": pages, "rot": rng.choice([d, d, d // 2]), "inter": rng.random() < 0.5,
                "run": "prefill" if tokens >= 512 else "decode",
                "in": rng.choice(["f32", t16]), "type": t16}
    if op == "attn":
        hkv = rng.choice([1, 2, 4, 8, 8])
        hq = hkv * rng.choice([1, 2, 4, 7, 8])
        d = rng.choice([64, 128, 128, 256])
        new = rng.choice([1, 1, 1, 4, _log_int(rng, 2, 256)])
        batch = max(1, min(_log_int(rng, 1, 96), 2048 // new))
        prefix = rng.choice([0, _log_int(rng, 1, 16000)])
        suffix = new + _log_int(rng, 1, 4000)
        # no more work than the largest listed cases
        while batch * new * hq * d * (prefix + suffix) > 2.0e11 and batch > 1:
            batch = batch // 2
        return {"op": op, "batch": batch, "hq": hq, "hkv": hkv, "d": d,
                "page": rng.choice([8, 16, 32, 64, 128]), "prefix": prefix, "suffix": suffix,
                "new": new, "ragged": rng.random() < 0.7, "type": t16}
    if op == "quant":
        return {"op": op, "m": _log_int(rng, 1, 4000),
                "k": rng.choice([1024, 4096, 8192, 16 * (2 * rng.randint(4, 340) + 1)]),
                "type": rng.choice(["f32", t16])}
    n = rng.choice([1024, 4096, 12288, rng.randint(100, 7000) * 2 + 1])
    k = rng.choice([1024, 2048, 4096, 16 * (2 * rng.randint(8, 127) + 1)])
    return {"op": op, "m": _log_int(rng, 1, 4000), "n": n, "k": k,
            "type": rng.choice(["f16", "bf16", "f32"])}


# ---- inputs -----------------------------------------------------------------
def _turns(rot, base=10000.0):
    """inv_freq / 2 pi as 64-bit fractions of a turn (two's complement in int64)."""
    f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot) / (2 * math.pi)
    v = [int(round(float(x) * 2.0 ** 64)) % 2 ** 64 for x in f]
    return np.array([x - 2 ** 64 if x >= 2 ** 63 else x for x in v], dtype=np.int64)


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
    return {"case": case, "q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "v": qkv[:, hq + hkv:],
            "pos": torch.from_numpy(pos.astype(np.int32)).to(DEV),
            "slots": torch.from_numpy(slots).to(DEV),
            "turns": torch.from_numpy(_turns(case["rot"])).to(DEV),
            "k_cache": torch.randn(P, hkv, ps, d, device=DEV, generator=g).to(ct),
            "v_cache": torch.randn(P, hkv, ps // 8, d, 8, device=DEV, generator=g).to(ct),
            "q_out": torch.empty(T, hq, d, device=DEV, dtype=ct)}


def _prepare_attn(case, seed, g):
    B, hq, hkv, d, ps = (case[k] for k in ("batch", "hq", "hkv", "d", "page"))
    t = TYPES[case["type"]]
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
    k = torch.randn(P, hkv, ps, d, device=DEV, generator=g, dtype=torch.float32).to(t)
    v = torch.randn(P, hkv, ps // 8, d, 8, device=DEV, generator=g, dtype=torch.float32).to(t)
    q = (1.5 * torch.randn(T, hq, d, device=DEV, generator=g)).to(t)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    row = np.repeat(np.arange(B), news)
    return {"case": case, "q": q, "k_cache": k, "v_cache": v, "pages": up(table),
            "lens": up(lens.astype(np.int32)), "prefix_pages": up(ids[:pp]) if pp else None,
            "start": up(start) if case["new"] > 1 else None,
            # the host's view of the same batch
            "seq": up(row), "tok": up(np.arange(T) - start[row]), "news": up(news),
            "most": int(news.max()), "rows": int(lens.max())}


def _prepare_quant(case, seed, g):
    x = torch.randn(case["m"], case["k"], device=DEV, generator=g)
    # a few channels are far larger than the others, as in trained models
    x *= torch.exp(1.2 * torch.randn(case["k"], device=DEV, generator=g))
    return {"case": case, "x": x.to(TYPES[case["type"]])}


def _codes(rows, cols, g):
    x = torch.randn(rows, cols, device=DEV, generator=g)
    return x.mul_(F8_MAX / 4).clamp_(-F8_MAX, F8_MAX).to(F8)


def _prepare_gemm(case, seed, g):
    m, n, k = case["m"], case["n"], case["k"]
    kb, nb = -(-k // 128), -(-n // 128)
    return {"case": case, "w": _codes(n, k, g), "x": _codes(m, k, g),
            "ws": torch.exp(0.3 * torch.randn(nb, kb, device=DEV, generator=g)) * (4 / F8_MAX / math.sqrt(k)),
            "xs": torch.exp(0.5 * torch.randn(kb, m, device=DEV, generator=g)) * (4 / F8_MAX)}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return {"append": _prepare_append, "attn": _prepare_attn, "quant": _prepare_quant,
            "gemm": _prepare_gemm}[case["op"]](case, int(seed), g)


# ---- plain forms ------------------------------------------------------------
def _rotate(x, c, s, rot, inter):
    x = x.float()
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_append(s):
    case, ct = s["case"], TYPES[s["case"]["type"]]
    ps = case["page"]
    phase = s["pos"].long()[:, None] * s["turns"][None]  # wraps: whole turns drop out
    angle = (phase >> 32).float() * (2 * math.pi / 2.0 ** 32)
    c, n = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    s["q_out"].copy_(_rotate(s["q"], c, n, case["rot"], case["inter"]))
    k = _rotate(s["k"], c, n, case["rot"], case["inter"]).to(ct)
    keep = s["slots"] >= 0
    slot, k, v = s["slots"][keep], k[keep], s["v"].to(ct)[keep]
    page, off = slot // ps, slot % ps
    s["k_cache"][page, :, off] = k
    s["v_cache"][page, :, off // 8, :, off % 8] = v
    return s["q_out"], s["k_cache"], s["v_cache"]


def _gather(cache, ids, v):
    """(pages of any shape) -> (shape, Hkv, tokens, D) in 32 bits."""
    x = cache[ids.long()].float()
    if v:  # [.., Hkv, ps/8, D, 8] -> [.., Hkv, ps, D]
        x = x.transpose(-1, -2).flatten(-3, -2)
    return x


def _plain_attn(s):
    case = s["case"]
    B, hq, hkv, d, ps = (case[k] for k in ("batch", "hq", "hkv", "d", "page"))
    G, L, N = hq // hkv, case["prefix"], s["most"]
    q = torch.zeros(B, N, hq, d, device=DEV)
    q[s["seq"], s["tok"]] = s["q"].float()
    q = q.view(B, N, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, N * G, d) / math.sqrt(d)
    mp = s["pages"].shape[1]
    # each sequence's own keys: [B, hkv, mp * ps, d]
    k = _gather(s["k_cache"], s["pages"], False).transpose(1, 2).flatten(2, 3)
    v = _gather(s["v_cache"], s["pages"], True).transpose(1, 2).flatten(2, 3)
    z = torch.matmul(q, k.transpose(-1, -2))
    key = torch.arange(mp * ps, device=DEV)
    tok = torch.arange(N, device=DEV)
    seen = key[None, None] <= (s["lens"] - s["news"])[:, None, None] + tok[None, :, None]
    seen = seen & (key < s["lens"][:, None, None])
    z = z.view(B, hkv, N, G, -1).masked_fill(~seen[:, None, :, None], -math.inf).flatten(2, 3)
    m = z.amax(-1)
    if L:
        kp = _gather(s["k_cache"], s["prefix_pages"], False).transpose(0, 1).flatten(1, 2)[:, :L]
        vp = _gather(s["v_cache"], s["prefix_pages"], True).transpose(0, 1).flatten(1, 2)[:, :L]
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


def _plain_quant(s):
    x = s["x"].float()
    m, k = x.shape
    kb = -(-k // 128)
    x = torch.nn.functional.pad(x, (0, kb * 128 - k)).view(m, kb, 128)
    scale = (x.abs().amax(-1) / F8_MAX).clamp_min(TINY)
    codes = (x / scale[..., None]).to(F8).view(m, kb * 128)[:, :k]
    return codes.contiguous(), scale.t().contiguous()


def _plain_gemm(s):
    n, k = s["w"].shape
    w = s["w"].float() * s["ws"].repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    x = s["x"].float() * s["xs"].t().repeat_interleave(128, 1)[:, :k]
    return torch.matmul(x, w.t()).to(TYPES[s["case"]["type"]])


# ---- the library's entry points ---------------------------------------------
def _own(s):
    import block_quantized_matmul_amd as bq
    case = s["case"]
    if case["op"] == "append":
        bq.lqmm_kv_append(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["k_cache"], s["v_cache"],
                          rope_turns=s["turns"], interleaved=case["inter"], q_out=s["q_out"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if case["op"] == "attn":
        return bq.lqmm_attn_prefix(s["q"], s["k_cache"], s["v_cache"], s["pages"], s["lens"],
                                   prefix_pages=s["prefix_pages"], prefix_len=case["prefix"],
                                   q_start=s["start"], max_q=s["most"], return_lse=True)
    if case["op"] == "quant":
        return bq.lqmm_quant_f8b128(s["x"])
    return bq.lqmm_gemm_f8b128(s["w"], s["ws"], s["x"], s["xs"], out_dtype=TYPES[case["type"]])


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "attn": _plain_attn, "quant": _plain_quant,
            "gemm": _plain_gemm}[state["case"]["op"]](state)


# ---- 64 bits ----------------------------------------------------------------
def _exact_append(s):
    case = s["case"]
    rot, ps, half = case["rot"], case["page"], case["rot"] // 2
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    ang = s["pos"].double()[:, None] * freq[None]
    unit = torch.polar(torch.ones_like(ang), ang)[:, None]

    def turn(x):
        y = x.double().clone()
        if case["inter"]:
            z = torch.view_as_complex(y[..., :rot].reshape(*y.shape[:-1], half, 2).contiguous()) * unit
            y[..., :rot] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :half], y[..., half:rot]) * unit
            y[..., :half], y[..., half:rot] = z.real, z.imag
        return y

    q, k, v = turn(s["q"]), turn(s["k"]), s["v"].double()
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    at = torch.nonzero(s["slots"] >= 0)[:, 0]
    slot = s["slots"][at]
    for h in range(case["hkv"]):
        kc[slot // ps, h, slot % ps] = k[at, h]
        vc[slot // ps, h, (slot % ps) // 8, :, slot % 8] = v[at, h]
    return q, kc, vc


def _exact_attn(s):
    case = s["case"]
    hq, hkv, d, ps, L = (case[k] for k in ("hq", "hkv", "d", "page", "prefix"))
    G = hq // hkv

    def dense(ids):
        n = ids.numel()
        k = s["k_cache"][ids.long()].double().permute(1, 0, 2, 3).reshape(hkv, n * ps, d)
        v = s["v_cache"][ids.long()].double().permute(1, 0, 2, 4, 3).reshape(hkv, n * ps, d)
        return k, v

    if L:
        pk, pv = dense(s["prefix_pages"])
        pk, pv = pk[:, :L].contiguous(), pv[:, :L].contiguous()
    lens, news = s["lens"].tolist(), s["news"].tolist()
    outs, lses, t0 = [], [], 0
    for b, (ln, nw) in enumerate(zip(lens, news)):
        k, v = dense(s["pages"][b])
        k, v = k[:, :ln], v[:, :ln]
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


def _exact_quant(s):
    m, k = s["x"].shape
    codes = torch.empty(m, k, device=DEV, dtype=torch.float64)
    scales = []
    for c in range(0, k, 128):
        x = s["x"][:, c:c + 128].double()
        sc = (x.abs().max(1).values / F8_MAX).clamp(min=TINY)
        y = x / sc[:, None]
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        codes[:, c:c + 128] = torch.round(y / step) * step
        scales.append(sc)
    return codes, torch.stack(scales)


def _exact_gemm(s):
    (m, k), n = s["x"].shape, s["w"].shape[0]
    y = torch.zeros(m, n, device=DEV, dtype=torch.float64)
    rows = torch.arange(n, device=DEV) // 128
    for b, c in enumerate(range(0, k, 1024)):
        cols = torch.arange(c, min(c + 1024, k), device=DEV) // 128
        x = s["x"][:, c:c + 1024].double() * s["xs"].double()[cols].t()
        w = s["w"][:, c:c + 1024].double() * s["ws"].double()[rows][:, cols]
        y += torch.matmul(x, w.t().contiguous())
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "quant": _exact_quant,
            "gemm": _exact_gemm}[case["op"]](s)


# ---- bytes and operations ---------------------------------------------------
def work(case):
    size = {"f16": 2, "bf16": 2, "f32": 4}
    e = size[case["type"]]
    if case["op"] == "append":
        T, heads, d = case["tokens"], case["hq"] + 2 * case["hkv"], case["d"]
        kept = T if case["run"] == "prefill" else sum(t % 16 != 9 for t in range(T))
        moved = case["hq"] * T + 2 * case["hkv"] * kept
        return {"bytes": moved * d * (size[case["in"]] + e) + T * 12 + case["rot"] * 4,
                "flops": 3 * T * (case["hq"] + case["hkv"]) * case["rot"]}
    if case["op"] == "attn":
        lens, news = _lens(case)
        T, row = sum(news), case["hkv"] * case["d"] * e
        pages = sum(-(-n // case["page"]) for n in [*lens, case["prefix"]])
        pairs = T * case["prefix"]
        for n, w in zip(lens, news):  # token i of a sequence sees n - w + i + 1 keys
            pairs += sum(max(0, n - w + i + 1) for i in range(w))
        return {"bytes": 2 * row * (sum(lens) + case["prefix"]) + T * case["hq"] * (2 * case["d"] * e + 4)
                + 4 * pages + 8 * case["batch"],
                "flops": 4 * pairs * case["hq"] * case["d"]}
    if case["op"] == "quant":
        m, k = case["m"], case["k"]
        return {"bytes": m * k * (e + 1) + 4 * m * -(-k // 128), "flops": 3 * m * k}
    m, n, k = case["m"], case["n"], case["k"]
    kb = -(-k // 128)
    return {"bytes": n * k + m * k + 4 * kb * (m + -(-n // 128)) + m * n * e, "flops": 2 * m * n * k}
