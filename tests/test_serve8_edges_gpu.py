"""The serving operators in fewer bits at their edges: products of more tiles
than CUs, offsets and strides past 32 bits, launches in pieces, captured graphs,
graphs and threads beside each other."""
import numpy as np
import pytest

import block_quantized_matmul_amd as bq
import serve8_oracle as s8
from gpu_util import announce
from test_serve8_gpu import Batch, check_mx, compare, random_cache, up
from test_serve_gpu import DEV, np64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    bq.load()


# ---- products ------------------------------------------------------------------
@pytest.mark.parametrize("M, N, K", [
    (1, 70001, 64), (9, 40003, 160), (40, 20011, 320), (130, 9001, 288), (300, 8200, 96), (700, 9001, 160),
    (2500, 9000, 672), (4097, 8200, 32), (4097, 8200, 288), (1030, 16500, 544),
])
def test_mx_products_of_many_tiles(M, N, K):
    check_mx(M, N, K, "f16")


def test_mx_products_past_32_bits_of_outputs():
    """2.9e9 outputs: the last rows are those of a product of them alone."""
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    M, N, K = 71003, 40960, 32
    r = lambda *s: torch.randint(0, 256, s, device=DEV, generator=g, dtype=torch.uint8)  # noqa: E731
    w, x, ws, xs = r(N, K // 2), r(M, K // 2), torch.full((N, 1), 126, dtype=torch.uint8, device=DEV), r(M, 1) // 32 + 123
    announce("gemm_mxfp4 large output")
    y = bq.lqmm_gemm_mxfp4(w, ws, x, xs)
    tail = bq.lqmm_gemm_mxfp4(w, ws, x[-5:], xs[-5:])
    torch.cuda.synchronize()
    assert torch.equal(y[-5:], tail)
    first = bq.lqmm_gemm_mxfp4(w, ws, x[:5].contiguous(), xs[:5].contiguous())
    assert torch.equal(y[:5], first)


def test_mx_quant_of_many_rows_and_far_strides():
    g = torch.Generator(device=DEV)
    g.manual_seed(6)
    announce("quant_mxfp4 many rows")
    x = torch.randn(2 ** 26 + 3, 32, device=DEV, generator=g, dtype=torch.float16)
    c, s = bq.lqmm_quant_mxfp4(x)
    tail = bq.lqmm_quant_mxfp4(x[-999:])
    torch.cuda.synchronize()
    assert torch.equal(c[-999:], tail[0]) and torch.equal(s.view(torch.uint8)[-999:], tail[1].view(torch.uint8))
    del x, c, s
    announce("quant_mxfp4 far stride")
    x = torch.empty(3, 2 ** 31, dtype=torch.float16, device=DEV)[:, :96]
    x.copy_(torch.randn(3, 96, device=DEV, generator=g))
    c, s = bq.lqmm_quant_mxfp4(x)
    want = bq.lqmm_quant_mxfp4(x.contiguous())
    assert torch.equal(c, want[0]) and torch.equal(s.view(torch.uint8), want[1].view(torch.uint8))


# ---- cache ---------------------------------------------------------------------
@pytest.mark.parametrize("bits", [8, 16])
def test_append_of_many_tokens(bits):
    """More workgroups than one launch holds; most tokens are not appended."""
    T, hkv, d, ps, P = 3 * 2 ** 22 + 5, 2, 64, 16, 9
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    announce(f"append many tokens, {bits} bits")
    x = torch.randn(T, hkv, d, device=DEV, generator=g, dtype=torch.float16)
    slots = torch.full((T,), -1, dtype=torch.int64, device=DEV)
    slots[-ps * P:] = torch.arange(ps * P, device=DEV)
    out = []
    for n in (T, ps * P):
        if bits == 8:
            cache = [c.view(torch.uint8).zero_() for c in bq.kv_cache_empty(P, hkv, ps, d, dtype=F8)]
            cache += [s.view(torch.uint8) for s in bq.kv_scales_empty(P, hkv, ps)]
        else:
            cache = [c.zero_() for c in bq.kv_cache_empty(P, hkv, ps, d)]
        q = bq.lqmm_kv_append_norm(x[-n:], x[-n:], -x[-n:], None, slots[-n:], *cache,
                                   k_norm=torch.ones(d, device=DEV), q_norm=torch.ones(d, device=DEV))
        torch.cuda.synchronize()
        out.append((cache, q[-ps * P:].clone()))
    assert torch.equal(out[0][1], out[1][1])
    assert all(torch.equal(a, b) for a, b in zip(out[0][0], out[1][0]))


def test_rows_far_apart():
    """Row strides past 32 bits of q, k and v."""
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    T, hq, hkv, d, ps, P = 3, 4, 2, 64, 16, 3
    far = torch.empty(T, 2 ** 31, dtype=torch.float16, device=DEV)
    far[:, :(hq + 2 * hkv) * d] = torch.randn(T, (hq + 2 * hkv) * d, device=DEV, generator=g)
    view = far[:, :(hq + 2 * hkv) * d].unflatten(1, (hq + 2 * hkv, d))
    w = torch.rand(d, device=DEV, generator=g)
    got = []
    for x in (view, view.contiguous()):
        announce(f"append and attention, row stride {x.stride(0)}")
        cache = [c.view(torch.uint8).zero_() for c in bq.kv_cache_empty(P, hkv, ps, d, dtype=F8)]
        cache += [s.view(torch.uint8) for s in bq.kv_scales_empty(P, hkv, ps)]
        slots = torch.tensor([3, ps + 1, 2 * ps], device=DEV)
        q = bq.lqmm_kv_append_norm(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], None, slots, *cache, q_norm=w, k_norm=w)
        pages = torch.arange(3, dtype=torch.int32, device=DEV)[:, None].contiguous()
        lens = torch.tensor([5, 7, 1], dtype=torch.int32, device=DEV)
        o = bq.lqmm_attn_prefix_f8(x[:, :hq], *cache, pages, lens)
        torch.cuda.synchronize()
        got.append([q, o, *cache])
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("new", [1, 9, 130])
def test_attention_far_into_a_large_cache(new):
    """Pages whose offsets pass 32 bits: the bits of a cache of those pages alone."""
    P, hkv, ps, d, n = 2 ** 14 + 9, 16, 64, 256, 300
    used = [P - 1, 3, P - 7, P // 2 + 1, 2 ** 14 - 1, 77]
    r = np.random.default_rng(9)
    small = [up(a) for a in random_cache(r, len(used), hkv, ps, d)]
    announce(f"attention far, {new} new tokens")
    large = [torch.empty((P, *c.shape[1:]), dtype=torch.uint8, device=DEV) for c in small]
    for a, b in zip(large, small):
        a[torch.tensor(used, device=DEV)] = b
    q = torch.randn(new, 2 * hkv, d, device=DEV).half()
    i32 = dict(dtype=torch.int32, device=DEV)
    kw = dict(q_start=torch.tensor([0, new], **i32), max_q=new, prefix_len=60)
    got = [bq.lqmm_attn_prefix_f8(q, *cache, torch.tensor([ids[:5]], **i32), torch.tensor([n], **i32),
                                  prefix_pages=torch.tensor(ids[5:], **i32), **kw)
           for cache, ids in ((large, used), (small, list(range(len(used)))))]
    torch.cuda.synchronize()
    assert got[0].isfinite().all() and torch.equal(*got)


def test_sequences_that_share_pages():
    """The same page in several sequences, twice in one, and in the prefix."""
    b = Batch([40, 40, 33], [1, 1, 1], 4, 2, 64, 16, 40, "f16", seed=12)
    first = b.table[0, :2].copy()
    b.table[1, :3] = [first[0], first[1], first[0]]
    b.table[0, 2] = first[0]
    b.table[2, :3] = b.table[1, :3]
    b.pids[:2] = first
    b.pids[2] = first[1]
    compare(*b.run(), b.want())


# ---- graphs and threads ----------------------------------------------------------
def test_operators_in_a_captured_graph():
    """Append, read, quantization and product of one graph, replayed with other
    inputs and eager work between, give the bits of eager calls."""
    g = torch.Generator(device=DEV)
    g.manual_seed(11)
    T, hq, hkv, d, ps, P, hid = 33, 4, 2, 128, 16, 8, 416
    r = lambda *s: torch.randn(*s, device=DEV, generator=g)  # noqa: E731
    w, ws = bq.lqmm_quant_mxfp4(r((hq + 2 * hkv) * d, hid))
    norm, turns = r(d), bq.lqmm_rope_turns(10000.0 ** (-np.arange(0, d, 2) / d))
    slots = torch.randperm(P * ps, device=DEV, generator=g)[:T]
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    pages = torch.arange(P, dtype=torch.int32, device=DEV)[None].contiguous()
    starts = torch.tensor([0, P * ps], dtype=torch.int32, device=DEV)
    cache = [c.view(torch.uint8).zero_() for c in bq.kv_cache_empty(P, hkv, ps, d, dtype=F8)]
    cache += [s.view(torch.uint8) for s in bq.kv_scales_empty(P, hkv, ps)]
    x = r(T, hid).half()

    def run():
        y = bq.lqmm_gemm_mxfp4(w, ws, *bq.lqmm_quant_mxfp4(x)).view(T, hq + 2 * hkv, d)
        q = bq.lqmm_kv_append_norm(y[:, :hq], y[:, hq:hq + hkv], y[:, hq + hkv:], pos, slots, *cache,
                                   q_norm=norm, k_norm=norm, rope_turns=turns)
        return (y, q, *bq.lqmm_kv_read_f8(*cache, pages, starts, P * ps))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    announce("append, read, quantization and product in a graph")
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = run()
    for _ in range(4):
        x.copy_(r(T, hid))
        for c in cache[:2]:
            c.zero_()
        eager = [t.clone() for t in run()]
        kept = [c.clone() for c in cache]
        for t in (*outs, *cache):
            t.zero_()
        for c in cache[2:]:
            c.fill_(127)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, eager))
        assert all(torch.equal(a, b) for a, b in zip(cache, kept))


def split_call(seed, batch=24, prefix=700, new=1):
    """Arguments of a call whose keys are split, and its output by itself."""
    r = np.random.default_rng(seed)
    pp, hkv, d, ps = -(-prefix // 16), 2, 128, 16
    i32 = dict(dtype=torch.int32, device=DEV)
    q = torch.randn(batch * new, 8, d, device=DEV).half()
    args = (q, *map(up, random_cache(r, pp + 4 * batch, hkv, ps, d)),
            pp + torch.arange(4 * batch, **i32).view(batch, 4), torch.arange(batch, **i32) % 60 + 1)
    kw = dict(prefix_pages=torch.arange(pp, **i32), prefix_len=prefix, max_q=new)
    if new > 1:
        kw["q_start"] = new * torch.arange(batch + 1, **i32)
    assert bq.lqmm_attn_prefix_f8_workspace_bytes(prefix, 4, new, batch * new, batch, 8, hkv, d, ps) > 0
    out = bq.lqmm_attn_prefix_f8(*args, **kw)
    torch.cuda.synchronize()
    return args, kw, out


@pytest.mark.parametrize("new", [1, 20])
def test_graphs_of_one_capture_stream_run_beside_each_other(new):
    s, calls = torch.cuda.Stream(), [split_call(seed, new=new) for seed in (1, 2, 3)]
    graphs = []
    for args, kw, _ in calls[:2]:
        announce("attn_f8 graphs of one capture stream")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs = [bq.lqmm_attn_prefix_f8(*args, **kw) for _ in range(4)]
        graphs.append((graph, outs))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(6):
        torch.cuda.synchronize()
        for (graph, outs), on in zip(graphs, streams):
            with torch.cuda.stream(on):
                for o in outs:
                    o.zero_()
                graph.replay()
        with torch.cuda.stream(s):
            eager = [bq.lqmm_attn_prefix_f8(*calls[2][0], **calls[2][1]) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, calls[2][2]) for o in eager)
        for (_, outs), (_, _, want) in zip(graphs, calls):
            assert all(torch.equal(o, want) for o in outs), i


@pytest.mark.parametrize("where", ["current", "stream", "handle"])
def test_a_call_keeps_no_workspace(where):
    args, kw, want = split_call(1)
    announce(f"attn_f8 workspace of a call on {where}")
    out, s = torch.empty_like(want), torch.cuda.Stream()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for _ in range(3):
        bq.lqmm_attn_prefix_f8(*args, **kw, out=out, stream={"current": None, "stream": s, "handle": s.cuda_stream}[where])
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert torch.cuda.memory_allocated() == before


def test_threads_of_one_stream():
    import threading
    calls, wrong = [split_call(seed) for seed in (4, 5, 6)], []

    def work(args, kw, want):
        outs = [bq.lqmm_attn_prefix_f8(*args, **kw) for _ in range(100)]
        wrong.append(sum(not torch.equal(o, want) for o in outs))

    announce("attn_f8 from three threads on one stream")
    threads = [threading.Thread(target=work, args=c) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [0, 0, 0]


@pytest.mark.parametrize("hq, hkv, d, new, keys", [(32, 8, 128, 1, 5000), (8, 8, 64, 1, 9001), (4, 1, 256, 1, 3001),
                                                   (12, 2, 96, 1, 7000), (16, 4, 128, 40, 2000), (6, 6, 64, 100, 700)])
def test_many_parts_give_the_rows_of_each_sequence_alone(hq, hkv, d, new, keys):
    """Long keys split over many workgroups and joined: against 64 bits, with a
    sequence of one key, an empty one and rows of no sequence beside them."""
    b = Batch([keys, 1, 0], [new, 1, 1], hq, hkv, d, 16, 0, "f16", seed=keys)
    compare(*b.run(), b.want())


@pytest.mark.parametrize("hq, hkv, d, new, prefix", [(8, 2, 128, 1, 0), (4, 4, 64, 1, 90), (4, 1, 256, 3, 0), (16, 1, 96, 40, 33)])
def test_page_tables_wider_than_the_sequences(hq, hkv, d, new, prefix):
    """Most chunks of the table's length hold nothing: against 64 bits, with an
    empty sequence, and memory of the workspace that no part wrote is NaN."""
    b = Batch([300, 1, 0, 129, 64], [new, 1, 1, new, 1], hq, hkv, d, 16, prefix, "f16", seed=31)
    wide = np.full((5, 4096), -1, dtype=np.int32)
    wide[:, :b.table.shape[1]] = b.table
    b.table = wide
    need = bq.lqmm_attn_prefix_f8_workspace_bytes(prefix, 4096, new, sum(b.news), 5, hq, hkv, d, 16)
    assert need > 0
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    compare(*b.run(workspace=ws), b.want())


@pytest.mark.parametrize("M, N, K", [(64, 6144, 4096), (50, 8100, 1056), (128, 4090, 2080), (61, 5001, 96)])
def test_mx_products_of_sixty_four_rows(M, N, K):
    check_mx(M, N, K, "bf16")
