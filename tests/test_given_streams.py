"""Calls with ``stream=`` whose outputs are left out: the buffers a call allocates are written on that
stream and read by the caller on the current one, so neither stream's queued work may meet them
early or late.  The other stream is kept busy by a bounded sleep; every access stays inside live
allocations of the process, so a wrong order shows as wrong values."""

import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_sa_b200 as sa
from chunk_ref import Batch

gpu = pytest.mark.gpu
SLEEP = 300_000_000  # clock cycles, about 0.2 s: the calls below are queued long before


def bits(t):
    return t.contiguous().view(torch.uint8)


def new_token_calls(geom):
    b = Batch(geom, [40, 1], [200, 77], seed=41, sigma=0.5)
    g = b.g
    d = {k: b.to(getattr(b, k)) for k in ("cu", "table", "seq", "k_cache", "v_cache")}
    q, k = b.normal(b.n, g.Hq, g.Dk).cuda(), b.normal(b.n, g.Hkv, g.Dk).cuda()
    v = None if b.latent else b.normal(b.n, g.Hkv, g.Dv).cuda()
    ws = sa.Workspace.for_chunk(g, b.n)
    kc = d["k_cache"].clone()
    vc = None if b.latent else d["v_cache"].clone()
    return {
        "append_kv": lambda stream: (sa.append_kv(g, k, v, d["cu"], d["table"], d["seq"], kc, vc,
                                                  ws, q=q, stream=stream),),
        "attend_chunk": lambda stream: sa.attend_chunk(
            g, q, d["cu"], d["k_cache"], d["v_cache"], d["table"], d["seq"], g.Dk ** -0.5, ws,
            stream=stream),
    }


def check_streams(call):
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()

    # 1. blocks that the current stream has given back but still reads
    torch.cuda.empty_cache()
    busy = [torch.full_like(x, 3) for x in want]
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    copies = [x.clone() for x in busy]
    del busy
    got = call(side)
    torch.cuda.synchronize()
    for x, c, w in zip(got, copies, want):
        assert bool((c == 3).all())
        assert torch.equal(bits(x), bits(w))

    # 2. results dropped before the call has written them
    del got, copies
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(SLEEP)
    call(side)
    zeros = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    for z in zeros:
        assert not bool(bits(z).any())

    # 3. results dropped while the current stream still reads them
    del zeros
    torch.cuda.empty_cache()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(SLEEP)
    copies = [x.clone() for x in got]
    del got
    with torch.cuda.stream(side):
        fill = [torch.full_like(w, 5) for w in want]
    torch.cuda.synchronize()
    for c, w in zip(copies, want):
        assert torch.equal(bits(c), bits(w))
    del fill


@gpu
@pytest.mark.parametrize("name", ["append_kv", "attend_chunk"])
@pytest.mark.parametrize("geom", ["llama", "latent"])
def test_new_token_calls_on_a_given_stream(geom, name):
    check_streams(new_token_calls(geom)[name])


def decode_calls(geom, fp8):
    b = Batch(geom, [1] * 4, [200, 177, 130, 160], seed=42, sigma=0.5)
    g = b.g
    table, seq = b.table.cuda(), b.seq.cuda()
    k = b.k_cache.nan_to_num(0).cuda()
    v = None if b.latent else b.v_cache.nan_to_num(0).cuda()
    q = b.normal(g.B, g.Hq, g.Dk).cuda()
    budget, sink, window = 2 * g.P, 0, g.P
    ws = sa.Workspace.for_decode(g, budget)
    summ = torch.zeros(g.n_pool, g.Hkv, 2, g.Dk, dtype=torch.bfloat16, device="cuda")
    sa.page_summaries(g, k, table, seq, summ)
    sel, count = sa.select_pages(g, q, summ, table, seq, budget, sink, window, ws)
    args = (g, q, k, v, summ, table, seq, budget, sink, window, 0.1)
    calls = {
        "page_scores": lambda s: (sa.page_scores(g, q, summ, table, seq, ws, stream=s),),
        "select_pages": lambda s: sa.select_pages(g, q, summ, table, seq, budget, sink, window, ws,
                                                  stream=s),
        "sparse_decode": lambda s: sa.sparse_decode(*args, ws, stream=s),
        "sparse_decode_noalloc": lambda s: sa.sparse_decode_noalloc(*args, stream=s),
        "attend_selected": lambda s: sa.attend_selected(g, q, k, v, table, seq, sel, count, 0.1,
                                                        ws, stream=s),
    }
    if not b.latent:
        calls["sparse_decode_fused"] = lambda s: sa.sparse_decode_fused(*args, ws, stream=s)
    if fp8:
        summ8 = sa.empty_summaries_fp8(g)
        sa.page_summaries_fp8(g, k, table, seq, summ8)
        calls = {
            "page_scores_fp8": lambda s: (sa.page_scores_fp8(g, q, summ8, table, seq, ws,
                                                             stream=s),),
            "sparse_decode_fp8": lambda s: sa.sparse_decode_fp8(
                g, q, k, v, summ8, table, seq, budget, sink, window, 0.1, ws, stream=s),
        }
    return calls


@gpu
@pytest.mark.parametrize("geom,name", [
    (geom, name) for geom in ("llama", "latent")
    for name in ("page_scores", "select_pages", "sparse_decode", "sparse_decode_noalloc",
                 "attend_selected")] + [("llama", "sparse_decode_fused")])
def test_decode_calls_on_a_given_stream(geom, name):
    check_streams(decode_calls(geom, False)[name])


@gpu
@pytest.mark.parametrize("name", ["page_scores_fp8", "sparse_decode_fp8"])
def test_fp8_calls_on_a_given_stream(name):
    check_streams(decode_calls("llama", True)[name])


@gpu
def test_prune_on_a_given_stream():
    b = Batch("llama", [1, 1], [200, 77], seed=43, extra_pages=40)
    g = b.g
    table, seq = b.table.cuda(), b.seq.cuda()
    k, v = b.k_cache.nan_to_num(0).cuda(), b.v_cache.nan_to_num(0).cuda()
    keep = (torch.rand(g.B, g.max_pages * g.P, generator=b.gen) < 0.5).to(torch.uint8).cuda()
    used = set(b.table[b.table >= 0].tolist())
    free = torch.tensor([p for p in range(g.n_pool) if p not in used], dtype=torch.int32).cuda()
    summ = torch.zeros(g.n_pool, g.Hkv, 2, g.Dk, dtype=torch.bfloat16, device="cuda")
    ws = sa.Workspace.for_prune(g)
    check_streams(lambda s: sa.prune_compact(g, k, v, table, seq, keep, free, k, v, summ, ws,
                                             stream=s))
    assert ws.status() == sa.SA_OK


@gpu
def test_workspace_of_a_given_stream():
    """The buffer is zeroed on the stream it is made for."""
    side = torch.cuda.Stream()
    busy = torch.full((1 << 16,), 3, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    copy = busy.clone()
    del busy
    ws = sa.Workspace(1 << 16, stream=side)
    torch.cuda.synchronize()
    assert bool((copy == 3).all()) and ws.status(side) == sa.SA_OK
    assert not bool(ws.buf[:256].any())


@gpu
@pytest.mark.parametrize("geom", ["llama", "latent"])
def test_a_given_stream_inside_a_capture(geom):
    """A captured step whose calls run on a second stream: the outputs are the graph's."""
    calls = new_token_calls(geom)
    want = calls["append_kv"](None) + calls["attend_chunk"](None)
    torch.cuda.synchronize()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        got = calls["append_kv"](side) + calls["attend_chunk"](side)
        main.wait_stream(side)
        copies = [x.clone() for x in got]
    for _ in range(3):
        for x in got + tuple(copies):
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, c, w in zip(got, copies, want):
            assert torch.equal(bits(x), bits(w)) and torch.equal(bits(c), bits(w))


@gpu
def test_any_object_with_a_stream_handle():
    """A stream of another library: only its handle is looked at."""
    side = torch.cuda.Stream()

    class Handle:
        cuda_stream = side.cuda_stream
    calls = dict(new_token_calls("llama"), **decode_calls("llama", False))
    for name in ("append_kv", "attend_chunk", "sparse_decode"):
        want = calls[name](None)
        torch.cuda.synchronize()
        got = calls[name](Handle)
        torch.cuda.synchronize()
        for x, w in zip(got, want):
            assert torch.equal(bits(x), bits(w))
