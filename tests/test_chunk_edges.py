"""Calls of append_kv and attend_chunk that a serving loop makes at its edges: many whole items,
caches beyond 32-bit offsets, shared prefixes, evicted pages, rows in front of the first
sequence, two streams at once, workspaces and scratch that other calls have left.
Tolerances as in test_attend_chunk.py and test_append_kv.py."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_sa_b200 as sa
from chunk_ref import Batch
from test_attend_chunk import call, check, run_case

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("geom,new,lens,sink,window", [
    ("llama", [5000, 100, 1], [5000, 3000, 700], 16, 64),   # items drawn one by one
    ("g8", [5000], [5100], 0, 1),
    ("latent", [500, 3], [600, 90], 4, 64),                 # items taken in turn
])
def test_many_more_items_than_ctas(geom, new, lens, sink, window):
    b, q, out, lse = run_case(geom, new, lens, sink=sink, window=window, seed=21)
    # the item counter is back at zero: the same call again, and another on its workspace
    ws = sa.Workspace.for_chunk(b.g, b.n)
    for _ in range(3):
        o, l = call(b, q, sink, window, ws=ws)
        assert torch.equal(o.view(torch.int16), out.view(torch.int16)) and torch.equal(l, lse)


@gpu
@pytest.mark.parametrize("geom,pages", [("llama", 140000), ("latent", 62000)])
def test_offsets_beyond_32_bits(geom, pages):
    """Used pages at the end of a pool of more than 2^32 bytes, and 2^31 elements, per tensor."""
    b = Batch(geom, [5, 1], [300, 77], seed=22, sigma=0.5)
    g = b.g
    small_k, small_v, table = b.k_cache, b.v_cache, b.table.clone()
    shift = pages - g.n_pool
    assert pages * g.Hkv * g.P * g.Dk > 2 ** 31
    big = sa.Geometry(**{**g.__dict__, "n_pool": pages})
    k = torch.empty(pages, g.Hkv, g.P, g.Dk, dtype=torch.bfloat16, device="cuda")
    k[shift:] = small_k.cuda()
    v = None
    if not b.latent:
        v = torch.empty(pages, g.Hkv, g.P, g.Dv, dtype=torch.bfloat16, device="cuda")
        v[shift:] = small_v.cuda()
    far = torch.where(table >= 0, table + shift, table).cuda()
    ws = sa.Workspace.for_chunk(big, b.n)
    q = b.normal(b.n, g.Hq, g.Dk).cuda()
    out, lse = sa.attend_chunk(big, q, b.to(b.cu), k, v, far, b.to(b.seq), g.Dk ** -0.5, ws)
    near, nlse = call(b, q)
    assert torch.equal(out.view(torch.int16), near.view(torch.int16)) and torch.equal(lse, nlse)
    kn = b.normal(b.n, g.Hkv, g.Dk).cuda()
    vn = None if b.latent else b.normal(b.n, g.Hkv, g.Dv).cuda()
    summ = torch.empty(pages, g.Hkv, 2, g.Dk, dtype=torch.bfloat16, device="cuda")
    summ[shift:] = 0
    ks, vs = b.to(small_k), b.to(small_v)
    ss = torch.zeros(g.n_pool, g.Hkv, 2, g.Dk, dtype=torch.bfloat16, device="cuda")
    sa.append_kv(big, kn, vn, b.to(b.cu), far, b.to(b.seq), k, v, ws, summ=summ)
    sa.append_kv(g, kn, vn, b.to(b.cu), b.to(table), b.to(b.seq), ks, vs, ws, summ=ss)
    bits = lambda x: x.view(torch.int16)
    assert torch.equal(bits(k[shift:]), bits(ks)) and torch.equal(bits(summ[shift:]), bits(ss))
    assert b.latent or torch.equal(bits(v[shift:]), bits(vs))
    assert ws.status() == sa.SA_OK


@gpu
@pytest.mark.parametrize("geom", ["llama", "latent"])
def test_shared_prefix(geom):
    """Two sequences whose first pages are the same physical pages."""
    b = Batch(geom, [3, 7], [500, 700], seed=23, sigma=0.5)
    n = 400 // b.g.P
    b.table[1, :n] = b.table[0, :n]
    q = b.normal(b.n, b.g.Hq, b.g.Dk).cuda()
    check(b, q, *call(b, q))


@gpu
@pytest.mark.parametrize("geom,P", [("llama", 16), ("ragged", 32), ("latent", 64),
                                    ("latent16", 16)])
def test_pages_out_of_the_window_may_be_gone(geom, P):
    """Pages that only hold hidden tokens are not looked at: -1 in the table, NaN in the pool."""
    new, lens, sink, window = [4, 40], [1000, 1500], 20, 200
    b = Batch(geom, new, lens, seed=24, sigma=0.5)
    q = b.normal(b.n, b.g.Hq, b.g.Dk).cuda()
    k, v, table = b.k_cache.clone(), None if b.latent else b.v_cache.clone(), b.table.clone()
    for i, (n, L) in enumerate(zip(new, lens)):
        for lp in range(-(-L // P)):
            if lp * P >= sink and (lp + 1) * P <= L - n - window + 1:
                page = int(table[i, lp])
                b.k_cache[page] = float("nan")
                if v is not None:
                    b.v_cache[page] = float("nan")
                b.table[i, lp] = -1 if lp % 2 else b.g.n_pool + 5
    out, lse = call(b, q, sink, window)
    b.k_cache, b.v_cache, b.table = k, v, table
    check(b, q, out, lse, sink, window)


@gpu
def test_rows_in_front_of_the_first_sequence():
    b = Batch("llama", [6, 2], [90, 300], pad=0, seed=25)
    g = b.g
    q = torch.full((11, g.Hq, g.Dk), float("nan"), dtype=torch.bfloat16)
    q[3:] = b.normal(8, g.Hq, g.Dk)
    k, v = b.normal(11, g.Hkv, g.Dk), b.normal(11, g.Hkv, g.Dv)
    cu = (b.cu + 3).cuda()
    kc, vc = b.to(b.k_cache), b.to(b.v_cache)
    ws = sa.Workspace.for_chunk(g, 11)
    qo = torch.full_like(q, 3.0).cuda()
    sa.append_kv(g, k.cuda(), v.cuda(), cu, b.to(b.table), b.to(b.seq), kc, vc, ws, q=q.cuda(),
                 q_out=qo)
    assert bool((qo[:3] == 3.0).all())
    assert torch.equal(qo[3:].cpu().view(torch.int16), q[3:].view(torch.int16))
    b.k_cache, b.v_cache = kc.cpu(), vc.cpu()
    out = torch.full((11, g.Hq, g.Dv), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((11, g.Hq), 5.0, device="cuda")
    sa.attend_chunk(g, qo, cu, kc, vc, b.to(b.table), b.to(b.seq), g.Dk ** -0.5, ws, out=out,
                    lse=lse)
    assert ws.status() == sa.SA_OK
    assert bool((out[:3] == 5.0).all()) and bool((lse[:3] == 5.0).all())
    check(b, q[3:].cuda(), out[3:], lse[3:])


@gpu
@pytest.mark.parametrize("first,second", [("llama", "tiny"), ("latent", "llama"),
                                          ("latent", "latent")])
def test_two_streams_at_once(first, second):
    """Calls that overlap in time, each on its own stream and workspace."""
    jobs = []
    for i, geom in enumerate((first, second)):
        b = Batch(geom, [64, 1, 9], [900, 2000, 9], seed=26 + i, sigma=0.5)
        q = b.normal(b.n, b.g.Hq, b.g.Dk).cuda()
        want = call(b, q)
        dev = [b.to(x) for x in (b.cu, b.k_cache, b.v_cache, b.table, b.seq)]
        jobs.append((b, q, want, dev, torch.cuda.Stream(), sa.Workspace.for_chunk(b.g, b.n), []))
    torch.cuda.synchronize()
    for _ in range(20):
        for b, q, _, dev, stream, ws, got in jobs:
            with torch.cuda.stream(stream):
                got.append(sa.attend_chunk(b.g, q, *dev, b.g.Dk ** -0.5, ws))
    torch.cuda.synchronize()
    for b, _, (out, lse), _, stream, ws, got in jobs:
        assert ws.status(stream) == sa.SA_OK
        for o, l in got:
            assert torch.equal(o.view(torch.int16), out.view(torch.int16))
            assert torch.equal(l, lse)


@gpu
def test_append_and_attend_back_to_back_without_a_wait():
    """Steps enqueued one behind another, as the kernels may start before the last has ended:
    every step reads what the step before wrote."""
    g0 = Batch("llama", [1, 1], [64, 200], seed=28)
    steps = 40
    b = Batch("llama", [steps, steps], [64 + steps, 200 + steps], seed=28)
    g = b.g
    q, k, v = (b.normal(steps, 2, h, 128).cuda() for h in (32, 8, 8))
    inv = (10000.0 ** (-torch.arange(64) / 64)).float().cuda()
    cu = torch.tensor([0, 1, 2], dtype=torch.int32).cuda()
    lens = [torch.tensor([65 + i, 201 + i], dtype=torch.int32).cuda() for i in range(steps)]
    table, ws = b.to(b.table), sa.Workspace.for_chunk(g, 2 * steps)

    def loop(wait):
        kc, vc = b.to(b.k_cache), b.to(b.v_cache)
        outs = []
        for i in range(steps):
            qr = sa.append_kv(g, k[i], v[i], cu, table, lens[i], kc, vc, ws, q=q[i], inv_freq=inv)
            if wait:
                torch.cuda.synchronize()
            outs.append(sa.attend_chunk(g, qr, cu, kc, vc, table, lens[i], 128 ** -0.5, ws))
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return torch.stack([o for o, _ in outs]), torch.stack([l for _, l in outs]), kc
    a, c = loop(False), loop(True)
    for x, y in zip(a, c):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    assert ws.status() == sa.SA_OK and g0.g.Hq == g.Hq


@gpu
def test_workspace_grows_with_the_rows():
    b = Batch("g5", [3], [50], seed=29)
    sizes = [sa.chunk_workspace_size(b.g, n) for n in (0, 1, 2, 3, 24, 25, 26, 51, 1000, 100000)]
    assert sizes == sorted(sizes) and sizes[0] > 256
    q = b.normal(3, 5, 128).cuda()
    check(b, q, *call(b, q, ws=sa.Workspace(sizes[-1])))


def test_scale_limits():
    """The softmax works in base 2: a scale whose product with log2(e) is not finite is refused."""
    A = ctypes.c_void_p(1 << 20)
    c = sa.Geometry(B=2, Hq=8, Hkv=2, Dk=128, Dv=128, P=16, max_pages=64, n_pool=256).c()

    def st(scale):
        return sa.lib.sa_attend_chunk(ctypes.byref(c), A, 0, A, A, A, A, A, 0, 0, scale, A, A, A,
                                      1 << 40, None)
    assert st(1e-30) == sa.SA_OK and st(2e38) == sa.SA_OK
    assert st(2.5e38) == sa.SA_ERR_INVALID_ARG and st(3.3e38) == sa.SA_ERR_INVALID_ARG


def test_workspace_and_tensors_on_one_device():
    b = Batch("tiny", [2], [2], device="cpu")

    class Ws:
        buf, nbytes = torch.zeros(1 << 12, dtype=torch.uint8), 1 << 12
    with pytest.raises(ValueError):  # CPU tensors never reach the library
        sa.attend_chunk(b.g, torch.zeros(2, 4, 64, dtype=torch.bfloat16), b.cu, b.k_cache,
                        b.v_cache, b.table, b.seq, 0.1, Ws)
