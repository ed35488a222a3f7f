"""Attention of a ragged chunk of new tokens over the paged cache against the definition in
64 bits, refusals, and the operators of a serving step run together.

Tolerance of an output element o = sum_t w_t v_t with weights w: the probabilities enter the
product with V rounded to bf16 (half a step, 2^-8 of each w_t |v_t|), the result is rounded to
bf16 once (2^-8 of |o|); the exponential (2^-13), the fp32 sums and the fp32 scores (an error
e in a score changes its weight by a factor of 1 + e; |x| < 2^5 in these cases and its sum of
at most 576 products is good to 2^-16) stay below 2^-11 of the magnitude sum_t w_t |v_t|
together.  So |out - o| <= 2^-8 |o| + (2^-8 + 2^-11) sum_t w_t |v_t|, and the same errors
bound lse, a logarithm of the sum, by 2^-11.
"""

import ctypes

import pytest

torch = pytest.importorskip("torch")

import chunk_ref
import paged_kv_cache_sa_b200 as sa
from chunk_ref import Batch

gpu = pytest.mark.gpu


def check(b, q, out, lse, sink=0, window=0, scale=None, fill=None):
    want, want_lse, mag = chunk_ref.attend(b, q, sink, window, scale)
    n = sum(b.new)
    out, lse = out.double(), lse.double()
    if n:
        err = (out[:n] - want[:n]).abs()
        tol = 2.0 ** -8 * want[:n].abs() + (2.0 ** -8 + 2.0 ** -11) * mag[:n] + 1e-30
        assert bool((err <= tol).all()), "worst error %.3g of its bound" % float(
            (err / tol).nan_to_num(nan=float("inf")).max())
        assert bool(((lse[:n] - want_lse[:n]).abs() <= 2.0 ** -11).all())
    if fill is not None:
        assert bool((out[n:] == fill).all()) and bool((lse[n:] == fill).all())


def call(b, q, sink=0, window=0, scale=None, ws=None, fill=5.0):
    g = b.g
    ws = ws or sa.Workspace.for_chunk(g, b.n)
    out = torch.full((b.n, g.Hq, g.Dv), fill, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b.n, g.Hq), fill, dtype=torch.float32, device="cuda")
    got = sa.attend_chunk(g, q, b.to(b.cu), b.to(b.k_cache), b.to(b.v_cache), b.to(b.table),
                          b.to(b.seq), g.Dk ** -0.5 if scale is None else scale, ws, sink=sink,
                          window=window, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    assert ws.status() == sa.SA_OK
    return out, lse


def run_case(geom, new, lens, sink=0, window=0, pad=0, seed=0, sigma_q=1.5, scale=None):
    b = Batch(geom, new, lens, pad=pad, seed=seed, sigma=0.5 if "latent" in geom else 1.0)
    q = b.normal(b.n, b.g.Hq, b.g.Dk, sigma=sigma_q)
    q[sum(new):] = float("nan")  # rows of no sequence
    q = q.cuda()
    out, lse = call(b, q, sink, window, scale)
    check(b, q, out, lse, sink, window, scale, fill=5.0)
    return b, q, out, lse


GQA = ["tiny", "llama", "ragged", "one", "g3", "g5", "g7", "g8", "mha"]


@gpu
@pytest.mark.parametrize("geom", GQA)
@pytest.mark.parametrize("new,lens", [
    ([1], [1]), ([1], [15]), ([1], [129]), ([1], [1000]), ([1, 1, 1], [256, 3, 2049]),
    ([7], [7]), ([8, 0, 3], [300, 40, 67]), ([130], [130]), ([300], [1111]),
    ([31, 1, 130, 0, 17], [31, 500, 201, 0, 33]),
])
def test_lengths(geom, new, lens):
    run_case(geom, new, lens, pad=3, seed=len(new) * 1000 + lens[0])


@gpu
@pytest.mark.parametrize("geom", ["latent", "latent16"])
@pytest.mark.parametrize("new,lens", [
    ([1], [1]), ([1], [63]), ([1], [129]), ([1, 1], [1000, 64]), ([3, 0, 5], [300, 10, 5]),
    ([40], [333]),
])
def test_latent_lengths(geom, new, lens):
    run_case(geom, new, lens, pad=1, seed=len(new) * 1000 + lens[0])


@gpu
@pytest.mark.parametrize("geom", ["tiny", "llama", "g5", "latent"])
@pytest.mark.parametrize("sink,window", [(0, 1), (0, 100), (4, 1), (64, 128), (130, 257),
                                         (5000, 3), (0, 100000), (1, 127)])
def test_sink_and_window(geom, sink, window):
    new, lens = ([20, 1, 2], [700, 400, 2]) if geom == "latent" else ([200, 1, 3], [900, 1500, 3])
    run_case(geom, new, lens, sink=sink, window=window, seed=sink + window)


@gpu
@pytest.mark.parametrize("geom,new,lens", [
    ("llama", [1] * 8, [8192 + 17 * i for i in range(8)]),   # long rows, one token each
    ("llama", [1], [70001]),
    ("tiny", [1], [4096]),
    ("ragged", [8, 3, 5, 1], [9000, 20003, 16384, 33]),
    ("llama", [700], [4000]),                                 # many blocks of rows
    ("mha", [513, 64], [2000, 64]),
    ("g8", [100], [10000]),
    ("latent", [1] * 3, [4096, 5001, 64]),
    ("latent", [33], [2100]),
])
def test_longer(geom, new, lens):
    run_case(geom, new, lens, seed=7)


@gpu
def test_many_sequences():
    new = [1, 0, 2, 1, 5] * 80
    run_case("tiny", new, [n + (37 * i) % 300 for i, n in enumerate(new)], pad=5, seed=3)
    new = [1, 3] * 10
    run_case("latent", new, [n + (37 * i) % 200 for i, n in enumerate(new)], seed=4)


@gpu
@pytest.mark.parametrize("geom", ["llama", "tiny", "latent"])
def test_growing_and_large_scores(geom):
    """Keys that grow along the sequence, so that the running maximum moves again and again,
    and scores of every sign and some size: |x| < 2^5 holds by construction."""
    b = Batch(geom, [9], [1200], seed=5)
    g = b.g
    t = torch.arange(1200)
    page, slot = b.place(0, t)
    u = torch.randn(g.Dk, generator=b.gen)
    u = u / u.norm()
    ramp = (t.float() / 1200 * 5.0)[:, None, None] * u + 0.02 * torch.randn(
        1200, g.Hkv, g.Dk, generator=b.gen)
    b.k_cache[page, :, slot] = ramp.to(torch.bfloat16)
    q = (5.0 * u + 0.02 * torch.randn(9, g.Hq, g.Dk, generator=b.gen)).to(torch.bfloat16)
    q[4] = -q[4]
    q[5] = 0
    q = q.cuda()
    out, lse = call(b, q, scale=1.0)
    check(b, q, out, lse, scale=1.0)


@gpu
@pytest.mark.parametrize("geom", ["llama", "latent"])
def test_no_finite_difference_between_runs_or_company(geom):
    """Bit for bit the same on a second run, and through a captured graph."""
    b = Batch(geom, [17, 1], [800, 900], seed=6, sigma=0.5)
    q = b.normal(b.n, b.g.Hq, b.g.Dk).cuda()
    o1, l1 = call(b, q)
    o2, l2 = call(b, q)
    assert torch.equal(o1.view(torch.int16), o2.view(torch.int16)) and torch.equal(l1, l2)
    dev = [b.to(x) for x in (b.cu, b.k_cache, b.v_cache, b.table, b.seq)]
    ws = sa.Workspace.for_chunk(b.g, b.n)
    o3, l3 = torch.zeros_like(o1), torch.zeros_like(l1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            sa.attend_chunk(b.g, q, *dev, b.g.Dk ** -0.5, ws, out=o3, lse=l3)
    for _ in range(3):
        o3.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1.view(torch.int16), o3.view(torch.int16)) and torch.equal(l1, l3)
    assert ws.status() == sa.SA_OK


@gpu
def test_workspace_of_other_calls():
    """A workspace that other calls have used, and one of a decode call, serve."""
    a = Batch("llama", [40], [3000], seed=1)
    c = Batch("llama", [1, 1], [5000, 100], seed=2)
    qa = a.normal(a.n, 32, 128).cuda()
    qc = c.normal(c.n, 32, 128).cuda()
    size = max(sa.chunk_workspace_size(a.g, 40), sa.chunk_workspace_size(c.g, 2),
               sa.decode_workspace_size(c.g, 2048))
    ws = sa.Workspace(size)
    for _ in range(2):
        check(a, qa, *call(a, qa, ws=ws))
        check(c, qc, *call(c, qc, ws=ws))
        ws.buf[256:].fill_(255)  # NaN patterns in what calls leave behind


@gpu
@pytest.mark.parametrize("geom", ["tiny", "latent"])
def test_bad_pages_and_lengths_are_reported(geom):
    b = Batch(geom, [5, 2], [400, 90], seed=9)
    g = b.g
    q = b.normal(b.n, g.Hq, g.Dk).cuda()
    want, _ = call(b, q)
    ws = sa.Workspace.for_chunk(g, b.n)
    args = lambda t, c, s: (g, q, b.to(c), b.to(b.k_cache), b.to(b.v_cache), b.to(t), b.to(s),
                            g.Dk ** -0.5, ws)
    for bad in (-1, g.n_pool, 2 ** 31 - 1):
        t = b.table.clone()
        t[0, 2] = bad
        out, _ = sa.attend_chunk(*args(t, b.cu, b.seq))
        assert ws.status() == sa.SA_ERR_DEVICE_CHECK
        assert torch.equal(out[5:].view(torch.int16), want[5:].view(torch.int16))
    for seq, cu in [([4, 90], None), ([2 ** 30, 90], None), (None, [-3, 5, 7]),
                    (None, [0, 5, 7 + 1])]:
        s = b.seq if seq is None else torch.tensor(seq, dtype=torch.int32)
        c = b.cu if cu is None else torch.tensor(cu, dtype=torch.int32)
        out = torch.full((b.n, g.Hq, g.Dv), 5.0, dtype=torch.bfloat16, device="cuda")
        sa.attend_chunk(*args(b.table, c, s), out=out)
        assert ws.status() == sa.SA_ERR_DEVICE_CHECK
        left_out = slice(5, 7) if cu == [0, 5, 8] else slice(0, 5)
        sound = slice(0, 5) if cu == [0, 5, 8] else slice(5, 7)
        assert bool((out[left_out] == 5.0).all())
        assert torch.equal(out[sound].view(torch.int16), want[sound].view(torch.int16))


@gpu
def test_no_tokens_is_legal():
    b = Batch("tiny", [0, 0], [5, 0], seed=12)
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = call(b, q)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    b = Batch("llama", [0, 0], [5, 0], pad=3, seed=12)  # rows, but none of a sequence
    q = torch.full((3, 32, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    out, lse = call(b, q)
    assert bool((out == 5.0).all()) and bool((lse == 5.0).all())


@gpu
@pytest.mark.parametrize("geom,fp8", [("llama", False), ("ragged", True), ("latent", False)])
def test_prompt_then_decode_steps(geom, fp8):
    """A prompt in two chunks and two decode steps: append_kv, attend_chunk, then the sparse
    decode with the appended summaries.  With a budget of every page the decode and the chunk
    attention compute the same rows."""
    lens = [[90, 40], [200, 100], [201, 101], [202, 102]]
    b = Batch(geom, [lens[-1][i] for i in range(2)], lens[-1], seed=14, sigma=0.5)
    g = b.g
    latent = b.latent
    D, start = g.Dk, 512 if latent else 0
    inv = (10000.0 ** (-torch.arange(32, dtype=torch.float32) / 32)).cuda()
    kc = torch.full_like(b.k_cache, float("nan")).cuda()
    vc = None if latent else torch.full_like(b.v_cache, float("nan")).cuda()
    summ8 = torch.zeros(g.n_pool, g.Hkv, 2 * D + 16, dtype=torch.uint8, device="cuda")
    summ = torch.zeros(g.n_pool, g.Hkv, 2, D, dtype=torch.bfloat16, device="cuda")
    which = dict(summ8=summ8) if fp8 else dict(summ=summ)
    table = b.table.cuda()
    budget = g.max_pages * g.P
    ws = sa.Workspace(max(sa.chunk_workspace_size(g, 200), sa.decode_workspace_size(g, budget)))
    keys = [[], []]
    before = [0, 0]
    for step in lens:
        new = [s - o for s, o in zip(step, before)]
        before = step
        n = sum(new)
        cu = torch.tensor([0, new[0], n], dtype=torch.int32).cuda()
        sl = torch.tensor(step, dtype=torch.int32).cuda()
        q, k = b.normal(n, g.Hq, D).cuda(), b.normal(n, g.Hkv, D, sigma=0.5).cuda()
        v = None if latent else b.normal(n, g.Hkv, g.Dv).cuda()
        qr = sa.append_kv(g, k, v, cu, table, sl, kc, vc, ws, q=q, inv_freq=inv, rot_start=start,
                          interleaved=latent, **which)
        out, lse = sa.attend_chunk(g, qr, cu, kc, vc, table, sl, D ** -0.5, ws)
        # the cache now holds the step's rows: the definition reads them from there
        b.new, b.lens, b.n = new, step, n
        b.k_cache = kc.cpu()
        b.v_cache = None if latent else vc.cpu()
        check(b, qr, out, lse)
        if n == 2:
            dec = sa.sparse_decode_fp8 if fp8 else sa.sparse_decode
            od, ld = dec(g, qr, kc, vc, summ8 if fp8 else summ, table, sl, budget, 0, 0,
                         D ** -0.5, ws)
            check(b, qr, od, ld)
    assert ws.status() == sa.SA_OK


def test_refusals():
    """Bad arguments come back before any CUDA call (so this runs without a GPU)."""
    A, MIS = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 4)
    INV, UNS, WSE = sa.SA_ERR_INVALID_ARG, sa.SA_ERR_UNSUPPORTED, sa.SA_ERR_WORKSPACE
    gqa = sa.Geometry(B=2, Hq=8, Hkv=2, Dk=128, Dv=128, P=16, max_pages=64, n_pool=256)
    lat = sa.Geometry(B=2, Hq=128, Hkv=1, Dk=576, Dv=512, P=64, max_pages=64, n_pool=256,
                      v_aliases_k=1)

    def call(g=gqa, q=A, n=4, cu=A, kc=A, vc=A, pt=A, sl=A, sink=0, window=0, scale=0.1, out=A,
             lse=A, ws=A, nbytes=1 << 40):
        c = g.c()
        return sa.lib.sa_attend_chunk(ctypes.byref(c), q, n, cu, kc, vc, pt, sl, sink, window,
                                      scale, out, lse, ws, nbytes, None)
    assert call(n=0) == sa.SA_OK
    assert call(g=lat, vc=None, n=0) == sa.SA_OK
    inf = float("inf")
    for kw in (dict(n=-1), dict(q=None), dict(cu=None), dict(kc=None), dict(vc=None),
               dict(pt=None), dict(sl=None), dict(out=None), dict(lse=None), dict(sink=-1),
               dict(window=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=inf),
               dict(scale=float("nan")), dict(q=MIS), dict(kc=MIS), dict(vc=MIS), dict(out=MIS)):
        assert call(**kw) == INV, kw
    need = sa.chunk_workspace_size(gqa, 4)
    assert need >= 256
    for kw in (dict(ws=None), dict(ws=MIS), dict(nbytes=need - 1)):
        assert call(**kw) == WSE, kw
    bad = sa.Geometry(B=2, Hq=8, Hkv=2, Dk=96, Dv=96, P=16, max_pages=64, n_pool=256)
    assert call(g=bad) == UNS and sa.chunk_workspace_size(bad, 4) == 0
    assert sa.chunk_workspace_size(gqa, -1) == 0


def test_binding_checks_shapes():
    b = Batch("tiny", [2], [2], device="cpu")
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)

    class Ws:
        buf, nbytes = torch.zeros(1 << 12, dtype=torch.uint8), 1 << 12
    for bad in (q[:, :2], q.float(), q[0]):
        with pytest.raises(ValueError):
            sa.attend_chunk(b.g, bad, b.cu, b.k_cache, b.v_cache, b.table, b.seq, 0.1, Ws)
