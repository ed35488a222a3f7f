"""Appending new tokens to the paged cache: rotation, placement and the refreshed summaries
against the definition in 64 bits, refusals, and rows and storage that must stay as they were.

Tolerance of a rotated value: the result is rounded once to bf16 (2^-8 relative), and the
fp32 rotation is off by at most 2^-20 (|x| + |y|): the angle by 2^-25 turns (2^-22.3 rad)
plus sine and cosine within 2^-23 each, and three fp32 roundings.  Values that are only
copied, and the summaries of what the cache then holds, are compared bit for bit.
"""

import ctypes

import pytest

torch = pytest.importorskip("torch")

import oracle
import paged_kv_cache_sa_b200 as sa
from chunk_ref import Batch, rotated

gpu = pytest.mark.gpu
HALF_STEP = 2.0 ** -8


def freq(rot, base=500000.0):
    half = rot // 2
    return base ** (-torch.arange(half, dtype=torch.float32) / half)


def summaries_of(b, k_cache, seq, fp8=False):
    k = k_cache.cpu().view(torch.int16).numpy().view("uint16")
    f = oracle.page_summaries_fp8 if fp8 else oracle.page_summaries
    return torch.from_numpy(f(b.g, k, b.table.numpy(), seq.numpy()).view("uint8"))


def touched(b):
    return sorted({int(b.table[i, lp]) for i, (n, L) in enumerate(zip(b.new, b.lens)) if n
                   for lp in range((L - n) // b.g.P, (L - 1) // b.g.P + 1)})


def run_case(b, rot=64, start=0, interleaved=False, logical=None, summ="bf16", with_q=True,
             fused_input=True):
    g = b.g
    if b.latent or not fused_input:
        q, k = b.normal(b.n, g.Hq, g.Dk), b.normal(b.n, g.Hkv, g.Dk)
        v = None if b.latent else b.normal(b.n, g.Hkv, g.Dv)
        dq, dk, dv = b.to(q), b.to(k), b.to(v)
    else:  # slices of one projection output
        qkv = b.normal(b.n, g.Hq + 2 * g.Hkv, g.Dk)
        q, k, v = qkv.split([g.Hq, g.Hkv, g.Hkv], dim=1)
        dq, dk, dv = b.to(qkv).split([g.Hq, g.Hkv, g.Hkv], dim=1)
    inv = freq(rot) if rot else None
    k_cache, v_cache = b.to(b.k_cache), b.to(b.v_cache)
    kw = {}
    fill = torch.full((g.n_pool, g.Hkv, 2, g.Dk), 7.0, dtype=torch.bfloat16)
    fill8 = torch.full((g.n_pool, g.Hkv, 2 * g.Dk + 16), 77, dtype=torch.uint8)
    if summ == "bf16":
        kw["summ"] = b.to(fill)
    elif summ == "fp8":
        kw["summ8"] = b.to(fill8)
    q_out = torch.full((b.n, g.Hq, g.Dk), 3.0, dtype=torch.bfloat16, device=b.device)
    ws = sa.Workspace.for_chunk(g, b.n)
    got = sa.append_kv(g, dk, dv, b.to(b.cu), b.to(b.table), b.to(b.seq), k_cache, v_cache, ws,
                       q=dq if with_q else None, q_out=q_out if with_q else None,
                       inv_freq=b.to(inv), rot_start=start, interleaved=interleaved,
                       logical_lens=None if logical is None else b.to(
                           torch.tensor(logical, dtype=torch.int32)), **kw)
    assert ws.status() == sa.SA_OK
    assert (got is q_out) if with_q else (got is None)

    # the definition
    want_k = b.k_cache.double()
    want_v = None if b.latent else b.v_cache.clone()
    tol_k = torch.zeros_like(want_k)
    want_q, tol_q = torch.full((b.n, g.Hq, g.Dk), 3.0, dtype=torch.float64), 0
    tol_q = torch.zeros_like(want_q)
    at = 0
    for i, (n, L) in enumerate(zip(b.new, b.lens)):
        s = torch.arange(L - n, L)
        pos = s + ((logical[i] - L) if logical is not None else 0)
        page, slot = b.place(i, s)
        rows = slice(at, at + n)
        at += n
        kk, qq = k[rows].double(), q[rows].double()
        mk, mq = kk.abs(), qq.abs()
        if rot:
            kk, mk = rotated(kk, pos, inv, start, interleaved)
            qq, mq = rotated(qq, pos, inv, start, interleaved)
        want_k[page, :, slot] = kk
        tol_k[page, :, slot] = HALF_STEP * kk.abs() + 2.0 ** -20 * mk
        want_q[rows] = qq
        tol_q[rows] = HALF_STEP * qq.abs() + 2.0 ** -20 * mq
        if want_v is not None:
            want_v[page, :, slot] = v[rows]
    bits = lambda x: x.cpu().contiguous().view(torch.int16)
    got_k = k_cache.cpu().double()
    same = torch.isnan(want_k) & torch.isnan(got_k)
    assert bool((same | ((got_k - want_k).abs() <= tol_k)).all())
    if want_v is not None:
        assert torch.equal(bits(v_cache), bits(want_v))
    if with_q:
        assert bool(((q_out.cpu().double() - want_q).abs() <= tol_q).all())
    pages = touched(b)
    rest = [p for p in range(g.n_pool) if p not in pages]
    if summ == "bf16":
        ref = summaries_of(b, k_cache, b.seq).view(torch.int16)
        assert torch.equal(bits(kw["summ"])[pages], ref[pages])
        assert torch.equal(bits(kw["summ"])[rest], bits(fill)[rest])
    elif summ == "fp8":
        ref = summaries_of(b, k_cache, b.seq, fp8=True)
        assert torch.equal(kw["summ8"].cpu()[pages], ref[pages])
        assert torch.equal(kw["summ8"].cpu()[rest], fill8[rest])
    return k_cache


@gpu
@pytest.mark.parametrize("geom", ["tiny", "llama", "ragged", "one", "g3", "g5", "g7", "g8",
                                  "mha", "latent", "latent16"])
@pytest.mark.parametrize("new,lens", [
    ([1], [1]), ([1], [16]), ([1], [17]), ([1], [1000]), ([64], [64]), ([65, 0, 3], [65, 40, 67]),
    ([31, 1, 130, 0, 17], [31, 500, 201, 0, 33]),
])
def test_geometries_and_lengths(geom, new, lens):
    b = Batch(geom, new, lens, pad=2, seed=len(new) + lens[0])
    latent = b.latent
    run_case(b, rot=64, start=512 if latent else 0, interleaved=latent)


@gpu
@pytest.mark.parametrize("geom,rot,start", [
    ("tiny", 0, 0), ("tiny", 16, 8), ("tiny", 64, 0), ("tiny", 48, 16), ("llama", 128, 0),
    ("llama", 32, 96), ("llama", 112, 8), ("latent", 64, 512), ("latent", 128, 0),
    ("latent", 16, 560),
])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("summ", ["bf16", "fp8", None])
def test_rotated_ranges(geom, rot, start, interleaved, summ):
    b = Batch(geom, [33, 1, 20], [50, 300, 20], seed=rot + start)
    if b.latent and summ == "fp8":
        pytest.skip("fp8 records are for the grouped-query geometry")
    run_case(b, rot=rot, start=start, interleaved=interleaved, summ=summ)


@gpu
@pytest.mark.parametrize("ahead", [0, 12345, 1 << 20, (1 << 30) - 7])
def test_positions_ahead_of_slots(ahead):
    b = Batch("llama", [40, 1], [50, 77], seed=ahead % 97)
    run_case(b, rot=128, logical=[50 + ahead, 77 + ahead])


@gpu
def test_without_queries_and_dense_inputs():
    run_case(Batch("llama", [20, 1], [20, 40], seed=3), with_q=False, fused_input=False)
    run_case(Batch("ragged", [20, 1], [20, 40], seed=4), fused_input=False)


@gpu
def test_many_sequences_and_a_long_prompt():
    # more sequences than one scan round of the kernel covers, and more pages than CTAs
    new = [1, 0, 2] * 100 + [1]
    b = Batch("tiny", new, [n + (7 * i) % 40 for i, n in enumerate(new)], seed=8)
    run_case(b, rot=64)
    run_case(Batch("llama", [5000, 1], [5003, 9], seed=9), rot=128)


@gpu
def test_rotation_in_place():
    b = Batch("llama", [5], [21], seed=10)
    q, k, v = b.normal(5, 32, 128).cuda(), b.normal(5, 8, 128).cuda(), b.normal(5, 8, 128).cuda()
    inv = freq(128).cuda()
    args = (b.to(b.cu), b.to(b.table), b.to(b.seq), b.to(b.k_cache), b.to(b.v_cache),
            sa.Workspace.for_chunk(b.g, 5))
    apart = sa.append_kv(b.g, k, v, *args, q=q, inv_freq=inv)
    sa.append_kv(b.g, k, v, *args, q=q, q_out=q, inv_freq=inv)
    assert torch.equal(apart.view(torch.int16), q.view(torch.int16))


@gpu
@pytest.mark.parametrize("interleaved,rot,start,in_place", [
    (True, 64, 512, False), (False, 64, 512, True), (False, 48, 40, False)])
def test_latent_queries_of_many_tokens(interleaved, rot, start, in_place):
    """More tokens than the CTAs look up at a time; rows apart from one another or rotated in
    place; a sequence whose page is bad and rows of no sequence stay as they were."""
    new = [2500, 0, 1, 3000, 7, 1700] + [5] * 20
    b = Batch("latent", new, [n + 11 * i for i, n in enumerate(new)], pad=9, seed=rot)
    g, bad = b.g, 4
    table = b.table.clone()
    table[bad] = -1
    gen = torch.Generator("cuda").manual_seed(1)
    big = torch.randn(b.n, 128 + (0 if in_place else 1), 576, device="cuda", generator=gen,
                      dtype=torch.bfloat16)
    q, k = big[:, :128], b.normal(b.n, 1, 576).cuda()
    before = q.clone()
    q_out = q if in_place else torch.full((b.n, 128, 576), 3.0, dtype=torch.bfloat16,
                                          device="cuda")
    was = q_out[-1:].clone() if not in_place else None
    ws = sa.Workspace.for_chunk(g, b.n)
    inv = freq(rot)
    sa.append_kv(g, k, None, b.to(b.cu), b.to(table), b.to(b.seq), b.to(b.k_cache), None, ws,
                 q=q, q_out=q_out, inv_freq=inv.cuda(), rot_start=start, interleaved=interleaved)
    assert ws.status() == sa.SA_ERR_DEVICE_CHECK
    at = 0
    for i, (n, L) in enumerate(zip(new, b.lens)):
        for lo in range(0, n, 500):
            r = slice(at + lo, at + min(lo + 500, n))
            if i == bad:
                want = before[r] if in_place else was.expand(r.stop - r.start, -1, -1)
                assert torch.equal(q_out[r], want)
                continue
            pos = torch.arange(r.start, r.stop, device="cuda") - at + L - n
            half = rot // 2
            j = torch.arange(half, device="cuda")
            first = start + (2 * j if interleaved else j)
            second = first + (1 if interleaved else half)
            angle = torch.outer(pos.double(), inv.double().cuda())[:, None]
            c, sn = angle.cos(), angle.sin()
            x = before[r].double()
            u, w = x[..., first], x[..., second]
            got = q_out[r].double()
            for ch, want in ((first, u * c - w * sn), (second, w * c + u * sn)):
                tol = HALF_STEP * want.abs() + 2.0 ** -20 * (u.abs() + w.abs())
                assert bool(((got[..., ch] - want).abs() <= tol).all())
            rest = torch.ones(576, dtype=torch.bool, device="cuda")
            rest[first] = rest[second] = False
            assert torch.equal(got[..., rest], x[..., rest])
        at += n
    want = before[at:] if in_place else was.expand(b.n - at, -1, -1)
    assert torch.equal(q_out[at:], want)


@gpu
def test_bad_pages_and_lengths_are_reported_and_left_out():
    b = Batch("tiny", [20, 3, 1], [40, 3, 9], pad=1, seed=11)
    g = b.g
    q, k, v = b.normal(b.n, 4, 64).cuda(), b.normal(b.n, 1, 64).cuda(), b.normal(b.n, 1, 64).cuda()

    def call(table, cu, seq):
        kc, vc = b.to(b.k_cache), b.to(b.v_cache)
        qo = torch.full_like(q, 3.0)
        ws = sa.Workspace.for_chunk(g, b.n)
        sa.append_kv(g, k, v, b.to(cu), b.to(table), b.to(seq), kc, vc, ws, q=q, q_out=qo)
        return kc.cpu(), qo.cpu(), ws.status()
    good_k, good_q, st = call(b.table, b.cu, b.seq)
    assert st == sa.SA_OK
    bits = lambda x: x.contiguous().view(torch.int16)
    for bad in (-1, g.n_pool):
        t = b.table.clone()
        page = int(t[0, 1])
        t[0, 1] = bad              # sequence 0 adds tokens 20..39: page 1 takes 20..31
        kc, qo, st = call(t, b.cu, b.seq)
        assert st == sa.SA_ERR_DEVICE_CHECK
        want_k, want_q = good_k.clone(), good_q.clone()
        want_k[page] = b.k_cache[page]
        want_q[0:12] = 3.0
        assert torch.equal(bits(kc), bits(want_k)) and torch.equal(bits(qo), bits(want_q))
    for seq, cu in [([40, 2, 9], None), ([40, 3, 9999], None), (None, [0, 20, 23, 99])]:
        s = b.seq if seq is None else torch.tensor(seq, dtype=torch.int32)
        c = b.cu if cu is None else torch.tensor(cu, dtype=torch.int32)
        kc, qo, st = call(b.table, c, s)
        assert st == sa.SA_ERR_DEVICE_CHECK
        assert torch.equal(bits(qo[:20]), bits(good_q[:20]))  # the sound sequence is done
        page = int(b.table[0, 2])
        assert torch.equal(bits(kc[page]), bits(good_k[page]))


@gpu
def test_no_tokens_is_legal():
    b = Batch("tiny", [0, 0], [5, 0], seed=12)
    e = lambda h: torch.empty(0, h, 64, dtype=torch.bfloat16, device="cuda")
    kc = b.to(b.k_cache)
    ws = sa.Workspace.for_chunk(b.g, 0)
    out = sa.append_kv(b.g, e(1), e(1), b.to(b.cu), b.to(b.table), b.to(b.seq), kc,
                       b.to(b.v_cache), ws, q=e(4))
    assert out.shape == (0, 4, 64) and ws.status() == sa.SA_OK
    assert torch.equal(kc.cpu().view(torch.int16), b.k_cache.view(torch.int16))


def test_refusals():
    """Bad arguments come back before any CUDA call (so this runs without a GPU)."""
    A, MIS = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 4)
    INV, UNS, WSE = sa.SA_ERR_INVALID_ARG, sa.SA_ERR_UNSUPPORTED, sa.SA_ERR_WORKSPACE
    gqa = sa.Geometry(B=2, Hq=8, Hkv=2, Dk=128, Dv=128, P=16, max_pages=64, n_pool=256)
    lat = sa.Geometry(B=2, Hq=128, Hkv=1, Dk=576, Dv=512, P=64, max_pages=64, n_pool=256,
                      v_aliases_k=1)
    B2 = ctypes.c_void_p(1 << 24)

    def call(g=gqa, q=A, qs=None, k=A, ks=None, v=A, vs=None, n=4, cu=A, pt=A, sl=A, ll=None,
             fq=A, start=0, rot=64, inter=0, qo=B2, kc=A, vc=A, summ=None, summ8=None, ws=A,
             nbytes=1 << 20):
        qs = g.Hq * g.Dk if qs is None else qs
        ks = g.Hkv * g.Dk if ks is None else ks
        vs = g.Hkv * g.Dv if vs is None else vs
        c = g.c()
        return sa.lib.sa_append_kv(ctypes.byref(c), q, qs, k, ks, v, vs, n, cu, pt, sl, ll, fq,
                                   start, rot, inter, qo, kc, vc, summ, summ8, ws, nbytes, None)
    assert call(n=0) == sa.SA_OK                       # nothing to do, nothing launched
    for kw in (dict(n=-1), dict(k=None), dict(v=None), dict(cu=None), dict(pt=None),
               dict(sl=None), dict(kc=None), dict(vc=None), dict(qo=None), dict(fq=None),
               dict(rot=24), dict(rot=-16), dict(start=4), dict(start=-8), dict(start=72),
               dict(summ=A, summ8=A), dict(qs=8 * 128 - 8), dict(qs=8 * 128 + 4),
               dict(ks=2 * 128 - 8), dict(ks=2 * 128 + 2), dict(vs=0), dict(q=MIS), dict(k=MIS),
               dict(v=MIS), dict(kc=MIS), dict(vc=MIS), dict(qo=MIS), dict(summ=MIS),
               dict(summ8=MIS), dict(qo=A, qs=8 * 128 + 8)):
        assert call(**kw) == INV, kw
    assert call(rot=0, fq=None, n=0) == sa.SA_OK
    assert call(g=lat, rot=144) == UNS                 # at most 128 rotated channels
    assert call(g=lat, summ8=A) == UNS                 # fp8 records: grouped-query only
    assert call(g=lat, v=None, vc=None, n=0, start=512) == sa.SA_OK
    for kw in (dict(ws=None), dict(ws=MIS), dict(nbytes=255)):
        assert call(**kw) == WSE, kw
    bad = sa.Geometry(B=2, Hq=8, Hkv=2, Dk=96, Dv=96, P=16, max_pages=64, n_pool=256)
    assert call(g=bad) == UNS


def test_binding_checks_shapes():
    """The library sees plain pointers, so the binding checks shapes, types and devices."""
    b = Batch("tiny", [2], [2], device="cpu")
    x = lambda h: torch.zeros(2, h, 64, dtype=torch.bfloat16)

    class Ws:
        buf, nbytes = torch.zeros(1 << 12, dtype=torch.uint8), 1 << 12
    for kw in (dict(k=x(2)), dict(v=x(1).float()), dict(seq=b.seq.long()), dict(cu=b.cu[:1])):
        d = dict(k=x(1), v=x(1), cu=b.cu, seq=b.seq)
        d.update(kw)
        with pytest.raises(ValueError):
            sa.append_kv(b.g, d["k"], d["v"], d["cu"], b.table, d["seq"], b.k_cache, b.v_cache,
                         Ws)
