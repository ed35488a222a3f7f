"""One row a call: the stride of a dimension of one row says nothing about the memory, and torch
leaves the fused projection's stride there."""

import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_sa_b200 as sa
from chunk_ref import Batch

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("geom", ["llama", "latent"])
def test_a_slice_of_a_fused_row_is_rotated_in_place(geom):
    b = Batch(geom, [1], [21], seed=51)
    g = b.g
    width = g.Hq + 2 * g.Hkv
    fused = b.normal(1, width, g.Dk).cuda()
    q, k, v = fused.split([g.Hq, g.Hkv, g.Hkv], dim=1)
    assert q.stride(0) == width * g.Dk and q.is_contiguous()
    v = None if b.latent else v
    inv = (10000.0 ** (-torch.arange(32) / 32)).float().cuda()
    ws = sa.Workspace.for_chunk(g, 1)

    def call(q, q_out):
        kc, vc = b.to(b.k_cache), b.to(b.v_cache)
        got = sa.append_kv(g, k, v, b.to(b.cu), b.to(b.table), b.to(b.seq), kc, vc, ws, q=q,
                           q_out=q_out, inv_freq=inv)
        assert ws.status() == sa.SA_OK
        return got, kc
    tail = fused[:, g.Hq:].clone()
    apart, k_apart = call(q.clone(), None)
    got, k_got = call(q, q)
    assert got is q
    assert torch.equal(q.view(torch.int16), apart.view(torch.int16))
    assert torch.equal(fused[:, g.Hq:].view(torch.int16), tail.view(torch.int16))
    assert torch.equal(k_got.view(torch.int16), k_apart.view(torch.int16))


@gpu
@pytest.mark.parametrize("stride", [8, 128, 4096, 100000])
def test_any_stride_of_a_single_row(stride):
    b = Batch("llama", [1], [21], seed=52)
    g = b.g
    args = lambda: (b.to(b.cu), b.to(b.table), b.to(b.seq), b.to(b.k_cache), b.to(b.v_cache),
                    sa.Workspace.for_chunk(g, 1))
    dense = [b.normal(1, h, 128).cuda() for h in (g.Hkv, g.Hkv, g.Hq)]
    k, v, q = (x.as_strided(x.shape, (stride, 128, 1)) for x in dense)
    want = sa.append_kv(g, dense[0], dense[1], *args(), q=dense[2])
    got = sa.append_kv(g, k, v, *args(), q=q)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
