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
