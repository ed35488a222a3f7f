"""Refusals of the Python binding of append_kv and attend_chunk: every tensor is checked against
the geometry before its address goes to the library, which could not tell."""

import pytest
import torch

import paged_kv_cache_sa_b200 as sa

from chunk_ref import Batch

gpu = pytest.mark.gpu


def append_args(b):
    g = b.g
    d = dict(k=b.normal(b.n, g.Hkv, g.Dk), v=b.normal(b.n, g.Hkv, g.Dv), cu_new=b.cu,
             page_table=b.table, seq_lens=b.seq, k_cache=b.k_cache, v_cache=b.v_cache,
             q=b.normal(b.n, g.Hq, g.Dk), q_out=b.normal(b.n, g.Hq, g.Dk),
             inv_freq=torch.ones(g.Dk // 2), logical_lens=b.seq.clone(),
             summ=torch.zeros(g.n_pool, g.Hkv, 2, g.Dk, dtype=torch.bfloat16))
    return {k: x.cuda() for k, x in d.items()}


def attend_args(b):
    g = b.g
    d = dict(q=b.normal(b.n, g.Hq, g.Dk), cu_new=b.cu, k_cache=b.k_cache, v_cache=b.v_cache,
             page_table=b.table, seq_lens=b.seq,
             out=torch.zeros(b.n, g.Hq, g.Dv, dtype=torch.bfloat16), lse=torch.zeros(b.n, g.Hq))
    return {k: x.cuda() for k, x in d.items()}


def run(b, name, d, **kw):
    ws = sa.Workspace.for_chunk(b.g, b.n)
    if name == "append":
        got = sa.append_kv(b.g, ws=ws, **d, **kw)
    else:
        got = sa.attend_chunk(b.g, ws=ws, scale=0.1, **d, **kw)
    assert ws.status() == sa.SA_OK
    return got


@gpu
@pytest.mark.parametrize("name", ["append", "attend"])
def test_wrong_tensors_are_refused(name):
    b = Batch("tiny", [3, 2], [20, 2], seed=1)
    args = append_args if name == "append" else attend_args
    good = args(b)
    run(b, name, good)
    for key, x in good.items():
        wide = torch.cat([x, x], dim=-1)
        other = torch.float64 if x.dtype != torch.float64 else torch.float32
        bad = [x.cpu(), x.to(other), x[..., :-1].contiguous(), x[None],
               wide[..., ::2], "x", x.sum().cpu()]
        if key in ("k_cache", "page_table", "seq_lens", "summ", "out", "lse", "q_out"):
            bad.append(x[:-1].contiguous())
        if key not in ("k", "v", "q") or name == "attend":
            bad.append(wide[..., :x.shape[-1]])  # rows apart
        if key in ("k", "v", "q") and name == "append":
            bad.append(torch.cat([x, x], dim=0))
        for t in bad:
            if isinstance(t, torch.Tensor) and t.shape == x.shape and t.dtype == x.dtype and \
                    t.is_cuda and t.is_contiguous():
                continue  # one element: the same tensor
            if key == "inv_freq" and isinstance(t, torch.Tensor) and t.is_cuda and \
                    t.dtype == x.dtype and t.dim() == 1 and t.is_contiguous():
                continue  # any dense row of fp32 is a width (the library judges it)
            with pytest.raises((ValueError, TypeError, AttributeError)):
                run(b, name, dict(good, **{key: t}))
    for key in ("v", "v_cache") if name == "append" else ("v_cache",):
        with pytest.raises(ValueError):
            run(b, name, dict(good, **{key: None}))
    if name == "append":
        with pytest.raises(OverflowError):
            run(b, name, good, rot_start=1 << 40)
        with pytest.raises(RuntimeError):
            run(b, name, good, interleaved=torch.ones(2))  # no truth value
        with pytest.raises(sa.SaError):
            run(b, name, good, rot_start=4)
    else:
        with pytest.raises(OverflowError):
            run(b, name, good, window=1 << 31)
        with pytest.raises(sa.SaError):
            run(b, name, good, sink=-1)
        with pytest.raises(TypeError):
            run(b, name, good, sink="4")
    run(b, name, good)  # a refusal leaves nothing behind


@gpu
@pytest.mark.parametrize("name", ["append", "attend"])
def test_bit_patterns_and_a_given_stream(name):
    """bf16 values may come as 16-bit integers; an explicit stream is the one that is used."""
    b = Batch("tiny", [3, 2], [20, 2], seed=2)
    d = (append_args if name == "append" else attend_args)(b)
    want = run(b, name, {k: x.clone() for k, x in d.items()})
    as_int = {k: x.view(torch.int16) if x.dtype == torch.bfloat16 else x for k, x in d.items()}
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = run(b, name, as_int, stream=st)
    torch.cuda.synchronize()
    for x, y in zip((want,) if name == "append" else want,
                    (got,) if name == "append" else got):
        assert torch.equal(x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32),
                           y.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32))
