"""Refusals of append_kv and attend_chunk by their messages: each check of the compiled binding is the
one that refuses, on tensors that live where they should."""

import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_sa_b200 as sa
from chunk_ref import Batch
from test_chunk_binding import append_args, attend_args, run

gpu = pytest.mark.gpu


@gpu
def test_refusals_say_what_is_wrong():
    b = Batch("tiny", [3, 2], [20, 2], seed=3)
    a, t = append_args(b), attend_args(b)
    for name, good, key, bad, match in [
            ("append", a, "k", a["k"].float(), "^k: need bfloat16 rows"),
            ("append", a, "v", a["v"][:, :, :32], "^v: need bfloat16 rows"),
            ("append", a, "q", torch.cat([a["q"]] * 2, 2)[:, :, :64], "^q: need the heads"),
            ("append", a, "cu_new", a["cu_new"][:1], "^cu_new: need a dense int32"),
            ("append", a, "seq_lens", a["seq_lens"].long(), "^seq_lens: need a dense int32"),
            ("append", a, "inv_freq", a["inv_freq"].double(), "^inv_freq: need a dense float32"),
            ("append", a, "summ", a["summ"][1:], "^summ: need a dense bfloat16"),
            ("attend", t, "q", t["q"][:, :2], "^q: need a dense bfloat16"),
            ("attend", t, "lse", t["lse"].half(), "^lse: need a dense float32"),
            ("attend", t, "page_table", t["page_table"].t(), "^page_table: need a dense int32"),
            ("attend", t, "v_cache", t["v_cache"].cpu(), "^v_cache: need .* on cpu$"),
            ("attend", t, "k_cache", t["k_cache"].cpu(), "must live on a CUDA device")]:
        with pytest.raises(ValueError, match=match):
            run(b, name, dict(good, **{key: bad}))


@gpu
@pytest.mark.parametrize("name", ["append", "attend"])
def test_a_workspace_elsewhere_is_refused(name):
    b = Batch("tiny", [3, 2], [20, 2], seed=4)

    class Ws:
        buf, nbytes = torch.zeros(1 << 20, dtype=torch.uint8), 1 << 20
    d = (append_args if name == "append" else attend_args)(b)
    with pytest.raises(ValueError, match="the workspace lives on cpu"):
        if name == "append":
            sa.append_kv(b.g, ws=Ws, **d)
        else:
            sa.attend_chunk(b.g, ws=Ws, scale=0.1, **d)
