"""Attention of batches of more than 32 sequences whose items are dealt out whole (the work list walks
the batch in groups of 32), some groups without any new token.  Tolerance as in
test_attend_chunk.py.

Why nothing is cut here: an item costs its steps and 2 more, and lists of at least four times the
longest item's cost per CTA are dealt whole.  All items below have the same cost c, so what counts
is their number: at least 4 x 148 = 592 items of the grouped-query geometry (rows of one sequence
and KV head), 4 x 74 = 296 latent rows (pairs of CTAs)."""

import pytest

torch = pytest.importorskip("torch")

from chunk_ref import Batch
from test_attend_chunk import call, check

gpu = pytest.mark.gpu


def lengths(count, first):
    return [first + (7 * i) % 100 for i in range(count)]  # in the third tile of 128 keys


@gpu
@pytest.mark.parametrize("geom,new", [
    ("llama", [1] * 100),                       # 800 items
    ("llama", [0] * 40 + [2] * 90 + [0] * 33),  # groups without new tokens
    ("mha", [1] * 199 + [3]),                   # 600 items
    ("latent", [4] * 80),                       # 320 rows
    ("latent", [3] * 45 + [0] * 50 + [5] * 35),  # 310 rows
])
@pytest.mark.parametrize("sink,window", [(0, 0), (20, 400)])
def test_whole_items_of_many_sequences(geom, new, sink, window):
    b = Batch(geom, new, lengths(len(new), 270), pad=2, seed=61, sigma=0.5)
    q = b.normal(b.n, b.g.Hq, b.g.Dk)
    q[sum(new):] = float("nan")
    q = q.cuda()
    out, lse = call(b, q, sink, window)
    check(b, q, out, lse, sink, window, fill=5.0)
    o, l = call(b, q, sink, window)
    assert torch.equal(o.view(torch.int16), out.view(torch.int16)) and torch.equal(l, lse)
