"""Rows whose softmax warps hold nothing but padding: such a warp still zeroes its rows of the last
tile's values, behind the sequence's end, before the product over that tile may start.  One new
token per sequence and every length of the last tile, with NaN in the storage behind the end: a
product that started early would multiply it by a probability of zero.  Tolerance as in
test_attend_chunk.py."""

import pytest

torch = pytest.importorskip("torch")

from chunk_ref import Batch
from test_attend_chunk import call, check

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("geom,n", [
    ("tiny", 1),    # 4 of 128 rows used: three of the four warps of a chain are padding
    ("one", 1),     # a single row
    ("llama", 1),
    ("llama", 9),   # 36 rows: two warps of padding
    ("g8", 1),
])
def test_every_length_of_the_last_tile(geom, n):
    lens = [n + i for i in range(256)]  # one and two tiles, so either chain meets the tail
    b = Batch(geom, [n] * len(lens), lens, seed=31)
    q = b.normal(b.n, b.g.Hq, b.g.Dk).cuda()
    out, lse = call(b, q)
    check(b, q, out, lse)
    for _ in range(5):
        o, l = call(b, q)
        assert torch.equal(o.view(torch.int16), out.view(torch.int16)) and torch.equal(l, lse)
