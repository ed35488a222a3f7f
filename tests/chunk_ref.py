"""Ragged batches of new tokens for the append and chunk-attention tests, and the plain
definitions of both operators in 64 bits (torch, one loop per sequence and head).

Storage that belongs to no token (page slots behind a sequence's end, unused pages) is
filled with NaN, so that any use of it shows.
"""

import torch

GEOMS = {
    "tiny": dict(Hq=4, Hkv=1, Dk=64, Dv=64, P=16),
    "llama": dict(Hq=32, Hkv=8, Dk=128, Dv=128, P=16),
    "ragged": dict(Hq=32, Hkv=8, Dk=128, Dv=128, P=32),
    "one": dict(Hq=1, Hkv=1, Dk=128, Dv=128, P=64),
    "g3": dict(Hq=6, Hkv=2, Dk=64, Dv=64, P=32),
    "g5": dict(Hq=5, Hkv=1, Dk=128, Dv=128, P=16),
    "g8": dict(Hq=16, Hkv=2, Dk=64, Dv=64, P=64),
    "g7": dict(Hq=7, Hkv=1, Dk=128, Dv=128, P=32),
    "mha": dict(Hq=3, Hkv=3, Dk=128, Dv=128, P=16),
    "latent": dict(Hq=128, Hkv=1, Dk=576, Dv=512, P=64, latent=True),
    "latent16": dict(Hq=128, Hkv=1, Dk=576, Dv=512, P=16, latent=True),
}


class Batch:
    """One call's tensors.  ``new``/``lens``: new tokens and length after the append of every
    sequence; ``pad`` rows of no sequence follow the last one."""

    def __init__(self, geom, new, lens, pad=0, seed=0, extra_pages=3, sigma=1.0, device="cuda",
                 spare_width=1):
        import paged_kv_cache_sa_b200 as sa
        c = dict(GEOMS[geom])
        self.latent = c.pop("latent", False)
        self.new, self.lens, self.pad = list(new), list(lens), pad
        P, B = c["P"], len(new)
        pages = [-(-v // P) for v in lens]
        width = max(max(pages), 1) + spare_width
        pool = sum(pages) + extra_pages
        self.g = sa.Geometry(B=B, max_pages=width, n_pool=pool, v_aliases_k=int(self.latent), **c)
        g = self.g
        gen = torch.Generator().manual_seed(seed)
        self.gen = gen
        table = torch.full((B, width), -1, dtype=torch.int32)
        order = torch.randperm(pool, generator=gen).to(torch.int32)
        at = 0
        for b, n in enumerate(pages):
            table[b, :n] = order[at:at + n]
            at += n
        self.n = sum(new) + pad
        self.cu = torch.tensor([0] + list(new)).cumsum(0).to(torch.int32)
        self.table, self.seq = table, torch.tensor(lens, dtype=torch.int32)
        self.k_cache = self._cache(g.Dk, sigma)
        self.v_cache = None if self.latent else self._cache(g.Dv, 1.0)
        self.device = device

    def normal(self, *shape, sigma=1.0):
        return (torch.randn(shape, generator=self.gen) * sigma).to(torch.bfloat16)

    def _cache(self, width, sigma):
        g = self.g
        x = torch.full((g.n_pool, g.Hkv, g.P, width), float("nan"), dtype=torch.bfloat16)
        for b, length in enumerate(self.lens):
            for lp in range(-(-length // g.P)):
                m = min(g.P, length - lp * g.P)
                x[self.table[b, lp], :, :m] = self.normal(g.Hkv, m, width, sigma=sigma)
        return x

    def place(self, b, t):
        """(physical page, slot) of tokens t of sequence b."""
        return self.table[b].long()[t // self.g.P], t % self.g.P

    def to(self, x):
        return None if x is None else x.to(self.device)


def rotated(x, pos, inv_freq, start, interleaved):
    """x [n, H, D] float64 turned by pos * inv_freq; also |x| + |y| of every pair, the
    magnitude that rounding errors of the rotation scale with."""
    half = inv_freq.numel()
    j = torch.arange(half)
    first = start + (2 * j if interleaved else j)
    second = first + (1 if interleaved else half)
    angle = torch.outer(pos.double(), inv_freq.double())[:, None]
    c, s = angle.cos(), angle.sin()
    out, mag = x.clone(), x.abs()
    a, b = x[..., first], x[..., second]
    out[..., first], out[..., second] = a * c - b * s, b * c + a * s
    mag[..., first] = mag[..., second] = a.abs() + b.abs()
    return out, mag


def visible(slots, length, sink, window):
    """[rows, length] truth: token t is seen from slot s."""
    t = torch.arange(length, device=slots.device)
    s = slots[:, None]
    seen = t <= s
    if window > 0:
        seen &= (t > s - window) | (t < sink)
    return seen


def attend(batch, q, sink=0, window=0, scale=None, device="cuda"):
    """(out, lse, magnitude) in float64, magnitude = sum_t softmax(x)_t |v_t|; rows of no
    sequence are NaN."""
    g = batch.g
    G = g.Hq // g.Hkv
    scale = g.Dk ** -0.5 if scale is None else scale
    nan = float("nan")
    out = torch.full((batch.n, g.Hq, g.Dv), nan, dtype=torch.float64, device=device)
    mag = torch.full_like(out, nan)
    lse = torch.full((batch.n, g.Hq), nan, dtype=torch.float64, device=device)
    at = 0
    for b, (n, length) in enumerate(zip(batch.new, batch.lens)):
        if n == 0:
            continue
        page, slot = batch.place(b, torch.arange(length))
        seen = visible(torch.arange(length - n, length, device=device), length, sink, window)
        for h in range(g.Hkv):
            k = batch.k_cache[page, h, slot].to(device).double()
            v = k[:, :g.Dv] if batch.latent else batch.v_cache[page, h, slot].to(device).double()
            rows, heads = slice(at, at + n), slice(h * G, (h + 1) * G)
            x = torch.einsum("ngd,td->ngt", q[rows, heads].to(device).double(), k) * scale
            x.masked_fill_(~seen[:, None], -float("inf"))
            z = torch.logsumexp(x, -1)
            p = torch.where(seen[:, None], (x - z[..., None]).exp(), torch.zeros_like(x))
            lse[rows, heads] = z
            out[rows, heads] = torch.einsum("ngt,td->ngd", p, v)
            mag[rows, heads] = torch.einsum("ngt,td->ngd", p, v.abs())
        at += n
    return out, lse, mag
