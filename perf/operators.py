"""Appending to the paged KV cache and attention of new tokens over it: cases to measure.

Two operators of a serving step, each in its plain form (elementary torch operations) and as
the call a user makes of the framework:

* ``append``: the new tokens' keys and values go to the pages that the page table names, the
  position rotation is applied to the keys (and to the queries, into a buffer of their own)
  and the per-page key summaries of every page that received a token are refreshed, as bf16
  min/max rows or as fp8 records.
* ``attend``: exact softmax attention of the new tokens (one to thousands per sequence) over
  the cache, causal by slot, optionally restricted to sink tokens and a local window.

Geometries are the repository's workloads: Llama-3.1-8B attention (32 query / 8 KV heads of
128 channels, pages of 16), its ragged variant (pages of 32), the tiny one (4 / 1 heads of 64
channels) and the latent one (128 heads over one 576-wide latent row, pages of 64).  Lengths
are texts of comma-separated numbers: ``new`` the new tokens of each sequence, ``lens`` its
length after the append.
"""

import math

import torch

own = False

GEOMETRY = {
    "tiny": dict(Hq=4, Hkv=1, Dk=64, Dv=64, P=16, latent=False),
    "llama": dict(Hq=32, Hkv=8, Dk=128, Dv=128, P=16, latent=False),
    "ragged": dict(Hq=32, Hkv=8, Dk=128, Dv=128, P=32, latent=False),
    "latent": dict(Hq=128, Hkv=1, Dk=576, Dv=512, P=64, latent=True),
}


def _text(values):
    return ",".join(str(v) for v in values)


def _numbers(text):
    return [int(v) for v in text.split(",")]


def listed():
    return [
        # one decode step of a batch of eight at 32K tokens: eight rows into eight pages
        dict(name="append_decode", op="append", geom="llama", new=_text([1] * 8),
             lens=_text([32768] * 8), pad=0, summ="bf16", rot=128, interleaved=False,
             pruned=0, pool=16384),
        # prompts of several sessions arriving together: streaming bandwidth
        dict(name="append_prompts", op="append", geom="llama", new="8192,1,4097,2500,1600",
             lens="8192,30001,4097,12500,9999", pad=13, summ="bf16", rot=128, interleaved=False,
             pruned=0, pool=4200),
        # after pruning (positions run ahead of the slots), fp8 records, half of the channels
        # rotated in neighbouring pairs
        dict(name="append_pruned_fp8", op="append", geom="ragged", new="700,5,33,1",
             lens="9000,12005,33,20000", pad=0, summ="fp8", rot=64, interleaved=True,
             pruned=100000, pool=1400),
        # latent rows: 16 sequences, a small chunk each; the last 64 channels are rotated
        dict(name="append_latent", op="append", geom="latent", new=_text([64] * 15 + [1]),
             lens=_text([4096 + 77 * i for i in range(16)]), pad=0, summ="bf16", rot=64,
             interleaved=True, pruned=0, pool=1300),
        # the smallest call: one token of one short sequence
        dict(name="attend_tiny", op="attend", geom="tiny", new="1", lens="4096", pad=0, sink=0,
             window=0, pool=300),
        # dense decode step at 32K: one row per sequence, bandwidth of the whole cache
        dict(name="attend_decode_32k", op="attend", geom="llama", new=_text([1] * 8),
             lens=_text([32768] * 8), pad=0, sink=0, window=0, pool=16400),
        # drafted tokens checked against long ragged contexts
        dict(name="attend_drafts_ragged", op="attend", geom="ragged", new="8,3,5,1",
             lens="65536,100003,131072,81931", pad=3, sink=0, window=0, pool=12000),
        # a chunk of a long prompt: the largest, bound by the tensor cores
        dict(name="attend_chunk_8k", op="attend", geom="llama", new="8192", lens="32768", pad=0,
             sink=0, window=0, pool=2100),
        # a mixed batch: fresh prompts, a continued one, decode rows, odd sizes
        dict(name="attend_mixed", op="attend", geom="llama", new="2048,1,517,1,1300,64,1,33",
             lens="2048,8192,517,4001,5555,8000,17,7033", pad=9, sink=0, window=0, pool=2400),
        # A-shape prefill: sink tokens and a local window
        dict(name="attend_window", op="attend", geom="llama", new="8192", lens="16384", pad=0,
             sink=64, window=512, pool=1100),
        # latent decode step
        dict(name="attend_latent_decode", op="attend", geom="latent", new=_text([1] * 16),
             lens=_text([16384] * 16), pad=0, sink=0, window=0, pool=4200),
        # latent prompt chunk
        dict(name="attend_latent_chunk", op="attend", geom="latent", new="256,100",
             lens="16384,5001", pad=0, sink=0, window=0, pool=400),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend"])
    geom = rng.choice(["tiny", "llama", "llama", "ragged", "latent"])
    g = GEOMETRY[geom]
    batch = _log(rng, 1, 16)
    kind = rng.choice(["decode", "drafts", "chunk", "mixed"])
    # bounds keep a draw below the largest listed case: new tokens x length x heads
    longest = 32768 if geom != "latent" else 8192
    lens, new = [], []
    budget = 2 ** 27 if geom != "latent" else 2 ** 21
    for _ in range(batch):
        length = _log(rng, 1, longest)
        most = max(1, min(length, budget // (batch * longest)))
        n = {"decode": 1, "drafts": _log(rng, 1, 16), "chunk": _log(rng, 1, 8192),
             "mixed": rng.choice([1, _log(rng, 1, 8192)])}[kind]
        lens.append(length)
        new.append(min(n, most))
    pages = sum(-(-v // g["P"]) for v in lens)
    case = dict(op=op, geom=geom, new=_text(new), lens=_text(lens), pad=rng.choice([0, 0, 1, 7]),
                pool=pages + rng.randint(1, 64))
    if op == "append":
        rot = 64 if geom in ("latent", "tiny") else rng.choice([32, 64, 128])
        fp8 = not g["latent"] and pages <= 1800 and rng.random() < 0.5
        case.update(summ="fp8" if fp8 else "bf16", rot=rot, interleaved=rng.random() < 0.5,
                    pruned=rng.choice([0, 0, _log(rng, 1, 200000)]))
    else:
        masked = rng.random() < 0.3
        case.update(sink=rng.choice([0, 4, 64, 130]) if masked else 0,
                    window=_log(rng, 1, 4096) if masked else 0)
    return case


def _shapes(case):
    g = GEOMETRY[case["geom"]]
    new, lens = _numbers(case["new"]), _numbers(case["lens"])
    return g, new, lens, sum(new) + case["pad"]


def _normal(shape, gen, sigma=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    return x.normal_(0.0, sigma, generator=gen)


def prepare(case, seed):
    g, new, lens, n_rows = _shapes(case)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    batch, P = len(new), g["P"]
    width = max(-(-v // P) for v in lens) + 1
    order = torch.randperm(case["pool"], generator=gen, device=dev).to(torch.int32)
    table = torch.full((batch, width), -1, dtype=torch.int32)
    at = 0
    order_host = order.cpu()
    for b, v in enumerate(lens):
        n = -(-v // P)
        table[b, :n] = order_host[at:at + n]
        at += n
    cu = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32)
    s = dict(case=case, g=g, n_rows=n_rows, most_new=max(new), most_len=max(lens),
             page_table=table.to(dev), cu_new=cu.to(dev),
             seq_lens=torch.tensor(lens, dtype=torch.int32, device=dev))
    sigma = 0.5 if g["latent"] else 1.0
    s["k_cache"] = _normal((case["pool"], g["Hkv"], P, g["Dk"]), gen, sigma)
    s["v_cache"] = None if g["latent"] else _normal((case["pool"], g["Hkv"], P, g["Dv"]), gen)
    if case["op"] == "append":
        if g["latent"]:
            s["q"] = _normal((n_rows, g["Hq"], g["Dk"]), gen)
            s["k"] = _normal((n_rows, 1, g["Dk"]), gen, sigma)
            s["v"] = None
        else:  # slices of one projection's output, as a model produces them
            qkv = _normal((n_rows, g["Hq"] + 2 * g["Hkv"], g["Dk"]), gen)
            s["q"], s["k"], s["v"] = qkv.split([g["Hq"], g["Hkv"], g["Hkv"]], dim=1)
        s["q_out"] = torch.zeros((n_rows, g["Hq"], g["Dk"]), dtype=torch.bfloat16, device=dev)
        half = case["rot"] // 2
        s["inv_freq"] = 500000.0 ** (-torch.arange(half, dtype=torch.float32, device=dev) / half)
        s["rot_start"] = g["Dk"] - 64 if g["latent"] else 0
        s["logical_lens"] = s["seq_lens"] + case["pruned"] if case["pruned"] else None
        if case["summ"] == "fp8":
            s["summ8"] = torch.zeros((case["pool"], g["Hkv"], 2 * g["Dk"] + 16),
                                     dtype=torch.uint8, device=dev)
        else:
            s["summ"] = torch.zeros((case["pool"], g["Hkv"], 2, g["Dk"]), dtype=torch.bfloat16,
                                    device=dev)
    else:
        s["q"] = _normal((n_rows, g["Hq"], g["Dk"]), gen, 1.0 if g["latent"] else 2.0)
        s["scale"] = g["Dk"] ** -0.5
        s["out"] = torch.zeros((n_rows, g["Hq"], g["Dv"]), dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.zeros((n_rows, g["Hq"]), dtype=torch.float32, device=dev)
    if own:  # what a serving loop keeps: the geometry and one workspace
        import paged_kv_cache_sa_b200 as sa
        s["geom"] = sa.Geometry(B=batch, Hq=g["Hq"], Hkv=g["Hkv"], Dk=g["Dk"], Dv=g["Dv"], P=P,
                                max_pages=width, n_pool=case["pool"],
                                v_aliases_k=int(g["latent"]))
        s["ws"] = sa.Workspace.for_chunk(s["geom"], n_rows)
    return s


def run(s):
    return _append(s) if s["case"]["op"] == "append" else _attend(s)


def _append_outputs(s):
    out = dict(q_out=s["q_out"], k_cache=s["k_cache"])
    if s["v_cache"] is not None:
        out["v_cache"] = s["v_cache"]
    if "summ8" in s:
        d = s["g"]["Dk"]
        out["codes"] = s["summ8"][..., :2 * d].view(torch.float8_e4m3fn)
        out["exponents"] = s["summ8"][..., 2 * d].view(torch.int8)
    else:
        out["summ"] = s["summ"]
    return out


def _append(s):
    c = s["case"]
    if own:
        import paged_kv_cache_sa_b200 as sa
        sa.append_kv(s["geom"], s["k"], s["v"], s["cu_new"], s["page_table"], s["seq_lens"],
                     s["k_cache"], s["v_cache"], s["ws"], q=s["q"], q_out=s["q_out"],
                     inv_freq=s["inv_freq"], rot_start=s["rot_start"],
                     interleaved=c["interleaved"], logical_lens=s["logical_lens"],
                     summ=s.get("summ"), summ8=s.get("summ8"))
    else:
        _append_plain(s)
    return _append_outputs(s)


def _rotate(x, cos, sin, start, rot, interleaved):
    """x [T, H, D] rotated in 32 bits, rounded once; cos, sin [T, rot / 2]."""
    x = x.float()
    y = x.clone()
    r = x[..., start:start + rot]
    z = y[..., start:start + rot]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        z[..., 0::2] = a * cos - b * sin
        z[..., 1::2] = b * cos + a * sin
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        z[..., :rot // 2] = a * cos - b * sin
        z[..., rot // 2:] = b * cos + a * sin
    return y.to(torch.bfloat16)


def _append_plain(s):
    g, c = s["g"], s["case"]
    P = g["P"]
    cu, lens = s["cu_new"].long(), s["seq_lens"].long()
    new = cu[1:] - cu[:-1]
    n = s["n_rows"] - c["pad"]
    row = torch.arange(n, device=cu.device)
    b = torch.searchsorted(cu[1:], row, right=True)
    i = row - cu[b]
    slot = lens[b] - new[b] + i
    logical = s["logical_lens"].long() if s["logical_lens"] is not None else lens
    pos = logical[b] - new[b] + i
    angle = pos.double()[:, None] * s["inv_freq"].double()  # 64 bits: far positions
    cos, sin = angle.cos().float(), angle.sin().float()
    args = (s["rot_start"], c["rot"], c["interleaved"])
    s["q_out"][:n] = _rotate(s["q"][:n], cos, sin, *args)
    page = s["page_table"][b, slot // P].long()
    s["k_cache"][page, :, slot % P] = _rotate(s["k"][:n], cos, sin, *args)
    if s["v_cache"] is not None:
        s["v_cache"][page, :, slot % P] = s["v"][:n]
    # summaries of the touched pages: one entry per first new row of a page
    first = (i == 0) | (slot % P == 0)
    fb, lp, fp = b[first], slot[first] // P, page[first]
    valid = (lens[fb] - lp * P).clamp(max=P)
    rows = s["k_cache"][fp].float()
    there = torch.arange(P, device=cu.device) < valid[:, None]
    there = there[:, None, :, None]
    low = rows.masked_fill(~there, float("inf")).amin(2)
    high = rows.masked_fill(~there, float("-inf")).amax(2)
    if "summ8" in s:
        s["summ8"][fp] = _records(low, high)
    else:
        s["summ"][fp] = torch.stack([low, high], 2).to(torch.bfloat16)


def _records(low, high):
    """fp8 records of min and max rows [.., Dk]: E4M3 codes rounded outward, exponent, zeros."""
    largest = torch.maximum(low.abs(), high.abs()).amax(-1, keepdim=True)
    f, x = torch.frexp(largest)
    e = torch.where(f <= 0.875, x - 9, x - 8)
    e = torch.where(largest == 0, torch.zeros_like(e), e)

    def codes(v, rounding):
        y = torch.ldexp(v, -e)
        _, k = torch.frexp(y)
        step = torch.ldexp(torch.ones_like(y), (k - 1).clamp(min=-6) - 3)
        return (rounding(y / step) * step).to(torch.float8_e4m3fn).view(torch.uint8)

    lo, hi = codes(low, torch.floor), codes(high, torch.ceil)
    # zero is the code 0x00
    lo, hi = lo.masked_fill(lo == 128, 0), hi.masked_fill(hi == 128, 0)
    tail = torch.zeros(low.shape[:-1] + (16,), dtype=torch.uint8, device=low.device)
    tail[..., 0] = e[..., 0].to(torch.int8).view(torch.uint8)
    return torch.cat([lo, hi, tail], -1)


def _attend(s):
    c = s["case"]
    if own:
        import paged_kv_cache_sa_b200 as sa
        return sa.attend_chunk(s["geom"], s["q"], s["cu_new"], s["k_cache"], s["v_cache"],
                               s["page_table"], s["seq_lens"], s["scale"], s["ws"],
                               sink=c["sink"], window=c["window"], out=s["out"], lse=s["lse"])
    _attend_plain(s)
    return s["out"], s["lse"]


def _attend_plain(s):
    """The batch padded to its longest sequence and its most new tokens; scores in 32 bits."""
    g, c = s["g"], s["case"]
    P, Hkv, G = g["P"], g["Hkv"], g["Hq"] // g["Hkv"]
    cu, lens = s["cu_new"].long(), s["seq_lens"].long()
    new = cu[1:] - cu[:-1]
    B, n, pages = len(new), s["most_new"], -(-s["most_len"] // P)
    dev = cu.device
    table = s["page_table"][:, :pages].long().clamp(min=0)
    k = s["k_cache"][table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, pages * P, -1).float()
    # tokens behind a sequence's end are not part of it, whatever their pages hold
    there = torch.arange(pages * P, device=dev) < lens[:, None]
    k.masked_fill_(~there[:, None, :, None], 0.0)
    i = torch.arange(n, device=dev)
    row = (cu[:-1, None] + i).clamp(max=s["n_rows"] - 1)
    q = s["q"][row].float().view(B, n, Hkv, G, -1).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(B, Hkv, G * n, -1), k.transpose(2, 3))
    x.mul_(s["scale"])
    slot = (lens - new)[:, None] + i
    t = torch.arange(pages * P, device=dev)
    hidden = t > slot[:, :, None]
    if c["window"]:
        hidden |= (t <= slot[:, :, None] - c["window"]) & (t >= c["sink"])
    x = x.view(B, Hkv, G, n, -1).masked_fill_(hidden[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    m.masked_fill_(m == float("-inf"), 0.0)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    if g["latent"]:
        v = k[..., :g["Dv"]]
    else:
        v = s["v_cache"][table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, pages * P, -1).float()
        v.masked_fill_(~there[:, None, :, None], 0.0)
    o = torch.matmul(p.view(B, Hkv, G * n, -1), v).view(B, Hkv, G, n, -1)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (m + total.log())[..., 0]
    real = i < new[:, None]
    s["out"][row[real]] = o.permute(0, 3, 1, 2, 4).reshape(B, n, g["Hq"], -1)[real].to(
        torch.bfloat16)
    s["lse"][row[real]] = lse.permute(0, 3, 1, 2).reshape(B, n, g["Hq"])[real]


def _visible(n, length, sink, window):
    """(visible pairs, distinct visible tokens) of one sequence's new rows."""
    first = length - n
    if not window:
        return n * first + n * (n + 1) // 2, length
    pairs = 0
    for s in range(first, length):
        near = min(window, s + 1)
        pairs += near + min(sink, s + 1 - near)
    start = max(0, first - window + 1)
    return pairs, length - start + min(sink, start)


def work(case):
    g, new, lens, _ = _shapes(case)
    rows, P = sum(new), g["P"]
    widths = g["Dk"] + (0 if g["latent"] else g["Dv"])
    if case["op"] == "append":
        kv = g["Hkv"] * widths * 2
        moved = rows * (2 * kv + 2 * g["Hq"] * g["Dk"] * 2)
        for n, length in zip(new, lens):
            old = (length - n) % P  # rows before the first new one in its page
            moved += old * g["Hkv"] * g["Dk"] * 2
            pages = (length - 1) // P - (length - n) // P + 1
            record = 2 * g["Dk"] + 16 if case["summ"] == "fp8" else 4 * g["Dk"]
            moved += pages * (g["Hkv"] * record + 4)
        turned = rows * (g["Hq"] + g["Hkv"]) * case["rot"] // 2
        return dict(bytes=moved, flops=6 * turned)
    pairs = tokens = pages = 0
    for n, length in zip(new, lens):
        p, t = _visible(n, length, case["sink"], case["window"])
        pairs, tokens, pages = pairs + p, tokens + t, pages + -(-t // P)
    moved = tokens * g["Hkv"] * widths * 2 + pages * 4
    moved += rows * g["Hq"] * (g["Dk"] * 2 + g["Dv"] * 2 + 4)
    return dict(bytes=moved, flops=2 * (g["Dk"] + g["Dv"]) * g["Hq"] * pairs)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)


def _places(s, b, count):
    """Physical page and slot of the first `count` tokens of sequence b."""
    P = s["g"]["P"]
    t = torch.arange(count, device="cuda")
    return s["page_table"][b].long()[t // P], t % P


def _exact_append(s):
    g, c = s["g"], s["case"]
    half, start = c["rot"] // 2, s["rot_start"]
    q_out, k_cache = s["q_out"].double(), s["k_cache"].double()
    v_cache = None if s["v_cache"] is None else s["v_cache"].double()
    summ = None if "summ8" in s else s["summ"].double()
    j = torch.arange(half, device="cuda")
    first = start + (2 * j if c["interleaved"] else j)
    second = first + (1 if c["interleaved"] else half)
    at = 0
    for b, (n, length) in enumerate(zip(_numbers(c["new"]), _numbers(c["lens"]))):
        pos = torch.arange(length - n, length, device="cuda", dtype=torch.float64) + c["pruned"]
        turn = torch.polar(torch.ones(n, half, dtype=torch.float64, device="cuda"),
                           torch.outer(pos, s["inv_freq"].double()))[:, None]
        done = []
        for x in (s["q"], s["k"]):
            x = x[at:at + n].double()
            z = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = z.real, z.imag
            done.append(x)
        q_out[at:at + n] = done[0]
        page, slot = _places(s, b, length)
        k_cache[page[-n:], :, slot[-n:]] = done[1]
        if v_cache is not None:
            v_cache[page[-n:], :, slot[-n:]] = s["v"][at:at + n].double()
        if summ is not None:
            keys = k_cache[page, :, slot]
            for lp in range((length - n) // g["P"], (length - 1) // g["P"] + 1):
                part = keys[lp * g["P"]:(lp + 1) * g["P"]]
                summ[page[lp * g["P"]]] = torch.stack([part.amin(0), part.amax(0)], 1)
        at += n
    out = dict(q_out=q_out, k_cache=k_cache)
    if v_cache is not None:
        out["v_cache"] = v_cache
    if summ is None:
        out.update(codes=None, exponents=None)
    else:
        out["summ"] = summ
    return out


def _exact_attend(s):
    g, c = s["g"], s["case"]
    G = g["Hq"] // g["Hkv"]
    out, lse = s["out"].double(), s["lse"].double()
    at = 0
    for b, (n, length) in enumerate(zip(_numbers(c["new"]), _numbers(c["lens"]))):
        page, slot = _places(s, b, length)
        t = torch.arange(length, device="cuda")
        for h in range(g["Hkv"]):
            k = s["k_cache"][page, h, slot].double()
            v = k[:, :g["Dv"]] if g["latent"] else s["v_cache"][page, h, slot].double()
            for i in range(0, n, 1024):
                e = min(n, i + 1024)
                mine = torch.arange(length - n + i, length - n + e, device="cuda")[:, None]
                seen = t <= mine
                if c["window"]:
                    seen = seen & ((mine - t < c["window"]) | (t < c["sink"]))
                q = s["q"][at + i:at + e, h * G:(h + 1) * G].double()
                x = torch.einsum("ngd,td->ngt", q, k) * s["scale"]
                x.masked_fill_(~seen[:, None], float("-inf"))
                z = torch.logsumexp(x, -1)
                lse[at + i:at + e, h * G:(h + 1) * G] = z
                out[at + i:at + e, h * G:(h + 1) * G] = torch.einsum(
                    "ngt,td->ngd", x.sub_(z[..., None]).exp_(), v)
        at += n
    return out, lse
