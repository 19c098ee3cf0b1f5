"""Measured cases of the operators of a paged, quantised cache.

Five operators, in the order a server's step meets them:

  write    cache_write / cache_read with a page table: new rows quantised into the pages of each sequence, and read back.
  decode   decode with a page table: the newest token of every sequence over its pages.
  prefill  prefill: a chunk of new tokens of every sequence, a ragged batch, over its pages.
  weights  cache_weights: the attention weight that every key got, added to what it had.
  evict    cache_evict: the keys with the largest weights moved together into other pages, the rest given up.

`own` false computes a case in plain torch operations in 32 bits; `own` true makes the calls of the package. The pool of
pages is four planes: values [pages, Hkv, P, ...] and scales [pages, Hkv, P, D / 32] of K and of V; key j of sequence b is row
j % P of page table[b, j // P]. For every key of every head a plane holds blocks of 32 features: one fp16 scale d, and 32
signed bytes q (q8_0, value d * q) or 16 bytes with feature j in the low and feature j + 16 in the high nibble of byte j
(q4_0, value d * (nibble - 8)).
"""
import math

import torch

own = False

BLOCK = 32
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the newest token of 64 sequences, each to its own place in 4-bit pages, and those rows back: a step's latency
        dict(name="write_step_q4", op="write", B=64, Hkv=8, D=128, P=64, lo=1024, hi=8192, n=1, fmt="q4_0", dtype="bf16",
             ragged=False),
        # four prompts of up to 4095 tokens, a padded batch, into small 8-bit pages
        dict(name="write_prompt_q8", op="write", B=4, Hkv=8, D=128, P=16, lo=4095, hi=5000, n=4095, fmt="q8_0",
             dtype="bf16", ragged=True),
        # a token of each of 64 sequences of different lengths over 4-bit pages
        dict(name="decode_batch_q4", op="decode", B=64, Hq=32, Hkv=8, D=128, P=64, lo=1024, hi=8192, n=1, fmt="q4_0",
             window=0, empty=False),
        # a few short sequences of small heads in 8-bit pages, one slot of the batch unused: latency
        dict(name="decode_short_q8", op="decode", B=8, Hq=16, Hkv=8, D=64, P=16, lo=100, hi=1000, n=1, fmt="q8_0",
             window=0, empty=True),
        # a few tokens of each of 8 sequences, more than a step and less than a chunk (drafts to be verified)
        dict(name="prefill_drafts_q4", op="prefill", B=8, Hq=32, Hkv=8, D=128, P=64, lo=500, hi=4000, n=24, fmt="q4_0",
             window=0, ragged=True, empty=False),
        # the 512-token chunk at the end of a window of 67,584 keys
        dict(name="prefill_window_q4", op="prefill", B=1, Hq=16, Hkv=4, D=128, P=128, lo=67584, hi=67584, n=512,
             fmt="q4_0", window=0, ragged=False, empty=False),
        # two whole prompts of 4096 tokens of the causal LM
        dict(name="prefill_prompt_q8", op="prefill", B=2, Hq=32, Hkv=8, D=128, P=64, lo=4096, hi=4096, n=4096,
             fmt="q8_0", window=0, ragged=False, empty=False),
        # a ragged batch of chunks of small heads with a sliding window, one sequence unused
        dict(name="prefill_ragged_q8", op="prefill", B=6, Hq=16, Hkv=8, D=64, P=48, lo=300, hi=9000, n=777, fmt="q8_0",
             window=1024, ragged=True, empty=True),
        # the weights that a step's tokens gave to the keys of 64 sequences
        dict(name="weights_step_q4", op="weights", B=64, Hq=32, Hkv=8, D=128, P=64, lo=1024, hi=8192, n=1, fmt="q4_0",
             window=0, ragged=False, empty=False),
        # what a chunk of 512 gave to a window of 67,584
        dict(name="weights_window_q8", op="weights", B=1, Hq=16, Hkv=4, D=128, P=128, lo=67584, hi=67584, n=512,
             fmt="q8_0", window=0, ragged=False, empty=False),
        # 64 sequences of up to 8192 keys cut to 2048
        dict(name="evict_batch_q4", op="evict", B=64, Hkv=8, D=128, P=64, lo=1024, hi=8192, fmt="q4_0", keep=2048,
             sinks=4, recent=256),
        # the long window cut to an eighth
        dict(name="evict_window_q8", op="evict", B=1, Hkv=4, D=128, P=128, lo=67584, hi=67584, fmt="q8_0", keep=8448,
             sinks=4, recent=512),
    ]


HEADS = [(1, 1), (2, 1), (6, 2), (8, 8), (10, 2), (16, 4), (16, 8), (16, 16), (32, 4), (32, 8)]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["write", "decode", "decode", "prefill", "prefill", "prefill", "weights", "weights", "evict", "evict"])
    Hq, Hkv = rng.choice(HEADS)
    c = dict(op=op, Hkv=Hkv, D=rng.choice([64, 128]), P=rng.choice([16, 16, 32, 48, 64, 64, 112, 128, 256]),
             fmt=rng.choice(["q4_0", "q8_0"]))
    B = _spread(rng, 1, 64)
    most = max(1, min(67584, (1 << 22) // (B * Hkv)))   # keys of a sequence: the pool holds about 4 million at most
    if op == "write":
        n = _spread(rng, 1, max(1, min(4096, (1 << 17) // (B * Hkv))))
        lo = _spread(rng, n, max(n, most))
        return dict(c, B=B, lo=lo, hi=rng.randint(lo, max(lo, most)), n=n, dtype=rng.choice(["bf16", "f32"]),
                    ragged=rng.random() < 0.5)
    if op == "evict":
        lo = _spread(rng, 1, most)
        hi = rng.randint(lo, most)
        keep = _spread(rng, 1, hi)
        sinks = rng.randint(0, min(keep, 16))
        return dict(c, B=B, lo=lo, hi=hi, keep=keep, sinks=sinks, recent=rng.randint(0, keep - sinks))
    c["Hq"] = Hq
    if op == "decode":
        n = rng.choice([1, 1, 1, 2, 3, 4])
        lo = _spread(rng, 1, most)
        return dict(c, B=B, lo=lo, hi=rng.randint(lo, most), n=n, window=rng.choice([0, 0, 0, rng.randint(1, most)]),
                    empty=B > 1 and rng.random() < 0.3)
    n = _spread(rng, 1, 4096)
    pairs = 16 * 512 * 67584                              # padded rows times keys, at most
    B = max(1, min(B, pairs // (Hq * n * n)))
    most = max(1, min(most, pairs // (B * Hq * n)))
    lo = min(most, _spread(rng, n, max(n, most)))
    return dict(c, B=B, lo=lo, hi=rng.randint(lo, most), n=min(n, lo), window=rng.choice([0, 0, 0, rng.randint(1, most)]),
                ragged=rng.random() < 0.5, empty=B > 1 and rng.random() < 0.3)


# ---- inputs ------------------------------------------------------------------------------------------


def _lens(c):
    """Keys of each sequence: even over [lo, hi], so that their sum is the case's; one is 0 where a slot is unused."""
    n = torch.linspace(c["hi"], c["lo"], c["B"], dtype=torch.float64).round().to(torch.int64)
    if c.get("empty"):
        n[-1] = 0
    return n


def _counts(c):
    """New tokens of each sequence, in the order of _lens: all n, or from n down to about an eighth of it."""
    n = torch.full((c["B"],), c["n"], dtype=torch.int64)
    if c.get("ragged"):
        n = torch.linspace(c["n"], max(1, c["n"] // 8), c["B"], dtype=torch.float64).round().to(torch.int64)
    return torch.minimum(n, _lens(c))


def _normal(g, shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _pool(g, c, pages):
    """Pages that hold keys with a few strong features and values without: (k_q, k_d, v_q, v_d)."""
    got = []
    for strong in (True, False):
        x = torch.randn((pages, c["Hkv"], c["P"], c["D"]), generator=g, device="cuda")
        if strong:
            x[..., ::29] *= 3.0
        got += _quantise(x, c["fmt"])
        del x
    return got


def _empty_pool(c, pages):
    """Pages whose values are all 0."""
    rows = (pages, c["Hkv"], c["P"])
    out = []
    for _ in range(2):
        if c["fmt"] == "q4_0":
            out.append(torch.full(rows + (c["D"] // 2,), 0x88, dtype=torch.uint8, device="cuda"))
        else:
            out.append(torch.zeros(rows + (c["D"],), dtype=torch.int8, device="cuda"))
        out.append(torch.zeros(rows + (c["D"] // BLOCK,), dtype=torch.float16, device="cuda"))
    return out


def _table(g, c, keys, others=0):
    """Pages of each sequence for so many keys, in an order of the seed's, and the pages of the pool (some belong to no
    sequence); with `others`, a second table for so many keys, of further pages."""
    m, n = -(-keys // c["P"]), -(-others // c["P"])
    pages = c["B"] * (m + n) + 3
    at = torch.randperm(pages, generator=g, device="cuda")[:c["B"] * (m + n)].to(torch.int32).view(c["B"], m + n)
    return at[:, :m].contiguous(), at[:, m:].contiguous(), pages


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    order = torch.randperm(c["B"], generator=g, device="cuda")
    s = dict(case=c, lengths=_lens(c).cuda()[order])
    if c["op"] == "write":
        s["table"], _, pages = _table(g, c, c["hi"])
        s["planes"] = _empty_pool(c, pages)
        shape = (c["B"], c["Hkv"], c["n"], c["D"])
        s["k"], s["v"] = _normal(g, shape, DTYPES[c["dtype"]]), _normal(g, shape, DTYPES[c["dtype"]])
        s["k"][..., ::29] *= 3.0
        s["count"] = _counts(c).cuda()[order] if c["ragged"] else None
        s["begin"] = s["lengths"] - c["n"]   # the rows that are not padding are the first of the last n places
        return s
    if c["op"] == "evict":
        s["table"], s["table_out"], pages = _table(g, c, c["hi"], c["keep"])
        s["planes"] = _pool(g, c, pages)
        shape = (c["B"], c["Hkv"], c["hi"])
        # most of the weight on a few keys, in steps (a weight is a sum of probabilities held in 16 bits), many without any
        w = torch.rand(shape, generator=g, device="cuda").pow_(8).mul_(4).sub_(0.001).clamp_(min=0)
        s["weights"] = w.to(torch.bfloat16).float()
        s["weights_out"] = torch.zeros(shape, device="cuda")
        return s
    s["table"], _, pages = _table(g, c, c["hi"])
    s["planes"] = _pool(g, c, pages)
    s["q"] = _normal(g, (c["B"], c["Hq"], c["n"], c["D"]), torch.bfloat16)
    s["count"] = _counts(c).cuda()[order] if c["op"] != "decode" else None
    if c["op"] == "prefill":   # padding rows are left as they were
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(s["q"].shape[:3], device="cuda")
    if c["op"] == "weights":
        s["weights"] = torch.rand((c["B"], c["Hkv"], c["hi"]), generator=g, device="cuda")
        s["out"] = torch.zeros_like(s["weights"])
        s["lse"] = _lse(s)
    return s


# ---- the plain forms ---------------------------------------------------------------------------------


def _quantise(x, fmt):
    """(values, scales) of x [..., D]: the definition, in 32 bits."""
    b = x.float().unflatten(-1, (-1, BLOCK))
    if fmt == "q8_0":
        d = (b.abs().amax(-1) / 127.0).clamp(max=65504.0).to(torch.float16)
        df = d.float()[..., None]
        q = torch.where(df > 0, torch.round(b / df), torch.zeros_like(b)).clamp(-127, 127)
        return [q.to(torch.int8).flatten(-2), d]
    m = b.gather(-1, b.abs().argmax(-1, keepdim=True))[..., 0]   # the lowest index of the largest magnitude
    d = (m / -8.0).clamp(-65504.0, 65504.0).to(torch.float16)
    df = d.float()[..., None]
    q = (torch.where(df != 0, torch.round(b / df), torch.zeros_like(b)) + 8.0).clamp(0, 15).to(torch.uint8)
    return [(q[..., :16] | (q[..., 16:] << 4)).flatten(-2), d]


def _values(q, d):
    """The 32-bit values that (values, scales) stand for."""
    if q.dtype == torch.uint8:
        b = q.unflatten(-1, (-1, BLOCK // 2))
        n = torch.cat([b & 15, b >> 4], -1).float() - 8.0
    else:
        n = q.unflatten(-1, (-1, BLOCK)).float()
    return (n * d.float()[..., None]).flatten(-2)


def _gathered(plane, table):
    """A plane's pages as each sequence's keys: [B, Hkv, keys, ...]."""
    return plane[table.long()].transpose(1, 2).flatten(2, 3)


def _held(s, i):
    """32-bit values of K (i = 0) or V (i = 2) of each sequence: [B, Hkv, hi, D]."""
    q, d = (_gathered(s["planes"][i + j], s["table"])[:, :, :s["case"]["hi"]] for j in (0, 1))
    return _values(q, d)


def _positions(s):
    """Position of each token of the chunk, [B, n], and which of them are not padding."""
    i = torch.arange(s["case"]["n"], device="cuda")
    count = s["count"] if s["count"] is not None else torch.full_like(s["lengths"], s["case"]["n"])
    return (s["lengths"] - count)[:, None] + i, i < count[:, None]


def _parts(c):
    """Sequences that are taken together: as many as have at most 2^29 scores."""
    step = max(1, (1 << 29) // (c["Hq"] * c["n"] * c["hi"]))
    return [slice(b, min(c["B"], b + step)) for b in range(0, c["B"], step)]


def _scores(s, k, b):
    """Scores of the sequences of the slice b [.., Hkv, G, n, keys], with hidden pairs at -inf."""
    c = s["case"]
    q = s["q"][b].float().unflatten(1, (c["Hkv"], -1)).flatten(2, 3)
    x = (q @ k[b].transpose(-1, -2)).unflatten(2, (-1, c["n"])).mul_(1 / math.sqrt(c["D"]))
    at, real = (t[b, :, None] for t in _positions(s))
    j = torch.arange(c["hi"], device="cuda")
    seen = (j <= at) & real
    if c["window"] > 0:
        seen &= at - j <= c["window"]
    return x.masked_fill_(~seen[:, None, None], -math.inf)


def _attend(s, k, v):
    """(o, lse), those of padding 0."""
    out, logs = [], []
    for b in _parts(s["case"]):
        x = _scores(s, k, b)
        top = x.amax(-1, keepdim=True).clamp(min=-1e30)
        p = x.sub_(top).exp_()
        l = p.sum(-1, keepdim=True)
        o = (p.flatten(2, 3) @ v[b]).unflatten(2, p.shape[2:4]) / l.clamp(min=1e-37)
        out.append(o.flatten(1, 2).to(torch.bfloat16))
        logs.append(torch.where(l > 0, top + torch.log(l.clamp(min=1e-37)), torch.zeros_like(l)).flatten(1, 2)[..., 0])
    return torch.cat(out), torch.cat(logs)


def _bf16(x):
    """The serving chunk is defined, as the training one is, on the cache's values rounded to bf16."""
    return x.to(torch.bfloat16).float()


def _decode(s):
    return _attend(s, _held(s, 0), _held(s, 2))


def _prefill(s):
    return _attend(s, _bf16(_held(s, 0)), _bf16(_held(s, 2)))


def _lse(s):
    """What the attention of these tokens left, an input of their weights."""
    k = _bf16(_held(s, 0))
    got = [torch.logsumexp(_scores(s, k, b), -1).flatten(1, 2) for b in _parts(s["case"])]
    return torch.cat([torch.where(x > -1e30, x, torch.zeros_like(x)) for x in got])


def _weights(s):
    k = _bf16(_held(s, 0))
    out = s["weights"].clone()
    for b in _parts(s["case"]):
        x = _scores(s, k, b)
        out[b] += x.sub_(s["lse"][b].reshape(*x.shape[:-1], 1)).exp_().sum((2, 3), dtype=torch.float64).float()
    return [out]


def _write(s):
    """The rows into their pages, and the last n places back as bf16."""
    c = s["case"]
    r = torch.arange(c["n"], device="cuda")
    at = s["begin"][:, None] + r                                         # [B, n]
    page, row = s["table"].long().gather(1, at // c["P"]), at % c["P"]
    new = r < s["count"][:, None] if s["count"] is not None else torch.ones_like(at, dtype=torch.bool)
    for i, x in ((0, s["k"]), (2, s["v"])):
        for plane, got in zip(s["planes"][i:i + 2], _quantise(x, c["fmt"])):
            plane[page[new], :, row[new]] = got.transpose(1, 2)[new]
    return [_values(*(s["planes"][i + j][page, :, row].transpose(1, 2) for j in (0, 1))).to(torch.bfloat16) for i in (0, 2)]


def _evict(s):
    c = s["case"]
    n, keep = s["lengths"], c["keep"]
    j = torch.arange(c["hi"], device="cuda")
    w = s["weights"].masked_fill(((j < c["sinks"]) | (j >= n[:, None] - c["recent"]))[:, None], math.inf)
    w = w.masked_fill((j >= n[:, None])[:, None], -math.inf)
    kept = torch.sort(w, stable=True, dim=-1, descending=True).indices[..., :keep].sort(-1).values
    first = torch.arange(keep, device="cuda")
    kept = torch.where((n <= keep)[:, None, None], first.expand_as(kept), kept)
    left = n.clamp(max=keep)
    on = (first < left[:, None])[:, None].expand_as(kept)
    kept = torch.where(on, kept, torch.full_like(kept, -1))
    at, out = kept.clamp(min=0), s["weights_out"].zero_()
    out[..., :keep] = torch.where(on, s["weights"].gather(2, at), torch.zeros((), device="cuda"))
    b, h, i = on.nonzero(as_tuple=True)
    old, to = at[b, h, i], s["table_out"].long()
    for plane in s["planes"]:
        plane[to[b, i // c["P"]], h, i % c["P"]] = plane[s["table"].long()[b, old // c["P"]], h, old % c["P"]]
    k, v = (_values(*(_gathered(s["planes"][i + j], s["table_out"])[:, :, :keep] for j in (0, 1))).to(torch.bfloat16)
            for i in (0, 2))
    return [kept.to(torch.int32), left, out, k, v]


PLAIN = dict(write=_write, decode=_decode, prefill=_prefill, weights=_weights, evict=_evict)


# ---- the framework's calls ---------------------------------------------------------------------------


def _own(s):
    import backward_adapter_gb300 as fa

    c = s["case"]
    op, planes, table = c["op"], s["planes"], s["table"]
    if op == "write":
        fa.cache_write(s["k"], s["v"], *planes, s["begin"], s["count"], table=table)
        return fa.cache_read(*planes, s["begin"], c["n"], table=table)
    if op == "decode":
        return fa.decode(s["q"], *planes, s["lengths"], table=table, window=c["window"])
    if op == "prefill":
        return fa.prefill(s["q"], *planes, s["lengths"], s["count"], table=table, window=c["window"], out=s["out"],
                          lse=s["lse"])
    if op == "weights":
        return [fa.cache_weights(s["q"], s["lse"], planes[0], planes[1], s["lengths"], s["count"], table=table,
                                 window=c["window"], weights=s["weights"], out=s["out"])]
    kept, left = fa.cache_evict(*planes, s["weights"], s["lengths"], c["keep"], sinks=c["sinks"], recent=c["recent"],
                                table=table, table_out=s["table_out"], weights_out=s["weights_out"])
    return [kept, left, s["weights_out"], *fa.cache_read(*planes, 0, c["keep"], table=s["table_out"])]


def run(state):
    if own:
        return list(_own(state))
    return list(PLAIN[state["case"]["op"]](state))


# ---- what a pass cannot do without -------------------------------------------------------------------


def work(case):
    c = case
    D, Hkv, B = c["D"], c["Hkv"], c["B"]
    held = (D // 2 if c["fmt"] == "q4_0" else D) + D // BLOCK * 2   # bytes of a key in one plane
    lens = _lens(c)
    if c["op"] == "write":
        new = int(_counts(c).sum()) * Hkv
        es = 2 if c["dtype"] == "bf16" else 4
        # written and read back
        return {"bytes": 2 * (new * (D * es + held) + B * Hkv * c["n"] * (held + 2 * D)), "flops": 2 * new * 4 * D}
    if c["op"] == "evict":
        left = int(lens.clamp(max=c["keep"]).sum()) * Hkv
        rows = B * Hkv * c["keep"]
        # weights once in and once out, the kept rows moved, then read back
        return {"bytes": 4 * int(lens.sum()) * Hkv + 4 * B * Hkv * c["hi"] + 4 * rows + 2 * 2 * left * held
                + 2 * rows * (held + 2 * D), "flops": 2 * rows * D}
    # pairs of a token and a key that it sees, and keys that any token sees, of one head
    pairs = keys = 0
    for n, new in zip(lens.tolist(), _counts(c).tolist()):
        w = c["window"] if c["window"] > 0 else n
        first = n - new                                              # position of the first token
        at = torch.arange(first, n, dtype=torch.int64)
        pairs += int(torch.minimum(at + 1, torch.full_like(at, w + 1)).sum())
        keys += n - max(0, first - w)
    rows = int(_counts(c).sum()) * c["Hq"]
    if c["op"] == "weights":
        return {"bytes": keys * Hkv * held + 8 * B * Hkv * c["hi"] + rows * (2 * D + 4), "flops": 2 * D * pairs * c["Hq"]}
    return {"bytes": 2 * keys * Hkv * held + rows * (4 * D + 4) + 8 * B, "flops": 4 * D * pairs * c["Hq"]}


# ---- the definitions in 64 bits ----------------------------------------------------------------------


def _held64(q, d):
    """float64 values of quantised rows, by the definition of the formats."""
    out = torch.empty((*d.shape[:-1], d.shape[-1] * BLOCK), dtype=torch.float64, device=q.device)
    for f in range(0, out.shape[-1], BLOCK // 2):   # half a block at a time
        if q.dtype == torch.uint8:
            byte = q[..., f // 32 * 16:f // 32 * 16 + 16].to(torch.int32)
            n = (byte // 16 if f % 32 >= 16 else byte % 16) - 8
        else:
            n = q[..., f:f + 16].to(torch.int32)
        out[..., f:f + 16] = n.double() * d[..., f // 32, None].double()
    return out


def _stored64(x, fmt):
    """float64 values that x [..., D] has after it was stored: every block's scale, then each value's whole number."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for f in range(0, x.shape[-1], BLOCK):
        b = x[..., f:f + BLOCK].double()
        if fmt == "q8_0":
            d = (b.abs().max(-1, keepdim=True).values / 127).to(torch.float16).double()
            n = (b / torch.where(d == 0, torch.ones_like(d), d)).round().clamp(-127, 127)
        else:
            first = (b.abs() == b.abs().max(-1, keepdim=True).values).to(torch.int32).argmax(-1, keepdim=True)
            d = (b.gather(-1, first) / -8).to(torch.float16).double()
            n = (b / torch.where(d == 0, torch.ones_like(d), d)).round().clamp(-8, 7)
        out[..., f:f + BLOCK] = torch.where(d == 0, torch.zeros_like(n), n) * d
    return out


def _rows64(s, i, b, h, keys, rounded):
    """float64 K (i = 0) or V (i = 2) of some keys of one head of one sequence."""
    P = s["case"]["P"]
    page = s["table"][b].long()[keys // P]
    x = _held64(s["planes"][i][page, h, keys % P], s["planes"][i + 1][page, h, keys % P])
    return x.to(torch.bfloat16).double() if rounded else x


def _attention64(s):
    """(o, lse), or the weights, one head after the other, over the keys that its tokens see."""
    c = s["case"]
    G, scale = c["Hq"] // c["Hkv"], c["D"] ** -0.5
    out = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.zeros((c["B"], c["Hq"], c["n"], c["D"]), **out), torch.zeros((c["B"], c["Hq"], c["n"]), **out)
    got = s["weights"].double() if c["op"] == "weights" else None
    counts = s["count"].tolist() if s["count"] is not None else [c["n"]] * c["B"]
    for b, (n, new) in enumerate(zip(s["lengths"].tolist(), counts)):
        if n == 0 or new == 0:
            continue
        keys = torch.arange(max(0, n - new - c["window"]) if c["window"] else 0, n, device="cuda")
        back = torch.arange(n - new, n, device="cuda")[:, None] - keys       # keys before the token
        seen = (back >= 0) & ((back <= c["window"]) if c["window"] else (back >= 0))
        for h in range(c["Hkv"]):
            k = _rows64(s, 0, b, h, keys, c["op"] != "decode")
            v = _rows64(s, 2, b, h, keys, c["op"] != "decode") if got is None else None
            for m in range(h * G, h * G + G):
                x = scale * (s["q"][b, m, :new].double() @ k.T)
                if got is not None:
                    p = torch.exp(x - s["lse"][b, m, :new, None].double())
                    got[b, h, keys] += torch.where(seen, p, torch.zeros_like(p)).sum(0)
                    continue
                x = torch.where(seen, x, torch.full_like(x, -math.inf))
                log = torch.logsumexp(x, -1)
                some = seen.any(-1)
                log = torch.where(some, log, torch.zeros_like(log))
                o[b, m, :new] = torch.where(seen, torch.exp(x - log[:, None]), torch.zeros_like(x)) @ v
                lse[b, m, :new] = log
    return [got] if got is not None else [o, lse]


def _evict64(s):
    c = s["case"]
    shape = (c["B"], c["Hkv"], c["keep"])
    kept = torch.full(shape, -1, dtype=torch.int32, device="cuda")
    left = s["lengths"].clamp(max=c["keep"])
    out = torch.zeros(s["weights"].shape, dtype=torch.float64, device="cuda")
    to = s["table_out"].long()
    i = torch.arange(c["keep"], device="cuda")
    # what the pages of the second table held, where nothing is moved to
    k, v = (_held64(*(s["planes"][p + j][to[:, i // c["P"]], :, i % c["P"]].transpose(1, 2) for j in (0, 1))) for p in (0, 2))
    for b, n in enumerate(s["lengths"].tolist()):
        m = min(n, c["keep"])
        for h in range(c["Hkv"]):
            if n <= c["keep"]:
                at = torch.arange(n, device="cuda")
            else:
                a, z = c["sinks"], n - c["recent"]
                w, want = s["weights"][b, h, a:z].double(), c["keep"] - c["sinks"] - c["recent"]
                stay = torch.zeros(n, dtype=torch.bool, device="cuda")
                stay[:a] = True
                stay[z:] = True
                if want > 0:
                    border = torch.topk(w, want).values[-1]              # more than the border, then the first at it
                    more, at_border = w > border, w == border
                    room = want - more.sum()
                    stay[a:z] |= more | (at_border & (at_border.cumsum(0) <= room))
                at = stay.nonzero()[:, 0]
            kept[b, h, :m] = at.to(torch.int32)
            out[b, h, :m] = s["weights"][b, h, at].double()
            k[b, h, :m], v[b, h, :m] = _rows64(s, 0, b, h, at, False), _rows64(s, 2, b, h, at, False)
    return [kept, left, out, k, v]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        return _evict64(s)
    if case["op"] == "write":
        out = []
        for name in ("k", "v"):
            x = _stored64(s[name], case["fmt"])
            if s["count"] is not None:   # the padding's places keep their zeros
                x = x * (torch.arange(case["n"], device="cuda") < s["count"][:, None])[:, None, :, None]
            out.append(x)
        return out
    return _attention64(s)
