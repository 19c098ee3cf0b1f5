"""Measured cases of the operators around attention over a cached window.

Three operators, in the order a token meets them:

  rope    qk_norm_rope / qk_norm_rope_bwd: RMS norm of every query and key head, then the rotary
          position, in one pass; and the gradient of both.
  cache   cache_write / cache_read: K and V quantised into a q8_0 or q4_0 cache as they are written,
          and read back as values.
  attn    decode: the newest tokens of each sequence over its quantised cache; fwd_q4 / bwd_q4: the
          training forward and backward of a query chunk over a 4-bit cache.

`own` false computes a case in plain torch operations in 32 bits; `own` true makes the calls of the
package. A quantised cache holds, for every key of every key/value head, blocks of 32 features: one
fp16 scale d, and 32 signed bytes q (q8_0, value d * q) or 16 bytes with feature j in the low and
feature j + 16 in the high nibble of byte j (q4_0, value d * (nibble - 8)).
"""
import math

import torch

own = False

BLOCK = 32
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one new token of each of 8 sequences, at positions far apart: a decode step's latency
        dict(name="rope_fwd_step", op="rope_fwd", B=8, S=1, Hq=32, Hkv=8, D=128, rot=128, dtype="bf16", layout="bhsd",
             interleaved=False, norm=True, far=100000, factor=1.0),
        # the causal LM's chunk of 4096 tokens x 4, heads read in place from the fused projection's output
        dict(name="rope_fwd_prompt", op="rope_fwd", B=4, S=4096, Hq=32, Hkv=8, D=128, rot=128, dtype="bf16",
             layout="qkv", interleaved=False, norm=True, far=0, factor=1.0),
        # part of a small head, interleaved pairs, an odd length, scaled for a long context, 32 bits
        dict(name="rope_fwd_part_f32", op="rope_fwd", B=2, S=1021, Hq=16, Hkv=8, D=64, rot=32, dtype="f32",
             layout="bshd", interleaved=True, norm=True, far=65536, factor=1.2),
        # the gradient of the causal LM's 4096 tokens
        dict(name="rope_bwd_train", op="rope_bwd", B=2, S=4096, Hq=32, Hkv=8, D=128, rot=128, dtype="bf16",
             layout="bhsd", interleaved=False, norm=True, far=0, factor=1.0),
        # the newest token of 32 sequences, each to its own place in a 4-bit cache, and those rows back
        dict(name="cache_step_q4", op="write_read", B=32, Hkv=8, S=2048, D=128, n=1, fmt="q4_0", dtype="bf16"),
        # the 512-token chunk at the end of a window of 67,584 keys, 8 bits
        dict(name="cache_chunk_q8", op="write_read", B=1, Hkv=4, S=67584, D=128, n=512, fmt="q8_0", dtype="bf16"),
        # the whole 4-bit window read back, as a pass that wants values does
        dict(name="cache_window_q4", op="read", B=1, Hkv=4, S=67584, D=128, fmt="q4_0", dtype="bf16"),
        # one token over the long window: few heads, so the keys are what there is to split
        dict(name="decode_q4_window", op="decode", B=1, Sq=1, Hq=16, Hkv=4, S=67584, lo=67584, hi=67584, D=128,
             fmt="q4_0", window=0, empty=False),
        # a serving batch of sequences of different lengths
        dict(name="decode_q4_batch", op="decode", B=64, Sq=1, Hq=32, Hkv=8, S=8192, lo=1024, hi=8192, D=128,
             fmt="q4_0", window=0, empty=False),
        # a short 8-bit cache, small heads, one slot of the batch unused: latency
        dict(name="decode_q8_short", op="decode", B=4, Sq=1, Hq=16, Hkv=8, S=1024, lo=100, hi=1000, D=64, fmt="q8_0",
             window=0, empty=True),
        # the 512-token chunk over the 67,584-key window held in 4 bits: forward, and the gradients
        dict(name="chunk_fwd_q4", op="chunk_fwd", B=1, Hq=16, Hkv=4, Sq=512, Sk=67584, D=128, mask=False),
        dict(name="chunk_bwd_q4", op="chunk_bwd", B=1, Hq=16, Hkv=4, Sq=512, Sk=67584, D=128, mask=False),
    ]


HEADS = [(1, 1), (2, 1), (6, 2), (8, 8), (10, 2), (16, 4), (16, 8), (16, 16), (32, 4), (32, 8)]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope_fwd", "rope_fwd", "rope_bwd", "write_read", "read", "decode", "decode", "decode",
                     "chunk_fwd", "chunk_bwd"])
    Hq, Hkv = rng.choice(HEADS)
    D = rng.choice([64, 128])
    if op in ("rope_fwd", "rope_bwd"):
        B = _spread(rng, 1, 16)
        S = _spread(rng, 1, max(1, min(8192, (1 << 19) // (B * (Hq + Hkv)))))
        return dict(op=op, B=B, S=S, Hq=Hq, Hkv=Hkv, D=D, rot=16 * rng.randint(1, D // 16),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), layout=rng.choice(["bhsd", "bshd", "qkv"]),
                    interleaved=rng.random() < 0.4, norm=rng.random() < 0.8,
                    far=rng.choice([0, rng.randint(1, 1 << 20)]), factor=rng.choice([1.0, round(rng.uniform(1, 1.4), 3)]))
    fmt = rng.choice(["q4_0", "q4_0", "q8_0"])
    if op in ("write_read", "read"):
        B = _spread(rng, 1, 32)
        S = _spread(rng, 1, max(1, min(131072, (1 << 19) // (B * Hkv))))
        if op == "read":
            return dict(op=op, B=B, Hkv=Hkv, S=S, D=D, fmt=fmt, dtype=rng.choice(["bf16", "f32"]))
        return dict(op=op, B=B, Hkv=Hkv, S=S, D=D, n=_spread(rng, 1, S), fmt=fmt, dtype=rng.choice(["bf16", "f32"]))
    if op == "decode":
        B = _spread(rng, 1, 64)
        S = _spread(rng, 1, max(1, min(131072, (1 << 21) // (B * Hkv))))
        lo = rng.randint(1, S)
        hi = rng.randint(lo, S)
        return dict(op=op, B=B, Sq=rng.choice([1, 1, 1, 2, 3, 4]), Hq=Hq, Hkv=Hkv, S=S, lo=lo, hi=hi, D=D, fmt=fmt,
                    window=rng.choice([0, 0, 0, rng.randint(1, S)]), empty=B > 1 and rng.random() < 0.3)
    Sq = _spread(rng, 1, 1024)
    most = (16 * 512 * 67584) // (Hq * Sq)
    Sk = _spread(rng, Sq, max(Sq, min(67584, most)))
    B = max(1, min(4, most // Sk)) if rng.random() < 0.5 else 1
    # a mask tensor hides about a third of the keys, all of them for one row
    return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, Sq=Sq, Sk=Sk, D=D, mask=Sq * Sk <= 1 << 24 and rng.random() < 0.4)


# ---- inputs ------------------------------------------------------------------------------------------


def _normal(g, shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _planes(g, c):
    """A cache that holds keys with a few strong features and values without: (k_q, k_d, v_q, v_d)."""
    got = []
    for strong in (True, False):
        x = torch.randn((c["B"], c["Hkv"], c["S"], c["D"]), generator=g, device="cuda")
        if strong:
            x[..., ::29] *= 3.0
        got += _quantise(x, c["fmt"])
        del x
    return got


def _lengths(g, c):
    """Keys of each sequence: even over [lo, hi], in an order of the seed's, so that their sum is the case's."""
    n = torch.linspace(c["hi"], c["lo"], c["B"], dtype=torch.float64).round().to(torch.int64)
    if c["empty"]:
        n[-1] = 0
    return n.cuda()[torch.randperm(c["B"], generator=g, device="cuda")]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=c)
    if c["op"] in ("rope_fwd", "rope_bwd"):
        B, S, Hq, Hkv, D, dt = c["B"], c["S"], c["Hq"], c["Hkv"], c["D"], DTYPES[c["dtype"]]
        if c["layout"] == "qkv":   # the projection's output: queries, keys and values of a token side by side
            qkv = _normal(g, (B, S, Hq + 2 * Hkv, D), dt)
            s["q"], s["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]
        elif c["layout"] == "bshd":
            s["q"], s["k"] = _normal(g, (B, S, Hq, D), dt), _normal(g, (B, S, Hkv, D), dt)
        else:
            s["q"], s["k"] = _normal(g, (B, Hq, S, D), dt), _normal(g, (B, Hkv, S, D), dt)
        if c["op"] == "rope_bwd":
            s["dq"] = _normal(g, s["q"].shape, dt, 0.1)
            s["dk"] = _normal(g, s["k"].shape, dt, 0.1)
        s["qw"] = (1 + 0.2 * _normal(g, (D,))).to(dt) if c["norm"] else None
        s["kw"] = (1 + 0.2 * _normal(g, (D,))).to(dt) if c["norm"] else None
        first = torch.randint(0, c["far"] + 1, (B, 1), generator=g, device="cuda")
        s["pos"] = first + torch.arange(S, device="cuda")
        half = c["rot"] // 2
        s["inv_freq"] = 10000.0 ** -(torch.arange(half, dtype=torch.float32, device="cuda") / half)
        return s
    if c["op"] == "write_read":
        shape = (c["B"], c["Hkv"], c["n"], c["D"])
        s["k"], s["v"] = _normal(g, shape, DTYPES[c["dtype"]]), _normal(g, shape, DTYPES[c["dtype"]])
        s["k"][..., ::29] *= 3.0
        s["planes"] = _empty_planes(c)
        s["begin"] = c["S"] - c["n"]   # the chunk ends where the window does
        return s
    if c["op"] == "read":
        s["planes"] = _planes(g, c)
        return s
    if c["op"] == "decode":
        s["planes"] = _planes(g, c)
        s["q"] = _normal(g, (c["B"], c["Hq"], c["Sq"], c["D"]), torch.bfloat16)
        s["lengths"] = _lengths(g, c)
        return s
    s["planes"] = _planes(g, dict(c, S=c["Sk"], fmt="q4_0"))
    s["q"] = _normal(g, (c["B"], c["Hq"], c["Sq"], c["D"]), torch.bfloat16)
    s["mask"] = None
    if c["mask"]:
        s["mask"] = (torch.rand((1, c["Sq"], c["Sk"]), generator=g, device="cuda") < 0.7).to(torch.uint8)
        s["mask"][:, c["Sq"] // 2] = 0
    if c["op"] == "chunk_bwd":
        s["do"] = _normal(g, s["q"].shape, torch.bfloat16, 0.1)
        s["o"], s["lse"] = _chunk_fwd(s)
    return s


def _empty_planes(c):
    rows = (c["B"], c["Hkv"], c["S"])
    values = rows + (c["D"] // 2,) if c["fmt"] == "q4_0" else rows + (c["D"],)
    kind = torch.uint8 if c["fmt"] == "q4_0" else torch.int8
    scales = rows + (c["D"] // BLOCK,)
    return [torch.zeros(values, dtype=kind, device="cuda"), torch.zeros(scales, dtype=torch.float16, device="cuda"),
            torch.zeros(values, dtype=kind, device="cuda"), torch.zeros(scales, dtype=torch.float16, device="cuda")]


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


def _angles(s):
    a = s["pos"].double()[..., None] * s["inv_freq"].double()
    f = s["case"]["factor"]
    cos, sin = (a.cos() * f).float(), (a.sin() * f).float()
    return (cos[:, None], sin[:, None]) if s["case"]["layout"] == "bhsd" else (cos[:, :, None], sin[:, :, None])


def _turn(x, cos, sin, c, back=False):
    """x with its first rot features rotated, by minus the angle where `back`."""
    r, half = c["rot"], c["rot"] // 2
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else (x[..., :half], x[..., half:r])
    sin = -sin if back else sin
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, v], -1).flatten(-2) if c["interleaved"] else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _rope_fwd(s):
    c = s["case"]
    cos, sin = _angles(s)
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        f = x.float()
        if w is not None:
            f = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        out.append(_turn(f, cos, sin, c).to(x.dtype))
    return out


def _rope_bwd(s):
    c = s["case"]
    cos, sin = _angles(s)
    grads, weights = [], []
    for x, w, dy in ((s["q"], s["qw"], s["dq"]), (s["k"], s["kw"], s["dk"])):
        g = _turn(dy.float(), cos, sin, c, back=True)
        if w is None:
            grads.append(g.to(x.dtype))
            continue
        f = x.float()
        r = torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)
        n = f * r
        weights.append((g * n).sum((0, 1, 2), dtype=torch.float64).float())
        t = g * w.float()
        grads.append((r * (t - n * (t * n).mean(-1, keepdim=True))).to(x.dtype))
    return grads + weights


def _decode(s):
    c = s["case"]
    k_q, k_d, v_q, v_d = s["planes"]
    B, G, Sq, S = c["B"], c["Hq"] // c["Hkv"], c["Sq"], c["S"]
    k, v = _values(k_q, k_d), _values(v_q, v_d)
    q = s["q"].float().reshape(B, c["Hkv"], G * Sq, c["D"])
    x = (q @ k.transpose(-1, -2)).reshape(B, c["Hkv"], G, Sq, S) / math.sqrt(c["D"])
    at = s["lengths"][:, None] - Sq + torch.arange(Sq, device="cuda")       # position of each query token
    j = torch.arange(S, device="cuda")
    seen = j <= at[..., None]
    if c["window"] > 0:
        seen &= at[..., None] - j <= c["window"]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(x - top)
    l = p.sum(-1, keepdim=True)
    o = (p.reshape(B, c["Hkv"], G * Sq, S) @ v).reshape(B, c["Hkv"], G, Sq, c["D"]) / l.clamp(min=1e-37)
    lse = torch.where(l > 0, top + torch.log(l.clamp(min=1e-37)), torch.zeros_like(l))
    return o.reshape(B, c["Hq"], Sq, c["D"]).to(torch.bfloat16), lse.reshape(B, c["Hq"], Sq)


def _chunk_scores(s):
    """Scores of the chunk [B, Hkv, G, Sq, Sk], hidden pairs at -inf, with K and V. The training path is defined on the
    cache's values rounded to bf16, as it is for every other cache of the framework."""
    c = s["case"]
    k_q, k_d, v_q, v_d = s["planes"]
    k, v = (_values(q, d).to(torch.bfloat16).float() for q, d in ((k_q, k_d), (v_q, v_d)))
    G = c["Hq"] // c["Hkv"]
    q = s["q"].float().reshape(c["B"], c["Hkv"], G * c["Sq"], c["D"])
    x = (q @ k.transpose(-1, -2)).reshape(c["B"], c["Hkv"], G, c["Sq"], c["Sk"])
    x = x.mul_(1 / math.sqrt(c["D"]))
    i = torch.arange(c["Sq"], device="cuda") + (c["Sk"] - c["Sq"])
    hidden = torch.arange(c["Sk"], device="cuda") > i[:, None]
    if s["mask"] is not None:
        hidden = hidden | (s["mask"][0] == 0)
    return x.masked_fill_(hidden, -math.inf), q, k, v


def _chunk_fwd(s):
    c = s["case"]
    x, q, k, v = _chunk_scores(s)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = x.sub_(top).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).reshape(c["B"], c["Hkv"], -1, c["Sq"], c["D"]) / l.clamp(min=1e-37)
    lse = torch.where(l > 0, top + torch.log(l.clamp(min=1e-37)), torch.zeros_like(l))
    shape = (c["B"], c["Hq"], c["Sq"])
    return o.reshape(*shape, c["D"]).to(torch.bfloat16), lse.reshape(shape)


def _chunk_bwd(s):
    c = s["case"]
    x, q, k, v = _chunk_scores(s)
    rows = (c["B"], c["Hkv"], -1, c["D"])
    p = x.sub_(s["lse"].reshape(*x.shape[:-1], 1)).exp_().flatten(2, 3)
    do, o = s["do"].float().reshape(rows), s["o"].float().reshape(rows)
    dv = p.transpose(-1, -2) @ do
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(1 / math.sqrt(c["D"]))
    dq = (ds @ k).reshape(c["B"], c["Hq"], c["Sq"], c["D"])
    dk = ds.transpose(-1, -2) @ q
    return [t.to(torch.bfloat16) for t in (dq, dk, dv)]


def _write_read(s):
    c = s["case"]
    rows = slice(s["begin"], s["begin"] + c["n"])
    for i, x in ((0, s["k"]), (2, s["v"])):
        q, d = _quantise(x, c["fmt"])
        s["planes"][i][:, :, rows] = q
        s["planes"][i + 1][:, :, rows] = d
    k_q, k_d, v_q, v_d = (t[:, :, rows] for t in s["planes"])
    return [_values(k_q, k_d).to(torch.bfloat16), _values(v_q, v_d).to(torch.bfloat16)]


def _read(s):
    k_q, k_d, v_q, v_d = s["planes"]
    return [_values(k_q, k_d).to(DTYPES[s["case"]["dtype"]]), _values(v_q, v_d).to(DTYPES[s["case"]["dtype"]])]


PLAIN = dict(rope_fwd=_rope_fwd, rope_bwd=_rope_bwd, decode=_decode, chunk_fwd=_chunk_fwd, chunk_bwd=_chunk_bwd,
             write_read=_write_read, read=_read)


# ---- the framework's calls ---------------------------------------------------------------------------


def _own(s):
    import backward_adapter_gb300 as fa

    c = s["case"]
    op = c["op"]
    if op in ("rope_fwd", "rope_bwd"):
        kw = dict(q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, interleaved=c["interleaved"], factor=c["factor"],
                  layout="bhsd" if c["layout"] == "bhsd" else "bshd")
        if op == "rope_fwd":
            return fa.qk_norm_rope(s["q"], s["k"], s["inv_freq"], s["pos"], **kw)
        got = fa.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["inv_freq"], s["pos"], **kw)
        return got if c["norm"] else got[:2]
    if op == "write_read":
        fa.cache_write(s["k"], s["v"], *s["planes"], s["begin"])
        return fa.cache_read(*s["planes"], s["begin"], c["n"])
    if op == "read":
        return fa.cache_read(*s["planes"], dtype=DTYPES[c["dtype"]])
    if op == "decode":
        return fa.decode(s["q"], *s["planes"], s["lengths"], window=c["window"])
    if op == "chunk_fwd":
        return fa.fwd_q4(s["q"], *s["planes"], s["mask"], causal=True)
    return fa.bwd_q4(s["q"], *s["planes"], s["o"], s["lse"], s["do"], s["mask"], causal=True)


def run(state):
    if own:
        return list(_own(state))
    return list(PLAIN[state["case"]["op"]](state))


# ---- what a pass cannot do without -------------------------------------------------------------------


def work(case):
    c = case
    D = c["D"]
    if c["op"] in ("rope_fwd", "rope_bwd"):
        es = 2 if c["dtype"] == "bf16" else 4
        n = c["B"] * c["S"] * (c["Hq"] + c["Hkv"]) * D
        small = 8 * c["B"] * c["S"] + 2 * c["rot"] + (2 * D * es if c["norm"] else 0)
        if c["op"] == "rope_fwd":
            return {"bytes": 2 * n * es + small, "flops": 8 * n}
        # the gradient of a rotation alone does not need its input
        return {"bytes": (3 if c["norm"] else 2) * n * es + small + (8 * D if c["norm"] else 0), "flops": 16 * n}
    if c["op"] in ("write_read", "read"):
        es = 2 if c["dtype"] == "bf16" else 4
        n = 2 * c["B"] * c["Hkv"] * c.get("n", c["S"]) * D
        held = n // 2 if c["fmt"] == "q4_0" else n
        held += n // BLOCK * 2
        if c["op"] == "read":
            return {"bytes": held + n * es, "flops": 2 * n}
        return {"bytes": 2 * held + n * (es + 2), "flops": 6 * n}
    if c["op"] == "decode":
        lens = torch.linspace(c["hi"], c["lo"], c["B"], dtype=torch.float64).round().to(torch.int64)
        if c["empty"]:
            lens[-1] = 0
        used = lens.clamp(max=c["window"] + c["Sq"]) if c["window"] > 0 else lens
        keys = int(used.sum()) * c["Hkv"]
        per = 2 * (D // 2 if c["fmt"] == "q4_0" else D) + 2 * 2 * (D // BLOCK)
        rows = c["B"] * c["Hq"] * c["Sq"]
        return {"bytes": keys * per + rows * (4 * D + 4) + 8 * c["B"], "flops": 4 * D * int(used.sum()) * c["Hq"] * c["Sq"]}
    pairs = c["B"] * c["Hq"] * (c["Sq"] * c["Sk"] - c["Sq"] * (c["Sq"] - 1) // 2)
    held = 2 * c["B"] * c["Hkv"] * c["Sk"] * (D // 2 + D // BLOCK * 2) + (c["Sq"] * c["Sk"] if c["mask"] else 0)
    rows = c["B"] * c["Hq"] * c["Sq"]
    if c["op"] == "chunk_fwd":
        return {"bytes": held + rows * (4 * D + 4), "flops": 4 * D * pairs}
    return {"bytes": held + rows * (8 * D + 4) + 4 * c["B"] * c["Hkv"] * c["Sk"] * D, "flops": 10 * D * pairs}


# ---- the definitions in 64 bits ----------------------------------------------------------------------


def _held64(q, d):
    """float64 values of quantised planes, by the definition of the formats."""
    D = d.shape[-1] * BLOCK
    out = torch.empty((*d.shape[:-1], D), dtype=torch.float64, device=q.device)
    for f in range(D):
        if q.dtype == torch.uint8:
            byte = q[..., f // 32 * 16 + f % 16].to(torch.int32)
            n = (byte // 16 if f % 32 >= 16 else byte % 16) - 8
        else:
            n = q[..., f].to(torch.int32)
        out[..., f] = n.double() * d[..., f // 32].double()
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


def _complex(x, c):
    """The rotated features as complex numbers, and the others."""
    r = c["rot"]
    t = x[..., :r]
    z = torch.view_as_complex(t.unflatten(-1, (-1, 2)).contiguous()) if c["interleaved"] else \
        torch.complex(t[..., :r // 2].contiguous(), t[..., r // 2:].contiguous())
    return z, x[..., r:]


def _real(z, rest, c):
    t = torch.view_as_real(z).flatten(-2) if c["interleaved"] else torch.cat([z.real, z.imag], -1)
    return torch.cat([t, rest], -1)


def _rope64(s):
    c = s["case"]
    turn = torch.outer(s["pos"].double().flatten(), s["inv_freq"].double()).reshape(c["B"], c["S"], -1)
    turn = torch.polar(torch.full_like(turn, c["factor"]), turn)
    turn = turn.unsqueeze(1 if c["layout"] == "bhsd" else 2)
    first, second = [], []
    for name in ("q", "k"):
        x, w = s[name].double(), s[name + "w"]
        scale = 1 / (x.pow(2).sum(-1, keepdim=True) / c["D"] + 1e-6).sqrt()
        if c["op"] == "rope_fwd":
            z, rest = _complex(x * scale * w.double() if w is not None else x, c)
            first.append(_real(z * turn, rest, c))
            continue
        z, rest = _complex(s["d" + name].double(), c)
        g = _real(z * turn.conj(), rest, c)
        if w is None:
            first.append(g)
            continue
        h = g * w.double()
        first.append(scale * h - x * scale.pow(3) * (h * x).sum(-1, keepdim=True) / c["D"])
        second.append((g * x * scale).flatten(0, 2).sum(0))
    return first + second


def _attend64(q, k, v, seen, scale):
    """(o, lse) of one key/value head: q [rows, D], seen [rows, keys]."""
    x = torch.where(seen, scale * (q @ k.T), torch.full((), -math.inf, dtype=torch.float64, device=q.device))
    lse = torch.logsumexp(x, -1)
    p = torch.where(seen, torch.exp(x - torch.where(lse.isinf(), torch.zeros_like(lse), lse)[:, None]), torch.zeros_like(x))
    return p @ v, torch.where(lse.isinf(), torch.zeros_like(lse), lse)


def _decode64(s):
    c = s["case"]
    G, Sq = c["Hq"] // c["Hkv"], c["Sq"]
    o = torch.zeros((c["B"], c["Hq"], Sq, c["D"]), dtype=torch.float64, device="cuda")
    lse = torch.zeros((c["B"], c["Hq"], Sq), dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lengths"].tolist()):
        if n == 0:
            continue
        k, v = _held64(*(t[b, :, :n] for t in s["planes"][:2])), _held64(*(t[b, :, :n] for t in s["planes"][2:]))
        back = n - Sq + torch.arange(Sq, device="cuda")[:, None] - torch.arange(n, device="cuda")   # keys before the token
        seen = (back >= 0) & (back <= c["window"] if c["window"] else back >= 0)
        for h in range(c["Hkv"]):
            heads = slice(h * G, h * G + G)
            got = _attend64(s["q"][b, heads].double().flatten(0, 1), k[h], v[h], seen.repeat(G, 1), c["D"] ** -0.5)
            o[b, heads], lse[b, heads] = got[0].reshape(G, Sq, -1), got[1].reshape(G, Sq)
    return [o, lse]


def _chunk64(s):
    c = s["case"]
    G, scale = c["Hq"] // c["Hkv"], c["D"] ** -0.5
    shape = (c["B"], c["Hq"], c["Sq"])
    out = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.empty((*shape, c["D"]), **out), torch.empty(shape, **out)
    dq = torch.empty((*shape, c["D"]), **out)
    dk, dv = (torch.empty((c["B"], c["Hkv"], c["Sk"], c["D"]), **out) for _ in range(2))
    back = (c["Sk"] - c["Sq"]) + torch.arange(c["Sq"], device="cuda")[:, None] - torch.arange(c["Sk"], device="cuda")
    seen = back >= 0
    if s["mask"] is not None:
        seen = seen & s["mask"][0].bool()
    for b in range(c["B"]):
        for h in range(c["Hkv"]):
            k, v = (_held64(s["planes"][i][b, h], s["planes"][i + 1][b, h]).to(torch.bfloat16).double() for i in (0, 2))
            sk, sv = torch.zeros_like(k), torch.zeros_like(v)
            for n in range(h * G, h * G + G):
                q = s["q"][b, n].double()
                if c["op"] == "chunk_fwd":
                    o[b, n], lse[b, n] = _attend64(q, k, v, seen, scale)
                    continue
                p = torch.where(seen, torch.exp(scale * (q @ k.T) - s["lse"][b, n].double()[:, None]), 0.0)
                g = s["do"][b, n].double()
                d = p * (g @ v.T - (g * s["o"][b, n].double()).sum(-1, keepdim=True))
                dq[b, n] = scale * (d @ k)
                sk += scale * (d.T @ q)
                sv += p.T @ g
            dk[b, h], dv[b, h] = sk, sv
    return [o, lse] if c["op"] == "chunk_fwd" else [dq, dk, dv]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rope_fwd", "rope_bwd"):
        return _rope64(s)
    if case["op"] == "decode":
        return _decode64(s)
    if case["op"] in ("chunk_fwd", "chunk_bwd"):
        return _chunk64(s)
    if case["op"] == "write_read":
        return [_stored64(s["k"], case["fmt"]), _stored64(s["v"], case["fmt"])]
    k_q, k_d, v_q, v_d = s["planes"]
    return [_held64(k_q, k_d), _held64(v_q, v_d)]
