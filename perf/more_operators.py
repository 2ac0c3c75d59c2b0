"""Operators of a latent-attention layer around the latent rows, and the sizes they are measured at.

Operators that run one after another in a serving step of such a layer:
  add_rms_norm            residual addition and norm, in 16 bits or as E4M3 codes with scales
  latent_norm_rope_store  latent norm and rotary positions, one latent row a token into the cache
  latent_attention        attention over the rows that an index lists (a top-k selection)
  paged_latent_attention  a chunk of new tokens of each request over its paged latent rows

A latent row serves all query heads: 512 latent dims (keys and values) and 64 rotary dims (keys
only).  It is kept in 656 bytes (512 E4M3 codes, an fp32 scale for each 128 of them, 64 16-bit
rotary values) or as 576 16-bit values.

`own` selects the framework's calls; otherwise `run` computes the plain form.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
LATENT, ROPE, GROUP = 512, 64, 128
CODES, SCALES = LATENT, LATENT + 4 * (LATENT // GROUP)  # where a 656-byte row's scales and rotary values begin
ROW = SCALES + 2 * ROPE
EPS = 1e-6


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # a decode step's residual stream on its way into an 8-bit projection
        dict(name="norm, 32 tokens grouped", op="norm", tokens=32, dim=4096, dtype="bf16", residual=True, out=False, group=128),
        # an odd number of tokens, first layer (no residual yet), 16 bits for the router and codes with a scale a token
        dict(name="norm, 4097 tokens both", op="norm", tokens=4097, dim=2304, dtype="f16", residual=False, out=True, group=0),
        # the residual stream of several long prompts
        dict(name="norm, 16384 tokens grouped", op="norm", tokens=16384, dim=4096, dtype="bf16", residual=True, out=False, group=128),
        # a decode step's new latent rows, query heads split over GPUs
        dict(name="rows, 32 tokens", op="rows", tokens=32, heads=16, dtype="bf16", cache="fp8", inter=True, max_pos=131072),
        # a chunk of prompts with all query heads, the scatter benchmark's 4096 tokens with one more
        dict(name="rows, 4097 tokens 128 heads", op="rows", tokens=4097, heads=128, dtype="bf16", cache="fp8", inter=True, max_pos=131072),
        # long prompts into 16-bit rows
        dict(name="rows, 16384 tokens 16-bit", op="rows", tokens=16384, heads=16, dtype="f16", cache="same", inter=False, max_pos=32768),
        # two requests of a quiet server over their selected rows: latency
        dict(name="index, 2 tokens", op="index", tokens=2, heads=16, top_k=2048, hot=4096, dtype="bf16", cache="fp8", empty=0, sharp=2.0),
        # the decode-step benchmark: 32 requests, top-k 2048 in a hot buffer of 4096, all query heads
        dict(name="index, 32 tokens 128 heads", op="index", tokens=32, heads=128, top_k=2048, hot=4096, dtype="bf16", cache="fp8", empty=0, sharp=2.0),
        # the large batch of the stress benchmark, heads split over GPUs, some sequences shorter than the selection
        dict(name="index, 128 tokens 16 heads", op="index", tokens=128, heads=16, top_k=2048, hot=2048, dtype="bf16", cache="fp8", empty=1900, sharp=2.0),
        # a dense decode batch over long ragged contexts
        dict(name="paged, decode of 32", op="paged", batch=32, q_lo=1, q_hi=1, ctx_lo=2049, ctx_hi=16384, heads=16, dtype="bf16", cache="fp8", page=64, sharp=2.0),
        # drafted tokens under verification, all heads, 16-bit rows
        dict(name="paged, drafts 16-bit", op="paged", batch=13, q_lo=1, q_hi=4, ctx_lo=17, ctx_hi=4096, heads=128, dtype="bf16", cache="same", page=16, sharp=2.0),
        # chunked prompts of a few requests
        dict(name="paged, chunks", op="paged", batch=3, q_lo=129, q_hi=513, ctx_lo=0, ctx_hi=4099, heads=16, dtype="bf16", cache="fp8", page=64, sharp=2.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "rows", "index", "index", "paged", "paged"])
    dtype = rng.choice(["f16", "bf16", "bf16"])
    cache = rng.choice(["fp8", "fp8", "same"])
    heads = rng.choice([1, 2, 4, 8, 12, 16, 20, 32, 64, 128])
    if op == "norm":
        tokens, dim = _log(rng, 1, 16384), rng.choice([8, 16, 128]) * rng.randint(1, 64)
        while tokens * dim > 16384 * 4096:
            tokens = tokens * 3 // 4
        return dict(op=op, tokens=tokens, dim=dim, dtype=dtype, residual=rng.random() < 0.7, out=rng.random() < 0.5, group=rng.choice([0, 128]))
    if op == "rows":
        tokens = _log(rng, 1, 16384)
        while tokens * (heads + 9) > 4097 * 137:
            tokens = tokens * 3 // 4
        return dict(op=op, tokens=tokens, heads=heads, dtype=dtype, cache=cache, inter=rng.random() < 0.5, max_pos=_log(rng, 4096, 131072))
    if op == "index":
        tokens, top_k = _log(rng, 1, 128), _log(rng, 1, 2048)
        while tokens * top_k * max(heads, 16) > 32 * 2048 * 128:
            tokens = max(1, tokens * 3 // 4)
        hot = top_k + rng.randint(0, top_k)
        return dict(op=op, tokens=tokens, heads=heads, top_k=top_k, hot=hot, dtype=dtype, cache=cache, empty=rng.choice([0, rng.randint(0, top_k)]), sharp=rng.choice([1.0, 2.0]))
    batch = _log(rng, 1, 64)
    q_hi = 1 if rng.random() < 0.5 else _log(rng, 2, 513)
    ctx_hi = _log(rng, 1, 16384)
    while batch * q_hi * (q_hi // 2 + ctx_hi) * heads > 13_000_000 or batch * (q_hi + ctx_hi) > 32 * 9217:
        batch, q_hi, ctx_hi = max(1, batch * 3 // 4), max(1, q_hi * 7 // 8), max(1, ctx_hi * 7 // 8)
    return dict(op=op, batch=batch, q_lo=rng.randint(1, q_hi), q_hi=q_hi, ctx_lo=rng.randint(0, ctx_hi), ctx_hi=ctx_hi, heads=heads, dtype=dtype, cache=cache, page=rng.choice([1, 16, 48, 64, 128]), sharp=rng.choice([1.0, 2.0]))


def _ladder(lo, hi, n, step):
    """n whole numbers from lo to hi, spread by a stride so that neighbours differ; the same for every seed."""
    return [lo + (hi - lo) * ((i * step) % n) // max(1, n - 1) for i in range(n)]


def _lengths(case):
    """Each request's (context, new tokens), in an order that the seed changes later."""
    n = case["batch"]
    return list(zip(_ladder(case["ctx_lo"], case["ctx_hi"], n, 7), _ladder(case["q_lo"], case["q_hi"], n, 3)))


def _empties(case):
    """How many entries of each token's selection are empty: of every fourth token up to `empty`."""
    t = case["tokens"]
    return [case["empty"] * (i + 1) // t if i % 4 == 3 else 0 for i in range(t)]


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    host = np.random.default_rng(seed)
    return {"norm": _prepare_norm, "rows": _prepare_rows, "index": _prepare_index, "paged": _prepare_paged}[case["op"]](case, g, host)


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _prepare_norm(case, g, host):
    t, d, dt = case["tokens"], case["dim"], DTYPES[case["dtype"]]
    groups = -(-d // case["group"]) if case["group"] else 1
    # a stream whose channels differ in size, as they do behind some layers
    wide = torch.exp(_randn(g, d))
    state = dict(case=case, x=(_randn(g, t, d) * wide).to(dt), weight=(1 + 0.2 * _randn(g, d)).to(dt), residual=None, residual_out=None, out=None,
                 codes=torch.zeros(t, d, dtype=torch.float8_e4m3fn, device="cuda"), scales=torch.zeros(t, groups, device="cuda"))
    if case["residual"]:
        state["residual"] = (4 * _randn(g, t, d) * wide).to(dt)
        state["residual_out"] = torch.zeros_like(state["x"])
    if case["out"]:
        state["out"] = torch.zeros_like(state["x"])
    return state


def _latent_rows(n, case, g):
    """n latent rows as a cache holds them: normed latents with channels of different size, rotated keys."""
    dt = DTYPES[case["dtype"]]
    wide = torch.exp(0.5 * _randn(g, LATENT))
    rows = torch.empty(n, ROW, dtype=torch.uint8, device="cuda") if case["cache"] == "fp8" else torch.empty(n, LATENT + ROPE, dtype=dt, device="cuda")
    for a in range(0, n, 1 << 17):
        part = rows[a: a + (1 << 17)]
        x, pe = _randn(g, part.shape[0], LATENT) * wide, _randn(g, part.shape[0], ROPE)
        if case["cache"] == "fp8":
            x = x.view(-1, LATENT // GROUP, GROUP)
            scale = x.abs().amax(-1, keepdim=True) / 448
            part[:, :CODES] = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, LATENT)
            part[:, CODES:SCALES] = scale.view(-1, LATENT // GROUP).view(torch.uint8)
            part[:, SCALES:] = pe.to(dt).view(torch.uint8)
        else:
            part[:, :LATENT] = x.to(dt)
            part[:, LATENT:] = pe.to(dt)
    return rows


def _queries(t, case, g):
    # scores of a standard deviation of about `sharp`
    q = _randn(g, t, case["heads"], LATENT + ROPE)
    return (case["sharp"] * q).to(DTYPES[case["dtype"]])


def _scale():
    """One over the root of what the squares of a row sum up to: the wide channels' mean square is e^0.5."""
    return (LATENT * math.exp(0.5) + ROPE) ** -0.5


def _prepare_rows(case, g, host):
    t, h, dt = case["tokens"], case["heads"], DTYPES[case["dtype"]]
    half = ROPE // 2
    inv = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    ang = torch.arange(case["max_pos"], device="cuda", dtype=torch.float64)[:, None] * inv
    slots = 2 * t + 1
    # the down-projection's output holds latent and rotary key side by side, the queries' rotary part lies behind their
    # 128 other dims
    return dict(case=case, kv=(_randn(g, t, LATENT + ROPE) * torch.exp(_randn(g, t, 1))).to(dt), q=_randn(g, t, h, 2 * ROPE + ROPE).to(dt),
                weight=(1 + 0.2 * _randn(g, LATENT)).to(dt), cos_sin=torch.cat([ang.cos(), ang.sin()], 1).float(),
                positions=torch.randint(0, case["max_pos"], (t,), generator=g, device="cuda"),
                loc=torch.randperm(slots, generator=g, device="cuda")[:t], rows=_latent_rows(slots, case, g),
                q_all=torch.zeros(t, h, LATENT + ROPE, dtype=dt, device="cuda"), status=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _prepare_index(case, g, host):
    t, k, hot = case["tokens"], case["top_k"], case["hot"]
    # every token's request has hot + 1 rows of the buffer, and its selection is some of them
    index = np.stack([i * (hot + 1) + host.permutation(hot + 1)[:k] for i in range(t)]).astype(np.int32)
    for i, n in enumerate(_empties(case)):
        index[i, host.permutation(k)[:n]] = -1
    return dict(case=case, q=_queries(t, case, g), rows=_latent_rows(t * (hot + 1), case, g), index=_cuda(index),
                out=torch.zeros(t, case["heads"], LATENT, dtype=DTYPES[case["dtype"]], device="cuda"),
                status=torch.zeros(t, dtype=torch.int32, device="cuda"))


def _prepare_paged(case, g, host):
    ps = case["page"]
    lens = _lengths(case)
    order = host.permutation(len(lens))
    new = np.array([lens[i][1] for i in order], np.int64)
    seq = np.array([lens[i][0] for i in order], np.int64) + new
    held = -(-seq // ps)
    pages = int(held.sum()) + 3
    perm = host.permutation(pages).astype(np.int32)
    states = len(lens) + 2
    req = host.permutation(states)[: len(lens)]
    table = np.full((states, int(held.max()) + 1), -1, np.int32)
    at = 0
    for r, n in zip(req, held):
        table[r, :n] = perm[at: at + n]
        at += n
    t = int(new.sum())
    return dict(case=case, q=_queries(t, case, g), rows=_latent_rows(pages * ps, case, g), block_table=_cuda(table),
                req_state=_cuda(req.astype(np.int64)), cu_q=_cuda(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)),
                seq_lens=_cuda(seq.astype(np.int32)), max_q_len=int(new.max()),
                out=torch.zeros(t, case["heads"], LATENT, dtype=DTYPES[case["dtype"]], device="cuda"),
                status=torch.zeros(len(lens), dtype=torch.int32, device="cuda"))


# ---------------------------------------------------------------- one pass
def run(s):
    return {"norm": _run_norm, "rows": _run_rows, "index": _run_index, "paged": _run_paged}[s["case"]["op"]](s)


def _run_norm(s):
    c = s["case"]
    if own:
        import sparse_attention_kv_row_gb300 as hs
        hs.add_rms_norm(s["x"], s["weight"], s["out"], residual=s["residual"], residual_out=s["residual_out"], eps=EPS,
                        codes=s["codes"], scales=s["scales"], group=c["group"])
    else:
        _plain_norm(s)
    return {k: s[k] for k in ("residual_out", "out", "codes", "scales") if s[k] is not None}


def _plain_norm(s):
    c, x = s["case"], s["x"]
    if s["residual"] is not None:
        x = (x.float() + s["residual"].float()).to(x.dtype)
        s["residual_out"].copy_(x)
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    if s["out"] is not None:
        s["out"].copy_(y)
    t, d = y.shape
    n = c["group"] or d
    groups = -(-d // n)
    padded = torch.zeros(t, groups * n, device=y.device)
    padded[:, :d] = y
    padded = padded.view(t, groups, n)
    scale = padded.abs().amax(-1) * (1.0 / 448)
    inverse = torch.where(scale > 0, 1.0 / scale, 0.0)
    s["codes"].copy_((padded * inverse[..., None]).clamp(-448, 448).view(t, -1)[:, :d].to(torch.float8_e4m3fn))
    s["scales"].copy_(scale)


def _run_rows(s):
    kv, q = s["kv"], s["q"]
    latent, k_pe, q_pe, q_out = kv[:, :LATENT], kv[:, LATENT:], q[..., 2 * ROPE:], s["q_all"][..., LATENT:]
    if own:
        import sparse_attention_kv_row_gb300 as hs
        hs.latent_norm_rope_store(latent, k_pe, s["weight"], s["cos_sin"], s["positions"], s["rows"], s["loc"],
                                  q_pe=q_pe, q_out=q_out, eps=EPS, interleaved=s["case"]["inter"], status=s["status"])
    else:
        _plain_rows(s, latent, k_pe, q_pe, q_out)
    return {"q_out": q_out, **_parts(s["rows"], s["case"])}


def _parts(rows, case):
    """What a cache's rows hold: 16-bit values, or codes, scales and rotary values."""
    if case["cache"] != "fp8":
        return {"rows": rows}
    return {"codes": rows[:, :CODES].view(torch.float8_e4m3fn), "scales": rows.view(torch.float32)[:, CODES // 4: SCALES // 4],
            "rope": rows.view(DTYPES[case["dtype"]])[:, SCALES // 2:]}


def _plain_turn(x, cos, sin, inter):
    """Pairs (2i, 2i+1), or (i, i + half), turned."""
    half = ROPE // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :half], x[..., half:])
    both = (a * cos - b * sin, b * cos + a * sin)
    return torch.stack(both, -1).flatten(-2) if inter else torch.cat(both, -1)


def _plain_rows(s, latent, k_pe, q_pe, q_out):
    c, rows, loc = s["case"], s["rows"], s["loc"]
    cs = s["cos_sin"][s["positions"]]
    cos, sin = cs[:, : ROPE // 2], cs[:, ROPE // 2:]
    q_out.copy_(_plain_turn(q_pe.float(), cos[:, None], sin[:, None], c["inter"]))
    pe = _plain_turn(k_pe.float(), cos, sin, c["inter"]).to(k_pe.dtype)
    x = latent.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    if c["cache"] != "fp8":
        rows[loc] = torch.cat([x.to(rows.dtype), pe], 1)
        return
    x = x.view(-1, LATENT // GROUP, GROUP)
    scale = x.abs().amax(-1, keepdim=True) * (1.0 / 448)
    code = (x * torch.where(scale > 0, 1.0 / scale, 0.0)).clamp(-448, 448).to(torch.float8_e4m3fn).view(-1, LATENT)
    rows[loc] = torch.cat([code.view(torch.uint8), scale.view(-1, LATENT // GROUP).view(torch.uint8), pe.view(torch.uint8)], 1)


def _widened(rows, case):
    """Rows as 576 values in 32 bits."""
    if case["cache"] != "fp8":
        return rows.float()
    p = _parts(rows.reshape(-1, ROW), case)
    x = p["codes"].float().view(-1, LATENT // GROUP, GROUP) * p["scales"][..., None]
    return torch.cat([x.view(-1, LATENT), p["rope"].float()], 1).view(*rows.shape[:-1], LATENT + ROPE)


def _plain_softmax(p, seen):
    """Weights of the scores p where `seen`; rows that see nothing get zeros."""
    p = p.masked_fill(~seen, -math.inf)
    m = p.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(p - m)
    return p / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _run_index(s):
    if own:
        import sparse_attention_kv_row_gb300 as hs
        hs.latent_attention(s["q"], s["rows"], s["index"], s["out"], scale=_scale(), status=s["status"])
    else:
        kv = _widened(s["rows"][s["index"].clamp(min=0).long()], s["case"])
        p = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * _scale()
        s["out"].copy_(torch.matmul(_plain_softmax(p, (s["index"] >= 0)[:, None]), kv[..., :LATENT]))
    return s["out"]


def _run_paged(s):
    if own:
        import sparse_attention_kv_row_gb300 as hs
        hs.paged_latent_attention(s["q"], s["rows"], s["block_table"], s["req_state"], s["cu_q"], s["seq_lens"], s["out"],
                                  max_q_len=s["max_q_len"], page_size=s["case"]["page"], scale=_scale(), status=s["status"])
    else:
        _plain_paged(s)
    return s["out"]


def _plain_paged(s):
    """Every request padded to the longest; rows gathered through the block table; one softmax over them."""
    c = s["case"]
    cu, seq = s["cu_q"].long(), s["seq_lens"].long()
    new = cu[1:] - cu[:-1]
    batch, h, device = seq.numel(), c["heads"], cu.device
    table = s["block_table"][s["req_state"]].long().clamp(min=0)
    kv = _widened(s["rows"].view(-1, c["page"], s["rows"].shape[1])[table].flatten(1, 2), c)
    n = kv.shape[1]
    row = torch.arange(s["q"].shape[0], device=device)
    b = torch.searchsorted(cu[1:], row, right=True)
    i = row - cu[b]
    q = torch.zeros(batch, s["max_q_len"], h, LATENT + ROPE, device=device)
    q[b, i] = s["q"].float()
    p = torch.matmul(q.flatten(1, 2), kv.transpose(1, 2)).mul_(_scale()).view(batch, -1, h, n)
    pos = (seq - new)[:, None] + torch.arange(s["max_q_len"], device=device)
    seen = torch.arange(n, device=device) <= pos[..., None]
    seen &= (torch.arange(n, device=device) < seq[:, None])[:, None]
    o = torch.matmul(_plain_softmax(p, seen[:, :, None]).flatten(1, 2), kv[..., :LATENT])
    s["out"].copy_(o.view(batch, -1, h, LATENT)[b, i])


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    wide = 2
    if case["op"] == "norm":
        t, d = case["tokens"], case["dim"]
        groups = -(-d // case["group"]) if case["group"] else 1
        streams = 1 + 2 * case["residual"] + case["out"]
        return {"bytes": t * (d * (streams * wide + 1) + groups * 4) + d * wide, "flops": t * d * 8}
    row = ROW if case["cache"] == "fp8" else (LATENT + ROPE) * wide
    h = case["heads"]
    if case["op"] == "rows":
        t = case["tokens"]
        # latent and rotary key in, a row out; the queries' rotary part in and out; slot, position and angles
        return {"bytes": t * ((LATENT + ROPE) * wide + row + 2 * h * ROPE * wide + 16 + ROPE * 4) + LATENT * wide,
                "flops": t * (6 * LATENT + 3 * ROPE * (h + 1))}
    if case["op"] == "index":
        t, k = case["tokens"], case["top_k"]
        keys = pairs = t * k - sum(_empties(case))
        meta = t * k * 4
    else:
        lens = _lengths(case)
        keys = sum(c + q for c, q in lens)
        pairs = sum(q * c + q * (q + 1) // 2 for c, q in lens)
        t, meta = sum(q for _, q in lens), -(-keys // case["page"]) * 4
    return {"bytes": keys * row + meta + t * h * (2 * LATENT + ROPE) * wide, "flops": 2 * pairs * h * (2 * LATENT + ROPE)}


# ---------------------------------------------------------------- 64 bits, token by token
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "rows": _exact_rows, "index": _exact_index, "paged": _exact_paged}[case["op"]](s)


def _unit(x, weight):
    x = x.double()
    return x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) * weight.double()


def _coded(y, n):
    """(values that become codes, scales) of rows in groups of n."""
    parts = [(p / sc.clamp(min=1e-300), sc) for p in y.split(n, -1) for sc in (p.abs().amax(-1, keepdim=True) / 448,)]
    return torch.cat([p for p, _ in parts], -1), torch.cat([sc for _, sc in parts], -1)


def _exact_norm(s):
    c, x = s["case"], s["x"]
    got = {}
    if c["residual"]:
        x = (x.double() + s["residual"].double()).to(x.dtype)  # the sum is rounded to the stream's type
        got["residual_out"] = x.double()
    y = _unit(x, s["weight"])
    if c["out"]:
        got["out"] = y
    got["codes"], got["scales"] = _coded(y, c["group"] or c["dim"])
    return got


def _exact_turn(x, angle, inter):
    x = x.double()
    pair = x.unflatten(-1, (-1, 2)) if inter else x.unflatten(-1, (2, -1)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * angle)
    return z.flatten(-2) if inter else z.transpose(-1, -2).flatten(-2)


def _exact_rows(s):
    c = s["case"]
    cs = s["cos_sin"].double()[s["positions"]]
    angle = torch.complex(cs[:, : ROPE // 2].contiguous(), cs[:, ROPE // 2:].contiguous())
    got = {"q_out": _exact_turn(s["q"][..., 2 * ROPE:], angle[:, None], c["inter"])}
    latent, pe = _unit(s["kv"][:, :LATENT], s["weight"]), _exact_turn(s["kv"][:, LATENT:], angle, c["inter"])
    old = {k: v.double() for k, v in _parts(s["rows"], c).items()}
    if c["cache"] == "fp8":
        new = dict(zip(("codes", "scales"), _coded(latent, GROUP)), rope=pe)
    else:
        new = {"rows": torch.cat([latent, pe], 1)}
    for k, v in new.items():
        old[k][s["loc"]] = v
    return got | old


def _exact_values(rows, c):
    if c["cache"] != "fp8":
        return rows.double()
    p = _parts(rows, c)
    return torch.cat([p["codes"].double() * p["scales"].double().repeat_interleave(GROUP, 1), p["rope"].double()], 1)


def _exact_attend(q, kv, hidden=None):
    """One softmax of q [t, heads, 576] over kv [n, 576], without the pairs in `hidden` [t, n]."""
    z = torch.einsum("thd,nd->thn", q.double(), kv) * _scale()
    if hidden is not None:
        z.masked_fill_(hidden[:, None], -math.inf)
    return torch.einsum("thn,nd->thd", torch.softmax(z, -1), kv[:, :LATENT])


def _exact_index(s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for i, at in enumerate(s["index"]):
        at = at[at >= 0].long()
        if at.numel():
            out[i] = _exact_attend(s["q"][i: i + 1], _exact_values(s["rows"][at], s["case"]))[0]
    return out


def _exact_paged(s):
    c = s["case"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    cu, seq = s["cu_q"].tolist(), s["seq_lens"].tolist()
    for b, r in enumerate(s["req_state"].tolist()):
        n, a, e = seq[b], cu[b], cu[b + 1]
        pages = s["block_table"][r, : -(-n // c["page"])].long()
        at = (pages[:, None] * c["page"] + torch.arange(c["page"], device="cuda")).flatten()[:n]
        kv = _exact_values(s["rows"][at], c)
        for t in range(a, e, 64):  # some queries at a time
            u = min(e, t + 64)
            gap = torch.arange(n - e + t, n - e + u, device="cuda")[:, None] - torch.arange(n, device="cuda")
            out[t:u] = _exact_attend(s["q"][t:u], kv, gap < 0)
    return out
