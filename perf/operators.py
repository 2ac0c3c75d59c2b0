"""Serving operators around the paged KV cache, and the sizes they are measured at.

Three operators that run one after another in a serving step:
  assign_slots        block tables and slot maps from the requests' lengths
  qk_norm_rope_store  per-head norm and rotary positions, K/V into the paged cache
  paged_attention     a chunk of new tokens of each request over the paged cache

`own` selects the framework's calls; otherwise `run` computes the plain form.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of 32 requests: every request gets one token, a few cross into a new block
        dict(name="slots, decode of 32", op="slots", batch=32, new_lo=1, new_hi=1, ctx_hi=131072, block=64, pad=2),
        # a long ragged batch: prompts, chunks and single tokens together, small blocks
        dict(name="slots, 1000 ragged", op="slots", batch=1000, new_lo=0, new_hi=257, ctx_hi=4001, block=16, pad=24),
        # a decode step's new tokens, one per request
        dict(name="norm, 32 tokens bf16", op="norm", tokens=32, heads=32, kv_heads=8, dim=128, rot=128, inter=False, dtype="bf16", cache="same", page=64, max_pos=131072),
        # the scatter benchmark's 4096 tokens with one more, half the head rotated in pairs, into an FP8 cache
        dict(name="norm, 4097 tokens fp8", op="norm", tokens=4097, heads=24, kv_heads=8, dim=64, rot=32, inter=True, dtype="f16", cache="fp8", page=16, max_pos=32768),
        # the new tokens of several long prompts
        dict(name="norm, 16384 tokens bf16", op="norm", tokens=16384, heads=32, kv_heads=8, dim=128, rot=128, inter=False, dtype="bf16", cache="same", page=64, max_pos=131072),
        # two requests of a quiet server: latency
        dict(name="attention, decode of 2", op="attn", batch=2, q_lo=1, q_hi=1, ctx_lo=300, ctx_hi=1024, heads=32, kv_heads=8, dim=128, dtype="bf16", cache="same", page=16, window=0, sharp=2.0),
        # a full decode batch over long ragged contexts
        dict(name="attention, decode of 32", op="attn", batch=32, q_lo=1, q_hi=1, ctx_lo=2049, ctx_hi=16384, heads=32, kv_heads=8, dim=128, dtype="bf16", cache="same", page=64, window=0, sharp=2.0),
        # a large decode batch over an FP8 cache
        dict(name="attention, decode of 128 fp8", op="attn", batch=128, q_lo=1, q_hi=1, ctx_lo=100, ctx_hi=8192, heads=32, kv_heads=8, dim=128, dtype="bf16", cache="fp8", page=64, window=0, sharp=2.0),
        # drafted tokens under verification: one to five a request, a sliding window, three queries to a head
        dict(name="attention, drafts windowed", op="attn", batch=61, q_lo=1, q_hi=5, ctx_lo=17, ctx_hi=4096, heads=12, kv_heads=4, dim=64, dtype="f16", cache="same", page=32, window=1000, sharp=2.0),
        # chunked prefill and decode in one batch, FP8 cache
        dict(name="attention, mixed fp8", op="attn", batch=19, q_lo=1, q_hi=513, ctx_lo=0, ctx_hi=4099, heads=32, kv_heads=8, dim=128, dtype="bf16", cache="fp8", page=16, window=0, sharp=2.0),
        # four prompts from their first token
        dict(name="attention, 4 prompts", op="attn", batch=4, q_lo=2048, q_hi=2048, ctx_lo=0, ctx_hi=0, heads=32, kv_heads=8, dim=128, dtype="bf16", cache="same", page=64, window=0, sharp=2.0),
        # the next chunk of two long prompts
        dict(name="attention, 2 long chunks", op="attn", batch=2, q_lo=2048, q_hi=2048, ctx_lo=14336, ctx_hi=16384, heads=32, kv_heads=8, dim=128, dtype="bf16", cache="same", page=64, window=0, sharp=2.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["slots", "norm", "attn", "attn"])
    if op == "slots":
        batch = _log(rng, 1, 1000)
        hi = _log(rng, 1, 513)
        while batch * hi > 260000:
            hi = hi // 2 + 1
        return dict(op=op, batch=batch, new_lo=rng.randint(0, 1), new_hi=hi, ctx_hi=_log(rng, 1, 131072), block=rng.choice([1, 8, 16, 32, 48, 64, 128]), pad=rng.randint(0, batch // 4))
    dim = rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 6, 8])
    dtype = rng.choice(["f16", "bf16"])
    cache = rng.choice(["same", "fp8"])
    page = rng.choice([1, 8, 16, 32, 48, 64, 128])
    if op == "norm":
        tokens = _log(rng, 1, 16384)
        while tokens * (heads + 2 * kv_heads) * dim > 16384 * 48 * 128:
            tokens = tokens * 3 // 4
        return dict(op=op, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim, rot=rng.choice([dim // 2, dim]), inter=rng.random() < 0.5, dtype=dtype, cache=cache, page=page, max_pos=_log(rng, 4096, 131072))
    batch = _log(rng, 1, 128)
    q_hi = 1 if rng.random() < 0.4 else _log(rng, 2, 2048)
    ctx_hi = _log(rng, 1, 16384)
    while batch * q_hi * (q_hi + ctx_hi) * heads > 2 * 2048 * 18432 * 32 or batch * (q_hi + ctx_hi) * kv_heads * dim > 128 * 8192 * 1024:
        batch, q_hi, ctx_hi = max(1, batch * 3 // 4), max(1, q_hi * 7 // 8), max(1, ctx_hi * 7 // 8)
    window = _log(rng, 16, 4096) if rng.random() < 0.3 else 0
    return dict(op=op, batch=batch, q_lo=rng.randint(1, q_hi), q_hi=q_hi, ctx_lo=rng.randint(0, ctx_hi), ctx_hi=ctx_hi, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, cache=cache, page=page, window=window, sharp=rng.choice([1.0, 2.0]))


def _ladder(lo, hi, n, step):
    """n whole numbers from lo to hi, spread by a stride so that neighbours differ; the same for every seed."""
    return [lo + (hi - lo) * ((i * step) % n) // max(1, n - 1) for i in range(n)]


def _lengths(case):
    """Each request's (context, new tokens), in an order that the seed changes later."""
    n = case["batch"]
    if case["op"] == "slots":
        return list(zip(_ladder(0, case["ctx_hi"], n, 7), _ladder(case["new_lo"], case["new_hi"], n, 3)))
    return list(zip(_ladder(case["ctx_lo"], case["ctx_hi"], n, 7), _ladder(case["q_lo"], case["q_hi"], n, 3)))


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    host = np.random.default_rng(seed)
    return {"slots": _prepare_slots, "norm": _prepare_norm, "attn": _prepare_attn}[case["op"]](case, g, host)


def _cuda(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _prepare_slots(case, g, host):
    bs, pad = case["block"], case["pad"]
    lens = _lengths(case)
    order = host.permutation(len(lens))
    ctx = np.array([lens[i][0] for i in order], np.int32)
    new = np.array([lens[i][1] for i in order], np.int32)
    n = len(lens) + pad  # the last `pad` entries of the batch are padding
    states = n + 3
    cols = -(-(case["ctx_hi"] + case["new_hi"]) // bs) + 1
    held = -(-ctx.astype(np.int64) // bs)
    need = -(-(ctx.astype(np.int64) + new) // bs) - held
    blocks = host.permutation(int(held.sum() + need.sum()) + 17).astype(np.int32)
    table = np.full((states, cols), -1, np.int32)
    req = np.full(n, -1, np.int64)
    req[: len(lens)] = host.permutation(states)[: len(lens)]
    at = 0
    for r, h in zip(req[: len(lens)], held):
        table[r, :h] = blocks[at: at + h]
        at += h
    free = np.full(blocks.size, -1, np.int32)
    free[: blocks.size - at] = blocks[at:]
    tokens = int(new.sum())
    total = max(1, tokens + 5)  # room for a few more rows than the batch has
    return dict(case=case, ctx_lens=_cuda(np.concatenate([ctx, np.zeros(pad, np.int32)])),
                new_lens=_cuda(np.concatenate([new, np.full(pad, 1, np.int32)])), req_state=_cuda(req),
                block_table=_cuda(table), free_blocks=_cuda(free),
                free_top=_cuda(np.array([blocks.size - at], np.int32)),
                free_top_out=torch.zeros(1, dtype=torch.int32, device="cuda"),
                cu_new=torch.zeros(n + 1, dtype=torch.int32, device="cuda"),
                seq_lens=torch.zeros(n, dtype=torch.int32, device="cuda"),
                cache_loc=torch.zeros(total, dtype=torch.int64, device="cuda"),
                positions=torch.zeros(total, dtype=torch.int64, device="cuda"),
                token_row=torch.zeros(total, dtype=torch.int32, device="cuda"),
                status=torch.zeros(n, dtype=torch.int32, device="cuda"))


def _prepare_norm(case, g, host):
    t, h, hk, d, dt = case["tokens"], case["heads"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
    # the projection's output, with some heads much larger than others
    qkv = torch.randn(t, (h + 2 * hk) * d, generator=g, device="cuda") * torch.exp(
        torch.randn(t, (h + 2 * hk), generator=g, device="cuda")).repeat_interleave(d, 1)
    pages = -(-t // case["page"]) * 2 + 1
    half = case["rot"] // 2
    inv = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    ang = torch.arange(case["max_pos"], device="cuda", dtype=torch.float64)[:, None] * inv
    state = dict(case=case, qkv=qkv.to(dt),
                 q_weight=(1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt),
                 k_weight=(1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt),
                 cos_sin=torch.cat([ang.cos(), ang.sin()], 1).float(),
                 positions=torch.randint(0, case["max_pos"], (t,), generator=g, device="cuda"),
                 cache_loc=torch.randperm(pages * case["page"], generator=g, device="cuda")[:t],
                 q_out=torch.zeros(t, h, d, dtype=dt, device="cuda"),
                 status=torch.zeros(1, dtype=torch.int32, device="cuda"), k_scale=None, v_scale=None)
    shape = (pages, case["page"], hk, d)
    for name in ("k_cache", "v_cache"):
        c = torch.randn(shape, generator=g, device="cuda")
        state[name] = c.to(dt) if case["cache"] == "same" else c.to(torch.float8_e4m3fn)
    if case["cache"] == "fp8":
        state["k_scale"] = torch.tensor([0.031], device="cuda")
        state["v_scale"] = torch.tensor([0.11], device="cuda")
    return state


def _prepare_attn(case, g, host):
    h, hk, d, dt, ps = case["heads"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]], case["page"]
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
    fp8 = case["cache"] == "fp8"
    ks, vs = (0.031, 0.11) if fp8 else (1.0, 1.0)
    state = dict(case=case, q=(case["sharp"] * torch.randn(t, h, d, generator=g, device="cuda")).to(dt),
                 block_table=_cuda(table), req_state=_cuda(req.astype(np.int64)),
                 cu_q=_cuda(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)),
                 seq_lens=_cuda(seq.astype(np.int32)), max_q_len=int(new.max()),
                 out=torch.zeros(t, h, d, dtype=dt, device="cuda"),
                 lse=torch.zeros(t, h, device="cuda"),
                 status=torch.zeros(len(lens), dtype=torch.int32, device="cuda"),
                 k_scale=torch.tensor([ks], device="cuda") if fp8 else None,
                 v_scale=torch.tensor([vs], device="cuda") if fp8 else None)
    for name, sc in (("k_cache", ks), ("v_cache", vs)):
        c = torch.empty(pages, ps, hk, d, dtype=torch.float8_e4m3fn if fp8 else dt, device="cuda")
        step = max(1, (1 << 27) // (ps * hk * d))
        for a in range(0, pages, step):
            part = c[a: a + step]
            part.copy_((torch.randn(part.shape, generator=g, device="cuda") / sc).clamp(-448, 448))
        state[name] = c
    return state


# ---------------------------------------------------------------- one pass
def run(s):
    return {"slots": _run_slots, "norm": _run_norm, "attn": _run_attn}[s["case"]["op"]](s)


def _run_slots(s):
    if own:
        import sparse_attention_kv_row_gb300 as hs
        hs.assign_slots(s["ctx_lens"], s["new_lens"], s["req_state"], s["block_table"], s["free_blocks"],
                        s["free_top"], block_size=s["case"]["block"], cu_new=s["cu_new"],
                        seq_lens=s["seq_lens"], cache_loc=s["cache_loc"], positions=s["positions"],
                        token_row=s["token_row"], free_top_out=s["free_top_out"], status=s["status"])
    else:
        _plain_slots(s)
    return {k: s[k] for k in ("cu_new", "seq_lens", "cache_loc", "positions", "token_row", "block_table",
                              "free_top_out", "status")}


def _plain_slots(s):
    """Exclusive sums of the new tokens and of the blocks they open; each token's place by its row."""
    bs = s["case"]["block"]
    table, free = s["block_table"], s["free_blocks"]
    real = s["req_state"] >= 0
    r = s["req_state"].clamp(min=0)
    ctx = s["ctx_lens"].long()
    new = torch.where(real, s["new_lens"].long(), 0)
    cu = torch.cumsum(new, 0)
    held = (ctx + bs - 1) // bs
    need = torch.where(real, (ctx + new + bs - 1) // bs - held, 0)
    end = torch.cumsum(need, 0)
    col = torch.arange(table.shape[1], device=table.device)
    j = col[None, :] - held[:, None]  # the row's j-th new block
    opens = (j >= 0) & (j < need[:, None])
    taken = (s["free_top"].long() - 1 - (end - need)[:, None] - j).clamp(0, free.numel() - 1)
    rows = torch.where(opens, free[taken], table[r])
    keep = table.new_empty(table.shape[0] + 1, table.shape[1])  # padding writes to a row of its own
    keep[:-1] = table
    keep[torch.where(real, r, table.shape[0])] = rows
    table.copy_(keep[:-1])
    t = torch.arange(s["cache_loc"].numel(), device=table.device)
    b = torch.searchsorted(cu, t, right=True).clamp(max=cu.numel() - 1)
    inside = t < cu[-1]
    pos = t - (cu - new)[b] + ctx[b]
    block = rows[b, (pos // bs).clamp(0, table.shape[1] - 1)].long()
    s["cu_new"][1:] = cu
    s["cu_new"][0] = 0
    s["seq_lens"].copy_(ctx + new)
    s["cache_loc"].copy_(torch.where(inside, block * bs + pos % bs, -1))
    s["positions"].copy_(torch.where(inside, pos, -1))
    s["token_row"].copy_(torch.where(inside, b, -1))
    s["free_top_out"].copy_(s["free_top"] - end[-1])
    s["status"].zero_()


def _split(s):
    c = s["case"]
    h, hk, d = c["heads"], c["kv_heads"], c["dim"]
    x = s["qkv"].view(c["tokens"], h + 2 * hk, d)
    return x[:, :h], x[:, h: h + hk], x[:, h + hk:]


def _run_norm(s):
    c = s["case"]
    q, k, v = _split(s)
    if own:
        import sparse_attention_kv_row_gb300 as hs
        hs.qk_norm_rope_store(q, k, v, s["q_weight"], s["k_weight"], s["cos_sin"], s["positions"],
                              s["q_out"], s["k_cache"], s["v_cache"], s["cache_loc"], eps=1e-6,
                              interleaved=c["inter"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                              page_size=c["page"], status=s["status"])
    else:
        cs = s["cos_sin"][s["positions"]][:, None, :]
        s["q_out"].copy_(_plain_rope(_plain_norm(q, s["q_weight"]), cs, c))
        _plain_store(_plain_rope(_plain_norm(k, s["k_weight"]), cs, c), s["k_cache"], s["k_scale"], s["cache_loc"])
        _plain_store(v.float(), s["v_cache"], s["v_scale"], s["cache_loc"])
    return {k: s[k] for k in ("q_out", "k_cache", "v_cache")}


def _plain_norm(x, w):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()


def _plain_rope(x, cs, c):
    half = c["rot"] // 2
    cos, sin = cs[..., :half], cs[..., half:]
    y = x.clone()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if c["inter"] else (slice(0, half), slice(half, 2 * half))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _plain_store(x, cache, scale, loc):
    if scale is not None:
        x = (x * (1.0 / scale)).clamp(-448, 448)
        cache.view(torch.uint8).view(-1, *cache.shape[2:])[loc] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        cache.view(-1, *cache.shape[2:])[loc] = x.to(cache.dtype)


def _run_attn(s):
    c = s["case"]
    if own:
        import sparse_attention_kv_row_gb300 as hs
        hs.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["req_state"], s["cu_q"],
                           s["seq_lens"], s["out"], max_q_len=s["max_q_len"], scale=c["dim"] ** -0.5,
                           window=c["window"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                           page_size=c["page"], lse=s["lse"], status=s["status"])
    else:
        _plain_attn(s)
    return {"out": s["out"], "lse": s["lse"]}


def _plain_attn(s):
    """Every request padded to the longest; keys gathered through the block table; one softmax over them."""
    c = s["case"]
    h, hk, d, ps = c["heads"], c["kv_heads"], c["dim"], c["page"]
    cu, seq = s["cu_q"].long(), s["seq_lens"].long()
    new = cu[1:] - cu[:-1]
    t, batch = s["q"].shape[0], seq.numel()
    table = s["block_table"][s["req_state"]].long().clamp(min=0)
    n = table.shape[1] * ps

    def gathered(cache, scale):
        x = cache.view(torch.uint8)[table].view(cache.dtype) if scale is not None else cache[table]
        x = x.float().view(batch, n, hk, d).permute(0, 2, 1, 3)
        return x if scale is None else x * scale

    row = torch.arange(t, device=cu.device)
    b = torch.searchsorted(cu[1:], row, right=True)
    i = row - cu[b]
    q = torch.zeros(batch, s["max_q_len"], h, d, device=cu.device)
    q[b, i] = s["q"].float()
    q = q.view(batch, -1, hk, h // hk, d).permute(0, 2, 3, 1, 4).reshape(batch, hk, -1, d)
    p = torch.matmul(q, gathered(s["k_cache"], s["k_scale"]).transpose(2, 3)).mul_(d ** -0.5)
    p = p.view(batch, hk, h // hk, -1, n)
    pos = (seq - new)[:, None] + torch.arange(s["max_q_len"], device=cu.device)
    key = torch.arange(n, device=cu.device)
    seen = (key <= pos[..., None]) & (key < seq[:, None, None])
    if c["window"]:
        seen &= key > pos[..., None] - c["window"]
    p.masked_fill_(~seen[:, None, None], -math.inf)
    m = p.amax(-1, keepdim=True).clamp(min=-1e30)
    p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    p.div_(l.clamp(min=1e-30))
    o = torch.matmul(p.view(batch, hk, -1, n), gathered(s["v_cache"], s["v_scale"]))
    o = o.view(batch, hk, h // hk, -1, d).permute(0, 3, 1, 2, 4).reshape(batch, -1, h, d)
    lse = (m + torch.log(l)).squeeze(-1).permute(0, 3, 1, 2).reshape(batch, -1, h)
    s["out"].copy_(o[b, i])
    s["lse"].copy_(lse[b, i])


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "slots":
        lens = _lengths(case)
        n, t, bs = len(lens) + case["pad"], sum(x[1] for x in lens), case["block"]
        opened = sum(-(-(c + q) // bs) - -(-c // bs) for c, q in lens)
        # lengths, state rows, totals and status; a slot, a position and a row per token; the opened blocks,
        # and the entry of the block that each row fills up
        return {"bytes": n * (4 + 4 + 8 + 4 + 4 + 4) + 8 + t * 20 + opened * 8 + n * 4, "flops": 0}
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    wide = 4 if case["dtype"] == "f32" else 2
    kept = 1 if case["cache"] == "fp8" else wide
    if case["op"] == "norm":
        t = case["tokens"]
        return {"bytes": t * d * (2 * h * wide + 2 * hk * (wide + kept)) + t * (16 + case["rot"] * 4),
                "flops": t * (h + hk) * (4 * d + 3 * case["rot"])}
    lens, w = _lengths(case), case["window"]
    keys = pairs = 0
    for c, q in lens:
        first = max(0, c - w + 1) if w else 0
        keys += c + q - first
        pairs += sum(min(c + i + 1, w) if w else c + i + 1 for i in range(q))
    t = sum(q for _, q in lens)
    return {"bytes": keys * hk * d * 2 * kept + t * h * (2 * d * wide + 4), "flops": 4 * pairs * h * d}


# ---------------------------------------------------------------- 64 bits, request by request
def exact(case, seed):
    s = prepare(case, seed)
    return {"slots": _exact_slots, "norm": _exact_norm, "attn": _exact_attn}[case["op"]](s)


def _exact_slots(s):
    x = {k: v.cpu().numpy().copy() for k, v in s.items() if torch.is_tensor(v)}
    bs, top, at = s["case"]["block"], int(x["free_top"][0]), 0
    for k in ("cache_loc", "positions", "token_row"):
        x[k][:] = -1
    for b, r in enumerate(x["req_state"]):
        ctx = int(x["ctx_lens"][b])
        n = int(x["new_lens"][b]) if r >= 0 else 0
        for c in range(-(-ctx // bs), -(-(ctx + n) // bs)):
            top -= 1
            x["block_table"][r, c] = x["free_blocks"][top]
        pos = np.arange(ctx, ctx + n)
        x["cache_loc"][at: at + n] = x["block_table"][r, pos // bs].astype(np.int64) * bs + pos % bs
        x["positions"][at: at + n] = pos
        x["token_row"][at: at + n] = b
        at += n
        x["cu_new"][b + 1] = at
        x["seq_lens"][b] = ctx + n
    x["cu_new"][0] = 0
    x["free_top_out"][0] = top
    x["status"][:] = 0
    return {k: x[k] for k in ("cu_new", "seq_lens", "cache_loc", "positions", "token_row", "block_table",
                              "free_top_out", "status")}


def _exact_norm(s):
    c = s["case"]
    half, d = c["rot"] // 2, c["dim"]
    cs = s["cos_sin"].double()[s["positions"]]
    turn = torch.complex(cs[:, :half], cs[:, half:])[:, None]
    q, k, v = (x.double() for x in _split(s))
    done = []
    for x, w in ((q, s["q_weight"]), (k, s["k_weight"])):
        x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / d + 1e-6) * w.double()
        head = x[..., : 2 * half]
        pair = head.unflatten(-1, (half, 2)) if c["inter"] else head.unflatten(-1, (2, half)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        z = z.flatten(-2) if c["inter"] else z.transpose(-1, -2).flatten(-2)
        done.append(torch.cat([z, x[..., 2 * half:]], -1))
    out = {"q_out": done[0]}
    for name, x in (("k", done[1]), ("v", v)):
        cache, scale = s[name + "_cache"], s[name + "_scale"]
        x = x if scale is None else (x / scale.double()).clamp(-448, 448)
        kept = cache.double().reshape(-1, *cache.shape[2:])
        kept[s["cache_loc"]] = x
        out[name + "_cache"] = kept.view(cache.shape)
    return out


def _exact_attn(s):
    c = s["case"]
    h, hk, d, ps = c["heads"], c["kv_heads"], c["dim"], c["page"]
    cu, seq = s["cu_q"].tolist(), s["seq_lens"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    ks = 1.0 if s["k_scale"] is None else s["k_scale"].double()
    vs = 1.0 if s["v_scale"] is None else s["v_scale"].double()
    for b, r in enumerate(s["req_state"].tolist()):
        n, a, e = seq[b], cu[b], cu[b + 1]
        pages = s["block_table"][r, : -(-n // ps)].long()
        for g in range(hk):
            kk, vv = (x[pages, :, g].double().reshape(-1, d)[:n] * sc for x, sc in ((s["k_cache"], ks), (s["v_cache"], vs)))
            q = s["q"][a:e, g * (h // hk): (g + 1) * (h // hk)].double()
            z = torch.einsum("tgd,nd->tgn", q, kk) / math.sqrt(d)
            gap = torch.arange(n - (e - a), n, device="cuda")[:, None, None] - torch.arange(n, device="cuda")
            z.masked_fill_((gap < 0) | (gap >= (c["window"] or n + 1)), -math.inf)
            part = torch.logsumexp(z, -1)
            lse[a:e, g * (h // hk): (g + 1) * (h // hk)] = part
            out[a:e, g * (h // hk): (g + 1) * (h // hk)] = torch.einsum("tgn,nd->tgd", torch.exp(z - part[..., None]), vv)
    return {"out": out, "lse": lse}
