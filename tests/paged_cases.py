"""Plain statements, in 64 bits and request by request, of the paged-cache
operators, and the inputs their tests share."""
from __future__ import annotations

import math

import numpy as np
import torch

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16,
         "fp8": torch.float8_e4m3fn}
U32 = 2.0 ** -24


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


# ------------------------------------------------------------------ assign_slots
def slots_plain(ctx, new, req, table, free, top, bs, max_tokens):
    """assign_slots row by row; returns every output (``table`` is a changed copy)."""
    table = table.copy()
    states, cols = table.shape
    B = len(ctx)
    top = min(max(int(top), 0), len(free))
    out = dict(cu_new=np.zeros(B + 1, np.int64), seq_lens=np.array(ctx, np.int64),
               cache_loc=np.full(max_tokens, -1, np.int64),
               positions=np.full(max_tokens, -1, np.int64),
               token_row=np.full(max_tokens, -1, np.int32), status=np.zeros(B, np.int32))
    wanted = taken = 0
    for b in range(B):
        c, n, r = int(ctx[b]), int(new[b]), int(req[b])
        at = int(out["cu_new"][b])
        st, cnt = 0, 0
        if r >= 0:
            cnt = n if 0 <= n <= max_tokens else 0
            if (cnt != n or r >= states or not 0 <= c < 2 ** 31 or c + n > cols * bs
                    or c + n >= 2 ** 31):
                st = 32
            elif at + cnt > max_tokens:
                st = 64
        end = at + cnt
        out["cu_new"][b + 1] = min(end, 2 ** 31 - 1)
        ok = r >= 0 and st == 0
        if ok:
            held, upto = -(-c // bs), -(-(c + n) // bs)
            if upto > held:
                if wanted + upto - held > top:
                    st, ok = 128, False
                else:
                    for j in range(upto - held):
                        table[r, held + j] = free[top - 1 - wanted - j]
                    taken = wanted + upto - held
                wanted += upto - held
        if ok:
            out["seq_lens"][b] = c + n
        for i in range(cnt):
            t, p = at + i, c + i
            if t >= max_tokens:
                break
            out["positions"][t], out["token_row"][t] = p, b
            if ok:
                e = int(table[r, p // bs])
                if e >= 0:
                    out["cache_loc"][t] = e * bs + p % bs
                else:
                    st |= 64
        out["status"][b] = st
    out["table"], out["free_top"] = table, top - taken
    return out


# ------------------------------------------------------------------ qk_norm_rope_store
def norm_rope_plain(x, w, cs, eps, interleaved):
    """[T, heads, dim] in 64 bits with angles cs [T, rot]; returns (z, |y_a| + |y_b|)."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    size = x.abs()
    if cs is None:
        return x, size
    half = cs.shape[1] // 2
    co, si = cs[:, None, :half].double(), cs[:, None, half:].double()
    i = torch.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    z = x.clone()
    z[..., a] = x[..., a] * co - x[..., b] * si
    z[..., b] = x[..., b] * co + x[..., a] * si
    both = size.clone()
    both[..., a] = both[..., b] = size[..., a] + size[..., b]
    return z, both


# ------------------------------------------------------------------ paged_attention
def attention_plain(q, kc, vc, table, req, cu, seq, *, scale, window=0, ks=1.0, vs=1.0,
                    max_q=None):
    """Returns (out, lse, mean |v| under the weights, score error unit, keys seen, touched) per
    query, in 64 bits.  Caches are [pages, page, heads, dim]; `touched` marks the rows written."""
    T, H, D = q.shape
    pages, ps, HK, _ = kc.shape
    f = dict(dtype=torch.float64)
    out, lse = torch.zeros(T, H, D, **f), torch.full((T, H), -math.inf, **f)
    size, unit = torch.zeros(T, H, D, **f), torch.zeros(T, H, **f)
    seen_n, touched = torch.zeros(T, **f), torch.zeros(T, dtype=torch.bool)
    kc, vc, q = kc.double(), vc.double(), q.double()
    for b, r in enumerate(req):
        r, L, a, e = int(r), int(seq[b]), int(cu[b]), int(cu[b + 1])
        if (r < 0 or r >= table.shape[0] or a < 0 or e < a or e > T or L > table.shape[1] * ps
                or (max_q is not None and e - a > max_q)):
            continue
        touched[a:e] = True
        for t in range(a, e):
            p = L - (e - a) + (t - a)
            lo = max(0, p + 1 - window) if window else 0
            if p + 1 <= lo:
                continue
            j = np.arange(lo, p + 1)
            ent = table[r, j // ps].astype(np.int64)
            good = torch.from_numpy((ent >= 0) & (ent < pages))[:, None, None]
            ent = torch.from_numpy(np.where((ent >= 0) & (ent < pages), ent, 0))
            off = torch.from_numpy(j % ps)
            k = torch.where(good, kc[ent, off], 0.0).repeat_interleave(H // HK, 1)
            v = torch.where(good, vc[ent, off], 0.0).repeat_interleave(H // HK, 1)
            s = torch.einsum("hd,nhd->nh", q[t], k) * (scale * ks)
            lse[t] = torch.logsumexp(s, 0)
            w = torch.exp(s - lse[t])
            out[t] = torch.einsum("nh,nhd->hd", w, v) * vs
            size[t] = torch.einsum("nh,nhd->hd", w, v.abs()) * vs
            unit[t] = (torch.einsum("hd,nhd->nh", q[t].abs(), k.abs()) * abs(scale * ks)).amax(0)
            seen_n[t] = len(j)
    return out, lse, size, unit, seen_n, touched


class PagedInputs:
    """A paged cache with NaN in every byte that no request owns, random block tables, and
    queries for requests given as (context, new) pairs; a context of None is a padding row."""

    def __init__(self, lens, *, heads, kv_heads, dim, dtype, cache="same", page=16, flat=False,
                 seed=0, sharp=2.0, window=0, i64=True, scales=(0.031, 0.11), gap=0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        dt = TORCH[dtype]
        self.fp8 = cache == "fp8"
        cdt = torch.float8_e4m3fn if self.fp8 else dt
        self.ks, self.vs = scales if self.fp8 else (1.0, 1.0)
        self.page, self.window, self.scale = page, window, dim ** -0.5
        real = [(c, n) for c, n in lens if c is not None]
        seq = np.array([0 if c is None else c + n for c, n in lens], np.int64)
        held = -(-np.maximum(seq, 0) // page)
        pages = int(held.sum()) + 2
        cols = max(1, int(held.max(initial=0)))
        states = len(lens) + 2
        self.req = rng.permutation(states)[: len(lens)].astype(np.int64)
        perm = rng.permutation(pages)
        self.table = np.full((states, cols), -1, np.int32)
        at = 0
        kc = torch.full((pages, page, kv_heads, dim), math.nan)
        vc = kc.clone()
        for b, (c, n) in enumerate(lens):
            if c is None:
                self.req[b] = -1 - b
                continue
            self.table[self.req[b], : held[b]] = perm[at: at + held[b]]
            lo = max(0, c + 1 - window) if window else 0
            for j in range(held[b]):
                first, last = max(lo - j * page, 0), min(page, seq[b] - j * page)
                if last > first:
                    x = torch.randn(2, last - first, kv_heads, dim, generator=g)
                    kc[perm[at + j], first:last] = x[0] / self.ks
                    vc[perm[at + j], first:last] = x[1] / self.vs
            if lo:  # blocks behind the window have been given back
                self.table[self.req[b], : lo // page] = -1
            at += held[b]
        clamp = (lambda x: torch.where(x.isnan(), x, x.clamp(-448, 448))) if self.fp8 else (lambda x: x)
        self.kc, self.vc = clamp(kc).to(cdt), clamp(vc).to(cdt)
        new = np.array([0 if c is None else n for c, n in lens], np.int64)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.seq = seq
        self.T = int(self.cu[-1]) + gap  # `gap` rows behind the last request
        self.q = (sharp * torch.randn(self.T, heads, dim, generator=g)).to(dt)
        self.max_q = int(new.max(initial=0))
        self.dtype, self.flat, self.i64 = dt, flat, i64
        self.real = real

    def plain(self, max_q=None):
        return attention_plain(self.q, self.kc, self.vc, self.table, self.req, self.cu, self.seq,
                               scale=self.scale, window=self.window, ks=self.ks, vs=self.vs,
                               max_q=max_q)

    def tolerance(self, ref, tensor_cores):
        """Bounds on |out - plain| and |lse - plain|.  fp32 products and sums: a score is off by
        at most (D + 4) units of 2^-24 of sum |q k|; the two sums over n keys by n units; the
        weights' exponentials by 4 units.  On the tensor cores each weight is rounded to the
        compute type (half a step), as is the output; fp16 outputs have an absolute half step.
        fp16 weights have one too: they are kept as at least 2^6 times their share of a sum that
        is then at least 2^6, so half a step of fp16's subnormals, 2^-25, is at most 2^-31 of a
        value for each of n keys."""
        out, lse, size, unit, n, _ = ref
        D = self.q.shape[2]
        es = (D + 4) * U32 * unit  # [T, H]
        u = half_step(self.dtype)
        up, small = 0.0, 0.0
        if tensor_cores:
            kind = torch.float16 if self.fp8 else self.dtype
            up = half_step(kind)
            if kind == torch.float16:
                v = self.vc.float().abs()
                small = 2.0 ** -31 * float(v[v.isfinite()].max()) * self.vs if v.isfinite().any() else 0.0
        rel = 2 * es + (2 * n[:, None] + 16) * U32 + up
        tiny = 2.0 ** -25 if self.dtype == torch.float16 else 0.0
        tol_out = 1.01 * (rel[..., None] * size + u * out.abs() + small * n[:, None, None]) + tiny
        tol_lse = 1.01 * (es + (n[:, None] + 16) * U32 + 4 * U32 * lse.abs().nan_to_num(posinf=0.0))
        return tol_out, tol_lse

    def call(self, hs, dev, *, q=None, out=None, lse=None, status=None, max_q=None, **kw):
        """paged_attention on ``dev``; returns (out, lse, status) with untouched rows at -7."""
        t = lambda a, d=None: torch.from_numpy(np.ascontiguousarray(a)).to(dev) if d is None else \
            torch.from_numpy(np.ascontiguousarray(a)).to(d).to(dev)  # noqa: E731
        kc, vc = self.kc.to(dev), self.vc.to(dev)
        if self.flat:
            kc, vc = kc.flatten(0, 1), vc.flatten(0, 1)
        i = torch.int64 if self.i64 else torch.int32
        out = torch.full(self.q.shape, -7.0, dtype=self.dtype, device=dev) if out is None else out
        lse = torch.full(self.q.shape[:2], -7.0, device=dev) if lse is None else lse
        status = torch.full((len(self.seq),), -1, dtype=torch.int32, device=dev) \
            if status is None else status
        sc = lambda x: torch.tensor([x], device=dev) if self.fp8 else None  # noqa: E731
        inputs = (self.q.to(dev) if q is None else q, kc, vc, t(self.table), t(self.req, i), t(self.cu), t(self.seq, i))
        if "stream" in kw:  # the uploads are on the current stream
            torch.cuda.synchronize()
        hs.paged_attention(*inputs, out, max_q_len=self.max_q if max_q is None else max_q,
                           window=self.window, k_scale=sc(self.ks), v_scale=sc(self.vs),
                           page_size=self.page, lse=lse, status=status, **kw)
        if "stream" in kw:  # the inputs live as long as the call
            torch.cuda.synchronize()
        return out, lse, status

    def check(self, hs, dev, tensor_cores, **kw):
        out, lse, status = self.call(hs, dev, **kw)
        ref = self.plain(kw.get("max_q"))
        tol_out, tol_lse = self.tolerance(ref, tensor_cores)
        out, lse = out.cpu().double(), lse.cpu().double()
        seen = ref[5]
        assert bool((out[~seen] == -7).all()) and bool((lse[~seen] == -7).all()), "untouched rows"
        err = (out - ref[0]).abs()[seen]
        bad = ~(err <= tol_out[seen])
        assert not bool(bad.any()), (
            f"{int(bad.sum())} outputs off: worst {float(err.max()):.3g}, at most "
            f"{float((err / tol_out[seen]).nan_to_num(nan=9e9).max()):.3g} of the bound")
        none = seen[:, None] & (ref[1] == -math.inf)
        assert bool((lse[none] == -math.inf).all()) and bool((out[none.expand(lse.shape)] == 0).all())
        some = seen[:, None] & (ref[1] > -math.inf)
        err = (lse - ref[1]).abs()[some]
        assert bool((err <= tol_lse[some]).all()), f"lse off by {float(err.max()):.3g}"
        return out, lse, status
