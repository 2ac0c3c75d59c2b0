"""Plain statements, in 64 bits and token by token, of the latent-attention operators, and the
inputs their tests share."""
from __future__ import annotations

import math

import numpy as np
import torch

from paged_cases import TORCH, U32, half_step

GROUP = 128


def row_bytes(latent, rope):
    return latent + latent // 32 + 2 * rope


# ------------------------------------------------------------------ norm and codes
def norm_plain(x, w, eps):
    x = x.double()
    ms = (x * x).mean(-1, keepdim=True) + eps
    y = torch.where(ms == 0, torch.zeros_like(x), x / torch.sqrt(ms))
    return y if w is None else y * w.double()


def norm_error(dim):
    """Relative error of a normed value in fp32: a sum of dim squares (each partial sum off by at
    most one unit, half of which is left behind the root), the root, and three products."""
    return (dim / 2 + 12) * U32


def grouped(y, group):
    """[..., groups, n] of the last axis, zeros behind its end."""
    n = group or y.shape[-1]
    groups = -(-y.shape[-1] // n)
    z = torch.zeros(*y.shape[:-1], groups * n, dtype=y.dtype)
    z[..., : y.shape[-1]] = y
    return z.unflatten(-1, (groups, n))


def check_codes(y, rel, codes, scales, group, pow2):
    """Codes and scales of y (64 bits, relatively off by `rel` in the kernel).  A scale is 1/448 of
    the group's largest value, three roundings away; a code is half a step of E4M3 (2^-4 of it, or
    2^-10 where that is more) from the value over the scale that was stored."""
    z = grouped(y, group)
    want = z.abs().amax(-1) / 448
    s = scales.double()
    err = (rel + 4 * U32) * want
    if pow2:
        some = want > 0
        assert bool((torch.frexp(scales[some])[0] == 0.5).all()), "powers of two"
        assert bool((s >= want - err).all()) and bool((s <= 2 * (want + err)).all())
    else:
        assert bool(((s - want).abs() <= err).all()), float(((s - want).abs() / want).max())
    v = torch.where(s[..., None] > 0, z / s[..., None].clamp(min=1e-300), torch.zeros_like(z))
    v = v.flatten(-2)[..., : y.shape[-1]].clamp(-448, 448)
    got = codes.view(torch.float8_e4m3fn).double()
    assert bool(((got - v).abs() <= 1.01 * (2.0 ** -4 * v.abs() + 2 * rel * v.abs()) + 2.0 ** -10).all())


# ------------------------------------------------------------------ rows
def make_rows(values, fmt, dtype):
    """Latent rows [n, R + P] kept as `fmt` ("same" or "fp8"), and the values they hold (64 bits)."""
    R = values.shape[1] - 64 if fmt == "fp8" else None
    if fmt == "same":
        rows = values.to(dtype)
        return rows, rows.double()
    c, pe = values[:, :R], values[:, R:].to(dtype)
    g = c.unflatten(1, (-1, GROUP))
    scale = g.abs().amax(-1, keepdim=True) / 448
    codes = (g / torch.where(scale > 0, scale, 1.0)).clamp(-448, 448).to(torch.float8_e4m3fn)
    rows = torch.cat([codes.view(torch.uint8).flatten(1), scale.squeeze(-1).contiguous().view(torch.uint8),
                      pe.contiguous().view(torch.uint8)], 1)
    held = torch.cat([(codes.double() * scale.double()).flatten(1), pe.double()], 1)
    return rows, held


def spoil(rows, which, fmt):
    """NaN in every value of the rows `which`."""
    if fmt == "fp8":
        rows[which] = 0xFF
    else:
        rows[which] = math.nan


# ------------------------------------------------------------------ attention
def latent_plain(q, held, lists, R, scale):
    """Per token: out, lse, mean |value| under the weights, score unit, rows seen; `lists` has for
    each token the rows it sees (-2: a row of zeros), or None where it is not touched."""
    T, H, dims = q.shape
    f = dict(dtype=torch.float64)
    out, lse = torch.zeros(T, H, R, **f), torch.full((T, H), -math.inf, **f)
    size, unit, n = torch.zeros(T, H, R, **f), torch.zeros(T, H, **f), torch.zeros(T, **f)
    wide = torch.zeros(T, H, **f)
    q = q.double()
    for t, rows in enumerate(lists):
        if rows is None or len(rows) == 0:
            continue
        at = torch.as_tensor(rows, dtype=torch.int64)
        k = torch.where((at >= 0)[:, None], held[at.clamp(min=0)], 0.0)
        s = torch.einsum("hd,nd->nh", q[t], k) * scale
        lse[t] = torch.logsumexp(s, 0)
        w = torch.exp(s - lse[t])
        out[t] = torch.einsum("nh,nd->hd", w, k[:, :R])
        size[t] = torch.einsum("nh,nd->hd", w, k[:, :R].abs())
        unit[t] = (torch.einsum("hd,nd->nh", q[t].abs(), k.abs()) * scale).amax(0)
        wide[t] = q[t].abs().amax(1) * k.abs().sum(1).max() * scale
        n[t] = len(rows)
    return out, lse, size, unit, n, wide


class LatentInputs:
    """Latent rows with NaN in every one that no token sees, and queries for tokens that see
    `lists` of rows (by an index or by block tables)."""

    def __init__(self, *, heads, dtype, fmt, latent=512, rope=64, seed=0, sharp=2.0, spread=None):
        self.g = torch.Generator().manual_seed(seed)
        self.rng = np.random.default_rng(seed)
        self.H, self.R, self.P, self.fmt, self.dtype = heads, latent, rope, fmt, TORCH[dtype]
        self.scale, self.sharp = (latent * math.exp(0.5) + rope) ** -0.5, sharp
        # (a, b): rows of codes times up to 2^+-a, their groups times 2^-b to 1, some zeros
        self.spread = spread
        if spread is not None:
            self.scale *= 2.0 ** -spread[0]

    def _fill(self, n, seen, T):
        wide = torch.cat([torch.exp(0.5 * torch.randn(self.R, generator=self.g)), torch.ones(self.P)])
        values = torch.randn(n, self.R + self.P, generator=self.g) * wide
        if self.spread is not None:
            a, b = self.spread
            by = 2.0 ** torch.randint(-a, a + 1, (n, 1), generator=self.g).double()
            by = by * 2.0 ** -torch.randint(0, b + 1, (n, self.R // GROUP), generator=self.g).double()
            by[torch.rand(by.shape, generator=self.g) < 0.1] = 0.0
            values = values.double()
            values[:, : self.R] *= by.repeat_interleave(GROUP, 1)
            values = values.float()
        self.rows, self.held = make_rows(values, self.fmt, self.dtype)
        hidden = np.ones(n, bool)
        hidden[list(seen)] = False
        spoil(self.rows, torch.from_numpy(hidden), self.fmt)
        self.T = T
        self.q = (self.sharp * torch.randn(T, self.H, self.R + self.P, generator=self.g)).to(self.dtype)

    def indexed(self, T, top_k, pool, empty=(), bad=()):
        """Random selections; tokens in `empty` see nothing, those in `bad` have entries that are no
        rows of the pool."""
        self.index = np.stack([self.rng.permutation(pool)[:top_k] for _ in range(T)]).astype(np.int32) \
            if T and top_k else np.zeros((T, top_k), np.int32)
        if top_k > 2:
            self.index[self.rng.random((T, top_k)) < 0.1] = -1
        for t in empty:
            self.index[t] = -1 - self.rng.integers(0, 5, top_k)
        self.status = np.zeros(T, np.int32)
        for t in bad:
            self.index[t, self.rng.integers(0, top_k, max(1, top_k // 8))] = pool + self.rng.integers(0, 3)
            self.status[t] = 64
        self.lists = [[int(e) for e in row if 0 <= e < pool] for row in self.index]
        self._fill(pool, {e for row in self.lists for e in row}, T)
        return self

    def paged(self, lens, page, gap=0, bad_block=None):
        """Requests as (context, new) pairs; a context of None is a padding row."""
        seq = np.array([0 if c is None else c + n for c, n in lens], np.int64)
        new = np.array([0 if c is None else n for c, n in lens], np.int64)
        held = -(-np.maximum(seq, 0) // page)
        pages = int(held.sum()) + 2
        states = len(lens) + 2
        self.req = self.rng.permutation(states)[: len(lens)].astype(np.int64)
        perm = self.rng.permutation(pages)
        self.table = np.full((states, max(1, int(held.max(initial=0)))), -1, np.int32)
        at = 0
        self.status = np.zeros(len(lens), np.int32)
        for b, (c, n) in enumerate(lens):
            if c is None:
                self.req[b] = -1 - b
                continue
            self.table[self.req[b], : held[b]] = perm[at: at + held[b]]
            at += held[b]
        if bad_block is not None:
            b, c, e = bad_block
            self.table[self.req[b], c] = e
            self.status[b] = 64
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.seq, self.page, self.max_q = seq, page, int(new.max(initial=0))
        T = int(self.cu[-1]) + gap
        self.lists = [None] * T
        for b in range(len(lens)):
            for i in range(int(new[b])):
                p = int(seq[b] - new[b]) + i
                row = []
                for j in range(p + 1):
                    e = int(self.table[self.req[b], j // page])
                    row.append(e * page + j % page if 0 <= e < pages else -2)
                self.lists[int(self.cu[b]) + i] = row
        self._fill(pages * page, {e for row in self.lists if row for e in row if e >= 0}, T)
        return self

    def tolerance(self, ref, kind):
        """Bounds on |out - plain| and |lse - plain|.  fp32 products and sums: a score is off by at
        most (dims + 8) units of 2^-24 of sum |q k| (a code's scale and its product with the value
        among them); the sums over n rows by n units; the exponentials by 4 units.  On the tensor
        cores ("tiles") the weights are rounded to 16 bits (half a step; over codes they are fp16,
        times the scales), what codes stand for to fp16 (half a step in keys and in values), bf16
        queries over codes are taken as fp16, off by 2^-33 of the row's largest, and outputs by half
        a step; fp16 weights have an absolute half step, at most 2^-29 of the largest value for each
        of n rows."""
        out, lse, size, unit, n, wide = ref
        dims = self.R + self.P
        es = (dims + 8) * U32 * unit
        up, small = 0.0, 0.0
        if kind != "general":
            of = torch.float16 if self.fmt == "fp8" else self.dtype
            up = half_step(of) + 4 * U32
            if of == torch.float16:
                v = self.held[:, : self.R].abs()
                small = 2.0 ** -29 * float(v.max()) if v.numel() else 0.0
            if self.fmt == "fp8":
                es = es + 2.0 ** -33 * wide + half_step(torch.float16) * unit
                up += half_step(torch.float16)
                if self.spread is not None:
                    # Values below fp16's normal range are 2^-25 of 2^e off, at most twice the
                    # largest scale, 1/448 of a value; so are their scores.
                    off = 2.0 ** -25 * 2 / 448 * float(self.held[:, : self.R].abs().max())
                    es = es + off * self.q[..., : self.R].double().abs().sum(-1) * self.scale
                    small += off
        u = half_step(self.dtype) if self.dtype != torch.float32 else U32
        rel = 2 * es + (2 * n[:, None] + 16) * U32 + up
        tiny = 2.0 ** -25 if self.dtype == torch.float16 else 0.0
        tol_out = 1.01 * (rel[..., None] * size + u * out.abs() + small * n[:, None, None]) + tiny
        tol_lse = 1.01 * (es + (n[:, None] + 16) * U32 + 4 * U32 * lse.abs().nan_to_num(posinf=0.0))
        return tol_out, tol_lse

    def call(self, hs, dev, *, q=None, rows=None, out=None, lse=None, status=None, **kw):
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        q = self.q.to(dev) if q is None else q
        rows = self.rows.to(dev) if rows is None else rows
        out = torch.full((self.T, self.H, self.R), -7.0, dtype=self.dtype, device=dev) if out is None else out
        lse = torch.full((self.T, self.H), -7.0, device=dev) if lse is None else lse
        status = torch.full((len(self.status),), -1, dtype=torch.int32, device=dev) if status is None else status
        if hasattr(self, "index"):
            args = (q, rows, t(self.index), out)
            fn = hs.latent_attention
        else:
            args = (q, rows, t(self.table), t(self.req), t(self.cu), t(self.seq), out)
            kw = dict(max_q_len=self.max_q, page_size=self.page) | kw
            fn = hs.paged_latent_attention
        if "stream" in kw:
            torch.cuda.synchronize()
        fn(*args, scale=self.scale, lse=lse, status=status, **kw)
        if "stream" in kw:  # the inputs live as long as the call
            torch.cuda.synchronize()
        return out, lse, status

    def check(self, hs, dev, kind, **kw):
        out, lse, status = self.call(hs, dev, **kw)
        self.compare(out, lse, status, kind)
        return out, lse, status

    def compare(self, out, lse, status, kind):
        ref = latent_plain(self.q, self.held, self.lists, self.R, self.scale)
        tol_out, tol_lse = self.tolerance(ref, kind)
        out, lse = out.cpu().double(), lse.cpu().double()
        seen = torch.tensor([x is not None for x in self.lists], dtype=torch.bool)
        assert bool((out[~seen] == -7).all()) and bool((lse[~seen] == -7).all()), "untouched rows"
        err = (out - ref[0]).abs()[seen]
        if self.dtype == torch.float16:
            # What is past 65504 (or rounds there) is an infinity in fp16: 65520 is the half-way point.
            over = (out == math.inf) & (ref[0] + tol_out >= 65520) | (out == -math.inf) & (ref[0] - tol_out <= -65520)
            err = torch.where(over[seen], 0.0, err)
        bad = ~(err <= tol_out[seen])
        assert not bool(bad.any()), (
            f"{int(bad.sum())} outputs off: worst {float(err.max()):.3g}, at most "
            f"{float((err / tol_out[seen]).nan_to_num(nan=9e9).max()):.3g} of the bound")
        none = seen[:, None] & (ref[1] == -math.inf)
        assert bool((lse[none] == -math.inf).all()) and bool((out[none] == 0).all())
        some = seen[:, None] & (ref[1] > -math.inf)
        err = (lse - ref[1]).abs()[some]
        assert bool((err <= tol_lse[some]).all()), (
            f"lse off by {float(err.max()):.3g}, {float((err / tol_lse[some]).max()):.3g} of the bound")
        np.testing.assert_array_equal(status.cpu().numpy(), self.status)
