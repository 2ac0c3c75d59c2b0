"""Latent attention over codes whose scales lie far apart: outputs bounded by what each token sees,
under its weights, and rows that a token does not see."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from latent_cases import GROUP
from paged_cases import TORCH, U32, half_step

pytestmark = pytest.mark.gpu
R, P = 512, 64
GROUPS = R // GROUP
H16 = half_step(torch.float16)


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__

    __graft_entry__.build()
    return torch.device("cuda:0")


def rows_of(codes, scales, pe):
    """Rows of [n, 512] codes (float), [n, 4] scales and [n, 64] rotary values, and what they hold."""
    c = codes.to(torch.float8_e4m3fn)
    rows = torch.cat([c.view(torch.uint8), scales.float().contiguous().view(torch.uint8),
                      pe.contiguous().view(torch.uint8)], 1)
    held = torch.cat([c.double() * scales.double().repeat_interleave(GROUP, 1), pe.double()], 1)
    return rows, held


def some(g, n, dtype, scales):
    codes = (torch.randn(n, R, generator=g) * 100).clamp(-448, 448)
    return codes, torch.as_tensor(scales, dtype=torch.float64).expand(n, GROUPS).clone(), \
        torch.randn(n, P, generator=g).to(dtype)


def plain(q, held, scales, lists, scale, dtype):
    """Outputs and lse in 64 bits with bounds on their errors, a token and head at a time.

    With S the largest scale of a row, 2^e is below S / 64 and its values over 2^e are below 2^16.
    A value is kept as fp16 of code * (scale / 2^e): half a step, or 2^-25 of 2^e, for the value
    and a 2^-25 of 2^e for each unit of the code (at most 448) for the factor, which is two fp16
    values; in all `off` = 450 * 2^-25 * S / 64.  A score is off by that under |q|, by half a step
    of sum |q k|, by the fp32 sum and by 2^-33 of the largest query value.  A weight times 2^e is
    fp16, half a step off or 2^-25 where the largest one is at least 2^5: 2^-30 of the largest
    weight times 2^e, below S / 64, of a value below 2^16.  Sums in fp32 over n rows; the output
    once more half a step."""
    T, H, _ = q.shape
    f = dict(dtype=torch.float64)
    out, lse = torch.zeros(T, H, R, **f), torch.full((T, H), -np.inf, **f)
    tol, tol_lse = torch.zeros(T, H, R, **f), torch.zeros(T, H, **f)
    q = q.double()
    for t, rows in enumerate(lists):
        if not rows:
            continue
        k, top = held[rows], scales[rows].abs().amax(-1).clamp(min=2.0 ** -74)  # (2^e is at least 2^-80)
        n = len(rows)
        s = q[t] @ k.T * scale
        lse[t] = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[t][:, None])
        out[t] = p @ k[:, :R]
        off = 450 * 2.0 ** -25 * top / 64
        ds = scale * ((H16 + (R + P + 8) * U32) * (q[t].abs() @ k.abs().T) + 2.0 ** -33 * q[t][:, :R].abs().amax(-1)[:, None]
                      * k[:, :R].abs().sum(-1) + q[t][:, :R].abs().sum(-1)[:, None] * off)
        ds = ds + 8 * U32 * (s.abs() + lse[t].abs()[:, None])
        moved = torch.exp(s - lse[t][:, None] + ds) - p  # of the weights
        rel = H16 + (n + 16) * U32
        size = p @ k[:, :R].abs()
        small = n * 2.0 ** -30 * (p * top / 64).amax(-1) * 2.0 ** 16
        tol[t] = (moved @ k[:, :R].abs() + moved.sum(-1)[:, None] * out[t].abs() + (2 * H16 + rel) * size
                  + (p @ off)[:, None] + small[:, None] + half_step(dtype) * out[t].abs())
        tol_lse[t] = moved.sum(-1) + (n + 16) * U32 + 4 * U32 * lse[t].abs()
    return out, lse, 1.01 * tol, 1.01 * tol_lse


def check(dev, q, rows, held, scales, lists, scale, call):
    import sparse_attention_kv_row_gb300 as hs

    T, H, _ = q.shape
    out, lse = torch.zeros(T, H, R, dtype=q.dtype, device=dev), torch.zeros(T, H, device=dev)
    call(hs, q.to(dev), rows.to(dev), out, lse)
    ref, ref_lse, tol, tol_lse = plain(q, held, scales, lists, scale, q.dtype)
    got, got_lse = out.cpu().double(), lse.cpu().double()
    err = (got - ref).abs()
    assert bool((err <= tol).all()), f"{int((~(err <= tol)).sum())} outputs off, worst {float((err / tol).nan_to_num(9e9).max()):.3g} of the bound"
    err = (got_lse - ref_lse).abs()
    assert bool((err <= tol_lse).all()), f"lse, worst {float((err / tol_lse).max()):.3g} of the bound"
    return out, lse


def indexed(dev, q, rows, held, scales, index, scale):
    lists = [[int(e) for e in row if e >= 0] for row in index]

    def call(hs, q, rows, out, lse):
        hs.latent_attention(q, rows, torch.tensor(index, dtype=torch.int32, device=dev), out, scale=scale, lse=lse)

    return check(dev, q, rows, held, scales, lists, scale, call)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads", [3, 20, 64])
@pytest.mark.parametrize("place", [0, 100, 500])
@pytest.mark.parametrize("power", [10, 22, 31, 60, 110])
def test_large_row_without_weight(dev, dtype, heads, place, power):
    """A row 2^power times the others whose score is so far below theirs that it has no weight."""
    dt = TORCH[dtype]
    g = torch.Generator().manual_seed(power)
    n = 600
    codes, scales, pe = some(g, n, dt, 2.0 ** -7)
    # the first dim carries every score: small for the others, far below zero for the large row
    codes[:, 0] = 1.0
    codes[place, 0] = -256.0
    scales[place] = 2.0 ** (power - 7)
    rows, held = rows_of(codes, scales, pe)
    q = torch.zeros(2, heads, R + P)
    q[..., 0] = 64.0
    q[..., R:] = torch.randn(2, heads, P, generator=g)
    q = q.to(dt)
    index = [list(range(n)), list(range(n - 1, -1, -1))]
    indexed(dev, q, rows, held, scales, index, 0.125)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads", [3, 20, 64])
@pytest.mark.parametrize("power,apart", [(12, 12), (31, 31), (31, 20), (31, 40), (50, 55)])
def test_large_row_of_small_weight(dev, dtype, heads, power, apart):
    """Row 300 is 2^power times the others in three of its groups, and its weight 2^-apart of theirs;
    the first group and the rotary dims alone make the scores."""
    dt = TORCH[dtype] if power < 50 or dtype == "bf16" else torch.bfloat16
    g = torch.Generator().manual_seed(power)
    n = 500
    codes, scales, pe = some(g, n, dt, 2.0 ** -7)
    scales[300, 1:] = 2.0 ** (power - 7)
    codes[:, :GROUP] = 0.0
    pe.zero_()
    pe[:, 0] = torch.rand(n, generator=g).to(dt)
    pe[300, 0] = -float(apart)
    rows, held = rows_of(codes, scales, pe)
    q = torch.zeros(2, heads, R + P)
    q[..., R] = 1.0
    q = q.to(dt)
    if dt == torch.float16:  # (outputs within fp16)
        rows, held = rows_of(codes, scales * 2.0 ** -10, pe)
        scales = scales * 2.0 ** -10
    index = [list(range(n)), list(range(n - 1, -1, -1))]
    indexed(dev, q, rows, held, scales, index, float(np.log(2.0)))


@pytest.mark.parametrize("heads", [3, 20, 64])
@pytest.mark.parametrize("power", [-66, -40, 40, 60, 100])
def test_all_rows_small_or_large(dev, heads, power):
    g = torch.Generator().manual_seed(abs(power))
    codes, scales, pe = some(g, 700, torch.bfloat16, 2.0 ** power)
    pe.mul_(2.0 ** min(power + 7, 0))
    rows, held = rows_of(codes, scales, pe)
    size = min(2.0, 2.0 ** -(power + 9))
    q = (size * torch.randn(2, heads, R + P, generator=g)).to(torch.bfloat16)
    index = torch.stack([torch.randperm(700, generator=g)[:650] for _ in range(2)]).tolist()
    indexed(dev, q, rows, held, scales, index, (R + P) ** -0.5)


@pytest.mark.parametrize("heads", [3, 20, 64])
def test_equal_scores_of_rows_far_apart(dev, heads):
    """Queries of zeros: every row has the same weight, whatever its scale; some are zeros."""
    g = torch.Generator().manual_seed(3)
    n = 450
    codes, scales, pe = some(g, n, torch.bfloat16, 1.0)
    scales *= 2.0 ** torch.randint(-60, 61, (n, 1), generator=g).double()
    scales[::7] = 0.0
    rows, held = rows_of(codes, scales, pe)
    q = torch.zeros(2, heads, R + P, dtype=torch.bfloat16)
    index = torch.stack([torch.randperm(n, generator=g)[:400] for _ in range(2)]).tolist()
    indexed(dev, q, rows, held, scales, index, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads", [3, 20, 64])
@pytest.mark.parametrize("apart", [8, 14, 17, 20, 24])
@pytest.mark.parametrize("seen", [1, 250])
def test_small_groups(dev, dtype, heads, apart, seen):
    """A group 2^-apart of its row's largest, with scales that are no powers of two; a single row's
    outputs are its values."""
    dt = TORCH[dtype]
    g = torch.Generator().manual_seed(apart)
    n = 260
    codes, scales, pe = some(g, n, dt, 1.0)
    scales[:, 2] *= 2.0 ** -apart
    scales *= 0.5 + 0.5 * torch.rand(n, GROUPS, generator=g).double()
    scales = scales.float().double()
    rows, held = rows_of(codes, scales, pe)
    q = (0.05 * torch.randn(2, heads, R + P, generator=g)).to(dt)
    if seen == 1:
        q.zero_()
    index = torch.stack([torch.randperm(n, generator=g)[:seen] for _ in range(2)]).tolist()
    indexed(dev, q, rows, held, scales, index, (R + P) ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,new", [(1, 5), (4, 4), (5, 5), (8, 6), (16, 3), (64, 2), (20, 3)])
@pytest.mark.parametrize("ctx", [3, 126, 500])
def test_rows_of_later_tokens(dev, dtype, heads, new, ctx):
    """The last token's own row, which no earlier token of the request sees: whatever scale it has,
    the earlier tokens' outputs are the same bits."""
    import sparse_attention_kv_row_gb300 as hs

    dt = TORCH[dtype]
    g = torch.Generator().manual_seed(ctx)
    n = ctx + new
    q = (0.1 * torch.randn(new, heads, R + P, generator=g)).to(dt)
    codes, scales, pe = some(g, n, dt, 2.0 ** -7)
    table = torch.arange(n, dtype=torch.int32, device=dev)[None]
    cu = torch.tensor([0, new], dtype=torch.int32, device=dev)
    seq = torch.tensor([n], dtype=torch.int64, device=dev)
    req = torch.zeros(1, dtype=torch.int64, device=dev)
    lists = [list(range(ctx + i + 1)) for i in range(new)]
    first = None
    for power in (-7, 13, 24, 53, 105, -40):
        scales[n - 1] = 2.0 ** power
        rows, held = rows_of(codes, scales, pe)
        out, lse = torch.zeros(new, heads, R, dtype=dt, device=dev), torch.zeros(new, heads, device=dev)
        hs.paged_latent_attention(q.to(dev), rows.to(dev), table, req, cu, seq, out, max_q_len=new, page_size=1,
                                  scale=(R + P) ** -0.5, lse=lse)
        if first is None:
            first = out, lse
            ref, ref_lse, tol, tol_lse = plain(q, held, scales, lists, (R + P) ** -0.5, dt)
            assert bool(((out.cpu().double() - ref).abs() <= tol).all())
            assert bool(((lse.cpu().double() - ref_lse).abs() <= tol_lse).all())
        assert torch.equal(out[:-1], first[0][:-1]) and torch.equal(lse[:-1], first[1][:-1]), power
