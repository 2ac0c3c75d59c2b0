"""latent_norm_rope_store against its statement in 64 bits: formats, types, sizes, skipped tokens."""
from __future__ import annotations

import pytest
import torch

from latent_cases import GROUP, check_codes, norm_error, norm_plain, row_bytes
from paged_cases import TORCH, U32, half_step, norm_rope_plain

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__

    __graft_entry__.build()
    return torch.device("cuda:0")


def angles(max_pos, rope):
    half = rope // 2
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    return torch.cat([a.cos(), a.sin()], 1).float()


def close(got, want, rel, dt, size):
    u = half_step(dt) if dt != torch.float32 else U32
    tiny = 2.0 ** -25 if dt == torch.float16 else 0.0
    assert bool(((got.double() - want).abs() <= 1.01 * (rel * size + u * want.abs()) + tiny).all())


def run(dev, T, heads, dtype, fmt, *, R=512, P=64, inter=False, pow2=False, weight=True, rotate=True,
        seed=0, pad=0, shift=0, bad=True, in_place=False, eps=EPS, stream=None):
    import sparse_attention_kv_row_gb300 as hs

    dt = TORCH[dtype]
    g = torch.Generator().manual_seed(seed)
    kv = torch.randn(T, R + P + shift, generator=g).to(dt)
    kv[:, :R] *= torch.exp(torch.randn(T, 1, generator=g)).to(dt)
    q = torch.randn(T, heads, P + 8, generator=g).to(dt)
    w = (1 + 0.2 * torch.randn(R, generator=g)).to(dt) if weight else None
    N, max_pos = 2 * T + 3, 300
    cs = angles(max_pos, P) if rotate else None
    pos = torch.randint(0, max_pos, (T,), generator=g)
    loc = torch.randperm(N, generator=g)[:T]
    bad_pos = bad_loc = ()
    if bad and T > 4:
        loc[1], loc[3] = -1, N
        bad_loc = (1, 3)
        if rotate:
            pos[2], pos[4] = -1, max_pos
            bad_pos = (2, 4)
    if fmt == "fp8":
        rows = torch.randint(0, 256, (N, row_bytes(R, P) + pad), generator=g, dtype=torch.uint8)
        cols = row_bytes(R, P)
    else:
        rows = torch.randn(N, R + P + pad, generator=g).to(dt)
        cols = R + P
    d_kv, d_q, d_rows = kv.to(dev), q.to(dev), rows.to(dev)
    out = torch.full((T, heads, R + P), -7.0, dtype=dt, device=dev)
    q_pe, q_out = d_q[..., 8:], out[..., R:]
    if in_place:
        q_out = q_pe
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    up = lambda t: None if t is None else t.to(dev)  # noqa: E731
    torch.cuda.synchronize()
    hs.latent_norm_rope_store(d_kv[:, shift:shift + R], d_kv[:, shift + R:], up(w), up(cs), up(pos) if rotate else None,
                              d_rows[:, :cols], up(loc), q_pe=q_pe if heads else None, q_out=q_out if heads else None,
                              eps=eps, interleaved=inter, pow2_scales=pow2, status=status, stream=stream)
    torch.cuda.synchronize()
    assert int(status) == (64 if bad_pos or bad_loc else 0)
    ok = torch.ones(T, dtype=torch.bool)
    ok[list(bad_pos)] = False
    turn = cs[pos.clamp(0, max_pos - 1)] if rotate else None
    if heads:
        z, both = norm_rope_plain(q[..., 8:], None, turn, 0.0, inter)
        got = q_out.cpu()
        close(got[ok], z[ok], 4 * U32, dt, both[ok])
        assert torch.equal(got[~ok], q[..., 8:][~ok] if in_place else torch.full_like(got[~ok], -7.0))
        if not in_place:
            assert bool((out[..., :R] == -7).all())
    ok[list(bad_loc)] = False
    y = norm_plain(kv[:, shift:shift + R], w, eps) if weight else kv[:, shift:shift + R].double()
    rel = norm_error(R) if weight else 0.0
    k, both = norm_rope_plain(kv[:, None, shift + R:], None, turn, 0.0, inter)
    k, both = k[:, 0], both[:, 0]
    new = d_rows.cpu()
    at = loc[ok]
    if fmt == "fp8":
        codes, scales, pe = new[at, :R], new[at, R:R + R // 32], new[at, R + R // 32:cols]
        check_codes(y[ok], rel, codes.contiguous(), scales.contiguous().view(torch.float32), GROUP, pow2)
        pe = pe.contiguous().view(dt) if P else torch.zeros(len(at), 0, dtype=dt)
    else:
        close(new[at, :R], y[ok], rel, dt, y[ok].abs())
        pe = new[at, R:cols]
    close(pe, k[ok], 4 * U32, dt, both[ok])
    new[at, :cols] = rows[at, :cols]
    assert torch.equal(new.view(torch.uint8), rows.view(torch.uint8)), "other rows"


@pytest.mark.parametrize("fmt", ["fp8", "same"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,heads", [(1, 0), (2, 1), (7, 16), (33, 17), (130, 128)])
def test_lanes(dev, fmt, dtype, inter, T, heads):
    run(dev, T, heads, dtype, fmt, inter=inter, seed=T)


@pytest.mark.parametrize("R", [256, 768, 1024])
@pytest.mark.parametrize("fmt", ["fp8", "same"])
def test_other_latents(dev, R, fmt):
    run(dev, 9, 5, "bf16", fmt, R=R)


@pytest.mark.parametrize("R,P", [(128, 64), (512, 32), (384, 2), (100, 64), (1, 6), (1000, 256), (512, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_general(dev, R, P, dtype):
    run(dev, 9, 3 if P else 0, dtype, "same", R=R, P=P, inter=R == 384, rotate=P > 0)
    if dtype != "f32" and R % 128 == 0:
        run(dev, 9, 3 if P else 0, dtype, "fp8", R=R, P=P, rotate=P > 0)


def test_alignment(dev):
    run(dev, 9, 3, "bf16", "fp8", pad=4)      # rows not on 16 bytes
    run(dev, 9, 3, "bf16", "fp8", pad=16)
    run(dev, 9, 3, "bf16", "fp8", shift=1)    # inputs not on 16 bytes
    run(dev, 9, 3, "f16", "same", pad=1, shift=3)


@pytest.mark.parametrize("R,pad", [(256, 8), (256, 56), (768, 8), (768, 24), (512, 16), (1024, 16)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_padded_rows_of_codes(dev, R, pad, dtype):
    """Rows that begin on 16 bytes; their rotary values do so for multiples of 512 only."""
    assert (row_bytes(R, 64) + pad) % 16 == 0
    run(dev, 9, 5, dtype, "fp8", R=R, pad=pad)
    run(dev, 9, 0, dtype, "fp8", R=R, pad=pad, inter=True)


def test_options(dev):
    run(dev, 9, 4, "bf16", "fp8", pow2=True)
    run(dev, 9, 4, "bf16", "fp8", weight=False, rotate=False)
    run(dev, 9, 4, "bf16", "same", weight=False, rotate=False)
    run(dev, 9, 4, "bf16", "fp8", in_place=True, inter=True)
    run(dev, 9, 4, "f32", "same", R=64, in_place=True)
    run(dev, 40, 4, "bf16", "fp8", stream=torch.cuda.Stream())


def test_zero_latent(dev):
    import sparse_attention_kv_row_gb300 as hs

    for R in (512, 128):
        z = torch.zeros(2, R + 64, dtype=torch.bfloat16, device=dev)
        rows = torch.full((4, row_bytes(R, 64)), 9, dtype=torch.uint8, device=dev)
        hs.latent_norm_rope_store(z[:, :R], z[:, R:], torch.ones(R, dtype=torch.bfloat16, device=dev), None, None,
                                  rows, torch.tensor([2, 0], device=dev), eps=0.0)
        assert bool((rows[[0, 2]] == 0).all()) and bool((rows[[1, 3]] == 9).all())


@pytest.mark.parametrize("R", [512, 384])
@pytest.mark.parametrize("dtype,fmt", [("bf16", "fp8"), ("bf16", "same"), ("f32", "same")])
@pytest.mark.parametrize("size", [2.0 ** -133, 2.0 ** -128, 1e-37, 8e37])
def test_subnormal_and_largest_latents(dev, R, dtype, fmt, size):
    """Latents whose root's inverse leaves fp32's range, zeros among them, without eps."""
    import sparse_attention_kv_row_gb300 as hs

    dt = TORCH[dtype]
    g = torch.Generator().manual_seed(5)
    x = torch.randn(6, R, generator=g).clamp(-4, 4).double() * size
    x[torch.rand(6, R, generator=g) < 0.2] = 0.0
    x[2, 1:] = 0.0  # one value alone
    x[2, 0] = size
    x[5] = 0.0
    x = x.to(dt)
    w = (1 + 0.2 * torch.randn(R, generator=g)).to(dt)
    rows = torch.zeros(8, row_bytes(R, 64), dtype=torch.uint8, device=dev) if fmt == "fp8" else \
        torch.zeros(8, R + 64, dtype=dt, device=dev)
    hs.latent_norm_rope_store(x.to(dev), torch.zeros(6, 64, dtype=dt, device=dev), w.to(dev), None, None, rows,
                              torch.arange(6, device=dev), eps=0.0)
    y, got = norm_plain(x, w, 0.0), rows[:6].cpu()
    if fmt == "fp8":
        check_codes(y, norm_error(R), got[:, :R].contiguous(), got[:, R:R + R // 32].contiguous().view(torch.float32),
                    GROUP, False)
    else:
        close(got[:, :R], y, norm_error(R), dt, y.abs())


def test_long_offsets(dev):
    """Rows whose offsets pass 32 bits."""
    import sparse_attention_kv_row_gb300 as hs

    N = (1 << 32) // 656 + 100
    rows = torch.zeros(N, 656, dtype=torch.uint8, device=dev)
    kv = torch.randn(2, 576, device=dev).to(torch.bfloat16)
    hs.latent_norm_rope_store(kv[:, :512], kv[:, 512:], None, None, None, rows, torch.tensor([N - 1, 5], device=dev))
    check_codes(kv[:, :512].cpu().double(), 0.0, rows[[N - 1, 5], :512].cpu().contiguous(),
                rows[[N - 1, 5], 512:528].cpu().contiguous().view(torch.float32), GROUP, False)


def test_empty(dev):
    import sparse_attention_kv_row_gb300 as hs

    kv = torch.zeros(0, 576, dtype=torch.bfloat16, device=dev)
    hs.latent_norm_rope_store(kv[:, :512], kv[:, 512:], None, None, None,
                              torch.zeros(3, 656, dtype=torch.uint8, device=dev),
                              torch.zeros(0, dtype=torch.int64, device=dev))
