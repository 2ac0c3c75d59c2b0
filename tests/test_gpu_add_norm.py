"""add_rms_norm against its statement in 64 bits: types, sizes, groups, aliases, strides."""
from __future__ import annotations

import math

import pytest
import torch

from latent_cases import check_codes, norm_error, norm_plain
from paged_cases import TORCH, U32, half_step

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__

    __graft_entry__.build()
    return torch.device("cuda:0")


def run(dev, T, D, dtype, *, residual=True, out=True, group=None, pow2=False, weight=True, eps=EPS,
        seed=0, pad=0, x=None, uint8=False, transposed=False, alias=None):
    import sparse_attention_kv_row_gb300 as hs

    dt = TORCH[dtype]
    g = torch.Generator().manual_seed(seed)
    wide = torch.exp(torch.randn(D, generator=g))
    if x is None:
        x = (torch.randn(T, D, generator=g) * wide).to(dt)
    res = (4 * torch.randn(T, D, generator=g) * wide).to(dt) if residual else None
    w = (1 + 0.2 * torch.randn(D, generator=g)).to(dt) if weight else None

    def put(t, fill=None):
        """On the device, `pad` entries behind every row (which stay as they are)."""
        wide_t = torch.full((T, D + pad), -3.0, device=dev, dtype=torch.float32).to(t.dtype)
        wide_t[:, :D] = t.to(dev) if fill is None else fill
        return wide_t[:, :D], wide_t

    dx, dx_all = put(x)
    dres, _ = put(res) if residual else (None, None)
    keep, keep_all = put(x, -7.0) if residual else (None, None)
    o, o_all = put(x, -7.0) if out else (None, None)
    if alias == "in place":          # the sum over the residual, the result over x
        keep, o = (None if residual else None), dx if out else None
        keep_all, o_all = None, dx_all if out else None
    elif alias == "crossed":         # the sum over x, the result over the residual
        keep, o, keep_all, o_all = dx, dres if out else None, dx_all, None
    codes = scales = None
    if group is not None:
        groups = -(-D // group) if group else 1
        codes = torch.zeros(T, D + pad, dtype=torch.uint8, device=dev)[:, :D]
        codes = codes if uint8 else codes.view(torch.float8_e4m3fn)
        scales = torch.full((groups, T), -7.0, device=dev).t() if transposed else \
            torch.full((T, groups), -7.0, device=dev)
    hs.add_rms_norm(dx, None if w is None else w.to(dev), o, residual=dres, residual_out=keep, eps=eps,
                    codes=codes, scales=scales, group=group or 0, pow2_scales=pow2)
    torch.cuda.synchronize()
    r = x
    if residual:
        r = (x.float() + res.float()).to(dt)
        got = (dres if alias == "in place" else keep).cpu()
        assert torch.equal(got, r), "the kept sum"
    for a in (keep_all, o_all):
        if a is not None and pad:
            assert bool((a[:, D:].float() == -3).all()), "behind the rows"
    y = norm_plain(r, w, eps)
    rel = norm_error(D)
    if out:
        u = half_step(dt) if dt != torch.float32 else U32
        tiny = 2.0 ** -25 if dt == torch.float16 else 0.0
        err = (o.cpu().double() - y).abs()
        assert bool((err <= 1.01 * (rel + u) * y.abs() + tiny).all()), float((err / y.abs().clamp(min=1e-9)).max())
    if group is not None:
        check_codes(y, rel, codes.cpu().view(torch.uint8), scales.cpu(), group, pow2)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,D", [(1, 8), (3, 128), (5, 1000), (2, 4096), (7, 2304), (1, 16384),
                                 (400, 256), (401, 1024), (333, 1032), (310, 4104)])
def test_sizes(dev, dtype, T, D):
    run(dev, T, D, dtype, group=128, seed=T)
    run(dev, T, D, dtype, residual=False, group=0, seed=T + 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1, 7, 33, 4099, 65536])
def test_general(dev, dtype, D):
    run(dev, 3, D, dtype, group=128)
    run(dev, 3, D, dtype, residual=False, group=0)


@pytest.mark.parametrize("group", [8, 16, 64, 256, 24, 1, 1000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_groups(dev, group, dtype):
    run(dev, 5, 1040, dtype, group=group)
    run(dev, 5, 1040, dtype, group=group, pow2=True, transposed=True, uint8=True)


@pytest.mark.parametrize("T", [4, 700])
@pytest.mark.parametrize("alias", ["in place", "crossed"])
@pytest.mark.parametrize("D", [512, 2048, 1001])
def test_in_place(dev, T, alias, D):
    run(dev, T, D, "bf16", alias=alias, group=128)
    if alias == "in place":
        run(dev, T, D, "f16", residual=False, alias=alias, group=0)


@pytest.mark.parametrize("pad", [8, 3])
def test_strides(dev, pad):
    run(dev, 9, 1024, "bf16", pad=pad, group=128)
    run(dev, 500, 512, "f32", pad=pad, group=0)


def test_without_weight_or_norm_eps(dev):
    run(dev, 6, 512, "bf16", weight=False, eps=0.0, group=128)
    run(dev, 6, 512, "f16", weight=False, eps=1.0, out=False, group=0)


def test_zeros_and_tiny(dev):
    x = torch.zeros(4, 512)
    x[1, 130] = 2.0 ** -20
    x[2] = 1e-30
    run(dev, 4, 512, "f32", x=x, residual=False, eps=0.0, group=128)
    run(dev, 4, 512, "bf16", x=x.to(torch.bfloat16), residual=False, eps=1e-6, group=128, pow2=True)


@pytest.mark.parametrize("size", [1e-36, 1e-20, 1e25, 1e37])
@pytest.mark.parametrize("T,D", [(3, 512), (400, 256), (3, 1001)])
def test_squares_out_of_range(dev, size, T, D):
    """Values whose squares leave fp32's range."""
    x = torch.randn(T, D, generator=torch.Generator().manual_seed(1)) * size
    run(dev, T, D, "f32", x=x, residual=False, eps=0.0, group=128)


@pytest.mark.parametrize("size", [2.0 ** -148, 2.0 ** -140, 1e-40, 2.0 ** -128, 1e-37, 8e37])
@pytest.mark.parametrize("T,D", [(3, 512), (400, 256), (3, 1001)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_subnormal_and_largest_values(dev, size, T, D, dtype):
    """Roots whose inverse leaves fp32's range; some of the values, and a whole token, are zeros."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(T, D, generator=g).clamp(-4, 4).double() * size
    x[torch.rand(T, D, generator=g) < 0.2] = 0.0
    x[-1] = 0.0
    x[1, :-1] = 0.0  # one value alone
    x[1, -1] = size
    run(dev, T, D, dtype, x=x.to(TORCH[dtype]), residual=False, eps=0.0, group=128)
    run(dev, T, D, dtype, x=x.to(TORCH[dtype]), residual=False, eps=0.0, group=0, out=False, pow2=True)


def test_nan_and_infinity(dev):
    import sparse_attention_kv_row_gb300 as hs

    for D in (512, 513):
        x = torch.ones(3, D, dtype=torch.bfloat16, device=dev)
        x[0, 3], x[1, 200] = math.nan, math.inf
        out = torch.zeros_like(x)
        groups = -(-D // 128)
        codes, scales = torch.zeros(3, D, dtype=torch.uint8, device=dev), torch.zeros(3, groups, device=dev)
        hs.add_rms_norm(x, None, out, codes=codes, scales=scales, group=128)
        f = out.float().cpu()
        assert bool(f[0].isnan().all()) and bool(f[1, 200].isnan()) and int(f[1].isnan().sum()) == 1
        assert bool((f[1][~f[1].isnan()] == 0).all()) and bool(f[2].isfinite().all())
        c, s = codes.cpu() & 0x7F, scales.cpu()
        assert bool((c[0] == 0x7F).all()) and bool(s[0].isnan().all())
        assert s[1].isnan().tolist() == [g == 1 for g in range(groups)] and bool((c[1, 128:256] == 0x7F).all())
        assert bool(s[2].isfinite().all())


def test_stream_and_graph(dev):
    """On another stream than the current one, and captured: replays take what the inputs hold then."""
    import sparse_attention_kv_row_gb300 as hs

    x = torch.randn(64, 1024, device=dev).to(torch.bfloat16)
    res, out = torch.zeros_like(x), torch.zeros_like(x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    hs.add_rms_norm(x, None, out, residual=res, stream=s)
    s.synchronize()
    assert torch.equal(res, x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hs.add_rms_norm(x, None, out, residual=res)
    res.zero_()
    for n in range(1, 4):
        x.copy_(torch.full_like(x, float(n)))
        g.replay()
        torch.cuda.synchronize()
        assert bool((res == sum(range(1, n + 1))).all())
        assert bool((out == 1).all())


def test_long_offsets(dev):
    """Rows whose offsets pass 32 bits."""
    import sparse_attention_kv_row_gb300 as hs

    T, D, stride = 3, 512, (1 << 30) + 64
    buf = torch.zeros(2 * stride + D, dtype=torch.bfloat16, device=dev)
    x = buf.as_strided((T, D), (stride, 1))
    x.copy_(torch.randn(T, D, device=dev))
    out = torch.zeros(T, D, dtype=torch.bfloat16, device=dev)
    hs.add_rms_norm(x, None, out)
    y = norm_plain(x.cpu(), None, EPS)
    assert bool(((out.cpu().double() - y).abs() <= (norm_error(D) + 2.0 ** -8) * y.abs() * 1.01).all())


def test_empty(dev):
    import sparse_attention_kv_row_gb300 as hs

    x = torch.zeros(0, 512, dtype=torch.bfloat16, device=dev)
    hs.add_rms_norm(x, None, torch.zeros_like(x))
