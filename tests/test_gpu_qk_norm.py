"""qk_norm_rope_store against a plain 64-bit statement: every type and cache form,
head sizes that fill a lane group, do not, or need the general form, both pair
orders, partial rotation, in-place queries, views, bad slots and positions."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_cases import TORCH, U32, half_step, norm_rope_plain

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__

    __graft_entry__.build()
    return torch.device("cuda:0")


def _hs():
    import sparse_attention_kv_row_gb300 as hs

    return hs


def _angles(max_pos, rot):
    half = rot // 2
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(half, dtype=torch.float64) / max(1, half))
    return torch.cat([a.cos(), a.sin()], 1).float()


def _bound(z, both, D, dtype, normed):
    """The sum of squares is off by at most D units of 2^-24, half of that in the root; the root,
    two products and the rotation by 12 more, of |y_a| + |y_b|; then one rounding."""
    rel = ((D / 2 + 12) if normed else 4) * U32
    return rel * both, half_step(dtype) * z.abs() * (1 + rel), 2.0 ** -25 if dtype == torch.float16 else 1e-38


def _check(got, z, both, D, dtype, normed, what):
    a, b, tiny = _bound(z, both, D, dtype, normed)
    err = (got.cpu().double() - z).abs()
    assert bool((err <= a + b + tiny).all()), f"{what}: {float((err / (a + b + tiny)).max()):.3g} of the bound"


def _check_fp8(codes, z, both, D, scale, normed, what):
    """Against the unrounded scaled value: half a step of E4M3 (2^-4 relative, 2^-10 among the
    subnormals) and the error of the value itself; beyond 448 it saturates."""
    t = z / scale
    rel = ((D / 2 + 16) if normed else 8) * U32
    got = codes.view(torch.float8_e4m3fn).cpu().double()
    want = t.clamp(-448, 448)
    tol = 2.0 ** -4 * t.abs() + 2.0 ** -10 + 2 * rel * both / scale
    err = (got - want).abs()
    assert bool((err <= tol).all()), f"{what}: {float((err / tol).max()):.3g} of the bound"


def _run(dev, T, H, HK, D, dtype, cache="same", rot=None, inter=False, page=16, flat=False, seed=0,
         weights=True, in_place=False, shift=0, bad=True, head_gap=0, stream=None):
    hs = _hs()
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt, rot = TORCH[dtype], D if rot is None else rot
    max_pos = 5000
    rows = H + 2 * HK + head_gap
    base = torch.randn(T, rows, D, generator=g) * torch.exp(torch.randn(T, rows, 1, generator=g))
    base[0, 0] = 0  # a head of zeros
    buf = torch.zeros(base.numel() + shift, dtype=dt, device=dev)
    qkv = buf[shift:].view(base.shape)
    qkv.copy_(base)
    host = qkv.cpu()
    q, k, v = qkv[:, :H], qkv[:, H: H + HK], qkv[:, H + HK: H + 2 * HK]
    qw = (1 + 0.3 * torch.randn(D, generator=g)).to(dt) if weights else None
    kw = (1 + 0.3 * torch.randn(D, generator=g)).to(dt) if weights else None
    cs = _angles(max_pos, rot) if rot else None
    pos = torch.from_numpy(rng.integers(0, max_pos, T))
    pages = T // page + 3
    slots = pages * page
    loc = torch.from_numpy(rng.permutation(slots)[:T].astype(np.int64))
    bad_loc = bad_pos = None
    if bad and T > 6:
        bad_loc, bad_pos = [2, 5], [1, 4]
        loc[2], loc[5] = slots, -1
        if rot:
            pos[1], pos[4] = max_pos, -3
    shape = (slots, HK, D) if flat else (pages, page, HK, D)
    fp8 = cache == "fp8"
    ks, vs = 0.037, 0.4
    kc = torch.zeros(shape, dtype=torch.uint8 if fp8 else dt, device=dev) + 3
    vc = kc.clone()
    out = q if in_place else torch.full((T, H, D), -7.0, dtype=dt, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    d = lambda x: None if x is None else x.to(dev)  # noqa: E731
    given = (d(qw), d(kw), d(cs), d(pos) if rot else None)
    loc_d, scales = d(loc), [torch.tensor([x], device=dev) for x in (ks, vs)]
    torch.cuda.synchronize()  # the uploads are on the current stream
    hs.qk_norm_rope_store(q, k, v, *given, out, kc, vc, loc_d, eps=EPS, interleaved=inter,
                          k_scale=scales[0] if fp8 else None, v_scale=scales[1] if fp8 else None,
                          page_size=page, status=status, stream=stream)
    torch.cuda.synchronize()
    turn = cs[pos.clamp(0, max_pos - 1)] if rot else None
    zq, bq = norm_rope_plain(host[:, :H], qw, turn, EPS, inter)
    zk, bk = norm_rope_plain(host[:, H: H + HK], kw, turn, EPS, inter)
    zv = host[:, H + HK: H + 2 * HK].double()
    ok_pos, ok_loc = torch.ones(T, dtype=torch.bool), torch.ones(T, dtype=torch.bool)
    if bad_loc:
        ok_loc[bad_loc] = False
        if rot:
            ok_pos[bad_pos] = False
    assert int(status) == (64 if bad_loc else 0)
    o = out.cpu()
    _check(o[ok_pos], zq[ok_pos], bq[ok_pos], D, dt, weights, "q")
    keep = host[:, :H] if in_place else torch.full_like(o, -7.0)
    assert torch.equal(o[~ok_pos], keep[~ok_pos])
    if in_place:
        assert torch.equal(qkv[:, H:].cpu(), host[:, H:])
    for c, z, both, sc, ok, normed, what in (
            (kc, zk, bk, ks, ok_pos & ok_loc, weights, "k"), (vc, zv, zv.abs(), vs, ok_loc, False, "v")):
        rows_ = c.reshape(slots, HK, D)
        if fp8:
            _check_fp8(rows_[loc[ok].to(dev)], z[ok], both[ok], D, sc, normed, what)
        elif what == "v":
            assert torch.equal(rows_.cpu()[loc[ok]], z[ok].to(dt))
        else:
            _check(rows_.cpu()[loc[ok]], z[ok], both[ok], D, dt, normed, what)
        rest = torch.ones(slots, dtype=torch.bool)
        rest[loc[ok]] = False
        assert bool((rows_.cpu()[rest] == 3).all()), f"{what}: a row that no token names"


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cache", ["same", "fp8"])
@pytest.mark.parametrize("D,rot", [(128, 128), (64, 32), (8, 8), (80, 80), (96, 64), (256, 256),
                                   (192, 64), (40, 0), (512, 128), (1024, 1024), (18, 10), (1, 0)])
@pytest.mark.parametrize("inter", [False, True])
def test_sizes(dev, dtype, cache, D, rot, inter):
    _run(dev, 23, 5, 2, D, dtype, cache=cache, rot=rot, inter=inter, seed=D)


@pytest.mark.parametrize("T", [1, 2, 31, 257, 4097])
@pytest.mark.parametrize("H,HK", [(1, 1), (32, 8), (7, 1)])
def test_tokens_and_heads(dev, T, H, HK):
    _run(dev, T, H, HK, 64, "bf16", page=64, seed=T)
    _run(dev, T, H, HK, 128, "f16", cache="fp8", flat=True, page=1, inter=True, seed=T)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 18), ("f32", 64)])
def test_in_place_views_and_no_weights(dev, dtype, D):
    rot = D // 4 * 2
    _run(dev, 50, 6, 2, D, dtype, rot=rot, in_place=True)
    _run(dev, 50, 6, 2, D, dtype, rot=rot, in_place=True, inter=True)
    _run(dev, 50, 6, 2, D, dtype, rot=rot, weights=False)
    _run(dev, 50, 6, 2, D, dtype, rot=rot, head_gap=3)
    _run(dev, 50, 6, 2, D, dtype, rot=rot, shift=1)
    _run(dev, 50, 6, 2, D, dtype, rot=rot, shift=1, in_place=True, cache="fp8")
    _run(dev, 50, 6, 2, D, dtype, rot=rot, stream=torch.cuda.Stream())


def test_special_values_into_fp8(dev):
    """v as it is: infinities saturate, NaN stays NaN, signed zeros keep their sign."""
    hs = _hs()
    x = torch.zeros(4, 3, 8, dtype=torch.bfloat16, device=dev)
    x[0, 2] = torch.tensor([float("inf"), -float("inf"), float("nan"), -0.0, 1e30, -1e30, 448., 2e-3])
    kc = torch.zeros(8, 1, 8, dtype=torch.uint8, device=dev)
    vc = torch.zeros_like(kc)
    one = torch.ones(1, device=dev)
    hs.qk_norm_rope_store(x[:, :1], x[:, 1:2], x[:, 2:], None, None, None, None,
                          torch.empty_like(x[:, :1]), kc, vc, torch.arange(4, device=dev) * 2,
                          k_scale=one, v_scale=one, page_size=1)
    got = vc[0, 0].tolist()
    assert got[:2] == [0x7E, 0xFE] and got[2] & 0x7F == 0x7F and got[3] == 0x80
    assert got[4:7] == [0x7E, 0xFE, 0x7E] and got[7] == 1


def test_agrees_with_fp8_store_kv(dev):
    """Without norm and rotation it is the FP8 KV write, code by code."""
    hs = _hs()
    g = torch.Generator(device=dev).manual_seed(1)
    T, HK, D = 300, 4, 128
    x = (torch.randn(T, 2 * HK + 1, D, generator=g, device=dev) * 40).to(torch.bfloat16)
    loc = torch.randperm(T + 20, generator=g, device=dev)[:T]
    ks, vs = torch.tensor([0.37], device=dev), torch.tensor([3.1], device=dev)
    caches = [torch.zeros(20, 16, HK, D, dtype=torch.uint8, device=dev) for _ in range(4)]
    k, v = x[:, 1: 1 + HK], x[:, 1 + HK:]
    hs.fp8_store_kv(k, v, caches[0], caches[1], loc, k_scale=ks, v_scale=vs, page_size=16)
    hs.qk_norm_rope_store(x[:, :1], k, v, None, None, None, None, torch.empty_like(x[:, :1]),
                          caches[2], caches[3], loc, k_scale=ks, v_scale=vs, page_size=16)
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


def test_offsets_past_32_bits(dev):
    """Caches of more than 2^32 bytes, written at their end."""
    hs = _hs()
    T, HK, D, ps, pages = 40, 8, 128, 64, 34000  # 2.2 G elements, 4.4 GB each
    g = torch.Generator(device=dev).manual_seed(1)
    x = torch.randn(T, 2 * HK + 1, D, generator=g, device=dev).to(torch.bfloat16)
    kc = torch.empty(pages, ps, HK, D, dtype=torch.bfloat16, device=dev)
    vc = torch.empty_like(kc)
    loc = pages * ps - 1 - torch.arange(T, device=dev)
    hs.qk_norm_rope_store(x[:, :1], x[:, 1: 1 + HK], x[:, 1 + HK:], None, None, None, None,
                          torch.empty_like(x[:, :1]), kc, vc, loc, page_size=ps)
    assert torch.equal(kc.view(-1, HK, D)[-T:].flip(0), x[:, 1: 1 + HK])
    assert torch.equal(vc.view(-1, HK, D)[-T:].flip(0), x[:, 1 + HK:])


def test_no_tokens(dev):
    hs = _hs()
    x = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=dev)
    kc = torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16, device=dev)
    hs.qk_norm_rope_store(x[:, :2], x[:, 2:3], x[:, 3:], None, None, None, None, x[:, :2], kc, kc.clone(),
                          torch.zeros(0, dtype=torch.int64, device=dev))
    torch.cuda.synchronize()


@pytest.mark.parametrize("fp8", [False, True])
def test_caches_with_a_page_per_head(dev, fp8):
    """[pages, heads, page, dim] memory, seen as [pages, page, heads, dim]."""
    hs = _hs()
    g = torch.Generator(device=dev).manual_seed(1)
    T, HK, D, ps = 60, 3, 64, 16
    x = torch.randn(T, 2 * HK + 1, D, generator=g, device=dev).to(torch.bfloat16)
    loc = torch.randperm(5 * ps, generator=g, device=dev)[:T]
    kind = torch.uint8 if fp8 else torch.bfloat16
    one = torch.ones(1, device=dev) if fp8 else None
    caches = []
    for turned in (False, True):
        kc, vc = (torch.zeros((5, HK, ps, D) if turned else (5, ps, HK, D), dtype=kind, device=dev)
                  for _ in range(2))
        if turned:
            kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
        hs.qk_norm_rope_store(x[:, :1], x[:, 1: 1 + HK], x[:, 1 + HK:], None, None, None, None,
                              torch.empty_like(x[:, :1]), kc, vc, loc, k_scale=one, v_scale=one,
                              page_size=ps)
        caches.append((kc, vc))
    for a, b in zip(*caches):
        assert torch.equal(a, b) and bool(a.view(torch.uint8).any())


def test_no_slots_and_repeated_rows(dev):
    """A cache of no pages takes no K or V and says so; one q row may stand for every token."""
    hs = _hs()
    g = torch.Generator(device=dev).manual_seed(3)
    x = torch.randn(1, 4, 64, generator=g, device=dev).to(torch.bfloat16)
    T, w = 37, torch.ones(64, dtype=torch.bfloat16, device=dev)
    kc = torch.zeros(0, 16, 1, 64, dtype=torch.bfloat16, device=dev)
    loc, st = torch.arange(T, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    got = []
    for rows in (x.expand(T, 4, 64), x.repeat(T, 1, 1)):
        out = torch.empty(T, 2, 64, dtype=torch.bfloat16, device=dev)
        st.zero_()
        hs.qk_norm_rope_store(rows[:, :2], rows[:, 2:3], rows[:, 3:], w, w, None, None, out, kc,
                              kc.clone(), loc, status=st)
        assert int(st) == 64
        got.append(out)
    assert torch.equal(*got)


@pytest.mark.parametrize("D,inter", [(128, False), (128, True), (18, False)])
def test_tokens_far_apart(dev, D, inter):
    """Inputs and outputs whose offsets pass 2^32 bytes: as near ones, bit for bit."""
    hs = _hs()
    g = torch.Generator(device=dev).manual_seed(4)
    T, step = 4, 800_000_000  # 1.6 GB a token
    x = torch.randn(T, 4, D, generator=g, device=dev).to(torch.bfloat16)
    w = torch.randn(D, generator=g, device=dev).to(torch.bfloat16)
    angle = torch.randn(T, D // 2, generator=g, device=dev)
    cs = torch.cat([angle.cos(), angle.sin()], 1)
    pos, loc = torch.arange(T, device=dev), torch.arange(T, device=dev).flip(0)

    def far(heads):
        return torch.empty((T - 1) * step + heads * D, dtype=torch.bfloat16, device=dev).as_strided(
            (T, heads, D), (step, D, 1))

    got = []
    for make in (None, far):
        src = x if make is None else make(4).copy_(x)
        out = torch.empty_like(x[:, :2]) if make is None else make(2)
        kc, vc = (torch.zeros(1, 16, 1, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
        hs.qk_norm_rope_store(src[:, :2], src[:, 2:3], src[:, 3:], w, w, cs, pos, out, kc, vc, loc,
                              interleaved=inter)
        got.append((out, kc, vc))
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,rot,inter", [(128, 128, False), (64, 32, True), (18, 10, False), (80, 0, True)])
@pytest.mark.parametrize("fp8", [False, True])
def test_heads_of_zeros_without_eps(dev, dtype, D, rot, inter, fp8):
    """With eps = 0 a head of zeros stays zero; the others are normed as ever."""
    hs = _hs()
    g = torch.Generator().manual_seed(D)
    T, H, HK, dt = 9, 3, 2, TORCH[dtype]
    x = torch.randn(T, H + 2 * HK, D, generator=g).to(dt)
    x[::2, 1] = 0   # a q head
    x[::3, 3] = 0   # a k head
    w = (1 + 0.3 * torch.randn(2, D, generator=g)).to(dt)
    cs = _angles(50, rot) if rot else None
    pos, loc = torch.arange(T) * 5, torch.arange(T).flip(0) * 2
    d = lambda a: None if a is None else a.to(dev)  # noqa: E731
    kc = torch.full((2, 16, HK, D), 3, dtype=torch.uint8 if fp8 else dt, device=dev)
    out = torch.full((T, H, D), -7.0, dtype=dt, device=dev)
    y = d(x)
    hs.qk_norm_rope_store(y[:, :H], y[:, H: H + HK], y[:, H + HK:], d(w[0]), d(w[1]), d(cs), d(pos) if rot else None,
                          out, kc, kc.clone(), d(loc), eps=0.0, interleaved=inter)
    turn = cs[pos] if rot else None
    zq, bq = (a.nan_to_num(nan=0.0) for a in norm_rope_plain(x[:, :H], w[0], turn, 0.0, inter))
    zk, bk = (a.nan_to_num(nan=0.0) for a in norm_rope_plain(x[:, H: H + HK], w[1], turn, 0.0, inter))
    _check(out, zq, bq, D, dt, True, "q")
    assert bool((out[::2, 1] == 0).all())
    got = kc.view(-1, HK, D)[d(loc)]
    if fp8:
        _check_fp8(got, zk, bk, D, 1.0, True, "k")
    else:
        _check(got, zk, bk, D, dt, True, "k")
