"""The serving operators one after another, as a decode loop uses them: slots from
lengths, norm and rotation with the cache write, attention over the cache; prompts
first, then tokens one by one, eagerly and as one captured graph that carries
lengths and free blocks from replay to replay; and attention over caches that
store_kv and fp8_store_kv wrote."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_cases import U32, attention_plain, half_step, norm_rope_plain, slots_plain

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__

    __graft_entry__.build()
    return torch.device("cuda:0")


class Server:
    """Device state of a few requests, and the same state in plain arrays."""

    def __init__(self, dev, cache, dim, heads, kv_heads, bs=16, blocks=40, cols=6, B=5):
        import sparse_attention_kv_row_gb300 as hs

        self.hs, self.dev, self.bs, self.B = hs, dev, bs, B
        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        g = torch.Generator().manual_seed(dim)
        self.g, self.fp8 = g, cache == "fp8"
        self.free = np.random.default_rng(1).permutation(blocks).astype(np.int32)
        self.req = np.array([3, 0, -1, 5, 1][:B], np.int64)
        self.top, self.table = blocks, np.full((7, cols), -1, np.int32)
        self.len = np.zeros(B, np.int64)
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        self.d = dict(req=t(self.req), table=t(self.table), free=t(self.free), len=t(self.len),
                      top=t(np.array([blocks], np.int32)))
        kind = torch.uint8 if self.fp8 else torch.bfloat16
        self.kc = torch.zeros(blocks, bs, kv_heads, dim, dtype=kind, device=dev)
        self.vc = torch.zeros_like(self.kc)
        self.qw = (1 + 0.2 * torch.randn(dim, generator=g)).to(torch.bfloat16)
        self.kw = (1 + 0.2 * torch.randn(dim, generator=g)).to(torch.bfloat16)
        half = dim // 2
        a = torch.arange(cols * bs, dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(half, dtype=torch.float64) / half)
        self.cs = torch.cat([a.cos(), a.sin()], 1).float()
        self.scales = (0.02, 0.03) if self.fp8 else (1.0, 1.0)
        self.dw = dict(qw=self.qw.to(dev), kw=self.kw.to(dev), cs=self.cs.to(dev))
        self.ds = [torch.tensor([x], device=dev) if self.fp8 else None for x in self.scales]

    def buffers(self, max_tokens):
        z = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt, device=self.dev)  # noqa: E731
        i64, bf = torch.int64, torch.bfloat16
        return dict(new=z(self.B), cu=z(self.B + 1), loc=z(max_tokens, dt=i64), pos=z(max_tokens, dt=i64),
                    row=z(max_tokens), slot_st=z(self.B), norm_st=z(1), attn_st=z(self.B),
                    qkv=z(max_tokens, self.heads + 2 * self.kv_heads, self.dim, dt=bf),
                    q=z(max_tokens, self.heads, self.dim, dt=bf),
                    out=z(max_tokens, self.heads, self.dim, dt=bf) - 7)

    def step(self, b, max_q):
        hs, d, h, k = self.hs, self.d, self.heads, self.kv_heads
        hs.assign_slots(d["len"], b["new"], d["req"], d["table"], d["free"], d["top"],
                        block_size=self.bs, cu_new=b["cu"], seq_lens=d["len"], cache_loc=b["loc"],
                        positions=b["pos"], token_row=b["row"], status=b["slot_st"])
        x = b["qkv"]
        hs.qk_norm_rope_store(x[:, :h], x[:, h:h + k], x[:, h + k:], self.dw["qw"], self.dw["kw"],
                              self.dw["cs"], b["pos"], b["q"], self.kc, self.vc, b["loc"], eps=EPS,
                              k_scale=self.ds[0], v_scale=self.ds[1], page_size=self.bs,
                              status=b["norm_st"])
        hs.paged_attention(b["q"], self.kc, self.vc, d["table"], d["req"], b["cu"], d["len"], b["out"],
                           max_q_len=max_q, k_scale=self.ds[0], v_scale=self.ds[1],
                           page_size=self.bs, status=b["attn_st"])

    def check(self, b, new, qkv, padded):
        """Every intermediate of the step that just ran; `new` and `qkv` are what it was given."""
        torch.cuda.synchronize()
        max_tokens = b["loc"].numel()
        ref = slots_plain(self.len, new, self.req, self.table, self.free, self.top, self.bs, max_tokens)
        self.len, self.table, self.top = ref["seq_lens"], ref["table"], ref["free_top"]
        for name, key in (("cu", "cu_new"), ("loc", "cache_loc"), ("pos", "positions"),
                          ("row", "token_row"), ("slot_st", "status")):
            np.testing.assert_array_equal(b[name].cpu().numpy(), ref[key], err_msg=name)
        np.testing.assert_array_equal(self.d["table"].cpu().numpy(), self.table)
        np.testing.assert_array_equal(self.d["len"].cpu().numpy(), self.len)
        assert int(self.d["top"]) == self.top
        T = int(ref["cu_new"][-1])
        assert int(b["norm_st"]) == (64 if padded else 0)  # slots of -1 behind the last token
        b["norm_st"].zero_()
        h, k, D = self.heads, self.kv_heads, self.dim
        turn = self.cs[torch.from_numpy(ref["positions"][:T])]
        rel = (D / 2 + 12) * U32
        z, both = norm_rope_plain(qkv[:T, :h], self.qw, turn, EPS, False)
        q = b["q"][:T].cpu()
        assert bool(((q.double() - z).abs() <= rel * both + half_step(q.dtype) * z.abs() * 1.01).all())
        z, both = norm_rope_plain(qkv[:T, h:h + k], self.kw, turn, EPS, False)
        loc = torch.from_numpy(ref["cache_loc"][:T])
        kc, vc = self.kc.cpu(), self.vc.cpu()
        if self.fp8:
            kc, vc = kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn)
        got = kc.flatten(0, 1).double()[loc]
        sc = self.scales[0]
        bound = (2.0 ** -4 * (z / sc).abs() + 2.0 ** -10 if self.fp8
                 else half_step(torch.bfloat16) * z.abs() * 1.01) + 2 * rel * both / sc
        assert bool(((got - (z / sc).clamp(-448, 448) if self.fp8 else got - z).abs() <= bound).all())
        if not self.fp8:
            assert torch.equal(vc.flatten(0, 1)[loc], qkv[:T, h + k:])
        out, lse, size, unit, n, seen = attention_plain(
            q, kc, vc, self.table, self.req, ref["cu_new"], self.len, scale=D ** -0.5,
            ks=self.scales[0], vs=self.scales[1])
        up = half_step(torch.float16 if self.fp8 else torch.bfloat16)
        tol = 1.01 * ((2 * (D + 4) * U32 * unit + (2 * n[:, None] + 16) * U32 + up)[..., None] * size
                      + half_step(torch.bfloat16) * out.abs())
        assert bool(seen.all())
        got = b["out"].cpu()
        assert bool(((got[:T].double() - out).abs() <= tol).all())
        assert bool((got[T:] == -7).all())
        assert not bool(b["attn_st"].any())


@pytest.mark.parametrize("cache", ["same", "fp8"])
@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 6, 2), (128, 8, 1), (40, 4, 2)])
def test_prompts_then_tokens(dev, cache, dim, heads, kv_heads):
    s = Server(dev, cache, dim, heads, kv_heads)
    for new in ([33, 5, 9, 0, 60], [1, 12, 1, 20, 7], [1, 1, 1, 1, 1], [0, 3, 2, 1, 2]):
        new = np.array(new, np.int32)
        T = int(new[s.req >= 0].sum())
        b = s.buffers(T)
        b["new"].copy_(torch.from_numpy(new))
        qkv = torch.randn(b["qkv"].shape, generator=s.g).to(torch.bfloat16)
        b["qkv"].copy_(qkv)
        s.step(b, int(new.max()))
        s.check(b, new, qkv, False)


@pytest.mark.parametrize("cache", ["same", "fp8"])
@pytest.mark.parametrize("chunk", [1, 3])
def test_captured_decode_loop(dev, cache, chunk):
    """One graph for a step of at most `chunk` tokens a request, replayed with other inputs;
    the buffers have room for more tokens than a step has."""
    s = Server(dev, cache, 128, 16, 2)
    b = s.buffers(s.B * chunk + 2)
    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):  # a step of no tokens loads everything
        s.step(b, chunk)
    torch.cuda.synchronize()
    b["norm_st"].zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step(b, chunk)
    rng = np.random.default_rng(3)
    for _ in range(20):
        new = rng.integers(0, chunk + 1, s.B).astype(np.int32)
        qkv = torch.randn(b["qkv"].shape, generator=s.g).to(torch.bfloat16)
        b["new"].copy_(torch.from_numpy(new))
        b["qkv"].copy_(qkv)
        b["out"].fill_(-7)
        graph.replay()
        s.check(b, new, qkv, True)


@pytest.mark.parametrize("fp8", [False, True])
def test_over_caches_of_the_movers(dev, fp8):
    """store_kv and fp8_store_kv write the cache, paged_attention reads it."""
    import sparse_attention_kv_row_gb300 as hs

    g = torch.Generator().manual_seed(1)
    T, H, HK, D, bs = 150, 8, 2, 128, 16
    x = torch.randn(2, T, HK, D, generator=g).to(torch.bfloat16)
    q = (2 * torch.randn(T, H, D, generator=g)).to(torch.bfloat16)
    table = np.random.default_rng(0).permutation(14)[:10].astype(np.int32)[None]
    pos = np.arange(T)
    loc = torch.from_numpy(table[0, pos // bs].astype(np.int64) * bs + pos % bs).to(dev)
    kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
    kc = torch.zeros(14, bs, HK, D, dtype=torch.bfloat16, device=dev).to(kind)
    vc = torch.zeros_like(kc)
    k, v = x[0].to(dev), x[1].to(dev)
    sc = [torch.tensor([0.01], device=dev)] * 2 if fp8 else [None, None]
    if fp8:
        hs.fp8_store_kv(k, v, kc, vc, loc, k_scale=sc[0], v_scale=sc[1], page_size=bs)
    else:
        hs.store_kv(k, v, kc.flatten(0, 1), vc.flatten(0, 1), loc)
    out = torch.zeros(T, H, D, dtype=torch.bfloat16, device=dev)
    i = lambda *a, dt=torch.int32: torch.tensor(a, dtype=dt, device=dev)  # noqa: E731
    hs.paged_attention(q.to(dev), kc, vc, torch.from_numpy(table).to(dev), i(0), i(0, T), i(T), out,
                       max_q_len=T, k_scale=sc[0], v_scale=sc[1], page_size=bs)
    s = 0.01 if fp8 else 1.0
    ref, _, size, unit, n, _ = attention_plain(q, kc.cpu(), vc.cpu(), table, [0], [0, T], [T],
                                               scale=D ** -0.5, ks=s, vs=s)
    up = half_step(torch.float16 if fp8 else torch.bfloat16)
    tol = 1.01 * ((2 * (D + 4) * U32 * unit + (2 * n[:, None] + 16) * U32 + up)[..., None] * size
                  + half_step(torch.bfloat16) * ref.abs())
    assert bool(((out.cpu().double() - ref).abs() <= tol).all())
