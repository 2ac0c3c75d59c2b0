"""paged_attention against a plain 64-bit statement: decode steps, short and long
chunks, mixed batches, every type and cache form, page sizes that end inside a
tile, odd head counts, windows, padding and empty rows, bad blocks, strided and
unaligned inputs; unowned cache bytes hold NaN throughout."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_cases import PagedInputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__

    __graft_entry__.build()
    return torch.device("cuda:0")


def _hs():
    import sparse_attention_kv_row_gb300 as hs

    return hs


DECODE = [(5, 1), (0, 1), (63, 1), (64, 1), (None, 0), (700, 1), (31, 1), (1500, 1)]
DRAFTS = [(40, 4), (0, 3), (None, 0), (257, 1), (600, 5), (3, 0), (127, 2)]
CHUNKS = [(0, 130), (None, 0), (300, 257), (500, 1), (77, 64), (3, 0), (0, 1), (1000, 33)]


@pytest.mark.parametrize("lens", [DECODE, DRAFTS, CHUNKS], ids=["decode", "drafts", "chunks"])
@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("f16", "same"), ("bf16", "fp8"),
                                         ("f16", "fp8")])
@pytest.mark.parametrize("dim", [64, 128])
def test_types(dev, lens, dtype, cache, dim):
    x = PagedInputs(lens, heads=8, kv_heads=2, dim=dim, dtype=dtype, cache=cache, page=16, seed=dim)
    _, _, status = x.check(_hs(), dev, True)
    assert not bool(status.any())


@pytest.mark.parametrize("dtype,cache,dim", [("f32", "same", 64), ("f32", "fp8", 128),
                                             ("bf16", "same", 40), ("f16", "fp8", 96),
                                             ("bf16", "same", 256), ("f16", "same", 1),
                                             ("bf16", "fp8", 320)])
def test_general_form(dev, dtype, cache, dim):
    x = PagedInputs([(0, 3), (70, 1), (None, 0), (33, 40), (100, 0)], heads=6, kv_heads=2, dim=dim,
                    dtype=dtype, cache=cache, page=8, seed=dim, i64=False)
    x.check(_hs(), dev, False)


@pytest.mark.parametrize("page,flat", [(1, False), (3, False), (8, True), (48, False), (64, True),
                                       (128, False), (256, False)])
@pytest.mark.parametrize("lens", [DECODE, CHUNKS], ids=["decode", "chunks"])
@pytest.mark.parametrize("cache", ["same", "fp8"])
def test_page_sizes(dev, page, flat, lens, cache):
    x = PagedInputs(lens, heads=4, kv_heads=1, dim=128, dtype="bf16", cache=cache, page=page,
                    flat=flat, seed=page)
    x.check(_hs(), dev, True)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 1), (5, 5), (12, 4), (16, 1), (7, 1), (48, 3)])
@pytest.mark.parametrize("lens", [DECODE, DRAFTS, CHUNKS], ids=["decode", "drafts", "chunks"])
def test_head_groups(dev, heads, kv_heads, lens):
    x = PagedInputs(lens, heads=heads, kv_heads=kv_heads, dim=64, dtype="f16", page=16, seed=heads)
    x.check(_hs(), dev, True)


@pytest.mark.parametrize("window", [1, 2, 33, 100, 128, 500, 100000])
@pytest.mark.parametrize("lens", [DECODE, DRAFTS, CHUNKS], ids=["decode", "drafts", "chunks"])
def test_window(dev, window, lens):
    """Blocks behind the window are given back: their entries are -1 and their bytes NaN."""
    x = PagedInputs(lens, heads=4, kv_heads=2, dim=128, dtype="bf16", page=16, window=window, seed=window)
    _, _, status = x.check(_hs(), dev, True)
    assert not bool(status.any())


def test_window_fp8(dev):
    x = PagedInputs(CHUNKS + DECODE, heads=4, kv_heads=2, dim=64, dtype="bf16", cache="fp8", page=16,
                    window=77, seed=5)
    x.check(_hs(), dev, True)


@pytest.mark.parametrize("dim,dtype,tensor_cores", [(128, "bf16", True), (80, "f16", False)])
@pytest.mark.parametrize("long", [False, True])
def test_rows_without_keys_and_bad_rows(dev, dim, dtype, tensor_cores, long):
    """A chunk longer than its sequence, an empty sequence, a state row past the table, a
    sequence past the table's blocks, too many queries; rows behind the last sequence."""
    lens = [(20, 4), (9, 3), (30, 2), (10, 40 if long else 1), (50, 1)]
    x = PagedInputs(lens, heads=4, kv_heads=2, dim=dim, dtype=dtype, page=16, seed=3, gap=3)
    x.seq[0] = 2        # two of the four queries see nothing
    x.seq[1] = 0        # none of three sees a key
    x.req[2] = x.table.shape[0]
    x.seq[4] = x.table.shape[1] * 16 + 1
    out, lse, status = x.check(_hs(), dev, tensor_cores)
    assert status.tolist() == [0, 0, 32, 0, 32]
    if long:
        _, _, status = x.check(_hs(), dev, tensor_cores, max_q=39)
        assert status.tolist() == [0, 0, 32, 32, 32]


def test_bad_cu(dev):
    x = PagedInputs([(20, 4), (9, 3), (30, 2)], heads=4, kv_heads=2, dim=128, dtype="bf16", seed=3)
    x.cu[3] = 50       # past the tokens
    x.cu[1] = 8        # row 1 runs backwards, row 0 has more queries than announced
    _, _, status = x.check(_hs(), dev, True, max_q=4)
    assert status.tolist() == [32, 32, 32]


@pytest.mark.parametrize("cache", ["same", "fp8"])
@pytest.mark.parametrize("dim,tensor_cores", [(128, True), (64, True), (48, False)])
@pytest.mark.parametrize("n", [1, 50])
def test_bad_blocks_are_zero_keys(dev, cache, dim, tensor_cores, n):
    x = PagedInputs([(300, n), (200, n), (150, 1)], heads=4, kv_heads=2, dim=dim, dtype="bf16",
                    cache=cache, page=16, seed=9)
    x.table[x.req[0], 3] = x.kc.shape[0]
    x.table[x.req[0], 7] = -1
    x.table[x.req[2], 0] = 2 ** 31 - 1
    _, _, status = x.check(_hs(), dev, tensor_cores)
    assert status.tolist() == [64, 0, 64]


@pytest.mark.parametrize("lens", [DECODE, CHUNKS], ids=["decode", "chunks"])
def test_large_and_equal_scores(dev, lens):
    """Scores of several hundred (weights that are nearly one-hot), and all scores equal."""
    for sharp in (60.0, 0.0):
        x = PagedInputs(lens, heads=4, kv_heads=1, dim=128, dtype="bf16", seed=4, sharp=sharp)
        x.check(_hs(), dev, True)


@pytest.mark.parametrize("lens", [DECODE, CHUNKS], ids=["decode", "chunks"])
def test_fp8_keeps_small_and_huge_queries(dev, lens):
    """bf16 queries beyond fp16's range on both sides, against an FP8 cache."""
    for power in (18, -30):
        x = PagedInputs(lens, heads=4, kv_heads=1, dim=128, dtype="bf16", cache="fp8", seed=4,
                        scales=(2.0 ** -5, 0.11))
        x.q *= 2.0 ** power
        x.ks *= 2.0 ** -power
        x.check(_hs(), dev, True)


@pytest.mark.parametrize("lens", [DECODE, CHUNKS], ids=["decode", "chunks"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,page,tensor_cores", [(128, 16, True), (64, 48, True), (40, 16, False)])
def test_every_fp8_code(dev, lens, dtype, dim, page, tensor_cores):
    """Caches of random codes: subnormals, both zeros, the largest; then NaN codes, which make
    the rows that see them NaN and leave the others alone."""
    x = PagedInputs(lens, heads=4, kv_heads=2, dim=dim, dtype=dtype, cache="fp8", page=page, seed=4,
                    scales=(0.003, 0.02))
    g = torch.Generator().manual_seed(1)
    for c in (x.kc, x.vc):
        codes = torch.randint(0, 256, c.shape, generator=g, dtype=torch.uint8)
        codes[(codes & 0x7F) == 0x7F] = 0x81
        c.view(torch.uint8).copy_(torch.where(c.float().isnan(), c.view(torch.uint8), codes))
    x.check(_hs(), dev, tensor_cores)
    for which in ("kc", "vc"):
        y = PagedInputs(lens, heads=4, kv_heads=2, dim=dim, dtype=dtype, cache="fp8", page=page, seed=4)
        b = 5  # a request of one token over 500 or 700
        getattr(y, which).view(torch.uint8)[y.table[y.req[3 if lens is CHUNKS else b], 100 // page],
                                            100 % page, 1, 7] = 0xFF
        out, _, _ = y.call(_hs(), dev)
        row = int(y.cu[3 if lens is CHUNKS else b])
        bad = out.float().isnan().any(-1).cpu()
        want = torch.zeros_like(bad)
        want[row, 2:] = True
        assert torch.equal(bad, want)


@pytest.mark.parametrize("lens", [DECODE, CHUNKS], ids=["decode", "chunks"])
@pytest.mark.parametrize("cache", ["same", "fp8"])
def test_views_and_layouts(dev, lens, cache):
    """q a slice of a packed projection, out strided, K and V interleaved in one cache."""
    hs = _hs()
    x = PagedInputs(lens, heads=4, kv_heads=2, dim=128, dtype="bf16", cache=cache, page=16, seed=8)
    ref = x.plain()
    tol, _ = x.tolerance(ref, True)
    packed = torch.randn(x.T, 9, 128).to(torch.bfloat16)
    packed[:, 2:6] = x.q
    q = packed.to(dev)[:, 2:6]
    both = torch.stack([x.kc.view(torch.uint8) if x.fp8 else x.kc,
                        x.vc.view(torch.uint8) if x.fp8 else x.vc], 2).to(dev)
    out = torch.full((x.T, 4, 2, 128), -7.0, dtype=torch.bfloat16, device=dev)
    t = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
    sc = lambda v: torch.tensor([v], device=dev) if x.fp8 else None  # noqa: E731
    hs.paged_attention(q, both[:, :, 0], both[:, :, 1], t(x.table), t(x.req), t(x.cu), t(x.seq),
                       out[:, :, 0], max_q_len=x.max_q + 13, page_size=16, k_scale=sc(x.ks),
                       v_scale=sc(x.vs))
    seen = ref[5]
    assert bool(((out[:, :, 0].cpu().double() - ref[0]).abs() <= tol)[seen].all())
    assert bool((out[:, :, 1] == -7).all())


@pytest.mark.parametrize("lens", [DECODE, CHUNKS], ids=["decode", "chunks"])
@pytest.mark.parametrize("cache,page", [("same", 16), ("same", 128), ("fp8", 16), ("same", 3)])
def test_caches_with_a_page_per_head(dev, lens, cache, page):
    """[pages, heads, page, dim] memory, seen as [pages, page, heads, dim]."""
    x = PagedInputs(lens, heads=8, kv_heads=2, dim=128, dtype="bf16", cache=cache, page=page, seed=8)
    x.kc, x.vc = (c.transpose(1, 2).contiguous().transpose(1, 2) for c in (x.kc, x.vc))
    assert x.kc.to(dev).stride() == x.kc.stride()
    _, _, status = x.check(_hs(), dev, True)
    assert not bool(status.any())


@pytest.mark.parametrize("max_q", [None, 64])
def test_largest_batch(dev, max_q):
    """2048 requests of a token each, by either kernel."""
    x = PagedInputs([(i % 5, 1) for i in range(2048)], heads=2, kv_heads=1, dim=64, dtype="bf16", seed=3)
    _, _, status = x.check(_hs(), dev, True, **({"max_q": max_q} if max_q else {}))
    assert not bool(status.any())


@pytest.mark.parametrize("heads,tensor_cores", [(100, True), (128, True), (200, False)])
def test_many_query_heads_to_one(dev, heads, tensor_cores):
    x = PagedInputs([(40, 1), (3, 5), (300, 2)], heads=heads, kv_heads=1, dim=64, dtype="bf16", seed=3)
    x.check(_hs(), dev, tensor_cores)


def test_unaligned_caches_and_queries(dev):
    """Addresses that allow no 16-byte loads."""
    hs = _hs()
    x = PagedInputs([(40, 1), (100, 30)], heads=4, kv_heads=2, dim=64, dtype="f16", page=16, seed=8)
    ref = x.plain()
    tol, _ = x.tolerance(ref, True)

    def shifted(a, by):
        buf = torch.zeros(a.numel() + by, dtype=a.dtype, device=dev)
        v = buf[by:].view(a.shape)
        v.copy_(a)
        return v

    t = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
    for bq, bk in ((1, 0), (0, 1), (3, 5)):
        out = torch.zeros(x.q.shape, dtype=torch.float16, device=dev)
        hs.paged_attention(shifted(x.q, bq), shifted(x.kc, bk), shifted(x.vc, bk), t(x.table),
                           t(x.req), t(x.cu), t(x.seq), out, max_q_len=x.max_q, page_size=16)
        assert bool(((out.cpu().double() - ref[0]).abs() <= tol).all())


@pytest.mark.parametrize("lens", [DECODE, CHUNKS], ids=["decode", "chunks"])
def test_repeat_is_bitwise_and_streams(dev, lens):
    """The same call gives the same bits; it runs on a given stream with its own workspace."""
    hs = _hs()
    x = PagedInputs(lens, heads=8, kv_heads=2, dim=128, dtype="bf16", seed=2)
    a = x.call(hs, dev)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    b = x.call(hs, dev, stream=s)
    c = x.call(hs, dev, stream=s.cuda_stream)
    torch.cuda.synchronize()
    for u, v, w in zip(a, b, c):
        assert torch.equal(u, v) and torch.equal(u, w)


def test_batch_order_and_company(dev):
    """A request's result is that of the request alone, up to the order of fp32 sums."""
    hs = _hs()
    x = PagedInputs(DECODE + CHUNKS, heads=8, kv_heads=2, dim=64, dtype="f16", seed=2)
    x.check(hs, dev, True)


def test_one_long_context(dev):
    """One request, a long context: the keys are split over the whole GPU."""
    for lens in ([(20000, 1)], [(9000, 40)]):
        x = PagedInputs(lens, heads=4, kv_heads=1, dim=64, dtype="bf16", page=64, seed=6, sharp=1.0)
        x.check(_hs(), dev, True)


def test_many_short_requests(dev):
    lens = [(i % 7, 1 + i % 3) for i in range(700)]
    x = PagedInputs(lens, heads=2, kv_heads=1, dim=64, dtype="bf16", page=16, seed=6)
    _, _, status = x.check(_hs(), dev, True)
    assert not bool(status.any())
    lens = [(i % 7, 20 + i % 30) for i in range(150)]
    x = PagedInputs(lens, heads=2, kv_heads=1, dim=64, dtype="bf16", page=16, seed=6)
    _, _, status = x.check(_hs(), dev, True)
    assert not bool(status.any())


def test_offsets_past_32_bits(dev):
    """A cache of more than 2^32 bytes whose last pages are read."""
    hs = _hs()
    pages, ps, hk, d = 70000, 16, 8, 128  # 2.3 G elements, 4.6 GB each
    lens = [(45, 1), (100, 30)]
    x = PagedInputs(lens, heads=16, kv_heads=hk, dim=d, dtype="bf16", page=ps, seed=1)
    ref = x.plain()
    tol, _ = x.tolerance(ref, True)
    n = x.kc.shape[0]
    kc = torch.empty(pages, ps, hk, d, dtype=torch.bfloat16, device=dev)
    vc = torch.empty_like(kc)
    kc[pages - n:] = x.kc.to(dev)
    vc[pages - n:] = x.vc.to(dev)
    table = np.where(x.table >= 0, x.table + (pages - n), x.table).astype(np.int32)
    t = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
    for sel in ([0], [1]):  # the single token and the chunk
        out = torch.zeros(x.q.shape, dtype=torch.bfloat16, device=dev)
        a, e = int(x.cu[sel[0]]), int(x.cu[sel[0] + 1])
        hs.paged_attention(x.q.to(dev)[a:e], kc, vc, t(table), t(x.req[sel]),
                           torch.tensor([0, e - a], dtype=torch.int32, device=dev), t(x.seq[sel]),
                           out[a:e], max_q_len=e - a, page_size=ps)
        assert bool(((out.cpu().double() - ref[0]).abs() <= tol)[a:e].all())


def test_captured_and_replayed(dev):
    """Two captured calls with a workspace each; lengths and queries change between replays."""
    hs = _hs()
    for lens in (DECODE, CHUNKS):
        x = PagedInputs(lens, heads=8, kv_heads=2, dim=128, dtype="bf16", seed=2)
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        q, kc, vc, table, req, cu, seq = (x.q.to(dev), x.kc.to(dev), x.vc.to(dev), t(x.table),
                                          t(x.req), t(x.cu), t(x.seq))
        outs = [torch.zeros_like(q) for _ in range(2)]
        kw = dict(max_q_len=x.max_q, page_size=16)
        n = hs.paged_attention_workspace_bytes(q, kc, vc, table, req, cu, seq, outs[0], **kw)
        spaces = [torch.empty(n, dtype=torch.uint8, device=dev) for _ in outs]
        call = lambda i: hs.paged_attention(q, kc, vc, table, req, cu, seq, outs[i],  # noqa: E731
                                            workspace=spaces[i] if n else None, **kw)
        call(0)
        torch.cuda.synchronize()
        graphs = []
        for i in range(2):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[i]):
                call(i)
        streams = [torch.cuda.Stream() for _ in graphs]
        for step in range(3):
            x.seq = np.maximum(x.seq - step, 0)
            x.q = (x.q * (1 + step)).to(torch.bfloat16)
            seq.copy_(t(x.seq))
            q.copy_(x.q)
            torch.cuda.synchronize()
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
            torch.cuda.synchronize()
            ref = x.plain()
            tol, _ = x.tolerance(ref, True)
            assert torch.equal(outs[0], outs[1])
            assert bool(((outs[0].cpu().double() - ref[0]).abs() <= tol)[ref[5]].all())


def test_empty_calls(dev):
    hs = _hs()
    x = PagedInputs([(20, 0), (None, 0)], heads=4, kv_heads=2, dim=128, dtype="bf16", seed=3)
    _, _, status = x.call(hs, dev)
    assert status.tolist() == [0, 0]
    q = torch.zeros(0, 4, 128, dtype=torch.bfloat16, device=dev)
    kc = torch.zeros(0, 16, 2, 128, dtype=torch.bfloat16, device=dev)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    hs.paged_attention(q, kc, kc, torch.zeros(0, 0, dtype=torch.int32, device=dev), i32(), i32(0),
                       i32(), q.clone(), max_q_len=0)
    torch.cuda.synchronize()


def test_axes_of_one_entry_may_have_any_stride(dev):
    """One request, one token, one head, one page: torch gives such axes strides that mean nothing."""
    hs = _hs()
    g = torch.Generator(device=dev).manual_seed(1)
    for dim in (128, 40):
        q = torch.randn(dim, generator=g, device=dev).to(torch.bfloat16).as_strided((1, 1, dim), (0, 3, 1))
        kv = torch.randn(2, 1, 16, 1, dim, generator=g, device=dev).to(torch.bfloat16)
        kc, vc = (c.as_strided((1, 16, 1, dim), (1, dim, 1, 1), c.storage_offset()) for c in kv)
        table = torch.zeros(1, dtype=torch.int32, device=dev).as_strided((1, 1), (0, 0))
        out = torch.zeros(dim, dtype=torch.bfloat16, device=dev).as_strided((1, 1, dim), (7, 0, 1))
        i = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
        hs.paged_attention(q, kc, vc, table, i(0), i(0, 1), i(9), out, max_q_len=1)
        k, v = kv[0, 0, :9, 0].double(), kv[1, 0, :9, 0].double()
        w = torch.softmax(k @ q[0, 0].double() * dim ** -0.5, 0)
        assert bool(((out[0, 0].double() - w @ v).abs() <= 2.0 ** -6).all())


@pytest.mark.parametrize("dtype,cache,page,dim", [("bf16", "same", 16, 128), ("f16", "same", 48, 64),
                                                  ("bf16", "fp8", 64, 128), ("f16", "fp8", 3, 128)])
def test_waits_that_run_out_hand_control_back(dev, dtype, cache, page, dim):
    """Every bounded wait of the long-chunk kernel gives up at once: all rows report the
    time-out, and the calls that follow are right."""
    hs = _hs()
    x = PagedInputs(CHUNKS, heads=8, kv_heads=2, dim=dim, dtype=dtype, cache=cache, page=page, seed=3)
    t = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
    sc = [torch.tensor([v], device=dev) if x.fp8 else None for v in (x.ks, x.vs)]
    args = (x.q.to(dev), x.kc.to(dev), x.vc.to(dev), t(x.table), t(x.req), t(x.cu), t(x.seq))
    for _ in range(3):
        status = torch.zeros(len(CHUNKS), dtype=torch.int32, device=dev)
        hs.paged_attention_timeout_selftest(*args, torch.zeros_like(args[0]), max_q_len=x.max_q,
                                            k_scale=sc[0], v_scale=sc[1], page_size=page, status=status)
        assert status.tolist() == [16] * len(CHUNKS)
        x.check(hs, dev, True)


@pytest.mark.parametrize("cache,page", [("same", 16), ("fp8", 16), ("same", 48)])
def test_many_units_of_one_tile(dev, cache, page):
    """Several short units per SM, with one half and with two in turn: no wait runs out."""
    lens = [(0, 64 if i % 3 else 20) for i in range(70)]
    x = PagedInputs(lens, heads=32, kv_heads=8, dim=64, dtype="bf16", cache=cache, page=page, seed=3)
    _, _, status = x.check(_hs(), dev, True)
    assert not bool(status.any())


@pytest.mark.parametrize("n", [1, 40])
def test_longest_rows_are_bounded(dev, n):
    """A length past 2^30 is refused, for its row alone."""
    hs = _hs()
    x = PagedInputs([(20, 1), (30, 1), (9, n)], heads=2, kv_heads=1, dim=64, dtype="bf16",
                    page=1 << 15, seed=3)
    wide = np.zeros((x.table.shape[0], 1 << 16), np.int32)
    wide[:, :1] = x.table
    x.table = wide
    x.seq[1] = (1 << 30) + 1
    t = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
    status = torch.zeros(3, dtype=torch.int32, device=dev)
    out = torch.full(x.q.shape, -7.0, dtype=torch.bfloat16, device=dev)
    hs.paged_attention(x.q.to(dev), x.kc.to(dev), x.vc.to(dev), t(x.table), t(x.req), t(x.cu), t(x.seq),
                       out, max_q_len=n, page_size=1 << 15, status=status)
    assert status.tolist() == [0, 32, 0]
    x.req[1] = -1
    ref = x.plain()
    tol, _ = x.tolerance(ref, True)
    assert bool(((out.cpu().double() - ref[0]).abs() <= tol)[ref[5]].all())
    assert bool((out[1] == -7).all())


@pytest.mark.parametrize("cache", ["same", "fp8"])
@pytest.mark.parametrize("lens", [[(200, 1)] * 3, [(100, 3), (None, 0), (50, 200)]])
def test_one_query_row_for_every_token(dev, lens, cache):
    """q with a token stride of 0."""
    x = PagedInputs(lens, heads=8, kv_heads=2, dim=128, dtype="bf16", cache=cache, seed=11)
    x.q = x.q[:1].expand(x.T, 8, 128)
    x.check(_hs(), dev, True, q=x.q[:1].to(dev).expand(x.T, 8, 128))


def test_no_states(dev):
    """A block table of no rows: every request is refused."""
    x = PagedInputs([(20, 2), (5, 30)], heads=4, kv_heads=2, dim=64, dtype="f16", seed=12)
    x.table = x.table[:0]
    _, _, st = x.check(_hs(), dev, True)
    assert st.tolist() == [32, 32]


@pytest.mark.parametrize("lens", [[(300, 1)] * 4, [(100, 90)] * 3], ids=["split", "tiles"])
def test_own_workspaces_of_calls_at_the_same_time(dev, lens, monkeypatch):
    """A call on another stream gets no workspace that a call before it, on the current stream,
    may still be using."""
    from sparse_attention_kv_row_gb300 import _capi

    x = PagedInputs(lens, heads=8, kv_heads=2, dim=128, dtype="bf16", seed=13)
    used = []

    class Packer:
        @staticmethod
        def pack(*fields, block=_capi.PAGED_ATTENTION):
            used.append(fields[-2])
            return block.pack(*fields)

    monkeypatch.setattr(_capi, "PAGED_ATTENTION", Packer)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for kw in ({}, dict(stream=side[0]), dict(stream=side[1].cuda_stream), {}):
        x.check(_hs(), dev, True, **kw)
    assert all(used) and len(set(used[:3])) == 3 and used[0] == used[3]


@pytest.mark.parametrize("heads,kv_heads,dtype,cache", [
    (4, 2, "bf16", "same"), (4, 4, "f16", "fp8"), (16, 2, "bf16", "same"), (16, 2, "bf16", "fp8"),
    (2, 1, "f32", "same")])
def test_tokens_far_apart(dev, heads, kv_heads, dtype, cache):
    """Queries and outputs whose offsets pass 2^32 bytes."""
    x = PagedInputs([(50, 1), (70, 3)], heads=heads, kv_heads=kv_heads, dim=64, dtype=dtype,
                    cache=cache, seed=14)
    step = 1_100_000_000 // (2 if dtype == "f32" else 1) // 8 * 8  # 2.2 GB a token
    n = (x.T - 1) * step + heads * 64
    far = [torch.empty(n, dtype=x.dtype, device=dev).as_strided((x.T, heads, 64), (step, 64, 1))
           for _ in range(2)]
    far[0].copy_(x.q.to(dev))
    far[1].fill_(-7.0)
    x.check(_hs(), dev, dtype != "f32", q=far[0], out=far[1])


def _check_with_nan(x, dev, tensor_cores, b=None):
    """NaN where the plain statement has it, in outputs and log-sums alike; right elsewhere."""
    out, lse, _ = x.call(_hs(), dev)
    out, lse = out.cpu().double(), lse.cpu().double()
    ref = x.plain()
    tol_out, tol_lse = x.tolerance(ref, tensor_cores)
    nan = ref[1].isnan()
    assert bool(nan.any()) and not bool(nan.all())
    assert torch.equal(lse.isnan(), nan)
    assert torch.equal(out.isnan(), nan[..., None].expand(out.shape))
    some = ref[5][:, None] & ~nan & (ref[1] > -np.inf)
    assert bool(((out - ref[0]).abs() <= tol_out)[some].all())
    assert bool(((lse - ref[1]).abs() <= tol_lse)[some].all())
    none = ref[5][:, None] & (ref[1] == -np.inf)
    assert bool((lse[none] == -np.inf).all())


NAN_FORMS = [(8, 2, 128, "bf16", "same", 16, True), (12, 1, 64, "f16", "same", 16, True),
             (8, 2, 128, "bf16", "fp8", 16, True), (12, 1, 64, "f16", "fp8", 16, True),
             (8, 2, 128, "bf16", "same", 3, True), (8, 2, 64, "bf16", "fp8", 3, True),
             (4, 2, 40, "bf16", "same", 16, False)]


@pytest.mark.parametrize("lens", [DECODE, DRAFTS, CHUNKS], ids=["decode", "drafts", "chunks"])
@pytest.mark.parametrize("heads,kv_heads,dim,dtype,cache,page,tensor_cores", NAN_FORMS)
def test_nan_queries_and_keys_in_the_log_sum(dev, lens, heads, kv_heads, dim, dtype, cache, page,
                                             tensor_cores):
    """A row whose scores are all NaN is not a row that sees no key: its log-sum is NaN too."""
    kw = dict(heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, cache=cache, page=page, seed=21)
    x = PagedInputs(lens, **kw)
    for t in range(0, x.T, 3):  # every third token, in one head
        x.q[t, t % heads, t % dim] = np.nan
    _check_with_nan(x, dev, tensor_cores)
    x = PagedInputs(lens, **kw)
    for b in (0, 1, 5):  # every key of some requests, in one kv head
        pages = x.table[x.req[b]]
        x.kc.view(torch.uint8 if x.fp8 else x.dtype)[pages[pages >= 0], :, kv_heads - 1, 1] = (
            0x7F if x.fp8 else float("nan"))
    _check_with_nan(x, dev, tensor_cores)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("cache", ["same", "fp8"])
def test_nan_in_one_part_of_a_long_context(dev, n, cache):
    """Keys that are NaN for a stretch in the middle: whole parts of a split request."""
    x = PagedInputs([(9000, n), (40, 1)], heads=4, kv_heads=2, dim=64, dtype="bf16", cache=cache,
                    page=64, seed=22)
    pages = x.table[x.req[0], 40:80]
    x.kc.view(torch.uint8 if x.fp8 else x.dtype)[pages, :, 1] = 0x7F if x.fp8 else float("nan")
    _check_with_nan(x, dev, True)


@pytest.mark.parametrize("lens", [DECODE, DRAFTS, CHUNKS], ids=["decode", "drafts", "chunks"])
@pytest.mark.parametrize("dim,page,tensor_cores", [(128, 16, True), (64, 3, True), (40, 16, False)])
def test_scores_of_minus_infinity(dev, lens, dim, page, tensor_cores):
    """Keys whose score is -inf weigh nothing; where every key's is, the row is zeros and -inf."""
    hs = _hs()
    x = PagedInputs(lens, heads=4, kv_heads=2, dim=dim, dtype="bf16", page=page, seed=26)
    x.q[:, :, 1] = x.q[:, :, 1].abs() + 1
    finite = x.kc.clone()
    x.kc[..., 1, 1] = float("-inf")     # kv head 1: every key
    x.kc[:, ::2, 0, 1] = float("-inf")  # kv head 0: every other place of a page
    out, lse, _ = x.call(hs, dev)
    out, lse = out.cpu().double(), lse.cpu().double()
    ref = list(x.plain())
    seen = ref[5]
    assert bool((out[seen, 2:] == 0).all()) and bool((lse[seen, 2:] == -np.inf).all())
    some = seen[:, None] & (ref[1] > -np.inf)
    assert bool(some[:, :2].any()) and not bool(some[:, 2:].any())
    x.kc = finite
    ref[3] = x.plain()[3]  # sum |q k| of the finite keys, which bounds those that weigh
    tol_out, tol_lse = x.tolerance(ref, tensor_cores)
    assert bool(((out - ref[0]).abs() <= tol_out)[some].all())
    assert bool(((lse - ref[1]).abs() <= tol_lse)[some].all())


@pytest.mark.parametrize("batch,max_q", [(255, 131072), (256, 131072), (2048, 16384), (64, 524288)])
@pytest.mark.parametrize("cache", ["same", "fp8"])
def test_a_large_bound_on_chunks_changes_nothing(dev, batch, max_q, cache):
    """max_q_len is only a bound: the kernel, its workspace and the results are those of a tight one."""
    hs = _hs()
    x = PagedInputs([(i % 50, 1 + (i % 40 == 3) * 30) for i in range(batch)], heads=32, kv_heads=8,
                    dim=128, dtype="bf16", cache=cache, seed=23)
    t = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
    q, kc = x.q.to(dev), x.kc.to(dev)
    need = [hs.paged_attention_workspace_bytes(q, kc, kc, t(x.table), t(x.req), t(x.cu), t(x.seq), q,
                                               max_q_len=m, page_size=16) for m in (x.max_q, max_q)]
    assert need[0] == need[1] > 0
    tight = x.check(hs, dev, True)
    wide = x.check(hs, dev, True, max_q=max_q)
    for a, b in zip(tight, wide):
        assert torch.equal(a, b)


@pytest.mark.parametrize("length", [0, -1, -5000])
def test_more_empty_rows_than_tiles_can_be_counted(dev, length):
    """2^20 kv heads and 700 rows: one tile a unit is more than 32 bits count.  Every row is refused,
    also where its length is negative (which counts as 0)."""
    hs = _hs()
    B, heads, dim = 700, 1 << 20, 64
    q = torch.zeros(1, heads, dim, dtype=torch.bfloat16, device=dev).expand(B, heads, dim)
    out = torch.full((1, heads, dim), -7.0, dtype=torch.bfloat16, device=dev)
    kc = torch.zeros(1, 1, heads, dim, dtype=torch.bfloat16, device=dev)
    i = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)  # noqa: E731
    status = i(np.full(B, -1))
    hs.paged_attention(q, kc, kc, i(np.zeros((B, 1))), i(np.arange(B)), i(np.arange(B + 1)),
                       i(np.full(B, length)), out.expand(B, heads, dim), max_q_len=17, page_size=1,
                       status=status)
    assert bool((status == 32).all()) and bool((out == -7).all())


def test_negative_lengths_count_as_none(dev):
    """Rows of a negative length see no key: zeros and -inf, in every kernel."""
    for lens, dim, tensor_cores in ((DECODE, 64, True), (CHUNKS, 128, True), (CHUNKS, 40, False)):
        for i64 in (True, False):
            x = PagedInputs(lens, heads=4, kv_heads=2, dim=dim, dtype="bf16", seed=27, i64=i64)
            x.seq[0], x.seq[3] = -1, -2 ** 31
            _, lse, status = x.check(_hs(), dev, tensor_cores)
            assert not bool(status.any()) and bool((lse[int(x.cu[3]): int(x.cu[4])] == -np.inf).all())


def test_workspace_sizes_are_asked_for_once(dev):
    """The size follows from types, head size and the kernel: other token counts, bounds and batches
    of a running server need no new look-up."""
    hs = _hs()
    g = torch.Generator(device=dev).manual_seed(1)
    kv = torch.randn(2, 40, 16, 2, 64, generator=g, device=dev).to(torch.bfloat16)
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    table = torch.arange(36, dtype=torch.int32, device=dev).view(3, 12)
    hs._attention_workspace.cache_clear()
    for n in range(1, 60):
        q = torch.randn(n + 2, 4, 64, generator=g, device=dev).to(torch.bfloat16)
        for batch, cu in ((3, i(0, n, n + 1, n + 2)), (1, i(0, n))):
            hs.paged_attention(q, kv[0], kv[1], table, i(0, 1, 2)[:batch], cu, i(n, 40, 50)[:batch],
                               torch.empty_like(q), max_q_len=n)
    assert hs._attention_workspace.cache_info().misses <= 20


@pytest.mark.parametrize("over", [0, 1])
def test_longest_row_of_a_large_call(dev, over):
    """The bound on a row's length where units of whole tokens are counted, at its last length and
    one past it: 2^20 tokens in units of 32, 8 kv heads."""
    hs = _hs()
    T, heads, kv_heads, dim, ps = 1 << 20, 64, 8, 64, 1 << 15
    units = T // (2 * (128 // (heads // kv_heads))) + 1
    most = ((2 ** 31 - 1) // (units * kv_heads) - 8) * 128
    assert most == 1047424
    g = torch.Generator(device=dev).manual_seed(1)
    q = torch.randn(1, heads, dim, generator=g, device=dev).to(torch.bfloat16).expand(T, heads, dim)
    out = torch.full((1, heads, dim), -7.0, dtype=torch.bfloat16, device=dev).expand(T, heads, dim)
    kc = torch.zeros(1, ps, kv_heads, dim, dtype=torch.bfloat16, device=dev)
    vc = torch.ones_like(kc)
    i = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    status = i(-1)
    hs.paged_attention(q, kc, vc, torch.zeros(1, 33, dtype=torch.int32, device=dev), i(0), i(0, 1),
                       i(most + over), out, max_q_len=64, page_size=ps, status=status)
    # equal weights, each of them 1: their sums are whole numbers, and their ratio is 1
    assert status.tolist() == [32 if over else 0]
    assert bool((out[0] == (-7.0 if over else 1.0)).all())


@pytest.mark.parametrize("lens", [DECODE, DRAFTS, CHUNKS], ids=["decode", "drafts", "chunks"])
@pytest.mark.parametrize("cache", ["same", "fp8"])
def test_other_requests_values_have_no_effect(dev, lens, cache):
    """Other queries, keys and values beside a request of the same lengths: its own bits stay."""
    hs = _hs()
    kw = dict(heads=8, kv_heads=2, dim=128, dtype="bf16", cache=cache, seed=24)
    x = PagedInputs(lens, **kw)
    first = x.call(hs, dev)
    for b, (c, n) in enumerate(lens):
        if c is None or n == 0:
            continue
        y = PagedInputs(lens, **kw)
        kept = y.table[y.req[b]]
        kept, rows = kept[kept >= 0], slice(int(y.cu[b]), int(y.cu[b + 1]))
        q = torch.full_like(y.q, 1000.0)
        q[rows] = y.q[rows]
        y.q = q
        others = torch.ones(len(y.kc), dtype=torch.bool)
        others[torch.from_numpy(kept).long()] = False
        for cache_, value in ((y.kc, 400.0), (y.vc, -400.0)):
            bits = torch.uint8 if y.fp8 else torch.int16
            cache_.view(bits)[others] = torch.tensor([value]).to(cache_.dtype).view(bits)
        out, lse, _ = y.call(hs, dev)
        assert torch.equal(out[rows], first[0][rows]) and torch.equal(lse[rows], first[1][rows])


@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("cache", ["same", "fp8"])
def test_requests_alone_and_in_another_order(dev, long, cache):
    """Requests of one tile of keys are never cut: the same bits alone, together and in any order.
    Longer ones are cut elsewhere, so that their weights are rounded by another running maximum:
    each within the bound, and so within twice the bound of each other."""
    hs = _hs()
    lens = DECODE + DRAFTS + (CHUNKS if long else [])
    kw = dict(heads=4, kv_heads=2, dim=64, dtype="bf16", cache=cache)
    x = PagedInputs(lens, seed=25, **kw)
    top = x.max_q
    together = x.call(hs, dev)
    tol_out, tol_lse = x.tolerance(x.plain(), True)
    one_tile = 128 if top * 2 > 16 else 32

    def pick(order):
        """The same data with the batch rows in `order`."""
        y = PagedInputs(lens, seed=25, **kw)
        rows = [np.arange(x.cu[b], x.cu[b + 1]) for b in order]
        y.q = x.q[np.concatenate(rows)]
        y.T = len(y.q)
        y.cu = np.concatenate([[0], np.cumsum([len(r) for r in rows])]).astype(np.int32)
        y.req, y.seq = x.req[order], x.seq[order]
        out, lse, _ = y.call(hs, dev, max_q=top)
        for i, b in enumerate(order):
            mine, theirs = slice(int(y.cu[i]), int(y.cu[i + 1])), torch.from_numpy(rows[i])
            for a, c, tol in ((out, together[0], tol_out), (lse, together[1], tol_lse)):
                a, c = a[mine].cpu(), c.cpu()[theirs]
                if x.seq[b] <= one_tile:
                    assert torch.equal(a, c)
                else:
                    assert bool(((a.double() - c.double()).abs() <= 2 * tol[theirs]).all())

    pick(list(range(len(lens)))[::-1])
    for b, (c, n) in enumerate(lens):
        if c is not None and n > 0:
            pick([b])
