"""latent_attention and paged_latent_attention against their statement in 64 bits."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from latent_cases import LatentInputs

pytestmark = pytest.mark.gpu



@pytest.fixture(scope="module")
def hs(dev):
    import sparse_attention_kv_row_gb300

    return sparse_attention_kv_row_gb300


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__

    __graft_entry__.build()
    return torch.device("cuda:0")


# ------------------------------------------------------------------ the general kernel
@pytest.mark.parametrize("latent,rope,dtype,fmt", [
    (512, 64, "f32", "same"), (128, 64, "bf16", "fp8"), (256, 64, "f16", "fp8"), (64, 32, "bf16", "same"),
    (100, 0, "f32", "same"), (1, 1, "f16", "same"), (512, 256, "bf16", "same")])
def test_general(hs, dev, latent, rope, dtype, fmt):
    a = LatentInputs(heads=3, dtype=dtype, fmt=fmt, latent=latent, rope=rope)
    a.indexed(5, 70, 200, empty=[2], bad=[1]).check(hs, dev, "general")
    a = LatentInputs(heads=3, dtype=dtype, fmt=fmt, latent=latent, rope=rope)
    a.paged([(40, 1), (0, 3), (None, 0), (17, 2), (0, 0)], 16, gap=2).check(hs, dev, "general")


def test_general_unaligned(hs, dev):
    """Rows and queries that allow no 16-byte accesses."""
    a = LatentInputs(heads=2, dtype="bf16", fmt="fp8").indexed(4, 40, 100)
    rows = torch.zeros(100, 660, dtype=torch.uint8, device=dev)[:, :656]
    rows.copy_(a.rows)
    a.check(hs, dev, "general", rows=rows)
    a = LatentInputs(heads=2, dtype="f16", fmt="same").paged([(30, 2), (5, 1)], 8)
    q = torch.zeros(a.T, 2, 577, dtype=torch.float16, device=dev)[..., 1:]
    q.copy_(a.q)
    a.check(hs, dev, "general", q=q)


# ------------------------------------------------------------------ the tensor-core kernels
TYPES = [("bf16", "fp8"), ("f16", "fp8"), ("bf16", "same"), ("f16", "same")]


@pytest.mark.parametrize("dtype,fmt", TYPES)
@pytest.mark.parametrize("heads", [1, 5, 16])
@pytest.mark.parametrize("T,top_k", [(1, 1), (3, 31), (2, 33), (5, 300), (40, 64), (500, 20), (2, 2048)])
def test_indexed(hs, dev, dtype, fmt, heads, T, top_k):
    a = LatentInputs(heads=heads, dtype=dtype, fmt=fmt, seed=T)
    a.indexed(T, top_k, 2 * top_k + 5, empty=[T // 2] if T > 2 else [], bad=[T - 1] if T > 1 else [])
    a.check(hs, dev, "tiles")


@pytest.mark.parametrize("dtype,fmt", TYPES)
@pytest.mark.parametrize("heads,page", [(16, 64), (3, 1), (8, 48), (16, 7)])
@pytest.mark.parametrize("lens", [
    [(0, 1)], [(31, 1), (32, 1), (63, 1)], [(700, 1), (None, 0), (3, 2), (0, 0), (40, 3)], [(0, 5), (129, 4)],
    [(i * 7 % 50, 1 + i % 2) for i in range(40)]])
def test_paged(hs, dev, dtype, fmt, heads, page, lens):
    a = LatentInputs(heads=heads, dtype=dtype, fmt=fmt, seed=page)
    a.paged(lens, page, gap=3).check(hs, dev, "tiles")


@pytest.mark.parametrize("dtype,fmt", TYPES)
@pytest.mark.parametrize("heads,T,top_k", [(17, 3, 200), (32, 2, 129), (64, 40, 260), (65, 3, 100), (128, 5, 700),
                                           (128, 160, 140), (100, 2, 1), (20, 2, 5000)])
def test_indexed_heads(hs, dev, dtype, fmt, heads, T, top_k):
    a = LatentInputs(heads=heads, dtype=dtype, fmt=fmt, seed=T)
    a.indexed(T, top_k, 2 * top_k + 5, empty=[T // 2] if T > 2 else [], bad=[T - 1])
    a.check(hs, dev, "tiles")


@pytest.mark.parametrize("dtype,fmt", TYPES)
@pytest.mark.parametrize("heads,page", [(16, 64), (128, 16), (12, 7), (64, 1)])
@pytest.mark.parametrize("lens", [
    [(0, 9)], [(120, 7), (128, 1), (200, 20)], [(700, 3), (None, 0), (3, 2), (0, 0), (0, 140)],
    [(i * 37 % 290, 1 + i % 5) for i in range(30)]])
def test_paged_chunks(hs, dev, dtype, fmt, heads, page, lens):
    a = LatentInputs(heads=heads, dtype=dtype, fmt=fmt, seed=page)
    a.paged(lens, page, gap=3).check(hs, dev, "tiles")


# ------------------------------------------------------------------ values at their limits
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads", [4, 40])
@pytest.mark.parametrize("spread", [(0, 6), (30, 0), (60, 14)])
def test_scales_far_apart(hs, dev, dtype, heads, spread):
    a = LatentInputs(heads=heads, dtype=dtype, fmt="fp8", seed=heads, spread=spread)
    a.indexed(6, 700, 1500).check(hs, dev, "tiles")
    a = LatentInputs(heads=heads, dtype=dtype, fmt="fp8", seed=heads + 1, spread=spread)
    a.paged([(500, 3), (129, 1)], 16).check(hs, dev, "tiles")


@pytest.mark.parametrize("dtype,fmt", TYPES)
@pytest.mark.parametrize("heads", [2, 30, 128])
@pytest.mark.parametrize("rising", [True, False])
def test_sharp_scores(hs, dev, dtype, fmt, heads, rising):
    """Scores in the hundreds, that rise from tile to tile or fall."""
    a = LatentInputs(heads=heads, dtype=dtype, fmt=fmt, seed=7, sharp=40.0).indexed(3, 900, 1900)
    s = torch.einsum("td,nd->tn", a.q[:, 0].double(), a.held.nan_to_num()).numpy()
    for t in range(3):
        order = np.argsort(s[t, np.maximum(a.index[t], 0)])
        a.index[t] = a.index[t, order if rising else order[::-1]]
    a.check(hs, dev, "tiles")


@pytest.mark.parametrize("dtype,fmt", TYPES)
@pytest.mark.parametrize("heads", [3, 64])
def test_queries_that_are_not_finite(hs, dev, dtype, fmt, heads):
    """They make their own head NaN and leave every other bit as it was."""
    a = LatentInputs(heads=heads, dtype=dtype, fmt=fmt, seed=1).indexed(3, 400, 900)
    out, lse, _ = a.check(hs, dev, "tiles")
    q = a.q.clone()
    q[1, 2, 5], q[2, 0, 570] = math.inf, math.nan
    out2, lse2, status = a.call(hs, dev, q=q.to(dev))
    mask = torch.zeros(3, heads, dtype=torch.bool, device=dev)
    mask[1, 2] = mask[2, 0] = True
    assert bool(out2[mask].isnan().all()) and bool(lse2[mask].isnan().all())
    assert torch.equal(out2[~mask], out[~mask]) and torch.equal(lse2[~mask], lse[~mask])
    assert not bool(status.any())


@pytest.mark.parametrize("dtype,fmt", TYPES)
def test_rows_that_are_not_finite(hs, dev, dtype, fmt):
    """They reach the tokens that see them, and no other."""
    a = LatentInputs(heads=9, dtype=dtype, fmt=fmt, seed=2).indexed(4, 300, 4000)
    a.index[1:][np.isin(a.index[1:], a.index[0, :1])] = -1
    out, lse, _ = a.call(hs, dev)
    rows = a.rows.clone()
    if fmt == "fp8":
        rows[a.index[0, 0], 77] = 0x7F
    else:
        rows[a.index[0, 0], 77] = math.nan
    assert a.index[0, 0] >= 0
    out2, lse2, _ = a.call(hs, dev, rows=rows.to(dev))
    assert bool(lse2[0].isnan().all()) and bool(out2[0].isnan().all())
    assert torch.equal(out2[1:], out[1:]) and torch.equal(lse2[1:], lse[1:])


# ------------------------------------------------------------------ layouts and sizes
@pytest.mark.parametrize("dtype,fmt", TYPES)
@pytest.mark.parametrize("heads", [5, 70])
def test_views(hs, dev, dtype, fmt, heads):
    """Queries, outputs and rows inside wider tensors; what is around them stays."""
    for a in (LatentInputs(heads=heads, dtype=dtype, fmt=fmt, seed=3).indexed(4, 200, 500),
              LatentInputs(heads=heads, dtype=dtype, fmt=fmt, seed=3).paged([(100, 2), (300, 1)], 8, gap=1)):
        q = torch.zeros(a.T, heads + 1, 640, dtype=a.dtype, device=dev)[:, 1:, 32:608]
        q.copy_(a.q)
        n, cols = a.rows.shape
        pad = 16 if fmt == "fp8" else 8
        rows = torch.zeros(n, cols + 2 * pad, dtype=a.rows.dtype, device=dev)[:, pad:-pad]
        rows.copy_(a.rows)
        whole = torch.full((a.T, heads, 640), -7.0, dtype=a.dtype, device=dev)
        a.check(hs, dev, "tiles", q=q, rows=rows, out=whole[..., 64:576])
        assert bool((whole[..., :64] == -7).all()) and bool((whole[..., 576:] == -7).all())


@pytest.mark.parametrize("fmt,n", [("fp8", 7_000_000), ("same", 4_000_000)])
def test_rows_past_32_bits(hs, dev, fmt, n):
    """The same rows at the end of a pool of 4.6 GB: the same bits."""
    a = LatentInputs(heads=16, dtype="bf16", fmt=fmt, seed=4).indexed(3, 300, 700)
    near = a.check(hs, dev, "tiles")
    pool = torch.empty(n, a.rows.shape[1], dtype=a.rows.dtype, device=dev)
    shift = n - a.rows.shape[0]
    pool[shift:] = a.rows.to(dev)
    a.index = np.where(a.index >= 0, a.index + shift, a.index).astype(np.int32)
    for x, y in zip(near, a.call(hs, dev, rows=pool)):
        assert torch.equal(x, y)
    a = LatentInputs(heads=16, dtype="bf16", fmt=fmt, seed=5).paged([(250, 2), (40, 1)], 16)
    near = a.check(hs, dev, "tiles")
    at = n // 16 - a.rows.shape[0] // 16
    pool[at * 16: at * 16 + a.rows.shape[0]] = a.rows.to(dev)
    a.table = np.where(a.table >= 0, a.table + at, a.table).astype(np.int32)
    for x, y in zip(near, a.call(hs, dev, rows=pool)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("heads,batch", [(64, 1024), (64, 1100), (16, 2048)])
def test_many_requests(hs, dev, heads, batch):
    a = LatentInputs(heads=heads, dtype="bf16", fmt="fp8", seed=6)
    a.paged([(i % 7, 1) if i % 11 else (None, 0) for i in range(batch)], 4, gap=1).check(hs, dev, "tiles")


def test_bad_blocks(hs, dev):
    """Blocks outside the pool stand for rows of zeros, and are reported."""
    for fmt in ("fp8", "same"):
        a = LatentInputs(heads=8, dtype="f16", fmt=fmt, seed=8)
        a.paged([(40, 2), (150, 1)], 16, bad_block=(1, 3, 1 << 20)).check(hs, dev, "tiles")


@pytest.mark.parametrize("dtype,fmt", TYPES)
def test_nothing_to_see(hs, dev, dtype, fmt):
    a = LatentInputs(heads=20, dtype=dtype, fmt=fmt)
    a.indexed(3, 150, 300, empty=[0, 1, 2]).check(hs, dev, "tiles")
    a.indexed(2, 0, 10).check(hs, dev, "tiles")
    a.indexed(2, 5, 10, empty=[0, 1]).check(hs, dev, "general", rows=a.rows[:0].to(dev))


@pytest.mark.parametrize("dtype,fmt,kind", [(*t, "tiles") for t in TYPES] + [("f32", "same", "general")])
def test_more_new_tokens_than_rows(hs, dev, dtype, fmt, kind):
    """The first tokens of a request that is shorter than what is new of it see nothing."""
    a = LatentInputs(heads=16, dtype=dtype, fmt=fmt, seed=10)
    a.paged([(-3, 5), (10, 2), (-4, 4), (-1, 140)], 16).check(hs, dev, kind)


@pytest.mark.parametrize("dtype,fmt", TYPES)
def test_rows_listed_twice(hs, dev, dtype, fmt):
    a = LatentInputs(heads=7, dtype=dtype, fmt=fmt, seed=11).indexed(3, 290, 600)
    a.index[0] = np.repeat(a.index[0, :29], 10)
    a.index[2, 1:200:2] = a.index[2, 0:199:2]
    a.lists = [[int(e) for e in row if e >= 0] for row in a.index]
    a.check(hs, dev, "tiles")


def test_longest_row(hs, dev):
    """The longest row that the limit's formula allows is served, one past it is refused: rows
    outside the pool, so that every score is 0."""
    T, L = 16 * 1023, 128 * ((2 ** 31 - 1) // 1024 - 4)
    assert 1024 * (L + 512) <= 2 ** 38 - 128 < 1024 * (L + 128 + 512)
    f = dict(device=dev)
    q = torch.zeros(T, 1, 576, dtype=torch.bfloat16, **f)
    out, lse = torch.zeros(T, 1, 512, dtype=torch.bfloat16, **f), torch.zeros(T, 1, **f)
    rows, status = torch.zeros(16, 656, dtype=torch.uint8, **f), torch.zeros(1, dtype=torch.int32, **f)
    for n, want in ((L, 64), (L + 1, 32), (L + 127, 32)):
        out.fill_(-7)
        lse.fill_(-7)
        hs.paged_latent_attention(q, rows, torch.zeros(1, 1, dtype=torch.int32, **f), torch.zeros(1, dtype=torch.int64, **f),
                                  torch.tensor([0, 1], dtype=torch.int32, **f), torch.tensor([n], **f), out, max_q_len=1,
                                  page_size=1 << 28, scale=1.0, lse=lse, status=status)
        assert int(status) == want
        assert bool((out[1:] == -7).all()) and bool((lse[1:] == -7).all())
        if want == 64:
            assert bool((out[0] == 0).all()) and abs(float(lse[0, 0]) - math.log(n)) < 1e-3
        else:
            assert bool((out[0] == -7).all()) and bool((lse[0] == -7).all())


# ------------------------------------------------------------------ streams, graphs, workspaces
@pytest.mark.parametrize("fmt", ["fp8", "same"])
@pytest.mark.parametrize("heads", [16, 64])
def test_streams_and_workspaces(hs, dev, fmt, heads):
    """Two calls at once on streams of their own, each with its workspace: the bits of calls one
    after the other, every time."""
    two = [LatentInputs(heads=heads, dtype="bf16", fmt=fmt, seed=9 + i).indexed(30, 700 + i, 2000) for i in range(2)]
    alone = [a.check(hs, dev, "tiles") for a in two]
    t = [(a.q.to(dev), a.rows.to(dev), torch.from_numpy(a.index).to(dev)) for a in two]
    outs = [torch.zeros_like(x[0]) for x in alone]
    n = [hs.latent_attention_workspace_bytes(*x, o) for x, o in zip(t, outs)]
    space = [torch.empty(m, dtype=torch.uint8, device=dev) for m in n]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for own in (True, False):
        for _ in range(5):
            for o in outs:
                o.fill_(-3)
            torch.cuda.synchronize()
            for i in range(2):
                hs.latent_attention(*t[i], outs[i], scale=two[i].scale, workspace=space[i] if own else None,
                                    stream=streams[i])
            torch.cuda.synchronize()
            for o, want in zip(outs, alone):
                assert torch.equal(o, want[0])
    with pytest.raises(hs.HisparseError, match="workspace"):
        hs.latent_attention(*t[0], outs[0], scale=1.0, workspace=space[0][: n[0] - 256])
    with pytest.raises(hs.HisparseError, match="workspace"):
        wide = torch.empty(n[0] + 16, dtype=torch.uint8, device=dev)
        hs.latent_attention(*t[0], outs[0], scale=1.0, workspace=wide[16:])


@pytest.mark.parametrize("fmt", ["fp8", "same"])
@pytest.mark.parametrize("keep", [True, False])
def test_captured(hs, dev, fmt, keep):
    """A captured call follows its inputs: lengths, tables and queries that change in place."""
    lens = [[(300, 2), (0, 1), (77, 2)], [(10, 1), (500, 2), (None, 0)], [(0, 0), (128, 2), (127, 1)]]
    runs = [LatentInputs(heads=16, dtype="bf16", fmt=fmt, seed=20 + i).paged(x, 16) for i, x in enumerate(lens)]
    rows_n, cols = max(a.rows.shape[0] for a in runs), max(a.table.shape[1] for a in runs)
    T = 5
    f = dict(device=dev)
    q = torch.zeros(T, 16, 576, dtype=torch.bfloat16, **f)
    rows = torch.zeros(rows_n, runs[0].rows.shape[1], dtype=runs[0].rows.dtype, **f)
    table = torch.full((runs[0].table.shape[0], cols), -1, dtype=torch.int32, **f)
    req, cu, seq = (torch.zeros(3, dtype=torch.int64, **f), torch.zeros(4, dtype=torch.int32, **f),
                    torch.zeros(3, dtype=torch.int64, **f))
    out, lse = torch.zeros(T, 16, 512, dtype=torch.bfloat16, **f), torch.zeros(T, 16, **f)
    status = torch.zeros(3, dtype=torch.int32, **f)

    def load(a):
        q[: a.T] = a.q.to(dev)
        rows[: a.rows.shape[0]] = a.rows.to(dev)
        table.fill_(-1)
        table[:, : a.table.shape[1]] = torch.from_numpy(a.table).to(dev)
        req.copy_(torch.from_numpy(a.req))
        cu.copy_(torch.from_numpy(a.cu))
        seq.copy_(torch.from_numpy(a.seq))
        out.fill_(-7)
        lse.fill_(-7)

    args = (q, rows, table, req, cu, seq, out)
    kw = dict(max_q_len=2, page_size=16, scale=runs[0].scale, lse=lse, status=status)
    space = None
    if keep:
        n = hs.paged_latent_attention_workspace_bytes(*args, max_q_len=2, page_size=16)
        space = torch.empty(n, dtype=torch.uint8, device=dev)
    load(runs[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        hs.paged_latent_attention(*args, workspace=space, **kw)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hs.paged_latent_attention(*args, workspace=space, **kw)
    for a in (runs[1], runs[2], runs[0]):
        load(a)
        graph.replay()
        torch.cuda.synchronize()
        assert bool((out[a.T:] == -7).all()) and bool((lse[a.T:] == -7).all())
        a.compare(out[: a.T], lse[: a.T], status, "tiles")


@pytest.mark.parametrize("fmt", ["fp8", "same"])
def test_graphs_that_share_a_workspace(hs, dev, fmt):
    """Replayed in turn in one stream: what one left in the workspace is nothing to the other."""
    two = [LatentInputs(heads=h, dtype="bf16", fmt=fmt, seed=40 + h).indexed(t, k, 2 * k) for h, t, k in
           ((64, 9, 900), (16, 3, 2000))]
    alone = [a.check(hs, dev, "tiles")[0] for a in two]
    t = [(a.q.to(dev), a.rows.to(dev), torch.from_numpy(a.index).to(dev)) for a in two]
    outs = [torch.zeros_like(x) for x in alone]
    n = max(hs.latent_attention_workspace_bytes(*x, o) for x, o in zip(t, outs))
    space = torch.full((n,), 0xFF, dtype=torch.uint8, device=dev)
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            hs.latent_attention(*t[i], outs[i], scale=two[i].scale, workspace=space)
        graphs.append(g)
    for i in (0, 1, 1, 0, 1, 0):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], alone[i])


@pytest.mark.parametrize("fmt", ["fp8", "same"])
@pytest.mark.parametrize("heads", [16, 32, 64])
def test_time_out(hs, dev, fmt, heads):
    a = LatentInputs(heads=heads, dtype="bf16", fmt=fmt, seed=30).indexed(20, 600, 1300, bad=[3])
    t = (a.q.to(dev), a.rows.to(dev), torch.from_numpy(a.index).to(dev))
    out = torch.zeros(20, heads, 512, dtype=torch.bfloat16, device=dev)
    status = torch.zeros(20, dtype=torch.int32, device=dev)
    for _ in range(2):
        hs.latent_attention_timeout_selftest(*t, out, scale=a.scale, status=status)
        assert status.tolist() == [16 | x for x in a.status]
        a.check(hs, dev, "tiles")


def test_time_out_needs_waits(hs, dev):
    a = LatentInputs(heads=2, dtype="f32", fmt="same").indexed(2, 10, 30)
    with pytest.raises(hs.HisparseError, match="no bounded waits"):
        hs.latent_attention_timeout_selftest(a.q.to(dev), a.rows.to(dev), torch.from_numpy(a.index).to(dev),
                                             torch.zeros(2, 2, 512, device=dev), scale=1.0)
