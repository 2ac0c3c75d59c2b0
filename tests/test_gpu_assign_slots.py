"""assign_slots against a plain row-by-row statement, entry by entry."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from paged_cases import slots_plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    import __graft_entry__

    __graft_entry__.build()
    return torch.device("cuda:0")


def _hs():
    import sparse_attention_kv_row_gb300 as hs

    return hs


def _case(B, bs, ctx_hi, new_hi, seed, pad=0, spare=3, extra=2):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, ctx_hi + 1, B)
    new = rng.integers(0, new_hi + 1, B)
    states = B + 4
    req = rng.permutation(states)[:B]
    req[rng.permutation(B)[:pad]] = -1
    cols = -(-(ctx_hi + new_hi) // bs) + 1
    held = -(-ctx // bs)
    need = np.where(req >= 0, -(-(ctx + new) // bs) - held, 0)
    blocks = rng.permutation(int(held.sum() + need.sum()) + spare).astype(np.int32)
    table = np.full((states, cols), -1, np.int32)
    at = 0
    for r, h in zip(req, held):
        if r >= 0:
            table[r, :h] = blocks[at: at + h]
            at += h
    free = blocks[at:]
    tokens = int(np.where(req >= 0, new, 0).sum()) + extra
    return dict(ctx=ctx, new=new.astype(np.int32), req=req, table=table, free=free,
                top=int(need.sum()) + min(spare, 2), bs=bs, max_tokens=tokens)


def _run(dev, c, i64=True, in_place=False, optional=True, stride=0):
    hs = _hs()
    ref = slots_plain(c["ctx"], c["new"], c["req"], c["table"], c["free"], c["top"], c["bs"],
                      c["max_tokens"])
    it = torch.int64 if i64 else torch.int32
    t = lambda a, d: torch.from_numpy(np.ascontiguousarray(a)).to(d).to(dev)  # noqa: E731
    B, n = len(c["ctx"]), c["max_tokens"]
    ctx = t(c["ctx"], it)
    wide = torch.full((c["table"].shape[0], c["table"].shape[1] + stride), -9, dtype=torch.int32,
                      device=dev)
    table = wide[:, : c["table"].shape[1]]
    table.copy_(t(c["table"], torch.int32))
    top = torch.tensor([c["top"]], dtype=torch.int32, device=dev)
    out = dict(cu_new=torch.full((B + 1,), -9, dtype=torch.int32, device=dev),
               seq_lens=ctx if in_place else torch.full((B,), -9, dtype=it, device=dev),
               cache_loc=torch.full((n,), -9, dtype=torch.int64, device=dev),
               positions=torch.full((n,), -9, dtype=torch.int64, device=dev),
               token_row=torch.full((n,), -9, dtype=torch.int32, device=dev),
               status=torch.full((B,), -9, dtype=torch.int32, device=dev))
    top_out = top if in_place else torch.full((1,), -9, dtype=torch.int32, device=dev)
    if not optional:
        out["positions"] = out["token_row"] = out["status"] = None
    hs.assign_slots(ctx, t(c["new"], torch.int32), t(c["req"], it), table,
                    t(c["free"], torch.int32), top, block_size=c["bs"],
                    free_top_out=None if in_place else top_out, **out)
    torch.cuda.synchronize()
    for name, x in out.items():
        if x is not None:
            np.testing.assert_array_equal(x.cpu().numpy(), ref[name], err_msg=name)
    np.testing.assert_array_equal(table.cpu().numpy(), ref["table"])
    assert bool((wide[:, c["table"].shape[1]:] == -9).all())
    assert int(top_out) == ref["free_top"]
    if not in_place:
        np.testing.assert_array_equal(ctx.cpu().numpy(), c["ctx"])
    return ref


@pytest.mark.parametrize("B,bs,ctx_hi,new_hi,pad", [
    (1, 16, 0, 1, 0), (1, 1, 5, 3, 0), (2, 64, 1000, 1, 1), (33, 16, 300, 1, 5),
    (32, 64, 131072, 1, 0), (100, 7, 50, 40, 10), (1000, 16, 400, 60, 100),
    (1024, 128, 100, 2, 0), (1025, 8, 9, 5, 1025), (4096, 16, 40, 3, 7), (4, 16, 10, 30000, 0)])
@pytest.mark.parametrize("i64", [True, False])
def test_sizes(dev, B, bs, ctx_hi, new_hi, pad, i64):
    _run(dev, _case(B, bs, ctx_hi, new_hi, seed=B + bs, pad=pad), i64=i64)


def test_in_place_optional_and_strided(dev):
    for B, new_hi in ((40, 5), (500, 100)):
        c = _case(B, 16, 200, new_hi, seed=B)
        _run(dev, c, in_place=True)
        _run(dev, c, optional=False)
        _run(dev, c, stride=5)


@pytest.mark.parametrize("B,new_hi", [(20, 30), (600, 60)])
def test_free_blocks_run_out(dev, B, new_hi):
    """Rows are served in order until one does not fit; rows that open none still are."""
    c = _case(B, 16, 100, new_hi, seed=1)
    for top in (0, 1, c["top"] // 2, c["top"] // 2 + 1, -5, len(c["free"]) + 100):
        c["top"] = top
        ref = _run(dev, c)
        if 0 < top < len(c["free"]) // 2:
            assert 128 in ref["status"] and 0 in ref["status"]


@pytest.mark.parametrize("B,new_hi", [(20, 30), (600, 60)])
def test_bad_rows(dev, B, new_hi):
    c = _case(B, 16, 100, new_hi, seed=2)
    free_rows = set(range(c["table"].shape[0])) - set(c["req"].tolist())
    assert free_rows
    c["req"][3] = c["table"].shape[0]          # past the table
    c["ctx"][4] = -1
    c["ctx"][5] = c["table"].shape[1] * 16     # beyond the row's blocks, with any new token
    c["new"][5] = 1
    c["new"][6] = -2
    c["new"][7] = c["max_tokens"] + 1
    c["ctx"][8] = 17
    c["new"][8] = 2
    c["table"][c["req"][8], 1] = -1            # its half-filled block is missing
    ref = _run(dev, c)
    assert [int(ref["status"][i]) for i in (3, 4, 5, 6, 7, 8)] == [32, 32, 32, 32, 32, 64]
    c["max_tokens"] //= 2                      # the later rows' tokens have no room
    ref = _run(dev, c)
    assert ref["status"][-1] == 64
    c["max_tokens"] = 0
    _run(dev, c)


def test_lengths_past_32_bits_are_refused_per_row(dev):
    c = _case(5, 16, 10, 3, seed=2)
    c["ctx"] = c["ctx"].astype(np.int64)
    c["ctx"][1] = 2 ** 31 + 5
    c["new"][1] = 0  # (positions of a refused row say nothing)
    ref = _run(dev, c)
    assert ref["status"][1] == 32


def test_negative_free_block(dev):
    c = _case(10, 16, 100, 30, seed=4)
    c["free"][c["top"] - 2] = -1
    ref = _run(dev, c)
    assert 64 in ref["status"]


def test_captured_decode_loop(dev):
    """Lengths and stack carried in place from replay to replay until the blocks run out."""
    hs = _hs()
    B, bs, cols, n_free = 6, 4, 5, 17
    free = np.random.default_rng(0).permutation(n_free).astype(np.int32)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    table, ctx = np.full((B, cols), -1, np.int32), np.zeros(B, np.int64)
    new, req = np.ones(B, np.int32), np.arange(B)[::-1].copy()
    g = dict(ctx=t(ctx), new=t(new), req=t(req), table=t(table), free=t(free),
             top=t(np.array([n_free], np.int32)), cu=t(np.zeros(B + 1, np.int32)),
             loc=t(np.zeros(B, np.int64)), st=t(np.zeros(B, np.int32)))

    def step():
        hs.assign_slots(g["ctx"], g["new"], g["req"], g["table"], g["free"], g["top"], block_size=bs,
                        cu_new=g["cu"], seq_lens=g["ctx"], cache_loc=g["loc"], status=g["st"])

    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            step()
    top = n_free
    for i in range(16):
        graph.replay()
        ref = slots_plain(ctx, new, req, table, free, top, bs, B)
        ctx, table, top = ref["seq_lens"], ref["table"], ref["free_top"]
        torch.cuda.synchronize()
        np.testing.assert_array_equal(g["loc"].cpu().numpy(), ref["cache_loc"])
        np.testing.assert_array_equal(g["ctx"].cpu().numpy(), ctx)
        np.testing.assert_array_equal(g["table"].cpu().numpy(), table)
        np.testing.assert_array_equal(g["st"].cpu().numpy(), ref["status"])
        assert int(g["top"]) == top
    assert 128 in ref["status"]


def test_empty_batch(dev):
    """No rows: the token count is 0, the stack keeps its height, every entry is -1."""
    c = _case(1, 16, 10, 3, seed=5)
    for n in (0, 1, 700):
        for i64 in (True, False):
            e = dict(c, ctx=c["ctx"][:0], new=c["new"][:0], req=c["req"][:0], top=2, max_tokens=n)
            _run(dev, e, i64=i64)
            _run(dev, e, i64=i64, in_place=True, optional=False)


def test_empty_tables(dev):
    """No states, no columns, no free blocks: every row with tokens is refused."""
    for shape, code in (((0, 4), 32), ((9, 0), 32), ((9, 4), 128)):
        c = _case(3, 16, 0, 3, seed=6)
        c.update(table=np.full(shape, -1, np.int32), free=c["free"][:0], top=0)
        c["new"][:] = 2
        c["req"] = np.arange(3)
        ref = _run(dev, c)
        assert (ref["status"] & code == code).all()


def test_positions_of_refused_rows_past_32_bits(dev):
    """A refused row's tokens keep their positions, also where these pass 32 bits."""
    for ctx in (2 ** 31 + 5, 2 ** 32 + 3, 2 ** 40 + 7, -1, -2 ** 33 - 9):
        c = _case(5, 16, 10, 3, seed=2, extra=20)
        c["ctx"] = c["ctx"].astype(np.int64)
        c["ctx"][1], c["new"][1] = ctx, 4
        ref = _run(dev, c)
        assert ref["status"][1] == 32
        at = int(ref["cu_new"][1])
        assert ref["positions"][at: at + 4].tolist() == [ctx + i for i in range(4)]


def test_first_call_of_a_process_captured(dev):
    """The device's limits are asked for during the first call, which may be a captured one, of a
    size that takes the largest cluster."""
    import os
    import subprocess
    import sys

    code = """
import torch, sparse_attention_kv_row_gb300 as hs
dev = torch.device("cuda:0")
z = lambda n, d=torch.int32: torch.zeros(n, dtype=d, device=dev)
n, bs = 20000, 16
new, table = z(2), torch.full((2, 1300), -1, dtype=torch.int32, device=dev)
new[:] = 9000
free, top = torch.arange(1300, dtype=torch.int32, device=dev), z(1)
top[:] = 1300
cu, seq, loc, ctx, req = z(3), z(2), z(n, torch.int64), z(2), torch.arange(2, device=dev)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    hs.assign_slots(ctx, new, req, table, free, top, block_size=bs, cu_new=cu, seq_lens=seq, cache_loc=loc)
graph.replay()
torch.cuda.synchronize()
assert cu.tolist() == [0, 9000, 18000] and int(top) == 1300 - 2 * 563
assert sorted(loc[:18000].tolist())[0] >= 0 and bool((loc[18000:] == -1).all())
assert len(set(loc[:18000].tolist())) == 18000
print("good")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "good" in r.stdout, r.stderr[-2000:]
