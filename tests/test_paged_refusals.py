"""What the paged-cache operators refuse, before anything reaches a GPU."""
from __future__ import annotations

import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def hs():
    import sparse_attention_kv_row_gb300 as hs
    from sparse_attention_kv_row_gb300 import build

    build.build()
    return hs


@pytest.fixture(scope="module")
def lib(hs):
    from sparse_attention_kv_row_gb300 import _capi

    return _capi.load()


def _slots(lib, **kw):
    a = dict(ctx=256, new=256, req=256, batch=2, flags=0, table=256, stride=4, states=2, blocks=4, bs=16,
             free=256, num_free=8, top=256, top_out=256, cu=256, seq=256, loc=256, pos=None, row=None,
             max_tokens=4, status=None)
    a.update(kw)
    return lib.hs_assign_slots(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), 1), (dict(bs=0), 1), (dict(stride=3), 1), (dict(flags=4), 1), (dict(num_free=-1), 1),
    (dict(max_tokens=-1), 1), (dict(states=-1), 1), (dict(batch=4097), 2), (dict(max_tokens=1 << 31), 2),
    (dict(num_free=1 << 31), 2), (dict(ctx=None), 1), (dict(cu=None), 1), (dict(free=None), 1),
    (dict(loc=None), 1), (dict(top_out=None), 1), (dict(batch=0, top_out=None), 1),
    (dict(batch=0, ctx=None, cu=None), 1), (dict(table=None), 1)])
def test_assign_slots_rejects(lib, kw, code):
    assert _slots(lib, **kw) == code
    if code:
        assert b"hs_assign_slots" in lib.hs_last_error()


def _norm(lib, **kw):
    from sparse_attention_kv_row_gb300._capi import QkNormRopeArgs

    a = dict(n_tokens=4, num_heads=4, num_kv_heads=2, head_dim=64, rot_dim=64, in_dtype=2, cache_dtype=2,
             flags=0, page_size=16, eps=1e-6, q=256, q_stride_token=512, q_stride_head=64, k=256,
             k_stride_token=512, k_stride_head=64, v=256, v_stride_token=512, v_stride_head=64,
             cos_sin=256, max_pos=10, positions=256, q_out=512, out_stride_token=256,
             out_stride_head=64, k_cache=256, v_cache=256, cache_stride_page=4096,
             cache_stride_offset=256, cache_stride_head=128, num_slots=64, cache_loc=256)
    a.update(kw)
    return lib.hs_qk_norm_rope_store(C.byref(QkNormRopeArgs(**a)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(in_dtype=3), 1), (dict(cache_dtype=1), 1), (dict(flags=2), 1), (dict(rot_dim=63), 1),
    (dict(rot_dim=66), 1), (dict(rot_dim=-2), 1), (dict(head_dim=0), 1), (dict(page_size=0), 1),
    (dict(n_tokens=-1), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(num_kv_heads=0), 1),
    (dict(head_dim=1025, q_stride_head=2000), 2), (dict(num_slots=1 << 32), 2),
    (dict(num_heads=1 << 26), 2), (dict(k_scale=256), 1), (dict(q=None), 1), (dict(v_cache=None), 1),
    (dict(cos_sin=None), 1), (dict(positions=None), 1), (dict(q_stride_head=63), 1),
    (dict(cache_stride_head=127), 1), (dict(q=257), 1), (dict(k_cache=257), 1),
    (dict(cache_stride_offset=257), 1), (dict(cos_sin=258), 1), (dict(n_tokens=0, q=None), 0)])
def test_qk_norm_rope_store_rejects(lib, kw, code):
    assert _norm(lib, **kw) == code
    if code:
        assert b"hs_qk_norm_rope_store" in lib.hs_last_error()
    assert lib.hs_qk_norm_rope_store(None, None) == 1


def _attn_args(**kw):
    from sparse_attention_kv_row_gb300._capi import PagedAttentionArgs

    a = dict(batch=2, num_heads=4, num_kv_heads=2, head_dim=48, in_dtype=2, cache_dtype=2, flags=0,
             page_size=16, max_q_len=2, window=0, scale=0.1, table_blocks=4, n_tokens=4, q=256,
             q_stride_token=192, q_stride_head=48, out=256, out_stride_token=192, out_stride_head=48,
             k_cache=256, v_cache=256, cache_stride_page=4096, cache_stride_offset=192,
             cache_stride_head=96, num_pages=8, block_table=256, block_table_stride=4, num_states=2,
             req_state=256, cu_q=256, seq_lens=256)
    a.update(kw)
    return C.byref(PagedAttentionArgs(**a))


@pytest.mark.parametrize("kw,code", [
    (dict(in_dtype=3), 1), (dict(cache_dtype=0), 1), (dict(flags=4), 1), (dict(batch=-1), 1),
    (dict(num_heads=3), 1), (dict(num_kv_heads=0), 1), (dict(head_dim=0), 1), (dict(page_size=0), 1),
    (dict(max_q_len=-1), 1), (dict(window=-1), 1), (dict(block_table_stride=3), 1),
    (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1), (dict(k_scale=256), 1),
    (dict(head_dim=513, q_stride_head=600), 2), (dict(batch=4097), 2), (dict(max_q_len=1 << 30), 2),
    (dict(n_tokens=1 << 31), 2), (dict(q=None), 1), (dict(out=None), 1), (dict(block_table=None), 1),
    (dict(cu_q=None), 1), (dict(k_cache=None), 1), (dict(q_stride_head=47), 1),
    (dict(cache_stride_head=95), 1), (dict(q=257), 1), (dict(k_cache=257), 1),
    (dict(cache_stride_page=4097), 1), (dict(batch=0, q=None), 0)])
def test_paged_attention_rejects(lib, kw, code):
    assert lib.hs_paged_attention(_attn_args(**kw), None) == code
    if code:
        assert b"hs_paged_attention" in lib.hs_last_error()
    assert lib.hs_paged_attention(None, None) == 1
    assert lib.hs_paged_attention_workspace_bytes(None) == -1
    assert lib.hs_paged_attention_workspace_bytes(_attn_args(num_heads=3)) == -1


def test_status_name(lib):
    assert lib.hs_status_string(128) == b"HS_ST_NO_BLOCK"


def _i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def _i64(*s):
    return torch.zeros(*s, dtype=torch.int64)


def _slot_call(hs, **kw):
    a = dict(ctx_lens=_i64(2), new_lens=_i32(2), req_state=_i64(2), block_table=_i32(3, 4), free_blocks=_i32(5),
             free_top=_i32(1), block_size=16, cu_new=_i32(3), seq_lens=_i64(2), cache_loc=_i64(7))
    a.update(kw)
    hs.assign_slots(**a)


@pytest.mark.parametrize("kw,err", [
    (dict(new_lens=_i64(2)), TypeError), (dict(ctx_lens=_i64(3)), ValueError),
    (dict(seq_lens=_i32(2)), TypeError), (dict(cu_new=_i32(2)), ValueError), (dict(cache_loc=_i32(7)), TypeError),
    (dict(positions=_i64(6)), ValueError), (dict(token_row=_i64(7)), TypeError), (dict(status=_i32(1)), ValueError),
    (dict(free_top=_i32(2)), ValueError), (dict(block_table=_i32(4, 3).t()), ValueError),
    (dict(req_state=torch.zeros(2)), TypeError), (dict(), ValueError)])  # the last: not on a GPU
def test_assign_slots_binding(hs, kw, err):
    with pytest.raises(err):
        _slot_call(hs, **kw)


def _h(*s, dtype=torch.bfloat16):
    return torch.zeros(*s, dtype=dtype)


def _norm_call(hs, **kw):
    a = dict(q=_h(5, 4, 64), k=_h(5, 2, 64), v=_h(5, 2, 64), q_weight=_h(64), k_weight=_h(64),
             cos_sin=torch.zeros(10, 64), positions=_i64(5), q_out=_h(5, 4, 64), k_cache=_h(3, 16, 2, 64),
             v_cache=_h(3, 16, 2, 64), cache_loc=_i64(5))
    a.update(kw)
    hs.qk_norm_rope_store(**a)


@pytest.mark.parametrize("kw,err", [
    (dict(q=_h(5, 4, 64, dtype=torch.float64)), TypeError), (dict(q=_h(5, 256)), ValueError),
    (dict(k=_h(5, 2, 64, dtype=torch.float16)), TypeError), (dict(v=_h(4, 2, 64)), ValueError),
    (dict(q_weight=_h(32)), ValueError), (dict(k_weight=torch.zeros(64)), TypeError),
    (dict(cos_sin=_h(10, 64)), TypeError), (dict(positions=_i32(5)), TypeError), (dict(positions=_i64(4)), ValueError), (dict(positions=None), ValueError),
    (dict(cache_loc=_i64(6)), ValueError), (dict(page_size=8), ValueError),
    (dict(v_cache=_h(3, 16, 2, 64, dtype=torch.float16)), TypeError), (dict(k_scale=torch.ones(1)), ValueError),
    (dict(k_cache=_h(2, 16, 2, 64)), ValueError), (dict(status=_i64(1)), TypeError), (dict(), ValueError)])
def test_qk_norm_binding(hs, kw, err):
    with pytest.raises(err):
        _norm_call(hs, **kw)


def test_qk_norm_partly_in_place(hs):
    x = _h(5, 9, 64)
    with pytest.raises(ValueError, match="q_out"):
        _norm_call(hs, q=x[:, :8:2], q_out=x[:, :4])


def _attn_call(hs, **kw):
    a = dict(q=_h(5, 4, 64), k_cache=_h(3, 16, 2, 64), v_cache=_h(3, 16, 2, 64), block_table=_i32(2, 3),
             req_state=_i64(2), cu_q=_i32(3), seq_lens=_i64(2), out=_h(5, 4, 64), max_q_len=3)
    a.update(kw)
    hs.paged_attention(**a)


@pytest.mark.parametrize("kw,err", [
    (dict(q=_i32(5, 4, 64)), TypeError), (dict(out=_h(5, 4, 32)), ValueError), (dict(cu_q=_i64(3)), TypeError),
    (dict(seq_lens=_i64(3)), ValueError), (dict(lse=torch.zeros(4, 5)), ValueError),
    (dict(lse=_h(5, 4)), TypeError), (dict(status=_i32(3)), ValueError), (dict(block_table=_i64(2, 3)), TypeError),
    (dict(v_scale=torch.ones(1)), ValueError), (dict(page_size=32), ValueError),
    (dict(k_cache=_h(3, 16, 2, 64, dtype=torch.float16)), TypeError), (dict(), ValueError)])
def test_paged_attention_binding(hs, kw, err):
    with pytest.raises(err):
        _attn_call(hs, **kw)
