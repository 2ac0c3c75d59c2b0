"""Arguments that the latent-attention operators refuse, before any device call."""
from __future__ import annotations

import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_kv_row_gb300 import _capi, build

    build.build()
    return _capi.load()


def _norm(**kw):
    from sparse_attention_kv_row_gb300._capi import AddRmsNormArgs

    base = dict(n_tokens=2, dim=64, dtype=2, eps=1e-6, x=4096, x_stride=64, out=8192, out_stride=64)
    base.update(kw)
    return AddRmsNormArgs(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), 1), (dict(flags=2), 1), (dict(dim=0), 1), (dict(n_tokens=-1), 1), (dict(group=-1), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(dim=65537, x_stride=65537, out_stride=65537), 2),
    (dict(x=None), 1), (dict(out=None), 1), (dict(codes=4096), 1), (dict(scales=4096), 1),
    (dict(residual_out=4096), 1), (dict(out_stride=63), 1), (dict(x_stride=-1), 1),
    (dict(x=4097), 1), (dict(codes=4096, codes_stride=64, scales=4098), 1),
    (dict(residual=16384, residual_stride=64, residual_out=8192, residual_out_stride=64), 1),  # out too
    (dict(out=4096, out_stride=128), 1),                                                       # x, other stride
    (dict(residual=8192, residual_stride=128), 1),                                             # out, other stride
])
def test_add_rms_norm(lib, kw, code):
    assert lib.hs_add_rms_norm(C.byref(_norm(**kw)), None) == code
    assert lib.hs_last_error() != b""


def test_nothing_to_do(lib):
    from sparse_attention_kv_row_gb300._capi import LatentAttentionArgs, LatentRowsArgs

    assert lib.hs_add_rms_norm(C.byref(_norm(n_tokens=0, x=None, out=None)), None) == 0
    assert lib.hs_latent_norm_rope_store(C.byref(LatentRowsArgs(latent_dim=512, rope_dim=64, in_dtype=2, row_stride=656, row_format=1)), None) == 0
    a = dict(num_heads=16, latent_dim=512, rope_dim=64, in_dtype=2, row_format=1, scale=1.0, page_size=1, row_stride=656,
             q_stride_head=576, out_stride_head=512)
    assert lib.hs_latent_attention(C.byref(LatentAttentionArgs(**a)), None) == 0
    assert lib.hs_latent_attention(C.byref(LatentAttentionArgs(flags=4, **a)), None) == 0
    for fn in (lib.hs_add_rms_norm, lib.hs_latent_norm_rope_store, lib.hs_latent_attention):
        assert fn(None, None) == 1
    assert lib.hs_latent_attention_workspace_bytes(None) == -1


def _rows(**kw):
    from sparse_attention_kv_row_gb300._capi import LatentRowsArgs

    base = dict(n_tokens=2, latent_dim=512, rope_dim=64, num_heads=2, in_dtype=2, row_format=1, eps=1e-6, latent=4096,
                latent_stride=576, k_pe=4096, k_pe_stride=576, q_pe=4096, q_stride_token=128, q_stride_head=64,
                q_out=8192, out_stride_token=128, out_stride_head=64, rows=16384, row_stride=656, num_rows=10, loc=4096)
    base.update(kw)
    return LatentRowsArgs(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(in_dtype=3), 1), (dict(row_format=2), 1), (dict(flags=4), 1), (dict(latent_dim=0), 1), (dict(rope_dim=63), 1),
    (dict(num_heads=-1), 1), (dict(num_rows=-1), 1), (dict(eps=-1.0), 1), (dict(in_dtype=0), 2), (dict(latent_dim=500), 2),
    (dict(latent_dim=1152, row_stride=2048), 2), (dict(rope_dim=258, row_stride=2048), 2), (dict(cos_sin=4096), 1),
    (dict(positions=4096), 1), (dict(latent=None), 1), (dict(loc=None), 1), (dict(k_pe=None), 1), (dict(q_out=None), 1),
    (dict(rows=None), 1), (dict(row_stride=655), 1), (dict(row_stride=658), 1), (dict(q_stride_head=63), 1),
    (dict(q_out=4096, out_stride_head=128), 1), (dict(latent=4097), 1), (dict(rows=16386), 1),
    (dict(num_heads=1 << 26), 2),
])
def test_latent_rows(lib, kw, code):
    assert lib.hs_latent_norm_rope_store(C.byref(_rows(**kw)), None) == code
    assert lib.hs_last_error() != b""


def _attn(**kw):
    from sparse_attention_kv_row_gb300._capi import LatentAttentionArgs

    base = dict(batch=2, num_heads=16, latent_dim=512, rope_dim=64, in_dtype=2, row_format=1, page_size=16, max_q_len=1,
                scale=0.1, table_blocks=4, n_tokens=2, q=4096, q_stride_token=9216, q_stride_head=576, out=8192,
                out_stride_token=8192, out_stride_head=512, rows=16384, row_stride=656, num_rows=64, block_table=4096,
                block_table_stride=4, num_states=2, req_state=4096, cu_q=4096, seq_lens=4096)
    base.update(kw)
    return LatentAttentionArgs(**base)


INDEX = dict(flags=4, batch=0, row_index=4096, row_index_stride=8, top_k=8)


@pytest.mark.parametrize("kw,code", [
    (dict(in_dtype=3), 1), (dict(row_format=2), 1), (dict(flags=8), 1), (dict(num_heads=0), 1), (dict(latent_dim=0), 1),
    (dict(rope_dim=-1), 1), (dict(n_tokens=-1), 1), (dict(num_rows=-1), 1), (dict(batch=-1), 1), (dict(scale=0.0), 1),
    (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(page_size=0), 1),
    (dict(block_table_stride=3), 1), (dict(in_dtype=0), 2), (dict(latent_dim=500), 2), (dict(latent_dim=640, row_stride=2048, q_stride_head=704, out_stride_head=640), 2),
    (dict(rope_dim=257, row_stride=2048, q_stride_head=1024), 2), (dict(batch=2049), 2), (dict(num_rows=1 << 31), 2),
    (dict(n_tokens=1 << 31), 2), (dict(max_q_len=1 << 28), 2), (dict(q_stride_head=575), 1), (dict(out_stride_head=511), 1),
    (dict(row_stride=655), 1), (dict(row_stride=658), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(rows=None), 1),
    (dict(cu_q=None), 1), (dict(block_table=None), 1), (dict(q=4097), 1),
    (INDEX | dict(batch=1), 1), (INDEX | dict(row_index=None), 1), (INDEX | dict(row_index_stride=7), 1),
    (INDEX | dict(top_k=-1), 1), (INDEX | dict(top_k=(1 << 30) + 1, row_index_stride=1 << 31), 2),
])
def test_latent_attention(lib, kw, code):
    assert lib.hs_latent_attention(C.byref(_attn(**kw)), None) == code
    assert lib.hs_last_error() != b""


def test_python_checks():
    """The binding's own checks come before anything touches a device."""
    import sparse_attention_kv_row_gb300 as hs

    bf = torch.bfloat16
    x = torch.zeros(4, 64, dtype=bf)
    w = torch.zeros(64, dtype=bf)
    for bad, err in (
            (lambda: hs.add_rms_norm(x.double(), w, x), TypeError),
            (lambda: hs.add_rms_norm(x[0], w, x[0]), ValueError),
            (lambda: hs.add_rms_norm(x, w), ValueError),
            (lambda: hs.add_rms_norm(x, w[:5], x), ValueError),
            (lambda: hs.add_rms_norm(x, w, x[:3]), ValueError),
            (lambda: hs.add_rms_norm(x, w, x.float()), TypeError),
            (lambda: hs.add_rms_norm(x, w, x, residual_out=x), ValueError),
            (lambda: hs.add_rms_norm(x.t(), w, x.t()), ValueError),
            (lambda: hs.add_rms_norm(x, w, x, group=-1), ValueError),
            (lambda: hs.add_rms_norm(x, w, codes=torch.zeros(4, 64, dtype=torch.uint8)), ValueError),
            (lambda: hs.add_rms_norm(x, w, codes=torch.zeros(4, 64, dtype=torch.uint8), scales=torch.zeros(4, 2)), ValueError),
            (lambda: hs.add_rms_norm(x, w, codes=torch.zeros(4, 64, dtype=torch.int32), scales=torch.zeros(4, 1)), TypeError),
            (lambda: hs.add_rms_norm(x, w, x), ValueError)):  # not on a CUDA device
        with pytest.raises(err):
            bad()
    c, pe, rows, loc = torch.zeros(4, 512, dtype=bf), torch.zeros(4, 64, dtype=bf), torch.zeros(9, 656, dtype=torch.uint8), torch.zeros(4, dtype=torch.int64)
    cs, pos, q = torch.zeros(10, 64), torch.zeros(4, dtype=torch.int64), torch.zeros(4, 2, 64, dtype=bf)
    for bad, err in (
            (lambda: hs.latent_norm_rope_store(c, pe, None, cs, None, rows, loc), ValueError),
            (lambda: hs.latent_norm_rope_store(c, pe[:3], None, cs, pos, rows, loc), ValueError),
            (lambda: hs.latent_norm_rope_store(c, pe, None, cs[:, :32], pos, rows, loc), ValueError),
            (lambda: hs.latent_norm_rope_store(c, pe, None, cs, pos, rows[:, :600], loc), ValueError),
            (lambda: hs.latent_norm_rope_store(c, pe, None, cs, pos, rows.float(), loc), TypeError),
            (lambda: hs.latent_norm_rope_store(c, pe, None, cs, pos, rows, loc.int()), TypeError),
            (lambda: hs.latent_norm_rope_store(c, pe, None, cs, pos, rows, loc, q_pe=q), ValueError),
            (lambda: hs.latent_norm_rope_store(c, pe.float(), None, cs, pos, rows, loc), TypeError),
            (lambda: hs.latent_norm_rope_store(c, pe, None, cs, pos, rows, loc, q_pe=q, q_out=q[:, :1]), ValueError)):
        with pytest.raises(err):
            bad()
    q, out, idx = torch.zeros(4, 2, 576, dtype=bf), torch.zeros(4, 2, 512, dtype=bf), torch.zeros(4, 8, dtype=torch.int32)
    for bad, err in (
            (lambda: hs.latent_attention(q.double(), rows, idx, out, scale=1.0), TypeError),
            (lambda: hs.latent_attention(q, rows, idx[:3], out, scale=1.0), ValueError),
            (lambda: hs.latent_attention(q, rows, idx.long(), out, scale=1.0), TypeError),
            (lambda: hs.latent_attention(q, rows, idx, out.float(), scale=1.0), TypeError),
            (lambda: hs.latent_attention(q, rows[:, :600], idx, out, scale=1.0), ValueError),
            (lambda: hs.latent_attention(q, rows, idx, out[:, :1], scale=1.0), ValueError),
            (lambda: hs.latent_attention(q, rows, idx, out, scale=1.0, lse=torch.zeros(4, 3)), ValueError),
            (lambda: hs.latent_attention(q, rows, idx, out, scale=1.0, status=torch.zeros(3, dtype=torch.int32)), ValueError),
            (lambda: hs.latent_attention(q, rows, idx, out, scale=1.0), ValueError)):  # not on a CUDA device
        with pytest.raises(err):
            bad()
    t, i, cu = torch.zeros(4, 8, dtype=torch.int32), torch.zeros(4, dtype=torch.int64), torch.zeros(5, dtype=torch.int32)
    kw = dict(max_q_len=1, page_size=1, scale=1.0)
    for bad, err in (
            (lambda: hs.paged_latent_attention(q, rows, t, i[:3], cu, i, out, **kw), ValueError),
            (lambda: hs.paged_latent_attention(q, rows, t, i, cu.long(), i, out, **kw), TypeError),
            (lambda: hs.paged_latent_attention(q, rows, t[0], i, cu, i, out, **kw), ValueError),
            (lambda: hs.paged_latent_attention(q, rows, t, i, cu, i.float(), out, **kw), TypeError)):
        with pytest.raises(err):
            bad()


@pytest.mark.parametrize("tokens,group,strides", [
    (3, 16, (0, 1)), (3, 16, (4, 0)), (3, 16, (0, 0)), (3, 16, (1, 1)), (3, 16, (3, 1)), (3, 16, (1, 2)), (3, 16, (2, 2)),
    (3, 16, (-2, 1)), (3, 16, (1 << 40, 0)), (2, 0, (0, 1)), (1, 16, (4, 0))])
def test_scales_strides(lib, tokens, group, strides):
    """Two scales in one place would race."""
    places = [t * strides[0] + g * strides[1] for t in range(tokens) for g in range(64 // group if group else 1)]
    assert len(set(places)) < len(places)
    a = _norm(n_tokens=tokens, group=group, codes=16384, codes_stride=64, scales=4096, scales_stride_token=strides[0],
              scales_stride_group=strides[1])
    assert lib.hs_add_rms_norm(C.byref(a), None) == 1
    assert b"scales" in lib.hs_last_error()


@pytest.mark.parametrize("tokens,heads,strides", [
    (2, 1, (0, 64)), (2, 2, (0, 64)), (3, 2, (63, 64)), (2, 2, (64, 64)), (3, 4, (128, 64)), (2, 3, (128, 128)), (4, 3, (192, 288))])
def test_outputs_that_share_places(lib, tokens, heads, strides):
    """Two tokens' outputs in one place would race."""
    a = _rows(n_tokens=tokens, num_heads=heads, out_stride_token=strides[0], out_stride_head=strides[1])
    assert lib.hs_latent_norm_rope_store(C.byref(a), None) == 1
    assert b"q_out" in lib.hs_last_error()
    for kw in ({}, INDEX):
        a = _attn(**kw | dict(n_tokens=tokens, num_heads=heads, out_stride_token=strides[0] * 8, out_stride_head=strides[1] * 8,
                              q_stride_token=9216))
        assert lib.hs_latent_attention(C.byref(a), None) == 1
        assert b"outputs" in lib.hs_last_error()
