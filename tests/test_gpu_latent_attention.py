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
