"""Calls at the edges of the expert layer's operators: what no group or row of them may notice (GPU)."""

import numpy as np
import pytest
import torch

import group_scale_factor_amd as gsf
from test_experts_products_gpu import DEV, ends_of, random_codes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("empty", [[1], [0, 7], [2, 3, 4]])
def test_empty_token_groups_leave_the_others_bits(empty):
    """Scales that are powers of two: with a group of no tokens or without it, the other groups' sums take the same
    instructions. More large tiles than compute units, so that a workgroup goes on from an empty group's tile."""
    sizes, M, N = [500, 700, 1, 128, 256, 384] * 2, 1272, 1528
    with_empty = list(sizes)
    for g in empty:
        with_empty.insert(g, 0)
    T = sum(sizes)
    gen = torch.Generator(device=DEV).manual_seed(len(empty))
    Tp = gsf.fp8_quantize_cols_K_groups_tokens(T, len(with_empty))
    codes = [random_codes(gen, n, Tp) for n in (M, N)]
    scales = [torch.exp2(torch.randint(-12, 12, (Tp // 128, n), generator=gen, device=DEV).double()).float()
              for n in (M, N)]
    res = []
    for these in (sizes, with_empty):
        tp = gsf.fp8_quantize_cols_K_groups_tokens(T, len(these))
        (a, b), (asc, bsc) = [c[:, :tp].contiguous() for c in codes], [s[: tp // 128].contiguous() for s in scales]
        res.append(gsf.fp8_grouped_mm_K_groups(a, asc, b, bsc, ends_of(these)))
    kept = torch.tensor([n > 0 for n in with_empty], device=DEV)
    assert torch.equal(res[1][kept], res[0])
    assert bool((res[1][~kept] == 0).all())


@pytest.mark.parametrize("k,E", [(1, 2049), (8, 4096), (64, 2048), (2, 3)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort_of_no_tokens_writes_the_ends(k, E, dtype):
    ends = torch.full((E,), 7, dtype=torch.int32, device=DEV)
    order = torch.empty(0, dtype=torch.int32, device=DEV)
    position = torch.empty((0, k), dtype=torch.int32, device=DEV)
    got = gsf.moe_sort_tokens(torch.empty((0, k), dtype=dtype, device=DEV), E, out=(ends, order, position))
    assert got[0] is ends and bool((ends == 0).all())


@pytest.mark.parametrize("kind", ["mx", "fp8"])
@pytest.mark.parametrize("sizes,tail,N", [([3, 0, 5], 2, 40), ([1], 0, 16), ([300], 0, 300)])
def test_row_products_over_no_depth_are_zeros(kind, sizes, tail, N):
    rows, E = sum(sizes) + tail, len(sizes)
    a = torch.empty((rows, 0), dtype=torch.uint8, device=DEV)
    w = torch.empty((E, N, 0), dtype=torch.uint8, device=DEV)
    if kind == "mx":
        asc = wsc = torch.empty(0, dtype=torch.uint8, device=DEV)
    else:
        asc = torch.empty((0, rows), device=DEV)
        wsc = torch.empty((E, -(-N // 128), 0), device=DEV)
    out = torch.full((rows, N), 3.0, dtype=torch.bfloat16, device=DEV)
    mm = gsf.mx_grouped_mm_M_groups if kind == "mx" else gsf.fp8_grouped_mm_M_groups
    assert mm(a, asc, w, wsc, ends_of(sizes), out=out) is out
    assert bool((out == 0).all())
