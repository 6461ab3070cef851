"""Calls at the edges of the expert layer's operators (GPU): no tokens, no depth, groups of no tokens among others,
scales of another kind, workgroups that start with rows in no group. Products are held to the bounds that
test_experts_products_gpu.py derives."""

import pytest
import torch

import group_scale_factor_amd as gsf
from test_experts_products_gpu import (DEV, ends_of, fp8_dequant, fp8_m_inputs, k_reference, m_reference, mx_dequant,
                                       mx_m_inputs, near, random_codes)

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


# Block-128 scales that are no powers of two among large tiles of token groups, whose workgroups change over to
# multiplications there: (step of 36, row, value) at the first, a middle and the last step of a tile and of a workgroup,
# in the first and the last row, next to a tile's edge, in several; a zero, a negative, a subnormal and a huge number.
TOKEN_OTHERS = [[(35, 0, 1.5)], [(35, -1, 0.75)], [(3, 255, 2.0 ** -130), (4, 256, 1e30)], [(4, 0, -2.0)], [(9, 511, 0.0)],
                [(17, -1, 3.0), (18, 0, 3.0)], [(0, -1, 0.7), (11, 3, 1e-3), (34, 257, -5.0)],
                [(b, 7 * b, 0.7) for b in range(36)]]


@pytest.mark.parametrize("others", TOKEN_OTHERS)
@pytest.mark.parametrize("side", [0, 1])
def test_other_scales_among_large_token_tiles(others, side):
    sizes, M, N = [500, 0, 700, 1, 128] * 3, 1272, 1528
    padded = [-(-n // 128) * 128 for n in sizes]
    ends, T = ends_of(sizes), sum(sizes)
    Tp = gsf.fp8_quantize_cols_K_groups_tokens(T, len(sizes))
    gen = torch.Generator(device=DEV).manual_seed(100 + side)
    codes = [random_codes(gen, n, Tp, narrow=True) for n in (M, N)]
    scales = [torch.exp2(torch.randint(-12, 12, (Tp // 128, n), generator=gen, device=DEV).double()).float()
              for n in (M, N)]
    for step, row, value in others:
        scales[side][step, row] = value
    got = gsf.fp8_grouped_mm_K_groups(codes[0], scales[0], codes[1], scales[1], ends)
    near(got, *k_reference(fp8_dequant(codes[0], scales[0].t()), fp8_dequant(codes[1], scales[1].t()), padded),
         max(padded), narrow=True)
    again = gsf.fp8_grouped_mm_K_groups(codes[0], scales[0], codes[1], scales[1], ends)
    assert torch.equal(got, again)


# Large tiles whose workgroups start with rows in no group: fewer tiles than compute units, and no rows in groups at all
@pytest.mark.parametrize("sizes,tail,K,N", [([584] * 16, 896, 2048, 1024), ([0] * 16, 10240, 256, 1024),
                                            ([0, 2600, 0], 7000, 384, 1500)])
@pytest.mark.parametrize("kind", ["mx", "fp8"])
def test_workgroups_that_start_with_rows_in_no_group(kind, sizes, tail, K, N):
    make = mx_m_inputs if kind == "mx" else fp8_m_inputs
    a, asc, w, wsc, ends = make(sizes, tail, K, N, K + N, narrow=True)
    rows = a.shape[0]
    out = torch.full((rows, N), 3.0, dtype=torch.bfloat16, device=DEV)
    if kind == "mx":
        av, wv = mx_dequant(a, asc), lambda e: mx_dequant(w[e], wsc[e])
        gsf.mx_grouped_mm_M_groups(a, gsf.mx_block_rearrange_M_groups(asc, ends), w, gsf.mx_block_rearrange_3d(wsc), ends,
                                   out=out)
    else:
        av, wv = fp8_dequant(a, asc.t()), lambda e: fp8_dequant(w[e], wsc[e].repeat_interleave(128, 0)[:N])
        gsf.fp8_grouped_mm_M_groups(a, asc, w, wsc, ends, out=out)
    near(out, *m_reference(av, wv, sizes, rows, N), K, narrow=True)
    assert bool((out[rows - tail:] == 0).all())
