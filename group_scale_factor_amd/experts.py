"""Expert-layer operators around the grouped casts: tokens sorted by expert and back,
and the grouped products of 8-bit operands.

Thin binding over the C ABI in ``include/moe/``: checks, sizes, output allocation
and the call on the current torch stream, as in the package's other entry points.

    ends, order, position = moe_sort_tokens(expert_ids, num_experts)
    rows = moe_gather_tokens(x, position)                            # into the token groups
    dx = moe_gather_tokens_backward(drows, position)
    out = moe_combine_tokens(y, position, weights)                   # and back
    dy, dweights = moe_combine_tokens_backward(dout, y, position, weights)

    out = mx_grouped_mm_M_groups(q, scales, w_q, w_scales, ends)     # MXFP8 casts' codes and blocked scales
    dw = mx_grouped_mm_K_groups(doutT, dout_scales, xT, x_scales, ends)

    q, scales = fp8_quantize_rows(x)                                 # one scale for each block of 128
    w_q, w_scales = fp8_quantize_tiles(w, transposed=False)
    qT, scales = fp8_quantize_cols_K_groups(x, ends)
    out = fp8_grouped_mm_M_groups(q, scales, w_q, w_scales, ends)
    dw = fp8_grouped_mm_K_groups(doutT, dout_scales, xT, x_scales, ends)

Codes are uint8 tensors or float8_e4m3fn ones. With ``stream`` (a raw hipStream_t
handle) the call runs there, and what it allocates belongs to that stream; inputs
have to be ready on it, and a caller that uses the result elsewhere orders that
itself. Without, everything happens on torch's current stream.
"""

import ctypes
import os

from . import _build

LIBRARY = _build.EXPERTS_LIBRARY

# Set on the first call: importing the package does not import torch, and no call looks either up again (a call
# of a few microseconds' work is as long as its checks).
_lib = None
torch = None
_package = None


def _load():
    global _lib, _package, torch
    if _lib is not None:
        return _lib
    if not os.path.exists(LIBRARY):
        raise ImportError(
            "HIP library %s is not built; run __graft_entry__.build() (hipcc --offload-arch=gfx950)" % LIBRARY)
    lib = ctypes.CDLL(LIBRARY)
    i64, i32, vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
    arguments = {
        "moe_sort_tokens": [vp, i32, i64, i32, i64, i32, vp, vp, vp, vp, vp],
        "moe_gather_tokens": [vp, i32, i64, i32, i64, i64, vp, vp, i64, vp],
        "moe_combine_tokens": [vp, i32, i64, i32, i64, i64, vp, vp, vp, i64, vp],
        "moe_combine_tokens_backward": [vp, i32, i64, i32, i64, i64, vp, i64, vp, vp, vp, i64, vp, vp],
        "mx_grouped_mm_M_groups": [vp, vp, i64, i64, i64, vp, vp, i64, i64, i64, vp, i32, vp, i64, vp],
        "mx_grouped_mm_K_groups": [vp, vp, i64, vp, vp, i64, i64, vp, i32, vp, vp],
        "fp8_quantize_rows": [vp, i64, i64, i64, vp, vp, vp],
        "fp8_quantize_tiles": [vp, i64, i64, i64, i64, i64, i32, vp, vp, vp],
        "fp8_quantize_cols_K_groups": [vp, i64, i64, i64, vp, i32, vp, vp, vp],
        "fp8_grouped_mm_M_groups": [vp, vp, i64, i64, i64, vp, vp, i64, i64, i64, vp, i32, vp, i64, vp],
        "fp8_grouped_mm_K_groups": [vp, vp, i64, vp, vp, i64, i64, vp, i32, vp, vp],
    }
    for name, args in arguments.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    import torch as _torch

    import group_scale_factor_amd as package

    torch, _package = _torch, package
    _lib = lib
    return lib


def experts_library():
    """The loaded ctypes handle of libmoeexperts.so."""
    return _load()


# The headers' size helpers, restated as the package's other entry points restate theirs; a CPU test
# compiles the headers and checks both.

def moe_sort_tokens_workspace_bytes(tokens, topk, num_experts):
    """4 * (E + 1) * (runs of 1024 slots + 1); 0 up to 16384 slots and 2048 experts, and for no tokens; -1 for
    invalid sizes (include/moe/moe_tokens.h)."""
    if tokens < 0 or not 1 <= topk <= 64 or not 1 <= num_experts <= 4096 or tokens > (0x7fffffff - 4096) // topk:
        return -1
    if tokens == 0 or tokens * topk <= 16384 and num_experts <= 2048:
        return 0
    return 4 * (num_experts + 1) * ((tokens * topk + 1023) // 1024 + 1)


def fp8_quantize_cols_K_groups_tokens(T, num_groups):
    """round_up(T, 128) + 128*G; -1 for invalid sizes (include/moe/fp8_block128.h)."""
    if T < 0 or num_groups < 1:
        return -1
    return (T + 127) // 128 * 128 + 128 * num_groups


def _blocks(n):
    return (n + 127) // 128


def _handle(stream, device):
    # torch's current stream as its raw handle: a torch.cuda.Stream object would take longer to make than a launch
    return (torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream) or None


def _empty(shape, dtype, device, stream):
    """An uninitialised tensor of the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    on = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    with torch.cuda.stream(on):
        return torch.empty(shape, dtype=dtype, device=device)


def _output(out, name, shape, dtype, device, stream):
    """`out` checked as a dense tensor, or a new one."""
    if out is None:
        return _empty(shape, dtype, device, stream)
    if out.dtype != dtype or tuple(out.shape) != shape or out.device != device or not out.is_contiguous():
        raise ValueError("%s must be a contiguous %s %s tensor on the inputs' device" % (name, shape, dtype))
    return out


def _rows_output(out, name, rows, cols, dtype, device, stream):
    """`out` checked as a (rows, cols) tensor of unit column stride and any row stride, or a new one; its row stride."""
    if out is None:
        return _empty((rows, cols), dtype, device, stream), cols
    if out.dtype != dtype or tuple(out.shape) != (rows, cols) or out.device != device or (
            rows > 0 and cols > 1 and out.stride(1) != 1):
        raise ValueError("%s must be a (%d, %d) %s tensor with unit column stride on the inputs' device"
                         % (name, rows, cols, dtype))
    return out, out.stride(0) if rows > 1 else cols


def _check_rows(t, name, dtypes, dims=2):
    """Row stride of a GPU tensor of one of `dtypes` with unit column stride."""
    if t.dtype not in dtypes or t.dim() != dims:
        raise TypeError("%s must be a %d-D tensor of %s" % (name, dims, " or ".join(str(d) for d in dtypes)))
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    shape, stride = t.shape, t.stride()
    if stride[-1] != 1 and shape[-1] > 1 and t.numel() > 0:
        raise ValueError("%s must have unit column stride" % name)
    return stride[-2] if shape[-2] > 1 and shape[-1] > 0 else shape[-1]     # no second row, or rows of nothing: as dense


def _check_codes(t, name, dims):
    """Row stride of E4M3 codes (their type does not matter to a data pointer)."""
    if t.dtype != torch.uint8 and t.dtype != torch.float8_e4m3fn:
        raise TypeError("%s must hold E4M3 codes (uint8 or float8_e4m3fn)" % name)
    return _check_rows(t, name, (t.dtype,), dims)


def _check_flat(t, name, dtype, shape, count, device):
    """A dense tensor of `dtype`: of that shape, or (shape None) with at least `count` elements."""
    if t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise TypeError("%s must be a contiguous %s tensor on the inputs' device" % (name, dtype))
    if shape is None:
        if t.numel() < count:
            raise ValueError("%s must hold at least %d elements" % (name, count))
    elif tuple(t.shape) != shape:
        raise ValueError("%s must have the shape %s" % (name, shape))


def _ptr(t):
    return None if t is None else t.data_ptr() or None


def _check(rc):
    if rc != 0:
        raise _package.RearrangeError(rc)


# ------------------------------------------------------------------ tokens


def moe_sort_tokens(expert_ids, num_experts, out=None, workspace=None, stream=None):
    """Slots (token, choice) sorted by expert: the plan of an expert layer's token groups.

    ``expert_ids``: (T, k) int32 or int64 CUDA tensor, unit column stride; an id outside
    [0, num_experts) drops its slot. Returns int32 tensors (group_end_offsets (E,), order (T*k,),
    position (T, k)): sorted row r holds slot ``order[r]``, slot t*k+j lies in row
    ``position[t, j]``; dropped slots fill the rows past the last end, both as ``~`` of the number.
    Slots of one expert keep their order. ``out``: those three to write into; ``workspace``: a flat
    uint8 tensor of ``moe_sort_tokens_workspace_bytes`` bytes, allocated when it is None.
    """
    lib = _lib or _load()
    stride = _check_rows(expert_ids, "expert_ids", (torch.int64, torch.int32))
    T, k = expert_ids.shape
    dev = expert_ids.device
    n = moe_sort_tokens_workspace_bytes(T, k, num_experts)
    if n < 0:
        raise ValueError("invalid sizes tokens=%d topk=%d num_experts=%d" % (T, k, num_experts))
    ends, order, position = out if out is not None else (None, None, None)
    ends = _output(ends, "group_end_offsets", (num_experts,), torch.int32, dev, stream)
    order = _output(order, "order", (T * k,), torch.int32, dev, stream)
    position = _output(position, "position", (T, k), torch.int32, dev, stream)
    if workspace is not None:
        _check_flat(workspace, "workspace", torch.uint8, None, n, dev)
    elif n > 0:
        workspace = _empty(n, torch.uint8, dev, stream)
    _check(lib.moe_sort_tokens(_ptr(expert_ids), expert_ids.element_size(), T, k, stride, num_experts, _ptr(ends),
                               _ptr(order), _ptr(position), _ptr(workspace), _handle(stream, dev)))
    return ends, order, position


def _row_type(t, name):
    """(type number, row stride) of a tensor of rows to move."""
    number = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}.get(t.dtype, -1)
    if number < 0:
        raise TypeError("%s must be a 2-D tensor of bfloat16, float16 or float32" % name)
    return number, _check_rows(t, name, (t.dtype,))


def _check_plan(position, device, rows=None):
    if position.dtype != torch.int32 or position.dim() != 2 or not position.is_contiguous():
        raise TypeError("position must be a contiguous 2-D torch.int32 tensor")
    if position.device != device:
        raise ValueError("position must be on the rows' device")
    if rows is not None and rows != position.numel():
        raise ValueError("the sorted rows must be as many as the plan's slots (%d)" % position.numel())


def moe_gather_tokens(x, position, out=None, stream=None):
    """Tokens copied into their groups: out[position[t, j]] = x[t]; rows of dropped slots are zero.

    ``x``: (T, D) bf16, f16 or f32 CUDA tensor, unit column stride; ``position``: (T, k) of
    ``moe_sort_tokens``. Returns (T*k, D) of x's type; ``out`` may have any row stride.
    """
    lib = _lib or _load()
    number, stride = _row_type(x, "x")
    dev = x.device
    _check_plan(position, dev)
    T, D = x.shape
    if position.shape[0] != T:
        raise ValueError("x must have the plan's %d tokens" % position.shape[0])
    k = position.shape[1]
    out, out_stride = _rows_output(out, "out", T * k, D, x.dtype, dev, stream)
    _check(lib.moe_gather_tokens(_ptr(x), number, T, k, D, stride, _ptr(position), _ptr(out), out_stride,
                                 _handle(stream, dev)))
    return out


def moe_combine_tokens(y, position, weights=None, out=None, stream=None):
    """The experts' rows summed back: out[t] = sum_j weights[t, j] * y[position[t, j]], dropped slots left out.

    ``y``: (T*k, D) bf16, f16 or f32; ``weights``: (T, k) f32, or None for ones. Sums are 32-bit, in
    the order of j, rounded once. Returns (T, D) of y's type; ``out`` may have any row stride.
    """
    lib = _lib or _load()
    number, stride = _row_type(y, "y")
    dev = y.device
    rows, D = y.shape
    _check_plan(position, dev, rows)
    T, k = position.shape
    if weights is not None:
        _check_flat(weights, "weights", torch.float32, (T, k), 0, dev)
    out, out_stride = _rows_output(out, "out", T, D, y.dtype, dev, stream)
    _check(lib.moe_combine_tokens(_ptr(y), number, T, k, D, stride, _ptr(position), _ptr(weights), _ptr(out),
                                  out_stride, _handle(stream, dev)))
    return out


def moe_gather_tokens_backward(drows, position, out=None, stream=None):
    """Gradient of ``moe_gather_tokens``: dx[t] = sum_j drows[position[t, j]], dropped slots left out."""
    return moe_combine_tokens(drows, position, None, out, stream)


def moe_combine_tokens_backward(dout, y, position, weights, dy=None, dweights=None, stream=None):
    """Gradients of ``moe_combine_tokens``: dy[position[t, j]] = weights[t, j] * dout[t] (zero rows for
    dropped slots) and dweights[t, j] = <dout[t], y[position[t, j]]> (0 for dropped slots).

    ``dout``: (T, D) of y's type. Returns (dy (T*k, D), dweights (T, k) f32). ``dy`` must not overlap y.
    """
    lib = _lib or _load()
    number, stride = _row_type(y, "y")
    dout_stride = _check_rows(dout, "dout", (y.dtype,))
    dev = y.device
    rows, D = y.shape
    _check_plan(position, dev, rows)
    T, k = position.shape
    _check_flat(weights, "weights", torch.float32, (T, k), 0, dev)
    if tuple(dout.shape) != (T, D) or dout.device != dev:
        raise ValueError("dout must be a (%d, %d) tensor on y's device" % (T, D))
    dy, dy_stride = _rows_output(dy, "dy", rows, D, y.dtype, dev, stream)
    dweights = _output(dweights, "dweights", (T, k), torch.float32, dev, stream)
    _check(lib.moe_combine_tokens_backward(_ptr(dout), number, T, k, D, dout_stride, _ptr(y), stride, _ptr(position),
                                           _ptr(weights), _ptr(dy), dy_stride, _ptr(dweights), _handle(stream, dev)))
    return dy, dweights


# ------------------------------------------------------------------ products


def _mm_M(mx, a, a_scales, w, w_scales, offs, out, stream):
    lib = _lib or _load()
    a_stride, w_row = _check_codes(a, "a", 2), _check_codes(w, "w", 3)
    dev = a.device
    rows, K = a.shape
    G, N, wK = w.shape
    if wK != K or w.device != dev:
        raise ValueError("w must be (experts, N, %d) on a's device" % K)
    _package._check_offsets(offs, dev)
    if offs.numel() != G:
        raise ValueError("group_end_offsets must have one end for each of w's %d experts" % G)
    if mx:
        count = _package.mx_rearrange_M_groups_out_bytes(rows, K // 32, G)
        _check_flat(a_scales, "a_scales", torch.uint8, None, count, dev)
        _check_flat(w_scales, "w_scales", torch.uint8, None, _package.mx_rearrange_3d_out_bytes(G, N, K // 32), dev)
    else:
        _check_flat(a_scales, "a_scales", torch.float32, (_blocks(K), rows), 0, dev)
        _check_flat(w_scales, "w_scales", torch.float32, (G, _blocks(N), _blocks(K)), 0, dev)
    out, out_stride = _rows_output(out, "out", rows, N, torch.bfloat16, dev, stream)
    fn = lib.mx_grouped_mm_M_groups if mx else lib.fp8_grouped_mm_M_groups
    _check(fn(_ptr(a), _ptr(a_scales), rows, K, a_stride, _ptr(w), _ptr(w_scales), N,
              w.stride(0) if G > 1 and K > 0 else N * w_row, w_row, _ptr(offs), G, _ptr(out), out_stride,
              _handle(stream, dev)))
    return out


def mx_grouped_mm_M_groups(a, a_scales, w, w_scales, group_end_offsets, out=None, stream=None):
    """Grouped product of MXFP8 operands, groups along the rows: out[r] = a[r] . w[group of r]^T, bf16.

    ``a``: (rows, K) E4M3 codes, K a multiple of 32, with ``a_scales`` the flat M-groups blocked scales
    (``mx_quantize_dim0_M_groups``); ``w``: (E, N, K) codes with the flat per-expert blocked
    ``w_scales`` (``mx_quantize_dim1_3d``). Rows in no group come out zero. Rows and experts may be
    strided by multiples of 16 bytes. Returns (rows, N) torch.bfloat16.
    """
    return _mm_M(True, a, a_scales, w, w_scales, group_end_offsets, out, stream)


def fp8_grouped_mm_M_groups(a, a_scales, w, w_scales, group_end_offsets, out=None, stream=None):
    """Grouped product of operands with a scale for each block of 128, groups along the rows, bf16.

    ``a``: (rows, K) E4M3 codes, K a multiple of 16, with ``a_scales`` (ceil(K/128), rows) f32
    (``fp8_quantize_rows``); ``w``: (E, N, K) codes with ``w_scales`` (E, ceil(N/128), ceil(K/128)) f32
    (``fp8_quantize_tiles``, or a checkpoint's). Rows in no group come out zero. Rows and experts may
    be strided by multiples of 16 bytes. Returns (rows, N) torch.bfloat16.
    """
    return _mm_M(False, a, a_scales, w, w_scales, group_end_offsets, out, stream)


def _mm_K(mx, a, a_scales, b, b_scales, offs, out, stream):
    lib = _lib or _load()
    _check_codes(a, "a", 2)
    _check_codes(b, "b", 2)
    if not (a.is_contiguous() and b.is_contiguous()):
        raise ValueError("a and b must be contiguous")
    dev = a.device
    M, T = a.shape
    N = b.shape[0]
    if b.shape[1] != T or b.device != dev:
        raise ValueError("b must be (N, %d) on a's device" % T)
    _package._check_offsets(offs, dev)
    G = offs.numel()
    if mx:
        count = _package.mx_rearrange_K_groups_out_bytes
        _check_flat(a_scales, "a_scales", torch.uint8, None, count(M, T // 32, G), dev)
        _check_flat(b_scales, "b_scales", torch.uint8, None, count(N, T // 32, G), dev)
    else:
        if T % 128 != 0 or T < 128 * G:
            raise ValueError("a and b must hold the round_up(T, 128) + 128*G padded tokens of their casts")
        _check_flat(a_scales, "a_scales", torch.float32, (T // 128, M), 0, dev)
        _check_flat(b_scales, "b_scales", torch.float32, (T // 128, N), 0, dev)
    out = _output(out, "out", (G, M, N), torch.bfloat16, dev, stream)
    fn = lib.mx_grouped_mm_K_groups if mx else lib.fp8_grouped_mm_K_groups
    _check(fn(_ptr(a), _ptr(a_scales), M, _ptr(b), _ptr(b_scales), N, T, _ptr(offs), G, _ptr(out),
              _handle(stream, dev)))
    return out


def mx_grouped_mm_K_groups(a, a_scales, b, b_scales, token_group_end_offsets, out=None, stream=None):
    """Grouped product of MXFP8 operands, groups of tokens along the summed axis: out[g] = a_g . b_g^T, bf16.

    ``a``: (M, T) and ``b``: (N, T) dense E4M3 codes with flat K-groups blocked scales, as
    ``mx_quantize_dim1_K_groups`` writes both for the same offsets (multiples of 32). An empty group's
    matrix is zero. Returns (G, M, N) torch.bfloat16: the weight gradient of each expert.
    """
    return _mm_K(True, a, a_scales, b, b_scales, token_group_end_offsets, out, stream)


def fp8_grouped_mm_K_groups(a, a_scales, b, b_scales, token_group_end_offsets, out=None, stream=None):
    """Grouped product of operands with a scale for each block of 128 tokens, groups of tokens along the
    summed axis: out[g] = a_g . b_g^T, bf16.

    ``a``: (M, Tp) and ``b``: (N, Tp) dense E4M3 codes with (Tp/128, M) and (Tp/128, N) f32 scales, as
    ``fp8_quantize_cols_K_groups`` writes both for the same offsets. An empty group's
    matrix is zero. Returns (G, M, N) torch.bfloat16.
    """
    return _mm_K(False, a, a_scales, b, b_scales, token_group_end_offsets, out, stream)


# ------------------------------------------------------------------ casts


def fp8_quantize_rows(x, q=None, scales=None, stream=None):
    """E4M3 cast of rows with one power-of-two scale for each block of 128.

    ``x``: (rows, K) torch.bfloat16 CUDA tensor, K a multiple of 16, 16-byte aligned rows. Returns
    (q (rows, K) uint8 codes, scales (ceil(K/128), rows) f32).
    """
    lib = _lib or _load()
    stride = _check_rows(x, "x", (torch.bfloat16,))
    rows, K = x.shape
    dev = x.device
    q = _output(q, "q", (rows, K), torch.uint8, dev, stream)
    scales = _output(scales, "scales", (_blocks(K), rows), torch.float32, dev, stream)
    _check(lib.fp8_quantize_rows(_ptr(x), rows, K, stride, _ptr(q), _ptr(scales), _handle(stream, dev)))
    return q, scales


def fp8_quantize_tiles(w, transposed=False, q=None, scales=None, stream=None):
    """E4M3 cast of stacked weights with one power-of-two scale for each 128 x 128 block.

    ``w``: (E, N, K) torch.bfloat16 CUDA tensor, K a multiple of 16 (``transposed``: N too). Returns
    (q (E, N, K), scales (E, ceil(N/128), ceil(K/128))), or with ``transposed`` the same values as
    (E, K, N) and (E, ceil(K/128), ceil(N/128)), the weights of the input gradient.
    """
    lib = _lib or _load()
    stride = _check_rows(w, "w", (torch.bfloat16,), 3)
    E, N, K = w.shape
    dev = w.device
    shape, sshape = ((E, K, N), (E, _blocks(K), _blocks(N))) if transposed else ((E, N, K), (E, _blocks(N), _blocks(K)))
    q = _output(q, "q", shape, torch.uint8, dev, stream)
    scales = _output(scales, "scales", sshape, torch.float32, dev, stream)
    _check(lib.fp8_quantize_tiles(_ptr(w), E, N, K, w.stride(0) if E > 1 else N * stride, stride,
                                  1 if transposed else 0, _ptr(q), _ptr(scales), _handle(stream, dev)))
    return q, scales


def fp8_quantize_cols_K_groups(x, token_group_end_offsets, qT=None, scales=None, stream=None):
    """E4M3 cast along the tokens of padded groups, one power-of-two scale for each block of 128 tokens.

    ``x``: (T, N) torch.bfloat16 CUDA tensor, N a multiple of 8, 16-byte aligned rows. Each group's
    tokens are padded to a multiple of 128 (as ``mx_pad_M_groups`` places them). Returns (qT (N, Tp)
    uint8 codes, scales (Tp/128, N) f32), Tp = round_up(T, 128) + 128*G; padding is code 0.
    """
    lib = _lib or _load()
    stride = _check_rows(x, "x", (torch.bfloat16,))
    dev = x.device
    _package._check_offsets(token_group_end_offsets, dev)
    T, N = x.shape
    G = token_group_end_offsets.numel()
    Tp = fp8_quantize_cols_K_groups_tokens(T, G)
    if Tp < 0:
        raise ValueError("invalid sizes T=%d num_groups=%d" % (T, G))
    qT = _output(qT, "qT", (N, Tp), torch.uint8, dev, stream)
    scales = _output(scales, "scales", (Tp // 128, N), torch.float32, dev, stream)
    _check(lib.fp8_quantize_cols_K_groups(_ptr(x), T, N, stride, _ptr(token_group_end_offsets), G, _ptr(qT),
                                          _ptr(scales), _handle(stream, dev)))
    return qT, scales


__all__ = [
    "experts_library",
    "fp8_grouped_mm_K_groups",
    "fp8_grouped_mm_M_groups",
    "fp8_quantize_cols_K_groups",
    "fp8_quantize_cols_K_groups_tokens",
    "fp8_quantize_rows",
    "fp8_quantize_tiles",
    "moe_combine_tokens",
    "moe_combine_tokens_backward",
    "moe_gather_tokens",
    "moe_gather_tokens_backward",
    "moe_sort_tokens",
    "moe_sort_tokens_workspace_bytes",
    "mx_grouped_mm_K_groups",
    "mx_grouped_mm_M_groups",
]
