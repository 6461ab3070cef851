"""The expert layer's entry points from several host threads at once, each on its own stream (GPU).

The headers state that calls are thread-safe. The library raises the LDS allowance of a kernel on its first use, once
for each device. This test runs in a fresh process, so that the first calls of every entry point and of every kernel
with an allowance race one another: eight threads, each on its own torch stream, make the calls in different orders,
three times over outputs poisoned before each call. Their bits must be those of the same calls made afterwards one by
one (every kernel here gives the same bits on every run; other tests hold them to plain implementations).
"""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TESTS = os.path.dirname(os.path.abspath(__file__))

THREADED_CALLS = r"""
import sys
import threading

import torch

import group_scale_factor_amd as gsf
from test_experts_products_gpu import DEV, ends_of, fp8_m_inputs, mx_m_inputs, random_codes

THREADS, REPEATS = 8, 3
gen = torch.Generator(device=DEV).manual_seed(7)
cases = []          # (label, call(outs), (shape, type) of each output)
bf16, f16, f32, i32, u8 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.uint8


def add(label, call, *outs):
    cases.append((label, call, outs))


def randn(*shape):
    return torch.randn(shape, generator=gen, device=DEV)


# the sort: one workgroup with little and with much LDS, two and three launches
for T, k, E in ((300, 4, 16), (4096, 4, 2048), (9001, 4, 64), (40000, 4, 4096)):
    ids = torch.randint(-1, E, (T, k), generator=gen, device=DEV)
    add("sort %d x %d, %d experts" % (T, k, E),
        lambda o, ids=ids, E=E: gsf.moe_sort_tokens(ids, E, out=o), ((E,), i32), ((T * k,), i32), ((T, k), i32))

# the moves
T, k, D = 700, 3, 1409
slots = torch.randperm(T * k, generator=gen, device=DEV).to(i32).view(T, k)
position = torch.where(torch.rand((T, k), generator=gen, device=DEV) < 0.2, ~slots, slots)
weights = torch.rand((T, k), generator=gen, device=DEV)
for t in (bf16, f16, f32):
    x, y = randn(T, D).to(t), randn(T * k, D).to(t)
    add("gather %s" % t, lambda o, x=x: gsf.moe_gather_tokens(x, position, out=o[0]), ((T * k, D), t))
    add("combine %s" % t, lambda o, y=y: gsf.moe_combine_tokens(y, position, weights, out=o[0]), ((T, D), t))
    add("backward %s" % t, lambda o, x=x, y=y: gsf.moe_combine_tokens_backward(x, y, position, weights, dy=o[0],
                                                                             dweights=o[1]), ((T * k, D), t), ((T, k), f32))

# products of row groups: streamed, 32 x 128, 128 x 128 and 256 x 256 tiles
for sizes, K, N in (([1], 128, 16), ([1, 2, 1, 0, 4], 1408, 4096), ([1300, 0, 777, 1, 923], 1376, 1003),
                    ([5000, 7001], 256, 2056)):
    rows = sum(sizes)
    a, asc, w, wsc, ends = mx_m_inputs(sizes, 0, K, N, 1)
    asc, wsc = gsf.mx_block_rearrange_M_groups(asc, ends), gsf.mx_block_rearrange_3d(wsc)
    add("mx rows %s" % sizes, lambda o, v=(a, asc, w, wsc, ends): gsf.mx_grouped_mm_M_groups(*v, out=o[0]),
        ((rows, N), bf16))
    add("fp8 rows %s" % sizes, lambda o, v=fp8_m_inputs(sizes, 0, K, N, 2): gsf.fp8_grouped_mm_M_groups(*v, out=o[0]),
        ((rows, N), bf16))

# products of token groups; the casts
for sizes, M, N in (([32], 16, 16), ([640, 0, 2080], 40, 4000), ([640, 0, 2080], 1408, 1003),
                    ([512, 0, 704, 32, 128] * 3, 1272, 1528)):
    T, G, ends = sum(sizes), len(sizes), ends_of(sizes)
    a, b = random_codes(gen, M, T), random_codes(gen, N, T)
    asc, bsc = (gsf.mx_block_rearrange_K_groups(
        torch.randint(112, 140, (n, T // 32), generator=gen, device=DEV, dtype=u8), ends // 32) for n in (M, N))
    add("mx tokens %s, %d" % (sizes, M), lambda o, v=(a, asc, b, bsc, ends): gsf.mx_grouped_mm_K_groups(*v, out=o[0]),
        ((G, M, N), bf16))
    Tp = gsf.fp8_quantize_cols_K_groups_tokens(T, G)
    a, b = random_codes(gen, M, Tp), random_codes(gen, N, Tp)
    asc, bsc = (torch.exp2(torch.randint(-9, 9, (Tp // 128, n), generator=gen, device=DEV).float()) for n in (M, N))
    add("fp8 tokens %s, %d" % (sizes, M), lambda o, v=(a, asc, b, bsc, ends): gsf.fp8_grouped_mm_K_groups(*v, out=o[0]),
        ((G, M, N), bf16))
x, w, sizes = randn(777, 640).to(bf16), randn(3, 144, 272).to(bf16), [300, 0, 77, 400]
for G in (4, 70):
    ends = ends_of(sizes + [0] * (G - 4))
    Tp = gsf.fp8_quantize_cols_K_groups_tokens(777, G)
    add("cast of columns, %d groups" % G, lambda o, e=ends: gsf.fp8_quantize_cols_K_groups(x, e, qT=o[0], scales=o[1]),
        ((640, Tp), u8), ((Tp // 128, 640), f32))
add("cast of rows", lambda o: gsf.fp8_quantize_rows(x, q=o[0], scales=o[1]), ((777, 640), u8), ((5, 777), f32))
add("cast of tiles", lambda o: gsf.fp8_quantize_tiles(w, False, q=o[0], scales=o[1]), ((3, 144, 272), u8), ((3, 2, 3), f32))
add("cast of tiles, transposed", lambda o: gsf.fp8_quantize_tiles(w, True, q=o[0], scales=o[1]),
    ((3, 272, 144), u8), ((3, 3, 2), f32))


def buffers():
    return [[torch.empty(shape, dtype=t, device=DEV) for shape, t in c[2]] for c in cases]


def poison(outs, byte):
    for o in outs:
        o.view(u8).fill_(byte & 0xFF)


def bits(t):
    return t.view(u8)


streams = [torch.cuda.Stream() for _ in range(THREADS)]
outs = [[buffers() for _ in range(REPEATS)] for _ in range(THREADS)]
torch.cuda.synchronize()
failures = []
start = threading.Barrier(THREADS)
count_lock = threading.Lock()
done = [0]


def worker(t):
    try:
        order = [(t * 5 + i) % len(cases) for i in range(len(cases))]
        if t % 2:
            order.reverse()
        with torch.cuda.stream(streams[t]):
            start.wait(timeout=120)
            for rep in range(REPEATS):
                for i in order:
                    poison(outs[t][rep][i], 0x5A + 17 * t + rep)
                    cases[i][1](outs[t][rep][i])
                    with count_lock:
                        done[0] += 1
            streams[t].synchronize()
    except BaseException as exc:   # a thread that dies must fail the run, not vanish
        failures.append("thread %d raised %r" % (t, exc))


threads = [threading.Thread(target=worker, args=(t,)) for t in range(THREADS)]
for th in threads:
    th.start()
for th in threads:
    th.join()
torch.cuda.synchronize()
wanted = buffers()
for i, (label, call, _) in enumerate(cases):
    poison(wanted[i], 0xA5)
    call(wanted[i])
    for t in range(THREADS):
        for rep in range(REPEATS):
            for n, (o, want) in enumerate(zip(outs[t][rep][i], wanted[i])):
                if not torch.equal(bits(o), bits(want)):
                    failures.append("thread %d repeat %d %s output %d" % (t, rep, label, n))
print("threads %d, cases %d, repeats %d, calls %d" % (THREADS, len(cases), REPEATS, done[0]))
if failures or done[0] != THREADS * REPEATS * len(cases):
    print("\n".join(failures[:20]))
    sys.exit(1)
print("threaded calls: ok")
"""


def test_expert_layer_calls_from_many_threads_give_the_bits_of_single_ones():
    from group_scale_factor_amd import _build

    if not os.path.exists(_build.EXPERTS_LIBRARY):
        _build.build()
    print("case threaded calls of the expert layer in a fresh process", flush=True)
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([ROOT, TESTS, os.environ.get("PYTHONPATH", "")]))
    res = subprocess.run([sys.executable, "-c", THREADED_CALLS], capture_output=True, text=True, timeout=300, env=env,
                         cwd=ROOT)
    print(res.stdout[-3000:])
    assert res.returncode == 0, res.stdout[-3000:] + res.stderr[-3000:]
    assert res.stdout.strip().endswith("threaded calls: ok")
