"""GPU tests of the block-scaled e4m3 quantiser and product against the 64-bit
reference (tests/fp8_reference.py, where the tolerances are derived): codes and
scales bit for bit, Y within its bound."""
from __future__ import annotations

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import int8_quantized_matmul_02_b200 as i8
from tests import fp8_reference as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.float16, torch.bfloat16]


def _x(M, K, dtype, seed, outliers=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g)
    if outliers:
        cols = torch.randperm(K, generator=g)[: max(1, K // 256)]
        x[:, cols] *= 40
    return x.to(dtype)


def _np(t):
    return t.double().cpu().numpy()


def _same_codes(codes, q):
    return np.array_equal(_np(codes.float()), q)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (16, 256), (7, 4112), (257, 1040), (1000, 11008)])
def test_quantize(cuda_ok, M, K, dtype):
    X = _x(M, K, dtype, M + K)
    codes, scales = i8.quantize_fp8(X.cuda())
    q, s = ref.quantize(_np(X))
    assert np.array_equal(_np(scales), s)
    assert _same_codes(codes, q)


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_every_value(cuda_ok, dtype):
    """Every finite value of the type, each in a block whose maximum is a power
    of two times a few mantissas (ties of every kind, subnormal codes)."""
    v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(dtype)
    v = v[torch.isfinite(v.float())]
    v = v[torch.argsort(v.float().abs(), stable=True)]
    v = v[: v.numel() // 128 * 128].view(-1, 128)
    rows = [v]
    for top in (1.0, 1.75, 448.0, 500.0, 30000.0):
        w = v.clone()
        w[w.float().abs() > top] = 0
        w[:, 0] = top
        rows.append(w)
    X = torch.cat(rows)
    codes, scales = i8.quantize_fp8(X.cuda())
    q, s = ref.quantize(_np(X))
    assert np.array_equal(_np(scales), s)
    assert _same_codes(codes, q)


@pytest.mark.parametrize("dtype", DTYPES)
def test_scale_of_every_maximum(cuda_ok, dtype):
    """Each finite value of the type as the maximum of a block, in the
    quantiser (the product's kernel forms its scales by the same function)."""
    v = torch.arange(0, 32768, dtype=torch.int32).to(torch.int16).view(dtype)
    v = v[torch.isfinite(v.float())]
    v = v[: v.numel() // 256 * 256].view(-1, 256)          # row: 256 blocks
    X = torch.zeros(v.shape[0], 256, 128, dtype=dtype)
    X[:, :, 77] = -v
    X = X.view(v.shape[0], -1)
    codes, scales = i8.quantize_fp8(X.cuda())
    q, s = ref.quantize(_np(X))
    assert np.array_equal(_np(scales), s) and _same_codes(codes, q)


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_zero_tiny_and_large_blocks(cuda_ok, dtype):
    X = torch.zeros(6, 272, dtype=dtype)
    X[1, 5] = torch.finfo(dtype).smallest_normal
    X[2, :] = torch.finfo(dtype).smallest_normal * 2.0 ** -3   # subnormal values
    X[3, 130] = torch.finfo(dtype).max
    X[4, 271] = -torch.finfo(dtype).max                         # the last, short block
    X[5, :] = 1.0
    codes, scales = i8.quantize_fp8(X.cuda())
    q, s = ref.quantize(_np(X))
    assert np.array_equal(_np(scales), s) and _same_codes(codes, q)
    assert torch.isfinite(scales).all() and (scales > 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K,N", [(16, 16), (128, 128), (144, 272), (4112, 400)])
def test_prepare_weight(cuda_ok, K, N, dtype):
    W = (_x(K, N, dtype, K * N).float() * 0.02).to(dtype)
    w = i8.prepare_weight_fp8(W.cuda())
    q, s = ref.quantize_weight(_np(W))
    assert np.array_equal(_np(w.scales), s)
    assert _same_codes(w.codes, q)


def _case(M, K, N, dtype, seed):
    X = _x(M, K, dtype, seed)
    W = (_x(K, N, torch.float16, seed + 1).float() / K ** 0.5).half()
    w = i8.prepare_weight_fp8(W.cuda())
    return X, w


def _want(X, w):
    xv = ref.row_values(*ref.quantize(_np(X)))
    return ref.product(xv, ref.weight_values(_np(w.codes.float()), _np(w.scales)))


def _check(Y, X, w):
    y, err = _want(X, w)
    ref.check(Y, y, ref.out_bound(y, err, X.dtype))


SHAPES = [
    (1, 16, 16),          # the smallest layer
    (1, 4096, 528),
    (2, 144, 1040),       # K ends inside a block
    (16, 256, 384),
    (17, 2064, 400),      # 32 columns of rows
    (33, 1040, 272),      # 64
    (64, 512, 128),
    (65, 640, 144),       # 128, two halves of a block of channels
    (100, 11008, 256),
    (129, 272, 4112),
    (300, 4112, 272),     # N and M end inside tiles
    (513, 128, 640),      # one block of k
    (1025, 400, 528),
]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_product(cuda_ok, M, K, N, dtype):
    X, w = _case(M, K, N, dtype, M + K + N)
    ws = i8.Fp8Workspace(M, K, N)
    Xd = X.cuda()
    Y = i8.forward_fp8(Xd, w, workspace=ws)
    assert i8.device_status(ws)[0] == 0
    _check(Y, X, w)
    # the same call again, and after a call on other values: every bit as before
    other = i8.forward_fp8(-Xd, w, workspace=ws)
    again = i8.forward_fp8(Xd, w, workspace=ws)
    assert torch.equal(Y, again) and torch.equal(other, -Y)


@pytest.mark.parametrize("path", ["gemm", "decode"])
@pytest.mark.parametrize("M,K,N", SHAPES[:-1])
def test_product_forced_paths(cuda_ok, M, K, N, path):
    X, w = _case(M, K, N, torch.bfloat16, M + K + N + 7)
    ws = i8.Fp8Workspace(M, K, N)
    Y = i8.forward_fp8(X.cuda(), w, workspace=ws, path=path)
    assert i8.device_status(ws)[0] == 0
    _check(Y, X, w)


@pytest.mark.parametrize("M,K,N", [
    (8, 8192, 1024),      # few tiles: a cluster's blocks take pieces of one
    (16, 1040, 144),
    (3, 16384, 272),
    (24, 4112, 528),
    (31, 528, 4112),      # a tile per block
    (40, 2064, 400),
    (100, 528, 1040),
    (128, 8208, 272),
    (8, 2064, 20496),     # more tiles than SMs: runs that begin and end inside tiles
    (30, 784, 20496),
    (50, 400, 19216),
    (120, 272, 19216),
])
def test_product_however_tiles_are_shared_out(cuda_ok, M, K, N):
    X, w = _case(M, K, N, torch.bfloat16, K + N + M)
    ws = i8.Fp8Workspace(M, K, N)
    Y = i8.forward_fp8(X.cuda(), w, workspace=ws)
    assert i8.device_status(ws)[0] == 0
    _check(Y, X, w)
    assert torch.equal(i8.forward_fp8(X.cuda(), w, workspace=ws), Y)


@pytest.mark.parametrize("M", [8, 24, 60])
def test_wait_limit_in_a_cluster_reports_timeout_and_recovers(cuda_ok, M):
    K, N = 8192, 256
    X, w = _case(M, K, N, torch.float16, 31)
    Xd, ws = X.cuda(), i8.Fp8Workspace(M, K, N)
    want = i8.forward_fp8(Xd, w, workspace=ws)
    i8.forward_fp8(Xd, w, workspace=ws, wait_limit_ns=50_000_000, test_flags=1)
    assert i8.device_status(ws)[0] == 6
    ws.reset()
    assert torch.equal(i8.forward_fp8(Xd, w, workspace=ws), want)
    assert i8.device_status(ws)[0] == 0


@pytest.mark.parametrize("path,M", [("decode", 5), ("decode", 20), ("decode", 40), ("decode", 150), ("gemm", 300)])
def test_rows_that_are_not_finite_stay_alone(cuda_ok, path, M):
    K, N = 656, 272
    X, w = _case(M, K, N, torch.float16, 5)
    clean = i8.forward_fp8(X.cuda(), w, path=path)
    X[1, 300] = float("nan")
    X[M - 1, 640] = float("inf")
    X[2] = 0
    Y = i8.forward_fp8(X.cuda(), w, path=path)
    assert torch.isnan(Y[1]).all() and torch.isnan(Y[M - 1]).all()
    assert (Y[2] == 0).all()
    keep = [m for m in range(M) if m not in (1, 2, M - 1)]
    assert torch.equal(Y[keep], clean[keep])


def test_memory_around_the_output_is_left_alone(cuda_ok):
    for path, M in (("decode", 3), ("decode", 70), ("gemm", 300)):
        X, w = _case(M, 272, 400, torch.bfloat16, 11)
        big = torch.full((M + 40, 400), 7.0, dtype=torch.bfloat16, device="cuda")
        i8.forward_fp8(X.cuda(), w, out=big[8: 8 + M], path=path)
        assert (big[:8] == 7).all() and (big[8 + M:] == 7).all()
        _check(big[8: 8 + M], X, w)


def test_a_view_of_rows_and_a_checkpoint_weight(cuda_ok):
    """X as rows of a larger tensor (any row start is 32-byte aligned), codes
    and scales as parts of larger tensors."""
    X, w = _case(40, 272, 400, torch.float16, 12)
    pool = torch.zeros(3, 400, 272, device="cuda").to(torch.float8_e4m3fn)
    pool.view(torch.uint8)[1] = w.codes.view(torch.uint8)
    scales = torch.zeros(3, 4, 3, device="cuda")
    scales[1] = w.scales
    w2 = i8.weight_fp8(pool[1], scales[1])
    Y = i8.forward_fp8(X.cuda()[9:20], w2)
    _check(Y, X[9:20], w)


def test_new_weights_in_place_are_seen_by_the_next_call(cuda_ok):
    """A kernel that overwrites the weight right before a call, and after it."""
    X, w = _case(8, 4096, 2048, torch.float16, 13)
    Xd = X.cuda()
    ws = i8.Fp8Workspace(8, 4096, 2048)
    first = i8.forward_fp8(Xd, w, workspace=ws)
    flipped = (-w.codes.float()).to(torch.float8_e4m3fn)
    saved = w.codes.clone()
    torch.cuda.synchronize()
    for _ in range(20):
        w.codes.view(torch.uint8).copy_(flipped.view(torch.uint8))
        b = i8.forward_fp8(Xd, w, workspace=ws)
        w.codes.view(torch.uint8).copy_(saved.view(torch.uint8))
        a = i8.forward_fp8(Xd, w, workspace=ws)
        assert torch.equal(b, -first) and torch.equal(a, first)


@pytest.mark.parametrize("M", [3, 24, 100, 400, 1100])
def test_weights_and_rows_written_just_before_the_call(cuda_ok, M):
    """The kernels start while earlier ones end; what those wrote is read all the same."""
    K, N = 1040, 2064
    X, w = _case(M, K, N, torch.float16, 41)
    Xd, ws = X.cuda(), i8.Fp8Workspace(M, K, N)
    filler = torch.zeros(1 << 24, device="cuda")
    codes = [w.codes.view(torch.uint8).roll(k, 1).contiguous() for k in range(4)]
    rows = [Xd.roll(k, 0).contiguous() for k in range(4)]
    want = []
    for k in range(4):
        want.append(i8.forward_fp8(rows[k], i8.weight_fp8(codes[k].view(torch.float8_e4m3fn), w.scales)))
        torch.cuda.synchronize()
    got, x = [], torch.empty_like(Xd)
    for k in range(4):
        filler.add_(1)
        x.copy_(rows[k])
        w.codes.view(torch.uint8).copy_(codes[k])
        got.append(i8.forward_fp8(x, w, workspace=ws))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_the_first_call_of_a_process_may_be_captured(cuda_ok):
    """Nothing that a first call sets up (kernel attributes, occupancy) is barred while a graph is captured."""
    code = """
import torch, int8_quantized_matmul_02_b200 as i8
g = torch.Generator(device="cuda").manual_seed(1)
codes = torch.randint(0, 120, (1024, 8192), dtype=torch.uint8, device="cuda", generator=g).view(torch.float8_e4m3fn)
w = i8.weight_fp8(codes, torch.rand(8, 64, device="cuda", generator=g))
xs = [torch.randn(M, 8192, device="cuda", generator=g).half() for M in (8, 24, 50, 100, 1030)]
wss = [i8.Fp8Workspace(x.shape[0], 8192, 1024) for x in xs]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    ys = [i8.forward_fp8(x, w, workspace=s) for x, s in zip(xs, wss)]
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(y, i8.forward_fp8(x, w)) for x, y in zip(xs, ys))
print("same")
"""
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert out.returncode == 0 and out.stdout.strip() == "same", out.stderr[-2000:]


@pytest.mark.parametrize("M", [8, 40, 300])
def test_another_stream_and_a_captured_call(cuda_ok, M):
    X, w = _case(M, 1040, 528, torch.bfloat16, 21)
    Xd = X.cuda()
    want = i8.forward_fp8(Xd, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Y = i8.forward_fp8(Xd, w, stream=side)     # workspace and Y belong to `side`
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(Y, want)
    ws, ws2 = i8.Fp8Workspace(M, 1040, 528), i8.Fp8Workspace(M, 1040, 528)
    Xs, Ys = Xd.clone(), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        i8.forward_fp8(Xs, w, workspace=ws, out=Ys)
    for k in range(3):
        Xs.copy_(Xd * (k - 1))
        graph.replay()
        eager = i8.forward_fp8(Xs, w, workspace=ws2)
        torch.cuda.synchronize()
        assert torch.equal(Ys, eager)


def test_two_calls_at_once(cuda_ok):
    """Two streams, a workspace each."""
    X, w = _case(16, 4096, 4096, torch.float16, 22)
    Xd = X.cuda()
    want = i8.forward_fp8(Xd, w)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [i8.Fp8Workspace(16, 4096, 4096) for _ in streams]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for s, ws in zip(streams, spaces):
            got.append(i8.forward_fp8(Xd, w, workspace=ws, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


@pytest.mark.parametrize("path,M", [("decode", 8), ("decode", 100), ("gemm", 300)])
def test_wait_limit_reports_timeout_and_recovers(cuda_ok, path, M):
    X, w = _case(M, 1040, 528, torch.float16, 23)
    Xd = X.cuda()
    ws = i8.Fp8Workspace(M, 1040, 528)
    i8.forward_fp8(Xd, w, workspace=ws, path=path, wait_limit_ns=50_000_000, test_flags=1)
    assert i8.device_status(ws)[0] == 6
    ws.reset()
    Y = i8.forward_fp8(Xd, w, workspace=ws, path=path)
    assert i8.device_status(ws)[0] == 0
    _check(Y, X, w)


def test_large_offsets(cuda_ok):
    """A weight and an output past 2^31 bytes and elements: sampled columns."""
    M, K, N = 1040, 1024, 2 ** 21 + 272
    g = torch.Generator(device="cuda").manual_seed(3)
    codes = torch.randint(0, 120, (N, K), dtype=torch.uint8, device="cuda", generator=g).view(torch.float8_e4m3fn)
    scales = torch.rand((N + 127) // 128, K // 128, device="cuda", generator=g) * 1e-3
    w = i8.weight_fp8(codes, scales)
    X = _x(M, K, torch.float16, 31)
    cols = torch.tensor([0, 5, 2 ** 20 + 3, 2 ** 21 - 1, 2 ** 21, N - 1])
    xv = ref.row_values(*ref.quantize(_np(X)))
    q = _np(codes.view(torch.uint8)[cols.cuda()].view(torch.float8_e4m3fn).float())
    s = _np(scales[(cols // 128).cuda()])
    wv = q * np.repeat(s, 128, -1)
    for rows in (M, 8):
        Y = i8.forward_fp8(X[:rows].cuda(), w)
        y, err = ref.product(xv[:rows], wv)
        ref.check(Y[:, cols.cuda()], y, ref.out_bound(y, err, torch.float16))
        del Y
