"""GPU tests of the ways in which the weight-streaming e4m3 kernel shares out
its tiles: each case names the way that it is there for, and is checked to
take it, against the 64-bit reference (tests/fp8_reference.py)."""
from __future__ import annotations

import pytest
import torch

import int8_quantized_matmul_02_b200 as i8
from tests import fp8_reference as ref
from tests.launches import launches, the
from tests.test_gpu_fp8 import _case as product_case, _check as check_product
from tests.test_gpu_moe import _case as layer_case, _check as check_layer, _want as want_layer

pytestmark = pytest.mark.gpu

ROWS, DOWN = "k_fp8_rowsILi0E", "k_fp8_rowsILi2E"  # the kernel as plain and as down product


def _way(launch, tiles: int) -> str:
    """How `tiles` tiles are shared out on the blocks of a launch."""
    if launch.cluster > 1:
        assert launch.grid == launch.cluster * tiles
        return "clusters"
    return "whole" if launch.grid == tiles else "runs"


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M,K,N,path,way", [
    # several blocks of 128 rows; tiles begin and end inside a share and are joined through memory
    (256, 8192, 5120, "auto", "runs"),
    (1000, 8192, 1280, "auto", "runs"),         # the last of 8 row blocks has 104 rows
    (250, 8208, 5136, "auto", "runs"),          # K, N and M end inside a tile
    (140, 400, 9616, "decode", "runs"),         # more tiles than SMs
    (1024, 144, 2576, "decode", "runs"),
    (129, 272, 4112, "auto", "whole"),
    (300, 4112, 272, "auto", "clusters"),
    (8, 8192, 1024, "auto", "clusters"),
    (24, 4112, 528, "auto", "clusters"),
    (31, 528, 4112, "auto", "whole"),
    (8, 2064, 20496, "auto", "runs"),
])
def test_product(cuda_ok, M, K, N, path, way, dtype):
    X, w = product_case(M, K, N, dtype, K + N + M + 1)
    ws, Xd = i8.Fp8Workspace(M, K, N), X.cuda()
    rows = 16 if M <= 16 else 32 if M <= 32 else 64 if M <= 64 else 128
    found = launches(lambda: i8.forward_fp8(Xd, w, workspace=ws, path=path))
    assert _way(the(found, ROWS), -(-N // 128) * -(-M // rows)) == way
    Y = i8.forward_fp8(Xd, w, workspace=ws, path=path)
    assert i8.device_status(ws)[0] == 0
    check_product(Y, X, w)
    other = i8.forward_fp8(-Xd, w, workspace=ws, path=path)
    assert torch.equal(i8.forward_fp8(Xd, w, workspace=ws, path=path), Y) and torch.equal(other, -Y)


LAYERS = [
    (3, 8, 2, 8192, 272, "clusters"),           # of two blocks
    (20, 8, 2, 8208, 272, "clusters"),
    (50, 8, 2, 1040, 272, "clusters"),
    # of four blocks and more, where the GPU runs enough of them at once (its SMs are not
    # the same in every part of it); else runs
    (1, 8, 2, 4096, 528, "clusters or runs"),
    (5, 8, 3, 2576, 656, "clusters or runs"),
    (24, 8, 2, 4096, 528, "clusters or runs"),
    (32, 16, 4, 4112, 144, "clusters or runs"),
    # (too few units for pieces that keep four in five SMs busy)
    (5, 8, 3, 2064, 272, "runs"),
    (24, 8, 2, 4096, 272, "runs"),
    (2, 8, 2, 528, 1040, "runs"),
    (20, 8, 2, 528, 1040, "runs"),
]


@pytest.mark.parametrize("dtype,renorm", [(torch.float16, False), (torch.bfloat16, True)])
@pytest.mark.parametrize("T,E,top_k,H,I,way", LAYERS)
def test_layer(cuda_ok, T, E, top_k, H, I, way, dtype, renorm):  # noqa: E741
    X, w = layer_case(T, E, H, I, dtype, T + E + H + I + 1)
    ws, Xd = i8.MoeWorkspace(T, w, top_k), X.cuda()
    call = lambda **kw: i8.forward_moe_fp8(Xd, w, top_k, renormalize=renorm, workspace=ws, **kw)  # noqa: E731
    assert _way(the(launches(call), DOWN), -(-H // 128)) in way
    got = call(return_routing=True)
    assert i8.device_status(ws)[0] == 0
    check_layer(got, X, w, top_k, renorm)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y = call()
    for _ in range(3):
        Y.zero_()
        graph.replay()
        assert torch.equal(Y, got[0])
    assert torch.equal(call(), got[0])


@pytest.mark.parametrize("which", ["up", "down", "down scales"])
@pytest.mark.parametrize("T", [4, 20])
def test_weights_that_are_not_finite_stay_with_their_tokens_in_a_cluster(cuda_ok, T, which):
    E, H, I = 8, 8192, 272  # noqa: E741
    X, w = layer_case(T, E, H, I, torch.bfloat16, 14)
    X[:, 0], w.router[:, 0] = 0, 0
    X[0, 0], w.router[5, 0] = 64, 64      # the first token chooses expert 5
    Xd = X.cuda()
    assert _way(the(launches(lambda: i8.forward_moe_fp8(Xd, w, 2)), DOWN), 64) == "clusters"
    clean, ids, _ = i8.forward_moe_fp8(Xd, w, 2, return_routing=True)
    chose = (ids == 5).any(1)
    assert chose[0] and not chose.all()
    if which == "down scales":
        w.down[1][5] = float("-inf")
    else:
        (w.up if which == "up" else w.down)[0].view(torch.uint8)[5, ::3] = 0xFF      # a NaN code
    Y = i8.forward_moe_fp8(Xd, w, 2)
    assert torch.equal(Y[~chose], clean[~chose])
    assert not torch.isfinite(Y[chose]).all(1).any()


@pytest.mark.parametrize("T", [4, 20])
def test_tokens_that_are_not_finite_stay_alone_in_a_cluster(cuda_ok, T):
    X, w = layer_case(T, 8, 8192, 272, torch.float16, 15)
    X[1, 70] = float("nan")
    X[T - 1, 8191] = float("-inf")
    Xd = X.cuda()
    assert _way(the(launches(lambda: i8.forward_moe_fp8(Xd, w, 2)), DOWN), 64) == "clusters"
    Y = i8.forward_moe_fp8(Xd, w, 2)
    assert torch.isnan(Y[1]).all() and torch.isnan(Y[T - 1]).all()
    keep = [t for t in range(T) if t not in (1, T - 1)]
    y, err, _, _ = want_layer(X[keep], w, 2, True)
    ref.check(Y[keep], y, ref.out_bound(y, err, torch.float16))


@pytest.mark.parametrize("T", [3, 20])
def test_wait_limit_before_a_clustered_down_product(cuda_ok, T):
    X, w = layer_case(T, 8, 8192, 272, torch.float16, 16)
    ws, Xd = i8.MoeWorkspace(T, w, 2), X.cuda()
    assert _way(the(launches(lambda: i8.forward_moe_fp8(Xd, w, 2, workspace=ws)), DOWN), 64) == "clusters"
    want = i8.forward_moe_fp8(Xd, w, 2, workspace=ws)
    i8.forward_moe_fp8(Xd, w, 2, workspace=ws, wait_limit_ns=50_000_000, test_flags=1)
    assert i8.device_status(ws)[0] == 6
    ws.reset()
    assert torch.equal(i8.forward_moe_fp8(Xd, w, 2, workspace=ws), want)
    assert i8.device_status(ws)[0] == 0
