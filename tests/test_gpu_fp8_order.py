"""GPU tests of the order of kernels that let the next one start before they
end: the kernel ahead of a call is one of the library's own that does so and is
still writing the call's weights, or its rows, when the call's first blocks may
start.  No synchronisation in between; every result bit for bit that of the
same steps taken one at a time."""
from __future__ import annotations

import pytest
import torch

import int8_quantized_matmul_02_b200 as i8

pytestmark = pytest.mark.gpu
ROUNDS = 12


def _alternate(write, call, out_of=lambda y: y):
    """call() after write(0) and write(1) in turn, against synchronised results."""
    want = []
    for k in range(2):
        write(k)
        torch.cuda.synchronize()
        want.append(out_of(call()).clone())
        torch.cuda.synchronize()
    assert not torch.equal(*want)
    write(1)
    call()
    got = []
    for r in range(ROUNDS):
        write(r & 1)
        got.append(out_of(call()))
    torch.cuda.synchronize()
    assert [torch.equal(y, want[r & 1]) for r, y in enumerate(got)] == [True] * ROUNDS


def _writer(rows, cols, g):
    """(codes rows x cols, write): write(k) fills the codes with set k by the
    quantiser, whose blocks come to the last rows last and all at once."""
    src = [torch.randn(rows, cols, device="cuda", generator=g).half() for _ in range(2)]
    codes = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(rows, (cols + 127) // 128, device="cuda")
    return codes, lambda k: i8.quantize_fp8(src[k], codes=codes, scales=scales)


def _busy_writer(g):
    """(1228800 codes, write): write(k) fills them with set k by a product of 38
    tiles on as many pairs of SMs, so that what comes next finds room at once.
    Its rows have a single one each, and its outputs are the integers -7 .. 7,
    whose fp16 halves are e4m3 codes that are finite (a zero and 0x3C to 0x47,
    with either sign)."""
    M, K, N = 64, 8192, 9600
    v = torch.randint(-7, 8, (N, K), device="cuda", generator=g)
    w = i8.weight_fp8(v.float().to(torch.float8_e4m3fn), torch.ones(N // 128, K // 128, device="cuda"))
    src = torch.zeros(2, M, K, device="cuda").half()
    for k in range(2):
        src[k, torch.arange(M), torch.randint(0, K, (M,), device="cuda", generator=g)] = 1
    Y, ws = torch.empty(M, N, device="cuda").half(), i8.Fp8Workspace(M, K, N)
    return Y.view(-1).view(torch.float8_e4m3fn), lambda k: i8.forward_fp8(src[k], w, out=Y, workspace=ws, path="gemm")


@pytest.mark.parametrize("M", [3, 16, 24, 40, 100, 400, 1100])
def test_product_beside_the_kernel_that_writes_its_weight(cuda_ok, M):
    K, N = 1200, 1024
    g = torch.Generator(device="cuda").manual_seed(6)
    codes, write = _busy_writer(g)
    w = i8.weight_fp8(codes.view(N, K), torch.full((N // 128, 10), 1e-2, device="cuda"))
    X, ws = torch.randn(M, K, device="cuda", generator=g).half(), i8.Fp8Workspace(M, K, N)
    _alternate(write, lambda: i8.forward_fp8(X, w, workspace=ws))


@pytest.mark.parametrize("T", [1, 12, 24, 50])
def test_layer_beside_the_kernel_that_writes_its_weights(cuda_ok, T):
    E, H, I = 4, 320, 320  # noqa: E741
    g = torch.Generator(device="cuda").manual_seed(7)
    codes, write = _busy_writer(g)
    pairs = [(c, torch.full((E, 3, 3), 1e-2, device="cuda")) for c in codes.view(3, E, I, H)]
    w = i8.moe_weight_fp8(torch.randn(E, H, device="cuda", generator=g).half(), *pairs)
    X, ws = torch.randn(T, H, device="cuda", generator=g).half(), i8.MoeWorkspace(T, w, 2)
    _alternate(write, lambda: i8.forward_moe_fp8(X, w, 2, workspace=ws))


@pytest.mark.parametrize("M", [3, 16, 24, 40, 100, 400, 1100])
def test_product_behind_the_kernel_that_writes_its_weight(cuda_ok, M):
    K, N = 4096, 2064
    g = torch.Generator(device="cuda").manual_seed(1)
    codes, write = _writer(8192, K, g)
    w = i8.weight_fp8(codes[-N:], torch.rand(-(-N // 128), K // 128, device="cuda", generator=g) * 1e-3)
    X, ws = torch.randn(M, K, device="cuda", generator=g).half(), i8.Fp8Workspace(M, K, N)
    _alternate(write, lambda: i8.forward_fp8(X, w, workspace=ws))


@pytest.mark.parametrize("T", [1, 12, 24, 50])
def test_layer_behind_the_kernel_that_writes_its_weights(cuda_ok, T):
    E, H, I = 8, 1024, 512  # noqa: E741
    g = torch.Generator(device="cuda").manual_seed(2)
    codes, write = _writer(48 * 1024, H, g)
    n = E * I
    pair = lambda c, a, b: (c.view(E, a, b), torch.full((E, a // 128, b // 128), 1e-3, device="cuda"))  # noqa: E731
    router = torch.randn(E, H, device="cuda", generator=g).half()
    w = i8.moe_weight_fp8(router, pair(codes[-3 * n: -2 * n], I, H), pair(codes[-2 * n: -n], I, H), pair(codes[-n:], H, I))
    X, ws = torch.randn(T, H, device="cuda", generator=g).half(), i8.MoeWorkspace(T, w, 2)
    _alternate(write, lambda: i8.forward_moe_fp8(X, w, 2, workspace=ws))


def _rows_writer(M, N, g):
    """(X M x N, write): write(k) makes X by a product that leaves SMs idle near its end."""
    K = 8192
    codes = torch.randint(0, 120, (N, K), dtype=torch.uint8, device="cuda", generator=g)
    codes ^= torch.randint(0, 2, (N, K), dtype=torch.uint8, device="cuda", generator=g) << 7
    w = i8.weight_fp8(codes.view(torch.float8_e4m3fn), torch.full((-(-N // 128), K // 128), 1e-4, device="cuda"))
    src = [torch.randn(M, K, device="cuda", generator=g).half() for _ in range(2)]
    X, ws = torch.empty(M, N, device="cuda").half(), i8.Fp8Workspace(M, K, N)
    return X, lambda k: i8.forward_fp8(src[k], w, out=X, workspace=ws)


@pytest.mark.parametrize("M", [3, 16, 24, 40, 100, 400, 1100])
def test_product_behind_the_kernel_that_writes_its_rows(cuda_ok, M):
    g = torch.Generator(device="cuda").manual_seed(3)
    X, write = _rows_writer(M, 9600, g)
    w = i8.weight_fp8(torch.randint(0, 120, (2064, 9600), dtype=torch.uint8, device="cuda", generator=g)
                      .view(torch.float8_e4m3fn), torch.full((17, 75), 1e-5, device="cuda"))
    ws = i8.Fp8Workspace(M, 9600, 2064)
    _alternate(write, lambda: i8.forward_fp8(X, w, workspace=ws))


@pytest.mark.parametrize("M", [3, 40, 400, 1100])
def test_quantiser_behind_the_kernel_that_writes_its_rows(cuda_ok, M):
    g = torch.Generator(device="cuda").manual_seed(4)
    X, write = _rows_writer(M, 9600, g)
    _alternate(write, lambda: i8.quantize_fp8(X), lambda y: y[0].view(torch.uint8))


@pytest.mark.parametrize("T", [1, 12, 24, 50])
def test_layer_behind_the_kernel_that_writes_its_tokens(cuda_ok, T):
    E, H, I = 8, 9600, 256  # noqa: E741
    g = torch.Generator(device="cuda").manual_seed(5)
    X, write = _rows_writer(T, H, g)
    pair = lambda a, b: (torch.randint(0, 120, (E, a, b), dtype=torch.uint8, device="cuda", generator=g)  # noqa: E731
                         .view(torch.float8_e4m3fn), torch.full((E, a // 128, b // 128), 1e-4, device="cuda"))
    w = i8.moe_weight_fp8(torch.randn(E, H, device="cuda", generator=g).half(), pair(I, H), pair(I, H), pair(H, I))
    ws = i8.MoeWorkspace(T, w, 2)
    _alternate(write, lambda: i8.forward_moe_fp8(X, w, 2, workspace=ws))
