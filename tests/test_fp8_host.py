"""Host-only checks of the block-scaled e4m3 calls: sizes, refusals before the
device is touched, the Python front's checks, and the 64-bit reference itself
(no compute call runs here)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import int8_quantized_matmul_02_b200 as i8
from int8_quantized_matmul_02_b200 import _abi
from tests import fp8_reference as ref

FAKE = 0x7F0000000000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from int8_quantized_matmul_02_b200 import build

    build.build()
    return _abi.load()


def _quant(lib, X=FAKE, dtype=0, M=4, K=256, codes=FAKE, scales=FAKE):
    return lib.int8mm_quantize_fp8(X, dtype, M, K, codes, scales, None)


def test_quantize_refusals(lib):
    assert _quant(lib, X=None) == 1
    assert _quant(lib, codes=None) == 1
    assert _quant(lib, scales=None) == 1
    assert _quant(lib, dtype=2) == 1 and _quant(lib, dtype=-1) == 1
    assert _quant(lib, M=0) == 1
    assert _quant(lib, K=0) == 1 and _quant(lib, K=250) == 1 and _quant(lib, K=131088) == 1
    assert _quant(lib, X=FAKE + 8) == 2
    assert _quant(lib, codes=FAKE + 8) == 2
    assert _quant(lib, scales=FAKE + 2) == 2


def _weight(K=256, N=384, codes=FAKE, scales=FAKE):
    return _abi.Fp8Weight(K, N, codes, scales)


def _fwd(lib, X=FAKE, dtype=0, M=8, w=None, Y=FAKE, ws=FAKE, nbytes=1 << 40, opts=None):
    w = w or _weight()
    return lib.int8mm_forward_fp8(X, dtype, M, ctypes.byref(w), Y, ws, nbytes, ctypes.byref(opts) if opts else None,
                                  None)


def test_forward_refusals(lib):
    for kw in ({"X": None}, {"Y": None}, {"ws": None}, {"dtype": 5}, {"M": 0}, {"w": _weight(K=264)},
               {"w": _weight(N=100)}, {"w": _weight(codes=None)}, {"w": _weight(scales=None)},
               {"opts": _abi.ForwardOpts(3, None, 0)}, {"opts": _abi.ForwardOpts(9, None, 0)},
               {"opts": _abi.ForwardOpts(0, FAKE, 0)},                # no int32 sums here
               {"opts": _abi.ForwardOpts(0, None, 0, FAKE, None)},    # one event without the other
               {"M": 1025, "opts": _abi.ForwardOpts(2, None, 0)}):    # too many rows to stream the weight for
        assert _fwd(lib, **kw) == 1, kw
    for kw in ({"X": FAKE + 8}, {"Y": FAKE + 8}, {"ws": FAKE + 64}, {"w": _weight(codes=FAKE + 8)},
               {"w": _weight(scales=FAKE + 2)}):
        assert _fwd(lib, **kw) == 2, kw
    for M in (1, 40, 3000):
        need = lib.int8mm_fp8_workspace_bytes(M, 256, 384)
        assert _fwd(lib, M=M, nbytes=need - 1) == 3


@pytest.mark.skipif(torch.cuda.is_available(), reason="the pointers are not memory")
@pytest.mark.parametrize("M", [1, 100, 1000, 1024, 1025])
def test_a_weight_that_fills_the_memory_is_not_refused(lib, M):
    """131072 x 1048576, 128 GB of codes: the call gets as far as the device, which is not there."""
    K, N, GB = 131072, 1 << 20, 1 << 30
    assert lib.int8mm_fp8_workspace_bytes(M, K, N) > 0
    w = _weight(K, N, codes=FAKE, scales=FAKE + 130 * GB)
    assert _fwd(lib, M=M, w=w, X=FAKE + 140 * GB, Y=FAKE + 150 * GB, ws=FAKE + 160 * GB) in (4, 5)


def test_overlapping_buffers_are_refused(lib):
    """A few rows are quantised while other blocks store results, so Y may not
    lie on X; nor may codes or scales lie on X or on one another."""
    assert _quant(lib, codes=FAKE) == 1 and _quant(lib, codes=FAKE + 2032) == 1  # X: 4 x 256 values, 2048 bytes
    assert _quant(lib, codes=FAKE + 4096, scales=FAKE + 2044) == 1
    assert _quant(lib, codes=FAKE + 4096, scales=FAKE + 4096 + 1020) == 1
    for M in (8, 40, 300):
        w = _weight(256, 256)
        assert _fwd(lib, M=M, w=w, Y=FAKE) == 1
        assert _fwd(lib, M=M, w=w, Y=FAKE + M * 512 - 16) == 1
        assert _fwd(lib, M=M, w=w, X=FAKE + M * 512 - 16) == 1


def test_prepare_refusals(lib):
    out = _abi.Fp8Weight()
    need = lib.int8mm_fp8_weight_bytes(256, 384)
    assert need >= 256 * 384 + 2 * 3 * 4
    assert lib.int8mm_fp8_weight_bytes(250, 384) == 0 and lib.int8mm_fp8_weight_bytes(256, 8) == 0

    def call(W=FAKE, dtype=1, K=256, N=384, buf=FAKE, nbytes=need):
        return lib.int8mm_prepare_weight_fp8(W, dtype, K, N, buf, nbytes, ctypes.byref(out), None)

    assert call(W=None) == 1 and call(buf=None) == 1 and call(dtype=3) == 1 and call(K=100) == 1
    assert call(W=FAKE + 2) == 2 and call(buf=FAKE + 16) == 2
    assert call(nbytes=need - 1) == 3


def _moe_weight(E=8, H=256, I=384, **kw):
    names = ("router", "gate_codes", "gate_scales", "up_codes", "up_scales", "down_codes", "down_scales")
    return _abi.MoeWeight(E, H, I, *(kw.get(n, FAKE) for n in names))


def _moe(lib, X=FAKE, dtype=0, T=4, w=None, top_k=2, Y=FAKE, ids=None, wts=None, ws=FAKE, nbytes=1 << 40, opts=None):
    w = w or _moe_weight()
    return lib.int8mm_forward_moe_fp8(X, dtype, T, ctypes.byref(w), top_k, 1, Y, ids, wts, ws, nbytes,
                                      ctypes.byref(opts) if opts else None, None)


def test_moe_refusals(lib):
    for kw in ({"X": None}, {"Y": None}, {"ws": None}, {"dtype": 2}, {"T": 0}, {"T": 65}, {"top_k": 0}, {"top_k": 9},
               {"top_k": 17, "w": _moe_weight(E=64)}, {"w": _moe_weight(E=0)}, {"w": _moe_weight(E=257)},
               {"w": _moe_weight(H=250)}, {"w": _moe_weight(I=8)}, {"w": _moe_weight(router=None)},
               {"w": _moe_weight(gate_codes=None)}, {"w": _moe_weight(up_scales=None)},
               {"w": _moe_weight(down_codes=None)}, {"opts": _abi.ForwardOpts(2, None, 0)},
               {"opts": _abi.ForwardOpts(0, None, 0, FAKE, FAKE)}):
        assert _moe(lib, **kw) == 1, kw
    for kw in ({"X": FAKE + 8}, {"Y": FAKE + 2}, {"ws": FAKE + 16}, {"w": _moe_weight(router=FAKE + 4)},
               {"w": _moe_weight(up_codes=FAKE + 8)}, {"w": _moe_weight(down_scales=FAKE + 1)}, {"ids": FAKE + 2},
               {"wts": FAKE + 1}):
        assert _moe(lib, **kw) == 2, kw
    need = lib.int8mm_moe_workspace_bytes(4, 256, 384, 8, 2)
    assert _moe(lib, nbytes=need - 1) == 3
    assert lib.int8mm_moe_workspace_bytes(65, 256, 384, 8, 2) == 0
    assert lib.int8mm_moe_workspace_bytes(4, 256, 384, 8, 9) == 0


def test_overlapping_buffers_of_the_layer_are_refused(lib):
    """Routing is stored while X is read, and what lies in topk_ids and in the
    workspace is used as an index: nothing that is written lies on anything
    else, but for Y on X.  Calls that pass get as far as the device, which is
    not there (the pointers are not memory, so where there is one this test
    makes no such call)."""
    T, E, H, I, k = 4, 8, 256, 384, 2
    MB = 1 << 20
    names = ("router", "gate_codes", "gate_scales", "up_codes", "up_scales", "down_codes", "down_scales")
    size = {"router": E * H * 2, "gate_codes": E * H * I, "up_codes": E * H * I, "down_codes": E * H * I,
            "gate_scales": E * 6 * 4, "up_scales": E * 6 * 4, "down_scales": E * 6 * 4, "X": T * H * 2, "Y": T * H * 2,
            "ids": T * k * 4, "wts": T * k * 4, "ws": lib.int8mm_moe_workspace_bytes(T, H, I, E, k)}
    apart = {n: FAKE + 64 * MB * i for i, n in enumerate(size)}
    assert max(size.values()) < 64 * MB

    def call(**moved):
        at = {**apart, **moved}
        return _moe(lib, X=at["X"], T=T, w=_moe_weight(E, H, I, **{n: at[n] for n in names}), top_k=k, Y=at["Y"],
                    ids=at["ids"], wts=at["wts"], ws=at["ws"], nbytes=size["ws"])

    for a in ("ids", "wts", "Y", "ws"):
        for b in size:
            if a == b or {a, b} == {"X", "Y"}:
                continue
            step = 256  # keeps every alignment
            assert call(**{a: apart[b]}) == 1, (a, b)
            assert call(**{a: apart[b] + (size[b] - 1) // step * step}) == 1, (a, b)
            assert call(**{a: apart[b] - (size[a] - 1) // step * step}) == 1, (a, b)
    if not torch.cuda.is_available():
        for fine in ({}, {"Y": apart["X"]}, {"Y": apart["X"] + 1024}, {"ids": None}, {"wts": None},
                     {"ids": None, "wts": None}, {"ids": apart["X"] + size["X"]}, {"wts": apart["ids"] + size["ids"]},
                     {"wts": apart["ids"] - size["wts"]}):
            assert call(**fine) in (4, 5), fine


def test_python_front_refuses(lib):
    """Tensors on the CPU, wrong types, shapes and strides: an error before any call."""
    with pytest.raises(ValueError):
        i8.quantize_fp8(torch.zeros(4, 256, dtype=torch.float16))
    with pytest.raises(ValueError):
        i8.prepare_weight_fp8(torch.zeros(256, 256, dtype=torch.float32))
    codes, scales = torch.zeros(384, 256).to(torch.float8_e4m3fn), torch.zeros(3, 2)
    with pytest.raises(ValueError):
        i8.weight_fp8(codes, scales)          # not on a GPU
    with pytest.raises(ValueError):
        i8.moe_weight_fp8(torch.zeros(8, 256, dtype=torch.float16), (codes, scales), (codes, scales), (codes, scales))
    with pytest.raises(i8.Int8mmError):
        i8.Fp8Workspace(0, 256, 384)


def test_reference_rounds_as_torch_does():
    """The reference's e4m3 rounding against torch's conversion, on every e4m3
    value, the borders between neighbours and numbers next to the borders."""
    v = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()  # 0 .. 448
    mid = (v[1:] + v[:-1]) / 2
    x = np.concatenate([v, mid, np.nextafter(mid.astype(np.float32), np.float32(0)).astype(np.float64),
                        np.nextafter(mid.astype(np.float32), np.float32(1e9)).astype(np.float64)])
    x = np.concatenate([x, -x])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3_round(x)[0], want)


def test_reference_layer_without_quantisation_error():
    """Small integers quantise without error in blocks whose maximum is 448:
    the reference product is then the exact integer product."""
    g = np.random.default_rng(1)
    X = g.integers(-8, 9, (3, 256)).astype(float)
    W = g.integers(-8, 9, (256, 128)).astype(float)
    X[:, ::128] = 448
    W[::128, 0] = 448
    q, s = ref.quantize(X)
    wq, ws = ref.quantize_weight(W)
    assert np.all(s == 1) and np.all(ws == 1)
    y, _ = ref.product(ref.row_values(q, s), ref.weight_values(wq, ws))
    assert np.array_equal(y, X @ W)


def test_reference_routing():
    X = np.array([[1.0, 0.0], [0.0, 0.0]])
    R = np.array([[1.0, 0], [3.0, 0], [3.0, 1], [2.0, 5]])
    ids, p = ref.route(X, R, 2, True)
    assert ids.tolist() == [[1, 2], [0, 1]]
    assert np.allclose(p, 0.5)
    _, p = ref.route(X, R, 4, False)
    assert np.allclose(p.sum(1), 1.0) and np.allclose(p[1], 0.25)
