"""GPU tests of the block-scaled e4m3 calls on tensors of more than 2^31
elements (the product's are in test_gpu_fp8.py): sampled rows, and the experts
that were chosen, against the 64-bit reference."""
from __future__ import annotations

import pytest
import torch

import int8_quantized_matmul_02_b200 as i8
from tests import fp8_reference as ref
from tests.test_gpu_fp8 import _np, _same_codes

pytestmark = pytest.mark.gpu


def test_quantise_past_2_31_values(cuda_ok):
    M, K = 2 ** 21 + 5, 1040
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(4096, K, device="cuda", generator=g).bfloat16().repeat(M // 4096 + 1, 1)[:M]
    rows = torch.tensor([0, 7, 2 ** 20, 2 ** 31 // K - 1, 2 ** 31 // K, 2 ** 31 // K + 1, M - 1], device="cuda")
    X[rows] *= torch.arange(1, 8, device="cuda")[:, None]      # rows like no others
    codes, scales = i8.quantize_fp8(X)
    q, s = ref.quantize(_np(X[rows]))
    assert (_np(scales[rows]) == s).all() and _same_codes(codes.view(torch.uint8)[rows].view(codes.dtype), q)


class _Experts:
    """Dequantised weights of one expert at a time."""

    def __init__(self, codes, scales):
        self.codes, self.scales = codes, scales

    def __getitem__(self, e):
        e = int(e)
        return ref.weight_values(_np(self.codes[e].float()), _np(self.scales[e]))


def test_layer_with_weights_past_2_31_bytes(cuda_ok):
    T, E, H, I, k = 3, 128, 8208, 2064, 2  # noqa: E741
    assert E * H * I > 2 ** 31 and (E - 2) * H * I < 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(2)

    def weight(n, m):
        codes = torch.randint(0, 120, (E, n, m), dtype=torch.uint8, device="cuda", generator=g)
        codes |= torch.randint(0, 2, (E, n, m), dtype=torch.uint8, device="cuda", generator=g) << 7
        scales = 2e-2 / m ** 0.5 * (1 + torch.rand(E, (n + 127) // 128, (m + 127) // 128, device="cuda", generator=g))
        return codes.view(torch.float8_e4m3fn), scales

    router = (torch.randn(E, H, device="cuda", generator=g) / H ** 0.5).bfloat16()
    X = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    X[:, 0], router[:, 0] = 8, 0
    router[E - 3:, 0] = 4                                       # every token chooses two of the last three experts
    w = i8.moe_weight_fp8(router, weight(I, H), weight(I, H), weight(H, I))
    Y, ids, wts = i8.forward_moe_fp8(X, w, k, return_routing=True)
    y, err, want_ids, _ = ref.moe(_np(X), _np(router), _Experts(*w.gate), _Experts(*w.up), _Experts(*w.down), k, True)
    assert (ids >= E - 3).all() and (ids.cpu().numpy() == want_ids).all() and (ids == E - 1).any()
    ref.check(Y, y, ref.out_bound(y, err, torch.bfloat16))
