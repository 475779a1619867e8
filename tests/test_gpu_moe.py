"""GPU tests of the mixture-of-experts layer against the 64-bit reference
(tests/fp8_reference.py, where the tolerances are derived): the chosen experts
exactly, weights and Y within their bounds."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import int8_quantized_matmul_02_b200 as i8
from tests import fp8_reference as ref

pytestmark = pytest.mark.gpu


def _np(t):
    return t.double().cpu().numpy()


def _case(T, E, H, I, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(T, H, generator=g)
    X[:, torch.randperm(H, generator=g)[:2]] *= 20
    R = (torch.randn(E, H, generator=g) / H ** 0.5).to(dtype)
    gate, up = ((torch.randn(E, H, I, generator=g) / H ** 0.5).to(dtype) for _ in range(2))
    down = (torch.randn(E, I, H, generator=g) / I ** 0.5).to(dtype)
    w = i8.prepare_moe_weight_fp8(R.cuda(), gate.cuda(), up.cuda(), down.cuda())
    return X.to(dtype), w


def _values(pair):
    return ref.weight_values(_np(pair[0].float()), _np(pair[1]))


def _want(X, w, top_k, renorm):
    return ref.moe(_np(X), _np(w.router), _values(w.gate), _values(w.up), _values(w.down), top_k, renorm)


def _check(got, X, w, top_k, renorm):
    Y, ids, wts = got
    y, err, ref_ids, ref_w = _want(X, w, top_k, renorm)
    assert np.array_equal(ids.cpu().numpy(), ref_ids)
    # exp, the sum over at most 256 experts and a division, each within 2 steps
    assert np.all(np.abs(_np(wts) - ref_w) <= (2 * 4 + 256) * ref.U * ref_w)
    ref.check(Y, y, ref.out_bound(y, err, X.dtype))


@pytest.mark.parametrize("dtype,renorm", [(torch.float16, True), (torch.bfloat16, False)])
@pytest.mark.parametrize("T,E,top_k,H,I", [
    (1, 1, 1, 16, 16),         # the smallest layer
    (1, 8, 2, 256, 384),
    (1, 256, 16, 144, 128),    # the most experts, the most choices
    (4, 8, 8, 272, 144),       # every expert for every token; sizes that end inside a block
    (5, 64, 6, 512, 272),
    (16, 16, 2, 1040, 528),
    (17, 5, 3, 256, 640),      # 32 columns
    (33, 33, 4, 128, 128),     # 64 columns, an expert in a second group of 32
    (64, 12, 4, 400, 400),
    # more than three whole tiles per block, so that its slots of sums are used again
    (2, 256, 16, 128, 2064),
    (24, 64, 8, 144, 1040),
    (50, 80, 3, 128, 1040),
])
def test_layer(cuda_ok, T, E, top_k, H, I, dtype, renorm):
    X, w = _case(T, E, H, I, dtype, T + E + H + I)
    ws = i8.MoeWorkspace(T, w, top_k)
    Xd = X.cuda()
    got = i8.forward_moe_fp8(Xd, w, top_k, renormalize=renorm, workspace=ws, return_routing=True)
    assert i8.device_status(ws)[0] == 0
    _check(got, X, w, top_k, renorm)
    # after other tokens through the same workspace, every bit as before; without the routing too
    i8.forward_moe_fp8(Xd.flip(0).contiguous() * 3, w, top_k, renormalize=renorm, workspace=ws)
    assert torch.equal(i8.forward_moe_fp8(Xd, w, top_k, renormalize=renorm, workspace=ws), got[0])


def test_equal_scores_take_the_lower_expert(cuda_ok):
    X, w = _case(6, 40, 256, 128, torch.bfloat16, 2)
    w.router[20:] = w.router[:20]         # experts e and e + 20 score the same
    w.router[7] = w.router[3]
    X[5] = 0                              # every score zero: experts 0, 1, 2, 3
    got = i8.forward_moe_fp8(X.cuda(), w, 4, return_routing=True)
    _check(got, X, w, 4, True)
    assert got[1][5].tolist() == [0, 1, 2, 3]


def test_all_tokens_on_one_expert(cuda_ok):
    X, w = _case(64, 9, 256, 256, torch.float16, 3)
    X[:] = X[:1]
    got = i8.forward_moe_fp8(X.cuda(), w, 1, return_routing=True)
    _check(got, X, w, 1, True)
    assert (got[0] == got[0][:1]).all()


@pytest.mark.parametrize("T", [4, 20, 50])
def test_tokens_that_are_not_finite_stay_alone(cuda_ok, T):
    X, w = _case(T, 8, 272, 256, torch.bfloat16, 4)
    clean, ids, _ = i8.forward_moe_fp8(X.cuda(), w, 2, return_routing=True)
    X[1, 70] = float("nan")
    X[T - 1, 271] = float("inf")
    Y, ids2, _ = i8.forward_moe_fp8(X.cuda(), w, 2, return_routing=True)
    assert torch.isnan(Y[1]).all() and torch.isnan(Y[T - 1]).all()
    keep = [t for t in range(T) if t not in (1, T - 1)]
    assert torch.equal(ids2[keep], ids[keep])
    assert ((ids2 >= 0) & (ids2 < 8)).all()
    y, err, _, _ = _want(X[keep], w, 2, True)
    ref.check(Y[keep], y, ref.out_bound(y, err, torch.bfloat16))


@pytest.mark.parametrize("which", ["gate", "down", "down scales"])
@pytest.mark.parametrize("T", [4, 20, 50])
def test_weights_that_are_not_finite_reach_their_own_tokens_only(cuda_ok, T, which):
    X, w = _case(T, 8, 272, 256, torch.bfloat16, 10)
    X[:, 0], w.router[:, 0] = 0, 0
    X[0, 0], w.router[5, 0] = 64, 64      # the first token chooses expert 5
    clean, ids, _ = i8.forward_moe_fp8(X.cuda(), w, 2, return_routing=True)
    chose = (ids == 5).any(1)
    assert chose[0] and not chose.all()
    if which == "down scales":
        w.down[1][5] = float("inf")
    else:
        codes = (w.gate if which == "gate" else w.down)[0]
        codes.view(torch.uint8)[5, ::3] = 0x7F      # the NaN code
    Y = i8.forward_moe_fp8(X.cuda(), w, 2)
    assert torch.equal(Y[~chose], clean[~chose])
    assert not torch.isfinite(Y[chose]).all(1).any()


@pytest.mark.parametrize("T", [3, 20, 50])
def test_a_down_scale_of_any_value_counts(cuda_ok, T):
    """The lowest fp32 number as an expert's down scale, next to a scale of h of
    exactly one: its tokens get that multiple of their sums, the other expert's
    tokens theirs.  Every step is exact: g = 64 (silu(64) = 64 in fp32), u = 7,
    h = 448 with scale 1, the sum 448 * 2^-9 = 0.875, and bf16 holds 0.875 and
    0.875 * 2^128; -0.875 * FLT_MAX rounds to the latter's negative."""
    H = I = 128
    one = {v: int(torch.tensor(float(v)).to(torch.float8_e4m3fn).view(torch.uint8)) for v in (64, 7, 2.0 ** -9)}
    gate, up, down = (torch.zeros(2, 128, 128, dtype=torch.uint8, device="cuda") for _ in range(3))
    gate[:, 0, 1], up[:, 0, 1], down[:, :, 0] = one[64], one[7], one[2.0 ** -9]
    scales = [torch.ones(2, 1, 1, device="cuda") for _ in range(3)]
    scales[2][0] = torch.finfo(torch.float32).min
    router = torch.zeros(2, H, dtype=torch.bfloat16, device="cuda")
    router[0, 2], router[1, 2] = 8, -8
    w = i8.moe_weight_fp8(router, *((c.view(torch.float8_e4m3fn), s) for c, s in zip((gate, up, down), scales)))
    X = torch.zeros(T, H, dtype=torch.bfloat16)
    X[:, 0], X[:, 1] = 448, 1                 # the block's scale is 1; the gate and up weights read column 1
    X[:, 2] = 1
    X[1::2, 2] = -1                           # every other token chooses expert 1
    Y, ids, wts = i8.forward_moe_fp8(X.cuda(), w, 1, return_routing=True)
    assert ids.flatten().tolist() == [t % 2 for t in range(T)] and (wts == 1).all()
    assert (Y[1::2].double() == 0.875).all()
    assert (Y[::2].double() == -0.875 * 2.0 ** 128).all()


def test_output_in_place_of_the_tokens(cuda_ok):
    X, w = _case(7, 8, 272, 256, torch.float16, 11)
    Xd = X.cuda()
    want = i8.forward_moe_fp8(Xd, w, 3)
    assert torch.equal(i8.forward_moe_fp8(Xd, w, 3, out=Xd), want)


def test_another_stream_and_a_captured_call(cuda_ok):
    X, w = _case(12, 16, 528, 272, torch.float16, 5)
    Xd = X.cuda()
    want = i8.forward_moe_fp8(Xd, w, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Y = i8.forward_moe_fp8(Xd, w, 4, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(Y, want)
    ws, ws2 = i8.MoeWorkspace(12, w, 4), i8.MoeWorkspace(12, w, 4)
    Xs, Ys = Xd.clone(), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        i8.forward_moe_fp8(Xs, w, 4, workspace=ws, out=Ys)
    for k in range(3):
        Xs.copy_(Xd.roll(k, 0) * (k + 1))
        graph.replay()
        eager = i8.forward_moe_fp8(Xs, w, 4, workspace=ws2)
        torch.cuda.synchronize()
        assert torch.equal(Ys, eager)


@pytest.mark.parametrize("T", [2, 20, 60])
def test_weights_and_tokens_written_just_before_the_call(cuda_ok, T):
    """The kernels start while earlier ones end; what those wrote is read all the same."""
    X, w = _case(T, 8, 528, 272, torch.float16, 12)
    Xd, ws = X.cuda(), i8.MoeWorkspace(T, w, 3)
    filler = torch.zeros(1 << 24, device="cuda")
    parts = [w.router, *(p.view(torch.uint8) for p, _ in (w.gate, w.up, w.down)), Xd]
    kept = [[p.roll(k, 0).contiguous() for p in parts] for k in range(4)]

    def write(k):
        for p, v in zip(parts, kept[k]):
            p.copy_(v)

    want, got = [], []
    for k in range(4):
        write(k)
        torch.cuda.synchronize()
        want.append(i8.forward_moe_fp8(Xd, w, 3))
        torch.cuda.synchronize()
    for k in range(4):
        filler.add_(1)
        write(k)
        got.append(i8.forward_moe_fp8(Xd, w, 3, workspace=ws))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_calls_at_once(cuda_ok):
    X, w = _case(16, 16, 512, 512, torch.bfloat16, 6)
    Xd = X.cuda()
    want = i8.forward_moe_fp8(Xd, w, 2)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [i8.MoeWorkspace(16, w, 2) for _ in streams]
    torch.cuda.synchronize()
    got = [i8.forward_moe_fp8(Xd, w, 2, workspace=ws, stream=s)
           for _ in range(20) for s, ws in zip(streams, spaces)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_wait_limit_reports_timeout_and_recovers(cuda_ok):
    X, w = _case(3, 8, 256, 256, torch.float16, 7)
    Xd = X.cuda()
    ws = i8.MoeWorkspace(3, w, 2)
    want = i8.forward_moe_fp8(Xd, w, 2, workspace=ws)
    i8.forward_moe_fp8(Xd, w, 2, workspace=ws, wait_limit_ns=50_000_000, test_flags=1)
    assert i8.device_status(ws)[0] == 6
    ws.reset()
    assert torch.equal(i8.forward_moe_fp8(Xd, w, 2, workspace=ws), want)
    assert i8.device_status(ws)[0] == 0


def test_layers_in_a_row(cuda_ok):
    """A decode step of two layers as a model runs them: a block-scaled
    projection, the mixture-of-experts layer, a projection back; one stream,
    workspaces kept, no synchronisation in between, against the same steps
    taken one at a time."""
    T, H, E = 8, 512, 16
    g = torch.Generator().manual_seed(8)
    proj = [i8.prepare_weight_fp8((torch.randn(H, H, generator=g) / H ** 0.5).bfloat16().cuda()) for _ in range(2)]
    layers = [_case(T, E, H, 256, torch.bfloat16, 9 + k)[1] for k in range(2)]
    x0 = torch.randn(T, H, generator=g).bfloat16().cuda()
    pws, mws = i8.Fp8Workspace(T, H, H), i8.MoeWorkspace(T, layers[0], 4)
    x = x0
    for w, layer in zip(proj, layers):
        x = i8.forward_moe_fp8(i8.forward_fp8(x, w, workspace=pws), layer, 4, workspace=mws)
    z = x0
    for w, layer in zip(proj, layers):
        a = i8.forward_fp8(z, w)
        torch.cuda.synchronize()
        y, err = ref.product(ref.row_values(*ref.quantize(_np(z))), ref.weight_values(_np(w.codes.float()), _np(w.scales)))
        ref.check(a, y, ref.out_bound(y, err, torch.bfloat16))
        z, ids, wts = i8.forward_moe_fp8(a, layer, 4, return_routing=True)
        torch.cuda.synchronize()
        _check((z, ids, wts), a, layer, 4, True)
    assert torch.equal(x, z)
