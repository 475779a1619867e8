"""GPU tests of the block-scaled e4m3 calls on another stream than their tensors'."""
from __future__ import annotations

import pytest
import torch

import int8_quantized_matmul_02_b200 as i8

pytestmark = pytest.mark.gpu


def _codes(*shape, g):
    return torch.randint(0, 120, shape, dtype=torch.uint8, device="cuda", generator=g).view(torch.float8_e4m3fn)


def _quantize(g):
    X = torch.randn(64, 4096, device="cuda", generator=g).half()
    return lambda s: i8.quantize_fp8(X, stream=s)[0].view(torch.uint8)


def _prepare(g):
    W = torch.randn(4096, 512, device="cuda", generator=g).half()
    return lambda s: i8.prepare_weight_fp8(W, stream=s).codes.view(torch.uint8)


def _product(g):
    X = torch.randn(40, 4096, device="cuda", generator=g).half()
    w = i8.weight_fp8(_codes(1024, 4096, g=g), torch.rand(8, 32, device="cuda", generator=g) * 1e-3)
    return lambda s: i8.forward_fp8(X, w, stream=s)


def _moe_weight(E, H, I, g):  # noqa: E741
    pair = lambda n, k: (_codes(E, n, k, g=g), torch.rand(E, n // 128, k // 128, device="cuda", generator=g) * 1e-3)  # noqa: E731
    return i8.moe_weight_fp8(torch.randn(E, H, device="cuda", generator=g).half(), pair(I, H), pair(I, H), pair(H, I))


def _layer(g):
    X = torch.randn(24, 512, device="cuda", generator=g).half()
    w = _moe_weight(4, 512, 256, g)
    return lambda s: i8.forward_moe_fp8(X, w, 2, stream=s)


@pytest.mark.parametrize("make", [_quantize, _prepare, _product, _layer])
def test_inputs_dropped_while_the_other_stream_has_yet_to_run(cuda_ok, make):
    """The caller drops the inputs and weights that it gave to a call on a stream
    that is still busy, and allocates and writes on its own stream meanwhile.
    (Inputs and weights only: they are values to the kernels, and whatever lies
    in their memory gives wrong numbers at most.)"""
    call = make(torch.Generator(device="cuda").manual_seed(5))  # the call alone holds them
    want = call(None).clone()
    torch.full((1,), 0x11, dtype=torch.uint8, device="cuda")    # (its kernel is loaded now)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)       # about a fifth of a second
    got = call(side)
    del call
    # the sizes of the tensors above
    junk = [torch.full((n,), 0x11, dtype=torch.uint8, device="cuda")
            for n in [64 * 4096 * 2, 4096 * 512 * 2, 40 * 4096 * 2, 1024 * 4096, 24 * 512 * 2, 4 * 512 * 256] * 4
            + [1 << s for s in range(9, 23)] * 8]
    torch.cuda.current_stream().synchronize()
    assert not side.query()                  # it had yet to run
    side.synchronize()
    assert torch.equal(got, want)
    del junk


def test_everything_that_a_call_takes_is_recorded_on_its_stream(cuda_ok, monkeypatch):
    g = torch.Generator(device="cuda").manual_seed(6)
    side = torch.cuda.Stream()
    X, W = torch.randn(24, 512, device="cuda", generator=g).half(), torch.randn(512, 256, device="cuda", generator=g).half()
    codes, scales = torch.empty_like(X, dtype=torch.float8_e4m3fn), torch.empty(24, 4, device="cuda")
    w, m = i8.prepare_weight_fp8(W), _moe_weight(4, 512, 256, g)
    Y, Z = torch.empty(24, 256, device="cuda").half(), torch.empty_like(X)
    ws, mws = i8.Fp8Workspace(24, 512, 256), i8.MoeWorkspace(24, m, 2)
    torch.cuda.synchronize()
    seen, record = [], torch.Tensor.record_stream

    def spy(t, stream):
        seen.append((t.untyped_storage().data_ptr(), stream))
        record(t, stream)

    monkeypatch.setattr(torch.Tensor, "record_stream", spy)
    for call, used in [
        (lambda s: i8.quantize_fp8(X, codes, scales, stream=s), (X, codes, scales)),
        (lambda s: i8.prepare_weight_fp8(W, stream=s), (W,)),
        (lambda s: i8.forward_fp8(X, w, out=Y, workspace=ws, stream=s), (X, w.codes, w.scales, Y, ws.buf)),
        (lambda s: i8.forward_fp8(X, w, stream=s), (X, w.codes, w.scales)),
        (lambda s: i8.forward_moe_fp8(X, m, 2, out=Z, workspace=mws, stream=s),
         (X, m.router, *m.gate, *m.up, *m.down, Z, mws.buf)),
        (lambda s: i8.forward_moe_fp8(X, m, 2, stream=s), (X, m.router, *m.gate, *m.up, *m.down)),
    ]:
        seen.clear()
        call(side)
        assert {p for p, s in seen if s == side} == {t.untyped_storage().data_ptr() for t in used}
        seen.clear()
        call(None)                           # on the current stream nothing is recorded
        side.synchronize()
        torch.cuda.synchronize()
        assert not seen


def test_tensors_that_a_call_refuses_are_refused_with_a_stream_too(cuda_ok):
    g = torch.Generator(device="cuda").manual_seed(7)
    side = torch.cuda.Stream()
    X = torch.randn(24, 512, device="cuda", generator=g).half()
    w, m = i8.weight_fp8(_codes(256, 512, g=g), torch.ones(2, 4, device="cuda")), _moe_weight(4, 512, 256, g)
    for call in (lambda **kw: i8.forward_fp8(X, w, out=torch.empty(24, 256).half(), **kw),
                 lambda **kw: i8.forward_fp8(X.cpu(), w, **kw),
                 lambda **kw: i8.forward_moe_fp8(X, m, 2, out=torch.empty(24, 512).half(), **kw),
                 lambda **kw: i8.quantize_fp8(X, codes=torch.empty(24, 512).to(torch.float8_e4m3fn), **kw),
                 lambda **kw: i8.quantize_fp8(X, scales=torch.empty(24, 4), **kw)):
        for kw in ({}, {"stream": side}):
            with pytest.raises(ValueError):
                call(**kw)


@pytest.mark.parametrize("make", [_quantize, _product, _layer])
def test_a_call_with_its_stream_named_in_a_capture(cuda_ok, make):
    """stream= is the capturing stream; what was captured runs after the caller's
    other tensors have come and gone."""
    call = make(torch.Generator(device="cuda").manual_seed(8))
    want = call(None).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = call(side)
    torch.full((1 << 22,), 0x11, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        got.zero_()
        graph.replay()
        assert torch.equal(got, want)
