"""Cases that measure the block-scaled 8-bit floating point operators.

Three operators, each in plain torch (32-bit arithmetic, one rounding at the
end) and through the library:

- ``quantize``: 16-bit activations to e4m3 codes with one fp32 scale per row
  and block of 128 consecutive k;
- ``product``: Y = X W with X quantised that way per call and W held as e4m3
  codes with one fp32 scale per 128 x 128 block;
- ``moe``: a mixture-of-experts layer for a few tokens (router, top-k, gated
  experts with block-scaled weights, weighted sum).

The rule of the codes, for a block of values with absolute maximum a (all steps
in fp32): s = max(a / 448, 2^-126), code = e4m3(x * (1 / s)), value = code * s.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -126
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the activations of a decode step of the decode-shaped feed-forward layer
        {"name": "quantize-decode", "op": "quantize", "M": 8, "K": 4096, "dtype": "fp16"},
        # the activations of a prefill of the 175B-scale feed-forward layer
        {"name": "quantize-175b", "op": "quantize", "M": 4096, "K": 12288, "dtype": "bf16"},
        # the smallest layer of the tests: latency only
        {"name": "product-tiny", "op": "product", "M": 16, "K": 256, "N": 384, "dtype": "fp16"},
        # one decode step of the decode-shaped feed-forward up-projection
        {"name": "product-decode", "op": "product", "M": 8, "K": 4096, "N": 11008, "dtype": "fp16"},
        # a single token through the 175B-scale up-projection
        {"name": "product-token", "op": "product", "M": 1, "K": 12288, "N": 49152, "dtype": "bf16"},
        # a mid-sized batch of decode rows through a down-projection
        {"name": "product-batch", "op": "product", "M": 100, "K": 11008, "N": 4096, "dtype": "bf16"},
        # odd row count, K and N that end inside a block of 128
        {"name": "product-ragged", "op": "product", "M": 333, "K": 4112, "N": 5136, "dtype": "bf16"},
        # prefill of the prefill-shaped feed-forward layer
        {"name": "product-prefill", "op": "product", "M": 2048, "K": 8192, "N": 28672, "dtype": "fp16"},
        # prefill of the 175B-scale feed-forward layer
        {"name": "product-175b", "op": "product", "M": 4096, "K": 12288, "N": 49152, "dtype": "bf16"},
        # one token, few large experts (the decode-shaped layer as each expert)
        {"name": "moe-token", "op": "moe", "T": 1, "E": 8, "k": 2, "H": 4096, "I": 11008, "dtype": "bf16", "renorm": True},
        # a decode batch over many small experts
        {"name": "moe-batch", "op": "moe", "T": 16, "E": 64, "k": 8, "H": 2048, "I": 1408, "dtype": "bf16", "renorm": True},
        # a larger batch, every expert busy, an intermediate size that ends inside a block
        {"name": "moe-many", "op": "moe", "T": 61, "E": 32, "k": 4, "H": 4096, "I": 2064, "dtype": "fp16", "renorm": False},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "moe"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "quantize":
        return {"op": op, "M": _log(rng, 1, 4096), "K": _log(rng, 16, 12288, 16), "dtype": dtype}
    if op == "product":
        return {"op": op, "M": _log(rng, 1, 4096), "K": _log(rng, 64, 12288, 16), "N": _log(rng, 64, 49152, 16),
                "dtype": dtype}
    E = _log(rng, 2, 64)
    return {"op": op, "T": _log(rng, 1, 64), "E": E, "k": rng.randint(1, min(8, E)), "H": _log(rng, 256, 4096, 16),
            "I": _log(rng, 128, 2064, 16), "dtype": dtype, "renorm": rng.random() < 0.5}


def work(case):
    if case["op"] == "quantize":
        M, K = case["M"], case["K"]
        return {"bytes": 3 * M * K + 4 * M * -(-K // 128), "flops": 3 * M * K}
    if case["op"] == "product":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": 2 * M * K + K * N + 4 * -(-K // 128) * -(-N // 128) + 2 * M * N, "flops": 2 * M * N * K}
    T, E, k, H, I = case["T"], case["E"], case["k"], case["H"], case["I"]
    busy = E * (1 - (1 - k / E) ** T)  # experts that T tokens choosing evenly are expected to reach
    scales = 4 * -(-H // 128) * -(-I // 128)
    return {"bytes": busy * 3 * (H * I + scales) + 2 * E * H + 4 * T * H + 8 * T * k,
            "flops": 2 * T * E * H + 6 * T * k * H * I}


# ------------------------------------------------------------------ inputs

def _activations(M, K, dtype, g):
    """N(0, 1) with a few large feature columns, as a transformer's activations have them."""
    x = torch.randn(M, K, device="cuda", generator=g)
    cols = torch.randperm(K, device="cuda", generator=g)[: max(1, K // 1024)]
    x[:, cols] *= 20 + 40 * torch.rand(cols.numel(), device="cuda", generator=g)
    return x.to(DTYPES[dtype])


def _weight(rows, cols, g, lead=()):
    """e4m3 codes (rows x cols: one row per output channel) and 128 x 128 block scales of random weights."""
    nb, kb = -(-rows // 128), -(-cols // 128)
    codes, scales = [], []
    for _ in range(math.prod(lead)):
        w = torch.zeros(nb * 128, kb * 128, device="cuda")
        w[:rows, :cols] = torch.randn(rows, cols, device="cuda", generator=g) * (1.0 / math.sqrt(cols))
        w = w.view(nb, 128, kb, 128)
        s = w.abs().amax((1, 3)) / E4M3_MAX
        q = (w / s[:, None, :, None]).clamp_(-E4M3_MAX, E4M3_MAX)
        codes.append(q.view(nb * 128, kb * 128)[:rows, :cols].to(torch.float8_e4m3fn))
        scales.append(s)
    return torch.stack(codes).view(*lead, rows, cols), torch.stack(scales).view(*lead, nb, kb)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case, "op": case["op"]}
    if case["op"] == "moe":
        E, H, I = case["E"], case["H"], case["I"]
        st["X"] = _activations(case["T"], H, case["dtype"], g)
        st["router"] = (torch.randn(E, H, device="cuda", generator=g) / math.sqrt(H)).to(DTYPES[case["dtype"]])
        for name, rows, cols in (("gate", I, H), ("up", I, H), ("down", H, I)):
            st[name] = _weight(rows, cols, g, (E,))
        if own:
            import int8_quantized_matmul_02_b200 as i8

            st["w"] = i8.moe_weight_fp8(st["router"], st["gate"], st["up"], st["down"])
            st["ws"] = i8.MoeWorkspace(case["T"], st["w"], case["k"])
        return st
    st["X"] = _activations(case["M"], case["K"], case["dtype"], g)
    if case["op"] == "product":
        codes, scales = _weight(case["N"], case["K"], g)
        st["codes"], st["scales"] = codes, scales
        if own:
            import int8_quantized_matmul_02_b200 as i8

            st["w"] = i8.weight_fp8(codes, scales)
            st["ws"] = i8.Fp8Workspace(case["M"], case["K"], case["N"])
    return st


# ------------------------------------------------------------------ plain forms

def _quantize(x):
    """(e4m3 codes, scales) of the last axis of an fp32 tensor, in blocks of 128."""
    K = x.shape[-1]
    kb = -(-K // 128)
    b = torch.nn.functional.pad(x, (0, kb * 128 - K)).unflatten(-1, (kb, 128))
    a = b.abs().amax(-1)
    s = torch.clamp(a / torch.full_like(a, E4M3_MAX), min=TINY)
    q = (b * torch.reciprocal(s)[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    return q.flatten(-2)[..., :K].to(torch.float8_e4m3fn), s


def _rows_value(q, s):
    return q.float() * s.repeat_interleave(128, -1)[..., : q.shape[-1]]


def _weight_value(q, s):
    s = s.repeat_interleave(128, -1)[..., : q.shape[-1]]
    return q.float() * s.repeat_interleave(128, -2)[..., : q.shape[-2], :]


def _plain_moe(st):
    c, X = st["case"], st["X"]
    T, E, k = c["T"], c["E"], c["k"]
    # two experts whose scores are near each other must not change places: 64-bit sums
    logits = X.double() @ st["router"].double().t()
    top, ids = torch.sort(logits, dim=-1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    p = torch.exp((top - top[:, :1]).float())
    p = p / (p if c["renorm"] else torch.exp((logits - top[:, :1]).float())).sum(-1, keepdim=True)
    x = _rows_value(*_quantize(X.float()))
    if T * k < E:  # only the chosen experts' weights, one set for each (token, choice)
        pick = ids.flatten()
        gate, up, down = (_weight_value(q.view(torch.uint8)[pick].view(q.dtype), s[pick])
                          for q, s in (st["gate"], st["up"], st["down"]))
        x = x.repeat_interleave(k, 0)[:, None]
        comb = p.flatten()
    else:  # every expert on every token, the ones not chosen at weight zero
        gate, up, down = (_weight_value(*st[n]) for n in ("gate", "up", "down"))
        x = x[None].expand(E, T, -1)
        comb = torch.zeros(T, E, device=X.device).scatter(1, ids, p)
    a = x @ gate.transpose(1, 2)
    h = a / (1 + torch.exp(-a)) * (x @ up.transpose(1, 2))
    y = _rows_value(*_quantize(h)) @ down.transpose(1, 2)
    if T * k < E:
        y = (y[:, 0] * comb[:, None]).view(T, k, -1).sum(1)
    else:
        y = (y * comb.t()[:, :, None]).sum(0)
    return y.to(X.dtype), ids.int(), p


def run(st):
    if own:
        import int8_quantized_matmul_02_b200 as i8

        if st["op"] == "quantize":
            return i8.quantize_fp8(st["X"])
        if st["op"] == "product":
            return i8.forward_fp8(st["X"], st["w"], workspace=st["ws"])
        c = st["case"]
        return i8.forward_moe_fp8(st["X"], st["w"], c["k"], renormalize=c["renorm"], workspace=st["ws"],
                                  return_routing=True)
    if st["op"] == "quantize":
        return _quantize(st["X"].float())
    if st["op"] == "product":
        y = _rows_value(*_quantize(st["X"].float())) @ _weight_value(st["codes"], st["scales"]).t()
        return y.to(st["X"].dtype)
    return _plain_moe(st)


# ------------------------------------------------------------------ 64-bit results

def _exact_codes(x):
    """Codes (as doubles) and scales of x (double holding fp32 values), rounding on the e4m3 grid by hand.

    The scale, its reciprocal and the scaled value are rounded to fp32, as the
    definition has it; a double quotient or product rounded to fp32 is the
    correctly rounded fp32 one."""
    f32 = lambda v: v.to(torch.float32).double()  # noqa: E731
    M, K = x.shape
    kb = (K + 127) // 128
    padded = x.new_zeros(M, kb * 128)
    padded[:, :K] = x
    padded = padded.view(M, kb, 128)
    s = f32(padded.abs().max(dim=2).values / E4M3_MAX).clamp(min=TINY)
    v = f32(padded * f32(1.0 / s)[:, :, None])
    exponent = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))).clamp(max=8)
    step = torch.exp2(exponent - 3)
    q = (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
    return q.view(M, kb * 128)[:, :K], s


def _exact_product(q, s, codes, scales):
    M, K = q.shape
    N = codes.shape[0]
    xs = s[:, :, None].expand(-1, -1, 128).reshape(M, -1)[:, :K]
    y = q.new_empty(M, N)
    for n in range(0, N, 4096):  # bands of output channels bound the memory
        m = min(N, n + 4096)
        ws = scales[n // 128: (m + 127) // 128].double()[:, None, :, None].expand(-1, 128, -1, 128)
        ws = ws.reshape(-1, scales.shape[1] * 128)[: m - n, :K]
        y[:, n:m] = (q * xs) @ (codes[n:m].double() * ws).t()
    return y


def exact(case, seed):
    st = prepare(case, seed)
    X = st["X"].double()
    q, s = _exact_codes(X)
    if case["op"] == "quantize":
        return q, s
    if case["op"] == "product":
        return _exact_product(q, s, st["codes"], st["scales"])
    T, E, k = case["T"], case["E"], case["k"]
    logits = X @ st["router"].double().t()
    order = torch.empty(T, k, dtype=torch.int64, device=X.device)
    left = logits.clone()
    for j in range(k):
        best = left.max(dim=1, keepdim=True).values
        first = torch.where(left == best, torch.arange(E, device=X.device), E).min(dim=1).values
        order[:, j] = first
        left.scatter_(1, first[:, None], -math.inf)
    weights = torch.softmax(logits, dim=1).gather(1, order)
    if case["renorm"]:
        weights = weights / weights.sum(dim=1, keepdim=True)
    y = torch.zeros(T, case["H"], dtype=torch.float64, device=X.device)
    for e in range(E):
        t, j = torch.nonzero(order == e, as_tuple=True)
        if not t.numel():
            continue
        gate, up, down = ((st[n][0][e], st[n][1][e]) for n in ("gate", "up", "down"))
        a = _exact_product(q[t], s[t], *gate)
        h = a * torch.sigmoid(a) * _exact_product(q[t], s[t], *up)
        hq, hs = _exact_codes(h.to(torch.float32).double())
        y.index_add_(0, t, _exact_product(hq, hs, *down) * weights[t, j][:, None])
    return y, order.int(), weights
