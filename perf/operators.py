"""The block-scaled FP8 operators on the sizes they are used at: plain forms, inputs and 64-bit values.

A row of activations is held in E4M3 with one power-of-two scale (E8M0) for
each 128 consecutive values, a weight matrix with one for each 128 x 128
block.  The operators: the two quantisers, the linear layer on their codes,
the weight gradient taken from the 8-bit codes kept of the forward pass, and
the GELU's backward pass from an 8-bit checkpoint of its input.

Sizes: the single-stream DiT (4096 -> 4096 -> 16384, 4096 tokens), the video
DiT (1536 -> 8960, 21 frames of 1560 patches = 32760 tokens), the tiny layer
(64 tokens of 256), single tokens, and ragged sizes between them.
"""

import math

import torch

own = False

BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token's input of a 4096-wide layer: the latency of the quantiser
        {"name": "quantize_token", "op": "quantize", "T": 1, "d": 4096, "dtype": "bf16", "gelu": False, "checkpoint": False},
        # a video step's MLP hidden rows: GELU, codes for the down projection, codes of the input for the backward pass
        {"name": "quantize_video_gelu", "op": "quantize", "T": 32760, "d": 8960, "dtype": "bf16", "gelu": True, "checkpoint": True},
        # fp32 master weights of an attention projection, inference layout only
        {"name": "weights_4096_f32", "op": "weights", "N": 4096, "K": 4096, "dtype": "f32", "transposed": False},
        # the MLP up projection in both layouts, as a training step lays it out
        {"name": "weights_16384x4096", "op": "weights", "N": 16384, "K": 4096, "dtype": "bf16", "transposed": True},
        # a single token through an attention projection: bound by reading the weights
        {"name": "linear_token", "op": "linear", "M": 1, "N": 4096, "K": 4096},
        # a ragged batch of text tokens and widths that fill neither a tile nor a scale block
        {"name": "linear_ragged", "op": "linear", "M": 333, "N": 1001, "K": 1552},
        # the MLP up projection of the single-stream DiT
        {"name": "linear_mlp_up", "op": "linear", "M": 4096, "N": 16384, "K": 4096},
        # the MLP down projection of a whole video
        {"name": "linear_video_down", "op": "linear", "M": 32760, "N": 1536, "K": 8960},
        # weight gradient of an attention projection from one frame's tokens: few output tiles
        {"name": "wgrad_frame", "op": "wgrad", "M": 1560, "N": 1536, "K": 1536},
        # weight gradient of the MLP up projection
        {"name": "wgrad_mlp_up", "op": "wgrad", "M": 4096, "N": 16384, "K": 4096},
        # the GELU's backward pass of the tiny layer: latency
        {"name": "gelu_backward_tiny", "op": "gelu_backward", "T": 64, "d": 256, "quantize": False},
        # the GELU's backward pass of the MLP, its result also in FP8 for the input gradient
        {"name": "gelu_backward_mlp", "op": "gelu_backward", "T": 4096, "d": 16384, "quantize": True},
    ]


def _size(rng, lo, hi, step=1):
    """A size in [lo, hi], a multiple of `step`, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


MOST_ELEMS = 32760 * 8960
MOST_MACS = 4096 * 4096 * 16384


def draw(rng):
    op = rng.choice(["quantize", "weights", "linear", "linear", "wgrad", "gelu_backward"])
    if op in ("quantize", "gelu_backward"):
        d = _size(rng, 64, 16384, 16)
        T = _size(rng, 1, min(32768, MOST_ELEMS // (2 * d)))
        if op == "gelu_backward":
            return {"op": op, "T": T, "d": d, "quantize": rng.random() < 0.5}
        gelu = rng.random() < 0.5
        return {"op": op, "T": T, "d": d, "dtype": rng.choice(["bf16", "bf16", "f32"]), "gelu": gelu,
                "checkpoint": gelu and rng.random() < 0.5}
    if op == "weights":
        return {"op": op, "N": _size(rng, 64, 16384, 16), "K": _size(rng, 64, 4096, 16),
                "dtype": rng.choice(["bf16", "f32"]), "transposed": rng.random() < 0.5}
    K = _size(rng, 64, 16384, 16)
    if op == "wgrad":
        N = _size(rng, 64, 16384, 16)
        return {"op": op, "M": _size(rng, 1, max(1, min(32768, MOST_MACS // (N * K)))), "N": N, "K": K}
    N = _size(rng, 64, 16384)
    return {"op": op, "M": _size(rng, 1, max(1, min(32768, MOST_MACS // (N * K)))), "N": N, "K": K}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(g, T, d, dtype):
    """Student-t(3) values with 1 % of the channels 30 times larger, as the DiT layers' inputs have."""
    x = torch.randn((T, d), generator=g, device="cuda")
    chi = torch.zeros_like(x)
    for _ in range(3):
        chi += torch.randn((T, d), generator=g, device="cuda").square_()
    x /= (chi / 3).sqrt_()
    wide = torch.randperm(d, generator=g, device="cuda")[: max(1, d // 100)]
    x[:, wide] *= 30.0
    return x.to(dtype)


def _preactivations(g, T, d, dtype):
    """A GELU's input: normal values, channels of different widths and means."""
    x = torch.randn((T, d), generator=g, device="cuda")
    x *= 0.5 + torch.rand((1, d), generator=g, device="cuda") * 2
    x += torch.randn((1, d), generator=g, device="cuda") * 0.5
    return x.to(dtype)


def _weights(g, N, K, dtype):
    w = torch.randn((N, K), generator=g, device="cuda") * 0.02
    w[torch.rand((N, K), generator=g, device="cuda") < 0.01] *= 10.0
    return w.to(dtype)


def _gradients(g, T, d):
    """Gradients: small, and of different sizes from token to token."""
    y = torch.randn((T, d), generator=g, device="cuda")
    y *= 1e-3 * torch.exp(torch.randn((T, 1), generator=g, device="cuda"))
    return y.to(torch.bfloat16)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    state = dict(case)
    if op == "quantize":
        make = _preactivations if case["gelu"] else _activations
        state["X"] = make(g, case["T"], case["d"], DTYPES[case["dtype"]])
    elif op == "weights":
        state["W"] = _weights(g, case["N"], case["K"], DTYPES[case["dtype"]])
    elif op == "linear":
        state["a"] = _quantize_rows(_activations(g, case["M"], case["K"], torch.bfloat16).float())
        state["w"] = _quantize_blocks(_weights(g, case["N"], case["K"], torch.bfloat16).float())
    elif op == "wgrad":
        state["dY"] = _gradients(g, case["M"], case["N"])
        state["a"] = _quantize_rows(_activations(g, case["M"], case["K"], torch.bfloat16).float())
    else:
        state["dH"] = _gradients(g, case["T"], case["d"])
        state["x"] = _quantize_rows(_preactivations(g, case["T"], case["d"], torch.bfloat16).float())
    return state


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _padded(x, rows, cols):
    return torch.nn.functional.pad(x, (0, -x.shape[1] % cols, 0, -x.shape[0] % rows))


def _scale_byte(amax):
    """E8M0 byte of the smallest power of two s with amax / s <= 448, from the fp32 bits of amax; at least 2^-117."""
    bits = amax.contiguous().view(torch.int32)
    byte = (bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)
    return byte.clamp(10, 247)


def _power(byte):
    """2^(byte - 127) as fp32, bytes 1 to 254."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _encode(x, rows):
    """Codes and scales of fp32 x with a scale for each block of rows x 128."""
    n, d = x.shape
    p = _padded(x, rows, BLOCK)
    b = p.view(p.shape[0] // rows, rows, p.shape[1] // BLOCK, BLOCK)
    byte = _scale_byte(b.abs().amax(dim=(1, 3)))
    q = (b * _power(254 - byte)[:, None, :, None]).view(p.shape)[:n, :d]
    return q.to(torch.float8_e4m3fn), byte.to(torch.uint8).view(torch.float8_e8m0fnu)


def _quantize_rows(x):
    return _encode(x, 1)


def _quantize_blocks(w):
    return _encode(w, BLOCK)


def _spread(scale, rows, n, d):
    return scale.repeat_interleave(rows, 0)[:n].repeat_interleave(BLOCK, 1)[:, :d]


def _decode(codes, scale, rows):
    return codes.float() * _spread(_power(scale.view(torch.uint8)), rows, *codes.shape)


def _gelu(x):
    return 0.5 * x * torch.special.erfc(x * -math.sqrt(0.5))


def _gelu_slope(x):
    return 0.5 * torch.special.erfc(x * -math.sqrt(0.5)) + x * torch.exp(-0.5 * x * x) * (1 / math.sqrt(2 * math.pi))


def run(state):
    op = state["op"]
    if own:
        import rotation_bit_ptq_b200 as rbq
        if op == "quantize":
            return rbq.quantize_fp8(state["X"], activation="gelu" if state["gelu"] else None,
                                    checkpoint=state["checkpoint"])
        if op == "weights":
            return rbq.quantize_weights_fp8(state["W"], transposed=state["transposed"])
        if op == "linear":
            return rbq.qlinear_fp8(*state["a"], *state["w"])
        if op == "wgrad":
            return rbq.qlinear_fp8_wgrad(state["dY"], *state["a"])
        return rbq.gelu_backward_fp8(state["dH"], *state["x"], quantize=state["quantize"])
    if op == "quantize":
        x = state["X"].float()
        out = _quantize_rows(_gelu(x) if state["gelu"] else x)
        return (*out, *_quantize_rows(x)) if state["checkpoint"] else out
    if op == "weights":
        codes, scale = _quantize_blocks(state["W"].float())
        if not state["transposed"]:
            return codes, scale
        return codes, scale, codes.view(torch.uint8).t().contiguous().view(codes.dtype), \
            scale.view(torch.uint8).t().contiguous().view(scale.dtype)
    if op == "linear":
        return (_decode(*state["a"], 1) @ _decode(*state["w"], BLOCK).t()).to(torch.bfloat16)
    if op == "wgrad":
        return (state["dY"].float().t() @ _decode(*state["a"], 1)).to(torch.bfloat16)
    dx = (state["dH"].float() * _gelu_slope(_decode(*state["x"], 1))).to(torch.bfloat16)
    return (dx, *_quantize_rows(dx.float())) if state["quantize"] else dx


# ---------------------------------------------------------------------------
# what a pass cannot do without, and the values in 64 bits
# ---------------------------------------------------------------------------

def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    op = case["op"]
    if op in ("quantize", "gelu_backward"):
        T, d = case["T"], case["d"]
        code_row = d + _blocks(d)
        if op == "quantize":
            moved = T * (d * (2 if case["dtype"] == "bf16" else 4) + code_row * (2 if case["checkpoint"] else 1))
        else:
            moved = T * (4 * d + code_row * (2 if case["quantize"] else 1))
        return {"bytes": moved, "flops": 2 * T * d}
    if op == "weights":
        N, K = case["N"], case["K"]
        layouts = 2 if case["transposed"] else 1
        return {"bytes": N * K * (2 if case["dtype"] == "bf16" else 4) + layouts * (N * K + _blocks(N) * _blocks(K)),
                "flops": 2 * N * K}
    M, N, K = case["M"], case["N"], case["K"]
    codes = M * (K + _blocks(K))
    if op == "linear":
        return {"bytes": codes + N * K + _blocks(N) * _blocks(K) + 2 * M * N, "flops": 2 * M * N * K}
    return {"bytes": codes + 2 * M * N + 2 * N * K, "flops": 2 * M * N * K}


def _exact_scale(amax):
    """2^ceil(log2(amax / 448)), at least 2^-117, in 64 bits."""
    m, e = torch.frexp(amax / 448.0)          # amax / 448 = m 2^e with m in [1/2, 1)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(amax > 0, e, torch.full_like(e, -117)).clamp(-117, 120)
    return torch.ldexp(torch.ones_like(amax), e)


def _exact_codes(x, rows):
    """x over its blocks' scales, and the scales: the codes before their rounding to E4M3."""
    n, d = x.shape
    N, D = _blocks(n) * BLOCK if rows == BLOCK else n, _blocks(d) * BLOCK
    p = x.new_zeros((N, D))
    p[:n, :d] = x
    amax = p.abs().reshape(N // rows, rows, D // BLOCK, BLOCK).amax(3).amax(1)
    s = _exact_scale(amax)
    return x / _spread(s, rows, n, d), s


def _exact_values(codes, scale, rows):
    return codes.double() * _spread(scale.double(), rows, *codes.shape)


def _exact_cdf(x):
    return 0.5 * torch.special.erfc(-x / math.sqrt(2.0))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["X"].double()
        out = _exact_codes(x * _exact_cdf(x) if case["gelu"] else x, 1)
        return (*out, *_exact_codes(x, 1)) if case["checkpoint"] else out
    if op == "weights":
        codes, scale = _exact_codes(s["W"].double(), BLOCK)
        return (codes, scale, codes.t().contiguous(), scale.t().contiguous()) if case["transposed"] else (codes, scale)
    if op == "linear":
        return _exact_values(*s["a"], 1) @ _exact_values(*s["w"], BLOCK).t()
    if op == "wgrad":
        return s["dY"].double().t() @ _exact_values(*s["a"], 1)
    x = _exact_values(*s["x"], 1)
    dx = s["dH"].double() * (_exact_cdf(x) + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi))
    # the codes are those of the BF16 result
    return (dx, *_exact_codes(dx.to(torch.bfloat16).double(), 1)) if case["quantize"] else dx
