"""The block-scaled FP8 layer on the GPU against the fp64 oracle.

Tolerances, all relative to the fp64 value computed from the same codes:

* codes and scales of plain values: exact (x / s is exact in fp32, the scale a
  function of the bits of the maximum);
* of GELU(x): the kernel's h is within E_h = 4e-7 |x| of the exact one (the
  CDF's published 1.5e-7 / 2, and the roundings of its exponential, reciprocal
  and products, 2e-7 in all for |cdf| <= 1), so the decoded code is within half an
  E4M3 step (2^-4 of the value, 2^-10 s below the normal range) plus E_h of it;
* BF16 results: 2^-8 |y| for the rounding (at most half a step), plus the fp32 sum's own error:
  each of the (terms / 32) steps of the tensor core's accumulation (/ 16 on
  BF16 operands) loses at most 2^-21 of the absolute sum so far, so
  (steps + 8) 2^-21 sum |a b| in all.
"""

import numpy as np
import pytest

import oracle
import synth
from parity import bf16_to_numpy, poison, torch_bf16

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import rotation_bit_ptq_b200 as rbq  # noqa: E402

F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture(autouse=True)
def _no_device_error():
    yield
    torch.cuda.synchronize()
    assert rbq.device_error() == 0


def _code_values(codes):
    return codes.double().cpu().numpy()


def _exponents(scale):
    return scale.view(torch.uint8).cpu().numpy().astype(np.int64) - 127


def _held(codes, scale, rows=1):
    return oracle.fp8_decode(_code_values(codes), _exponents(scale), rows)


def _values(g, shape, dtype):
    """Heavy-tailed values whose blocks differ by many binades."""
    x = (g.standard_t(3, shape) * np.exp(g.normal(0, 3, (shape[0], 1)))).astype(np.float32)
    x[:, ::37] *= np.float32(30.0)
    return synth.to_bf16(x) if dtype == "bf16" else x


def _tensor(x, dtype):
    return torch_bf16(x) if dtype == "bf16" else torch.from_numpy(x).cuda()


def _random_codes(g, n, d, rows=1):
    q, s = (rbq.quantize_fp8 if rows == 1 else rbq.quantize_weights_fp8)(_tensor(_values(g, (n, d), "bf16"), "bf16"))
    return q, s, _held(q, s, rows)


def _close(got, ref, absum, steps):
    tol = 2.0 ** -8 * np.abs(ref) + (steps + 8) * 2.0 ** -21 * absum
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.max(np.abs(got - ref) / tol)))


# ---- quantisers ---------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 16), (1, 4096), (3, 128), (33, 144), (100, 1040), (257, 640)])
def test_quantize_rows_exact(T, d, dtype):
    x = _values(np.random.default_rng(T + d), (T, d), dtype)
    q, s = rbq.quantize_fp8(_tensor(x, dtype))
    rq, re = oracle.fp8_encode(x)
    assert q.dtype == F8 and s.dtype == E8 and s.shape == (T, rbq.fp8_blocks(d))
    assert np.array_equal(_exponents(s), re)
    assert np.array_equal(_code_values(q), rq)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K", [(1, 16), (16, 16), (128, 128), (272, 400), (130, 1552), (512, 640)])
def test_quantize_weights_exact(N, K, dtype):
    w = _values(np.random.default_rng(N + K), (N, K), dtype)
    trans = N % 16 == 0
    out = rbq.quantize_weights_fp8(_tensor(w, dtype), transposed=trans)
    rq, re = oracle.fp8_encode(w, 128)
    assert np.array_equal(_exponents(out[1]), re)
    assert np.array_equal(_code_values(out[0]), rq)
    if trans:
        assert out[2].shape == (K, N) and out[3].shape == (rbq.fp8_blocks(K), rbq.fp8_blocks(N))
        assert np.array_equal(_code_values(out[2]), rq.T)
        assert np.array_equal(_exponents(out[3]), re.T)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_edge_values(dtype):
    """Zero blocks, values next to a scale's border and to a code's, infinities
    and NaN beside ordinary values, the smallest and the largest values."""
    x = np.zeros((10, 256), dtype=np.float32)
    x[0, :3] = 448.0, -1.0, 2.0 ** -9
    x[1, :3] = 450.0, 7.0, -0.0
    x[2, :4] = np.inf, -np.inf, np.nan, 5.0
    x[2, 128] = np.nan
    x[3, :2] = 3.3e38, -1.0
    x[4, :2] = 2.0 ** -120, 2.0 ** -126
    x[5, :2] = 2.0 ** -133, -(2.0 ** -133)                       # subnormal in fp32 and BF16
    x[6, :8] = 256.0, 17.0, 17.5, 18.5, 19.5, 0.0009765625, 0.001953125, 0.0029296875     # ties
    x[7, :] = -1.0
    x[8, 127], x[8, 128] = 1e-30, 1e30                             # neighbours in different blocks
    x[9, :] = np.inf
    if dtype == "bf16":
        with np.errstate(invalid="ignore"):
            keep = ~np.isfinite(x)
            x = np.where(keep, x, synth.to_bf16(np.where(keep, 0, x)))
        t = torch.from_numpy(x).to(torch.bfloat16).cuda()
    else:
        t = torch.from_numpy(x).cuda()
    rq, re = oracle.fp8_encode(x)
    q, s = rbq.quantize_fp8(t)
    assert np.array_equal(_exponents(s), re)
    assert np.array_equal(_code_values(q), rq, equal_nan=True)
    rq, re = oracle.fp8_encode(x, 128)
    q, s, qt, st = rbq.quantize_weights_fp8(torch.cat([t, torch.zeros_like(t[:6])]), transposed=True)
    assert np.array_equal(_exponents(s), re) and np.array_equal(_exponents(st), re.T)
    assert np.array_equal(_code_values(q)[:10], rq, equal_nan=True)
    assert np.array_equal(_code_values(qt)[:, :10], rq.T, equal_nan=True)


def test_decoded_values_are_exact_in_bf16():
    """(exp(25 z) is infinite for z > 3.55, which one run in 80 draws: such a
    value's code is NaN, and NaN is compared as equal to itself.)"""
    x = torch.randn(64, 512, device="cuda") * torch.exp(torch.randn(64, 1, device="cuda") * 25)
    q, s = rbq.quantize_fp8(x.contiguous())
    v = q.float() * s.float().repeat_interleave(128, 1)
    assert torch.allclose(v, v.bfloat16().float(), rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,ck", [(1, 16, False), (1, 4096, True), (77, 400, True), (130, 1024, False)])
def test_quantize_gelu_and_checkpoint(T, d, ck, dtype):
    g = np.random.default_rng(T + d)
    x = (g.standard_normal((T, d)) * 2.5).astype(np.float32)
    x = synth.to_bf16(x) if dtype == "bf16" else x
    out = rbq.quantize_fp8(_tensor(x, dtype), activation="gelu", checkpoint=ck)
    h = oracle.gelu(x.astype(np.float64))
    held = _held(*out[:2])
    s = oracle.fp8_scales(_exponents(out[1]), 1, x.shape)
    tol = np.maximum(2.0 ** -4 * np.abs(h), 2.0 ** -10 * s) + 4e-7 * np.abs(x)
    assert np.all(np.abs(held - h) <= tol)
    # the scale is the smallest that holds the block (its maximum known to 4e-7)
    pad = -d % 128
    amax = np.pad(np.abs(h), ((0, 0), (0, pad))).reshape(T, -1, 128).max(2)
    e = np.ldexp(1.0, _exponents(out[1]))
    assert np.all(amax <= 448 * e * (1 + 1e-6)) and np.all((amax > 224 * e * (1 - 1e-6)))
    if ck:
        rq, re = oracle.fp8_encode(x)
        assert np.array_equal(_exponents(out[3]), re)
        assert np.array_equal(_code_values(out[2]), rq)


@pytest.mark.parametrize("quantize", [False, True])
@pytest.mark.parametrize("T,d", [(1, 16), (64, 256), (77, 400), (5, 4096)])
def test_gelu_backward(T, d, quantize):
    g = np.random.default_rng(T * d)
    xq, xs = rbq.quantize_fp8(_tensor((g.standard_normal((T, d)) * 3).astype(np.float32), "f32"))
    dh = synth.to_bf16((g.standard_normal((T, d)) * np.exp(g.normal(-5, 2, (T, 1)))).astype(np.float32))
    out = rbq.gelu_backward_fp8(torch_bf16(dh), xq, xs, quantize=quantize)
    dx = out[0] if quantize else out
    x = _held(xq, xs)
    ref = dh * oracle.gelu_slope(x)
    got = bf16_to_numpy(dx)
    # half a BF16 step, and the slope's own error: CDF 2e-7, x phi(x) 2e-7 |x|
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 4e-7 * (1 + np.abs(x)) * np.abs(dh))
    # ... and against differences of the GELU itself
    step = 1e-4
    slope = (oracle.gelu(x + step) - oracle.gelu(x - step)) / (2 * step)
    assert np.all(np.abs(got - dh * slope) <= (2.0 ** -8 * np.abs(slope) + 1e-6 * (1 + np.abs(x))) * np.abs(dh))
    if quantize:
        rq, re = oracle.fp8_encode(got)          # the codes of the BF16 gradient
        assert np.array_equal(_exponents(out[2]), re)
        assert np.array_equal(_code_values(out[1]), rq)


def test_gelu_backward_in_place():
    g = np.random.default_rng(1)
    xq, xs, _ = _random_codes(g, 300, 1040)
    dh = torch.randn(300, 1040, device="cuda").bfloat16()
    ref = rbq.gelu_backward_fp8(dh, xq, xs)
    out = dh.clone()
    assert rbq.gelu_backward_fp8(out, xq, xs, out=out) is out
    assert torch.equal(out, ref)


def test_gelu_of_extreme_values():
    """Zeros of both signs, subnormals, values far out on both sides, infinities
    and NaN, each alone in its block."""
    v = np.array([0.0, -0.0, 1e-40, -1e-40, 2.0 ** -126, 6.0, -6.0, 13.0, -13.0, 100.0, -100.0, 1e5, -1e5, 1e30, -1e30,
                  3.3e38, -3.3e38, np.inf, -np.inf, np.nan], dtype=np.float32)
    x = np.zeros((len(v), 128), dtype=np.float32)
    x[:, 5] = v
    q, s, xq, xs = rbq.quantize_fp8(torch.from_numpy(x).cuda(), activation="gelu", checkpoint=True)
    with np.errstate(invalid="ignore"):
        h = oracle.gelu(v.astype(np.float64))
    got = _held(q, s)
    fin = np.isfinite(h)
    assert np.array_equal(np.isnan(got[:, 5]), ~fin)
    # as test_quantize_gelu_and_checkpoint; below the smallest scale a code's step is 2^-9 2^-117
    tol = np.maximum(2.0 ** -4 * np.abs(h), 2.0 ** -127) + 4e-7 * np.abs(v)
    assert np.all(np.abs(got[:, 5] - h)[fin] <= tol[fin])
    assert not np.nan_to_num(np.delete(got, 5, 1)).any()
    with np.errstate(invalid="ignore"):
        rq, re = oracle.fp8_encode(x)
    assert np.array_equal(_exponents(xs), re) and np.array_equal(_code_values(xq), rq, equal_nan=True)


def test_gelu_far_below_zero_keeps_its_digits():
    """Blocks that hold nothing but x in [-7, -3], where GELU(x) is x times the
    normal tail: the tail is known to 9e-4 of itself to -5 and 4e-3 to -7 (the fit's error,
    computed in 64 bits over [0, 7] when it was made), and exp2 and the roundings of its argument, of
    magnitude up to 43 and so 2^-19 each, add 9 * 2^-19 ln 2 + 2^-22 < 2e-5."""
    x = np.linspace(-7, -3, 64 * 128, dtype=np.float32).reshape(64, 128)
    q, s = rbq.quantize_fp8(torch.from_numpy(x).cuda(), activation="gelu")
    h = oracle.gelu(x.astype(np.float64))
    got, sc = _held(q, s), oracle.fp8_scales(_exponents(s), 1, x.shape)
    rel = np.where(x >= -5, 9e-4, 4.2e-3) + 2e-5
    assert np.all(np.abs(got - h) <= np.maximum(2.0 ** -4 * np.abs(h), 2.0 ** -10 * sc) + rel * np.abs(h) * (1 + 2.0 ** -4))


def test_gelu_backward_of_what_is_not_finite():
    """NaN in the checkpoint or the gradient reaches its own value and its own code only."""
    g = np.random.default_rng(2)
    xq, xs, _ = _random_codes(g, 6, 256)
    dh = torch.randn(6, 256, device="cuda").bfloat16()
    ref = rbq.gelu_backward_fp8(dh, xq, xs)
    xq.view(torch.uint8)[1, 7], xq.view(torch.uint8)[2, 130] = 0x7F, 0xFF
    dh[3, 9], dh[4, 200] = float("nan"), float("inf")
    xs.view(torch.uint8)[5, 1] = 255
    dx, q, s = rbq.gelu_backward_fp8(dh, xq, xs, quantize=True)
    bad = torch.zeros(6, 256, dtype=torch.bool, device="cuda")
    bad[1, 7] = bad[2, 130] = bad[3, 9] = bad[4, 200] = True
    bad[5, 128:] = True
    assert torch.equal(~torch.isfinite(dx), bad) and torch.equal(dx[~bad], ref[~bad])
    rq, re = oracle.fp8_encode(dx.double().cpu().numpy())
    assert np.array_equal(_exponents(s), re) and np.array_equal(_code_values(q), rq, equal_nan=True)


# ---- the layer ------------------------------------------------------------------------

@pytest.mark.parametrize("M,N,K", [(1, 128, 128), (1, 1, 16), (1, 1536, 1536), (1, 1001, 2064), (2, 999, 1552),
                                   (3, 130, 4112), (4, 33, 6000), (4, 1002, 272), (2, 64, 8960), (1, 4096, 4096), (2, 1000, 2048), (15, 300, 1040),
                                   (16, 256, 512), (17, 129, 272), (33, 1001, 640), (64, 512, 1536), (65, 130, 400),
                                   (128, 384, 2064), (129, 127, 128), (255, 500, 1552), (256, 256, 8960),
                                   (257, 256, 128), (300, 1001, 1552), (511, 8, 4096), (513, 264, 656),
                                   (700, 1536, 1536), (1025, 2049, 400)])
def test_layer(M, N, K):
    g = np.random.default_rng(M + 7 * N + K)
    aq, asc, a = _random_codes(g, M, K)
    wq, wsc, w = _random_codes(g, N, K, 128)
    out = poison((M, N), torch.bfloat16)
    y = rbq.qlinear_fp8(aq, asc, wq, wsc, out=out)
    assert y is out
    _close(bf16_to_numpy(y), a @ w.T, np.abs(a) @ np.abs(w).T, K / 32)


# Enough tiles for the kernel of CTA pairs; rows of Y by TMA (N a multiple of
# 8), of whole words (even N) and of halves; rows of scales that are
# multiples of 16, of 4 and of nothing, in one slot of 16 slices and in several.
@pytest.mark.parametrize("M,N,K", [(4097, 3001, 272), (4100, 3002, 528), (4096, 3004, 512), (4000, 3008, 2048),
                                   (3000, 4104, 4112), (33000, 264, 144), (2305, 6001, 16)])
def test_layer_of_many_tokens(M, N, K):
    g = np.random.default_rng(M + N + K)
    aq, asc, a = _random_codes(g, M, K)
    wq, wsc, w = _random_codes(g, N, K, 128)
    ref, absum = a @ w.T, np.abs(a) @ np.abs(w).T
    for off in (0, 1, 2):                                   # elements from a 16-byte boundary
        buf = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        y = rbq.qlinear_fp8(aq, asc, wq, wsc, out=buf[off:off + M * N].view(M, N))
        _close(bf16_to_numpy(y), ref, absum, K / 32)
        assert (buf[:off] == 7).all() and (buf[off + M * N:] == 7).all()


# Few tokens and a long K: split over a cluster, several slots of scales in each part.
@pytest.mark.parametrize("M,N,K", [(5, 130, 16384), (1, 1000, 40000), (40, 64, 33024), (130, 72, 20480)])
def test_layer_of_few_tokens_and_many_slices(M, N, K):
    g = np.random.default_rng(M + N + K)
    aq, asc, a = _random_codes(g, M, K)
    wq, wsc, w = _random_codes(g, N, K, 128)
    _close(bf16_to_numpy(rbq.qlinear_fp8(aq, asc, wq, wsc)), a @ w.T, np.abs(a) @ np.abs(w).T, K / 32)


def test_scales_at_any_address():
    """Scales that begin 1, 2, 3, 4 and 8 bytes from a boundary, at both ends of
    their buffers, for both kernels."""
    g = np.random.default_rng(8)
    for M, N, K in ((9, 260, 2048), (4097, 2600, 2048), (4097, 2600, 640)):
        aq, asc, a = _random_codes(g, M, K)
        wq, wsc, w = _random_codes(g, N, K, 128)
        ref = rbq.qlinear_fp8(aq, asc, wq, wsc)
        for off in (1, 2, 3, 4, 8):
            moved = []
            for t in (asc, wsc):
                buf = torch.zeros(t.numel() + off, dtype=torch.uint8, device="cuda")
                buf[off:] = t.view(torch.uint8).flatten()
                moved.append(buf[off:].view(E8).view(t.shape))
            assert torch.equal(rbq.qlinear_fp8(aq, moved[0], wq, moved[1]), ref)


def test_layer_uses_each_scale():
    """One non-zero code per row and scale block pins which scale meets which
    K slice and row: all sums are single exact products."""
    M, N, K = 300, 260, 1552
    g = np.random.default_rng(5)
    kb = rbq.fp8_blocks(K)
    for rows in (7, M):
        q = np.zeros((rows, K), dtype=np.float32)
        at = np.arange(rows) % kb * 128
        q[np.arange(rows), at] = 1.0
        e = g.integers(110, 140, (rows, kb))
        aq = torch.from_numpy(q).cuda().to(F8)
        asc = torch.from_numpy(e.astype(np.uint8)).cuda().view(E8)
        ew = g.integers(110, 140, (rbq.fp8_blocks(N), kb))
        wq = torch.ones(N, K, device="cuda").to(F8)
        wsc = torch.from_numpy(ew.astype(np.uint8)).cuda().view(E8)
        y = rbq.qlinear_fp8(aq, asc, wq, wsc)
        blk = np.arange(rows) % kb
        ref = np.ldexp(1.0, e[np.arange(rows), blk][:, None] - 127 + ew[np.arange(N) // 128][:, blk].T - 127)
        assert np.array_equal(bf16_to_numpy(y), ref)


def test_layer_with_far_scales():
    """Scales at the ends of what the quantisers choose, whose product is an
    ordinary number (or, both small, the smallest): single products, exact."""
    N, K = 260, 1552
    kb = rbq.fp8_blocks(K)
    g = np.random.default_rng(6)
    for rows in (1, 2, 4, 9, 300, 4100):
        q = np.zeros((rows, K), dtype=np.float32)
        blk = np.arange(rows) % kb
        q[np.arange(rows), blk * 128] = 1.0
        e = g.choice([10, 20, 127, 200, 247], (rows, kb))
        ew = g.choice([10, 20, 127, 200, 247], (rbq.fp8_blocks(N), kb))
        y = rbq.qlinear_fp8(torch.from_numpy(q).cuda().to(F8), torch.from_numpy(e.astype(np.uint8)).cuda().view(E8),
                            torch.ones(N, K, device="cuda").to(F8),
                            torch.from_numpy(ew.astype(np.uint8)).cuda().view(E8))
        exp = e[np.arange(rows), blk][:, None] - 127 + ew[np.arange(N) // 128][:, blk].T - 127
        sure = (exp >= -126) & (exp <= 127)
        got = bf16_to_numpy(y)
        assert np.array_equal(got[sure], np.ldexp(1.0, exp)[sure]), rows
        assert np.all(np.abs(got[exp < -126]) <= 2.0 ** -126) and np.all(np.isinf(got[exp > 127]))


def test_layer_nan_scales_and_codes_reach_only_their_rows():
    for M in (4, 5, 300):
        g = np.random.default_rng(M)
        aq, asc, a = _random_codes(g, M, 640)
        wq, wsc, w = _random_codes(g, 256, 640, 128)
        y0 = rbq.qlinear_fp8(aq, asc, wq, wsc)
        asc.view(torch.uint8)[3, 2] = 255
        aq.view(torch.uint8)[1, 7] = 0x7F
        y = rbq.qlinear_fp8(aq, asc, wq, wsc)
        rows = torch.isnan(y).all(1)
        assert rows[1] and rows[3] and int(rows.sum()) == 2
        keep = ~rows
        assert torch.equal(y[keep], y0[keep])


@pytest.mark.parametrize("M,N,K", [(64, 256, 256), (1, 8, 16), (1, 16, 64), (63, 24, 144), (100, 272, 400),
                                   (300, 264, 1040), (1560, 512, 384), (3001, 64, 128), (4096, 768, 272)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_weight_gradient(M, N, K, dtype):
    g = np.random.default_rng(M + N + K)
    aq, asc, a = _random_codes(g, M, K)
    dy = synth.to_bf16((g.standard_normal((M, N)) * np.exp(g.normal(-6, 2, (M, 1)))).astype(np.float32))
    out = poison((N, K), dtype)
    dW = rbq.qlinear_fp8_wgrad(torch_bf16(dy), aq, asc, out=out)
    assert dW is out
    ref, absum = dy.T.astype(np.float64) @ a, np.abs(dy).T.astype(np.float64) @ np.abs(a)
    got = dW.double().cpu().numpy()
    tol = (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23) * np.abs(ref) + (M / 16 + 8) * 2.0 ** -21 * absum
    assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) / tol))


# Wide tiles, narrow ones in several parts, and the last token alone in its slice.
@pytest.mark.parametrize("M,N,K", [(300, 4096, 4096), (4097, 512, 1040), (6000, 40, 48), (20001, 264, 272)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_weight_gradient_tiles_and_parts(M, N, K, dtype):
    test_weight_gradient(M, N, K, dtype)


def test_weight_gradient_is_the_difference_of_the_loss():
    """L(W) = <dY, X^ W^T> is linear in W: its difference along any D is <dW, D>."""
    g = np.random.default_rng(11)
    M, N, K = 200, 64, 272
    aq, asc, a = _random_codes(g, M, K)
    dy = synth.to_bf16(g.standard_normal((M, N)).astype(np.float32))
    dW = rbq.qlinear_fp8_wgrad(torch_bf16(dy), aq, asc, dtype=torch.float32).double().cpu().numpy()
    W, D = g.standard_normal((N, K)), g.standard_normal((N, K))
    diff = np.sum(dy * (a @ (W + D).T)) - np.sum(dy * (a @ W.T))
    absum = np.sum((np.abs(dy).T @ np.abs(a)) * np.abs(D))
    assert abs(np.sum(dW * D) - diff) <= ((M / 16 + 8) * 2.0 ** -21 + 2.0 ** -23) * absum


# ---- empty, strided, misplaced -----------------------------------------------------------

def test_empty():
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    q, s = rbq.quantize_fp8(x)
    assert q.shape == (0, 256) and s.shape == (0, 2)
    assert [tuple(t.shape) for t in rbq.quantize_fp8(x, activation="gelu", checkpoint=True)] == \
        [(0, 256), (0, 2), (0, 256), (0, 2)]
    w, ws = rbq.quantize_weights_fp8(torch.randn(32, 256, device="cuda"))
    assert rbq.qlinear_fp8(q, s, w, ws).shape == (0, 32)
    assert [tuple(t.shape) for t in rbq.quantize_weights_fp8(x, transposed=True)] == [(0, 256), (0, 2), (256, 0), (2, 0)]
    assert rbq.qlinear_fp8(w, torch.ones(32, 2, device="cuda").to(E8), q, s).shape == (32, 0)
    dy = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")
    dW = rbq.qlinear_fp8_wgrad(dy, q, s, out=poison((32, 256), torch.bfloat16))
    assert dW.shape == (32, 256) and not dW.any()
    assert rbq.gelu_backward_fp8(x, q, s).shape == (0, 256)


def test_binding_refusals():
    x = torch.randn(64, 256, device="cuda")
    q, s = rbq.quantize_fp8(x)
    w, ws = rbq.quantize_weights_fp8(x)
    dy = torch.randn(64, 32, device="cuda").bfloat16()
    for call in (lambda: rbq.quantize_fp8(x.t()), lambda: rbq.quantize_fp8(x[:, :128]), lambda: rbq.quantize_fp8(x[0]),
                 lambda: rbq.quantize_fp8(x[:, :40].contiguous()), lambda: rbq.quantize_fp8(x, activation="relu"),
                 lambda: rbq.quantize_fp8(x, checkpoint=True), lambda: rbq.quantize_fp8(x, codes=q[:32]),
                 lambda: rbq.quantize_fp8(x, scale=s[:, :1].contiguous()),
                 lambda: rbq.quantize_weights_fp8(x[:40], transposed=True),
                 lambda: rbq.qlinear_fp8(q, s[:32], w, ws), lambda: rbq.qlinear_fp8(q, s, w, s),
                 lambda: rbq.qlinear_fp8(q[:, :128].contiguous(), s[:, :1].contiguous(), w, ws),
                 lambda: rbq.qlinear_fp8(q, s, w, ws, out=torch.empty(64, 32, device="cuda").bfloat16()),
                 lambda: rbq.qlinear_fp8_wgrad(dy[:32], q, s),
                 lambda: rbq.qlinear_fp8_wgrad(dy[:, :12].contiguous(), q, s),
                 lambda: rbq.gelu_backward_fp8(dy, q, s),
                 lambda: rbq.linear_fp8(x, x[:40]), lambda: rbq.linear_fp8(x[:, :240], x)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: rbq.quantize_fp8(x.half()), lambda: rbq.quantize_fp8(x, codes=q.view(torch.uint8)),
                 lambda: rbq.qlinear_fp8(q.view(torch.uint8), s, w, ws), lambda: rbq.qlinear_fp8(q, s.float(), w, ws),
                 lambda: rbq.qlinear_fp8(q, s, w, ws, out=torch.empty(64, 64, device="cuda")),
                 lambda: rbq.qlinear_fp8_wgrad(dy.float(), q, s),
                 lambda: rbq.qlinear_fp8_wgrad(dy, q, s, dtype=torch.float16),
                 lambda: rbq.gelu_backward_fp8(x, q, s), lambda: rbq.linear_fp8(x.half(), x)):
        with pytest.raises(TypeError):
            call()
    flat = torch.randn(64 * 256 + 1, device="cuda")
    with pytest.raises(rbq.RBQError) as e:
        rbq.quantize_fp8(flat[1:].view(64, 256))
    assert e.value.code == rbq.RBQ_EALIGN


def test_unaligned_views_and_guard_rows():
    """Scales, Y and codes that start inside a larger buffer at the least
    alignment allowed, and nothing written outside them."""
    M, K, N = 300, 400, 264
    g = np.random.default_rng(3)
    x = _values(g, (M, K), "bf16")
    codes = torch.full((M * K + 64,), 0x11, dtype=torch.uint8, device="cuda")
    scales = torch.full((M * 4 + 8,), 0x22, dtype=torch.uint8, device="cuda")
    q, s = codes[16:16 + M * K].view(F8).view(M, K), scales[3:3 + 4 * M].view(E8).view(M, 4)
    rbq.quantize_fp8(torch_bf16(x), codes=q, scale=s)
    rq, re = oracle.fp8_encode(x)
    assert np.array_equal(_code_values(q), rq) and np.array_equal(_exponents(s), re)
    assert (codes[:16] == 0x11).all() and (codes[16 + M * K:] == 0x11).all()
    assert (scales[:3] == 0x22).all() and (scales[3 + 4 * M:] == 0x22).all()
    wq, wsc, w = _random_codes(g, N, K, 128)
    a = oracle.fp8_decode(rq, re)
    for rows in (M, 9):
        buf = torch.full((rows * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        for off in (1, 8, 16):
            buf.fill_(7.0)
            out = buf[off:off + rows * N].view(rows, N)
            rbq.qlinear_fp8(q[:rows], s[:rows], wq, wsc, out=out)
            _close(bf16_to_numpy(out), a[:rows] @ w.T, np.abs(a[:rows]) @ np.abs(w).T, K / 32)
            assert (buf[:off] == 7).all() and (buf[off + rows * N:] == 7).all()
    dy = synth.to_bf16(g.standard_normal((M, N)).astype(np.float32))
    for dtype in (torch.bfloat16, torch.float32):
        buf = torch.full((N * K + 64,), 7.0, dtype=dtype, device="cuda")
        off = 16 // buf.element_size()
        rbq.qlinear_fp8_wgrad(torch_bf16(dy), q, s, out=buf[off:off + N * K].view(N, K))
        ref, absum = dy.T.astype(np.float64) @ a, np.abs(dy).T.astype(np.float64) @ np.abs(a)
        _close(buf[off:off + N * K].view(N, K).double().cpu().numpy(), ref, absum, M / 16)
        assert (buf[:off] == 7).all() and (buf[off + N * K:] == 7).all()


def test_more_than_2_31_elements():
    T, d = 140000, 16384
    x = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, d, device="cuda").bfloat16()
    q, s = rbq.quantize_fp8(x)
    rq, rs = rbq.quantize_fp8(x[-3:].contiguous())
    assert torch.equal(q[-3:].view(torch.uint8), rq.view(torch.uint8))
    assert torch.equal(s[-3:].view(torch.uint8), rs.view(torch.uint8))
    del x
    w, ws = rbq.quantize_weights_fp8(torch.randn(128, d, device="cuda"))
    y = rbq.qlinear_fp8(q, s, w, ws)
    # both against the 64-bit values: layers of 140000 and of 259 tokens add
    # their products in different orders (the latter splits K), so that their
    # fp32 sums, each within the bound of the exact one, need not be equal
    a, b = _held(q[-3:], s[-3:]), _held(w, ws, 128)
    for rows in (y[-3:], rbq.qlinear_fp8(q[-259:].contiguous(), s[-259:].contiguous(), w, ws)[-3:]):
        _close(bf16_to_numpy(rows), a @ b.T, np.abs(a) @ np.abs(b).T, d / 32)
    assert not y[:-3].any()
    del q, s, y
    a, asc = rbq.quantize_fp8(torch.randn(70000, 16, device="cuda"))
    w, ws = rbq.quantize_weights_fp8(torch.randn(32768, 16, device="cuda"))
    y = rbq.qlinear_fp8(a, asc, w, ws)
    av, wv = _held(a[-2:], asc[-2:]), _held(w, ws, 128)
    for rows in (y[-2:], rbq.qlinear_fp8(a[-300:].contiguous(), asc[-300:].contiguous(), w, ws)[-2:]):
        _close(bf16_to_numpy(rows), av @ wv.T, np.abs(av) @ np.abs(wv).T, 1)


def test_native_and_checked_calls_agree():
    """The ordinary call (made by _rbq_call.so) and the one with buffers given
    (made in Python) are the same call."""
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(300, 400, device="cuda", generator=g).bfloat16()
    w = torch.nn.Parameter(torch.randn(272, 400, device="cuda", generator=g))
    dy = torch.randn(300, 272, device="cuda", generator=g).bfloat16()

    def like(*ts):
        return [torch.full_like(t.view(torch.uint8), 0x55).view(t.dtype) for t in ts]

    a = rbq.quantize_fp8(x, activation="gelu")
    ca, cs = like(*a)
    assert _same(a, rbq.quantize_fp8(x, activation="gelu", codes=ca, scale=cs)) and _same(a, (ca, cs))
    wq = rbq.quantize_weights_fp8(w)
    assert all(not t.requires_grad for t in wq)
    cw, cws = like(*wq)
    assert _same(wq, rbq.quantize_weights_fp8(w, codes=cw, scale=cws))
    y = rbq.qlinear_fp8(*a, *wq)
    assert torch.equal(y, rbq.qlinear_fp8(*a, *wq, out=torch.empty_like(y)))
    for dtype in (torch.bfloat16, torch.float32):
        dW = rbq.qlinear_fp8_wgrad(dy, *a, dtype=dtype)
        assert dW.dtype == dtype and torch.equal(dW, rbq.qlinear_fp8_wgrad(dy, *a, out=torch.empty_like(dW)))
    ck = rbq.quantize_fp8(x, activation="gelu", checkpoint=True)
    dx = rbq.gelu_backward_fp8(x, *ck[2:])
    assert torch.equal(dx, rbq.gelu_backward_fp8(x, *ck[2:], out=torch.empty_like(dx)))
    assert _same(ck[:2], a)


# ---- streams, graphs, repeated calls ---------------------------------------------------------

def _step(x, w, dy):
    a = rbq.quantize_fp8(x, activation="gelu", checkpoint=True)
    wq = rbq.quantize_weights_fp8(w, transposed=True)
    y = rbq.qlinear_fp8(*a[:2], *wq[:2])
    dh = rbq.qlinear_fp8(*rbq.quantize_fp8(dy), *wq[2:])
    dx = rbq.gelu_backward_fp8(dh, *a[2:], quantize=True)
    return (*a, *wq, y, dh, *dx, rbq.qlinear_fp8_wgrad(dy, *a[:2]))


def _same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def _step_inputs(M, K, N, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(M, K, device="cuda", generator=g).bfloat16(),
            torch.randn(N, K, device="cuda", generator=g) * 0.05,
            torch.randn(M, N, device="cuda", generator=g).bfloat16())


@pytest.mark.parametrize("M,K,N", [(5, 256, 384), (700, 1040, 272), (4200, 1040, 2048)])
def test_results_do_not_depend_on_the_run_or_the_stream(M, K, N):
    ins = [_step_inputs(M, K, N, i) for i in range(2)]
    ref = [_step(*i) for i in ins]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):                                   # two at once, workspaces and all
        with torch.cuda.stream(s1):
            a = _step(*ins[0])
        with torch.cuda.stream(s2):
            b = _step(*ins[1])
        torch.cuda.synchronize()
        assert _same(a, ref[0]) and _same(b, ref[1])


def test_stream_argument():
    x, w, dy = _step_inputs(300, 400, 272, 1)
    ref = _step(x, w, dy)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    a = rbq.quantize_fp8(x, activation="gelu", checkpoint=True, stream=st)
    wq = rbq.quantize_weights_fp8(w, transposed=True, stream=st)
    y = rbq.qlinear_fp8(*a[:2], *wq[:2], stream=st)
    dq = rbq.quantize_fp8(dy, stream=st)
    dh = rbq.qlinear_fp8(*dq, *wq[2:], stream=st)
    dx = rbq.gelu_backward_fp8(dh, *a[2:], quantize=True, stream=st)
    dW = rbq.qlinear_fp8_wgrad(dy, *a[:2], stream=st)
    st.synchronize()
    assert _same((*a, *wq, y, dh, *dx, dW), ref)


@pytest.mark.parametrize("M,K,N", [(3, 512, 1024), (700, 1040, 272), (4200, 1040, 2048)])
def test_captured_steps_share_nothing(M, K, N):
    """Two graphs of the whole step, replayed in turn and together on new inputs."""
    ins = [_step_inputs(M, K, N, i) for i in range(2)]
    _step(*ins[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in ins:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(_step(*i))
        graphs.append(gr)
    for seed in (10, 20):
        new = [_step_inputs(M, K, N, seed + i) for i in range(2)]
        ref = [_step(*n) for n in new]
        for i, n in zip(ins, new):
            for t, v in zip(i, n):
                t.copy_(v)
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        for gr, st in zip(graphs, (s1, s2)):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        assert _same(outs[0], ref[0]) and _same(outs[1], ref[1])


# ---- the layer as a differentiable function ----------------------------------------------------

@pytest.mark.parametrize("act", [None, "gelu"])
@pytest.mark.parametrize("shape,N,xdt,wdt", [((5, 256), 128, torch.bfloat16, torch.float32),
                                             ((2, 150, 400), 272, torch.float32, torch.bfloat16),
                                             ((64,), 16, torch.bfloat16, torch.bfloat16)])
def test_linear_gradients(shape, N, xdt, wdt, act):
    g = torch.Generator(device="cuda").manual_seed(N)
    K = shape[-1]
    X = (torch.randn(shape, device="cuda", generator=g) * 2).to(xdt).requires_grad_()
    W = (torch.randn(N, K, device="cuda", generator=g) * 0.1).to(wdt).requires_grad_()
    y = rbq.linear_fp8(X, W, activation=act)
    assert y.shape == (*shape[:-1], N) and y.dtype == torch.bfloat16
    dy = torch.randn(y.shape, device="cuda", generator=g).bfloat16()
    y.backward(dy)
    assert X.grad.dtype == xdt and W.grad.dtype == wdt and X.grad.shape == X.shape
    x2, dy2 = X.detach().reshape(-1, K), dy.reshape(-1, N)
    a = rbq.quantize_fp8(x2, activation=act)
    wq = rbq.quantize_weights_fp8(W.detach())
    av, wv = _held(*a), _held(*wq, 128)
    dyv = dy2.double().cpu().numpy()
    _close(y.detach().reshape(-1, N).double().cpu().numpy(), av @ wv.T, np.abs(av) @ np.abs(wv).T, K / 32)
    _close(W.grad.double().cpu().numpy(), dyv.T @ av, np.abs(dyv).T @ np.abs(av), len(dyv) / 16)
    dq = _held(*rbq.quantize_fp8(dy2.contiguous()))
    ref, absum = dq @ wv, np.abs(dq) @ np.abs(wv)
    tol = 2.0 ** -8 * np.abs(ref) + (N / 32 + 8) * 2.0 ** -21 * absum
    if act:
        xv = _held(*rbq.quantize_fp8(x2))
        slope = oracle.gelu_slope(xv)
        ref = ref * slope
        # dh is rounded to BF16 before the slope, the product once more
        tol = tol * np.abs(slope) * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref) + \
            4e-7 * (1 + np.abs(xv)) * (np.abs(dq @ wv) * (1 + 2.0 ** -8) + tol)
    got = X.grad.reshape(-1, K).double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) / tol))


def test_linear_partial_and_broadcast_gradients():
    X = torch.randn(40, 64, device="cuda").bfloat16()
    W = torch.randn(32, 64, device="cuda")
    wg = W.clone().requires_grad_()
    rbq.linear_fp8(X, wg).sum().backward()                   # an expanded dY
    xg = X.clone().requires_grad_()
    rbq.linear_fp8(xg, W, activation="gelu").sum().backward()
    both_x, both_w = X.clone().requires_grad_(), W.clone().requires_grad_()
    rbq.linear_fp8(both_x, both_w).sum().backward()
    assert torch.equal(both_w.grad, wg.grad) and xg.grad.isfinite().all()
    assert not rbq.linear_fp8(X, W).requires_grad
    # a shared weight and a transposed (strided) input
    xt = torch.randn(64, 40, device="cuda", requires_grad=True)
    w = W.clone().requires_grad_()
    (rbq.linear_fp8(xt.t(), w).sum() + rbq.linear_fp8(xt.t(), w).sum()).backward()
    one = W.clone().requires_grad_()
    x1 = xt.detach().clone().requires_grad_()
    rbq.linear_fp8(x1.t(), one).sum().backward()
    assert torch.equal(w.grad, 2 * one.grad) and torch.equal(xt.grad, 2 * x1.grad)


def test_linear_empty_batch():
    X = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    W = torch.randn(32, 64, device="cuda", requires_grad=True)
    rbq.linear_fp8(X, W).sum().backward()
    assert X.grad.shape == (0, 64) and not W.grad.any()


def test_training_step_in_a_graph():
    """Forward and backward of an MLP captured once; replays on new inputs equal eager steps."""
    g = torch.Generator(device="cuda").manual_seed(0)
    w1 = (torch.randn(512, 256, device="cuda", generator=g) * 0.05).requires_grad_()
    w2 = (torch.randn(256, 512, device="cuda", generator=g) * 0.05).requires_grad_()
    x = torch.randn(300, 256, device="cuda", generator=g).bfloat16()

    def step():
        y = rbq.linear_fp8(rbq.linear_fp8(x, w1), w2, activation="gelu")
        return torch.autograd.grad((y.float() ** 2).sum(), (w1, w2))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = step()
    for i in range(2):
        x.copy_(torch.randn(300, 256, device="cuda", generator=g).bfloat16())
        gr.replay()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


# ---- together with the rotation ------------------------------------------------------------------

def test_rotated_layer_end_to_end():
    """rotate_act, quantisers and product: the rotation cancels, so the layer is
    X W^T up to its two 8-bit roundings.  Each operand's relative error is at
    most 2^-4 per value and random between (uniform in a step: 2^-4 / sqrt 3 at
    most, 2.6e-2 measured on Gaussian values), so the result's is at most
    sqrt 2 * 2^-4 / sqrt 3 + the BF16 roundings of x', w' and y (3 * 2^-8)."""
    d, N, T = 1024, 512, 300
    g = np.random.default_rng(0)
    X, _ = synth.student_t_act(T, d, 1)
    W = synth.to_bf16(synth.gaussian_weights(g, N, d, outlier_frac=0.01))
    r = rbq.RPBH(d, 3)
    a = rbq.quantize_fp8(rbq.rotate_act(r, torch_bf16(X)))
    w = rbq.quantize_weights_fp8(rbq.rotate_act(r, torch_bf16(W)))
    y = bf16_to_numpy(rbq.qlinear_fp8(*a, *w))
    ref = X.astype(np.float64) @ W.astype(np.float64).T
    err = np.linalg.norm(y - ref) / np.linalg.norm(ref)
    print(f"rotated FP8 layer: rel. Frobenius error {err:.2e}")
    assert err <= np.sqrt(2) * 2.0 ** -4 / np.sqrt(3) + 3 * 2.0 ** -8
