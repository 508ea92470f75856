"""The block-scaled FP8 layer where its numbers leave the ordinary range, and
where a lost token or a lost thread would not show in a sum's tolerance.

What can be exact is compared exactly; other bounds are derived at their test."""

import numpy as np
import pytest

import oracle
from parity import bf16_to_numpy

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


def _codes(values):
    return torch.from_numpy(np.asarray(values, dtype=np.float32)).cuda().to(F8)


def _scales(bytes_):
    return torch.from_numpy(np.asarray(bytes_).astype(np.uint8)).cuda().view(E8)


# ---- far scales -----------------------------------------------------------------------

@pytest.mark.parametrize("M", [1, 2, 3, 4, 9, 300, 4100])
def test_sums_of_large_codes_under_far_scales(M):
    """Sixteen products 448 * 448 under scales whose own product may be anything: a token
    has the same result alone and beside tokens of other scales, and a sum
    overflows only where the result does.  16 * 448^2 = 49 * 2^16 is a BF16 number, so
    every result in its normal range is exact."""
    eb = np.array([10, 127, 244, 100, 247, 20, 150])
    K, N = 128, 128 * len(eb)
    q = np.zeros((M, K))
    q[:, 16:32] = 448.0
    w = np.zeros((N, K))
    w[:, 16:32] = 448.0
    e = eb[np.arange(M) % len(eb)]
    y = bf16_to_numpy(rbq.qlinear_fp8(_codes(q), _scales(e[:, None]), _codes(w), _scales(eb[:, None])))
    exp = e[:, None] + eb[np.arange(N) // 128][None, :] - 254
    ref = np.ldexp(49.0 * 2 ** 16, exp)
    sure = ref >= 2.0 ** -126
    fits = ref <= float(torch.finfo(torch.bfloat16).max)
    assert (sure & fits).any()
    assert np.array_equal(y[sure & fits], ref[sure & fits])
    assert np.all(np.isinf(y[ref >= 2.0 ** 128])) and np.all(np.abs(y[~sure]) <= 2.0 ** -126)


# ---- the GELU's slope at the ends -------------------------------------------------------

@pytest.mark.parametrize("quantize", [False, True])
def test_gelu_backward_of_the_largest_values(quantize):
    """Where the checkpoint holds 2^128 (a code 256 under 2^120) the slope is 1 or 0
    as anywhere far out: dX is dH or 0, not NaN."""
    v = np.array([3.4e38, -3.4e38, 3.3e38, -3.3e38, 3.2e38, -3.2e38, 1e30, -1e30], dtype=np.float32)
    x = np.zeros((len(v), 128), dtype=np.float32)
    x[:, 3] = v
    xq, xs = rbq.quantize_fp8(torch.from_numpy(x).cuda())
    dh = torch.full((len(v), 128), 0.75, device="cuda").bfloat16()
    out = rbq.gelu_backward_fp8(dh, xq, xs, quantize=quantize)
    dx = bf16_to_numpy(out[0] if quantize else out)
    assert np.array_equal(dx[:, 3], np.where(v > 0, 0.75, 0.0))
    assert np.all(np.delete(dx, 3, 1) == 0.375)


def test_gelu_backward_under_every_scale():
    """Zero, the smallest, 1 and the largest code of both signs under all 256 scale bytes."""
    codes = np.array([0.0, 2.0 ** -9, 1.0, 448.0, -(2.0 ** -9), -1.0, -448.0, 0.0] * 16)
    q = _codes(np.tile(codes, (256, 1)))
    dx = bf16_to_numpy(rbq.gelu_backward_fp8(torch.ones(256, 128, device="cuda").bfloat16(), q,
                                             _scales(np.arange(256)[:, None])))
    assert np.isnan(dx[255]).all()
    x = np.ldexp(codes[None, :], np.arange(255)[:, None] - 127)
    ref = oracle.gelu_slope(np.clip(x, -1e30, 1e30))          # there the slope is 0 or 1 to 64 bits
    # half a BF16 step; the slope's own error, 4e-7 (1 + |x|) while it is neither 0 nor 1
    assert np.all(np.abs(dx[:255] - ref) <= 2.0 ** -8 * np.abs(ref) + 4e-7 * (1 + np.minimum(np.abs(x), 14)))
    far = np.abs(x) >= 14
    assert np.array_equal(dx[:255][far], (x[far] > 0).astype(np.float64))


# ---- operands and gradients that begin anywhere -----------------------------------------

def test_linear_takes_views_at_any_address():
    """X and W inside flat buffers, and a gradient that is a view into the gradient
    of a concatenation: none begins on a 16-byte boundary."""
    g = torch.Generator(device="cuda").manual_seed(1)
    T, K, N = 40, 64, 32
    x = torch.randn(T * K + 3, device="cuda", generator=g).bfloat16()
    w = torch.randn(N * K + 1, device="cuda", generator=g)
    head = torch.randn(5, device="cuda", generator=g).bfloat16().requires_grad_()
    up = torch.randn(5 + T * N, device="cuda", generator=g).bfloat16()

    def step(X, W):
        y = rbq.linear_fp8(X, W, activation="gelu")
        torch.cat([head, y.flatten()]).backward(up)
        return y

    xv, wv = x[3:].view(T, K).detach().requires_grad_(), w[1:].view(N, K).detach().requires_grad_()
    assert xv.data_ptr() % 16 and wv.data_ptr() % 16 and up[5:].data_ptr() % 16
    y = step(xv, wv)
    xc, wc = xv.detach().clone().requires_grad_(), wv.detach().clone().requires_grad_()
    assert torch.equal(y, step(xc, wc))
    assert torch.equal(xv.grad, xc.grad) and torch.equal(wv.grad, wc.grad)
    dy = up[5:].clone().view(T, N)
    y2 = rbq.linear_fp8(xc, wc, activation="gelu")
    gx, gw = torch.autograd.grad(y2, (xc, wc), dy)
    assert torch.equal(gx, xc.grad) and torch.equal(gw, wc.grad)


# ---- other threads ------------------------------------------------------------------------

def test_native_calls_release_the_interpreter_lock():
    """The entry points are replaced by PyGILState_Check, which takes no arguments and
    returns 1 if the calling thread holds the lock: the native binding takes that
    for an error code and answers None, and 0 for success.  Nothing is launched."""
    import ctypes

    from rotation_bit_ptq_b200 import _fp8
    native = _fp8._ordinary()
    x = torch.randn(32, 256, device="cuda").bfloat16()
    a, w = rbq.quantize_fp8(x), rbq.quantize_weights_fp8(x)
    check = ctypes.cast(ctypes.pythonapi.PyGILState_Check, ctypes.c_void_p).value
    native.bind(*[check] * 5)
    try:
        got = [native.quantize_fp8(x, 0, False), native.quantize_weights_fp8(x, True), native.qlinear_fp8(*a, *w),
               native.qlinear_fp8_wgrad(x, *a, False), native.gelu_backward_fp8(x, *a, True)]
    finally:
        _fp8._native = None
        _fp8._ordinary()                                  # binds librbq.so again
    assert [r is not None for r in got] == [True] * 5
    assert torch.equal(rbq.quantize_fp8(x)[0].view(torch.uint8), a[0].view(torch.uint8))


def test_threads_at_once():
    """Four threads, each with a stream of its own, get what each gets alone."""
    import threading

    def work(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn(100 + seed, 400, device="cuda", generator=g).bfloat16()
        w = (torch.randn(272, 400, device="cuda", generator=g) * 0.1).requires_grad_()
        out = []
        for _ in range(20):
            y = rbq.linear_fp8(x, w, activation="gelu")
            out.append((y.detach(), *torch.autograd.grad(y, w, torch.ones_like(y))))
        return out

    ref = [work(s) for s in range(4)]
    torch.cuda.synchronize()
    got = [None] * 4

    def run(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            got[i] = work(i)
            torch.cuda.current_stream().synchronize()

    ts = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    for r, o in zip(ref, got):
        assert all(torch.equal(p, q) for a, b in zip(r, o) for p, q in zip(a, b))


# ---- every token and every value counts ---------------------------------------------------

# Sums of small integers: exact in fp32 whatever their order, so that one lost,
# doubled or misplaced term shows.  (With heavy-tailed operands a few tokens carry
# the sum, and the others fall within the tolerance of a long sum.)

def _integers(g, n, d, rows, lo, hi):
    """Codes of integers lo..hi under scales 1, 2 and 4, and the values as fp64 on the GPU."""
    v = torch.randint(lo, hi + 1, (n, d), device="cuda", generator=g)
    e = torch.randint(0, 3, (-(-n // rows), -(-d // 128)), device="cuda", generator=g)
    s = torch.exp2(e.double()).repeat_interleave(rows, 0)[:n].repeat_interleave(128, 1)[:, :d]
    return v.float().to(F8), (e + 127).to(torch.uint8).view(E8), v.double() * s


# One token, the last one alone in its slice of 64, the last one missing from it;
# narrow and wide tiles, one part and several.
@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (63, 264, 272), (64, 264, 272), (65, 264, 272), (3001, 64, 128),
                                   (4033, 64, 128), (4031, 64, 128), (1561, 520, 400), (1599, 520, 400),
                                   (6017, 40, 48), (20033, 264, 272), (321, 4096, 4096), (319, 4096, 4096),
                                   (4097, 4096, 1040), (8001, 1536, 1536), (2047, 2048, 2064)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_weight_gradient_counts_every_token(M, N, K, dtype):
    """Token m's gradient is one entry of size 1 to 3 in column m % N, its codes are 1 to 3: without it
    row m % N differs everywhere.  The sums stay below 2^24."""
    g = torch.Generator(device="cuda").manual_seed(M + N)
    aq, asc, a = _integers(g, M, K, 1, 1, 3)
    rows = torch.arange(M, device="cuda")
    up = torch.randint(1, 4, (M,), device="cuda", generator=g).double()
    dy = torch.zeros(M, N, device="cuda", dtype=torch.bfloat16)
    dy[rows, rows % N] = up.bfloat16()
    ref = torch.zeros(N, K, device="cuda", dtype=torch.float64).index_add_(0, rows % N, a * up[:, None])
    dW = rbq.qlinear_fp8_wgrad(dy, aq, asc, dtype=dtype)
    assert float(ref.max()) < 2 ** 24
    assert torch.equal(dW, ref.to(dtype))


# Every kernel: dot products of one to four tokens, 16 to 256 tokens to a tile
# with K in one part and in several, and CTA pairs; whole and short last blocks of K.
@pytest.mark.parametrize("M,N,K", [(1, 1001, 2064), (2, 130, 144), (3, 136, 4112), (4, 1000, 2048), (15, 300, 1040),
                                   (9, 1000, 40000), (33, 1001, 656), (64, 512, 1536), (100, 520, 1040),
                                   (255, 500, 1552), (300, 1001, 1552), (513, 2056, 656), (40, 64, 33024),
                                   (4097, 3001, 272), (4100, 2600, 8960), (2000, 2048, 2064)])
def test_layer_counts_every_value(M, N, K):
    """Integers -2 to 2 under scales 1 to 4: the sums (below 2^24) are exact, the result their BF16 rounding."""
    g = torch.Generator(device="cuda").manual_seed(M + N)
    aq, asc, a = _integers(g, M, K, 1, -2, 2)
    wq, wsc, w = _integers(g, N, K, 128, -2, 2)
    assert 64 * K < 2 ** 24
    assert torch.equal(rbq.qlinear_fp8(aq, asc, wq, wsc), (a @ w.t()).to(torch.bfloat16))


# ---- the GELU's own error ---------------------------------------------------------------

def _gelu_preimage(b, lo, hi):
    """x in [lo, hi] with x Phi(x) = b, by bisection in 64 bits (monotone there)."""
    lo, hi = np.full_like(b, lo), np.full_like(b, hi)
    up = oracle.gelu(hi) > oracle.gelu(lo)
    for _ in range(100):
        mid = 0.5 * (lo + hi)
        left = (oracle.gelu(mid) < b) == up
        lo, hi = np.where(left, mid, lo), np.where(left, hi, mid)
    return 0.5 * (lo + hi)


@pytest.mark.parametrize("j", range(-6, 6))
def test_gelu_beside_every_border_of_the_codes(j):
    """The stated |error| <= 2.5e-7 |x| decides the code of an x whose GELU lies further than
    that from the border of two codes.  Such x are taken as close to the borders as fp32
    lets them, on both sides, and their codes compared with the exact ones.

    The bound: h = max(x, 0) - |x| t with t = 2^q.  The polynomial, its fp32
    evaluation included, is off by 8e-8 of Phi(-|x|) (the maximum over [0, 16], taken in 64 bits
    with every FMA rounded); ex2.approx by 2^-22 t, t <= 1/2; the last FMA by
    2^-24 |h|.  Over [0, 16] the sum is at most 2.2e-7 |x|."""
    bound, s = 2.5e-7, 2.0 ** j
    codes = torch.arange(0x7F, dtype=torch.uint8).view(F8).double().numpy()        # all that are >= 0
    borders = 0.5 * (codes[:-1] + codes[1:]) * s
    below = -borders[borders < 0.169]                  # the GELU's least value is -0.1700, at -0.752
    x0 = np.concatenate([_gelu_preimage(borders, 0.0, 1e6), _gelu_preimage(below, -0.75, 0.0),
                         _gelu_preimage(below, -6.0, -0.76)])
    step = bound * np.abs(x0) / np.maximum(np.abs(oracle.gelu_slope(x0)), 1e-3)
    x = np.concatenate([x0 + k * step for k in (1.1, -1.1, 2.0, -2.0)]).astype(np.float32)
    h = oracle.gelu(x.astype(np.float64))
    top = np.float32(440 * s)                          # in every block: it fixes the scale at s
    away = np.min(np.abs(h[:, None] - np.concatenate([-borders, borders])[None, :]), axis=1)
    x = x[(away > bound * np.abs(x)) & (np.abs(h) < top)]
    assert len(x) > 200
    x = np.pad(x, (0, -len(x) % 127)).reshape(-1, 127)
    x = np.concatenate([x, np.full((len(x), 1), top)], 1)
    q, sc = rbq.quantize_fp8(torch.from_numpy(x).cuda(), activation="gelu")
    rq, re = oracle.fp8_encode(oracle.gelu(x.astype(np.float64)))
    assert np.all(re == j) and np.all(sc.view(torch.uint8).cpu().numpy() == 127 + j)
    assert np.array_equal(q.double().cpu().numpy(), rq)


# ---- the two ways a call is made ---------------------------------------------------------

def _calls():
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(64, 256, device="cuda", generator=g)
    flat = torch.randn(64 * 256 + 4, device="cuda", generator=g)
    h = x.bfloat16()
    q, s = rbq.quantize_fp8(x)
    w, ws = rbq.quantize_weights_fp8(x[:48].contiguous())
    dy = torch.randn(64, 48, device="cuda", generator=g).bfloat16()
    q0, s0, h0 = q[:0], s[:0], h[:0]
    byte = torch.zeros(64 * 256 + 1, dtype=torch.uint8, device="cuda")
    odd = byte[1:].view(F8).view(64, 256)
    inputs = (x, h, x.half(), x.double(), x.t(), x[:, :128], x[0], x[:40], x[:, :40].contiguous(), x[:, :0], h0, x.cpu(),
              flat[4:].view(64, 256), flat[1:-3].view(64, 256), x.view(1, 64, 256), torch.nn.Parameter(x), None, [1.0])
    for t in inputs:
        for kw in ({}, {"activation": "gelu"}, {"activation": "gelu", "checkpoint": True}, {"checkpoint": True},
                   {"activation": "none"}, {"activation": "relu"}):
            yield rbq.quantize_fp8, (t,), kw
        for kw in ({}, {"transposed": True}, {"transposed": 1}):
            yield rbq.quantize_weights_fp8, (t,), kw
    pairs = ((q, s), (w, ws), (q0, s0), (q, s[:32]), (q, s[:, :1]), (q[:, :128].contiguous(), s[:, :1].contiguous()),
             (q.view(torch.uint8), s), (q, s.view(torch.uint8)), (q, s.float()), (q.cpu(), s.cpu()), (odd, s), (q.t(), s),
             (q[0], s[0]), (s, q), (None, s), (q, None))
    for a in pairs:
        for b in pairs:
            yield rbq.qlinear_fp8, (*a, *b), {}
        for t in (dy, h, dy.float(), dy[:32], dy[:, :12].contiguous(), dy.t(), dy[:0], dy[:, :0], h0, dy.cpu(), None):
            for kw in ({}, {"dtype": torch.float32}, {"dtype": torch.float16}):
                yield rbq.qlinear_fp8_wgrad, (t, *a), kw
            for kw in ({}, {"quantize": True}):
                yield rbq.gelu_backward_fp8, (t, *a), kw


def test_native_and_python_calls_accept_the_same(monkeypatch):
    """Whatever one way of making a call takes, refuses or answers, the other does."""
    from types import SimpleNamespace

    from rotation_bit_ptq_b200 import _fp8

    def outcome(f, args, kw):
        try:
            r = f(*args, **kw)
        except Exception as e:
            return type(e), None
        return None, r if isinstance(r, tuple) else (r,)

    calls = list(_calls())
    first = [outcome(*c) for c in calls]
    native = _fp8._ordinary()
    made = []

    def noted(name):
        def f(*args):
            r = getattr(native, name)(*args)
            made.append(r is not None)
            return r
        return f

    names = ("quantize_fp8", "quantize_weights_fp8", "qlinear_fp8", "qlinear_fp8_wgrad", "gelu_backward_fp8")
    monkeypatch.setattr(_fp8, "_native", SimpleNamespace(**{n: noted(n) for n in names}))
    natively = []
    for c in calls:
        made.clear()
        outcome(*c)
        natively.append(any(made))
    monkeypatch.setattr(_fp8, "_native", SimpleNamespace(**{n: lambda *a: None for n in names}))
    second = [outcome(*c) for c in calls]
    assert 50 < sum(natively) < len(calls) // 2
    for (e1, r1), (e2, r2), c, by in zip(first, second, calls, natively):
        what = (c[0].__name__, [getattr(t, "shape", t) for t in c[1]], c[2])
        assert e1 is e2, (*what, e1, e2)
        # (those without a row or a column may be left to Python)
        assert by == (e2 is None) or not all(t.numel() for t in c[1]), what
        if r1 is not None:
            assert len(r1) == len(r2) and all(a.dtype == b.dtype and a.shape == b.shape for a, b in zip(r1, r2)), what
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(r1, r2) if a.numel()), what


# ---- the weight gradient's workspace ----------------------------------------------------

# Panels of 15104 and 1280 columns, the second in several parts; of 1024 and 528, both in parts.
@pytest.mark.parametrize("M,N,K", [(70001, 16, 16384), (1000001, 40, 1552)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_weight_gradient_in_panels(M, N, K, dtype):
    """More than 2 GiB of BF16 values: panel by panel, exact as test_weight_gradient_counts_every_token."""
    g = torch.Generator(device="cuda").manual_seed(M + N)
    v = torch.randint(1, 4, (M, K), device="cuda", generator=g, dtype=torch.int8)
    e = torch.randint(0, 3, (M, -(-K // 128)), device="cuda", generator=g, dtype=torch.uint8)
    rows = torch.arange(M, device="cuda") % N
    up = torch.randint(1, 4, (M,), device="cuda", generator=g)
    dy = torch.zeros(M, N, device="cuda", dtype=torch.bfloat16)
    dy[torch.arange(M, device="cuda"), rows] = up.bfloat16()
    buf = torch.full((N + 2, K), 7.0, dtype=dtype, device="cuda")
    rbq.qlinear_fp8_wgrad(dy, v.float().to(F8), (e + 127).view(E8), out=buf[1:-1])
    assert (buf[0] == 7).all() and (buf[-1] == 7).all()
    for k in range(0, K, 128):
        a = v[:, k:k + 128].double() * torch.exp2(e[:, k // 128:k // 128 + 1].double())
        ref = torch.zeros(N, a.shape[1], device="cuda", dtype=torch.float64).index_add_(0, rows, a * up[:, None])
        assert float(ref.max()) < 2 ** 24 and torch.equal(buf[1:-1, k:k + 128], ref.to(dtype)), k


def test_weight_gradient_workspace_is_bounded():
    """300000 x 16384 values would take 9.8 GB as BF16; the call takes 2 GiB of the device's free memory (it
    stays in the library's pool) and what the driver adds."""
    M, N, K = 300000, 64, 16384
    q = torch.zeros(M, K, dtype=torch.uint8, device="cuda").view(F8)
    s = torch.full((M, K // 128), 127, dtype=torch.uint8, device="cuda").view(E8)
    dy = torch.ones(M, N, dtype=torch.bfloat16, device="cuda")
    out = torch.ones(N, K, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    rbq.qlinear_fp8_wgrad(dy, q, s, out=out)
    torch.cuda.synchronize()
    assert before - torch.cuda.mem_get_info()[0] <= (2 << 30) + (256 << 20)
    assert not out.any()


def test_captured_gradients_in_panels():
    """Two gradients of two panels each in one graph, replayed on new inputs."""
    M, N, K = 70001, 16, 16384
    g = torch.Generator(device="cuda").manual_seed(0)
    dy = torch.randn(M, N, device="cuda", generator=g).bfloat16()
    aq, asc, _ = _integers(g, M, 256, 1, -3, 3)
    aq = aq.view(torch.uint8).repeat(1, K // 256).view(F8)
    asc = asc.view(torch.uint8).repeat(1, K // 256).view(E8)
    rbq.qlinear_fp8_wgrad(dy, aq, asc)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = rbq.qlinear_fp8_wgrad(dy, aq, asc), rbq.qlinear_fp8_wgrad(dy, aq, asc, dtype=torch.float32)
    dy.copy_(torch.randn(M, N, device="cuda", generator=g).bfloat16())
    for _ in range(2):
        for o in out:
            o.zero_()
        gr.replay()
        ref = rbq.qlinear_fp8_wgrad(dy, aq, asc, dtype=torch.float32)
        assert torch.equal(out[1], ref) and torch.equal(out[0], ref.bfloat16())


# ---- large sizes ----------------------------------------------------------------------------

def test_more_than_2_31_weights_and_gradients():
    """The last rows of matrices of 2.3e9 values, against calls on those rows alone."""
    N, K = 140032, 16384
    tail = 256                                             # whole blocks of 128 rows
    w = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    w[-tail:] = torch.randn(tail, K, device="cuda").bfloat16()
    big = rbq.quantize_weights_fp8(w, transposed=True)
    small = rbq.quantize_weights_fp8(w[-tail:].contiguous(), transposed=True)
    cut = (big[0][-tail:], big[1][-2:], big[2][:, -tail:], big[3][:, -2:])
    for b, s in zip(cut, small):
        assert torch.equal(b.contiguous().view(torch.uint8), s.view(torch.uint8))
    assert not big[0][:-tail].view(torch.uint8).any() and not big[2][:, :-tail].view(torch.uint8).any()
    del big, small, cut
    xq, xs = rbq.quantize_fp8(w)
    big = rbq.gelu_backward_fp8(w, xq, xs, quantize=True)
    small = rbq.gelu_backward_fp8(w[-3:].contiguous(), xq[-3:].contiguous(), xs[-3:].contiguous(), quantize=True)
    for b, s in zip(big, small):
        assert torch.equal(b[-3:].view(torch.uint8), s.view(torch.uint8))
    del big
    # a gradient of 2.3e9 codes: all tokens but the last three have no weight
    dy = torch.zeros(N, 8, dtype=torch.bfloat16, device="cuda")
    dy[torch.arange(N - 3, N), torch.arange(3)] = 1.0
    dW = rbq.qlinear_fp8_wgrad(dy, xq, xs, dtype=torch.float32)
    held = xq[-3:].float() * xs[-3:].float().repeat_interleave(128, 1)
    assert torch.equal(dW[:3], held) and not dW[3:].any()


@pytest.mark.parametrize("M,N,K", [(1, 1000003, 16), (5, 1000003, 48), (300, 1000003, 16), (1000003, 3, 16),
                                   (1000003, 40, 144)])
def test_layers_of_very_long_sides(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M)
    aq, asc, a = _integers(g, M, K, 1, -2, 2)
    wq, wsc, w = _integers(g, N, K, 128, -2, 2)
    y = rbq.qlinear_fp8(aq, asc, wq, wsc)
    assert torch.equal(y, (a @ w.t()).to(torch.bfloat16))


@pytest.mark.parametrize("M,N,K", [(3, 1000000, 16), (1000001, 8, 16), (3, 8, 1000000 // 16 * 16)])
def test_gradients_of_very_long_sides(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M)
    aq, asc, a = _integers(g, M, K, 1, 1, 3)
    dy = torch.randint(0, 2, (M, N), device="cuda", generator=g)
    dW = rbq.qlinear_fp8_wgrad(dy.bfloat16(), aq, asc, dtype=torch.float32)
    assert torch.equal(dW, (dy.double().t() @ a).float())


# ---- the differentiable layer under torch's modes ---------------------------------------------

def test_linear_under_torchs_modes():
    """no_grad, inference_mode, autocast, a checkpointed segment, saved tensors kept on
    the CPU and a graph kept for a second backward pass change nothing."""
    from torch.utils.checkpoint import checkpoint
    g = torch.Generator(device="cuda").manual_seed(0)
    X = torch.randn(3, 50, 256, device="cuda", generator=g).bfloat16().requires_grad_()
    W = (torch.randn(272, 256, device="cuda", generator=g) * 0.1).requires_grad_()
    dy = torch.randn(3, 50, 272, device="cuda", generator=g).bfloat16()

    def layer(x, w):
        return rbq.linear_fp8(x, w, activation="gelu")

    y = layer(X, W)
    ref = torch.autograd.grad(y, (X, W), dy, retain_graph=True)
    again = torch.autograd.grad(y, (X, W), dy)
    assert all(torch.equal(a, b) for a, b in zip(ref, again))
    with torch.no_grad():
        assert torch.equal(layer(X, W), y) and not layer(X, W).requires_grad
    with torch.inference_mode():
        assert torch.equal(layer(X, W), y)
        assert torch.equal(rbq.qlinear_fp8(*rbq.quantize_fp8(X.flatten(0, 1), activation="gelu"),
                                           *rbq.quantize_weights_fp8(W)).view(y.shape), y)
    with torch.autocast("cuda", dtype=torch.bfloat16):
        got = torch.autograd.grad(layer(X, W), (X, W), dy)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    got = torch.autograd.grad(checkpoint(layer, X, W, use_reentrant=False), (X, W), dy)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    with torch.autograd.graph.save_on_cpu():
        y = layer(X, W)
    got = torch.autograd.grad(y, (X, W), dy)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
