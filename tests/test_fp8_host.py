"""The block-scaled FP8 layer without a GPU: the oracle's own pins, and every
refusal of the C ABI and of the binding (all checked before anything is
launched)."""

import ctypes

import numpy as np
import pytest

import oracle
import rotation_bit_ptq_b200 as rbq

torch = pytest.importorskip("torch")

FAKE, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004)     # never dereferenced
NONE, GELU = rbq.RBQ_ACT_NONE, rbq.RBQ_ACT_GELU


@pytest.fixture(scope="module")
def lib():
    return rbq.lib()


# ---- the oracle -----------------------------------------------------------------

def test_oracle_scale_exponent():
    for amax, e in ((448.0, 0), (np.nextafter(448.0, 500), 1), (1.75, -8), (1.7500001, -7), (1.0, -8), (0.875, -9),
                    (0.0, -117), (2.0 ** -200, -117), (float(np.finfo(np.float32).max), 120)):
        assert oracle.fp8_scale_exponent(amax) == e, amax


@pytest.mark.parametrize("rows,shape", [(1, (5, 300)), (128, (200, 400))])
def test_oracle_codes_are_pytorchs(rows, shape):
    g = np.random.default_rng(shape[0])
    x = g.standard_t(2, shape) * np.exp(g.normal(0, 4, shape))
    q, e = oracle.fp8_encode(x, rows)
    s = oracle.fp8_scales(e, rows, shape)
    assert np.array_equal(q, torch.from_numpy(x / s).to(torch.float8_e4m3fn).double().numpy())
    for i in range(e.shape[0]):
        for j in range(e.shape[1]):
            amax = np.abs(x[i * rows:(i + 1) * rows, j * 128:(j + 1) * 128]).max()
            assert 224.0 < amax / 2.0 ** e[i, j] <= 448.0


def test_oracle_non_finite_values_do_not_count():
    x = np.zeros((1, 256))
    x[0, 3], x[0, 4], x[0, 5] = np.inf, np.nan, 3.0
    q, e = oracle.fp8_encode(x)
    assert e.tolist() == [[-7, -117]] and np.isnan(q[0, 3]) and np.isnan(q[0, 4]) and q[0, 5] == 384.0
    assert np.all(q[0, 128:] == 0)


def test_oracle_gelu_slope_is_the_derivative():
    x = np.linspace(-8, 8, 4001)
    h = 1e-5
    d = (oracle.gelu(x + h) - oracle.gelu(x - h)) / (2 * h)
    # central differences: h^2/6 |f'''| <= 2e-11, and cancellation 2^-52 * 8 / h <= 2e-10
    assert np.max(np.abs(oracle.gelu_slope(x) - d)) < 1e-9


# ---- the C ABI's refusals ---------------------------------------------------------

def test_quantize_fp8_refusals(lib):
    f = lib.quantize_fp8
    bf = rbq.RBQ_BF16
    assert f(None, bf, 0, 64, NONE, None, None, None, None, None) == rbq.RBQ_OK
    for args in ((FAKE, 7, 4, 64, NONE, FAKE, FAKE, None, None), (FAKE, bf, -1, 64, NONE, FAKE, FAKE, None, None),
                 (FAKE, bf, 4, 0, NONE, FAKE, FAKE, None, None), (FAKE, bf, 4, 72, NONE, FAKE, FAKE, None, None),
                 (FAKE, bf, 4, 64, 2, FAKE, FAKE, None, None), (None, bf, 4, 64, NONE, FAKE, FAKE, None, None),
                 (FAKE, bf, 4, 64, NONE, None, FAKE, None, None), (FAKE, bf, 4, 64, NONE, FAKE, None, None, None),
                 (FAKE, bf, 4, 64, NONE, FAKE, FAKE, FAKE, FAKE),      # a checkpoint of what is already encoded
                 (FAKE, bf, 4, 64, GELU, FAKE, FAKE, FAKE, None), (FAKE, bf, 4, 64, GELU, FAKE, FAKE, None, FAKE)):
        assert f(*args, None) == rbq.RBQ_EINVAL, args
    for args in ((ODD, bf, 4, 64, NONE, FAKE, FAKE, None, None), (FAKE, bf, 4, 64, NONE, ODD, FAKE, None, None),
                 (FAKE, bf, 4, 64, GELU, FAKE, FAKE, ODD, FAKE)):
        assert f(*args, None) == rbq.RBQ_EALIGN, args


def test_quantize_weights_fp8_refusals(lib):
    f = lib.quantize_weights_fp8
    bf = rbq.RBQ_BF16
    assert f(None, bf, 0, 64, None, None, None, None, None) == rbq.RBQ_OK
    for args in ((FAKE, 3, 64, 64, FAKE, FAKE, None, None), (FAKE, bf, -1, 64, FAKE, FAKE, None, None),
                 (FAKE, bf, 64, 0, FAKE, FAKE, None, None), (FAKE, bf, 64, 40, FAKE, FAKE, None, None),
                 (FAKE, bf, 72, 64, FAKE, FAKE, FAKE, FAKE),           # the transpose's rows are not whole pieces
                 (FAKE, bf, 64, 64, FAKE, FAKE, FAKE, None), (FAKE, bf, 64, 64, FAKE, FAKE, None, FAKE),
                 (None, bf, 64, 64, FAKE, FAKE, None, None), (FAKE, bf, 64, 64, FAKE, None, None, None)):
        assert f(*args, None) == rbq.RBQ_EINVAL, args
    for args in ((ODD, bf, 64, 64, FAKE, FAKE, None, None), (FAKE, bf, 64, 64, ODD, FAKE, None, None),
                 (FAKE, bf, 64, 64, FAKE, FAKE, ODD, FAKE)):
        assert f(*args, None) == rbq.RBQ_EALIGN, args


def test_qlinear_fp8_refusals(lib):
    f = lib.qlinear_fp8
    assert f(None, None, None, None, 0, 8, 64, None, None) == rbq.RBQ_OK
    assert f(None, None, None, None, 8, 0, 64, None, None) == rbq.RBQ_OK
    for args in ((-1, 8, 64), (8, -1, 64), (8, 8, 0), (8, 8, 72), ((1 << 30) + 1, 8, 64), (8, (1 << 30) + 1, 64)):
        assert f(FAKE, FAKE, FAKE, FAKE, *args, FAKE, None) == rbq.RBQ_EINVAL, args
    for i in range(5):
        ptrs = [FAKE] * 5
        ptrs[i] = None
        assert f(*ptrs[:4], 8, 8, 64, ptrs[4], None) == rbq.RBQ_EINVAL, i
    assert f(ODD, FAKE, FAKE, FAKE, 8, 8, 64, FAKE, None) == rbq.RBQ_EALIGN
    assert f(FAKE, FAKE, ODD, FAKE, 8, 8, 64, FAKE, None) == rbq.RBQ_EALIGN
    assert f(FAKE, FAKE, FAKE, FAKE, 8, 8, 64, ctypes.c_void_p(0x10001), None) == rbq.RBQ_EALIGN


def test_qlinear_fp8_wgrad_refusals(lib):
    f = lib.qlinear_fp8_wgrad
    bf = rbq.RBQ_BF16
    assert f(None, None, None, 8, 0, 64, None, bf, None) == rbq.RBQ_OK
    for args in ((-1, 8, 64), (8, -8, 64), (8, 12, 64), (8, 8, 0), (8, 8, 72), ((1 << 30) + 1, 8, 64),
                 (8, (1 << 30) + 8, 64)):
        assert f(FAKE, FAKE, FAKE, *args, FAKE, bf, None) == rbq.RBQ_EINVAL, args
    assert f(FAKE, FAKE, FAKE, 8, 8, 64, FAKE, 2, None) == rbq.RBQ_EINVAL
    for i in range(4):
        ptrs = [FAKE] * 4
        ptrs[i] = None
        assert f(*ptrs[:3], 8, 8, 64, ptrs[3], bf, None) == rbq.RBQ_EINVAL, i
    for i in (0, 1, 3):
        ptrs = [FAKE] * 4
        ptrs[i] = ODD
        assert f(*ptrs[:3], 8, 8, 64, ptrs[3], bf, None) == rbq.RBQ_EALIGN, i


def test_gelu_backward_fp8_refusals(lib):
    f = lib.gelu_backward_fp8
    assert f(None, None, None, 0, 64, None, None, None, None) == rbq.RBQ_OK
    for args in ((-1, 64), (4, 0), (4, 24)):
        assert f(FAKE, FAKE, FAKE, *args, FAKE, None, None, None) == rbq.RBQ_EINVAL, args
    assert f(FAKE, FAKE, FAKE, 4, 64, FAKE, FAKE, None, None) == rbq.RBQ_EINVAL
    assert f(FAKE, FAKE, FAKE, 4, 64, FAKE, None, FAKE, None) == rbq.RBQ_EINVAL
    for i in range(4):
        ptrs = [FAKE] * 4
        ptrs[i] = None
        assert f(*ptrs[:3], 4, 64, ptrs[3], None, None, None) == rbq.RBQ_EINVAL, i
    for i in (0, 1, 3):
        ptrs = [FAKE] * 4
        ptrs[i] = ODD
        assert f(*ptrs[:3], 4, 64, ptrs[3], None, None, None) == rbq.RBQ_EALIGN, i
    assert f(FAKE, FAKE, FAKE, 4, 64, FAKE, ODD, FAKE, None) == rbq.RBQ_EALIGN


# ---- the binding's refusals of what is not on a GPU ----------------------------------

def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 64).to(torch.float8_e4m3fn), torch.ones(4, 1).to(torch.float8_e8m0fnu)
    for call in (lambda: rbq.quantize_fp8(x), lambda: rbq.quantize_weights_fp8(x), lambda: rbq.qlinear_fp8(q, s, q, s),
                 lambda: rbq.qlinear_fp8_wgrad(x, q, s), lambda: rbq.gelu_backward_fp8(x, q, s),
                 lambda: rbq.linear_fp8(x, x)):
        with pytest.raises(TypeError):
            call()


def test_fp8_blocks():
    assert [rbq.fp8_blocks(n) for n in (0, 1, 128, 129, 4096)] == [0, 1, 1, 2, 32]


def test_native_binding_leaves_other_calls_alone():
    """_rbq_call.so answers None -- make the call in Python -- for whatever is not
    an ordinary call, and raises nothing."""
    from rotation_bit_ptq_b200 import _fp8
    native = _fp8._ordinary()
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 64).to(torch.float8_e4m3fn), torch.ones(4, 1).to(torch.float8_e8m0fnu)
    for f, calls in ((native.quantize_fp8, ((x, 0, False), (None, 0, False), (x,), (x, "gelu", False))),
                     (native.quantize_weights_fp8, ((x, False), ([1.0], True), ())),
                     (native.qlinear_fp8, ((q, s, q, s), (1, 2, 3, 4), (q, s))),
                     (native.qlinear_fp8_wgrad, ((x, q, s, False), (None, q, s, False))),
                     (native.gelu_backward_fp8, ((x, q, s, True), (x, q, None, True)))):
        for args in calls:
            assert f(*args) is None, args
    with pytest.raises(TypeError):
        native.bind(1, 2)


def test_streams_of_another_device_are_refused():
    """Nothing is allocated or launched on a stream whose device is not the operands'."""
    from types import SimpleNamespace

    from rotation_bit_ptq_b200 import _fp8
    stream = SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=0)
    _fp8.check_stream_device(None, 0)
    _fp8.check_stream_device(stream, 1)
    with pytest.raises(ValueError):
        _fp8.check_stream_device(stream, 0)
    with pytest.raises(ValueError):
        _fp8._call("quantize_fp8", 0, stream, None, rbq.RBQ_BF16, 0, 64, NONE, None, None, None, None)
