"""The block-scaled FP8 layer: binding of quantize_fp8, quantize_weights_fp8,
qlinear_fp8, qlinear_fp8_wgrad and gelu_backward_fp8 (include/rbq.h), and
linear_fp8, the layer as a differentiable function.

Codes are torch.float8_e4m3fn and scales torch.float8_e8m0fnu tensors, so
``codes.float()`` times ``scale.float()`` of its block is the value held.
"""

import contextlib
import ctypes

from . import (RBQ_ACT_GELU, RBQ_ACT_NONE, RBQ_BF16, RBQ_F32, _ACTS, _check, _dtype_code, _need_cuda, _need_shape,
               check_same_device, lib)

BLOCK = 128


def fp8_blocks(n):
    """Scale blocks along n values."""
    return -(-int(n) // BLOCK)


def check_fp8_width(n, name, step=16):
    """Widths of FP8 rows: whole 16-byte pieces (pure Python, no device)."""
    if n <= 0 or n % step:
        raise ValueError(f"{name} must be a positive multiple of {step}, got {n}")


@contextlib.contextmanager
def _on(device, stream):
    """The operands' device current and, when a stream is given, the current
    stream too, so that what the call allocates belongs to the stream it is
    written on."""
    import torch
    with torch.cuda.device(device):
        with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
            yield


# A call on a few tokens is bound by the host.  The ordinary one -- plain
# contiguous CUDA tensors of the right types and shapes on the current device,
# on the current stream, with results to be allocated -- is made by _rbq_call.so
# (csrc/rbq_call.cpp), which returns None for any other and for one that fails.  Those
# are made here, with checks that word the error.
_native = None


def _ordinary():
    """The module _rbq_call, bound to librbq.so on first use."""
    global _native
    if _native is None:
        import torch  # noqa: F401  (loads the libraries _rbq_call.so links)

        from .build import built_for
        here = built_for()
        try:
            from . import _rbq_call
            if getattr(_rbq_call, "built_for", None) != here:
                raise ImportError(f"it was built for {getattr(_rbq_call, 'built_for', 'something else')}")
        except ImportError as e:
            raise RuntimeError(f"_rbq_call.so is missing or not built for {here}: build it with "
                               "`python -m rotation_bit_ptq_b200.build`") from e
        _rbq_call.bind(*(ctypes.cast(getattr(lib(), f), ctypes.c_void_p).value for f in (
            "quantize_fp8", "quantize_weights_fp8", "qlinear_fp8", "qlinear_fp8_wgrad", "gelu_backward_fp8")))
        _native = _rbq_call
    return _native


def _operand(t, name, dtype=None):
    """A contiguous CUDA tensor, of `dtype` if one is given; returns its device's index."""
    try:
        if t.is_cuda and t.is_contiguous() and (dtype is None or t.dtype is dtype):
            return t.get_device()
    except AttributeError:
        pass
    _need_cuda(t, name, dtype)
    return t.get_device()


def _matrix(t, name, dtype=None):
    """The same of a tensor with two dimensions."""
    try:
        if t.is_cuda and t.dim() == 2 and t.is_contiguous() and (dtype is None or t.dtype is dtype):
            return t.get_device()
    except AttributeError:
        pass
    dev = _operand(t, name, dtype)
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, got {t.dim()} dimensions")
    return dev


def check_stream_device(stream, dev):
    """A stream of the operands' device (a launch goes to the stream's device,
    which would read the operands through another's addresses)."""
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"the stream is of {stream.device}, the operands are of cuda:{dev}")


def _call(name, dev, stream, *args):
    """lib().name(*args, stream) with device number `dev` current."""
    import torch
    check_stream_device(stream, dev)
    fn = getattr(lib(), name)
    if stream is None and torch._C._cuda_getDevice() == dev:
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with _on(torch.device("cuda", dev), stream):
            rc = fn(*args, torch.cuda.current_stream().cuda_stream)
    if rc:
        _check(rc, name)


def _out(t, shape, dtype, like, stream, name, torch):
    """The caller's matrix `t` after its checks, or a new one on the device of `like`."""
    if t is None:
        if stream is None:
            return torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=like.device)
        check_stream_device(stream, like.get_device())
        with _on(like.device, stream):
            return torch.empty(shape, dtype=dtype, device=like.device)
    if _operand(t, name, dtype) != like.get_device():
        check_same_device(t, like)
    if t.shape != shape:
        _need_shape(t, shape, name)
    return t


def _codes(codes, scale, rows_per_scale, names, torch):
    """Checks a matrix of codes and its scales (`names`: what the caller calls
    them); returns its device's index and its shape."""
    dev = _matrix(codes, names[0], torch.float8_e4m3fn)
    if _matrix(scale, names[1], torch.float8_e8m0fnu) != dev:
        check_same_device(codes, scale)
    n, d = codes.shape
    if d <= 0 or d % 16:
        check_fp8_width(d, f"the width of {names[0]}")
    want = (n if rows_per_scale == 1 else -(-n // BLOCK), -(-d // BLOCK))
    if scale.shape != want:
        _need_shape(scale, want, names[1])
    return dev, n, d


_A, _W, _X = ("a_codes", "a_scale"), ("w_codes", "w_scale"), ("x_codes", "x_scale")


def quantize_fp8(X, activation=None, checkpoint=False, codes=None, scale=None, stream=None):
    """E4M3 codes [T, d] and E8M0 scales [T, ceil(d / 128)] of the rows of X
    (bfloat16 or float32), or of GELU(X) with activation='gelu'.

    checkpoint=True (with 'gelu') also returns the codes and scales of X
    itself, from which gelu_backward_fp8 takes the gradient: (codes, scale,
    x_codes, x_scale).  d a multiple of 16."""
    if codes is None and scale is None and stream is None and activation in _ACTS:
        r = (_native or _ordinary()).quantize_fp8(X, _ACTS[activation], bool(checkpoint))
        if r is not None:
            return r
    import torch
    dev = _matrix(X, "X")
    dtype = _dtype_code(X)
    if activation not in _ACTS:
        raise ValueError("activation must be None, 'none' or 'gelu'")
    act = _ACTS[activation]
    if checkpoint and act == RBQ_ACT_NONE:
        raise ValueError("checkpoint goes with an activation: without one the codes are X's own")
    T, d = X.shape
    check_fp8_width(d, "the width of X")
    blocks = (T, -(-d // BLOCK))
    codes = _out(codes, (T, d), torch.float8_e4m3fn, X, stream, "codes", torch)
    scale = _out(scale, blocks, torch.float8_e8m0fnu, X, stream, "scale", torch)
    if not checkpoint:
        _call("quantize_fp8", dev, stream, X.data_ptr(), dtype, T, d, act, codes.data_ptr(), scale.data_ptr(), None,
              None)
        return codes, scale
    x_codes = _out(None, (T, d), torch.float8_e4m3fn, X, stream, "x_codes", torch)
    x_scale = _out(None, blocks, torch.float8_e8m0fnu, X, stream, "x_scale", torch)
    _call("quantize_fp8", dev, stream, X.data_ptr(), dtype, T, d, act, codes.data_ptr(), scale.data_ptr(),
          x_codes.data_ptr(), x_scale.data_ptr())
    return codes, scale, x_codes, x_scale


def quantize_weights_fp8(W, transposed=False, codes=None, scale=None, stream=None):
    """E4M3 codes [N, K] and E8M0 scales [ceil(N / 128), ceil(K / 128)] of a
    weight matrix (bfloat16 or float32), one scale per 128 x 128 block.

    transposed=True also returns the codes and scales of W^T, the weights of
    the layer's input gradient: (codes, scale, codes_t [K, N], scale_t).
    K a multiple of 16, and N too when transposed."""
    if codes is None and scale is None and stream is None:
        r = (_native or _ordinary()).quantize_weights_fp8(W, bool(transposed))
        if r is not None:
            return r
    import torch
    dev = _matrix(W, "W")
    dtype = _dtype_code(W)
    N, K = W.shape
    check_fp8_width(K, "the width of W")
    if transposed and N:
        check_fp8_width(N, "the height of W (the width of its transpose)")
    codes = _out(codes, (N, K), torch.float8_e4m3fn, W, stream, "codes", torch)
    scale = _out(scale, (fp8_blocks(N), fp8_blocks(K)), torch.float8_e8m0fnu, W, stream, "scale", torch)
    if not transposed:
        _call("quantize_weights_fp8", dev, stream, W.data_ptr(), dtype, N, K, codes.data_ptr(), scale.data_ptr(), None,
              None)
        return codes, scale
    codes_t = _out(None, (K, N), torch.float8_e4m3fn, W, stream, "codes_t", torch)
    scale_t = _out(None, (fp8_blocks(K), fp8_blocks(N)), torch.float8_e8m0fnu, W, stream, "scale_t", torch)
    _call("quantize_weights_fp8", dev, stream, W.data_ptr(), dtype, N, K, codes.data_ptr(), scale.data_ptr(),
          codes_t.data_ptr() if N else None, scale_t.data_ptr() if N else None)
    return codes, scale, codes_t, scale_t


def qlinear_fp8(a_codes, a_scale, w_codes, w_scale, out=None, stream=None):
    """y[m, n] = sum_k (sa[m, k/128] qa[m, k]) (sw[n/128, k/128] qw[n, k]) as
    bfloat16 [M, N], on the codes of quantize_fp8 and quantize_weights_fp8."""
    if out is None and stream is None:
        y = (_native or _ordinary()).qlinear_fp8(a_codes, a_scale, w_codes, w_scale)
        if y is not None:
            return y
    import torch
    dev, M, K = _codes(a_codes, a_scale, 1, _A, torch)
    dev_w, N, K2 = _codes(w_codes, w_scale, BLOCK, _W, torch)
    if K != K2:
        raise ValueError("a_codes and w_codes disagree on K")
    if dev != dev_w:
        check_same_device(a_codes, w_codes)
    out = _out(out, (M, N), torch.bfloat16, a_codes, stream, "out", torch)
    _call("qlinear_fp8", dev, stream, a_codes.data_ptr(), a_scale.data_ptr(), w_codes.data_ptr(), w_scale.data_ptr(),
          M, N, K, out.data_ptr())
    return out


def qlinear_fp8_wgrad(dY, a_codes, a_scale, dtype=None, out=None, stream=None):
    """dW[n, k] = sum_m dY[m, n] (sa[m, k/128] qa[m, k]), the weight gradient
    of qlinear_fp8 from the bfloat16 dY [M, N] and the codes kept of the
    layer's input; bfloat16 (the default) or float32 [N, K].  N a multiple of 8.

    Takes a workspace of 2 M K bytes, at most 2 GiB (512 M bytes if that is
    more), from the library's memory pool, which keeps it for later calls: it
    is not torch's to reuse."""
    import torch
    if out is None and stream is None and dtype in (None, torch.bfloat16, torch.float32):
        dW = (_native or _ordinary()).qlinear_fp8_wgrad(dY, a_codes, a_scale, dtype is torch.float32)
        if dW is not None:
            return dW
    dev_y = _matrix(dY, "dY", torch.bfloat16)
    dev, M, K = _codes(a_codes, a_scale, 1, _A, torch)
    T, N = dY.shape
    if T != M:
        raise ValueError("dY and a_codes disagree on the number of tokens")
    if N:
        check_fp8_width(N, "the width of dY", 8)
    dtype = (torch.bfloat16 if out is None else out.dtype) if dtype is None else dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("the weight gradient is bfloat16 or float32")
    if dev != dev_y:
        check_same_device(dY, a_codes)
    out = _out(out, (N, K), dtype, dY, stream, "out", torch)
    _call("qlinear_fp8_wgrad", dev, stream, dY.data_ptr(), a_codes.data_ptr(), a_scale.data_ptr(), M, N, K,
          out.data_ptr(), RBQ_BF16 if dtype is torch.bfloat16 else RBQ_F32)
    return out


def gelu_backward_fp8(dH, x_codes, x_scale, quantize=False, out=None, stream=None):
    """dX = dH * (Phi(x) + x phi(x)) as bfloat16 [T, d], the GELU's backward
    pass from the 8-bit checkpoint of its input (quantize_fp8(...,
    checkpoint=True)); dH bfloat16.

    quantize=True also returns quantize_fp8(dX), for the product that follows:
    (dX, codes, scale)."""
    if out is None and stream is None:
        r = (_native or _ordinary()).gelu_backward_fp8(dH, x_codes, x_scale, bool(quantize))
        if r is not None:
            return r
    import torch
    dev_h = _matrix(dH, "dH", torch.bfloat16)
    dev, T, d = _codes(x_codes, x_scale, 1, _X, torch)
    if dH.shape != (T, d):
        _need_shape(dH, (T, d), "dH")
    if dev != dev_h:
        check_same_device(dH, x_codes)
    out = _out(out, (T, d), torch.bfloat16, dH, stream, "out", torch)
    if not quantize:
        _call("gelu_backward_fp8", dev, stream, dH.data_ptr(), x_codes.data_ptr(), x_scale.data_ptr(), T, d,
              out.data_ptr(), None, None)
        return out
    codes = _out(None, (T, d), torch.float8_e4m3fn, dH, stream, "codes", torch)
    scale = _out(None, x_scale.shape, torch.float8_e8m0fnu, dH, stream, "scale", torch)
    _call("gelu_backward_fp8", dev, stream, dH.data_ptr(), x_codes.data_ptr(), x_scale.data_ptr(), T, d,
          out.data_ptr(), codes.data_ptr(), scale.data_ptr())
    return out, codes, scale


_linear = None


def _rows(t):
    """The matrix [-1, t.shape[-1]], contiguous and on a 16-byte boundary.  A
    gradient may come as a view that begins anywhere (that of one part of a
    concatenation does), a weight as a piece of a flat buffer."""
    t = t.reshape(-1, t.shape[-1]).contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _linear_function():
    """The autograd function behind linear_fp8 (defined on first use: importing
    the package does not import torch)."""
    global _linear
    if _linear is not None:
        return _linear
    import torch
    from torch.autograd.function import once_differentiable

    class LinearFP8(torch.autograd.Function):
        @staticmethod
        def forward(ctx, X, W, activation):
            need_x, need_w = ctx.needs_input_grad[:2]
            x2 = _rows(X)
            gelu = _ACTS[activation] == RBQ_ACT_GELU
            keep_x = gelu and need_x
            aq, asc, *ck = quantize_fp8(x2, activation=activation, checkpoint=keep_x)
            wq, wsc, *wt = quantize_weights_fp8(_rows(W), transposed=need_x)
            y = qlinear_fp8(aq, asc, wq, wsc)
            ctx.save_for_backward(*((aq, asc) if need_w else (None, None)), *(wt or (None, None)),
                                  *(ck or (None, None)))
            ctx.x_shape, ctx.x_dtype, ctx.w_dtype = X.shape, X.dtype, W.dtype
            return y.view(*X.shape[:-1], W.shape[0])

        @staticmethod
        @once_differentiable
        def backward(ctx, dY):
            aq, asc, wt, wt_sc, xq, xsc = ctx.saved_tensors
            dy2 = _rows(dY)
            dX = dW = None
            if ctx.needs_input_grad[0]:
                dX = qlinear_fp8(*quantize_fp8(dy2), wt, wt_sc)
                if xq is not None:
                    dX = gelu_backward_fp8(dX, xq, xsc, out=dX)
                dX = dX.view(ctx.x_shape).to(ctx.x_dtype)
            if ctx.needs_input_grad[1]:
                dW = qlinear_fp8_wgrad(dy2, aq, asc, dtype=ctx.w_dtype)
            return dX, dW, None

    _linear = LinearFP8
    return _linear


def linear_fp8(X, W, activation=None):
    """act(X) W^T with both operands in block-scaled FP8: bfloat16 [..., N] from
    X [..., K] and W [N, K] (bfloat16 or float32), act = identity or 'gelu'.

    Differentiable in X and W.  What the backward pass needs is kept in 8
    bits: the codes of act(X) for dW, of X for the GELU's slope, and of W^T for
    dX (whose other operand, the incoming gradient, is quantised there).  W is
    quantised in every call.  N and K multiples of 16.  dX is rounded to bfloat16
    also for a float32 X, with 'gelu' before and after the slope; dW has W's
    type.  The backward pass takes qlinear_fp8_wgrad's workspace.  (rotate_act
    passes no gradient on: X of a layer on rotated inputs is where it ends.)"""
    import torch
    for t, name in ((X, "X"), (W, "W")):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        _dtype_code(t)
    if activation not in _ACTS:
        raise ValueError("activation must be None, 'none' or 'gelu'")
    if W.dim() != 2 or X.dim() < 1 or X.shape[-1] != W.shape[1]:
        raise ValueError(f"X [..., K] and W [N, K] are wanted, got {tuple(X.shape)} and {tuple(W.shape)}")
    check_fp8_width(W.shape[1], "K")
    check_fp8_width(W.shape[0], "N")
    check_same_device(X, W)
    return _linear_function().apply(X, W, activation)
