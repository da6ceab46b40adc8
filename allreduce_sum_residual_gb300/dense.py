"""The calls of a dense layer in 8 bits on torch tensors: the norms after and
before a block, quantisation, and products of 8-bit integers.

Argument marshalling only, called through the package (``arn.ar_i8_matmul``
and so on).  As in experts.py a call on the current stream goes through the
binding in one step, and what that does not take goes the long way here,
which names what is wrong."""
import ctypes

import torch

from . import ACTS, AR_ACT_SILU_MUL, AR_TYPE_F32
from . import lib as _lib
from .experts import (_BF16, _F16, _F32, _TENSOR, _call, _device_of, _fast, _new, _option, _type_code,
                      _want)

_I8 = torch.int8
_TYPE_CODES = {torch.float32: AR_TYPE_F32, torch.bfloat16: 1, torch.float16: 2}


def _type16(t, name):
    """AR_TYPE_* of a 16-bit float tensor."""
    if t.dtype is not _BF16 and t.dtype is not _F16:
        raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    return _type_code(t, name)


def _gate(gate, dtype, m, H, dev):
    """(address, stride, rows of out that share a row) of a gate [H] or [g, H]."""
    if gate is None:
        return None, H, 1
    if not isinstance(gate, _TENSOR):
        raise TypeError("gate must be a torch.Tensor")
    if gate.dim() not in (1, 2) or gate.shape[-1] != H:
        raise ValueError(f"gate must be [{H}] or [g, {H}], got {tuple(gate.shape)}")
    if gate.dtype is not dtype:
        raise TypeError(f"gate must be {str(dtype)[6:]}, got {gate.dtype}")
    if gate.get_device() != dev:
        raise ValueError(f"gate must be on cuda:{dev}, got {gate.device}")
    if gate.stride(-1) != 1 and H > 1:
        raise ValueError("the rows of gate must be contiguous")
    g = gate.shape[0] if gate.dim() == 2 else 1
    if g < 1 and m > 0 or g > 0 and m % g != 0:
        raise ValueError(f"the {g} rows of gate must share the {m} rows evenly")
    stride = gate.stride(0) if g > 1 else H
    return gate.data_ptr(), stride, max(1, m // g) if g else 1


def _block_operands(partials, residual, weight, post_weight, gate):
    """What the two block norms share: (device, m, H, type, arguments up to
    the residual, residual's type)."""
    partials = list(partials)
    if len(partials) < 1:
        raise ValueError("need at least one partial")
    dev = _device_of(partials[0], "partials[0]")
    kind = _type16(partials[0], "partials[0]")
    dtype, shape = partials[0].dtype, partials[0].shape
    if len(shape) != 2:
        raise ValueError("partials must be [m, H]")
    m, H = shape
    addresses = (ctypes.c_void_p * len(partials))(
        *[_want(p, f"partials[{k}]", dtype, shape, dev) for k, p in enumerate(partials)])
    if isinstance(residual, _TENSOR) and residual.dtype is _F32:
        ra, rtype = _want(residual, "residual", _F32, shape, dev), AR_TYPE_F32
    else:
        ra, rtype = _want(residual, "residual", dtype, shape, dev), kind
    wa = _want(weight, "weight", dtype, (H,), dev)
    pa = None if post_weight is None else _want(post_weight, "post_weight", dtype, (H,), dev)
    ga, stride, rows = _gate(gate, dtype, m, H, dev)
    return dev, m, H, dtype, (addresses, len(partials), kind, pa, ga, stride, rows), ra, rtype, wa


def _output(given, name, dtype, shape, like, dev, stream):
    """(tensor, address) of an output: the caller's, or a new one."""
    if given is None:
        t = _new(like, shape, dtype, stream)
        return t, t.data_ptr()
    return given, _want(given, name, dtype, shape, dev)


def ar_block_rmsnorm(partials, residual, weight, eps, post_weight=None, gate=None, block_scale=1.0,
                     residual_scale=1.0, weight_offset=0.0, out=None, residual_out=None, stream=None):
    """The norm after a block, its gate and scale, the residual add and the
    norm before the next block in one pass: (out, residual_out).

        b = sum of the partials, normed by post_weight where given
        r = residual_scale * residual + block_scale * gate * b
        out = r * rsqrt(mean(r^2) + eps) * (weight + weight_offset)

    partials: n [m, H] bfloat16 or float16, rank order = reduce order.
    residual: [m, H] of their type or float32, as residual_out.  weight,
    post_weight: [H]; weight_offset is added to both in fp32.  gate: [H], or
    [g, H] whose g rows (whole 16 bytes apart) share the m rows evenly, in order."""
    if stream is None:
        r = _fast().block_rmsnorm(partials, residual, weight, eps, post_weight, gate, block_scale,
                                  residual_scale, weight_offset, False, out, None, residual_out)
        if r is not None:
            return r
    dev, m, H, dtype, head, ra, rtype, wa = _block_operands(partials, residual, weight, post_weight,
                                                            gate)
    out, oa = _output(out, "out", dtype, (m, H), residual, dev, stream)
    residual_out, oo = _output(residual_out, "residual_out", residual.dtype, (m, H), residual, dev,
                               stream)
    _call(_lib().ar_block_rmsnorm, "ar_block_rmsnorm", dev, stream, *head, block_scale, ra, rtype,
          residual_scale, wa, weight_offset, eps, m, H, oa, oo)
    return out, residual_out


def ar_block_rmsnorm_i8(partials, residual, weight, eps, post_weight=None, gate=None,
                        block_scale=1.0, residual_scale=1.0, weight_offset=0.0, q=None, scales=None,
                        residual_out=None, stream=None):
    """ar_block_rmsnorm with its output in 8 bits, for an 8-bit product:
    (q [m, H] int8, scales [m] float32, residual_out); q * scales is out."""
    if stream is None:
        r = _fast().block_rmsnorm(partials, residual, weight, eps, post_weight, gate, block_scale,
                                  residual_scale, weight_offset, True, q, scales, residual_out)
        if r is not None:
            return r
    dev, m, H, dtype, head, ra, rtype, wa = _block_operands(partials, residual, weight, post_weight,
                                                            gate)
    q, qa = _output(q, "q", _I8, (m, H), residual, dev, stream)
    scales, sa = _output(scales, "scales", _F32, (m,), residual, dev, stream)
    residual_out, oo = _output(residual_out, "residual_out", residual.dtype, (m, H), residual, dev,
                               stream)
    _call(_lib().ar_block_rmsnorm_i8, "ar_block_rmsnorm_i8", dev, stream, *head, block_scale, ra,
          rtype, residual_scale, wa, weight_offset, eps, m, H, qa, sa, oo)
    return q, scales, residual_out


def ar_i8_quantize(x, q=None, scales=None, stream=None):
    """x [m, K] bfloat16 or float16 in 8 bits: (q [m, K] int8, scales [m]
    float32 = max|x| / 127 of each row); rows of any stride of whole 16 bytes.
    Halves go to even, decided as exact arithmetic does."""
    if stream is None:
        r = _fast().i8_quantize(x, q, scales)
        if r is not None:
            return r
    dev = _device_of(x, "x")
    kind = _type16(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [m, K]")
    m, K = x.shape
    row, unit = x.stride()
    if unit != 1 and K > 1:
        raise ValueError("the rows of x must be contiguous")
    if m <= 1:
        row = K
    q, qa = _output(q, "q", _I8, (m, K), x, dev, stream)
    scales, sa = _output(scales, "scales", _F32, (m,), x, dev, stream)
    _call(_lib().ar_i8_quantize, "ar_i8_quantize", dev, stream, x.data_ptr(), kind, row, m, K, qa, sa)
    return q, scales


def ar_i8_matmul(x, x_scales, w, w_scales, act="none", dtype=_BF16, out=None, stream=None):
    """x [m, K] int8 times w [N, K] int8, times x_scales [m] and w_scales [N]
    float32: out [m, N] of `dtype` (bfloat16, float16 or float32; that of `out`
    where it is given), or [m, N/2] with act="silu_mul" (rows [0, N/2) of w
    gate rows [N/2, N))."""
    if out is not None and isinstance(out, _TENSOR):
        dtype = out.dtype
    if dtype not in _TYPE_CODES:
        raise TypeError(f"dtype must be float32, bfloat16 or float16, got {dtype}")
    kind = _TYPE_CODES[dtype]
    if stream is None:
        r = _fast().i8_matmul(x, x_scales, w, w_scales, ACTS.get(act, act), kind, out)
        if r is not None:
            return r
    dev = _device_of(x, "x")
    of_x = x.shape
    if len(of_x) != 2:
        raise ValueError("x must be [m, K]")
    m, K = of_x
    if not isinstance(w, _TENSOR) or w.dim() != 2:
        raise ValueError("w must be a tensor [N, K]")
    N = w.shape[0]
    xa = _want(x, "x", _I8, of_x, dev)
    sa = _want(x_scales, "x_scales", _F32, (m,), dev)
    wa = _want(w, "w", _I8, (N, K), dev)
    za = _want(w_scales, "w_scales", _F32, (N,), dev)
    act = _option(ACTS, act, "act")
    shape = (m, N // 2 if act == AR_ACT_SILU_MUL else N)
    out, oa = _output(out, "out", dtype, shape, x, dev, stream)
    _call(_lib().ar_i8_matmul, "ar_i8_matmul", dev, stream, xa, sa, wa, za, m, N, K, act, kind, oa)
    return out
