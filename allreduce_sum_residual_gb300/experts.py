"""The expert-layer calls of libarnorm.so on torch tensors: routing, products
with 4-bit weights, the weighted sum of the experts' outputs.

Argument marshalling only, as in the package itself, which these functions
are called through (``arn.ar_route_experts`` and so on).  A call on the
current stream goes through the binding (csrc/binding.cpp), which checks,
allocates and calls in one step; what that does not take (a given stream,
another device than the current one, anything wrong) goes the long way here,
which names what is wrong, and so does everything where the binding is not
built."""
import ctypes
import importlib.util
import operator
import warnings

import torch

from . import (ACTS, AR_ACT_SILU_MUL, AR_TYPE_BF16, AR_TYPE_F16, AR_TYPE_F32, GROUP_SCORES,
               SCORES, ArError)
from . import lib as _lib

_TENSOR, _F32, _BF16, _F16 = torch.Tensor, torch.float32, torch.bfloat16, torch.float16
_I32, _U8 = torch.int32, torch.uint8
_empty = torch.empty
_raw_stream, _current = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice

_native = None     # the binding
_bound_to = None   # the library whose entry points it has


class _LongWay:
    """In the binding's place where there is none for this Python and torch."""
    route_experts = w4_matvec = w4_matvec_experts = combine = combine_rmsnorm = block_rmsnorm = \
        i8_quantize = i8_matmul = bind = staticmethod(lambda *_: None)


def _load_native():
    from . import _build
    path = _build.binding_path(torch.__version__, torch.version.git_version or "")
    try:
        spec = importlib.util.spec_from_file_location(__package__ + "._binding", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        return module
    except ImportError as e:
        warnings.warn("the expert-layer calls go through ctypes, some 10 us a call slower: build their "
                      "binding with `python -c \"import __graft_entry__ as g; g.build()\"` "
                      f"({e})", RuntimeWarning, stacklevel=4)
        return _LongWay


def _fast():
    """The binding, with the entry points of the loaded library."""
    global _native, _bound_to
    lib = _lib()
    if lib is not _bound_to:
        if _native is None:
            _native = _load_native()
        _native.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in
                       (lib.ar_route_experts, lib.ar_w4_matvec, lib.ar_w4_matvec_experts,
                        lib.ar_combine, lib.ar_combine_rmsnorm, lib.ar_block_rmsnorm,
                        lib.ar_block_rmsnorm_i8, lib.ar_i8_quantize, lib.ar_i8_matmul)))
        _bound_to = lib
    return _native


def _type_code(t, name):
    """AR_TYPE_* of a float tensor."""
    d = t.dtype
    if d is _BF16:
        return AR_TYPE_BF16
    if d is _F32:
        return AR_TYPE_F32
    if d is _F16:
        return AR_TYPE_F16
    raise TypeError(f"{name} must be float32, bfloat16 or float16, got {d}")


def _want(t, name, dtype, shape, dev):
    """Checks one tensor against device number `dev`; returns its address."""
    if isinstance(t, _TENSOR) and t.dtype is dtype and t.shape == shape and \
            t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, _TENSOR):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {str(dtype)[6:]}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _device_of(t, name):
    """The number of the CUDA device that `t` is on."""
    if isinstance(t, _TENSOR):
        if t.is_cuda:
            return t.get_device()
        raise ValueError(f"{name} must be on a CUDA device, got {t.device}")
    raise TypeError(f"{name} must be a torch.Tensor")


_INT_MAX = 2 ** 31 - 1


def _whole(value, name):
    """A whole number for a C int, which ctypes would cut off to 32 bits."""
    v = operator.index(value)
    if -_INT_MAX - 1 <= v <= _INT_MAX:
        return v
    raise ValueError(f"{name} must be a 32-bit whole number, got {v}")


def _size(n):
    """A tensor's size for a C int: one that does not fit is above every limit."""
    return n if n <= _INT_MAX else _INT_MAX


def _option(table, value, name):
    """An option by its name or its AR_* number (the library checks the number)."""
    if isinstance(value, str):
        if value in table:
            return table[value]
        raise ValueError(f"{name} must be one of {', '.join(sorted(table))}, got {value!r}")
    return _whole(value, name)


def _new(like, shape, dtype, stream):
    """An output tensor, in the memory of the stream that will write it."""
    if stream is None:
        return _empty(shape, dtype=dtype, device=like.device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device)
    with torch.cuda.stream(stream):
        return _empty(shape, dtype=dtype, device=like.device)


def _call(fn, name, dev, stream, *args):
    """Calls `fn` with its stream last and device number `dev` current."""
    if stream is None:
        handle = _raw_stream(dev)
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if _current() == dev:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, handle)
    if st:
        raise ArError(st, name)


def ar_route_experts(logits, k, bias=None, scoring="softmax", groups=1, topk_groups=None,
                     group_score="max", renorm=True, scale=1.0, weights=None, ids=None,
                     stream=None):
    """The k experts of each token and their weights: (weights [m, k] float32,
    ids [m, k] int32), largest choice first.

    logits: [m, E] float32, bfloat16 or float16, rows of any stride.
    bias: [E] float32 or None, added to the scores for the choice only.
    scoring: "softmax" or "sigmoid".  groups, topk_groups (default: all),
    group_score ("max" or "top2"): only experts of the topk_groups best of
    `groups` runs of experts are chosen.  renorm: divide the weights by
    their sum; scale: then multiply by this.
    Equal choices go to the lowest index, decided as in 64 bits."""
    if stream is None:
        r = _fast().route_experts(logits, k, bias, SCORES.get(scoring, scoring), groups, topk_groups,
                                  GROUP_SCORES.get(group_score, group_score), renorm, scale,
                                  weights, ids)
        if r is not None:
            return r
    dev = _device_of(logits, "logits")
    kind = _type_code(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be [m, E]")
    m, E = logits.shape
    row, unit = logits.stride()
    if unit != 1 and E > 1:
        raise ValueError("the rows of logits must be contiguous")
    if m <= 1:
        row = E
    k = _whole(k, "k")
    groups = _whole(groups, "groups")
    topk_groups = groups if topk_groups is None else _whole(topk_groups, "topk_groups")
    scoring = _option(SCORES, scoring, "scoring")
    group_score = _option(GROUP_SCORES, group_score, "group_score")
    shape = (m, k if k > 0 else 0)
    b = None if bias is None else _want(bias, "bias", _F32, (E,), dev)
    if weights is None:
        weights = _new(logits, shape, _F32, stream)
        w = weights.data_ptr()
    else:
        w = _want(weights, "weights", _F32, shape, dev)
    if ids is None:
        ids = _new(logits, shape, _I32, stream)
        i = ids.data_ptr()
    else:
        i = _want(ids, "ids", _I32, shape, dev)
    _call(_lib().ar_route_experts, "ar_route_experts", dev, stream, logits.data_ptr(), kind, row, b,
          m, _size(E), k, scoring, groups, topk_groups, group_score, 1 if renorm else 0, scale, w, i)
    return weights, ids


def _w4_operands(q, scales, zeros, K, lead, dev):
    """(N, group, addresses and type of scales and zeros) of 4-bit weights
    q [*lead, N, K/2]."""
    if not isinstance(q, _TENSOR):
        raise TypeError("q must be a torch.Tensor")
    if not isinstance(scales, _TENSOR):
        raise TypeError("scales must be a torch.Tensor")
    of_q, of_s = q.shape, scales.shape
    if len(of_q) != lead + 2:
        raise ValueError("q must be [E, N, K/2]" if lead else "q must be [N, K/2]")
    if len(of_s) != lead + 2:
        raise ValueError("scales must be a tensor of q's dimensions")
    ng = of_s[-1]
    if ng < 1 or K % ng != 0:
        raise ValueError(f"scales must hold one value per group of K = {K}, got {ng} a row")
    if of_q[-1] * 2 != K:
        raise ValueError(f"q must have K/2 = {K / 2:g} bytes a row (x has K = {K}), got {of_q[-1]}")
    shape = (of_q[0], of_q[1], ng) if lead else (of_q[0], ng)
    kind = _type_code(scales, "scales")
    qa = _want(q, "q", _U8, of_q, dev)
    sa = _want(scales, "scales", scales.dtype, shape, dev)
    za = None if zeros is None else _want(zeros, "zeros", _U8, shape, dev)
    return of_q[-2], _size(K // ng), qa, sa, kind, za


def ar_w4_matvec(x, q, scales, zeros=None, act="none", out=None, stream=None):
    """x [m, K] bf16 times 4-bit weights: out [m, N] bf16, or [m, N/2] with
    act="silu_mul" (rows [0, N/2) gate rows [N/2, N)).  m <= 64.

    q: [N, K/2] uint8, the low four bits hold the even k.  scales: [N, K/G]
    float32, bfloat16 or float16 with groups of G = 32, 64 or 128.  zeros:
    [N, K/G] uint8, or None for a zero point of 8."""
    if stream is None:
        r = _fast().w4_matvec(x, q, scales, zeros, ACTS.get(act, act), out)
        if r is not None:
            return r
    dev = _device_of(x, "x")
    of_x = x.shape
    if len(of_x) != 2:
        raise ValueError("x must be [m, K]")
    m, K = of_x
    xa = _want(x, "x", _BF16, of_x, dev)
    N, group, qa, sa, kind, za = _w4_operands(q, scales, zeros, K, 0, dev)
    act = _option(ACTS, act, "act")
    shape = (m, N // 2 if act == AR_ACT_SILU_MUL else N)
    if out is None:
        out = _new(x, shape, _BF16, stream)
        oa = out.data_ptr()
    else:
        oa = _want(out, "out", _BF16, shape, dev)
    _call(_lib().ar_w4_matvec, "ar_w4_matvec", dev, stream, xa, qa, sa, kind, za, m, N, K, group,
          act, oa)
    return out


def ar_w4_matvec_experts(x, ids, q, scales, zeros=None, act="none", first=0, out=None,
                         stream=None):
    """ar_w4_matvec with the weights of each token's experts: out [m, k, N]
    (or [m, k, N/2]) from x [m, K] (one row per token) or [m, k, K] (one per
    choice), ids [m, k] int32 and q [E, N, K/2], experts first .. first + E -
    1 of the layer.  A row whose id is none of these is zero.  m * k <=
    4096."""
    if stream is None:
        r = _fast().w4_matvec_experts(x, ids, q, scales, zeros, ACTS.get(act, act), first, out)
        if r is not None:
            return r
    dev = _device_of(x, "x")
    if not isinstance(ids, _TENSOR) or ids.dim() != 2:
        raise ValueError("ids must be a tensor [m, k]")
    of_ids, of_x = ids.shape, x.shape
    m, k = of_ids
    ia = _want(ids, "ids", _I32, of_ids, dev)
    per_pair = len(of_x) == 3
    if not per_pair and len(of_x) != 2:
        raise ValueError("x must be [m, K] or [m, k, K]")
    K = of_x[-1]
    xa = _want(x, "x", _BF16, (m, k, K) if per_pair else (m, K), dev)
    N, group, qa, sa, kind, za = _w4_operands(q, scales, zeros, K, 1, dev)
    act, first = _option(ACTS, act, "act"), _whole(first, "first")
    shape = (m, k, N // 2 if act == AR_ACT_SILU_MUL else N)
    if out is None:
        out = _new(x, shape, _BF16, stream)
        oa = out.data_ptr()
    else:
        oa = _want(out, "out", _BF16, shape, dev)
    _call(_lib().ar_w4_matvec_experts, "ar_w4_matvec_experts", dev, stream, xa,
          1 if per_pair else 0, ia, m, _size(k), qa, sa, kind, za, first, _size(q.shape[0]), N, K,
          group, act, oa)
    return out


def _combine_operands(y, weights, shared, slots):
    """(device, m, k, H, rows, addresses) of the combine calls."""
    dev = _device_of(y, "y")
    if not isinstance(weights, _TENSOR) or weights.dim() != 2:
        raise ValueError("weights must be a tensor [m, k]")
    of_w, of_y = weights.shape, y.shape
    m, k = of_w
    wa = _want(weights, "weights", _F32, of_w, dev)
    if slots is None:
        if len(of_y) != 3:
            raise ValueError("y must be [m, k, H] without slots")
        H = of_y[2]
        rows = m * k
        ya = _want(y, "y", _BF16, (m, k, H), dev)
        sa = None
    else:
        if len(of_y) != 2:
            raise ValueError("y must be [rows, H] with slots")
        rows, H = of_y
        ya = _want(y, "y", _BF16, of_y, dev)
        sa = _want(slots, "slots", _I32, of_w, dev)
    ha = None if shared is None else _want(shared, "shared", _BF16, (m, H), dev)
    return dev, m, k, H, rows, ya, sa, wa, ha


def ar_combine(y, weights, shared=None, slots=None, out=None, stream=None):
    """The weighted sum of each token's expert outputs, as bf16 [m, H] (a
    rank's partial): shared + sum_j weights[:, j] y[slots[:, j]].

    y: [m, k, H], or [rows, H] with slots [m, k] int32 (a slot outside
    [0, rows) adds nothing).  weights: [m, k] float32.  shared: [m, H]."""
    if stream is None:
        r = _fast().combine(y, weights, shared, slots, out)
        if r is not None:
            return r
    dev, m, k, H, rows, ya, sa, wa, ha = _combine_operands(y, weights, shared, slots)
    shape = (m, H)
    if out is None:
        out = _new(y, shape, _BF16, stream)
        oa = out.data_ptr()
    else:
        oa = _want(out, "out", _BF16, shape, dev)
    _call(_lib().ar_combine, "ar_combine", dev, stream, ya, rows, sa, wa, ha, m, _size(k), H, oa)
    return out


def ar_combine_rmsnorm(y, weights, residual, weight, eps, shared=None, slots=None, out=None,
                       residual_out=None, stream=None):
    """ar_combine's sum through the residual add and RMSNorm in one pass;
    residual, weight, eps and the outputs as in ar_rmsnorm.  Returns (out,
    residual_out)."""
    if stream is None:
        r = _fast().combine_rmsnorm(y, weights, residual, weight, eps, shared, slots, out,
                                    residual_out)
        if r is not None:
            return r
    dev, m, k, H, rows, ya, sa, wa, ha = _combine_operands(y, weights, shared, slots)
    shape = (m, H)
    ra = _want(residual, "residual", _BF16, shape, dev)
    ga = _want(weight, "weight", _BF16, (H,), dev)
    if out is None:
        out = _new(y, shape, _BF16, stream)
        oa = out.data_ptr()
    else:
        oa = _want(out, "out", _BF16, shape, dev)
    if residual_out is None:
        residual_out = _new(y, shape, _BF16, stream)
        oo = residual_out.data_ptr()
    else:
        oo = _want(residual_out, "residual_out", _BF16, shape, dev)
    _call(_lib().ar_combine_rmsnorm, "ar_combine_rmsnorm", dev, stream, ya, rows, sa, wa, ha, ra, ga,
          eps, m, _size(k), H, oa, oo)
    return out, residual_out
