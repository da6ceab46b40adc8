"""The expert-layer calls of libarnorm.so on torch tensors: routing, products
with 4-bit weights, the weighted sum of the experts' outputs.

Argument marshalling only, as in the package itself, which these functions
are called through (``arn.ar_route_experts`` and so on)."""
import torch

from . import (ACTS, AR_ACT_SILU_MUL, AR_OK, AR_TYPE_BF16, AR_TYPE_F16, AR_TYPE_F32, GROUP_SCORES,
               SCORES, ArError)
from . import lib as _lib

# The checks below run on every call of a decode step, where they cost more
# than the kernels: one combined test per tensor, the reasons only when it
# fails, and no torch helper that does more than it has to.

def _type_code(t, name):
    """AR_TYPE_* of a float tensor."""
    d = t.dtype
    if d is torch.bfloat16:
        return AR_TYPE_BF16
    if d is torch.float32:
        return AR_TYPE_F32
    if d is torch.float16:
        return AR_TYPE_F16
    raise TypeError(f"{name} must be float32, bfloat16 or float16, got {d}")


def _want(t, name, dtype, shape, device):
    """Checks one tensor of the expert-layer calls; returns its address."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and \
            t.device == device and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {str(dtype)[6:]}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _cuda_device(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device, got {t.device}")
    return t.device


def _option(table, value, name):
    """An option by its name or its AR_* number (the library checks the number)."""
    if isinstance(value, str):
        if value not in table:
            raise ValueError(f"{name} must be one of {', '.join(sorted(table))}, got {value!r}")
        return table[value]
    return int(value)


def _new(shape, dtype, device, stream):
    """An output tensor, in the memory of the stream that will write it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _on(device, fn, name, stream, *args):
    """Calls `fn` with its stream last and `device` current."""
    index = device.index
    if stream is None:
        # current_stream(device).cuda_stream, without the Stream object
        handle = torch._C._cuda_getCurrentRawStream(index)
    else:
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            st = fn(*args, handle)
    if st != AR_OK:
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
    dev = _cuda_device(logits, "logits")
    kind = _type_code(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be [m, E]")
    m, E = logits.shape
    if E > 1 and logits.stride(1) != 1:
        raise ValueError("the rows of logits must be contiguous")
    row = logits.stride(0) if m > 1 else E
    k = int(k)
    shape = (m, max(k, 0))
    b = None if bias is None else _want(bias, "bias", torch.float32, (E,), dev)
    if weights is None:
        weights = _new(shape, torch.float32, dev, stream)
        w = weights.data_ptr()
    else:
        w = _want(weights, "weights", torch.float32, shape, dev)
    if ids is None:
        ids = _new(shape, torch.int32, dev, stream)
        i = ids.data_ptr()
    else:
        i = _want(ids, "ids", torch.int32, shape, dev)
    _on(dev, _lib().ar_route_experts, "ar_route_experts", stream, logits.data_ptr(), kind, row, b, m,
        E, k, _option(SCORES, scoring, "scoring"), int(groups),
        int(groups if topk_groups is None else topk_groups),
        _option(GROUP_SCORES, group_score, "group_score"), 1 if renorm else 0, float(scale), w, i)
    return weights, ids


def _w4_operands(q, scales, zeros, K, lead, dev):
    """(N, group, addresses and type of scales and zeros) of 4-bit weights
    q [*lead, N, K/2]."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    if q.dim() != lead + 2:
        raise ValueError("q must be [E, N, K/2]" if lead else "q must be [N, K/2]")
    if not isinstance(scales, torch.Tensor) or scales.dim() != lead + 2:
        raise ValueError("scales must be a tensor of q's dimensions")
    shape = q.shape[:-1]
    ng = scales.shape[-1]
    if ng < 1 or K % ng != 0:
        raise ValueError(f"scales must hold one value per group of K = {K}, got {ng} a row")
    if q.shape[-1] * 2 != K:
        raise ValueError(f"q must have K/2 = {K / 2:g} bytes a row (x has K = {K}), got {q.shape[-1]}")
    kind = _type_code(scales, "scales")
    qa = _want(q, "q", torch.uint8, q.shape, dev)
    sa = _want(scales, "scales", scales.dtype, shape + (ng,), dev)
    za = None if zeros is None else _want(zeros, "zeros", torch.uint8, shape + (ng,), dev)
    return shape[-1], K // ng, qa, sa, kind, za


def ar_w4_matvec(x, q, scales, zeros=None, act="none", out=None, stream=None):
    """x [m, K] bf16 times 4-bit weights: out [m, N] bf16, or [m, N/2] with
    act="silu_mul" (rows [0, N/2) gate rows [N/2, N)).  m <= 64.

    q: [N, K/2] uint8, the low four bits hold the even k.  scales: [N, K/G]
    float32, bfloat16 or float16 with groups of G = 32, 64 or 128.  zeros:
    [N, K/G] uint8, or None for a zero point of 8."""
    dev = _cuda_device(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [m, K]")
    m, K = x.shape
    xa = _want(x, "x", torch.bfloat16, x.shape, dev)
    N, group, qa, sa, kind, za = _w4_operands(q, scales, zeros, K, 0, dev)
    act = _option(ACTS, act, "act")
    shape = (m, N // 2 if act == AR_ACT_SILU_MUL else N)
    if out is None:
        out = _new(shape, torch.bfloat16, dev, stream)
        oa = out.data_ptr()
    else:
        oa = _want(out, "out", torch.bfloat16, shape, dev)
    _on(dev, _lib().ar_w4_matvec, "ar_w4_matvec", stream, xa, qa, sa, kind, za, m, N, K, group, act,
        oa)
    return out


def ar_w4_matvec_experts(x, ids, q, scales, zeros=None, act="none", out=None, stream=None):
    """ar_w4_matvec with the weights of each token's experts: out [m, k, N]
    (or [m, k, N/2]) from x [m, K] (one row per token) or [m, k, K] (one per
    choice), ids [m, k] int32 and q [E, N, K/2].  A row whose id lies outside
    [0, E) is zero.  m * k <= 4096."""
    dev = _cuda_device(x, "x")
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be a tensor [m, k]")
    m, k = ids.shape
    ia = _want(ids, "ids", torch.int32, ids.shape, dev)
    if x.dim() not in (2, 3):
        raise ValueError("x must be [m, K] or [m, k, K]")
    per_pair = x.dim() == 3
    K = x.shape[-1]
    xa = _want(x, "x", torch.bfloat16, (m, k, K) if per_pair else (m, K), dev)
    N, group, qa, sa, kind, za = _w4_operands(q, scales, zeros, K, 1, dev)
    act = _option(ACTS, act, "act")
    shape = (m, k, N // 2 if act == AR_ACT_SILU_MUL else N)
    if out is None:
        out = _new(shape, torch.bfloat16, dev, stream)
        oa = out.data_ptr()
    else:
        oa = _want(out, "out", torch.bfloat16, shape, dev)
    _on(dev, _lib().ar_w4_matvec_experts, "ar_w4_matvec_experts", stream, xa, 1 if per_pair else 0,
        ia, m, k, qa, sa, kind, za, q.shape[0], N, K, group, act, oa)
    return out


def _combine_operands(y, weights, shared, slots):
    """(device, m, k, H, rows, addresses) of the combine calls."""
    dev = _cuda_device(y, "y")
    if not isinstance(weights, torch.Tensor) or weights.dim() != 2:
        raise ValueError("weights must be a tensor [m, k]")
    m, k = weights.shape
    wa = _want(weights, "weights", torch.float32, weights.shape, dev)
    if slots is None:
        if y.dim() != 3:
            raise ValueError("y must be [m, k, H] without slots")
        H = y.shape[2]
        rows = m * k
        ya = _want(y, "y", torch.bfloat16, (m, k, H), dev)
        sa = None
    else:
        if y.dim() != 2:
            raise ValueError("y must be [rows, H] with slots")
        rows, H = y.shape
        ya = _want(y, "y", torch.bfloat16, y.shape, dev)
        sa = _want(slots, "slots", torch.int32, (m, k), dev)
    ha = None if shared is None else _want(shared, "shared", torch.bfloat16, (m, H), dev)
    return dev, m, k, H, rows, ya, sa, wa, ha


def ar_combine(y, weights, shared=None, slots=None, out=None, stream=None):
    """The weighted sum of each token's expert outputs, as bf16 [m, H] (a
    rank's partial): shared + sum_j weights[:, j] y[slots[:, j]].

    y: [m, k, H], or [rows, H] with slots [m, k] int32 (a slot outside
    [0, rows) adds nothing).  weights: [m, k] float32.  shared: [m, H]."""
    dev, m, k, H, rows, ya, sa, wa, ha = _combine_operands(y, weights, shared, slots)
    if out is None:
        out = _new((m, H), torch.bfloat16, dev, stream)
        oa = out.data_ptr()
    else:
        oa = _want(out, "out", torch.bfloat16, (m, H), dev)
    _on(dev, _lib().ar_combine, "ar_combine", stream, ya, rows, sa, wa, ha, m, k, H, oa)
    return out


def ar_combine_rmsnorm(y, weights, residual, weight, eps, shared=None, slots=None, out=None,
                       residual_out=None, stream=None):
    """ar_combine's sum through the residual add and RMSNorm in one pass;
    residual, weight, eps and the outputs as in ar_rmsnorm.  Returns (out,
    residual_out)."""
    dev, m, k, H, rows, ya, sa, wa, ha = _combine_operands(y, weights, shared, slots)
    ra = _want(residual, "residual", torch.bfloat16, (m, H), dev)
    ga = _want(weight, "weight", torch.bfloat16, (H,), dev)
    if out is None:
        out = _new((m, H), torch.bfloat16, dev, stream)
        oa = out.data_ptr()
    else:
        oa = _want(out, "out", torch.bfloat16, (m, H), dev)
    if residual_out is None:
        residual_out = _new((m, H), torch.bfloat16, dev, stream)
        oo = residual_out.data_ptr()
    else:
        oo = _want(residual_out, "residual_out", torch.bfloat16, (m, H), dev)
    _on(dev, _lib().ar_combine_rmsnorm, "ar_combine_rmsnorm", stream, ya, rows, sa, wa, ha, ra, ga,
        float(eps), m, k, H, oa, oo)
    return out, residual_out
