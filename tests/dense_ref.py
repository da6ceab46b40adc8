"""Plain 64-bit forms of the 8-bit layer's operators, each with the bound of
its fp32 form's error.

u is half a step of fp32, relative.  A row's sum of H squares runs through at
most 8 multiply-adds, 5 shuffles, 32 warps, 16 CTAs and a few roundings
around: 80 u; rsqrt is within 2 steps, 4 u."""
import torch

U = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


def rounding(y, dtype):
    """What one rounding to dtype may be off by."""
    return half(dtype) * y.abs() + torch.finfo(dtype).smallest_normal * half(dtype)


def _norm(x, ex, w, offset, eps):
    """x / rms(x) * (w + offset) and its error bound, from x's bound."""
    H = x.shape[1]
    mean = (x * x).sum(1, keepdim=True) / H
    inv = 1 / torch.sqrt(mean + eps)
    f = w.double() + offset
    y = x * inv * f
    norm = x.norm(dim=1, keepdim=True)
    rel = torch.where(norm > 0, ex.norm(dim=1, keepdim=True) / norm, 0.0) + (40 + 4) * U
    return y, ex * inv * f.abs() + y.abs() * (rel + 4 * U)


def block(partials, residual, weight, eps, post_weight=None, gate=None, block_scale=1.0,
          residual_scale=1.0, weight_offset=0.0):
    """(y, its bound, r, its bound) in float64, before the outputs' rounding."""
    m = residual.shape[0]
    p = torch.stack([t.double() for t in partials])
    b, eb = p.sum(0), len(partials) * U * p.abs().sum(0)
    if post_weight is not None:
        b, eb = _norm(b, eb, post_weight, weight_offset, eps)
    if gate is not None:
        g = gate.double()
        g = g.view(1, -1) if g.dim() == 1 else g.repeat_interleave(m // g.shape[0], dim=0)
        eb = eb * g.abs() + (b * g).abs() * U
        b = b * g
    r1, r2 = residual_scale * residual.double(), block_scale * b
    r = r1 + r2
    er = abs(block_scale) * eb + 2 * U * (r1.abs() + r2.abs())
    y, ey = _norm(r, er, weight, weight_offset, eps)
    return y, ey, r, er


def quantise(x):
    """(q, scales) of 16-bit x [m, K]: decided in 64 bits, scales as fp32."""
    x = x.double()
    top = x.abs().amax(1, keepdim=True)
    fine = torch.isfinite(x).all(1, keepdim=True)
    q = torch.where(fine & (top > 0), torch.round(x * 127 / top), 0.0)
    s = torch.where(fine.squeeze(1), (top.squeeze(1).float() / torch.tensor(127.0, device=x.device)),
                    torch.nan)
    return q.to(torch.int8), s.float()


def product(x, xs, w, ws, act, chunk=1024):
    """(y, its bound) in float64 for sums that stay within 2^24."""
    s = torch.zeros((x.shape[0], w.shape[0]), dtype=torch.float64, device=x.device)
    for a in range(0, x.shape[1], chunk):
        s += (x[:, a:a + chunk].double() @ w[:, a:a + chunk].double().T)
    y = s * ws.double() * xs.double().unsqueeze(1)
    ey = 2 * U * y.abs() + 2.0 ** -149
    if act == "silu_mul":
        h = y.shape[1] // 2
        g, up = y[:, :h], y[:, h:]
        out = g * torch.sigmoid(g) * up
        # exp within 2 steps of an argument 2 u off, a sum, a quotient and a product
        ey = out.abs() * (2 * U * (2 + g.abs()) + 10 * U) + 2.0 ** -149
        return out, ey
    return y, ey
