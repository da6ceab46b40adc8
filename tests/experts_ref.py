"""Plain 64-bit forms of the expert-layer operators, for their tests.

Each also returns what its result's error bound needs: for a sum, the sum of
the terms' magnitudes, against which fp32 roundings count.
"""
import math

import torch

BF16 = 2.0 ** -8    # half a step of bf16, relative
F32 = 2.0 ** -24    # half a step of fp32, relative


def route(logits, k, bias=None, scoring="softmax", groups=1, topk_groups=None, group_score="max",
          renorm=True, scale=1.0):
    """(weights float64, ids) row by row, by sorting (choice, index)."""
    x = logits.double().cpu()
    m, E = x.shape
    topk_groups = groups if topk_groups is None else topk_groups
    gs = E // groups
    by_logit = bias is None and (group_score == "max" or topk_groups == groups)
    ws, out = [], []
    for r in range(m):
        row = x[r].tolist()
        if scoring == "softmax":
            top = max([v for v in row if not math.isnan(v)] + [-math.inf])
            shift = top if top > -math.inf else 0.0
            e = [0.0 if v == -math.inf else math.nan if math.isnan(v) or top == math.inf
                 else math.exp(v - shift) for v in row]
            total = sum(e)
            s = [v / total if total != 0 else 0.0 for v in e]
            if math.isnan(total):
                s = [math.nan] * E
        else:
            s = [math.nan if math.isnan(v) else 1 / (1 + math.exp(-v)) if v > -700 else 0.0
                 for v in row]
        b = [0.0] * E if bias is None else bias.double().cpu().tolist()
        c = [row[i] if by_logit else s[i] + b[i] for i in range(E)]
        c = [c[i] if row[i] > -math.inf and c[i] > -math.inf else -math.inf for i in range(E)]
        score = []
        for g in range(groups):
            best = sorted(c[g * gs:(g + 1) * gs], reverse=True)
            score.append(best[0] if group_score == "max" or groups == 1 else
                         best[0] + best[1] if best[1] > -math.inf else -math.inf)
        kept = sorted(range(groups), key=lambda g: (-score[g], g))[:topk_groups]
        cand = [i for i in range(E) if i // gs in kept]
        ids = sorted(cand, key=lambda i: (-c[i], i))[:k]
        w = [s[i] for i in ids]
        if renorm:
            t = sum(w)
            w = [v / t if t != 0 else 0.0 for v in w]
        ws.append([v * scale for v in w])
        out.append(ids)
    return torch.tensor(ws, dtype=torch.float64), torch.tensor(out, dtype=torch.int32)


def unpack(q, scales, zeros):
    """The weights as float64 [..., N, K]."""
    w = torch.stack((q.int() & 15, q.int() >> 4), dim=-1).flatten(-2).double()
    group = w.shape[-1] // scales.shape[-1]
    z = 8.0 if zeros is None else (zeros.int() & 15).double().repeat_interleave(group, -1)
    return (w - z) * scales.double().repeat_interleave(group, -1)


def product(x, q, scales, zeros):
    """x [r, K] times 4-bit weights [N, K/2]: (sums, error of an fp32 product).

    A matrix instruction adds 16 products to a running sum (at most 2^-23 of
    the magnitudes so far, truncation included), G/16 of them a group; the
    scale rounds once; the groups' sums pass K/128 adds at most, and up to
    128 joining warps and CTAs.  The magnitudes: sum |q - z| |s| |x|.  x
    itself is exact down to 2^-30 of its row's largest and off by at most
    2^-39 of that below, for weights of at most 15 |s|."""
    K = x.shape[1]
    group = K // scales.shape[-1]
    w = unpack(q, scales, zeros)
    x = x.double()
    roundings = 2 * group / 16 + 1 + K / 128 + 128
    tiny = 2.0 ** -39 * 15 * x.abs().amax(1, keepdim=True) * group * scales.double().abs().sum(1)
    return x @ w.T, roundings * F32 * (x.abs() @ w.abs().T) + tiny


def act(y, err, kind):
    """(result, error bound before the last rounding) of a product's epilogue."""
    if kind == "none":
        return y, err
    h = y.shape[-1] // 2
    gate, up, eg, eu = y[..., :h], y[..., h:], err[..., :h], err[..., h:]
    silu = gate * torch.sigmoid(gate)
    # |silu'| <= 1.1; exp, add, divide and multiply: at most 8 half steps.
    es = 1.1 * eg + 8 * F32 * silu.abs()
    return silu * up, es * up.abs() + silu.abs() * eu + es * eu + 2 * F32 * (silu * up).abs()


def close(got, ref, err):
    """A bf16 result against 64 bits: half a bf16 step of the value plus the
    error before that rounding (itself rounded along: 1 + 2^-8)."""
    tol = BF16 * ref.abs() + (1 + BF16) * err + 1e-38
    bad = ~((got.double() - ref).abs() <= tol)
    n = int(bad.sum())
    assert n == 0, (f"{n} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}: "
                    f"{got[bad][0].item()} for {ref[bad][0].item()}")


def combine(y, weights, shared, slots, rows, k):
    """(sum, magnitudes) of the weighted rows."""
    m = weights.shape[0]
    y = y.reshape(rows, -1).double()
    H = y.shape[1]
    acc = torch.zeros((m, H), dtype=torch.float64, device=weights.device)
    mag = torch.zeros_like(acc)
    if shared is not None:
        acc, mag = shared.double(), shared.double().abs()
    for j in range(k):
        at = (torch.arange(m, device=weights.device) * k + j if slots is None
              else slots[:, j].long())
        live = (at >= 0) & (at < rows)
        if not bool(live.any()):
            continue
        w = torch.where(live, weights[:, j].double(), 0.0).unsqueeze(1)
        v = torch.where(live.unsqueeze(1), y[at.clamp(0, rows - 1)], 0.0)
        acc = acc + w * v
        mag = mag + (w * v).abs()
    return acc, mag


def norm(r, err_r, weight, eps):
    """(out, error bound) of RMSNorm from r with error err_r: the square sum
    and its mean within 2^-15 (sums of at most 2^9 adds a thread and warp,
    plus the error of r, counted below), rsqrt within 2^-22, two multiplies."""
    ms = r.square().mean(1, keepdim=True)
    inv = 1 / torch.sqrt(ms + eps)
    w = weight.double()
    out = r * inv * w
    e_ms = (2 * r.abs() * err_r).mean(1, keepdim=True)  # of the mean square
    rel = 0.5 * e_ms / (ms + eps) + 2.0 ** -15
    return out, inv * w.abs() * err_r + out.abs() * rel
