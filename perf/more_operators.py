"""The operators of a layer in 8 bits, as cases to measure.

Three operators: the norms after and before a block with its gate and
residual scale (also with its output in 8 bits), the quantisation of
activations with a scale for each token, and the product of 8-bit integers
with scales for each token and channel.  ``run`` computes each in its plain
form (elementary torch operations) or, where ``own`` is true, through the
package's entry points.  What is quantised goes through the product that
reads it.
"""
import math

import torch

own = False

EPS = 1e-6
TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


# ---------------------------------------------------------------- cases

def _norms(name, m, H, n, post=True, gate="none", sequences=1, residual="bfloat16", block_scale=1.0,
           residual_scale=1.0, offset=0.0, dtype="bfloat16"):
    return dict(name=name, op="norms", m=m, H=H, n=n, post=post, gate=gate, sequences=sequences,
                residual=residual, block_scale=block_scale, residual_scale=residual_scale,
                offset=offset, dtype=dtype)


def _norms_linear(name, N, act="none", **norms):
    return dict(_norms(name, **norms), op="norms_linear", N=N, act=act)


def _linear(name, m, K, N, act="none", dtype="bfloat16"):
    return dict(name=name, op="linear", m=m, K=K, N=N, act=act, dtype=dtype)


def _matmul(name, m, K, N, act="none", dtype="bfloat16"):
    return dict(name=name, op="matmul", m=m, K=K, N=N, act=act, dtype=dtype)


def listed():
    return [
        # The end of a block in a decode step: a small batch, eight ranks' partials, a norm after
        # the block and one before the next.
        _norms("norms_decode", 16, 7168, 8, offset=1.0),
        # The same for a long prompt on one rank, with a gain for each channel of the block.
        _norms("norms_prompt", 8192, 6144, 1, gate="channel", residual_scale=0.5),
        # Odd sizes: sequences of one batch, each with its own gate (rows of a wider tensor), a
        # residual kept in fp32 and no norm after the block.
        _norms("norms_ragged", 1023, 5128, 3, post=False, gate="sequence", sequences=3,
               residual="float32", block_scale=0.22, dtype="float16"),
        # A decode step from the epilogue in 8 bits into the next projection.
        _norms_linear("norms_linear_decode", 8192, m=8, H=6144, n=4),
        # A prompt's epilogue in 8 bits into the gate and up projections.
        _norms_linear("norms_linear_prompt", 8192, m=2048, H=4096, n=2, gate="token",
                      act="silu_mul"),
        # One token through a square projection of the decode hidden size.
        _linear("linear_token", 1, 7168, 7168),
        # A prompt through a down projection: quantised rows, then the product.
        _linear("linear_prompt", 4096, 16384, 6144),
        # A ragged batch, quantised and multiplied.
        _linear("linear_ragged", 77, 5120, 1000, dtype="float16"),
        # A decode batch through a gate-up projection with its activation: the weights are read once.
        _matmul("matmul_gate_up", 32, 6144, 32768, act="silu_mul"),
        # A larger decode batch, or a short chunk of a prompt.
        _matmul("matmul_chunk", 192, 8192, 8192),
        # Odd sizes: a K that ends inside a tile, an odd number of outputs and tokens, fp32 out.
        _matmul("matmul_ragged", 333, 4112, 1001, dtype="float32"),
        # A long prompt through a gate-up projection.
        _matmul("matmul_prompt", 8192, 6144, 16384, act="silu_mul"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norms", "norms", "norms_linear", "linear", "matmul", "matmul"))
    m = _log(rng, 1, 8192)
    act = rng.choice(("none", "silu_mul"))
    dtype = rng.choice(("bfloat16", "bfloat16", "float16"))
    if op in ("norms", "norms_linear"):
        gate = rng.choice(("none", "channel", "sequence", "token"))
        sequences = 1
        if gate == "sequence":
            sequences = rng.randint(1, min(m, 8))
            m = max(1, m // sequences) * sequences
        H = 8 * _log(rng, 128, 2048) if op == "norms" else 16 * _log(rng, 64, 512)
        n = rng.randint(1, 8)
        while m * H * (n + 3) > 8192 * 6144 * 4 and n > 1:
            n -= 1
        H = min(H, 16 * (8192 * 6144 // m // 16))
        norms = dict(m=m, H=H, n=n, post=rng.random() < 0.6, gate=gate, sequences=sequences,
                     residual=rng.choice((dtype, dtype, "float32")),
                     block_scale=rng.choice((1.0, 1.0, 0.22)),
                     residual_scale=rng.choice((1.0, 1.0, 0.5)), offset=rng.choice((0.0, 1.0)),
                     dtype=dtype)
        if op == "norms":
            c = _norms(None, **norms)
        else:
            c = _norms_linear(None, 2 * _log(rng, 128, 4096), act, **norms)
    else:
        K, N = 16 * _log(rng, 32, 768), _log(rng, 256, 16384)
        if op == "matmul":
            dtype = rng.choice((dtype, "float32"))
        N = min(N, 8192 * 16384 * 6144 // (m * K))
        c = (_matmul if op == "matmul" else _linear)(
            None, m, K, N + N % 2 if act == "silu_mul" else N, act, dtype)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _weights8(g, N, K):
    """8-bit weights [N, K] and their channels' scales, which make the outputs about as large as
    the inputs."""
    w = (torch.randn((N, K), generator=g, device=g.device) * 38).round_().clamp_(-127, 127)
    s = (torch.rand(N, generator=g, device=g.device) + 0.5) / (38 * math.sqrt(K))
    return w.to(torch.int8), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = g.device
    t = TYPES[case["dtype"]]
    m = case["m"]

    def normal(*shape, std=1.0, mean=0.0, dtype=t):
        return (torch.randn(shape, generator=g, device=dev) * std + mean).to(dtype)

    st = dict(case=case)
    if case["op"] in ("norms", "norms_linear"):
        H = case["H"]
        st["partials"] = [normal(m, H, std=1 / math.sqrt(case["n"])) for _ in range(case["n"])]
        st["residual"] = normal(m, H, std=2.0, dtype=TYPES[case["residual"]])
        around = 1.0 - case["offset"]
        st["weight"] = normal(H, std=0.1, mean=around)
        st["post"] = normal(H, std=0.1, mean=around) if case["post"] else None
        st["gate"] = None
        if case["gate"] == "channel":
            st["gate"] = normal(H, std=0.3)
        elif case["gate"] == "sequence":  # one of six parts of a modulation
            st["gate"] = normal(case["sequences"], 6 * H, std=0.5)[:, 2 * H:3 * H]
        elif case["gate"] == "token":
            st["gate"] = normal(m, H, std=0.5)
        if case["op"] == "norms_linear":
            st["w"], st["ws"] = _weights8(g, case["N"], H)
    elif case["op"] == "linear":
        # Activations with a few channels that are far larger than the others.
        large = torch.rand(case["K"], generator=g, device=dev) < 0.002
        st["x"] = (normal(m, case["K"], dtype=torch.float32) * torch.where(large, 20.0, 1.0)).to(t)
        st["w"], st["ws"] = _weights8(g, case["N"], case["K"])
    else:
        x = torch.randn((m, case["K"]), generator=g, device=dev) * 32
        st["x"] = x.round_().clamp_(-127, 127).to(torch.int8)
        st["xs"] = (torch.rand(m, generator=g, device=dev) + 0.5) / 32
        st["w"], st["ws"] = _weights8(g, case["N"], case["K"])
    return st


# ---------------------------------------------------------------- the plain forms

def _plain_block(st):
    """(r, y) in fp32: the new residual and its norm."""
    case = st["case"]
    H = case["H"]
    b = torch.stack(st["partials"]).float().sum(0)
    if st["post"] is not None:
        b = b * torch.rsqrt(b.square().mean(1, keepdim=True) + EPS)
        b = b * (st["post"].float() + case["offset"])
    if st["gate"] is not None:
        gate = st["gate"].float().reshape(-1, 1, H)
        b = (b.view(gate.shape[0], -1, H) * gate).view(-1, H)
    r = case["residual_scale"] * st["residual"].float() + case["block_scale"] * b
    y = r * torch.rsqrt(r.square().mean(1, keepdim=True) + EPS)
    return r, y * (st["weight"].float() + case["offset"])


def _plain_quantised(x):
    amax = x.abs().amax(1, keepdim=True)
    q = torch.round(torch.where(amax > 0, x * 127 / amax, 0.0))
    return q, (amax / 127).squeeze(1)


def _plain_product(x, xs, w, ws, act, dtype):
    y = (x.float() @ w.float().T) * ws * xs.unsqueeze(1)
    if act == "silu_mul":
        gate, up = y.chunk(2, dim=-1)
        y = gate / (1 + torch.exp(-gate)) * up
    return y.to(TYPES[dtype])


def _plain(st):
    case = st["case"]
    if case["op"] == "norms":
        r, y = _plain_block(st)
        return y.to(TYPES[case["dtype"]]), r.to(TYPES[case["residual"]])
    if case["op"] == "norms_linear":
        r, y = _plain_block(st)
        q, s = _plain_quantised(y)
        out = _plain_product(q, s, st["w"], st["ws"], case["act"], case["dtype"])
        return out, r.to(TYPES[case["residual"]])
    if case["op"] == "linear":
        q, s = _plain_quantised(st["x"].float())
    else:
        q, s = st["x"], st["xs"]
    return _plain_product(q, s, st["w"], st["ws"], case["act"], case["dtype"])


def run(state):
    if not own:
        return _plain(state)
    import allreduce_sum_residual_gb300 as arn
    case = state["case"]
    op = case["op"]
    if op in ("norms", "norms_linear"):
        block = arn.ar_block_rmsnorm if op == "norms" else arn.ar_block_rmsnorm_i8
        r = block(state["partials"], state["residual"], state["weight"], EPS,
                  post_weight=state["post"], gate=state["gate"], block_scale=case["block_scale"],
                  residual_scale=case["residual_scale"], weight_offset=case["offset"])
        if op == "norms":
            return r
        q, s, residual_out = r
        return arn.ar_i8_matmul(q, s, state["w"], state["ws"], act=case["act"],
                                dtype=TYPES[case["dtype"]]), residual_out
    if op == "linear":
        q, s = arn.ar_i8_quantize(state["x"])
    else:
        q, s = state["x"], state["xs"]
    return arn.ar_i8_matmul(q, s, state["w"], state["ws"], act=case["act"],
                            dtype=TYPES[case["dtype"]])


# ---------------------------------------------------------------- what a pass has to do

def _size(name):
    return 4 if name == "float32" else 2


def work(case):
    """Bytes of the operator's inputs and outputs; the 8-bit rows between a norm or a
    quantisation and the product that reads them are not counted."""
    m, bytes_, flops = case["m"], 0, 0
    if case["op"] in ("norms", "norms_linear"):
        K = H = case["H"]
        gates = {"none": 0, "channel": 1, "sequence": case["sequences"], "token": m}[case["gate"]]
        bytes_ = 2 * m * H * case["n"] + 2 * _size(case["residual"]) * m * H
        bytes_ += 2 * H * (1 + int(case["post"]) + gates)
        flops = m * H * (case["n"] + 8)
        if case["op"] == "norms":
            return {"bytes": bytes_ + 2 * m * H, "flops": flops}
    else:
        K = case["K"]
        bytes_ = 2 * m * K if case["op"] == "linear" else m * K + 4 * m
    N = case["N"]
    width = N // 2 if case["act"] == "silu_mul" else N
    bytes_ += N * K + 4 * N + _size(case["dtype"]) * m * width
    return {"bytes": bytes_, "flops": flops + 2 * m * N * K}


# ---------------------------------------------------------------- 64 bits, from the definition

def _exact_block(st, case):
    m, H = case["m"], case["H"]
    b = torch.zeros((m, H), dtype=torch.float64, device="cuda")
    for p in st["partials"]:
        b += p.double()
    if case["post"]:
        b /= torch.sqrt((b * b).sum(1, keepdim=True) / H + EPS)
        b *= st["post"].double() + case["offset"]
    if case["gate"] == "channel":
        b *= st["gate"].double()
    elif case["gate"] != "none":
        b *= st["gate"].double().repeat_interleave(m // st["gate"].shape[0], dim=0)
    r = st["residual"].double() * case["residual_scale"] + b * case["block_scale"]
    rms = torch.sqrt((r * r).sum(1, keepdim=True) / H + EPS)
    return r, r / rms * (st["weight"].double() + case["offset"])


def _exact_rows8(x):
    top = torch.linalg.vector_norm(x, ord=math.inf, dim=1, keepdim=True)
    return torch.round(torch.nan_to_num(x * 127 / top, nan=0.0)), top.squeeze(1) / 127


def _exact_sums(x, w):
    """The whole numbers sum_k x w: 1024 products of 8-bit numbers are below 2^24, where sums of
    whole numbers in fp32 are exact in any order; the parts are added in 64 bits."""
    total = torch.zeros((x.shape[0], w.shape[0]), dtype=torch.float64, device="cuda")
    for a in range(0, x.shape[1], 1024):
        total += torch.matmul(x[:, a:a + 1024].float(), w[:, a:a + 1024].float().t()).double()
    return total


def exact(case, seed):
    st = prepare(case, seed)
    residual = None
    if case["op"] in ("norms", "norms_linear"):
        residual, y = _exact_block(st, case)
        if case["op"] == "norms":
            return y, residual
        q, s = _exact_rows8(y)
    elif case["op"] == "linear":
        q, s = _exact_rows8(st["x"].double())
    else:
        q, s = st["x"], st["xs"].double()
    out = _exact_sums(q, st["w"]) * torch.outer(s, st["ws"].double())
    if case["act"] == "silu_mul":
        half = case["N"] // 2
        out = out[:, :half] * torch.sigmoid(out[:, :half]) * out[:, half:]
    return out if residual is None else (out, residual)
