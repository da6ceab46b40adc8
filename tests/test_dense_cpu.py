"""The 8-bit layer's calls without a GPU: what they refuse, in the C ABI and
on tensors, before anything is launched."""
import ctypes

import pytest
import torch

VP = ctypes.c_void_p
A = 1 << 20  # a made-up, aligned address; nothing is read before the checks


def block(arlib, i8=False, n=1, type=1, post=None, gate=None, gate_stride=64, gate_rows=4,
          block_scale=1.0, residual=A * 2, residual_type=1, residual_scale=1.0, weight=A * 3,
          offset=0.0, eps=1e-6, m=4, H=64, out=A * 4, scales=A * 6, residual_out=A * 5, partials=(A,)):
    lib = arlib.lib()
    p = (VP * len(partials))(*partials) if partials is not None else None
    head = (p, n, type, post, gate, gate_stride, gate_rows, block_scale, residual, residual_type,
            residual_scale, weight, offset, eps, m, H, out)
    if i8:
        return lib.ar_block_rmsnorm_i8(*head, scales, residual_out, None)
    return lib.ar_block_rmsnorm(*head, residual_out, None)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(n=0), 1), (dict(n=17), 1), (dict(m=-1), 1), (dict(H=0), 1), (dict(H=12), 2),
    (dict(H=131080), 7), (dict(m=1 << 40), 7), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(type=0), 1), (dict(type=3), 1), (dict(residual_type=2), 1), (dict(residual_type=7), 1),
    (dict(block_scale=float("inf")), 1), (dict(residual_scale=float("nan")), 1),
    (dict(offset=float("inf")), 1),
    (dict(gate=A * 7, gate_rows=0), 1), (dict(gate=A * 7, gate_rows=-3), 1),
    (dict(gate=A * 7, gate_rows=1, gate_stride=56), 1), (dict(gate=A * 7, gate_rows=1, gate_stride=0), 1),
    (dict(gate=A * 7, gate_rows=1, gate_stride=68), 2),
    (dict(gate=A * 7, gate_rows=1, gate_stride=1 << 50), 7),
    (dict(partials=None), 1), (dict(partials=(None,)), 1), (dict(residual=None), 1),
    (dict(weight=None), 1), (dict(out=None), 1), (dict(residual_out=None), 1),
    (dict(partials=(A + 8,)), 2), (dict(residual=A * 2 + 4), 2), (dict(weight=A * 3 + 2), 2),
    (dict(out=A * 4 + 8), 2), (dict(residual_out=A * 5 + 8), 2), (dict(post=A * 7 + 8), 2),
    (dict(gate=A * 7 + 2), 2),
    (dict(out=A), 3), (dict(out=A * 2), 3), (dict(out=A * 3), 3), (dict(out=A * 5), 3),
    (dict(residual_out=A), 3), (dict(residual_out=A * 2 + 16), 3), (dict(residual_out=A * 3), 3),
    (dict(post=A * 7, out=A * 7), 3), (dict(gate=A * 7, residual_out=A * 7), 3),
    (dict(gate=A * 7, gate_rows=1, gate_stride=128, out=A * 7 + 128 * 6), 3),
])
def test_block_norm_refuses(arlib, i8, kw, status):
    assert block(arlib, i8, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(scales=None), 1), (dict(scales=A * 6 + 2), 2), (dict(scales=A), 3), (dict(scales=A * 2), 3),
    (dict(scales=A * 4 + 128), 3), (dict(scales=A * 5 + 64), 3), (dict(scales=A * 3), 3)])
def test_block_norm_in_bytes_refuses(arlib, kw, status):
    assert block(arlib, True, **kw) == status


def quantize(arlib, x=A, type=1, stride=64, m=4, K=64, q=A * 2, scales=A * 3):
    return arlib.lib().ar_i8_quantize(x, type, stride, m, K, q, scales, None)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), 1), (dict(K=0), 1), (dict(type=0), 1), (dict(type=5), 1), (dict(stride=56), 1),
    (dict(stride=68), 2), (dict(K=60), 2), (dict(K=131080, stride=131080), 7), (dict(m=1 << 31), 7),
    (dict(stride=1 << 39), 7), (dict(x=None), 1), (dict(q=None), 1), (dict(scales=None), 1),
    (dict(x=A + 2), 2), (dict(q=A * 2 + 8), 2), (dict(scales=A * 3 + 2), 2),
    (dict(q=A), 3), (dict(scales=A + 128), 3), (dict(scales=A * 2 + 64), 3),
    (dict(stride=512, q=A + 512 * 6), 3)])
def test_quantise_refuses(arlib, kw, status):
    assert quantize(arlib, **kw) == status


def matmul(arlib, x=A, xs=A * 2, w=A * 3, ws=A * 4, m=4, N=32, K=64, act=0, type=1, out=A * 5):
    return arlib.lib().ar_i8_matmul(x, xs, w, ws, m, N, K, act, type, out, None)


@pytest.mark.parametrize("kw,status", [
    (dict(m=-1), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(act=2), 1), (dict(act=-1), 1),
    (dict(type=3), 1), (dict(type=-1), 1), (dict(N=33, act=1), 1), (dict(K=72), 2),
    (dict(K=131072), 7), (dict(N=1048577), 7), (dict(m=4194305), 7),
    (dict(x=None), 1), (dict(xs=None), 1), (dict(w=None), 1), (dict(ws=None), 1), (dict(out=None), 1),
    (dict(x=A + 8), 2), (dict(w=A * 3 + 8), 2), (dict(xs=A * 2 + 2), 2), (dict(ws=A * 4 + 1), 2),
    (dict(out=A * 5 + 1), 2), (dict(out=A * 5 + 2, type=0), 2),
    (dict(out=A), 3), (dict(out=A * 2), 3), (dict(out=A * 3 + 1024), 3), (dict(out=A * 4), 3)])
def test_product_refuses(arlib, kw, status):
    assert matmul(arlib, **kw) == status


def test_empty_calls_need_no_pointers(arlib):
    nothing = dict(partials=None, residual=None, weight=None, out=None, residual_out=None, scales=None)
    assert block(arlib, m=0, **nothing) == 0 and block(arlib, True, m=0, **nothing) == 0
    assert quantize(arlib, m=0, x=None, q=None, scales=None) == 0
    assert matmul(arlib, m=0, x=None, xs=None, w=None, ws=None, out=None) == 0


def test_tensors_of_the_host_are_refused(arlib):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    q, s = torch.zeros((4, 64), dtype=torch.int8), torch.zeros(4)
    for f in (arlib.ar_block_rmsnorm, arlib.ar_block_rmsnorm_i8):
        with pytest.raises(ValueError, match="CUDA device"):
            f([x], x, w, 1e-6)
        with pytest.raises(ValueError, match="at least one"):
            f([], x, w, 1e-6)
        with pytest.raises(TypeError, match="partials"):
            f([None], x, w, 1e-6)
    with pytest.raises(ValueError, match="CUDA device"):
        arlib.ar_i8_quantize(x)
    with pytest.raises(ValueError, match="CUDA device"):
        arlib.ar_i8_matmul(q, s, q, s)
    with pytest.raises(TypeError, match="dtype must be"):
        arlib.ar_i8_matmul(q, s, q, s, dtype=torch.int8)


@pytest.mark.gpu
@pytest.mark.parametrize("long_way", [False, True])
def test_what_is_wrong_is_named(arlib, long_way):
    dev = "cuda:0"
    st = torch.cuda.current_stream() if long_way else None
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device=dev)
    w = torch.zeros(64, dtype=torch.bfloat16, device=dev)
    q, s = torch.zeros((4, 64), dtype=torch.int8, device=dev), torch.zeros(4, device=dev)

    def refused(error, match, f, *a, **kw):
        with pytest.raises(error, match=match):
            f(*a, stream=st, **kw)
    for f in (arlib.ar_block_rmsnorm, arlib.ar_block_rmsnorm_i8):
        refused(TypeError, "partials.0. must be bfloat16 or float16", f, [x.float()], x, w, 1e-6)
        refused(TypeError, "partials.1. must be bfloat16", f, [x, x.half()], x, w, 1e-6)
        refused(ValueError, "partials.1. must have shape", f, [x, x[:3]], x, w, 1e-6)
        refused(TypeError, "residual must be bfloat16", f, [x], x.half(), w, 1e-6)
        refused(ValueError, "residual must be contiguous", f, [x], x.t().contiguous().t(), w, 1e-6)
        refused(ValueError, "weight must have shape", f, [x], x, w[:32], 1e-6)
        refused(TypeError, "post_weight must be", f, [x], x, w, 1e-6, post_weight=w.float())
        refused(ValueError, "gate must be", f, [x], x, w, 1e-6, gate=w[:8])
        refused(TypeError, "gate must be bfloat16", f, [x], x, w, 1e-6, gate=w.half())
        refused(ValueError, "share the 4 rows", f, [x], x, w, 1e-6, gate=x[:3])
        refused(ValueError, "rows of gate must be contiguous", f, [x], x, w, 1e-6,
                gate=torch.zeros((64, 4), dtype=torch.bfloat16, device=dev).t())
        refused(ValueError, "gate must be on", f, [x], x, w, 1e-6, gate=w.cpu())
        refused(arlib.ArError, "status 1", f, [x], x, w, 1e-6, gate=x[:1].expand(2, 64))
        refused(arlib.ArError, "status 3", f, [x], x.clone(), w, 1e-6, residual_out=x)
        refused(arlib.ArError, "status 1", f, [x] * 17, x, w, 1e-6)
        refused(arlib.ArError, "status 1", f, [x], x, w, -1.0)
        refused(arlib.ArError, "status 1", f, [x], x, w, 1e-6, block_scale=float("nan"))
        refused(ValueError, "residual_out must have shape", f, [x], x, w, 1e-6, residual_out=x[:2])
    refused(TypeError, "x must be bfloat16 or float16", arlib.ar_i8_quantize, x.float())
    refused(ValueError, "x must be .m, K.", arlib.ar_i8_quantize, w)
    refused(ValueError, "rows of x must be contiguous", arlib.ar_i8_quantize, x.t())
    refused(arlib.ArError, "status 2", arlib.ar_i8_quantize, x[:, :60].contiguous())
    refused(arlib.ArError, "status 2", arlib.ar_i8_quantize, x.flatten()[4:196].view(3, 64))
    refused(TypeError, "q must be int8", arlib.ar_i8_quantize, x, q=x)
    refused(TypeError, "x must be int8", arlib.ar_i8_matmul, x, s, q, s)
    refused(ValueError, "x_scales must have shape", arlib.ar_i8_matmul, q, s[:3], q, s)
    refused(ValueError, "w must have shape", arlib.ar_i8_matmul, q, s, q[:, :32], s)
    refused(ValueError, "w_scales must have shape", arlib.ar_i8_matmul, q, s, q, s[:2])
    refused(ValueError, "act must be one of", arlib.ar_i8_matmul, q, s, q, s, act="gelu")
    refused(arlib.ArError, "status 1", arlib.ar_i8_matmul, q, s, q, s, act=9)
    refused(arlib.ArError, "status 1", arlib.ar_i8_matmul, q, s, q[:3], s[:3], act="silu_mul")
    refused(ValueError, "out must have shape", arlib.ar_i8_matmul, q, s, q, s, out=x)
    refused(TypeError, "dtype must be", arlib.ar_i8_matmul, q, s, q, s, out=q)
