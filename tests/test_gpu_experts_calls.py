"""Ways to call the expert-layer functions that the other tests do not take."""
import threading

import numpy as np
import pytest
import torch

import allreduce_sum_residual_gb300 as arn
from test_gpu_experts import DEV, gen, layer, layer_inputs, normal, weights4

pytestmark = pytest.mark.gpu


def test_the_default_stream_by_its_handle():
    d = layer_inputs(3, 91)
    logits = d["x"] @ d["router"].T
    want = arn.ar_route_experts(logits, 4)
    torch.cuda.synchronize()
    for s in (0, torch.cuda.default_stream(), torch.cuda.default_stream().cuda_stream):
        got = arn.ar_route_experts(logits, 4, stream=s)
        h = arn.ar_w4_matvec_experts(d["x"], got[1], *d["up"], stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(h, arn.ar_w4_matvec_experts(d["x"], want[1], *d["up"]))


def test_numbers_of_other_kinds():
    g = gen(92)
    x = normal(g, 5, 64)
    want = arn.ar_route_experts(x, 2, groups=4, topk_groups=2, scale=2.5)
    for n, f in ((np.int64, np.float32), (np.int32, np.float64), (torch.tensor, torch.tensor), (int, float)):
        got = arn.ar_route_experts(x, n(2), groups=n(4), topk_groups=n(2), scale=f(2.5))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_inference_mode_and_gradients_wanted():
    d = layer_inputs(4, 93)
    want = layer(**d)[0]
    with torch.inference_mode():
        got = layer(**d)[0]
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    d["x"].requires_grad_(True)
    d["weight"].requires_grad_(True)
    got = layer(**d)[0]
    assert torch.equal(got[0], want[0]) and not got[0].requires_grad


def test_threads_at_once():
    """Each thread with a stream of its own, all layers at the same time."""
    ins = [layer_inputs(1 + 5 * i, 94 + i) for i in range(4)]
    want = [layer(**d)[0] for d in ins]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got = layer(**ins[i])[0]
                torch.cuda.current_stream().synchronize()
            if not (torch.equal(got[0], want[i][0]) and torch.equal(got[1], want[i][1])):
                wrong.append(i)
        except Exception as e:  # reported by the main thread
            wrong.append((i, e))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_views_of_larger_tensors():
    """Operands that start inside a storage, at the alignment that is asked for."""
    g = gen(95)
    m, K, N = 4, 256, 40
    flat = normal(g, 16 + m * K)
    x = flat[16:].view(m, K)
    q, s, z = weights4(g, (3, N), K, 64, "f16", True)
    for i in range(3):  # 40 x 4 scales of two bytes: every matrix 64 bytes on from a 16-byte boundary
        got = arn.ar_w4_matvec(x, q[i], s[i], zeros=z[i])
        assert torch.equal(got, arn.ar_w4_matvec(x.clone(), q[i].clone(), s[i].clone(), zeros=z[i].clone()))
    with pytest.raises(arn.ArError) as e:
        arn.ar_w4_matvec(flat[3:3 + m * K].view(m, K), q[0], s[0], zeros=z[0])
    assert e.value.status == arn.AR_ERR_ALIGN
    out = torch.full((m * N + 3,), 7.0, dtype=torch.bfloat16, device=DEV)
    arn.ar_w4_matvec(x, q[0], s[0], zeros=z[0], out=out[1:1 + m * N].view(m, N))
    assert out[0] == 7 and bool((out[-2:] == 7).all())
    assert torch.equal(out[1:-2].view(m, N), arn.ar_w4_matvec(x, q[0], s[0], zeros=z[0]))
