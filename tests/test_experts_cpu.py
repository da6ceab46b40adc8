"""The expert-layer calls without a GPU: every refusal comes back as a code
before any CUDA call, and the binding checks its tensors."""
import math
import os
import re

import pytest
import torch

import experts_ref as ref

OK, ARG, ALIGN, ALIAS, WORKSPACE, CUDA, TIMEOUT, UNSUPPORTED = range(8)
BASE = 0x7F0000000000  # fake, never dereferenced
GAP = 1 << 34


def at(i):
    return BASE + i * GAP


def route(L, logits=at(0), kind=1, stride=None, bias=at(1), m=4, E=64, k=8, scoring=1, groups=8,
          topk_groups=4, group_score=1, renorm=1, scale=1.0, weights=at(2), ids=at(3)):
    return L.ar_route_experts(logits, kind, E if stride is None else stride, bias, m, E, k, scoring,
                              groups, topk_groups, group_score, renorm, scale, weights, ids, None)


@pytest.mark.parametrize("kw,status", [
    (dict(kind=3), ARG), (dict(kind=-1), ARG), (dict(m=-1), ARG), (dict(E=0), ARG), (dict(k=0), ARG),
    (dict(groups=0), ARG), (dict(groups=33, E=66), ARG), (dict(topk_groups=0), ARG),
    (dict(topk_groups=9), ARG), (dict(E=65), ARG), (dict(k=9, E=16, topk_groups=4), ARG),
    (dict(stride=63), ARG), (dict(scoring=2), ARG), (dict(group_score=2), ARG), (dict(renorm=2), ARG),
    (dict(scale=math.nan), ARG), (dict(scale=math.inf), ARG),
    (dict(E=8, k=4), ARG),                      # groups of one have no second choice
    (dict(E=520), UNSUPPORTED), (dict(k=17), UNSUPPORTED), (dict(m=1 << 40), UNSUPPORTED),
    (dict(logits=0), ARG), (dict(weights=0), ARG), (dict(ids=0), ARG),
    (dict(logits=at(0) + 1), ALIGN), (dict(kind=0, logits=at(0) + 2), ALIGN),
    (dict(bias=at(1) + 2), ALIGN), (dict(weights=at(2) + 2), ALIGN), (dict(ids=at(3) + 1), ALIGN),
    (dict(weights=at(3)), ALIAS), (dict(ids=at(0)), ALIAS), (dict(weights=at(1)), ALIAS),
    (dict(ids=at(0) + 4 * 64 * 2 - 4), ALIAS),
    (dict(m=0), OK), (dict(m=0, logits=0, weights=0, ids=0), OK),
])
def test_route_refusals(arlib, kw, status):
    assert route(arlib.lib(), **kw) == status


def w4(L, x=at(0), q=at(1), s=at(2), kind=1, z=at(3), m=4, N=64, K=256, group=64, act=0, out=at(4)):
    return L.ar_w4_matvec(x, q, s, kind, z, m, N, K, group, act, out, None)


def w4e(L, x=at(0), per=0, ids=at(5), m=4, k=2, q=at(1), s=at(2), kind=1, z=at(3), first=0, E=8,
        N=64, K=256, group=64, act=0, out=at(4)):
    return L.ar_w4_matvec_experts(x, per, ids, m, k, q, s, kind, z, first, E, N, K, group, act, out,
                                  None)


W4_BOTH = [
    (dict(m=-1), ARG), (dict(N=0), ARG), (dict(K=0), ARG), (dict(kind=3), ARG), (dict(group=16), ARG),
    (dict(group=256), ARG), (dict(K=288), ARG), (dict(act=2), ARG), (dict(act=1, N=63), ARG),
    (dict(K=32768 + 64), UNSUPPORTED), (dict(N=(1 << 20) + 2), UNSUPPORTED),
    (dict(x=0), ARG), (dict(q=0), ARG), (dict(s=0), ARG), (dict(out=0), ARG),
    (dict(x=at(0) + 8), ALIGN), (dict(q=at(1) + 4), ALIGN), (dict(s=at(2) + 2), ALIGN),
    (dict(z=at(3) + 1), ALIGN), (dict(out=at(4) + 1), ALIGN),
    (dict(out=at(0)), ALIAS), (dict(out=at(1) + 64), ALIAS), (dict(out=at(2)), ALIAS),
    (dict(out=at(3)), ALIAS), (dict(m=0), OK), (dict(m=0, x=0, q=0, s=0, out=0), OK),
]


@pytest.mark.parametrize("kw,status", W4_BOTH + [(dict(m=65), UNSUPPORTED)])
def test_w4_matvec_refusals(arlib, kw, status):
    assert w4(arlib.lib(), **kw) == status


@pytest.mark.parametrize("kw,status", W4_BOTH + [
    (dict(k=0), ARG), (dict(E=0), ARG), (dict(first=-1), ARG), (dict(per=2), ARG), (dict(ids=0), ARG), (dict(k=17), UNSUPPORTED),
    (dict(E=513), UNSUPPORTED), (dict(m=2049), UNSUPPORTED), (dict(ids=at(5) + 2), ALIGN),
    (dict(out=at(5)), ALIAS), (dict(per=1, out=at(0) + 4 * 256 * 2), ALIAS),
])
def test_w4_matvec_experts_refusals(arlib, kw, status):
    assert w4e(arlib.lib(), **kw) == status


def combine(L, y=at(0), rows=8, slots=None, w=at(1), shared=at(2), m=4, k=2, H=64, out=at(3)):
    return L.ar_combine(y, rows, slots, w, shared, m, k, H, out, None)


def combine_norm(L, y=at(0), rows=8, slots=None, w=at(1), shared=at(2), res=at(4), g=at(5), eps=1e-6,
                 m=4, k=2, H=64, out=at(3), rout=at(6)):
    return L.ar_combine_rmsnorm(y, rows, slots, w, shared, res, g, eps, m, k, H, out, rout, None)


COMBINE = [
    (dict(m=-1), ARG), (dict(H=0), ARG), (dict(H=60), ALIGN), (dict(H=131080), UNSUPPORTED),
    (dict(k=0), ARG), (dict(k=17, rows=68), UNSUPPORTED), (dict(rows=7), ARG), (dict(rows=-1), ARG),
    (dict(rows=1 << 35, slots=at(7)), UNSUPPORTED),
    (dict(y=0), ARG), (dict(w=0), ARG), (dict(out=0), ARG),
    (dict(y=at(0) + 8), ALIGN), (dict(shared=at(2) + 2), ALIGN), (dict(out=at(3) + 8), ALIGN),
    (dict(w=at(1) + 2), ALIGN), (dict(slots=at(7) + 2), ALIGN),
    (dict(out=at(0)), ALIAS), (dict(out=at(2)), ALIAS), (dict(out=at(7), slots=at(7)), ALIAS),
    (dict(m=0, rows=0), OK), (dict(m=0, rows=0, y=0, w=0, out=0), OK),
]


@pytest.mark.parametrize("kw,status", COMBINE)
def test_combine_refusals(arlib, kw, status):
    assert combine(arlib.lib(), **kw) == status


@pytest.mark.parametrize("kw,status", COMBINE + [
    (dict(eps=-1.0), ARG), (dict(eps=math.nan), ARG), (dict(res=0), ARG), (dict(g=0), ARG),
    (dict(rout=0), ARG), (dict(res=at(4) + 8), ALIGN), (dict(g=at(5) + 8), ALIGN),
    (dict(rout=at(6) + 8), ALIGN), (dict(rout=at(3)), ALIAS), (dict(rout=at(4) + 16), ALIAS),
    (dict(rout=at(0)), ALIAS), (dict(out=at(4)), ALIAS), (dict(rout=at(5)), ALIAS),
])
def test_combine_rmsnorm_refusals(arlib, kw, status):
    assert combine_norm(arlib.lib(), **kw) == status


@pytest.mark.skipif(torch.cuda.is_available(), reason="would launch on fake pointers")
def test_valid_calls_pass_the_checks(arlib):
    """Without a device a valid call stops at the first CUDA call."""
    L = arlib.lib()
    assert route(L) == CUDA and route(L, bias=None, kind=0, groups=1, topk_groups=1) == CUDA
    assert w4(L) == CUDA and w4(L, z=None, act=1) == CUDA and w4e(L) == CUDA
    assert combine(L) == CUDA and combine(L, shared=None, slots=at(7), rows=1) == CUDA
    assert combine(L, y=0, rows=0, slots=at(7)) == CUDA
    assert combine_norm(L) == CUDA and combine_norm(L, rout=at(4)) == CUDA  # in place


def test_the_binding_refuses_host_tensors_and_wrong_kinds(arlib):
    x = torch.zeros((4, 64))
    with pytest.raises(ValueError, match="CUDA device"):
        arlib.ar_route_experts(x, 2)
    with pytest.raises(TypeError, match="torch.Tensor"):
        arlib.ar_route_experts([1.0], 2)
    with pytest.raises(ValueError, match="CUDA device"):
        arlib.ar_w4_matvec(x, x, x)
    with pytest.raises(ValueError, match="CUDA device"):
        arlib.ar_w4_matvec_experts(x, x, x, x)
    with pytest.raises(ValueError, match="CUDA device"):
        arlib.ar_combine(x, x)
    with pytest.raises(ValueError, match="CUDA device"):
        arlib.ar_combine_rmsnorm(x, x, x, x, 1e-6)


def test_constants_match_the_header(arlib):
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                            "ar_rmsnorm.h")).read()
    names = [n for n in dir(arlib) if re.match(r"AR_(TYPE|SCORE|GROUP|ACT|MATVEC|MAX)_", n)]
    assert len(names) >= 16
    for n in names:
        m = re.search(rf"#define {n}\s+(\d+)", src)
        assert m and int(m.group(1)) == getattr(arlib, n), n


# The 64-bit forms themselves, on rows worked by hand.

def test_reference_route_by_hand():
    x = torch.tensor([[1.0, 3.0, 3.0, -math.inf], [0.0, 0.0, 0.0, 0.0]])
    w, ids = ref.route(x, 2)
    assert ids.tolist() == [[1, 2], [0, 1]] and w.tolist() == [[0.5, 0.5], [0.5, 0.5]]
    w, ids = ref.route(x, 2, groups=2, topk_groups=1)
    assert ids.tolist() == [[1, 0], [0, 1]]
    w, ids = ref.route(x, 2, groups=2, topk_groups=1, group_score="top2", scoring="sigmoid",
                       renorm=False, scale=2.0)
    assert ids.tolist() == [[1, 0], [0, 1]]
    assert abs(w[1, 0].item() - 1.0) < 1e-15 and abs(w[0, 1].item() - 2 / (1 + math.exp(-1))) < 1e-15
    w, ids = ref.route(torch.full((1, 4), -math.inf), 3)
    assert ids.tolist() == [[0, 1, 2]] and w.tolist() == [[0.0, 0.0, 0.0]]
    # The bias of an expert that is off does not bring it back.
    w, ids = ref.route(x[:1], 1, bias=torch.tensor([9.0, 0.0, 0.0, 99.0]), scoring="sigmoid")
    assert ids.tolist() == [[0]]


def test_reference_unpack_by_hand():
    q = torch.tensor([[0x21, 0x83]], dtype=torch.uint8).repeat(1, 8)  # 1, 2, 3, 8, ...
    w = ref.unpack(q, torch.tensor([[0.5]]), None)
    assert w.shape == (1, 32) and w[0, :4].tolist() == [-3.5, -3.0, -2.5, 0.0]
    w = ref.unpack(q, torch.tensor([[2.0]]), torch.tensor([[0x11]], dtype=torch.uint8))
    assert w[0, :4].tolist() == [0.0, 2.0, 4.0, 14.0]
