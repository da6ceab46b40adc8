"""A rank's part of a mixture-of-experts layer at decode batch sizes, from the
normed activations to the next layer's: the routing, the chosen experts'
4-bit products, a shared expert, their weighted sum, and the epilogue.

    x, r = moe(x, r, next_norm_weight, eps)

One rank sums the experts straight through the residual add and RMSNorm
(``ar_combine_rmsnorm``); a rank of a tensor-parallel or expert-parallel
group writes its partial into the group's buffer and calls the group's
epilogue (``peers.FusedAllReduceRMSNorm``).  The calls are asynchronous on
the current stream and can be captured in a CUDA graph.
"""
import torch

from .experts import (ar_combine, ar_combine_rmsnorm, ar_route_experts, ar_w4_matvec,
                      ar_w4_matvec_experts)


class ExpertLayer:
    """The weights of one layer on one rank.

    router: [experts of the layer, H] bf16 or fp32; its logits are fp32 either
    way (bf16's rounding would decide between experts).  up: (q, scales,
    zeros or None) of this rank's experts' gate and up rows, [E, 2 I, H]
    unpacked; down: the same of [E, H, I].  Layouts as in ``ar_w4_matvec``.
    first: the layer's number of this rank's first expert.  shared_up,
    shared_down: a dense expert that every token takes, or None (with a
    group: this rank's slice of it).  group: a
    ``peers.FusedAllReduceRMSNorm``, or None for one rank.  The routing
    options are ``ar_route_experts``'s.
    """

    def __init__(self, router, up, down, top_k, *, bias=None, scoring="softmax", groups=1,
                 topk_groups=None, group_score="max", renorm=True, scale=1.0, first=0,
                 shared_up=None, shared_down=None, group=None):
        if (shared_up is None) != (shared_down is None):
            raise ValueError("a shared expert needs both shared_up and shared_down")
        if router.dim() != 2:
            raise ValueError("router must be [experts, H]")
        if router.dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"router must be bfloat16 or float32, got {router.dtype}")
        if not 0 <= first <= router.shape[0] - up[0].shape[0]:
            raise ValueError(f"experts {first} .. {first + up[0].shape[0] - 1} are not all among the "
                             f"router's {router.shape[0]}")
        if down[0].shape[0] != up[0].shape[0]:
            raise ValueError(f"up holds {up[0].shape[0]} experts and down {down[0].shape[0]}")
        self.router, self.up, self.down = router.detach(), tuple(up), tuple(down)
        self.top_k, self.first, self.group = top_k, first, group
        self.shared_up, self.shared_down = shared_up, shared_down
        self.routing = dict(bias=bias, scoring=scoring, groups=groups, topk_groups=topk_groups,
                            group_score=group_score, renorm=renorm, scale=scale)

    def route(self, x):
        """(weights, ids) of the tokens x [m, H]."""
        if self.router.dtype is torch.bfloat16:
            logits = torch.mm(x, self.router.t(), out_dtype=torch.float32)
        else:
            with torch.autocast("cuda", enabled=False):
                logits = torch.mm(x.float(), self.router.t())
        return ar_route_experts(logits, self.top_k, **self.routing)

    def outputs(self, x):
        """(y, weights, shared): the chosen experts' rows [m, k, H] (zero where
        an expert is another rank's), their weights, the shared expert's rows
        or None."""
        weights, ids = self.route(x)
        h = ar_w4_matvec_experts(x, ids, *self.up, act="silu_mul", first=self.first)
        y = ar_w4_matvec_experts(h, ids, *self.down, first=self.first)
        shared = None
        if self.shared_up is not None:
            shared = ar_w4_matvec(ar_w4_matvec(x, *self.shared_up, act="silu_mul"),
                                  *self.shared_down)
        return y, weights, shared

    def partial(self, x, out=None):
        """This rank's partial [m, H] of the layer's sum."""
        y, weights, shared = self.outputs(x)
        return ar_combine(y, weights, shared=shared, out=out)

    def __call__(self, x, residual, weight, eps):
        """(out, residual_out) from the activations x [m, H], the residual and
        the next norm's weight."""
        if self.group is None:
            y, weights, shared = self.outputs(x)
            return ar_combine_rmsnorm(y, weights, residual, weight, eps, shared=shared)
        self.partial(x, out=self.group.partial(x.shape[0]))
        return self.group(residual, weight, eps)


__all__ = ["ExpertLayer"]
