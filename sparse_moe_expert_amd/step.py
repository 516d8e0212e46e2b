"""One routed-MoE step with preallocated outputs, for graph capture and reuse.

MoeStep owns every output and the workspace for fixed sizes (T, H, I, E, k)
and enqueues the library calls on torch's current stream.  Because no
call allocates or synchronises, `run` can be captured in a torch.cuda.CUDAGraph
(a HIP graph under ROCm) and replayed after the input tensors' contents change.
"""

from __future__ import annotations

from typing import Optional

import numpy as np
import torch

from ._lib import (
    ExpertWeights,
    _check,
    empty_buckets,
    load_library,
    make_workspace,
    moe_bucket_routes,
    moe_expert_ffn,
    moe_route_bucket,
    moe_route_topk,
    moe_router_logits,
    moe_step,
)
from .block import Fp8Experts, empty_fp8_tokens, make_block_ffn_workspace, moe_block_expert_ffn, moe_norm_quantize
from .layer import RouteRule, _int, moe_route_grouped, moe_route_grouped_bucket

_NULL_POINTER = 1        # MOE_ERR_NULL_POINTER


def expert_weights_from_numpy(bank, device) -> ExpertWeights:
    """Copy an NVFP4 expert bank (numpy arrays w_gate, s_gate, ..., g_scale) to the device."""
    dev = torch.device(device)
    to = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).to(dev, dt)  # noqa: E731
    return ExpertWeights(
        to(bank.w_gate, torch.uint8), to(bank.s_gate, torch.uint8),
        to(bank.w_up, torch.uint8), to(bank.s_up, torch.uint8),
        to(bank.w_down, torch.uint8), to(bank.s_down, torch.uint8),
        to(bank.g_scale, torch.float32))


class MoeStep:
    """Outputs and workspace for one step of fixed sizes, and the ways to run it.

    path "step": moe_step (the whole step in one call).  "packed":
    moe_step_packed, with the weights' packed copy passed to run().  "calls":
    moe_route_bucket then moe_expert_ffn.  "calls_unfused": moe_route_topk,
    moe_bucket_routes, moe_expert_ffn.  All of them produce the same outputs.
    With a `rule` (of the same k; "calls" and "calls_unfused" only) the experts
    are chosen by moe_route_grouped_bucket or moe_route_grouped in place of
    moe_route_bucket and moe_route_topk."""

    PATHS = ("step", "packed", "calls", "calls_unfused")

    def __init__(self, T: int, H: int, I: int, E: int, k: int, device, path: str = "step",
                 rule: Optional[RouteRule] = None):
        if path not in self.PATHS:
            raise ValueError(f"path must be one of {self.PATHS}")
        if rule is not None and path not in ("calls", "calls_unfused"):
            raise ValueError('a rule is used on paths "calls" and "calls_unfused"')
        if rule is not None and rule.k != k:
            raise ValueError(f"rule.k must be k={k}, got {rule.k}")
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.path = path
        self.rule = rule
        self.device = torch.device(device)
        self.topk_idx = torch.empty((T, k), dtype=torch.int32, device=self.device)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, device=self.device)
        self.buckets = empty_buckets(T, E, k, self.device)
        self.workspace = make_workspace(T, H, I, E, k, self.device)
        self.y = torch.empty((T, H), dtype=torch.bfloat16, device=self.device)

    def route(self, logits: torch.Tensor, bias: Optional[torch.Tensor]):
        if self.rule is not None:
            moe_route_grouped(logits, bias, self.rule, self.topk_idx, self.topk_w)
        else:
            moe_route_topk(logits, bias, self.k, self.topk_idx, self.topk_w)

    def bucket(self):
        moe_bucket_routes(self.topk_idx, self.E, self.buckets)

    def route_bucket(self, logits: torch.Tensor, bias: Optional[torch.Tensor]):
        if self.rule is not None:
            moe_route_grouped_bucket(logits, bias, self.rule, self.topk_idx, self.topk_w, self.buckets)
        else:
            moe_route_bucket(logits, bias, self.k, self.topk_idx, self.topk_w, self.buckets)

    def routing(self, logits: torch.Tensor, bias: Optional[torch.Tensor]):
        if self.path == "calls_unfused":
            self.route(logits, bias)
            self.bucket()
        else:
            self.route_bucket(logits, bias)

    def ffn(self, x: torch.Tensor, weights: ExpertWeights, stage: int = 3):
        moe_expert_ffn(x, weights, self.topk_w, self.buckets, self.workspace, self.y, stage=stage)

    def run(self, x: torch.Tensor, logits: torch.Tensor, bias: Optional[torch.Tensor],
            weights: ExpertWeights, packed: Optional[torch.Tensor] = None, stage: int = 3) -> torch.Tensor:
        """The step; stage 1 or 2 (paths "step" and "packed") runs one part of it."""
        if self.path in ("step", "packed"):
            if self.path == "packed" and packed is None:
                raise ValueError('path "packed" needs the packed weights (pack_weights)')
            moe_step(x, logits, bias, weights, self.k, self.topk_idx, self.topk_w, self.buckets,
                     self.workspace, self.y, packed=packed if self.path == "packed" else None, stage=stage)
        else:
            if stage != 3:
                raise ValueError('stages are run on paths "step" and "packed"')
            self.routing(logits, bias)
            self.ffn(x, weights)
        return self.y


class Fp8MoeStep:
    """The step in 8 bits, from the attention's output on: residual addition and
    norm, router, routing and buckets, the routed experts, all outputs and the
    workspace owned here (and the step capturable) as in MoeStep.

    run() computes r = x + residual and n = RMSNorm(r) * (norm_weight +
    weight_offset), routes n (moe_router_logits on n in bf16; top-k, or by
    `rule`) and returns y, the experts' output for n in 8 bits.  `residual`
    (bf16, or fp32 with residual_dtype) holds r afterwards; the next layer's x
    is y.  Sizes that one of the calls does not take (the router: H up to 4096)
    are refused here, with its MoeError."""

    def __init__(self, T: int, H: int, I: int, E: int, k: int, device, rule: Optional[RouteRule] = None,
                 residual_dtype: torch.dtype = torch.bfloat16, eps: float = 1e-6, weight_offset: float = 0.0):
        if residual_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"residual_dtype must be bfloat16 or float32, got {residual_dtype}")
        if rule is not None and rule.k != k:
            raise ValueError(f"rule.k must be k={k}, got {rule.k}")
        self._check_sizes(T, H, I, E, k)
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        self.rule, self.eps, self.weight_offset = rule, eps, weight_offset
        self.device = torch.device(device)
        self.residual = torch.empty((T, H), dtype=residual_dtype, device=self.device)
        self.hidden = torch.empty((T, H), dtype=torch.bfloat16, device=self.device)
        self.tokens = empty_fp8_tokens(T, H, self.device)
        self.logits = torch.empty((T, E), dtype=torch.float32, device=self.device)
        self.topk_idx = torch.empty((T, k), dtype=torch.int32, device=self.device)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, device=self.device)
        self.buckets = empty_buckets(T, E, k, self.device)
        self.workspace = make_block_ffn_workspace(T, H, I, E, k, self.device)
        self.y = torch.empty((T, H), dtype=torch.bfloat16, device=self.device)

    @staticmethod
    def _check_sizes(T: int, H: int, I: int, E: int, k: int):  # noqa: E741
        """The calls' own checks of sizes, which stand before those of pointers: all NULL here."""
        T, H, I, E, k = (_int(v, n) for v, n in zip((T, H, I, E, k), "THIEk"))  # noqa: E741
        lib = load_library()
        for name, args in (("moe_norm_quantize", [None, None, 0, None, 0.0, 1.0, T, H] + [None] * 5),
                           ("moe_router_logits", [None, None, T, H, E, None, None]),
                           ("moe_block_expert_ffn", [None] * 15 + [T, H, I, E, k, None, 0, None, None])):
            status = getattr(lib, name)(*args)
            if status != _NULL_POINTER:
                _check(name, status)

    def run(self, x: torch.Tensor, residual: torch.Tensor, norm_weight: torch.Tensor, w_router: torch.Tensor,
            bias: Optional[torch.Tensor], experts: Fp8Experts) -> torch.Tensor:
        """The step of bf16 x [T,H]; `residual` [T,H] may be self.residual, of the step before, and is
        zeros where there is none."""
        if residual is None:
            raise TypeError("residual must be a tensor: zeros where there is no residual stream yet")
        moe_norm_quantize(x, norm_weight, residual, self.eps, self.weight_offset, self.tokens, self.residual, self.hidden)
        moe_router_logits(self.hidden, w_router, self.logits)
        if self.rule is not None:
            moe_route_grouped_bucket(self.logits, bias, self.rule, self.topk_idx, self.topk_w, self.buckets)
        else:
            moe_route_bucket(self.logits, bias, self.k, self.topk_idx, self.topk_w, self.buckets)
        return moe_block_expert_ffn(self.tokens, experts, self.topk_w, self.buckets, self.workspace, self.y)
