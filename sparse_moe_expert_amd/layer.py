"""Binding of the operators around the routed experts: grouped routing, dense
products with 4-bit weights and the 4-bit shared expert (argument marshalling
only, as in _lib).

These calls are a few microseconds of GPU work each, less than a call costs
the host, so what does not change from call to call is checked once: a
RouteRule and a QuantWeight check themselves when they are made, and a call
checks its own tensors.
"""

from __future__ import annotations

from typing import Optional

import torch

from ._lib import Buckets, _check, _need, empty_buckets, load_library

_DTYPES = {torch.float32: 0, torch.bfloat16: 1}        # moe_dtype
_SCORES = {"softmax": 0, "sigmoid": 1}                 # moe_score
_FORMATS = {"nvfp4": (0, 16), "mxfp4": (1, 32)}        # moe_quant_format, weights per scale

Tensor = torch.Tensor
_MAX_INT = (1 << 31) - 1
_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
# the device and stream queries of torch.cuda without their Python layers, where
# this torch has them (one built without a GPU has not)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda index: torch.cuda.current_stream(index).cuda_stream)


def _int(value, name: str) -> int:
    """A whole number of 32 bits, as the library takes sizes: ctypes would drop
    what is beyond, and make another size of it."""
    n = int(value)
    if n != value:
        raise ValueError(f"{name} must be a whole number, got {value!r}")
    if not -_MAX_INT <= n <= _MAX_INT:
        raise ValueError(f"{name} must be at most 2^31 - 1, got {n}")
    return n


def _call(name: str, index: int, *args):
    """The library's call on the tensors' device, which it takes to be the
    current one, and on torch's current stream there."""
    fn = getattr(load_library(), name)
    if _current_device() == index:
        status = fn(*args, _current_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _current_stream(index))
    if status != 0:
        _check(name, status)


def _tensor(t, name: str, dtype, shape, device, index: int):
    """_need's checks, with the passing case in one expression."""
    if not (isinstance(t, Tensor) and t.dtype is dtype and t.get_device() == index and t.shape == shape
            and t.is_contiguous()):
        _need(t, name, dtype, shape, device)


class _Fixed:
    """Checked when made, so not to be changed afterwards."""

    __slots__ = ()

    def __setattr__(self, name, value):
        raise AttributeError(f"{type(self).__name__} cannot be changed; make another")

    def _set(self, **values):
        for name, value in values.items():
            object.__setattr__(self, name, value)


class RouteRule(_Fixed):
    """How moe_route_grouped selects: k experts by `score` ("softmax" or
    "sigmoid") plus the bias, from the `groups_kept` best of `groups` groups (a
    group's value: the sum of its `group_top` best), weights renormalised over
    the chosen experts or not, times `scale`."""

    __slots__ = ("k", "score", "groups", "groups_kept", "group_top", "renormalise", "scale", "_args")

    def __init__(self, k: int, score: str = "sigmoid", groups: int = 1, groups_kept: Optional[int] = None,
                 group_top: int = 2, renormalise: bool = True, scale: float = 1.0):
        if score not in _SCORES:
            raise ValueError(f"score must be one of {tuple(_SCORES)}, got {score!r}")
        self._set(k=_int(k, "k"), score=score, groups=_int(groups, "groups"), group_top=_int(group_top, "group_top"),
                  groups_kept=_int(groups if groups_kept is None else groups_kept, "groups_kept"),
                  renormalise=bool(renormalise), scale=float(scale))
        self._set(_args=(_SCORES[score], self.groups, self.groups_kept, self.group_top, int(self.renormalise), self.scale))


def _route_args(logits, bias, rule, topk_idx, topk_w):
    if not isinstance(logits, Tensor) or logits.dim() != 2:
        raise TypeError("logits must be a [T, E] tensor")
    dtype = _DTYPES.get(logits.dtype)
    if dtype is None:
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    (T, E), k, dev, index = logits.shape, rule.k, logits.device, logits.get_device()
    if T > _MAX_INT or E > _MAX_INT:
        raise ValueError(f"logits must have at most 2^31 - 1 tokens and experts, got {T} and {E}")
    if index < 0 or not logits.is_contiguous():
        _need(logits, "logits", logits.dtype)
    if bias is not None:
        _tensor(bias, "bias", _F32, (E,), dev, index)
    if topk_idx is None:
        topk_idx = torch.empty((T, max(k, 0)), dtype=_I32, device=dev)
    if topk_w is None:
        topk_w = torch.empty((T, max(k, 0)), dtype=_F32, device=dev)
    _tensor(topk_idx, "topk_idx", _I32, (T, k), dev, index)
    _tensor(topk_w, "topk_w", _F32, (T, k), dev, index)
    args = (logits.data_ptr(), dtype, None if bias is None else bias.data_ptr(), T, E, k, *rule._args,
            topk_idx.data_ptr(), topk_w.data_ptr())
    return args, T, E, k, dev, index, topk_idx, topk_w


def moe_route_grouped(logits: torch.Tensor, bias: Optional[torch.Tensor], rule: RouteRule,
                      topk_idx: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None):
    """Expert ids (int32 [T,k]) and gate weights (fp32 [T,k]) of fp32 or bf16
    logits [T,E] by a RouteRule; `bias` (fp32 [E]) counts in the selection only."""
    args, _, _, _, _, index, topk_idx, topk_w = _route_args(logits, bias, rule, topk_idx, topk_w)
    _call("moe_route_grouped", index, *args)
    return topk_idx, topk_w


def moe_route_grouped_bucket(logits: torch.Tensor, bias: Optional[torch.Tensor], rule: RouteRule,
                             topk_idx: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
                             out: Optional[Buckets] = None):
    """moe_route_grouped and moe_bucket_routes in one call: ids, weights, buckets."""
    args, T, E, k, dev, index, topk_idx, topk_w = _route_args(logits, bias, rule, topk_idx, topk_w)
    b = out if out is not None else empty_buckets(T, E, max(k, 0), dev)
    count, offset, active, n_active, src, pos = b
    _tensor(count, "expert_count", _I32, (E,), dev, index)
    _tensor(offset, "expert_offset", _I32, (E + 1,), dev, index)
    _tensor(active, "active_experts", _I32, (E,), dev, index)
    _tensor(n_active, "n_active", _I32, (1,), dev, index)
    _tensor(src, "route_src", _I32, (T * k,), dev, index)
    _tensor(pos, "route_pos", _I32, (T * k,), dev, index)
    _call("moe_route_grouped_bucket", index, *args, count.data_ptr(), offset.data_ptr(), active.data_ptr(),
          n_active.data_ptr(), src.data_ptr(), pos.data_ptr())
    return topk_idx, topk_w, b


class QuantWeight(_Fixed):
    """A dense 4-bit matrix [N, K] on the device: `codes` uint8 [N, K/2],
    `scales` uint8 [N, K/16] ("nvfp4") or [N, K/32] ("mxfp4") and the global
    scale, fp32 [1] (None: 1, "mxfp4" only).  The bytes are not read here: no
    scale is NaN or negative, and those of "mxfp4" are at most 252."""

    __slots__ = ("codes", "scales", "g_scale", "format", "N", "K", "device", "_format", "_index")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, g_scale: Optional[torch.Tensor] = None,
                 format: str = "nvfp4"):
        if format not in _FORMATS:
            raise ValueError(f"format must be one of {tuple(_FORMATS)}, got {format!r}")
        number, group = _FORMATS[format]
        if not isinstance(codes, torch.Tensor) or codes.dim() != 2:
            raise TypeError("codes must be a [N, K/2] tensor")
        N, K, device = codes.shape[0], 2 * codes.shape[1], codes.device
        if K % 32 != 0 or K == 0 or N == 0:
            raise ValueError(f"a 4-bit matrix needs N >= 1 and K a multiple of 32, got N={N}, K={K}")
        _int(N, "N"), _int(K, "K")
        _need(codes, "codes", torch.uint8, None, device)
        _need(scales, "scales", torch.uint8, (N, K // group), device)
        if g_scale is not None:
            _need(g_scale, "g_scale", torch.float32, (1,), device)
        elif format == "nvfp4":
            raise ValueError("nvfp4 weights need their global scale (g_scale)")
        self._set(codes=codes, scales=scales, g_scale=g_scale, format=format, N=N, K=K, device=device, _format=number,
                  _index=codes.get_device())

    @property
    def shape(self):
        return self.N, self.K

    def _ptrs(self):
        g = self.g_scale
        return self.codes.data_ptr(), self.scales.data_ptr(), None if g is None else g.data_ptr()


def _check_quant_x(x, weight: QuantWeight) -> int:
    if not isinstance(x, Tensor) or x.dim() != 2:
        raise TypeError("x must be a [T, K] tensor")
    T = x.shape[0]
    if T > _MAX_INT:
        raise ValueError(f"x must have at most 2^31 - 1 tokens, got {T}")
    _tensor(x, "x", _BF16, (T, weight.K), weight.device, weight._index)
    return T


QUANT_SUMS_BYTES = 8 << 20         # MOE_QUANT_SUMS_BYTES


def moe_quant_linear_workspace_size(T: int, N: int, K: int) -> int:
    return int(load_library().moe_quant_linear_workspace_size(_int(T, "T"), _int(N, "N"), _int(K, "K")))


def moe_quant_linear(x: torch.Tensor, weight: QuantWeight, bias: Optional[torch.Tensor] = None,
                     y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """bf16 y [T,N] = x W^T + bias for bf16 x [T,K], a QuantWeight [N,K] and an
    optional bf16 bias [N].  The workspace (uint8, for batches that need one;
    QUANT_SUMS_BYTES serve every batch) is allocated where none is given."""
    T, N, dev, index = _check_quant_x(x, weight), weight.N, weight.device, weight._index
    if bias is not None:
        _tensor(bias, "bias", _BF16, (N,), dev, index)
    if y is None:
        y = torch.empty((T, N), dtype=_BF16, device=dev)
    else:
        _tensor(y, "y", _BF16, (T, N), dev, index)
    if workspace is not None:
        _tensor(workspace, "workspace", _U8, getattr(workspace, "shape", None), dev, index)
    elif T > 4 or weight.K > 8192:                   # no workspace below that
        need = load_library().moe_quant_linear_workspace_size(T, N, weight.K)
        workspace = torch.empty((need,), dtype=_U8, device=dev) if need else None
    x_at, y_at = x.data_ptr(), y.data_ptr()
    if x_at == y_at and T > 0:
        raise ValueError("y must not be x: its rows are written while x is read")
    _call("moe_quant_linear", index, weight._format, x_at, *weight._ptrs(),
          None if bias is None else bias.data_ptr(), T, N, weight.K,
          None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel(), y_at)
    return y


def moe_quant_shared_expert_workspace_size(T: int, H: int, Is: int) -> int:
    return int(load_library().moe_quant_shared_expert_workspace_size(_int(T, "T"), _int(H, "H"), _int(Is, "Is")))


def make_quant_shared_workspace(T: int, H: int, Is: int, device) -> torch.Tensor:
    """A workspace for moe_quant_shared_expert, reusable across calls of these
    weights' sizes and of up to T tokens.  (The size that one call needs is not
    the largest for the largest batch.)"""
    up = lambda n: (n + 255) & ~255  # noqa: E731
    T, Is = max(T, 0), max(Is, 0)
    return torch.empty((up(2 * T * Is) + up(4 * T) + QUANT_SUMS_BYTES,), dtype=torch.uint8, device=device)


def moe_quant_shared_expert(x: torch.Tensor, gate: QuantWeight, up: QuantWeight, down: QuantWeight,
                            token_gate: Optional[torch.Tensor] = None, add: Optional[torch.Tensor] = None,
                            y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The 4-bit shared expert: bf16 y [T,H] = add + sigmoid(x . token_gate) *
    W_down (SiLU(W_gate x) * (W_up x)), gate/up [Is,H] and down [H,Is] of one
    format; `token_gate` (bf16 [H]) and `add` (bf16 [T,H], may be y) optional."""
    T, H, Is, dev, index = _check_quant_x(x, gate), gate.K, gate.N, gate.device, gate._index
    if up.N != Is or up.K != H or down.N != H or down.K != Is:
        raise ValueError(f"gate is {gate.shape}, up {up.shape}, down {down.shape}: up must be gate's shape, down its "
                         "transpose's")
    if not (gate._format == up._format == down._format):
        raise ValueError("gate, up and down must have one format")
    if not (up._index == index and down._index == index):
        raise ValueError(f"gate is on {dev}, up on {up.device}, down on {down.device}")
    if token_gate is not None:
        _tensor(token_gate, "token_gate", _BF16, (H,), dev, index)
    if add is not None:
        _tensor(add, "add", _BF16, (T, H), dev, index)
    if y is None:
        y = torch.empty((T, H), dtype=_BF16, device=dev)
    else:
        _tensor(y, "y", _BF16, (T, H), dev, index)
    if workspace is None:
        workspace = torch.empty((moe_quant_shared_expert_workspace_size(T, H, Is),), dtype=_U8, device=dev)
    else:
        _tensor(workspace, "workspace", _U8, getattr(workspace, "shape", None), dev, index)
    x_at, y_at = x.data_ptr(), y.data_ptr()
    if x_at == y_at and T > 0:
        raise ValueError("y must not be x: its rows are written while x is read")
    _call("moe_quant_shared_expert", index, gate._format, x_at, *gate._ptrs(), *up._ptrs(), *down._ptrs(),
          None if token_gate is None else token_gate.data_ptr(), None if add is None else add.data_ptr(),
          T, H, Is, workspace.data_ptr(), workspace.numel(), y_at)
    return y
