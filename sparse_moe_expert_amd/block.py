"""Binding of the block-scaled 8-bit operators: norm and quantiser, a dense
layer, the routed experts (argument marshalling only, as in _lib and layer).

Values are e4m3 codes (torch.float8_e4m3fn) with fp32 scales: of 128
consecutive values of a token, of a block of 128 x 128 of a weight.
"""

from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from ._lib import Buckets, _need, load_library
from .layer import _BF16, _DTYPES, _F32, _I32, _MAX_INT, _U8, _Fixed, _call, _int, _tensor

Tensor = torch.Tensor
_E4M3 = torch.float8_e4m3fn
BLOCK = 128                          # values that share a scale
BLOCK_SUMS_BYTES = 16 << 20          # MOE_BLOCK_SUMS_BYTES


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


class Fp8Tokens(NamedTuple):
    q: torch.Tensor        # float8_e4m3fn [T, K]
    scale: torch.Tensor    # fp32 [T, ceil(K/128)]


def empty_fp8_tokens(T: int, K: int, device) -> Fp8Tokens:
    return Fp8Tokens(torch.empty((T, K), dtype=_E4M3, device=device),
                     torch.empty((T, _blocks(K)), dtype=_F32, device=device))


def _check_weight(q, scale, name: str, dims: int, device=None):
    if not isinstance(q, Tensor) or q.dim() != dims:
        raise TypeError(f"{name} must be a tensor of {dims} dimensions")
    *lead, N, K = q.shape
    if K % 16 != 0 or K == 0 or N == 0:
        raise ValueError(f"{name}: an 8-bit matrix needs N >= 1 and K a multiple of 16, got N={N}, K={K}")
    _int(N, "N"), _int(K, "K")
    _need(q, name, _E4M3, None, device)
    _need(scale, f"{name}'s scale", _F32, (*lead, _blocks(N), _blocks(K)), q.device)


class Fp8Weight(_Fixed):
    """A dense 8-bit matrix [N, K] on the device: `q` float8_e4m3fn [N, K] and
    `scale` fp32 [ceil(N/128), ceil(K/128)], K a multiple of 16."""

    __slots__ = ("q", "scale", "N", "K", "device", "_index")

    def __init__(self, q: torch.Tensor, scale: torch.Tensor):
        _check_weight(q, scale, "q", 2)
        self._set(q=q, scale=scale, N=q.shape[0], K=q.shape[1], device=q.device, _index=q.get_device())

    @property
    def shape(self):
        return self.N, self.K


class Fp8Experts(_Fixed):
    """The 8-bit weights of E experts on the device: `w_gate`, `w_up`
    float8_e4m3fn [E, I, H], `w_down` [E, H, I] and the fp32 scales of their
    blocks, `s_gate`, `s_up` [E, ceil(I/128), ceil(H/128)], `s_down`."""

    __slots__ = ("w_gate", "s_gate", "w_up", "s_up", "w_down", "s_down", "E", "H", "I", "device", "_index")

    def __init__(self, w_gate: torch.Tensor, s_gate: torch.Tensor, w_up: torch.Tensor, s_up: torch.Tensor,
                 w_down: torch.Tensor, s_down: torch.Tensor):
        _check_weight(w_gate, s_gate, "w_gate", 3)
        _check_weight(w_up, s_up, "w_up", 3, w_gate.device)
        _check_weight(w_down, s_down, "w_down", 3, w_gate.device)
        E, I, H = w_gate.shape  # noqa: E741
        if tuple(w_up.shape) != (E, I, H) or tuple(w_down.shape) != (E, H, I):
            raise ValueError(f"w_gate is {tuple(w_gate.shape)}, w_up {tuple(w_up.shape)}, w_down {tuple(w_down.shape)}: "
                             "w_up must be w_gate's shape, w_down [E, H, I]")
        self._set(w_gate=w_gate, s_gate=s_gate, w_up=w_up, s_up=s_up, w_down=w_down, s_down=s_down, E=E, H=H, I=I,
                  device=w_gate.device, _index=w_gate.get_device())

    @property
    def shape(self):
        return self.E, self.H, self.I

    def _ptrs(self):
        return (self.w_gate.data_ptr(), self.s_gate.data_ptr(), self.w_up.data_ptr(), self.s_up.data_ptr(),
                self.w_down.data_ptr(), self.s_down.data_ptr())


def _rows(x, name: str):
    """The sizes and device of bf16 rows [T, K]"""
    if not isinstance(x, Tensor) or x.dim() != 2:
        raise TypeError(f"{name} must be a [T, K] tensor")
    (T, K), dev, index = x.shape, x.device, x.get_device()
    if T > _MAX_INT or K > _MAX_INT:
        raise ValueError(f"{name} must have at most 2^31 - 1 rows and columns, got {T} and {K}")
    if x.dtype is not _BF16 or index < 0 or not x.is_contiguous():
        _need(x, name, _BF16)
    return T, K, dev, index


def _tokens_out(out, T: int, K: int, dev, index: int):
    if out is None:
        return empty_fp8_tokens(T, K, dev)
    q, scale = out
    _tensor(q, "q", _E4M3, (T, K), dev, index)
    _tensor(scale, "scale", _F32, (T, _blocks(K)), dev, index)
    return out


def moe_norm_quantize(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                      eps: float = 1e-6, weight_offset: float = 0.0, out: Optional[Fp8Tokens] = None,
                      residual_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None):
    """(tokens, r): r = x + residual (bf16 or fp32 [T,H]; None without one) and
    the 8-bit form of y = RMSNorm(r) * (weight + weight_offset), for bf16 x
    [T,H] and weight [H].  `residual_out` may be `residual`; a bf16 `y` [T,H]
    receives y as well."""
    T, H, dev, index = _rows(x, "x")
    _tensor(weight, "weight", _BF16, (H,), dev, index)
    kind = 0
    if residual is not None:
        kind = _DTYPES.get(getattr(residual, "dtype", None))
        if kind is None:
            raise TypeError("residual must be a float32 or bfloat16 tensor")
        _tensor(residual, "residual", residual.dtype, (T, H), dev, index)
        if residual_out is None:
            residual_out = torch.empty_like(residual)
        else:
            _tensor(residual_out, "residual_out", residual.dtype, (T, H), dev, index)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if y is not None:
        _tensor(y, "y", _BF16, (T, H), dev, index)
    out = _tokens_out(out, T, H, dev, index)
    _call("moe_norm_quantize", index, x.data_ptr(), None if residual is None else residual.data_ptr(), kind,
          weight.data_ptr(), weight_offset, eps, T, H, None if residual_out is None else residual_out.data_ptr(),
          None if y is None else y.data_ptr(), out[0].data_ptr(), out[1].data_ptr())
    return out, residual_out


def moe_block_quantize(x: torch.Tensor, out: Optional[Fp8Tokens] = None) -> Fp8Tokens:
    """bf16 x [T,K] in 8 bits."""
    T, K, dev, index = _rows(x, "x")
    out = _tokens_out(out, T, K, dev, index)
    _call("moe_block_quantize", index, x.data_ptr(), T, K, out[0].data_ptr(), out[1].data_ptr())
    return out


def _check_tokens(x, K: int, dev, index: int) -> int:
    q, scale = x
    if not isinstance(q, Tensor) or q.dim() != 2:
        raise TypeError("q must be a [T, K] tensor")
    T = q.shape[0]
    if T > _MAX_INT:
        raise ValueError(f"q must have at most 2^31 - 1 tokens, got {T}")
    _tensor(q, "q", _E4M3, (T, K), dev, index)
    _tensor(scale, "scale", _F32, (T, _blocks(K)), dev, index)
    return T


def moe_block_linear_workspace_size(T: int, N: int, K: int) -> int:
    return int(load_library().moe_block_linear_workspace_size(_int(T, "T"), _int(N, "N"), _int(K, "K")))


def make_block_linear_workspace(device) -> torch.Tensor:
    """A workspace that serves every moe_block_linear call."""
    return torch.empty((BLOCK_SUMS_BYTES,), dtype=_U8, device=device)


def moe_block_linear(x: Fp8Tokens, weight: Fp8Weight, bias: Optional[torch.Tensor] = None,
                     y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """bf16 y [T,N] = x W^T + bias for 8-bit tokens [T,K], an Fp8Weight [N,K] and
    an optional bf16 bias [N].  The workspace (uint8, for sizes that need one)
    is allocated where none is given."""
    N, K, dev, index = weight.N, weight.K, weight.device, weight._index
    T = _check_tokens(x, K, dev, index)
    if bias is not None:
        _tensor(bias, "bias", _BF16, (N,), dev, index)
    if y is None:
        y = torch.empty((T, N), dtype=_BF16, device=dev)
    else:
        _tensor(y, "y", _BF16, (T, N), dev, index)
    if workspace is None:
        need = load_library().moe_block_linear_workspace_size(T, N, K)
        workspace = torch.empty((need,), dtype=_U8, device=dev) if need else None
    else:
        _tensor(workspace, "workspace", _U8, getattr(workspace, "shape", None), dev, index)
    x_at, y_at = x[0].data_ptr(), y.data_ptr()
    if x_at == y_at and T > 0:
        raise ValueError("y must not be x: its rows are written while x is read")
    _call("moe_block_linear", index, x_at, x[1].data_ptr(), weight.q.data_ptr(), weight.scale.data_ptr(),
          None if bias is None else bias.data_ptr(), T, N, K, None if workspace is None else workspace.data_ptr(),
          0 if workspace is None else workspace.numel(), y_at)
    return y


def moe_block_expert_ffn_workspace_size(T: int, H: int, I: int, E: int, k: int) -> int:
    return int(load_library().moe_block_expert_ffn_workspace_size(
        _int(T, "T"), _int(H, "H"), _int(I, "I"), _int(E, "E"), _int(k, "k")))


def make_block_ffn_workspace(T: int, H: int, I: int, E: int, k: int, device) -> torch.Tensor:
    """A workspace for moe_block_expert_ffn, reusable across calls of these sizes
    and of up to T tokens."""
    n = max(moe_block_expert_ffn_workspace_size(T, H, I, E, k), 256)
    return torch.empty((n,), dtype=_U8, device=device)


def moe_block_expert_ffn(x: Fp8Tokens, experts: Fp8Experts, topk_w: torch.Tensor, buckets: Buckets,
                         workspace: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """bf16 y [T,H] of the routed 8-bit experts for 8-bit tokens [T,H], gate
    weights fp32 topk_w [T,k] and the buckets of their ids."""
    E, H, I = experts.E, experts.H, experts.I  # noqa: E741
    dev, index = experts.device, experts._index
    T = _check_tokens(x, H, dev, index)
    if not isinstance(topk_w, Tensor) or topk_w.dim() != 2:
        raise TypeError("topk_w must be a [T, k] tensor")
    k = topk_w.shape[1]
    _tensor(topk_w, "topk_w", _F32, (T, k), dev, index)
    count, offset, active, n_active, src, pos = buckets
    _tensor(count, "expert_count", _I32, (E,), dev, index)
    _tensor(offset, "expert_offset", _I32, (E + 1,), dev, index)
    _tensor(active, "active_experts", _I32, (E,), dev, index)
    _tensor(n_active, "n_active", _I32, (1,), dev, index)
    _tensor(src, "route_src", _I32, (T * k,), dev, index)
    _tensor(pos, "route_pos", _I32, (T * k,), dev, index)
    if y is None:
        y = torch.empty((T, H), dtype=_BF16, device=dev)
    else:
        _tensor(y, "y", _BF16, (T, H), dev, index)
    if workspace is None:
        workspace = make_block_ffn_workspace(T, H, I, E, k, dev)
    else:
        _tensor(workspace, "workspace", _U8, getattr(workspace, "shape", None), dev, index)
    x_at, y_at = x[0].data_ptr(), y.data_ptr()
    if x_at == y_at and T > 0:
        raise ValueError("y must not be x: its rows are written while x is read")
    _call("moe_block_expert_ffn", index, x_at, x[1].data_ptr(), *experts._ptrs(), topk_w.data_ptr(),
          count.data_ptr(), offset.data_ptr(), active.data_ptr(), n_active.data_ptr(), src.data_ptr(), pos.data_ptr(),
          T, H, I, E, k, workspace.data_ptr(), workspace.numel(), y_at)
    return y
