"""PyTorch-facing helpers around the C ABI: they allocate the packed buffers as
torch tensors and call the entry points in order.  Device memory and streams
come from PyTorch; every step of the layer runs in the CUDA library.

    packed = pack_weight(R, lam, L_down, L_up, precision="nvfp4")   # once per layer
    y = svdq_linear(x, packed)                                      # quantize_act + gemm_w4a4

The 8-bit integer (W8A8) layer, for the layers that 4 bits cost too much:

    packed = pack_weight_w8a8(W, lam, bias)                         # once per layer
    y = w8a8_linear(x, packed)                                      # quantize_act_w8a8 + gemm_w8a8
    h, q = rms_norm_quantize_w8a8(x, residual, norm_weight, packed) # residual + RMSNorm + quantizer in one pass
    y = gemm_w8a8(q, packed)
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from dataclasses import dataclass, fields

import torch

from . import _lib, build

_U8 = torch.uint8


def _empty(nbytes: int, device) -> torch.Tensor:
    # 256-byte aligned by the caching allocator; at least one byte so data_ptr is valid
    return torch.empty(max(int(nbytes), 1), dtype=_U8, device=device)


@dataclass
class PackedWeight:
    precision: str
    N: int
    K: int
    rank: int
    w_codes: torch.Tensor
    w_scales: torch.Tensor
    w_tensor_scale: torch.Tensor | None
    inv_lambda: torch.Tensor
    L_down_t: torch.Tensor | None
    L_up_t: torch.Tensor | None
    bias: torch.Tensor | None

    @property
    def group_size(self) -> int:
        return _lib.GROUP_SIZES[self.precision]


@dataclass
class QuantizedAct:
    M: int
    x_codes: torch.Tensor
    x_scales: torch.Tensor
    x_tensor_scale: torch.Tensor | None
    lowrank_act: torch.Tensor | None
    workspace: torch.Tensor | None = None   # zero-filled once; the library keeps it zeroed


def pack_weight(R: torch.Tensor, lam: torch.Tensor, L_down: torch.Tensor | None, L_up: torch.Tensor | None,
                bias: torch.Tensor | None = None, precision: str = "nvfp4", stream=None) -> PackedWeight:
    N, K = R.shape
    rank = 0 if L_down is None else int(L_down.shape[1])
    dev = R.device
    sz = _lib.svdq_buffer_sizes(precision, N, K, rank)
    w_codes = _empty(sz["codes_bytes"], dev)
    w_scales = _empty(sz["w_scales_bytes"], dev)   # nvfp4: block layout, then the GEMM-ready copy
    w_ts = torch.empty(4, dtype=torch.float32, device=dev) if precision == "nvfp4" else None
    inv_lambda = torch.empty(K, dtype=torch.float32, device=dev)
    L_down_t = torch.empty(2, rank, K, dtype=torch.bfloat16, device=dev) if rank else None
    L_up_t = torch.empty(N, rank, dtype=torch.bfloat16, device=dev) if rank else None
    _lib.svdq_pack_weight(precision, _lib.GROUP_SIZES[precision], R.contiguous(), N, K, lam.contiguous(),
                          None if rank == 0 else L_down.contiguous(), None if rank == 0 else L_up.contiguous(),
                          rank, w_codes, w_scales, w_ts, inv_lambda, L_down_t, L_up_t, stream)
    return PackedWeight(precision, N, K, rank, w_codes, w_scales, w_ts, inv_lambda, L_down_t, L_up_t,
                        None if bias is None else bias.contiguous())


def alloc_act(packed: PackedWeight, M: int, device) -> QuantizedAct:
    sz = _lib.svdq_buffer_sizes(packed.precision, M, packed.K, packed.rank)
    ws = _lib.svdq_quantize_act_workspace_bytes(packed.precision, M, packed.K, packed.rank)
    return QuantizedAct(
        M,
        _empty(sz["codes_bytes"], device),
        _empty(sz["scales_bytes"], device),
        torch.empty(4, dtype=torch.float32, device=device) if packed.precision == "nvfp4" else None,
        torch.empty(2, M, packed.rank, dtype=torch.bfloat16, device=device) if packed.rank else None,
        torch.zeros(ws, dtype=torch.uint8, device=device) if ws else None,
    )


def quantize_act(x: torch.Tensor, packed: PackedWeight, out: QuantizedAct | None = None,
                 x_tensor_scale: float | torch.Tensor | None = None, stream=None) -> QuantizedAct:
    """x [M, K] bf16 -> codes, scales, rank-r activations.  x_tensor_scale None
    derives S_x from amax on the device; a float or a device tensor is used as
    a static scale."""
    M, K = x.shape
    assert K == packed.K
    q = out if out is not None else alloc_act(packed, M, x.device)
    compute = 1
    if packed.precision == "nvfp4" and x_tensor_scale is not None:
        compute = 0
        if isinstance(x_tensor_scale, torch.Tensor):
            q.x_tensor_scale[:1].copy_(x_tensor_scale.reshape(-1)[:1])
        else:
            q.x_tensor_scale.fill_(float(x_tensor_scale))
    _lib.svdq_quantize_act(packed.precision, packed.group_size, x, M, K, packed.inv_lambda, q.x_tensor_scale,
                           compute, packed.w_tensor_scale, packed.L_down_t, packed.rank, q.x_codes, q.x_scales,
                           q.lowrank_act, q.workspace, stream=stream)
    return q


def gemm(q: QuantizedAct, packed: PackedWeight, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    if y is None:
        y = torch.empty(q.M, packed.N, dtype=torch.bfloat16, device=q.x_codes.device)
    _lib.svdq_gemm_w4a4(packed.precision, packed.group_size, q.x_codes, q.x_scales, q.x_tensor_scale, q.M,
                        packed.w_codes, packed.w_scales, packed.w_tensor_scale, packed.N, packed.K, q.lowrank_act,
                        packed.L_up_t, packed.rank, packed.bias, y, stream)
    return y


def svdq_linear(x: torch.Tensor, packed: PackedWeight, x_tensor_scale=None, stream=None) -> torch.Tensor:
    """One forward of the SVDQ W4A4 linear layer: two launches, no host sync."""
    return gemm(quantize_act(x, packed, x_tensor_scale=x_tensor_scale, stream=stream), packed, stream=stream)


# ----------------------------------------------------------------- W8A8 layer
_DTYPES = {torch.bfloat16: _lib.SVDQ_BF16, torch.float16: _lib.SVDQ_F16, torch.float32: _lib.SVDQ_F32}


@dataclass(slots=True)
class PackedWeightW8A8:
    N: int
    K: int
    w_codes: torch.Tensor               # int8 [N, K]
    w_scales: torch.Tensor              # fp32 [N]
    inv_lambda: torch.Tensor | None     # fp32 [K]: 1 / lambda, None without smoothing
    bias: torch.Tensor | None           # [N], of the output's type


@dataclass(slots=True)
class QuantizedActW8A8:
    M: int
    x_codes: torch.Tensor               # int8 [M, K]
    x_scales: torch.Tensor              # fp32 [M]


def _raise_status(status: int, name: str) -> None:
    raise _lib.SvdqError(status, name)


class _Unloaded:
    """Stands for the native module of the W8A8 functions until one of them is called: what does not use it, the 4-bit
    layer, does not need it."""

    def __getattr__(self, name):
        global _front
        path = build.front_path()
        if not os.path.exists(path):
            raise ImportError(f"the native module of the W8A8 layer is not built for this Python and torch ({path}); "
                              "run __graft_entry__.build() (there is no fallback)")
        spec = importlib.util.spec_from_file_location(f"{__package__}._w8a8_front", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.bind(*(ctypes.cast(getattr(_lib.lib, fn), ctypes.c_void_p).value
                      for fn in ("svdq_pack_weight_w8a8", "svdq_quantize_act_w8a8", "svdq_rms_norm_quantize_w8a8",
                                 "svdq_gemm_w8a8")), _raise_status)
        _front = module
        return getattr(module, name)


# The operands' checks, the outputs' allocation and the library call are one call of a small native module: a layer
# call on few tokens is bound by what the host does for it, and in Python that was twice the GPU's time.
_front = _Unloaded()


def _tensors(v):
    """The tensors of an argument or a result."""
    if isinstance(v, torch.Tensor):
        yield v
    elif isinstance(v, (PackedWeightW8A8, QuantizedActW8A8)):
        yield from _tensors(tuple(getattr(v, f.name) for f in fields(v)))
    elif isinstance(v, tuple):
        for t in v:
            yield from _tensors(t)


def _on_stream(stream, x: torch.Tensor, fn, *args):
    """fn(*args) with `stream` (a torch stream or a raw handle) current, so that what it allocates is ordered with
    that stream's work.  The tensors it reads are marked as in use there, those it returns as in use on the caller's
    stream, so that the allocator hands out no memory early; the two streams' order is the caller's to keep."""
    if not isinstance(stream, int) and stream.device != x.device:
        raise ValueError(f"stream: expected a stream of {x.device}, where the operands are, got one of {stream.device}")
    caller = torch.cuda.current_stream(x.device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=x.device) if stream else torch.cuda.default_stream(x.device)
    with torch.cuda.stream(stream):
        result = fn(*args)
    if stream != caller:
        for t in _tensors(args):
            t.record_stream(stream)
        for t in _tensors(result):
            t.record_stream(caller)
    return result


def pack_weight_w8a8(W: torch.Tensor, lam: torch.Tensor | None = None, bias: torch.Tensor | None = None,
                     stream=None) -> PackedWeightW8A8:
    """W [N, K] bf16, fp16 or fp32 -> 8-bit codes and a scale per output channel.  With smoothing divisors
    lam [K] (fp32) the rows W * lam are quantised and activations are divided by lam."""
    if stream is not None:
        return _on_stream(stream, W, pack_weight_w8a8, W, lam, bias)
    w_codes, w_scales, inv_lambda = _front.pack(W, lam)
    N, K = W.shape
    if bias is not None:
        if bias.shape != (N,) or bias.dtype not in _DTYPES or bias.device != W.device:
            raise ValueError(f"bias: expected a bf16, fp16 or fp32 tensor of shape ({N},) on {W.device}, got "
                             f"{bias.dtype} {tuple(bias.shape)} on {bias.device}")
        bias = bias.contiguous()
    return PackedWeightW8A8(N, K, w_codes, w_scales, inv_lambda, bias)


def alloc_act_w8a8(packed: PackedWeightW8A8, M: int, device) -> QuantizedActW8A8:
    return QuantizedActW8A8(M, torch.empty(M, packed.K, dtype=torch.int8, device=device),
                            torch.empty(M, dtype=torch.float32, device=device))


def quantize_act_w8a8(x: torch.Tensor, packed: PackedWeightW8A8, out: QuantizedActW8A8 | None = None,
                      stream=None) -> QuantizedActW8A8:
    """x [M, K] bf16, fp16 or fp32 (rows may be apart) -> 8-bit codes and a scale per token."""
    if stream is not None:
        return _on_stream(stream, x, quantize_act_w8a8, x, packed, out)
    if out is not None:
        _front.quantize(x, packed.K, packed.inv_lambda, out.x_codes, out.x_scales)
        return out
    return QuantizedActW8A8(*_front.quantize(x, packed.K, packed.inv_lambda, None, None))


def rms_norm_quantize_w8a8(x: torch.Tensor, residual: torch.Tensor | None, norm_weight: torch.Tensor | None,
                           packed: PackedWeightW8A8, eps: float = 1e-6, h_out: torch.Tensor | None = None,
                           normed: torch.Tensor | None = None, out: QuantizedActW8A8 | None = None,
                           stream=None) -> tuple[torch.Tensor, QuantizedActW8A8]:
    """h = x + residual, its RMSNorm, and the 8-bit codes of that: returns (h, codes and scales).  h goes to h_out
    (a new tensor by default; x or residual itself for an update in place); with residual None and no h_out, h is
    x.  The normalised rows are also written, in x's type, to `normed` when that is given."""
    if stream is not None:
        return _on_stream(stream, x, rms_norm_quantize_w8a8, x, residual, norm_weight, packed, eps, h_out, normed,
                          out)
    codes, scales = (None, None) if out is None else (out.x_codes, out.x_scales)
    h, M, codes, scales = _front.norm(x, residual, norm_weight, packed.K, packed.inv_lambda, eps, h_out, normed,
                                      codes, scales)
    return h, (QuantizedActW8A8(M, codes, scales) if out is None else out)


def gemm_w8a8(q: QuantizedActW8A8, packed: PackedWeightW8A8, y: torch.Tensor | None = None,
              out_dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """y [M, N] = x_scales[m] w_scales[n] sum_k codes + bias, in out_dtype (default: y's type, else the bias's,
    else bf16); the bias has that type too."""
    if stream is not None:
        return _on_stream(stream, q.x_codes, gemm_w8a8, q, packed, y, out_dtype)
    bias = packed.bias
    if out_dtype is None:
        out_dtype = y.dtype if y is not None else bias.dtype if bias is not None else torch.bfloat16
    y_type = _DTYPES.get(out_dtype)
    if y_type is None:
        raise ValueError(f"out_dtype: expected bf16, fp16 or fp32, got {out_dtype}")
    return _front.gemm(q.x_codes, q.x_scales, q.M, packed.w_codes, packed.w_scales, packed.N, packed.K, bias, y_type, y)


def w8a8_linear(x: torch.Tensor, packed: PackedWeightW8A8, out_dtype: torch.dtype | None = None,
                stream=None) -> torch.Tensor:
    """One forward of the W8A8 linear layer: two launches, no host sync.  y is in out_dtype, by default the
    bias's type or, without one, x's."""
    if out_dtype is None:
        out_dtype = packed.bias.dtype if packed.bias is not None else x.dtype
    return gemm_w8a8(quantize_act_w8a8(x, packed, stream=stream), packed, out_dtype=out_dtype, stream=stream)
