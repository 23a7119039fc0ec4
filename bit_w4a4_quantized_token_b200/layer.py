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

from dataclasses import dataclass

import torch

from . import _lib

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


@dataclass
class PackedWeightW8A8:
    N: int
    K: int
    w_codes: torch.Tensor               # int8 [N, K]
    w_scales: torch.Tensor              # fp32 [N]
    inv_lambda: torch.Tensor | None     # fp32 [K]: 1 / lambda, None without smoothing
    bias: torch.Tensor | None           # [N], of the output's type


@dataclass
class QuantizedActW8A8:
    M: int
    x_codes: torch.Tensor               # int8 [M, K]
    x_scales: torch.Tensor              # fp32 [M]


# The small calls of this layer are bound by what the host does per call, so the current device and stream are
# asked for without building torch.cuda's objects (3 us for current_stream alone), and the library is called with
# plain addresses.
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


def _check_tensor(name: str, t: torch.Tensor, dtype, shape: tuple, index: int) -> None:
    """What the library cannot see of a contiguous operand behind its pointer (index: the call's GPU)."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on GPU {index}, got "
                         f"{t.dtype} {tuple(t.shape)} (strides {t.stride()}) on {t.device}")


def _check_rows(name: str, x: torch.Tensor, K: int) -> int:
    """The library's type of a matrix of activations; rows may be apart, elements of a row not."""
    dtype = _DTYPES.get(x.dtype)
    if dtype is None or x.dim() != 2 or x.shape[1] != K or not x.is_cuda or (x.stride(1) != 1 and K > 1):
        raise ValueError(f"{name}: expected a CUDA matrix [M, {K}] of bf16, fp16 or fp32 with contiguous rows, got "
                         f"{x.dtype} {tuple(x.shape)} (strides {x.stride()}) on {x.device}")
    return dtype


def _row_stride(x: torch.Tensor) -> int:
    return x.stride(0) if x.shape[0] > 1 else x.shape[1]


def _addr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _call(name: str, index: int, args: tuple) -> None:
    """Calls a library entry point on the current stream of GPU `index`."""
    if _current_device() != index:
        with torch.cuda.device(index):
            return _call(name, index, args)
    status = getattr(_lib.lib, name)(*args, _current_stream(index))
    if status != _lib.SVDQ_OK:
        raise _lib.SvdqError(status, name)


def _tensors(v):
    """The tensors of an argument or a result."""
    if isinstance(v, torch.Tensor):
        yield v
    elif isinstance(v, (PackedWeightW8A8, QuantizedActW8A8)):
        yield from _tensors(tuple(vars(v).values()))
    elif isinstance(v, tuple):
        for t in v:
            yield from _tensors(t)


def _on_stream(stream, x: torch.Tensor, fn, *args):
    """fn(*args) with `stream` (a torch stream or a raw handle) current, so that what it allocates is ordered with
    that stream's work.  The tensors it reads are marked as in use there, those it returns as in use on the caller's
    stream, so that the allocator hands out no memory early; the two streams' order is the caller's to keep."""
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
    N, K = W.shape
    w_type = _check_rows("W", W, K)
    W = W.contiguous()
    dev, index = W.device, W.get_device()
    if lam is not None:
        _check_tensor("lam", lam, torch.float32, (K,), index)
    if bias is not None and (bias.shape != (N,) or bias.dtype not in _DTYPES or bias.get_device() != index):
        raise ValueError(f"bias: expected a bf16, fp16 or fp32 tensor of shape ({N},) on {dev}, got {bias.dtype} "
                         f"{tuple(bias.shape)} on {bias.device}")
    w_codes = torch.empty(N, K, dtype=torch.int8, device=dev)
    w_scales = torch.empty(N, dtype=torch.float32, device=dev)
    inv_lambda = torch.empty(K, dtype=torch.float32, device=dev) if lam is not None else None
    _call("svdq_pack_weight_w8a8", index,
          (w_type, W.data_ptr(), N, K, _addr(lam), w_codes.data_ptr(), w_scales.data_ptr(), _addr(inv_lambda)))
    return PackedWeightW8A8(N, K, w_codes, w_scales, inv_lambda, None if bias is None else bias.contiguous())


def alloc_act_w8a8(packed: PackedWeightW8A8, M: int, device) -> QuantizedActW8A8:
    return QuantizedActW8A8(M, torch.empty((M, packed.K), dtype=torch.int8, device=device),
                            torch.empty((M,), dtype=torch.float32, device=device))


def _act_out(packed: PackedWeightW8A8, M: int, x: torch.Tensor, index: int,
             out: QuantizedActW8A8 | None) -> QuantizedActW8A8:
    if out is None:
        return alloc_act_w8a8(packed, M, x.device)
    _check_tensor("out.x_codes", out.x_codes, torch.int8, (M, packed.K), index)
    _check_tensor("out.x_scales", out.x_scales, torch.float32, (M,), index)
    return out


def quantize_act_w8a8(x: torch.Tensor, packed: PackedWeightW8A8, out: QuantizedActW8A8 | None = None,
                      stream=None) -> QuantizedActW8A8:
    """x [M, K] bf16, fp16 or fp32 (rows may be apart) -> 8-bit codes and a scale per token."""
    if stream is not None:
        return _on_stream(stream, x, quantize_act_w8a8, x, packed, out)
    K, inv_lambda = packed.K, packed.inv_lambda
    x_type = _check_rows("x", x, K)
    M, index = x.shape[0], x.get_device()
    if inv_lambda is not None:
        _check_tensor("packed.inv_lambda", inv_lambda, torch.float32, (K,), index)
    q = _act_out(packed, M, x, index, out)
    _call("svdq_quantize_act_w8a8", index,
          (x_type, x.data_ptr(), _row_stride(x), M, K, _addr(inv_lambda), q.x_codes.data_ptr(),
           q.x_scales.data_ptr()))
    return q


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
    K, inv_lambda = packed.K, packed.inv_lambda
    x_type = _check_rows("x", x, K)
    M, index, dt = x.shape[0], x.get_device(), x.dtype
    ldr = K
    if residual is not None:
        if _check_rows("residual", residual, K) != x_type or residual.shape[0] != M or residual.get_device() != index:
            raise ValueError(f"residual: expected {dt} {(M, K)} on {x.device}, got {residual.dtype} "
                             f"{tuple(residual.shape)} on {residual.device}")
        ldr = _row_stride(residual)
    if norm_weight is not None:
        _check_tensor("norm_weight", norm_weight, dt, (K,), index)
    if inv_lambda is not None:
        _check_tensor("packed.inv_lambda", inv_lambda, torch.float32, (K,), index)
    if h_out is not None:
        _check_tensor("h_out", h_out, dt, (M, K), index)
    elif residual is not None:
        h_out = torch.empty((M, K), dtype=dt, device=x.device)
    if normed is not None:
        _check_tensor("normed", normed, dt, (M, K), index)
    q = _act_out(packed, M, x, index, out)
    _call("svdq_rms_norm_quantize_w8a8", index,
          (x_type, x.data_ptr(), _row_stride(x), _addr(residual), ldr, M, K, _addr(norm_weight), eps,
           _addr(inv_lambda), _addr(h_out), _addr(normed), q.x_codes.data_ptr(), q.x_scales.data_ptr()))
    return (x if h_out is None else h_out), q


def gemm_w8a8(q: QuantizedActW8A8, packed: PackedWeightW8A8, y: torch.Tensor | None = None,
              out_dtype: torch.dtype | None = None, stream=None) -> torch.Tensor:
    """y [M, N] = x_scales[m] w_scales[n] sum_k codes + bias, in out_dtype (default: y's type, else the bias's,
    else bf16); the bias has that type too."""
    if stream is not None:
        return _on_stream(stream, q.x_codes, gemm_w8a8, q, packed, y, out_dtype)
    M, N, K, bias = q.M, packed.N, packed.K, packed.bias
    if out_dtype is None:
        out_dtype = y.dtype if y is not None else bias.dtype if bias is not None else torch.bfloat16
    y_type = _DTYPES.get(out_dtype)
    if y_type is None:
        raise ValueError(f"out_dtype: expected bf16, fp16 or fp32, got {out_dtype}")
    x_codes, x_scales, w_codes, w_scales = q.x_codes, q.x_scales, packed.w_codes, packed.w_scales
    index = x_codes.get_device()
    _check_tensor("q.x_codes", x_codes, torch.int8, (M, K), index)
    _check_tensor("q.x_scales", x_scales, torch.float32, (M,), index)
    _check_tensor("packed.w_codes", w_codes, torch.int8, (N, K), index)
    _check_tensor("packed.w_scales", w_scales, torch.float32, (N,), index)
    if bias is not None:
        _check_tensor("packed.bias", bias, out_dtype, (N,), index)
    if y is not None:
        _check_tensor("y", y, out_dtype, (M, N), index)
    if index < 0:
        raise ValueError(f"expected CUDA tensors, got tensors on {x_codes.device}")
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=x_codes.device)
    _call("svdq_gemm_w8a8", index,
          (x_codes.data_ptr(), x_scales.data_ptr(), M, w_codes.data_ptr(), w_scales.data_ptr(), N, K, _addr(bias),
           y_type, y.data_ptr()))
    return y


def w8a8_linear(x: torch.Tensor, packed: PackedWeightW8A8, out_dtype: torch.dtype | None = None,
                stream=None) -> torch.Tensor:
    """One forward of the W8A8 linear layer: two launches, no host sync.  y is in out_dtype, by default the
    bias's type or, without one, x's."""
    if out_dtype is None:
        out_dtype = packed.bias.dtype if packed.bias is not None else x.dtype
    return gemm_w8a8(quantize_act_w8a8(x, packed, stream=stream), packed, out_dtype=out_dtype, stream=stream)
