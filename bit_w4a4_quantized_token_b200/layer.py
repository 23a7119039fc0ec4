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

from dataclasses import dataclass, fields

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


_I8, _F32 = torch.int8, torch.float32


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


# A call of this layer on few tokens is bound by what the host does for it, so these functions ask torch for the
# current device and stream without building torch.cuda's objects (3 us for current_stream alone), allocate with the
# allocator's short form where torch has it (0.7 us a tensor, torch.empty 2.3), test operands in one expression each
# and put the message together only for a refusal, and call the library with plain addresses.
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream
try:
    from torch._C._dynamo.guards import _empty_strided_cuda as _empty_strided   # (sizes, strides, dtype)
except ImportError:
    def _empty_strided(size, stride, dtype):
        return torch.empty_strided(size, stride, dtype=dtype, device="cuda")


def _unfit(t: torch.Tensor, dtype, shape: tuple, index: int) -> bool:
    """Whether a contiguous operand is not what the library will take it for behind its pointer."""
    return t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous()


def _refuse(name: str, t: torch.Tensor, dtype, shape: tuple, index: int) -> None:
    raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on GPU {index}, got "
                     f"{t.dtype} {tuple(t.shape)} (strides {t.stride()}) on {t.device}")


def _rows(name: str, x: torch.Tensor, K: int) -> tuple[int, int, int]:
    """(library's type, rows, row stride) of a matrix of activations; rows may be apart, elements of a row not."""
    x_type, shape, strides = _DTYPES.get(x.dtype), x.shape, x.stride()
    if x_type is None or len(shape) != 2 or shape[1] != K or strides[1] != 1 or not x.is_cuda:
        raise ValueError(f"{name}: expected a CUDA matrix [M, {K}] of bf16, fp16 or fp32 with contiguous rows, got "
                         f"{x.dtype} {tuple(shape)} (strides {strides}) on {x.device}")
    return x_type, shape[0], (strides[0] if shape[0] > 1 else K)


def _addr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _check(status: int, name: str) -> None:
    if status:
        raise _lib.SvdqError(status, name)


def _on_device(index: int, fn, *args):
    """fn(*args) with GPU `index` current: where the operands are is where everything happens."""
    with torch.cuda.device(index):
        return fn(*args)


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
    w_type = _rows("W", W, K)[0]
    W = W.contiguous()
    dev, index = W.device, W.get_device()
    if lam is not None and _unfit(lam, _F32, (K,), index):
        _refuse("lam", lam, _F32, (K,), index)
    if bias is not None and (bias.shape != (N,) or bias.dtype not in _DTYPES or bias.get_device() != index):
        raise ValueError(f"bias: expected a bf16, fp16 or fp32 tensor of shape ({N},) on {dev}, got {bias.dtype} "
                         f"{tuple(bias.shape)} on {bias.device}")
    if index != _current_device():
        return _on_device(index, pack_weight_w8a8, W, lam, bias)
    w_codes = torch.empty(N, K, dtype=_I8, device=dev)
    w_scales = torch.empty(N, dtype=_F32, device=dev)
    inv_lambda = torch.empty(K, dtype=_F32, device=dev) if lam is not None else None
    _check(_lib.lib.svdq_pack_weight_w8a8(w_type, W.data_ptr(), N, K, _addr(lam), w_codes.data_ptr(),
                                          w_scales.data_ptr(), _addr(inv_lambda), _current_stream(index)),
           "svdq_pack_weight_w8a8")
    return PackedWeightW8A8(N, K, w_codes, w_scales, inv_lambda, None if bias is None else bias.contiguous())


def alloc_act_w8a8(packed: PackedWeightW8A8, M: int, device) -> QuantizedActW8A8:
    return QuantizedActW8A8(M, torch.empty(M, packed.K, dtype=_I8, device=device),
                            torch.empty(M, dtype=_F32, device=device))


def _act(M: int, K: int) -> QuantizedActW8A8:
    """alloc_act_w8a8 on the current GPU."""
    return QuantizedActW8A8(M, _empty_strided((M, K), (K, 1), _I8), _empty_strided((M,), (1,), _F32))


def _check_out(out: QuantizedActW8A8, M: int, K: int, index: int) -> None:
    if _unfit(out.x_codes, _I8, (M, K), index):
        _refuse("out.x_codes", out.x_codes, _I8, (M, K), index)
    if _unfit(out.x_scales, _F32, (M,), index):
        _refuse("out.x_scales", out.x_scales, _F32, (M,), index)


def quantize_act_w8a8(x: torch.Tensor, packed: PackedWeightW8A8, out: QuantizedActW8A8 | None = None,
                      stream=None) -> QuantizedActW8A8:
    """x [M, K] bf16, fp16 or fp32 (rows may be apart) -> 8-bit codes and a scale per token."""
    if stream is not None:
        return _on_stream(stream, x, quantize_act_w8a8, x, packed, out)
    K, inv_lambda = packed.K, packed.inv_lambda
    x_type, M, ldx = _rows("x", x, K)
    index = x.get_device()
    if index != _current_device():
        return _on_device(index, quantize_act_w8a8, x, packed, out)
    if inv_lambda is not None and _unfit(inv_lambda, _F32, (K,), index):
        _refuse("packed.inv_lambda", inv_lambda, _F32, (K,), index)
    if out is None:
        out = _act(M, K)
    else:
        _check_out(out, M, K, index)
    _check(_lib.lib.svdq_quantize_act_w8a8(x_type, x.data_ptr(), ldx, M, K, _addr(inv_lambda), out.x_codes.data_ptr(),
                                           out.x_scales.data_ptr(), _current_stream(index)), "svdq_quantize_act_w8a8")
    return out


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
    x_type, M, ldx = _rows("x", x, K)
    index, dt = x.get_device(), x.dtype
    if index != _current_device():
        return _on_device(index, rms_norm_quantize_w8a8, x, residual, norm_weight, packed, eps, h_out, normed, out)
    ldr, r_addr = K, None
    if residual is not None:
        r_type, r_rows, ldr = _rows("residual", residual, K)
        if r_type != x_type or r_rows != M or residual.get_device() != index:
            raise ValueError(f"residual: expected {dt} {(M, K)} on {x.device}, got {residual.dtype} "
                             f"{tuple(residual.shape)} on {residual.device}")
        r_addr = residual.data_ptr()
    if norm_weight is not None and _unfit(norm_weight, dt, (K,), index):
        _refuse("norm_weight", norm_weight, dt, (K,), index)
    if inv_lambda is not None and _unfit(inv_lambda, _F32, (K,), index):
        _refuse("packed.inv_lambda", inv_lambda, _F32, (K,), index)
    if h_out is not None:
        if _unfit(h_out, dt, (M, K), index):
            _refuse("h_out", h_out, dt, (M, K), index)
    elif residual is not None:
        h_out = _empty_strided((M, K), (K, 1), dt)
    if normed is not None and _unfit(normed, dt, (M, K), index):
        _refuse("normed", normed, dt, (M, K), index)
    if out is None:
        out = _act(M, K)
    else:
        _check_out(out, M, K, index)
    _check(_lib.lib.svdq_rms_norm_quantize_w8a8(
        x_type, x.data_ptr(), ldx, r_addr, ldr, M, K, _addr(norm_weight), eps, _addr(inv_lambda), _addr(h_out),
        _addr(normed), out.x_codes.data_ptr(), out.x_scales.data_ptr(), _current_stream(index)),
        "svdq_rms_norm_quantize_w8a8")
    return (x if h_out is None else h_out), out


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
    if _unfit(x_codes, _I8, (M, K), index):
        _refuse("q.x_codes", x_codes, _I8, (M, K), index)
    if _unfit(x_scales, _F32, (M,), index):
        _refuse("q.x_scales", x_scales, _F32, (M,), index)
    if _unfit(w_codes, _I8, (N, K), index):
        _refuse("packed.w_codes", w_codes, _I8, (N, K), index)
    if _unfit(w_scales, _F32, (N,), index):
        _refuse("packed.w_scales", w_scales, _F32, (N,), index)
    if bias is not None and _unfit(bias, out_dtype, (N,), index):
        _refuse("packed.bias", bias, out_dtype, (N,), index)
    if y is not None and _unfit(y, out_dtype, (M, N), index):
        _refuse("y", y, out_dtype, (M, N), index)
    if index != _current_device():
        if index < 0:
            raise ValueError(f"expected CUDA tensors, got tensors on {x_codes.device}")
        return _on_device(index, gemm_w8a8, q, packed, y, out_dtype)
    if y is None:
        y = _empty_strided((M, N), (N, 1), out_dtype)
    _check(_lib.lib.svdq_gemm_w8a8(x_codes.data_ptr(), x_scales.data_ptr(), M, w_codes.data_ptr(),
                                   w_scales.data_ptr(), N, K, _addr(bias), y_type, y.data_ptr(),
                                   _current_stream(index)), "svdq_gemm_w8a8")
    return y


def w8a8_linear(x: torch.Tensor, packed: PackedWeightW8A8, out_dtype: torch.dtype | None = None,
                stream=None) -> torch.Tensor:
    """One forward of the W8A8 linear layer: two launches, no host sync.  y is in out_dtype, by default the
    bias's type or, without one, x's."""
    if out_dtype is None:
        out_dtype = packed.bias.dtype if packed.bias is not None else x.dtype
    return gemm_w8a8(quantize_act_w8a8(x, packed, stream=stream), packed, out_dtype=out_dtype, stream=stream)
