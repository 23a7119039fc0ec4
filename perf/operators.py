"""Cases of the 8-bit integer (W8A8) linear path: what is measured, and the
plain form of every operator.

Three operators, used one after another in a transformer block:

* ``norm_linear``: the block's input step and its first projection.  The
  branch output x is added to the residual stream, h = x + residual; h is
  RMS-normalised, smoothed (x 1/lambda) and quantised to 8-bit integers with
  one scale per token; the codes are multiplied with a weight held in 8-bit
  integers with one scale per output channel:
      h = x + residual
      t = h * (w_norm / lambda);   a[m] = max_k |t[m, k]|
      codes = round_half_even(t * (127 / a));   scale[m] = a / 127 / sqrt(mean(h^2) + eps)
      y[m, n] = scale[m] * w_scale[n] * sum_k codes[m, k] * w_codes[n, k] + bias[n]
  It returns the new residual stream and y.
* ``linear``: the same without the norm (the projections whose input is not a
  normalised one: attention output, second MLP matrix): t = x / lambda,
  scale = a / 127.
* ``gemm``: the product alone, on codes and scales that are in hand.

A row of zeros (padding of a batch) has codes and scale zero, so its y is the bias.
"""
import math

import torch

own = False

EPS = 1e-6
#: rows whose largest magnitude is below this are taken as zero: 127 / a stays finite
TINY = 2.0 ** -100

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def _case(name, op, M, K, N, x="bf16", y="bf16", smooth=False, bias=False):
    return {"name": name, "op": op, "M": M, "K": K, "N": N, "x": x, "y": y, "smooth": smooth, "bias": bias}


def listed():
    return [
        # One token through an attention output projection: weights from L2 or HBM, latency counts.
        _case("linear one token", "linear", 1, 4096, 4096),
        # A decode batch of odd size through a gated MLP's wide matrix, fp16 with bias.
        _case("linear odd batch", "linear", 37, 2080, 11008, x="f16", y="f16", bias=True),
        # The MLP input projection of an image transformer: 4096 image + 512 text tokens, smoothed, with bias.
        _case("linear image tokens", "linear", 4608, 4096, 12288, smooth=True, bias=True),
        # One token through norm and a fused query/key/value projection with grouped heads.
        _case("norm one token", "norm_linear", 1, 8192, 10240, smooth=True),
        # A short ragged prompt in a small model with odd widths, fp16.
        _case("norm odd sizes", "norm_linear", 777, 1552, 1000, x="f16", y="f16", smooth=True, bias=True),
        # A long prompt into a narrow latent: the norm's traffic is most of the work.
        _case("norm long prompt latent", "norm_linear", 16384, 8192, 512),
        # A residual stream kept in fp32 (deep models), bf16 projections.
        _case("norm fp32 stream", "norm_linear", 2048, 4096, 6144, x="f32", smooth=True),
        # The smallest layer that is run: launch latency.
        _case("gemm tiny", "gemm", 64, 256, 256),
        # A decode batch over a weight larger than the L2: HBM-bound.
        _case("gemm decode wide", "gemm", 16, 8192, 28672),
        # The MLP output projection of an image transformer, fp32 results (summed over branches by the caller).
        _case("gemm image tokens", "gemm", 4608, 12288, 4096, y="f32"),
        # A prompt with sizes that divide no tile.
        _case("gemm ragged", "gemm", 1000, 4112, 4104, y="f16", bias=True),
        # A large prefill: tensor-bound.
        _case("gemm large prefill", "gemm", 16384, 8192, 8192),
    ]


_MOST_FLOPS = 2.0 * 16384 * 8192 * 8192
_MOST_VALUES = 16384 * 8192 * 1.5


def draw(rng):
    def spread(lo, hi, step):
        v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
        return max(lo, min(hi, int(v / step + 0.5) * step))

    op = rng.choice(("linear", "norm_linear", "gemm"))
    M, K, N = spread(1, 18432, 1), spread(128, 16384, 16), spread(64, 28672, 8)
    while 2.0 * M * N * K > _MOST_FLOPS or M * max(N, K) > _MOST_VALUES:
        M = max(1, M // 2 + rng.randrange(2))
        if rng.random() < 0.5:
            N = max(64, N // 2 // 8 * 8)
    x = rng.choice(("bf16", "bf16", "f16", "f32")) if op != "gemm" else "bf16"
    y = rng.choice(("bf16", "bf16", "f16"))
    if op == "gemm" and rng.random() < 0.25:
        y = "f32"
    return {"op": op, "M": M, "K": K, "N": N, "x": x, "y": y, "smooth": op != "gemm" and rng.random() < 0.5,
            "bias": rng.random() < 0.5}


def prepare(case, seed):
    """Inputs from the seed: activations ~ N(0, 1) with 1 % outlier channels x 20,
    a residual stream of several times their size, weights ~ N(0, 1 / sqrt(K))
    quantised per output channel, a few all-zero (padding) rows in larger batches."""
    M, K, N = case["M"], case["K"], case["N"]
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    def uniform(n, lo, hi):
        return torch.rand(n, generator=g, device="cuda", dtype=torch.float32) * (hi - lo) + lo

    outlier = 1.0 + 19.0 * (uniform(K, 0.0, 1.0) < 0.01).float()
    # the weight: 8-bit codes and a scale per output channel, as a program keeps it
    w = normal(N, K)
    w_amax = w.abs().amax(1, keepdim=True)
    s = {"w_codes": torch.round(w.mul_(127.0 / w_amax)).to(torch.int8),
         "w_scales": (w_amax[:, 0] / (127.0 * math.sqrt(K))).contiguous()}
    del w
    dt, yt = _TYPES[case["x"]], _TYPES[case["y"]]
    s["bias"] = (0.1 * normal(N)).to(yt) if case["bias"] else None
    s["inv_lambda"] = 1.0 / uniform(K, 0.5, 4.0) if case["smooth"] else None
    x = normal(M, K).mul_(outlier)
    if M > 8:
        x[M - 1 - M // 16:] = 0.0
    if case["op"] == "gemm":
        amax = x.abs().amax(1, keepdim=True)
        s["x_codes"] = torch.round(x * torch.where(amax > 0, 127.0 / amax, 0.0)).to(torch.int8)
        s["x_scales"] = (amax[:, 0] / 127.0).contiguous()
    else:
        s["x"] = x.to(dt)
    if case["op"] == "norm_linear":
        r = normal(M, K).mul_(3.0)
        if M > 8:
            r[M - 1 - M // 16:] = 0.0
        s["residual"] = r.to(dt)
        s["norm_weight"] = uniform(K, 0.5, 2.0).to(dt)
    s["case"] = case
    return s


def _quantize_plain(t):
    """Codes (as fp32 whole numbers) and scales of the rows of t, fp32."""
    a = t.abs().amax(1, keepdim=True)
    some = a >= TINY
    codes = torch.round(t * torch.where(some, 127.0 / a, 0.0))
    return codes, torch.where(some, a / 127.0, 0.0)


def _run_plain(s):
    case = s["case"]
    h = None
    if case["op"] == "gemm":
        codes, scale = s["x_codes"].float(), s["x_scales"][:, None]
    elif case["op"] == "linear":
        t = s["x"].float()
        if case["smooth"]:
            t = t * s["inv_lambda"]
        codes, scale = _quantize_plain(t)
    else:
        h = s["x"].float() + s["residual"].float()
        gain = s["norm_weight"].float()
        if case["smooth"]:
            gain = gain * s["inv_lambda"]
        codes, scale = _quantize_plain(h * gain)
        scale = scale * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
        h = h.to(_TYPES[case["x"]])
    y = (codes @ s["w_codes"].float().t()) * scale * s["w_scales"]
    if case["bias"]:
        y = y + s["bias"].float()
    y = y.to(_TYPES[case["y"]])
    return y if h is None else (h, y)


def _run_own(s):
    from bit_w4a4_quantized_token_b200 import layer

    case = s["case"]
    N, K = s["w_codes"].shape
    packed = layer.PackedWeightW8A8(N, K, s["w_codes"], s["w_scales"], s["inv_lambda"], s["bias"])
    h = None
    if case["op"] == "gemm":
        q = layer.QuantizedActW8A8(case["M"], s["x_codes"], s["x_scales"])
    elif case["op"] == "linear":
        q = layer.quantize_act_w8a8(s["x"], packed)
    else:
        h, q = layer.rms_norm_quantize_w8a8(s["x"], s["residual"], s["norm_weight"], packed, eps=EPS)
    y = layer.gemm_w8a8(q, packed, out_dtype=_TYPES[case["y"]])
    return y if h is None else (h, y)


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    M, K, N = case["M"], case["K"], case["N"]
    xb = _BYTES[case["x"]]
    moved = N * K + 4 * N + M * N * _BYTES[case["y"]]
    moved += N * _BYTES[case["y"]] if case["bias"] else 0
    moved += 4 * K if case["smooth"] else 0
    if case["op"] == "gemm":
        moved += M * K + 4 * M
    elif case["op"] == "linear":
        moved += M * K * xb
    else:
        moved += 3 * M * K * xb + K * xb
    return {"bytes": moved, "flops": 2 * M * N * K}


def exact(case, seed):
    """The definition in 64 bits, a block of rows at a time."""
    s = prepare(case, seed)
    f64 = torch.float64
    weight = s["w_codes"].to(f64) * s["w_scales"].to(f64)[:, None]      # [N, K], dequantised
    lam_inv = s["inv_lambda"].to(f64) if case["smooth"] else torch.ones(case["K"], dtype=f64, device="cuda")
    step = max(1, (1 << 26) // case["K"])
    hs, ys = [], []
    for m in range(0, case["M"], step):
        rows = slice(m, m + step)
        if case["op"] == "gemm":
            act = s["x_codes"][rows].to(f64) * s["x_scales"][rows].to(f64)[:, None]
        else:
            v = s["x"][rows].to(f64)
            if case["op"] == "norm_linear":
                v = v + s["residual"][rows].to(f64)
                hs.append(v)
                v = v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS) * s["norm_weight"].to(f64)
            v = v * lam_inv
            unit = v.abs().max(dim=1, keepdim=True).values / 127.0
            act = torch.where(unit > 0, torch.round(v / unit) * unit, 0.0)
        out = torch.matmul(act, weight.t())
        ys.append(out + s["bias"].to(f64) if case["bias"] else out)
    y = torch.cat(ys)
    return (torch.cat(hs), y) if hs else y
