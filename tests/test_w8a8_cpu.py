"""W8A8 layer on the CPU: pins of its oracle, and the refusals of its entry
points, which come before any launch and so need no GPU."""
from fractions import Fraction

import numpy as np
import pytest
import torch

FAKE = 1 << 20      # an aligned non-null address that no refused call reads
BIG = 1 << 40       # another one, far from it


@pytest.fixture(scope="module")
def L():
    from bit_w4a4_quantized_token_b200 import build

    build.build()
    from bit_w4a4_quantized_token_b200 import _lib

    return _lib


# ------------------------------------------------------------------ oracle pins
def test_codes_are_the_nearest_multiples_of_the_scale(oracle_mod):
    """Brute force in rationals: every code is a nearest whole multiple of a / 127, up to the fp32 steps (a code
    may be the other neighbour only within 127 * 2^-22 of the midpoint)."""
    rng = np.random.default_rng(0)
    t = rng.standard_normal((6, 48)).astype(np.float32) * np.float32(3.7)
    codes, scales = oracle_mod.w8a8_quantize_rows(t)
    for m in range(t.shape[0]):
        a = max(abs(Fraction(float(v))) for v in t[m])
        assert abs(Fraction(float(scales[m])) - a / 127) <= a / 127 * Fraction(1, 2 ** 24)
        for v, c in zip(t[m], codes[m]):
            assert abs(Fraction(float(v)) * 127 / a - int(c)) <= Fraction(1, 2) + Fraction(127, 2 ** 22)
        assert np.abs(codes[m]).max() == 127


def test_codes_on_the_grid_are_exact_and_ties_go_to_even(oracle_mod):
    c = np.arange(-127, 128, dtype=np.float32)[None, :]
    codes, scales = oracle_mod.w8a8_quantize_rows(c * np.float32(0.25))
    assert np.array_equal(codes[0], c[0].astype(np.int8)) and scales[0] == np.float32(0.25)
    t = np.array([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5]], np.float32)
    assert oracle_mod.w8a8_quantize_rows(t)[0].tolist() == [[127, 0, 2, 2, 0, -2, -2, 126]]


def test_special_rows(oracle_mod):
    t = np.zeros((5, 16), np.float32)
    t[1, 3] = np.inf
    t[2, 4] = np.nan
    t[3, 5] = 2.0 ** -101
    t[4, 6] = -2.0 ** -100
    codes, scales = oracle_mod.w8a8_quantize_rows(t)
    assert scales[0] == 0 and np.isnan(scales[1]) and np.isnan(scales[2]) and scales[3] == 0 and scales[4] > 0
    assert not codes[:4].any() and codes[4, 6] == -127


def test_norm_factor_leaves_the_codes(oracle_mod):
    """Codes of h g and of h g / rms are the same numbers (up to fp32 ties), so the factor may sit in the scale."""
    rng = np.random.default_rng(1)
    h, t = oracle_mod.w8a8_norm_rows(rng.standard_normal((4, 64)), rng.standard_normal((4, 64)),
                                     rng.uniform(0.5, 2, 64), rng.uniform(0.25, 2, 64))
    r = oracle_mod.w8a8_rstd(h, 1e-6)
    codes, scales = oracle_mod.w8a8_quantize_rows(t)
    v = t.astype(np.float64) * r[:, None]
    unit = np.abs(v).max(axis=1, keepdims=True) / 127
    assert np.abs(v / unit - codes).max() <= 0.5 + 127 * 2.0 ** -22
    assert np.allclose(scales * r, unit[:, 0], rtol=2.0 ** -23)


# -------------------------------------------------------------------- refusals
def _status(L, fn, **kw):
    try:
        getattr(L, fn)(**kw)
        return 0
    except L.SvdqError as e:
        return e.status


GEMM = dict(x_codes=FAKE, x_scales=FAKE, M=64, w_codes=FAKE, w_scales=FAKE, N=256, K=256, bias=None, y_type=0, y=BIG,
            stream=0)
QUANT = dict(x_type=0, x=FAKE, ldx=256, M=64, K=256, inv_lambda=None, x_codes=BIG, x_scales=2 * BIG, stream=0)
PACK = dict(w_type=0, W=FAKE, N=256, K=256, lam=None, w_codes=BIG, w_scales=2 * BIG, inv_lambda=None, stream=0)
NORM = dict(x_type=0, x=FAKE, ldx=256, residual=2 * BIG, ldr=256, M=64, K=256, norm_weight=7 * BIG, eps=1e-6,
            inv_lambda=8 * BIG, h_out=3 * BIG, normed=4 * BIG, x_codes=5 * BIG, x_scales=6 * BIG, stream=0)


@pytest.mark.parametrize("fn,base,bad", [
    ("svdq_gemm_w8a8", GEMM, dict(x_codes=None)), ("svdq_gemm_w8a8", GEMM, dict(x_scales=None)),
    ("svdq_gemm_w8a8", GEMM, dict(w_codes=FAKE + 8)), ("svdq_gemm_w8a8", GEMM, dict(w_scales=FAKE + 4)),
    ("svdq_gemm_w8a8", GEMM, dict(bias=FAKE + 2)), ("svdq_gemm_w8a8", GEMM, dict(y=None)),
    ("svdq_gemm_w8a8", GEMM, dict(y_type=3)), ("svdq_gemm_w8a8", GEMM, dict(y_type=-1)),
    ("svdq_quantize_act_w8a8", QUANT, dict(x=None)), ("svdq_quantize_act_w8a8", QUANT, dict(x=FAKE + 2)),
    ("svdq_quantize_act_w8a8", QUANT, dict(x_type=7)), ("svdq_quantize_act_w8a8", QUANT, dict(x_codes=None)),
    ("svdq_quantize_act_w8a8", QUANT, dict(x_scales=2 * BIG + 4)),
    ("svdq_quantize_act_w8a8", QUANT, dict(inv_lambda=FAKE + 4)),
    ("svdq_quantize_act_w8a8", QUANT, dict(x_codes=FAKE + 64 * 512 - 16)),      # codes in x's last row
    ("svdq_pack_weight_w8a8", PACK, dict(W=None)), ("svdq_pack_weight_w8a8", PACK, dict(lam=FAKE)),
    ("svdq_pack_weight_w8a8", PACK, dict(w_scales=None)), ("svdq_pack_weight_w8a8", PACK, dict(w_type=3)),
    ("svdq_rms_norm_quantize_w8a8", NORM, dict(x=None)), ("svdq_rms_norm_quantize_w8a8", NORM, dict(eps=0.0)),
    ("svdq_rms_norm_quantize_w8a8", NORM, dict(eps=1.0)),
    ("svdq_rms_norm_quantize_w8a8", NORM, dict(eps=float("nan"))),
    ("svdq_rms_norm_quantize_w8a8", NORM, dict(x_codes=None)),
    ("svdq_rms_norm_quantize_w8a8", NORM, dict(x_scales=None)),
    ("svdq_rms_norm_quantize_w8a8", NORM, dict(x_codes=None, x_scales=None, normed=None)),
    ("svdq_rms_norm_quantize_w8a8", NORM, dict(norm_weight=FAKE + 2)),
    ("svdq_rms_norm_quantize_w8a8", NORM, dict(h_out=2 * BIG + 16)),            # not quite in place
    ("svdq_rms_norm_quantize_w8a8", NORM, dict(h_out=2 * BIG, ldr=264)),        # in place, other stride
    ("svdq_rms_norm_quantize_w8a8", NORM, dict(h_out=FAKE, ldx=512)),
    ("svdq_rms_norm_quantize_w8a8", NORM, dict(normed=FAKE)), ("svdq_rms_norm_quantize_w8a8", NORM, dict(normed=3 * BIG)),
    ("svdq_rms_norm_quantize_w8a8", NORM, dict(x_codes=2 * BIG)),
    ("svdq_rms_norm_quantize_w8a8", NORM, dict(x_codes=4 * BIG)),
    ("svdq_rms_norm_quantize_w8a8", NORM, dict(h_out=FAKE + 128, ldx=264, M=1)),   # h in x's row, shifted
    # scales, y or a weight's side in memory that the call reads or writes otherwise
    ("svdq_gemm_w8a8", GEMM, dict(y=FAKE)), ("svdq_gemm_w8a8", GEMM, dict(y=FAKE + 64 * 256 - 16)),
    ("svdq_gemm_w8a8", GEMM, dict(bias=BIG + 64 * 256 * 2 - 16)),
    ("svdq_quantize_act_w8a8", QUANT, dict(x_scales=FAKE)), ("svdq_quantize_act_w8a8", QUANT, dict(x_scales=BIG + 16)),
    ("svdq_quantize_act_w8a8", QUANT, dict(inv_lambda=BIG)),
    ("svdq_pack_weight_w8a8", PACK, dict(w_codes=FAKE)), ("svdq_pack_weight_w8a8", PACK, dict(w_scales=BIG)),
    ("svdq_pack_weight_w8a8", PACK, dict(lam=FAKE, inv_lambda=FAKE)),
    ("svdq_rms_norm_quantize_w8a8", NORM, dict(x_scales=4 * BIG)),
    ("svdq_rms_norm_quantize_w8a8", NORM, dict(x_scales=3 * BIG + 64)),
    ("svdq_rms_norm_quantize_w8a8", NORM, dict(norm_weight=3 * BIG)),
])
def test_invalid_arguments(L, fn, base, bad):
    assert _status(L, fn, **dict(base, **bad)) == L.SVDQ_ERR_INVALID_ARG


@pytest.mark.parametrize("fn,base,bad", [
    ("svdq_gemm_w8a8", GEMM, dict(M=0)), ("svdq_gemm_w8a8", GEMM, dict(M=1 << 31)),
    ("svdq_gemm_w8a8", GEMM, dict(N=0)), ("svdq_gemm_w8a8", GEMM, dict(N=260)),
    ("svdq_gemm_w8a8", GEMM, dict(K=0)), ("svdq_gemm_w8a8", GEMM, dict(K=24)),
    ("svdq_gemm_w8a8", GEMM, dict(K=1 << 17)), ("svdq_gemm_w8a8", GEMM, dict(M=(1 << 31) - 1, N=(1 << 31) - 8)),
    ("svdq_quantize_act_w8a8", QUANT, dict(M=(1 << 31) - 1, ldx=(1 << 31) - 8)),
    ("svdq_quantize_act_w8a8", QUANT, dict(M=0)), ("svdq_quantize_act_w8a8", QUANT, dict(K=8)),
    ("svdq_quantize_act_w8a8", QUANT, dict(ldx=255)), ("svdq_quantize_act_w8a8", QUANT, dict(ldx=260)),
    ("svdq_quantize_act_w8a8", QUANT, dict(ldx=0)), ("svdq_quantize_act_w8a8", QUANT, dict(x_type=2, ldx=258)),
    ("svdq_pack_weight_w8a8", PACK, dict(N=0)), ("svdq_pack_weight_w8a8", PACK, dict(K=(1 << 17))),
    ("svdq_rms_norm_quantize_w8a8", NORM, dict(M=0)), ("svdq_rms_norm_quantize_w8a8", NORM, dict(ldr=128)),
    ("svdq_rms_norm_quantize_w8a8", NORM, dict(ldx=1 << 31)), ("svdq_rms_norm_quantize_w8a8", NORM, dict(K=40)),
])
def test_unsupported_shapes(L, fn, base, bad):
    assert _status(L, fn, **dict(base, **bad)) == L.SVDQ_ERR_UNSUPPORTED_SHAPE


def test_valid_arguments_reach_the_device_check(L):
    """With another device's capability every valid call stops at the device check (nothing is launched)."""
    L.svdq_debug_override_capability(9, 0)
    try:
        for fn, base, kw in [("svdq_gemm_w8a8", GEMM, {}), ("svdq_gemm_w8a8", GEMM, dict(K=(1 << 17) - 16, N=8)),
                             ("svdq_gemm_w8a8", GEMM, dict(y_type=2, bias=FAKE)),
                             ("svdq_quantize_act_w8a8", QUANT, {}),
                             ("svdq_quantize_act_w8a8", QUANT, dict(ldx=264)),
                             ("svdq_quantize_act_w8a8", QUANT, dict(x_type=2, ldx=260)),
                             ("svdq_pack_weight_w8a8", PACK, {}),
                             ("svdq_pack_weight_w8a8", PACK, dict(lam=FAKE, inv_lambda=3 * BIG)),
                             ("svdq_rms_norm_quantize_w8a8", NORM, {}),
                             ("svdq_rms_norm_quantize_w8a8", NORM, dict(h_out=2 * BIG)),
                             ("svdq_rms_norm_quantize_w8a8", NORM, dict(h_out=FAKE)),
                             ("svdq_rms_norm_quantize_w8a8", NORM, dict(M=1, h_out=FAKE, ldx=512)),
                             ("svdq_rms_norm_quantize_w8a8", NORM, dict(residual=None, ldr=0, h_out=None)),
                             ("svdq_rms_norm_quantize_w8a8", NORM, dict(x_codes=None, x_scales=None))]:
            assert _status(L, fn, **dict(base, **kw)) == L.SVDQ_ERR_UNSUPPORTED_DEVICE, (fn, kw)
    finally:
        L.svdq_debug_override_capability(-1)


def test_layer_refuses_what_a_pointer_hides(L):
    """Types, shapes, strides and devices are checked in the torch-facing layer (no GPU is touched)."""
    from bit_w4a4_quantized_token_b200 import layer

    codes, scales = torch.zeros(8, 32, dtype=torch.int8), torch.zeros(8)
    packed = layer.PackedWeightW8A8(8, 32, codes, scales, None, None)
    for x in (torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(32), torch.zeros(4, 16)):
        with pytest.raises(ValueError, match="x:"):
            layer.quantize_act_w8a8(x, packed)        # not on a GPU, not a matrix, other width
        with pytest.raises(ValueError, match="x:"):
            layer.rms_norm_quantize_w8a8(x, None, None, packed)
    q = layer.QuantizedActW8A8(8, codes, scales)
    with pytest.raises(ValueError, match="out_dtype"):
        layer.gemm_w8a8(q, packed, out_dtype=torch.float64)
    with pytest.raises(ValueError, match="x_codes"):
        layer.gemm_w8a8(layer.QuantizedActW8A8(8, codes.float(), scales), packed)
    with pytest.raises(ValueError, match="x_codes"):
        layer.gemm_w8a8(layer.QuantizedActW8A8(8, torch.zeros(32, 8, dtype=torch.int8).t(), scales), packed)
    with pytest.raises(ValueError, match="w_scales"):
        layer.gemm_w8a8(q, layer.PackedWeightW8A8(8, 32, codes, scales.double(), None, None))
    with pytest.raises(ValueError, match="bias"):
        layer.gemm_w8a8(q, layer.PackedWeightW8A8(8, 32, codes, scales, None, torch.zeros(8)),
                        out_dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="y:"):
        layer.gemm_w8a8(q, packed, y=torch.zeros(8, 16))
    with pytest.raises(ValueError, match="W:"):
        layer.pack_weight_w8a8(torch.zeros(8, 32))


def test_stream_of_another_device_is_refused(L):
    """A stream belongs to one GPU: work for an operand elsewhere would run on that operand's current stream."""
    from types import SimpleNamespace

    from bit_w4a4_quantized_token_b200 import layer

    other = SimpleNamespace(device=torch.device("cuda", 1))
    codes, scales = torch.zeros(8, 32, dtype=torch.int8), torch.zeros(8)
    packed = layer.PackedWeightW8A8(8, 32, codes, scales, None, None)
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    for call in (lambda: layer.quantize_act_w8a8(x, packed, stream=other),
                 lambda: layer.rms_norm_quantize_w8a8(x, None, None, packed, stream=other),
                 lambda: layer.gemm_w8a8(layer.QuantizedActW8A8(8, codes, scales), packed, stream=other),
                 lambda: layer.w8a8_linear(x, packed, stream=other),
                 lambda: layer.pack_weight_w8a8(torch.zeros(8, 32), stream=other)):
        with pytest.raises(ValueError, match="stream:"):
            call()
