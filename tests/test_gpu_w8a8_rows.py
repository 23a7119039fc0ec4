"""The row kernels of the W8A8 layer where a block takes many rows, against the
CPU oracle.

Rows of 16 KB and more (x, and the residual where there is one) stream through
a ring in shared memory.  Its later passes, in which a row lands where an
earlier one was, need more rows per block than the ring has places: the cases
give every block several passes on 148 SMs, on both sides of the switch from
two blocks per SM to one (16 rows per SM), with every row another.  Tolerances
as in test_gpu_w8a8.py: codes, plain scales and h bit for bit, the norm's
scales within the roundings counted there.
"""
import numpy as np
import pytest
import torch

from .test_gpu_w8a8 import BF16, EPS, F16, F32, U, _cuda, chain_length, draw, f32, packed_for, uniform  # noqa: F401

pytestmark = pytest.mark.gpu


def check_norm(O, q, x, r, w, il):
    """Codes bit for bit and scales within their roundings; returns fp32 h."""
    K = x.shape[1]
    h32, t = O.w8a8_norm_rows(f32(x), None if r is None else f32(r), None if w is None else f32(w),
                              None if il is None else f32(il))
    codes, plain = O.w8a8_quantize_rows(t)
    assert np.array_equal(q.x_codes.cpu().numpy(), codes)
    want = plain.astype(np.float64) * O.w8a8_rstd(h32, EPS)
    row = (4 + (chain_length(K) + 1) / 2) * U
    assert np.all(np.abs(q.x_scales.cpu().numpy() - want) <= row * want)
    return h32


@pytest.mark.parametrize("dtype,M,K,smooth", [
    (BF16, 2300, 8192, True), (BF16, 4999, 8192, False),      # places: 6 for each of two blocks
    (BF16, 2300, 16384, False), (F16, 2500, 16384, True),     # 3 for each of two blocks, 6 for one
    (F32, 3001, 4096, True), (F32, 2400, 8208, False)])       # 3 for each of four, 6 for one
def test_quantize_many_rows_per_block(oracle_mod, dtype, M, K, smooth):
    from bit_w4a4_quantized_token_b200 import layer

    x = draw(M, K, dtype, seed=M)
    il = 1.0 / uniform(K, 0.5, 4.0, seed=K) if smooth else None
    q = layer.quantize_act_w8a8(x.cuda(), packed_for(K, None if il is None else il.cuda()))
    codes, scales = oracle_mod.w8a8_quantize_rows(f32(x) * il.numpy() if smooth else f32(x))
    assert np.array_equal(q.x_codes.cpu().numpy(), codes) and np.array_equal(q.x_scales.cpu().numpy(), scales)


@pytest.mark.parametrize("dtype,M,K,res,weight,smooth", [
    (BF16, 2300, 8192, True, True, False), (BF16, 2400, 8192, True, False, True),   # two blocks per SM, one
    (F16, 4999, 4096, True, True, True), (F16, 3001, 8192, False, True, False),
    (F32, 2300, 4112, True, True, True), (F32, 2400, 4112, True, True, False), (BF16, 1500, 16400, True, True, True)])
def test_norm_many_rows_per_block(oracle_mod, dtype, M, K, res, weight, smooth):
    from bit_w4a4_quantized_token_b200 import layer

    x, r = draw(M, K, dtype, seed=M), draw(M, K, dtype, seed=M + 1, scale=2.0) if res else None
    w = uniform(K, 0.5, 2.0, seed=2, dtype=dtype) if weight else None
    il = 1.0 / uniform(K, 0.5, 4.0, seed=4) if smooth else None
    dev = lambda t: None if t is None else t.cuda()   # noqa: E731
    h, q = layer.rms_norm_quantize_w8a8(x.cuda(), dev(r), dev(w), packed_for(K, dev(il)), eps=EPS)
    h32 = check_norm(oracle_mod, q, x, r, w, il)
    assert torch.equal(h.cpu(), torch.from_numpy(h32).to(dtype))


@pytest.mark.parametrize("where", ["residual", "x"])
@pytest.mark.parametrize("dtype,M,K", [(BF16, 2300, 8192), (BF16, 2400, 8192), (F32, 1800, 4112)])
def test_norm_in_place_many_rows_per_block(oracle_mod, where, dtype, M, K):
    """h written over x or the residual while later rows of both are being fetched."""
    from bit_w4a4_quantized_token_b200 import layer

    x, r, w = draw(M, K, dtype, 1), draw(M, K, dtype, 2, scale=2.0), uniform(K, 0.5, 2.0, 3, dtype)
    xd, rd = x.cuda(), r.cuda()
    target, other, kept = (rd, xd, x) if where == "residual" else (xd, rd, r)
    h, q = layer.rms_norm_quantize_w8a8(xd, rd, w.cuda(), packed_for(K), eps=EPS, h_out=target)
    h32 = check_norm(oracle_mod, q, x, r, w, None)
    assert h.data_ptr() == target.data_ptr() and torch.equal(h.cpu(), torch.from_numpy(h32).to(dtype))
    assert torch.equal(other.cpu(), kept)


@pytest.mark.parametrize("dtype,M,K", [(BF16, 2000, 272), (BF16, 2400, 8192), (F32, 1500, 4112), (BF16, 700, 32768)])
def test_norm_special_rows_among_many(oracle_mod, dtype, M, K):
    """Zero rows, infinities, NaN and sums of squares that overflow, in each kernel and in late rows of a block: codes
    0 and scale NaN (0 for a zero row) there, every other row as it would be."""
    from bit_w4a4_quantized_token_b200 import layer

    x, r = draw(M, K, dtype, 5), draw(M, K, dtype, 6)
    rows = {M // 2: "zero", M // 2 + 1: "nan", M - 300: "inf", M - 200: "-inf", M - 100: "big", M - 1: "nan"}
    for m, kind in rows.items():
        if kind == "zero":
            x[m], r[m] = 0.0, 0.0
        elif kind == "inf":
            r[m, K - 1] = float("inf")
        elif kind == "big":
            x[m, K // 2] = 1e30                       # finite, its square is not
        else:
            x[m, m % K] = float(kind)
    w, packed = uniform(K, 0.5, 2.0, 7, dtype), packed_for(K)
    _, q = layer.rms_norm_quantize_w8a8(x.cuda(), r.cuda(), w.cuda(), packed, eps=EPS)
    s = q.x_scales.cpu()
    assert not q.x_codes[list(rows)].any()
    assert s[M // 2] == 0 and torch.isnan(s[[m for m, kind in rows.items() if kind != "zero"]]).all()
    rest = [m for m in range(M) if m not in rows]
    q.x_codes, q.x_scales = q.x_codes[rest], q.x_scales[rest]
    check_norm(oracle_mod, q, x[rest], r[rest], w, None)


@pytest.mark.parametrize("dtype,M,K", [(BF16, 300, 272), (BF16, 700, 8192), (F32, 40, 512), (F32, 700, 4112),
                                       (BF16, 40, 32768)])
def test_normed_of_rows_without_a_finite_sum(dtype, M, K):
    """A NaN, an infinity or finite values whose squares overflow: the whole normalised row is NaN (never zeros), and
    no other row changes."""
    from bit_w4a4_quantized_token_b200 import layer

    x, r = draw(M, K, dtype, 8), draw(M, K, dtype, 9)
    x[3, 5], x[M - 2, K - 1], r[M // 2, 0] = float("nan"), 1e30, float("-inf")
    bad = [3, M // 2, M - 2]
    rest = [m for m in range(M) if m not in bad]
    w, packed = uniform(K, 0.5, 2.0, 7, dtype).cuda(), packed_for(K)
    normed, alone = (torch.empty(n, K, dtype=dtype, device="cuda") for n in (M, M - 3))
    _, q = layer.rms_norm_quantize_w8a8(x.cuda(), r.cuda(), w, packed, normed=normed)
    layer.rms_norm_quantize_w8a8(x[rest].cuda(), r[rest].cuda(), w, packed, normed=alone)
    assert bool(torch.isnan(q.x_scales[bad]).all()) and bool(torch.isnan(normed[bad]).all())
    assert bool(torch.isfinite(alone).all()) and torch.equal(normed[rest], alone)
