"""The 8-bit integer (W8A8) layer against the CPU oracle: the quantizer, the
norm in front of it, the GEMM, and a run of them together.

Tolerances, in the order of the roundings they count (u = 2^-24, the largest
relative error of one fp32 rounding; half = finfo(type).eps / 2, of one
rounding to the output's type):
  * codes and the plain scales: bit-exact (the definition is in fp32 steps);
  * the norm's scale fl(fl(a / 127) rstd): one rounding each for a / 127, the
    product, the division by K, the addition of eps and the square root's
    reciprocal, and half the relative error of the sum of squares, whose terms
    are positive: at most (number of additions in a row + 1) u;
  * h: one rounding (bit-exact);  normed = fl(fl(h rstd) w): the row factor's
    error, two roundings, one rounding to the output's type;
  * y = round(fl(fl(float(sum) sx) sw + b)): the sum is exact; u for its
    conversion and u for the product with sx on the term sum sx sw, u for the
    fused multiply-add on y, half a step of the output's type on y, and half
    of fp16's smallest step where y is subnormal there.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [BF16, F16, F32]
EPS = 1e-6


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from bit_w4a4_quantized_token_b200 import _lib

    yield
    st, site = _lib.svdq_device_status(clear=True)
    assert st == 0, f"device status {st} (site {site})"


def half(dtype):
    return torch.finfo(dtype).eps / 2


def draw(M, K, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * scale
    x[:, torch.randperm(K, generator=g)[:max(1, K // 100)]] *= 20.0
    return x.to(dtype)


def uniform(n, lo, hi, seed, dtype=F32):
    return (torch.rand(n, generator=torch.Generator().manual_seed(seed)) * (hi - lo) + lo).to(dtype)


def f32(t):
    return t.float().cpu().numpy()


def packed_for(K, inv_lambda=None):
    """A weight of eight channels: what the quantizers read of it is its K and 1 / lambda."""
    from bit_w4a4_quantized_token_b200 import layer

    return layer.PackedWeightW8A8(8, K, torch.zeros(8, K, dtype=torch.int8, device="cuda"),
                                  torch.zeros(8, device="cuda"), inv_lambda, None)


def same_scales(got, want):
    got = got.cpu().numpy()
    return np.array_equal(got, want, equal_nan=True)


# ------------------------------------------------------------------- quantizer
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K,smooth", [(1, 16, False), (3, 48, True), (37, 2048, True), (5, 2064, False),
                                        (9, 8192, True), (2, 8208, False), (3, 16384, True), (2, 16400, True),
                                        (2, 65552, False), (1, 131056, True), (1500, 272, True)])
def test_quantize(oracle_mod, dtype, M, K, smooth):
    """Every block shape of the quantizer (rows in registers with 1, 2 and 4 vectors a thread, wide rows)."""
    from bit_w4a4_quantized_token_b200 import layer

    x = draw(M, K, dtype, seed=M + K)
    il = 1.0 / uniform(K, 0.5, 4.0, seed=K) if smooth else None
    q = layer.quantize_act_w8a8(x.cuda(), packed_for(K, None if il is None else il.cuda()))
    t = f32(x) * il.numpy() if smooth else f32(x)
    codes, scales = oracle_mod.w8a8_quantize_rows(t)
    assert np.array_equal(q.x_codes.cpu().numpy(), codes)
    assert same_scales(q.x_scales, scales)


@pytest.mark.parametrize("K", [2048, 4096, 32768])
def test_quantize_near_midpoints(oracle_mod, K):
    """Values within a few fp32 steps of half a unit: the product is rounded before the code is (the two roundings
    in one give other codes here)."""
    from bit_w4a4_quantized_token_b200 import layer

    rows = []
    for a in (1.0, 3.3, 97.1, 0.0123):
        inv = np.float32(127) / np.float32(a)
        mid = (np.arange(K) % 253 - 126.0) + 0.5
        t = (mid / np.float64(inv)).astype(np.float32)
        t = (t.view(np.int32) + (np.arange(K) // 253 % 5 - 2).astype(np.int32)).view(np.float32)
        t[0] = a
        rows.append(t)
    t = np.stack(rows)
    codes, scales = oracle_mod.w8a8_quantize_rows(t)
    inv = np.float32(127) / np.abs(t).max(1, keepdims=True)
    assert (np.rint(t.astype(np.float64) * inv) != codes).any()
    q = layer.quantize_act_w8a8(torch.from_numpy(t).cuda(), packed_for(K))
    assert np.array_equal(q.x_codes.cpu().numpy(), codes) and same_scales(q.x_scales, scales)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=str)
@pytest.mark.parametrize("K", [64, 4096, 32768])
def test_quantize_special_rows(oracle_mod, dtype, K):
    """Zero rows, values at the border of what counts as zero, ties, infinities and NaN: each alone in its row."""
    from bit_w4a4_quantized_token_b200 import layer

    x = draw(14, K, dtype, seed=K)
    x[0] = 0.0
    x[1] = 0.0
    x[1, K // 2] = 2.0 ** -101
    x[2] = 0.0
    x[2, K - 1] = -(2.0 ** -100)
    x[3, 5] = float("inf")
    x[4, K - 1] = float("-inf")
    x[5, 0] = float("nan")
    x[6, 7], x[6, 8] = float("nan"), float("inf")
    x[7] = 0.0
    x[7, :10] = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5, -127.0, 63.5])
    x[8] = -0.0
    x[9] = torch.finfo(dtype).max
    x[10] = -3.0
    x[11] = 0.0
    x[11, 3] = 1.0
    x[12] = torch.finfo(dtype).tiny
    q = layer.quantize_act_w8a8(x.cuda(), packed_for(K))
    codes, scales = oracle_mod.w8a8_quantize_rows(f32(x))
    assert np.array_equal(q.x_codes.cpu().numpy(), codes)
    assert same_scales(q.x_scales, scales)


def test_quantize_strided_rows_and_guards(oracle_mod):
    """x a column slice of a wider tensor; what lies behind the outputs stays as it was."""
    from bit_w4a4_quantized_token_b200 import layer

    wide = draw(19, 512, BF16, seed=3).cuda()
    x = wide[:, 64:64 + 272]
    store = torch.full((21 * 272,), 77, dtype=torch.int8, device="cuda")
    sstore = torch.full((32,), -5.0, device="cuda")
    out = layer.QuantizedActW8A8(19, store[:19 * 272].view(19, 272), sstore[:19])
    layer.quantize_act_w8a8(x, packed_for(272), out=out)
    codes, scales = oracle_mod.w8a8_quantize_rows(f32(x))
    assert np.array_equal(out.x_codes.cpu().numpy(), codes) and same_scales(out.x_scales, scales)
    assert bool((store[19 * 272:] == 77).all()) and bool((sstore[19:] == -5.0).all())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("N,K,smooth", [(8, 16, False), (72, 528, True), (130, 4096, True)])
def test_pack_weight(oracle_mod, dtype, N, K, smooth):
    from bit_w4a4_quantized_token_b200 import layer

    w = draw(N, K, dtype, seed=N)
    lam = uniform(K, 0.5, 4.0, seed=1) if smooth else None
    p = layer.pack_weight_w8a8(w.cuda(), None if lam is None else lam.cuda())
    codes, scales = oracle_mod.w8a8_quantize_rows(f32(w) * lam.numpy() if smooth else f32(w))
    assert np.array_equal(p.w_codes.cpu().numpy(), codes) and same_scales(p.w_scales, scales)
    if smooth:
        assert np.array_equal(p.inv_lambda.cpu().numpy(), np.float32(1) / lam.numpy())
    else:
        assert p.inv_lambda is None


# ------------------------------------------------------------------------ norm
def chain_length(K):
    """An upper bound of the additions in a row of any kernel's sum of squares: a thread's own, two warp trees."""
    return (32 if K <= 16384 else -(-K // 8192) * 8) + 10


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("M,K,res,weight,smooth", [
    (1, 16, True, True, True), (3, 48, False, True, False), (37, 2048, True, True, True),
    (5, 2064, True, False, True), (9, 8192, True, True, True), (4, 8208, True, True, False),
    (3, 16384, True, True, True), (2, 16400, True, True, True), (1, 131056, True, True, True),
    (6, 4096, False, False, False), (1500, 272, True, True, True)])
def test_norm(oracle_mod, dtype, M, K, res, weight, smooth):
    from bit_w4a4_quantized_token_b200 import layer

    x, r = draw(M, K, dtype, seed=M + K), draw(M, K, dtype, seed=M + K + 1, scale=2.0) if res else None
    w = uniform(K, 0.5, 2.0, seed=2, dtype=dtype) if weight else None
    il = 1.0 / uniform(K, 0.5, 4.0, seed=4) if smooth else None
    dev = lambda t: None if t is None else t.cuda()   # noqa: E731
    normed = torch.empty(M, K, dtype=dtype, device="cuda")
    h, q = layer.rms_norm_quantize_w8a8(x.cuda(), dev(r), dev(w), packed_for(K, dev(il)), eps=EPS, normed=normed)
    h32, t = oracle_mod.w8a8_norm_rows(f32(x), None if r is None else f32(r), None if w is None else f32(w),
                                       None if il is None else il.numpy())
    assert torch.equal(h.cpu(), torch.from_numpy(h32).to(dtype))
    codes, plain = oracle_mod.w8a8_quantize_rows(t)
    assert np.array_equal(q.x_codes.cpu().numpy(), codes)
    rstd = oracle_mod.w8a8_rstd(h32, EPS)
    row = (3 + (chain_length(K) + 1) / 2) * U         # rstd: sum of squares, / K, + eps (halved with it), the root
    want = plain.astype(np.float64) * rstd
    assert np.all(np.abs(q.x_scales.cpu().numpy() - want) <= (row + U) * want)
    n = h32.astype(np.float64) * rstd[:, None] * (1.0 if w is None else w.double().numpy())
    tol = (row + 2 * U + half(dtype) * (1 + 1e-3)) * np.abs(n) + torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    assert np.all(np.abs(normed.double().cpu().numpy() - n) <= tol)


@pytest.mark.parametrize("where", ["residual", "x"])
@pytest.mark.parametrize("K", [272, 8192, 24576])
def test_norm_in_place(oracle_mod, where, K):
    """The residual stream updated in place equals a separate output."""
    from bit_w4a4_quantized_token_b200 import layer

    x, r, w = draw(700, K, BF16, 1).cuda(), draw(700, K, BF16, 2).cuda(), uniform(K, 0.5, 2.0, 3, BF16).cuda()
    h, q = layer.rms_norm_quantize_w8a8(x, r, w, packed_for(K))
    target = r if where == "residual" else x
    h2, q2 = layer.rms_norm_quantize_w8a8(x, r, w, packed_for(K), h_out=target)
    assert h2.data_ptr() == target.data_ptr()
    assert torch.equal(h, h2) and torch.equal(q.x_codes, q2.x_codes) and torch.equal(q.x_scales, q2.x_scales)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_norm_without_residual_copies_the_stream(dtype):
    """h_out given and no residual: h_out is x; with neither, h is x itself; x as its own h_out."""
    from bit_w4a4_quantized_token_b200 import layer

    x = draw(33, 1040, dtype, 1).cuda()
    kept, buf, packed = x.clone(), torch.empty_like(x), packed_for(1040)
    h1, q1 = layer.rms_norm_quantize_w8a8(x, None, None, packed)
    h2, q2 = layer.rms_norm_quantize_w8a8(x, None, None, packed, h_out=buf)
    h3, q3 = layer.rms_norm_quantize_w8a8(x, None, None, packed, h_out=x)
    assert h1 is x and h2 is buf and h3 is x
    for h, q in ((h1, q1), (h2, q2), (h3, q3)):
        assert torch.equal(h, kept) and torch.equal(q.x_codes, q1.x_codes) and torch.equal(q.x_scales, q1.x_scales)


def test_norm_special_rows(oracle_mod):
    """A zero row, infinities and NaN, a sum of squares that overflows: no other row changes."""
    from bit_w4a4_quantized_token_b200 import layer

    K = 512
    x, r = draw(9, K, F32, 5), draw(9, K, F32, 6)
    x[1], r[1] = 0.0, 0.0
    x[3, 7] = float("nan")
    r[4, 8] = float("inf")
    x[6, 0] = 1e30                                     # finite, its square is not
    packed = packed_for(K)
    _, q = layer.rms_norm_quantize_w8a8(x.cuda(), r.cuda(), None, packed, eps=EPS)
    s, c = q.x_scales.cpu(), q.x_codes.cpu()
    assert s[1] == 0 and not c[1].any()
    assert torch.isnan(s[[3, 4, 6]]).all() and not c[[3, 4, 6]].any()
    rows = [0, 2, 5, 7, 8]
    _, q2 = layer.rms_norm_quantize_w8a8(x[rows].contiguous().cuda(), r[rows].contiguous().cuda(), None, packed, eps=EPS)
    assert torch.equal(c[rows], q2.x_codes.cpu()) and torch.equal(s[rows], q2.x_scales.cpu())


def test_norm_strides_and_normed_only():
    """Row strides of x and of the residual; normed without codes is the same normed."""
    from bit_w4a4_quantized_token_b200 import _lib, layer

    K, M = 400, 21
    xw, rw = draw(M, 640, F16, 7).cuda(), draw(M, 1000, F16, 8).cuda()
    x, r, w = xw[:, 8:8 + K], rw[:, 400:400 + K], uniform(K, 0.5, 2.0, 9, F16).cuda()
    n1, n2, n3 = (torch.empty(M, K, dtype=F16, device="cuda") for _ in range(3))
    h1, q1 = layer.rms_norm_quantize_w8a8(x, r, w, packed_for(K), normed=n1)
    h2, q2 = layer.rms_norm_quantize_w8a8(x.contiguous(), r.contiguous(), w, packed_for(K), normed=n2)
    assert torch.equal(h1, h2) and torch.equal(n1, n2)
    assert torch.equal(q1.x_codes, q2.x_codes) and torch.equal(q1.x_scales, q2.x_scales)
    _lib.svdq_rms_norm_quantize_w8a8(_lib.SVDQ_F16, x, 640, r, 1000, M, K, w, 1e-6, None, None, n3, None, None)
    assert torch.equal(n1, n3)


# ------------------------------------------------------------------------ GEMM
def codes_of(M, K, seed, lo=-127, hi=127):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, hi + 1, (M, K), generator=g, dtype=torch.int8)


def check_gemm(xc, xs, wc, ws, bias, y):
    acc = xc.double().cuda() @ wc.double().cuda().t()                    # exact: whole numbers below 2^53
    term = acc * xs.double().cuda()[:, None] * ws.double().cuda()
    want = term if bias is None else term + bias.double().cuda()
    tiny = torch.finfo(y.dtype).tiny * torch.finfo(y.dtype).eps / 2
    tol = 2.01 * U * term.abs() + 1.01 * U * want.abs() + half(y.dtype) * (1 + 1e-4) * want.abs() + tiny
    err = (y.double() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("out", TYPES, ids=str)
@pytest.mark.parametrize("M,N,K", [
    (1, 8, 16), (1, 128, 128), (1, 4096, 4096), (16, 264, 1024), (17, 1000, 80), (32, 136, 2064), (33, 512, 4096),
    (64, 256, 256), (65, 392, 1552), (128, 1024, 8192), (129, 128, 272), (300, 2056, 640), (777, 1000, 1552),
    (1000, 2504, 1040), (256, 12288, 128), (2500, 1288, 400), (5, 40, 131056)])
def test_gemm(out, M, N, K):
    """Every token tile of the narrow kernel, with and without a split of K, and the pair kernel; ragged sizes."""
    from bit_w4a4_quantized_token_b200 import layer

    xc, wc = codes_of(M, K, 1), codes_of(N, K, 2)
    xs, ws = uniform(M, 1e-3, 2e-2, 3), uniform(N, 1e-5, 1e-4, 4)
    bias = uniform(N, -1.0, 1.0, 5, out) if (M + N) % 3 else None
    packed = layer.PackedWeightW8A8(N, K, wc.cuda(), ws.cuda(), None, None if bias is None else bias.cuda())
    y = layer.gemm_w8a8(layer.QuantizedActW8A8(M, xc.cuda(), xs.cuda()), packed, out_dtype=out)
    check_gemm(xc, xs, wc, ws, bias, y)


@pytest.mark.parametrize("out", TYPES, ids=str)
@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (300, 520, 144), (513, 2312, 4112), (2100, 600, 1040), (64, 256, 20000)])
def test_both_kernels_give_the_same_bits(out, M, N, K):
    from bit_w4a4_quantized_token_b200 import _lib, layer

    xc, wc = codes_of(M, K, 1), codes_of(N, K, 2)
    xs, ws, bias = uniform(M, 1e-3, 2e-2, 3), uniform(N, 1e-5, 1e-4, 4), uniform(N, -1.0, 1.0, 5, out)
    packed = layer.PackedWeightW8A8(N, K, wc.cuda(), ws.cuda(), None, bias.cuda())
    q = layer.QuantizedActW8A8(M, xc.cuda(), xs.cuda())
    ys = []
    for mode in (1, 2, 0):
        _lib.svdq_debug_force_gemm_tiles(mode)
        try:
            ys.append(layer.gemm_w8a8(q, packed, out_dtype=out))
        finally:
            _lib.svdq_debug_force_gemm_tiles(0)
    check_gemm(xc, xs, wc, ws, bias, ys[0])
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


@pytest.mark.parametrize("mode", [1, 2])
def test_largest_sum_does_not_overflow(mode):
    """K at its limit with every code -128: the sum is 131056 * 2^14 < 2^31."""
    from bit_w4a4_quantized_token_b200 import _lib, layer

    M, N, K = 40, 136, (1 << 17) - 16
    xc = torch.full((M, K), -128, dtype=torch.int8)
    wc = torch.full((N, K), -128, dtype=torch.int8)
    one = torch.ones(M), torch.ones(N)
    _lib.svdq_debug_force_gemm_tiles(mode)
    try:
        y = layer.gemm_w8a8(layer.QuantizedActW8A8(M, xc.cuda(), one[0].cuda()),
                            layer.PackedWeightW8A8(N, K, wc.cuda(), one[1].cuda(), None, None), out_dtype=F32)
    finally:
        _lib.svdq_debug_force_gemm_tiles(0)
    assert bool((y == np.float32(131056 * 16384)).all())


@pytest.mark.parametrize("M,N,mode", [(20, 200, 1), (300, 328, 1), (300, 328, 2)])
def test_gemm_writes_its_rows_only_and_nan_rows_stay_alone(M, N, mode):
    from bit_w4a4_quantized_token_b200 import _lib, layer

    K = 336
    xc, wc = codes_of(M, K, 1).cuda(), codes_of(N, K, 2).cuda()
    xs, ws = uniform(M, 1e-3, 2e-2, 3), uniform(N, 1e-5, 1e-4, 4).cuda()
    xs[3], xs[7] = float("nan"), 0.0
    bias = uniform(N, -1.0, 1.0, 5, BF16).cuda()
    store = torch.full((M * N + 4096,), 7.0, dtype=BF16, device="cuda")
    y = store[2048:2048 + M * N].view(M, N)
    _lib.svdq_debug_force_gemm_tiles(mode)
    try:
        layer.gemm_w8a8(layer.QuantizedActW8A8(M, xc, xs.cuda()), layer.PackedWeightW8A8(N, K, wc, ws, None, bias), y=y)
    finally:
        _lib.svdq_debug_force_gemm_tiles(0)
    assert bool((store[:2048] == 7.0).all()) and bool((store[2048 + M * N:] == 7.0).all())
    assert bool(torch.isnan(y[3]).all()) and bool(torch.equal(y[7], bias))
    rest = [m for m in range(M) if m != 3]
    check_gemm(xc[rest].cpu(), xs[rest], wc.cpu(), ws.cpu(), bias.cpu(), y[rest])


# ------------------------------------------------------- a run of them together
def test_linear_types_by_default(oracle_mod):
    """Without a bias y has x's type, with one the bias's, unless it is said; fp32 in and out."""
    from bit_w4a4_quantized_token_b200 import layer

    W = draw(264, 528, F32, 3)
    packed = layer.pack_weight_w8a8(W.cuda())
    with_bias = layer.pack_weight_w8a8(W.cuda(), None, uniform(264, -1.0, 1.0, 1, F16).cuda())
    for dtype in TYPES:
        x = draw(50, 528, dtype, 2).cuda()
        y = layer.w8a8_linear(x, packed)
        assert y.dtype == dtype and layer.w8a8_linear(x, with_bias).dtype == F16
        assert layer.w8a8_linear(x, packed, out_dtype=BF16).dtype == BF16
        codes, scales = oracle_mod.w8a8_quantize_rows(f32(x))
        check_gemm(torch.from_numpy(codes), torch.from_numpy(scales), packed.w_codes.cpu(), packed.w_scales.cpu(), None, y)


def layer_inputs(M, K, N, dtype, smooth):
    x, r = draw(M, K, dtype, 11).cuda(), draw(M, K, dtype, 12, 3.0).cuda()
    W = (torch.randn(N, K, generator=torch.Generator().manual_seed(13)) / K ** 0.5).to(dtype).cuda()
    lam = uniform(K, 0.5, 4.0, 14).cuda() if smooth else None
    return x, r, W, lam, uniform(N, -0.1, 0.1, 15, dtype).cuda(), uniform(K, 0.5, 2.0, 16, dtype).cuda()


@pytest.mark.parametrize("M,K,N,dtype,smooth", [(1, 2048, 1024, BF16, True), (50, 528, 392, F16, False),
                                                (700, 1040, 2056, BF16, True)])
def test_layer_run(oracle_mod, M, K, N, dtype, smooth):
    """Norm and projection, and the plain linear, as a block calls them: against the oracle's own codes, and near
    the unquantised product (8-bit rounding noise: half a unit of each operand's scale per term, in the rms)."""
    from bit_w4a4_quantized_token_b200 import layer

    x, r, W, lam, bias, w = layer_inputs(M, K, N, dtype, smooth)
    packed = layer.pack_weight_w8a8(W, lam, bias)
    h, q = layer.rms_norm_quantize_w8a8(x, r, w, packed, eps=EPS)
    y = layer.gemm_w8a8(q, packed)
    z = layer.w8a8_linear(h, packed)
    assert y.dtype == z.dtype == dtype
    O = oracle_mod
    il = None if lam is None else np.float32(1) / lam.cpu().numpy()
    wc, ws = O.w8a8_quantize_rows(f32(W) if lam is None else f32(W) * lam.cpu().numpy())
    h32, t = O.w8a8_norm_rows(f32(x), f32(r), f32(w), il)
    xc, xs = O.w8a8_quantize_rows(t)
    assert torch.equal(h.cpu(), torch.from_numpy(h32).to(dtype))
    rstd = O.w8a8_rstd(h32, EPS)
    for got, codes, scales, extra in ((y, xc, xs * rstd, 8 + chain_length(K)),
                                      (z, *O.w8a8_quantize_rows(f32(h) * (1.0 if il is None else il)), 0)):
        want = O.w8a8_gemm(codes, scales, wc, ws, f32(bias))
        term = np.abs(want - f32(bias))
        tol = (4 + extra) * U * term + (U + half(dtype) * 1.001) * np.abs(want) + 2.0 ** -25
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)
    # the quantised layer is the unquantised one up to 8-bit noise: every code is off by at most half a unit, so
    # an output by at most sum_k (|v| sw / 2 + |w| sx / 2 + sx sw / 4)
    v = (h32.astype(np.float64) * rstd[:, None] * w.double().cpu().numpy())
    full = v @ W.double().cpu().numpy().T + bias.double().cpu().numpy()
    vs = v if il is None else v * il
    wsm = W.double().cpu().numpy() if lam is None else W.double().cpu().numpy() * lam.double().cpu().numpy()
    sx, sw = np.abs(vs).max(1) / 127, np.abs(wsm).max(1) / 127
    bound = (np.abs(vs).sum(1)[:, None] * sw + np.abs(wsm).sum(1)[None, :] * sx[:, None] + K / 2 * np.outer(sx, sw)) / 2
    assert np.all(np.abs(y.double().cpu().numpy() - full) <= bound * 1.01 + half(dtype) * 1.01 * np.abs(full))


def test_normed_rows_feed_the_4_bit_layer():
    """A block that mixes schemes: the norm's bf16 rows through the nvfp4 layer, its codes through the W8A8 one."""
    from bit_w4a4_quantized_token_b200 import layer
    from bit_w4a4_quantized_token_b200 import workloads as W

    case = W.scaled(W.QKV, M=200, K=512, N=256, name="mixed")
    inp = {k: v.cuda() for k, v in W.make_inputs(case).items()}
    p4 = layer.pack_weight(inp["R"], inp["lam"], inp["L_down"], inp["L_up"], inp["b"])
    p8 = layer.pack_weight_w8a8(inp["R"], inp["lam"], inp["b"])
    w = uniform(512, 0.5, 2.0, 1, BF16).cuda()
    normed = torch.empty_like(inp["x"])
    h, q = layer.rms_norm_quantize_w8a8(inp["x"], inp["x"], w, p8, normed=normed)
    y8 = layer.gemm_w8a8(q, p8)
    y4 = layer.svdq_linear(normed, p4)
    want = torch.nn.functional.rms_norm(h.float(), (512,), w.float(), EPS).to(BF16)
    # h is rounded before torch's norm and not before ours: half a step of h, and of n
    assert bool(((normed.float() - want.float()).abs() <= 3 * half(BF16) * want.float().abs() + 1e-6).all())
    assert torch.equal(y4, layer.svdq_linear(normed.clone(), p4))
    assert bool(torch.isfinite(y8).all()) and bool(torch.isfinite(y4).all())


# -------------------------------------------------------- streams, graphs, sizes
def test_captured_and_replayed_with_new_inputs():
    """The two calls in one CUDA graph (static buffers), replayed on other inputs, beside eager calls."""
    from bit_w4a4_quantized_token_b200 import layer

    x, r, W, lam, bias, w = layer_inputs(200, 1024, 2048, BF16, True)
    packed = layer.pack_weight_w8a8(W, lam, bias)
    out = layer.alloc_act_w8a8(packed, 200, x.device)
    h, y = torch.empty_like(x), torch.empty(200, 2048, dtype=BF16, device="cuda")

    def step():
        layer.rms_norm_quantize_w8a8(x, r, w, packed, h_out=h, out=out)
        layer.gemm_w8a8(out, packed, y=y)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (21, 22):
        x.copy_(draw(200, 1024, BF16, seed).cuda())
        graph.replay()
        got_h, got_y = h.clone(), y.clone()
        want_h, q = layer.rms_norm_quantize_w8a8(x, r, w, packed)
        assert torch.equal(got_h, want_h) and torch.equal(got_y, layer.gemm_w8a8(q, packed))


def test_two_streams_at_once():
    """Calls on two streams, given explicitly and as the current one, on tensors of their own; no state is shared."""
    from bit_w4a4_quantized_token_b200 import layer

    sets = [layer_inputs(130 + 7 * i, 2048, 1024 + 8 * i, BF16, True) for i in range(2)]
    packed = [layer.pack_weight_w8a8(s[2], s[3], s[4]) for s in sets]
    want = [layer.w8a8_linear(s[0], p) for s, p in zip(sets, packed)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        got[0].append(layer.w8a8_linear(sets[0][0], packed[0], stream=streams[0]))
        with torch.cuda.stream(streams[1]):
            got[1].append(layer.w8a8_linear(sets[1][0], packed[1]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


@pytest.mark.parametrize("M,K,layers", [(1, 1024, 12), (40, 2048, 12), (700, 2048, 6), (3000, 1024, 6)])
def test_layer_after_layer_without_waiting(M, K, layers):
    """Each kernel starts while the one before it ends: a stack of layers run without a wait between the calls
    equals the same stack with a wait after each, in place on the same residual stream and buffers."""
    from bit_w4a4_quantized_token_b200 import layer

    weights = [layer.pack_weight_w8a8((torch.randn(K, K, generator=torch.Generator().manual_seed(i)) / K ** 0.5)
                                      .to(BF16).cuda(), uniform(K, 0.5, 2.0, i).cuda()) for i in range(layers)]
    w = uniform(K, 0.5, 2.0, 99, BF16).cuda()
    x0, r0 = draw(M, K, BF16, 1).cuda(), draw(M, K, BF16, 2).cuda()

    def stack(wait):
        x, r = x0.clone(), r0.clone()
        q = layer.alloc_act_w8a8(weights[0], M, x.device)
        for p in weights:
            layer.rms_norm_quantize_w8a8(x, r, w, p, h_out=r, out=q)
            if wait:
                torch.cuda.synchronize()
            layer.gemm_w8a8(q, p, y=x)
            if wait:
                torch.cuda.synchronize()
            layer.quantize_act_w8a8(x, p, out=q)
            if wait:
                torch.cuda.synchronize()
            layer.gemm_w8a8(q, p, y=x)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return x, r

    want = stack(True)
    assert bool(torch.isfinite(want[0]).all())
    for _ in range(3):
        got = stack(False)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


FIRST_CALL_IN_CAPTURE = """
import torch
from bit_w4a4_quantized_token_b200 import layer
x = torch.randn(70, 512, device="cuda").bfloat16()
codes = torch.randint(-127, 128, (264, 512), dtype=torch.int8, device="cuda")
p = layer.PackedWeightW8A8(264, 512, codes, torch.rand(264, device="cuda"), None, None)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    h, q = layer.rms_norm_quantize_w8a8(x, x, None, p)
    y = layer.gemm_w8a8(q, p)
    z = layer.w8a8_linear(x, p)
g.replay()
torch.cuda.synchronize()
h2, q2 = layer.rms_norm_quantize_w8a8(x, x, None, p)
assert torch.equal(h, h2) and torch.equal(y, layer.gemm_w8a8(q2, p)) and torch.equal(z, layer.w8a8_linear(x, p))
print("captured")
"""


def test_first_call_of_a_process_inside_a_capture():
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_IN_CAPTURE], cwd=root, capture_output=True, text=True,
                       timeout=300, env=dict(os.environ, PYTHONPATH=root))
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_refusals_of_tensors_on_the_gpu():
    """No rows, rows that start off a 16-byte boundary, rows that overlap one another, other widths and types."""
    from bit_w4a4_quantized_token_b200 import _lib, layer

    packed = packed_for(64)
    wide = torch.zeros(8, 80, dtype=BF16, device="cuda")
    for x, status in ((wide[:0, :64], _lib.SVDQ_ERR_UNSUPPORTED_SHAPE), (wide[:, 1:65], _lib.SVDQ_ERR_INVALID_ARG),
                      (wide[:1, :64].expand(8, 64), _lib.SVDQ_ERR_UNSUPPORTED_SHAPE),
                      (torch.zeros(8, 68, dtype=BF16, device="cuda")[:, :64], _lib.SVDQ_ERR_UNSUPPORTED_SHAPE)):
        for call in (lambda: layer.quantize_act_w8a8(x, packed),
                     lambda: layer.rms_norm_quantize_w8a8(x, None, None, packed)):
            with pytest.raises(_lib.SvdqError) as e:
                call()
            assert e.value.status == status
    x = wide[:, :64].contiguous()
    for bad in (dict(residual=x.half()), dict(residual=x[:4]), dict(residual=x.cpu()), dict(norm_weight=x[0].float()),
                dict(norm_weight=x[0, :32]), dict(h_out=x[:, :32]), dict(normed=x.float()),
                dict(out=layer.alloc_act_w8a8(packed, 7, x.device))):
        kw = dict(dict(residual=None, norm_weight=None), **bad)
        with pytest.raises(ValueError):
            layer.rms_norm_quantize_w8a8(x, kw.pop("residual"), kw.pop("norm_weight"), packed, **kw)
    with pytest.raises(_lib.SvdqError):
        layer.rms_norm_quantize_w8a8(x, None, None, packed, eps=0.0)
    q = layer.quantize_act_w8a8(x, packed)
    for bad in (dict(y=torch.empty(8, 8, device="cuda").t()[::2]), dict(y=torch.empty(8, 16, dtype=BF16, device="cuda")),
                dict(out_dtype=torch.float64)):
        with pytest.raises(ValueError):
            layer.gemm_w8a8(q, packed, **bad)
    with pytest.raises(ValueError):
        layer.gemm_w8a8(layer.QuantizedActW8A8(8, q.x_codes, q.x_scales.cpu()), packed)
    # an odd number of channels is refused by the library
    odd = layer.PackedWeightW8A8(7, 64, torch.zeros(7, 64, dtype=torch.int8, device="cuda"),
                                 torch.zeros(7, device="cuda"), None, None)
    with pytest.raises(_lib.SvdqError) as e:
        layer.gemm_w8a8(q, odd)
    assert e.value.status == _lib.SVDQ_ERR_UNSUPPORTED_SHAPE


def test_same_call_twice_gives_the_same_bits():
    from bit_w4a4_quantized_token_b200 import layer

    x, r, W, lam, bias, w = layer_inputs(33, 4096, 4096, BF16, True)
    packed = layer.pack_weight_w8a8(W, lam, bias)
    runs = []
    for _ in range(3):
        h, q = layer.rms_norm_quantize_w8a8(x, r, w, packed)
        runs.append((h, q.x_codes, q.x_scales, layer.gemm_w8a8(q, packed)))
    for other in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], other))


def test_offsets_past_32_bits():
    """Activations and outputs of more than 2^31 elements: the last rows are right."""
    from bit_w4a4_quantized_token_b200 import layer

    M, K = 140000, 16384                                # 2.3e9 elements of x and of codes
    x = torch.zeros(M, K, dtype=BF16, device="cuda")
    x[-3:] = draw(3, K, BF16, 1).cuda()
    packed = packed_for(K)
    q = layer.quantize_act_w8a8(x, packed)
    ref = layer.quantize_act_w8a8(x[-3:].contiguous(), packed)
    assert torch.equal(q.x_codes[-3:], ref.x_codes) and torch.equal(q.x_scales[-3:], ref.x_scales)
    assert not bool(q.x_scales[:-3].any())
    _, qn = layer.rms_norm_quantize_w8a8(x, None, None, packed)
    assert torch.equal(qn.x_codes[-3:], ref.x_codes)
    del x, qn
    y = layer.gemm_w8a8(q, layer.PackedWeightW8A8(24, K, codes_of(24, K, 3).cuda(), torch.ones(24, device="cuda"),
                                                  None, None))
    y3 = layer.gemm_w8a8(ref, layer.PackedWeightW8A8(24, K, codes_of(24, K, 3).cuda(), torch.ones(24, device="cuda"),
                                                     None, None))
    assert torch.equal(y[-3:], y3) and not bool(y[:-3].any())
    del q, y
    M, N, K = 280000, 8192, 32                          # 2.3e9 elements of y
    xc, wc = codes_of(M, K, 4).cuda(), codes_of(N, K, 5).cuda()
    one = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    y = layer.gemm_w8a8(layer.QuantizedActW8A8(M, xc, one[0]), layer.PackedWeightW8A8(N, K, wc, one[1], None, None))
    want = (xc[-500:].double() @ wc.double().t()).to(BF16)
    assert torch.equal(y[-500:], want)


def test_other_device_than_the_current_one():
    """Tensors of another GPU than the current one are run there (needs two GPUs)."""
    if torch.cuda.device_count() < 2:
        pytest.skip("needs two GPUs")
    from bit_w4a4_quantized_token_b200 import layer

    x, r, W, lam, bias, w = (t.to("cuda:1") for t in layer_inputs(33, 512, 256, BF16, True))
    packed = layer.pack_weight_w8a8(W, lam, bias)
    y = layer.w8a8_linear(x, packed)
    with torch.cuda.device(1):
        assert torch.equal(y, layer.w8a8_linear(x, packed))
