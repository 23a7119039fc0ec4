// quantize_w8a8.cuh -- the activation side of the 8-bit integer (W8A8) linear
// layer (sm_100a): one pass over the rows of a matrix that quantises each to
// signed 8-bit codes and one fp32 scale, with or without a residual addition
// and an RMSNorm in front.
//
// Mathematics of a row v[0..K) (g = 1 / lambda, or 1):
//     plain:  t = v g                           scale = fl(a / 127)
//     norm:   h = x + r,  t = h fl(w g)         scale = fl(fl(a / 127) / sqrt(mean h^2 + eps))
//     a = max |t|,   code = round_half_even(fl(t fl(127 / a)))
// The factor 1 / sqrt(mean h^2 + eps) of a row is common to all of its
// values, so it leaves the codes and enters the scale alone: sum of squares
// and maximum come from one reduction, and the codes do not depend on the
// order of any sum.  All of it is fp32, each step rounded once; h enters
// unrounded (the stored h is rounded to the stream's type once).
//   * a < 2^-100 (127 / a near the end of fp32): codes and scale 0.
//   * a row that holds an infinity or a NaN, or whose sum of squares
//     overflows fp32: codes 0 and scale NaN, so that the whole output row,
//     and no other, is NaN, and the whole normalised row too.  The maximum is taken over the bit patterns of
//     |t| as unsigned integers, where NaN > infinity > every finite value.
//
// Bound: memory traffic.  Per element b read (2 b with a residual), 1 byte of
// code and b of h written.  The gains w g (2 + 4 bytes per column) would be
// read again for every row, as much as the row itself, so in two of the three
// kernels below the blocks are persistent and keep the gains of their columns
// in registers:
//   * rows held in registers, the next row's loads issued before the
//     reduction of the current one (rows below 16 KB, x and the residual
//     together, and fp32 norms of up to 4096 columns);
//   * rows streamed through a ring in shared memory (wider ones);
//   * two passes over the row (above 16384 columns, or where shared memory does
//     not hold two rows).
// One barrier per row in each.  Measured on a B200, data from HBM: norm, bf16,
// M = 16384, K = 8192 160 us (939 MB: 5.9 TB/s, 0.90 of a measured copy;
// 891 MB of DRAM traffic in ncu, none of it read twice), M = 4608, K = 4096
// 24.4 us (0.83), M = 4608, K = 2048 13.8 us (0.73); norm, fp32, M = 16384, K =
// 4096 148 us (0.90); quantise, bf16, M = 4608, K = 4096 12.6 us (0.69), M =
// 16384, K = 8192 74 us (0.82); quantise, fp32, M = 4608, K = 4096 18.4 us
// (0.78), M = 16384, K = 8192 117 us (0.87); one token, K = 8192 2.6 to 3.2 us,
// all latency.  With `normed` beside the codes, bf16: M = 16384, K = 8192 214 us
// (0.86), M = 4608, K = 4096 31.1 us (0.83); `normed` alone 193 (0.85) and 28.3
// (0.82).  Where there is little to move per value, instruction issue bounds:
// the norm without a residual, bf16, M = 4608, K = 4096 21.2 us (0.41; ncu: 65 %
// of the issue slots, a fifth of DRAM), M = 16384, K = 8192 112 us (0.55); the
// quantiser's 12.6 us above have 53 % of the slots and a third of DRAM.
#pragma once
#include "sm100_ptx.cuh"
#include "w8a8_plan.h"

namespace svdq {

// Wait for the phase with the given parity; false after the wait limit.  The
// first tries only suspend in the hardware: reading the timer and the limit
// from memory costs hundreds of cycles, which a wait that ends soon must not
// pay (a wait of every stage that paid them bounded the 128 x 64 tiles of the
// W8A8 GEMM at ~900 cycles a stage).
__device__ __forceinline__ bool bounded_wait(uint64_t* bar, uint32_t parity, uint32_t site) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    return mbar_wait_timed(bar, parity, site);
}

namespace q8 {
constexpr int kMaxThreads = 512;     // of the register-resident kernel
constexpr int kTwoPassThreads = 1024;
constexpr float kTiny = 7.888609052210118e-31f;   // 2^-100
}  // namespace q8

// Element types of rows that are quantised or stored (svdq_dtype of the C header).
enum : int { kBf16 = 0, kF16 = 1, kF32 = 2 };

struct QuantRowsArgs {
    const void* x;             // [M, ldx]
    const void* residual;      // [M, ldr] or null
    const void* norm_weight;   // [K] of x's type or null (norm only)
    const float* gain;         // [K] fp32 factors (1 / lambda, or lambda when packing) or null
    void* h_out;               // [M, K] or null (norm only)
    void* normed;              // [M, K] or null (norm only)
    uint8_t* codes;            // [M, K] or null (norm only)
    float* scales;             // [M] or null
    int64_t ldx, ldr;
    int M, K;
    float eps;
};

// Eight consecutive values of a row as they lie in memory.
template <int T>
struct Raw8 {
    uint4 w[T == kF32 ? 2 : 1];
};

// Plain (coherent) vector load: h_out may be the memory that x or the residual is read from.
__device__ __forceinline__ uint4 ld_v4(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

template <int T>
__device__ __forceinline__ Raw8<T> ld_raw8(const void* base, int64_t elem) {
    Raw8<T> r;
    const uint8_t* p = reinterpret_cast<const uint8_t*>(base) + elem * (T == kF32 ? 4 : 2);
    r.w[0] = ld_v4(p);
    if (T == kF32) r.w[T == kF32 ? 1 : 0] = ld_v4(p + 16);
    return r;
}

template <int T>
__device__ __forceinline__ void raw_to_f32(const Raw8<T>& r, float (&f)[8]) {
    if (T == kF32) {
        const uint4 a = r.w[0], b = r.w[T == kF32 ? 1 : 0];
        f[0] = __uint_as_float(a.x), f[1] = __uint_as_float(a.y), f[2] = __uint_as_float(a.z);
        f[3] = __uint_as_float(a.w), f[4] = __uint_as_float(b.x), f[5] = __uint_as_float(b.y);
        f[6] = __uint_as_float(b.z), f[7] = __uint_as_float(b.w);
    } else {
        const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (T == kBf16) {
                f[2 * i] = bf16lo_to_f32(w[i]);
                f[2 * i + 1] = bf16hi_to_f32(w[i]);
            } else {
                const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                f[2 * i] = v.x;
                f[2 * i + 1] = v.y;
            }
        }
    }
}

// Two fp32 rounded to bf16 or fp16 (nearest even), packed.
template <int T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if (T == kBf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <int T>
__device__ __forceinline__ void st_f32x8(void* base, int64_t elem, const float (&f)[8]) {
    uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(base) + elem * (T == kF32 ? 4 : 2));
    if (T == kF32) {
        p[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        p[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
    } else {
        p[0] = make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
    }
}

// Eight codes round_half_even(fl(t inv)), |t inv| <= 127 up to rounding, as
// bytes: adding 1.5 * 2^23 leaves the nearest integer (ties to even) in the
// low bits of the sum, and the low byte of that is the two's complement code.
// The addition is the scalar intrinsic: the packed one after a packed product
// was fused with it into one rounding (seen in the results, where t inv is
// within one rounding of a half).
__device__ __forceinline__ uint2 codes8(const float (&t)[8], float inv) {
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        float c0, c1;
        fmul2_rn(t[i], t[i + 1], inv, inv, c0, c1);
        b[i] = __float_as_uint(__fadd_rn(c0, kMagicI2F));
        b[i + 1] = __float_as_uint(__fadd_rn(c1, kMagicI2F));
    }
    uint2 r;
    r.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    r.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
    return r;
}

// The row's factors from its reduced maximum (bits of a) and sum of squares.
struct RowFactors {
    float inv;     // 127 / a; 0: every code of the row is zero
    float scale;
    float rstd;    // 1 / sqrt(mean h^2 + eps)
};
template <bool NORM>
__device__ __forceinline__ RowFactors row_factors(uint32_t abits, float ss, int K, float eps) {
    RowFactors f;
    const float a = __uint_as_float(abits);
    const bool some = a >= q8::kTiny && abits < 0x7F800000u;
    f.inv = some ? __fdiv_rn(127.0f, a) : 0.0f;
    f.scale = some ? __fdiv_rn(a, 127.0f) : 0.0f;
    f.rstd = 1.0f;
    bool bad = abits >= 0x7F800000u;
    if (NORM) {
        // an infinite sum has the factor NaN, not the 0 that its root gives:
        // the normalised values of a finite row would be zeros
        const bool lost = !(ss < __int_as_float(0x7F800000));
        f.rstd = lost ? __int_as_float(0x7FC00000) : __frsqrt_rn(__fadd_rn(__fdiv_rn(ss, (float)K), eps));
        f.scale = __fmul_rn(f.scale, f.rstd);
        bad = bad || lost;
    }
    if (bad) {
        f.inv = 0.0f;
        f.scale = __int_as_float(0x7FC00000);
    }
    return f;
}

// Maximum of abits and sum of ss over a group of warps of the block (this one
// is number `warp` of threads / 32); `slot` holds one entry per warp and is not
// written again before the group's next barrier but one.
template <bool NORM>
__device__ __forceinline__ void group_reduce(uint32_t& abits, float& ss, uint2* slot, int warp, int threads) {
    abits = __reduce_max_sync(0xffffffffu, abits);
    if (NORM) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    if (lane_id() == 0) slot[warp] = make_uint2(abits, __float_as_uint(ss));
    named_bar_sync(1, (uint32_t)threads);
    const int warps = threads >> 5;
    uint2 v = make_uint2(0u, 0u);
    if ((int)lane_id() < warps) v = slot[lane_id()];
    abits = __reduce_max_sync(0xffffffffu, v.x);
    if (NORM) {
        ss = __uint_as_float(v.y);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
}

// The block's next row (M when there is none); M may be near 2^31.
__device__ __forceinline__ int next_row(int row, int M) {
    return (int)min((int64_t)row + (int64_t)gridDim.x, (int64_t)M);
}

// max |t| of eight values, as bits
__device__ __forceinline__ uint32_t amax_bits8(const float (&t)[8], uint32_t m) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(t[i]) & 0x7FFFFFFFu);
    return m;
}

// Eight columns (vector c) of a row's outputs that need its factors.
template <int T, bool NORM>
__device__ __forceinline__ void store_row8(const QuantRowsArgs& a, int row, int c, const float (&h)[8],
                                           const float (&gain)[8], const RowFactors& f) {
    if (!NORM || a.codes) {
        float t[8];
#pragma unroll
        for (int i = 0; i < 8; i += 2) fmul2_rn(h[i], h[i + 1], gain[i], gain[i + 1], t[i], t[i + 1]);
        uint2 code = codes8(t, f.inv);
        if (f.inv == 0.0f) code = make_uint2(0u, 0u);   // also where t is not finite
        *reinterpret_cast<uint2*>(a.codes + (int64_t)row * a.K + 8 * (int64_t)c) = code;
    }
    if (NORM && a.normed) {
        float w[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
        if (a.norm_weight) raw_to_f32<T>(ld_raw8<T>(a.norm_weight, 8 * (int64_t)c), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __fmul_rn(__fmul_rn(h[i], f.rstd), w[i]);
        st_f32x8<T>(a.normed, (int64_t)row * a.K + 8 * (int64_t)c, w);
    }
}

// Rows held in registers: thread i of a block of T threads owns columns
// 8 (i + T v) .. + 7, v < V.  Every block takes rows blockIdx.x + j gridDim.x.
template <int T, bool NORM, int V>
__global__ void __launch_bounds__(q8::kMaxThreads) quantize_rows_w8_kernel(QuantRowsArgs a) {
    __shared__ uint2 slots[2][32];
    const int tid = (int)threadIdx.x, step = (int)blockDim.x;
    const int nvec = a.K >> 3;
    // the previous kernel of the stream wrote what is read here
    griddep_wait();
    griddep_launch_dependents();
    float gain[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = tid + v * step;
#pragma unroll
        for (int i = 0; i < 8; ++i) gain[v][i] = 1.0f;
        if (c < nvec) {
            if (NORM && a.norm_weight) raw_to_f32<T>(ld_raw8<T>(a.norm_weight, 8 * (int64_t)c), gain[v]);
            if (a.gain) {
                float g[8];
                raw_to_f32<kF32>(ld_raw8<kF32>(a.gain, 8 * (int64_t)c), g);
#pragma unroll
                for (int i = 0; i < 8; ++i) gain[v][i] = __fmul_rn(gain[v][i], g[i]);
            }
        }
    }
    Raw8<T> rx[V], rr[NORM ? V : 1];
    const bool has_res = NORM && a.residual != nullptr;
    auto load_row = [&](int row) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = tid + v * step;
            if (c < nvec) {
                rx[v] = ld_raw8<T>(a.x, (int64_t)row * a.ldx + 8 * c);
                if (NORM && has_res) rr[NORM ? v : 0] = ld_raw8<T>(a.residual, (int64_t)row * a.ldr + 8 * c);
            }
        }
    };
    int row = (int)blockIdx.x;
    if (row < a.M) load_row(row);
    for (int buf = 0; row < a.M; buf ^= 1) {
        float h[V][8];
        uint32_t abits = 0u;
        float ss = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = tid + v * step;
            if (c < nvec) {
                raw_to_f32<T>(rx[v], h[v]);
                if (NORM && has_res) {
                    float r[8];
                    raw_to_f32<T>(rr[NORM ? v : 0], r);
#pragma unroll
                    for (int i = 0; i < 8; i += 2)
                        fadd2_rn(h[v][i], h[v][i + 1], r[i], r[i + 1], h[v][i], h[v][i + 1]);
                }
                if (NORM) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss = fmaf(h[v][i], h[v][i], ss);
                    if (a.h_out) st_f32x8<T>(a.h_out, (int64_t)row * a.K + 8 * c, h[v]);
                }
                float t[8];
#pragma unroll
                for (int i = 0; i < 8; i += 2)
                    fmul2_rn(h[v][i], h[v][i + 1], gain[v][i], gain[v][i + 1], t[i], t[i + 1]);
                abits = amax_bits8(t, abits);
            }
        }
        const int next = next_row(row, a.M);
        if (next < a.M) load_row(next);
        group_reduce<NORM>(abits, ss, slots[buf], (int)warp_id(), step);
        const RowFactors f = row_factors<NORM>(abits, ss, a.K, a.eps);
        if (a.scales && tid == 0) a.scales[row] = f.scale;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = tid + v * step;
            if (c < nvec) store_row8<T, NORM>(a, row, c, h[v], gain[v], f);
        }
        row = next;
    }
}

// The same rows streamed: thread 0 copies whole rows (x, and the residual
// behind it) into a ring of shared memory, so that the bytes in flight are the
// ring's and not what the registers of the threads can hold.  The barrier of a
// row's reduction also says that every thread has read the row, so the copy
// of a later row into its place follows it without a barrier of its own.
namespace q8 {
constexpr int kRingThreads = 1024;
constexpr int kRingVec = 2;          // vectors of eight columns per thread (one: the same time; four: 96 registers)
constexpr int kMaxRing = 8;
constexpr int kRingBarBytes = 128;
}  // namespace q8
enum : uint32_t { kSiteQ8Full = 50, kSiteQ8Drain = 51 };

template <int T>
__device__ __forceinline__ Raw8<T> lds_raw8(const uint8_t* row, int vec) {
    Raw8<T> r;
    const uint4* p = reinterpret_cast<const uint4*>(row + (int64_t)vec * (T == kF32 ? 32 : 16));
    r.w[0] = p[0];
    if (T == kF32) r.w[T == kF32 ? 1 : 0] = p[1];
    return r;
}

template <int T, bool NORM>
__global__ void __launch_bounds__(q8::kRingThreads) quantize_rows_w8_ring_kernel(QuantRowsArgs a, int stages) {
    using namespace q8;
    constexpr int V = kRingVec;
    extern __shared__ __align__(128) uint8_t ring[];   // barriers, then `stages` rows (x, residual)
    __shared__ uint2 slots[2][32];
    uint64_t* full = reinterpret_cast<uint64_t*>(ring);
    uint8_t* rows = ring + kRingBarBytes;
    const int tid = (int)threadIdx.x, step = (int)blockDim.x;
    const int nvec = a.K >> 3;
    const bool has_res = NORM && a.residual != nullptr;
    const uint32_t row_bytes = (uint32_t)a.K * (T == kF32 ? 4u : 2u);
    const uint32_t stage_bytes = has_res ? 2u * row_bytes : row_bytes;
    if (tid == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
        fence_barrier_init();
    }
    __syncthreads();
    // the previous kernel of the stream wrote what is read here
    griddep_wait();
    griddep_launch_dependents();
    const auto fetch = [&](int row, int s) {   // thread 0
        constexpr int b = T == kF32 ? 4 : 2;
        uint8_t* dst = rows + (size_t)s * stage_bytes;
        mbar_arrive_expect_tx(&full[s], stage_bytes);
        bulk_load(dst, reinterpret_cast<const uint8_t*>(a.x) + (int64_t)row * a.ldx * b, row_bytes, &full[s]);
        if (has_res)
            bulk_load(dst + row_bytes, reinterpret_cast<const uint8_t*>(a.residual) + (int64_t)row * a.ldr * b,
                      row_bytes, &full[s]);
    };
    int ahead = (int)blockIdx.x;   // thread 0: the next row to fetch
    if (tid == 0)
        for (int s = 0; s < stages && ahead < a.M; ++s, ahead = next_row(ahead, a.M)) fetch(ahead, s);
    float gain[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = tid + v * step;
#pragma unroll
        for (int i = 0; i < 8; ++i) gain[v][i] = 1.0f;
        if (c < nvec) {
            if (NORM && a.norm_weight) raw_to_f32<T>(ld_raw8<T>(a.norm_weight, 8 * (int64_t)c), gain[v]);
            if (a.gain) {
                float g[8];
                raw_to_f32<kF32>(ld_raw8<kF32>(a.gain, 8 * (int64_t)c), g);
#pragma unroll
                for (int i = 0; i < 8; ++i) gain[v][i] = __fmul_rn(gain[v][i], g[i]);
            }
        }
    }
    int s = 0, buf = 0;
    uint32_t ph = 0u;
    int lost = -1;   // the row whose wait ran out
    for (int row = (int)blockIdx.x; row < a.M; row = next_row(row, a.M), buf ^= 1) {
        // after a timeout the block runs on without waiting and without fetching (its rows are void)
        if (lost < 0 && !bounded_wait(&full[s], ph, kSiteQ8Full)) lost = row;
        const uint8_t* src = rows + (size_t)s * stage_bytes;
        float h[V][8];
        uint32_t abits = 0u;
        float ss = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = tid + v * step;
            if (c < nvec) {
                raw_to_f32<T>(lds_raw8<T>(src, c), h[v]);
                if (has_res) {
                    float r[8];
                    raw_to_f32<T>(lds_raw8<T>(src + row_bytes, c), r);
#pragma unroll
                    for (int i = 0; i < 8; i += 2)
                        fadd2_rn(h[v][i], h[v][i + 1], r[i], r[i + 1], h[v][i], h[v][i + 1]);
                }
                float t[8];
#pragma unroll
                for (int i = 0; i < 8; i += 2)
                    fmul2_rn(h[v][i], h[v][i + 1], gain[v][i], gain[v][i + 1], t[i], t[i + 1]);
                abits = amax_bits8(t, abits);
                if (NORM) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss = fmaf(h[v][i], h[v][i], ss);
                }
            }
        }
        group_reduce<NORM>(abits, ss, slots[buf], (int)warp_id(), step);
        if (tid == 0 && lost < 0 && ahead < a.M) {
            fetch(ahead, s);
            ahead = next_row(ahead, a.M);
        }
        if (++s == stages) {
            s = 0;
            ph ^= 1u;
        }
        const RowFactors f = row_factors<NORM>(abits, ss, a.K, a.eps);
        if (a.scales && tid == 0) a.scales[row] = f.scale;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = tid + v * step;
            if (c < nvec) {
                if (NORM && a.h_out) st_f32x8<T>(a.h_out, (int64_t)row * a.K + 8 * c, h[v]);
                store_row8<T, NORM>(a, row, c, h[v], gain[v], f);
            }
        }
    }
    // no copy is in flight when the block ends, even after a timeout (best effort: each wait is bounded)
    if (tid == 0 && lost >= 0)
        drain_ring((int)blockIdx.x, (int)gridDim.x, lost, ahead, stages,
                   [&](int i, uint32_t parity) { mbar_wait(&full[i], parity, kSiteQ8Drain); });
}

// Rows too wide for the registers of one block: statistics in a first pass
// over the row, codes in a second one, which finds the row in the caches.
// h_out is written in the second pass only, each element by the thread that
// reads it, so it may be the memory of x or of the residual.
template <int T, bool NORM>
__global__ void __launch_bounds__(q8::kTwoPassThreads) quantize_rows_w8_wide_kernel(QuantRowsArgs a) {
    __shared__ uint2 slots[2][32];
    const int tid = (int)threadIdx.x, step = (int)blockDim.x;
    const int nvec = a.K >> 3;
    griddep_wait();
    griddep_launch_dependents();
    auto load_h = [&](int row, int c, float (&h)[8]) {
        raw_to_f32<T>(ld_raw8<T>(a.x, (int64_t)row * a.ldx + 8 * (int64_t)c), h);
        if (NORM && a.residual) {
            float r[8];
            raw_to_f32<T>(ld_raw8<T>(a.residual, (int64_t)row * a.ldr + 8 * (int64_t)c), r);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = __fadd_rn(h[i], r[i]);
        }
    };
    auto weight8 = [&](int c, float (&w)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.0f;
        if (NORM && a.norm_weight) raw_to_f32<T>(ld_raw8<T>(a.norm_weight, 8 * (int64_t)c), w);
    };
    auto gained = [&](int c, const float (&h)[8], const float (&w)[8], float (&t)[8]) {
        float g[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
        if (a.gain) raw_to_f32<kF32>(ld_raw8<kF32>(a.gain, 8 * (int64_t)c), g);
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = __fmul_rn(h[i], __fmul_rn(w[i], g[i]));
    };
    int buf = 0;
    for (int row = (int)blockIdx.x; row < a.M; row = next_row(row, a.M), buf ^= 1) {
        uint32_t abits = 0u;
        float ss = 0.0f;
#pragma unroll 2
        for (int c = tid; c < nvec; c += step) {
            float h[8], w[8], t[8];
            load_h(row, c, h);
            weight8(c, w);
            gained(c, h, w, t);
            if (NORM) {
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(h[i], h[i], ss);
            }
            abits = amax_bits8(t, abits);
        }
        group_reduce<NORM>(abits, ss, slots[buf], (int)warp_id(), step);
        const RowFactors f = row_factors<NORM>(abits, ss, a.K, a.eps);
        if (a.scales && tid == 0) a.scales[row] = f.scale;
#pragma unroll 2
        for (int c = tid; c < nvec; c += step) {
            float h[8], w[8];
            load_h(row, c, h);
            weight8(c, w);
            if (NORM && a.h_out) st_f32x8<T>(a.h_out, (int64_t)row * a.K + 8 * (int64_t)c, h);
            if (!NORM || a.codes) {
                float t[8];
                gained(c, h, w, t);
                uint2 code = codes8(t, f.inv);
                if (f.inv == 0.0f) code = make_uint2(0u, 0u);
                *reinterpret_cast<uint2*>(a.codes + (int64_t)row * a.K + 8 * (int64_t)c) = code;
            }
            if (NORM && a.normed) {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = __fmul_rn(__fmul_rn(h[i], f.rstd), w[i]);
                st_f32x8<T>(a.normed, (int64_t)row * a.K + 8 * (int64_t)c, w);
            }
        }
    }
}

}  // namespace svdq
