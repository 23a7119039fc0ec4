// gemm_w8a8.cuh -- the 8-bit integer GEMM of the W8A8 linear layer (sm_100a):
//     y[m, n] = round( float(sum_k qx[m, k] qw[n, k]) sx[m] sw[n] + b[n] )
// with signed 8-bit codes, one fp32 scale per token and per output channel,
// and the sum exact in int32 (K < 2^17, so that even codes of -128 cannot
// overflow it).  The scales are common to whole rows and columns of the
// product, so they stay out of the main loop: tcgen05.mma kind::i8 multiplies
// the codes as they lie in memory (K-major rows, 128-byte swizzled TMA boxes)
// and the epilogue scales once per output.
//
// Two kernels compute it, with the same bits (the host picks by an estimate of
// their times, w8_plan in w8a8_plan.h):
//  * gemm_w8a8_pair_kernel: 256 x 256 output tiles on two-CTA clusters, for
//    problems that fill the chip with such tiles;
//  * gemm_w8a8_narrow_kernel: 64 to 128 output channels x 16 to 128 tokens on
//    single CTAs, the K range split over a cluster if that pays, for few
//    tokens or few tiles.
//
// Bound.  Many tokens: the tensor pipe.  A pair's stage (two chunks of K, eight
// M256 N256 K32 MMAs) takes 1030 to 1060 cycles of 1024 at the pipe's 8192
// products per SM and cycle; ncu: pipe 90 % active at 4608 x 12288 x 4096, its
// operands read from DRAM once (69 MB).  The board's power cap then sets the
// clock (1.4 to 1.6 GHz).  Few tokens: the weight's bytes from HBM.  Measured
// on a B200 (M x N x K, bf16 out, data from HBM, us; P = 10^15 operations a
// second, 2 M N K; the measured bf16 GEMM peak doubled is 3.26 P, sustained
// 2.75 P; torch._int_mm, which leaves int32 sums, beside it):
//     16384 x 8192 x 8192   650-750  2.9-3.4 P   855
//     4608 x 12288 x 4096   152-169  2.7-3.0 P   207
//     4608 x 4096 x 12288   147-166  2.8-3.2 P   155
//     2048 x 6144 x 4096    38       2.7 P       47
//     1000 x 4104 x 4112    20.6     1.6 P       25   (rows off the 128-byte lines)
//     16 x 28672 x 8192     41.6     5.7 TB/s         (a plain stream of the weight: 39.9)
//     1 x 10240 x 8192      16.8     5.0 TB/s
//     1 x 4096 x 4096       6.6
//     64 x 256 x 256        2.6      (latency of one tile)
#pragma once
#include "gelu_mlp.cuh"        // st_shared_v4
#include "quantize_w8a8.cuh"   // the element types, pack2
#include "w8a8_plan.h"         // tile sizes, shared memory of the narrow kernel

namespace svdq {

struct GemmW8Args {
    const float* x_scales;   // [M]
    const float* w_scales;   // [N]
    const void* bias;        // [N] of y's type, or null
    void* y;                 // [M, N]
    int M, N;
    int chunks;              // ceil(K / 128): stages of 128 bytes of K
    int last_steps;          // 32-byte K-steps of the last chunk (1..4)
    int m_tiles, n_tiles;
    int group_m;             // pair kernel: row tiles that are walked together
    int stages;              // narrow kernel: ring depth
    int tile_n;              // narrow kernel: output channels of a tile (a multiple of 8, at most 128)
};

// D[tmem] (+)= A[smem] * B[smem]^T with signed 8-bit integers, s32 accumulate, on a CTA pair.
__device__ __forceinline__ void mma_s8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ float bias_at(const void* bias, int out, int n) {
    if (bias == nullptr) return 0.0f;
    if (out == kF32) return reinterpret_cast<const float*>(bias)[n];
    if (out == kF16) return __half2float(reinterpret_cast<const __half*>(bias)[n]);
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(bias)[n]);
}

enum : uint32_t {
    kSiteW8Empty = 56,
    kSiteW8Full = 57,
    kSiteW8Acc = 58,
    kSiteW8AccEmpty = 59,
    kSiteW8Drain = 60,
    kSiteW8NarrowEmpty = 61,
    kSiteW8NarrowFull = 62,
    kSiteW8NarrowAcc = 63,
    kSiteW8NarrowDrain = 64
};

// ------------------------------------------------------------ CTA-pair kernel
namespace w8p {
constexpr int kPer = 2;                       // chunks per stage
constexpr int kStages = 3;
constexpr int A_BYTES = 128 * BK;             // of one chunk
constexpr int B_BYTES = 128 * BK;
constexpr int STAGE_BYTES = kPer * (A_BYTES + B_BYTES);
constexpr int kWarpX = 0, kWarpW = 1, kWarpMma = 2, kWarpAlloc = 3;   // roles of warps 0..3
constexpr int kEpiWarp0 = 4;
constexpr int kEpiWarps = 8;                  // two per TMEM lane quarter, 128 columns each
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
constexpr uint32_t ACC_COLS = BN;             // two accumulators fill the 512 columns of TMEM
constexpr int kBoxBytes = 2048;               // y staging: 32 rows x 64 bytes per epilogue warp
constexpr int kColBytes = 128 * 4;            // one epilogue warp's 128 channel scales (and as much for the bias)
constexpr size_t BAR_OFF = (size_t)kStages * STAGE_BYTES;
constexpr size_t BOX_OFF = BAR_OFF + 1024;    // 1 KB aligned for the swizzle
constexpr size_t COL_OFF = BOX_OFF + (size_t)kEpiWarps * kBoxBytes;
constexpr size_t SMEM_BYTES = 1024 + COL_OFF + (size_t)kEpiWarps * 2 * kColBytes;
static_assert((2 * kStages + 4) * 8 + 4 <= 1024, "barriers do not fit");
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
}  // namespace w8p

// Tile of a running index: groups of group_m row tiles, the row tile fastest,
// so that the ~74 tiles in flight form a block that shares its operands in the
// L2 (a row-major walk keeps 74 different weight tiles in flight and re-reads
// the whole weight for every row tile).
__device__ __forceinline__ void w8_tile(int id, const GemmW8Args& a, int& m, int& n) {
    const int per_group = a.group_m * a.n_tiles;
    const int g = id / per_group, in = id - g * per_group;
    const int gm = min(a.group_m, a.m_tiles - g * a.group_m);
    n = in / gm;
    m = g * a.group_m + (in - n * gm);
}

template <int OUT>
__global__ void __launch_bounds__(w8p::kThreads, 1)
    gemm_w8a8_pair_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                          const __grid_constant__ CUtensorMap tm_y, GemmW8Args a) {
    using namespace w8p;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + BAR_OFF);
    uint64_t* empty = full + kStages;
    uint64_t* acc_full = empty + kStages;     // [2]
    uint64_t* acc_empty = acc_full + 2;       // [2]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
    __shared__ int s_failed;
    __shared__ int s_issued[kStages];         // phases this CTA's token loads started in each stage

    const uint32_t warp = warp_id(), lane = lane_id();
    const uint32_t rank = cluster_ctarank();  // 0: the CTA that issues the MMAs
    const int cluster = (int)(blockIdx.x >> 1), n_clusters = (int)(gridDim.x >> 1);
    const int total = a.m_tiles * a.n_tiles;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 2);           // CTA 0's two producers, for both CTAs' bytes
            mbar_init(&empty[s], 1);
            s_issued[s] = 0;
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 2 * kEpiWarps);   // both CTAs' epilogue warps
        }
        s_failed = 0;
        fence_barrier_init();
    }
    if (warp == kWarpX && lane == 0) {
        prefetch_tensormap(&tm_x);
        prefetch_tensormap(&tm_w);
        prefetch_tensormap(&tm_y);
    }
    if (warp == kWarpAlloc) {
        tmem_alloc_pair(tmem_slot, 2 * ACC_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // the first weight stages on their way into the L2 while the previous
    // kernel ends (only into the L2: that kernel may have written them)
    if (warp >= (uint32_t)kEpiWarp0 && lane == 0) {
        int m, n;
        w8_tile(cluster, a, m, n);
        const int c = (int)warp - kEpiWarp0;
        if (c < min(a.chunks, kStages * kPer)) tma_prefetch_l2_2d(&tm_w, c * BK, n * BN + 128 * (int)rank);
    }
    griddep_wait();   // everything above overlaps the end of the previous kernel

    if (warp == kWarpX || warp == kWarpW) {
        // ---------------------------------------------------------- producers
        // Each CTA loads its own 128 token rows and 128 weight rows of every
        // stage; all loads complete on CTA 0's barrier.
        if (lane == 0) {
            const bool is_x = warp == kWarpX;
            const CUtensorMap* map = is_x ? &tm_x : &tm_w;
            int s = 0;
            uint32_t ph = 1u;
            bool ok = true;
            for (int id = cluster; id < total && ok; id += n_clusters) {
                int m, n;
                w8_tile(id, a, m, n);
                const int row0 = (is_x ? m * BM : n * BN) + 128 * (int)rank;
                for (int c = 0; c < a.chunks; c += kPer) {
                    if (!bounded_wait(&empty[s], ph, kSiteW8Empty)) {
                        s_failed = 1;
                        ok = false;
                        break;
                    }
                    uint8_t* dst = smem + (size_t)s * STAGE_BYTES + (is_x ? 0 : kPer * A_BYTES);
                    const uint32_t bar = cluster_addr(&full[s], 0);
                    const bool both = c + 1 < a.chunks;
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], both ? 4u * A_BYTES : 2u * A_BYTES);
                    tma_load_2d_pair(dst, map, bar, c * BK, row0);
                    if (both) tma_load_2d_pair(dst + A_BYTES, map, bar, (c + 1) * BK, row0);
                    if (is_x) s_issued[s] = s_issued[s] + 1;
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
        }
    } else if (warp == kWarpMma) {
        // ------------------------------------------------- MMAs (CTA 0 only)
        if (rank == 0 && lane == 0) {
            const uint32_t idesc = idesc_m(idesc_s8_s32(BN), BM);
            const uint32_t smem0 = smem_u32(smem);
            int s = 0, local = 0;
            uint32_t ph = 0u;
            bool ok = true;
            for (int id = cluster; id < total && ok; id += n_clusters, ++local) {
                const uint32_t acc = tmem + (uint32_t)(local & 1) * ACC_COLS;
                if (!bounded_wait(&acc_empty[local & 1], ((uint32_t)(local >> 1) & 1u) ^ 1u, kSiteW8AccEmpty)) {
                    s_failed = 1;
                    break;
                }
                for (int c = 0; c < a.chunks; c += kPer) {
                    if (!bounded_wait(&full[s], ph, kSiteW8Full)) {
                        s_failed = 1;
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem0 + (uint32_t)s * STAGE_BYTES;
                    const uint64_t da = desc_sw128(sa), db = desc_sw128(sa + kPer * A_BYTES);
                    const uint32_t more = c > 0 ? 1u : 0u;
                    // K-step j of the stage: 32 bytes of K, 2 descriptor units apart inside a chunk
                    const auto mma = [&](int j) {
                        mma_s8_pair(acc, da + (uint64_t)(j >> 2) * (A_BYTES >> 4) + 2u * (j & 3),
                                    db + (uint64_t)(j >> 2) * (B_BYTES >> 4) + 2u * (j & 3), idesc, j == 0 ? more : 1u);
                    };
                    if (c + kPer < a.chunks || (c + kPer == a.chunks && a.last_steps == 4)) {
#pragma unroll
                        for (int j = 0; j < 4 * kPer; ++j) mma(j);
                    } else {   // the end of K inside a stage
                        const int n_steps = 4 * (a.chunks - c - 1) + a.last_steps;
                        for (int j = 0; j < n_steps; ++j) mma(j);
                    }
                    tc_commit_pair(&empty[s], 0x3);
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (ok) tc_commit_pair(&acc_full[local & 1], 0x3);
            }
        }
    } else if (warp >= (uint32_t)kEpiWarp0) {
        // ----------------------------------------------------------- epilogue
        const uint32_t q = warp & 3u, e = warp - kEpiWarp0;
        const int half = (int)(e >> 2);
        float* col_s = reinterpret_cast<float*>(smem + COL_OFF + (size_t)e * 2 * kColBytes);
        float* col_b = col_s + 128;
        constexpr int kBoxCols = OUT == kF32 ? 16 : 32, kBoxes = 128 / kBoxCols;
        static_assert(kEpiWarps * kBoxes * kBoxBytes <= BAR_OFF, "the last tile's boxes do not fit in the ring");
        int local = 0;
        for (int id = cluster; id < total; id += n_clusters, ++local) {
            int mt, nt;
            w8_tile(id, a, mt, nt);
            const int row0 = mt * BM + 128 * (int)rank + 32 * (int)q;   // the warp's first token
            const int row = row0 + (int)lane;
            const int n0 = nt * BN + 128 * half;
            // the warp's channel scales and bias, before the accumulator is ready
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = n0 + 32 * i + (int)lane;
                col_s[32 * i + lane] = n < a.N ? a.w_scales[n] : 0.0f;
                col_b[32 * i + lane] = n < a.N ? bias_at(a.bias, OUT, n) : 0.0f;
            }
            const float sx = row < a.M ? a.x_scales[row] : 0.0f;
            __syncwarp();
            if (!bounded_wait(&acc_full[local & 1], (uint32_t)(local >> 1) & 1u, kSiteW8Acc)) {
                s_failed = 1;
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + ((32u * q) << 16) + (uint32_t)(local & 1) * ACC_COLS + 128u * (uint32_t)half;
            // The main loop hides the epilogue of every tile but the last.
            // There each box has its own place in the ring, which is drained
            // by now, so that no box waits for the store of another.
            const bool last = id + n_clusters >= total;
            if (last) griddep_launch_dependents();
            const uint32_t box0 = last ? smem_u32(smem) + e * (uint32_t)(kBoxes * kBoxBytes)
                                       : smem_u32(smem + BOX_OFF) + e * (uint32_t)kBoxBytes;
            uint32_t v[32];
            tmem_ld_32x32b_x32(acc, v);
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                float o[32];
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = (float)(int)v[i];
                // the next columns are on their way while these are scaled and stored
                if (c < 3) tmem_ld_32x32b_x32(acc + 32u * (c + 1), v);
                if (c == 3) {   // drained: the accumulator may be overwritten
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(cluster_addr(&acc_empty[local & 1], 0));
                }
                if (n0 + 32 * c >= a.N) continue;   // warp-uniform
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 s4 = *reinterpret_cast<const float4*>(col_s + 32 * c + i);
                    const float4 b4 = *reinterpret_cast<const float4*>(col_b + 32 * c + i);
                    fmul2_rn(o[i], o[i + 1], sx, sx, o[i], o[i + 1]);
                    fmul2_rn(o[i + 2], o[i + 3], sx, sx, o[i + 2], o[i + 3]);
                    ffma2_rn(o[i], o[i + 1], s4.x, s4.y, b4.x, b4.y, o[i], o[i + 1]);
                    ffma2_rn(o[i + 2], o[i + 3], s4.z, s4.w, b4.z, b4.w, o[i + 2], o[i + 3]);
                }
#pragma unroll
                for (int p = 0; p < 32 / kBoxCols; ++p) {
                    // 32 rows x 64 bytes through the warp's box (64-byte swizzle), stored with TMA
                    const uint32_t box = last ? box0 + (uint32_t)((c * 32 / kBoxCols + p) * kBoxBytes) : box0;
                    if (!last) {
                        if (lane == 0) bulk_wait_group_read<0>();
                        __syncwarp();
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if (OUT == kF32) {
                                w[k] = __float_as_uint(o[(16 * p + 4 * j + k) & 31]);
                            } else {
                                w[k] = pack2<OUT>(o[(8 * j + 2 * k) & 31], o[(8 * j + 2 * k + 1) & 31]);
                            }
                        }
                        st_shared_v4(box + 64u * lane + ((uint32_t)(j ^ ((lane >> 1) & 3)) << 4), w[0], w[1], w[2],
                                     w[3]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    const int n = n0 + 32 * c + kBoxCols * p;
                    if (lane == 0 && row0 < a.M && n < a.N) {   // parts past M or N are clipped by the map
                        tma_store_2d(&tm_y, box, n, row0);
                        bulk_commit_group();
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_group<0>();
    }

    __syncwarp();
    __syncthreads();
    if (s_failed && rank == 0 && warp == 0 && lane == 0) {
        // after a timeout, let the loads already issued land before either CTA
        // exits (best effort: each wait is bounded)
        for (int s = 0; s < kStages; ++s) {
            const int n = *reinterpret_cast<volatile int*>(&s_issued[s]);
            if (n > 0) bounded_wait(&full[s], (uint32_t)(n - 1) & 1u, kSiteW8Drain);
        }
    }
    tc_fence_before();
    cluster_sync_all();   // no remote arrival or MMA may target a CTA that has exited
    if (warp == kWarpAlloc) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 2 * ACC_COLS);
    }
}

// -------------------------------------------------------------- narrow kernel
namespace w8n {
constexpr int kEpiWarps = 8;                  // two per TMEM lane quarter, taking turns of 16 tokens
// A thread issues a TMA load about every 300 cycles whatever the size of its
// box, so three share the loads: two take turns with the weight boxes, one
// loads the token boxes.
constexpr int kWarpW0 = 0, kWarpW1 = 1, kWarpX = 2;
// Two warps issue the MMAs of alternate stages into an accumulator each (the
// epilogue adds the two, exactly): one thread needs ~1000 cycles for the wait,
// the eight MMAs and the commit of a stage, which held a CTA below 40 bytes of
// weights a cycle.
constexpr int kWarpMma0 = 3, kWarpMma1 = 4, kEpiWarp0 = 5;
constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps);
static_assert((2 * kMaxStages + 1) * 8 + 4 <= kBarBytes, "barriers do not fit");
}  // namespace w8n

__device__ __forceinline__ uint32_t cluster_addr_u32(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_cluster_s32(uint32_t addr, int v) {
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <int OUT>
struct OutType {
    using type = __nv_bfloat16;
    __device__ static __nv_bfloat16 of(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct OutType<kF16> {
    using type = __half;
    __device__ static __half of(float v) { return __float2half_rn(v); }
};
template <>
struct OutType<kF32> {
    using type = float;
    __device__ static float of(float v) { return v; }
};

// The product transposed: the MMA's A operand (M = 128) holds weight rows, its
// B operand NT token rows, so that few tokens cost few tensor-core columns and
// few bytes of TMEM, and the weight streams through a ring as deep as shared
// memory allows.  The cluster's CTAs split the K range; each sends the int32
// partial sums of a token to the CTA that owns it (token i of the tile: CTA
// i mod split), which adds them (exact, so the split does not change y),
// scales and stores.
template <int NT, int OUT>
__global__ void __launch_bounds__(w8n::kThreads)
    gemm_w8a8_narrow_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                            GemmW8Args a) {
    using namespace w8n;
    constexpr int kPer = per(NT);
    constexpr int STAGE = stage_bytes(NT);
    constexpr uint32_t TCOLS = 2 * NT;   // two accumulators
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + (size_t)a.stages * STAGE);
    uint64_t* empty = full + kMaxStages;
    uint64_t* acc_full = empty + kMaxStages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
    float* s_sx = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(full) + kBarBytes);
    int* s_part = reinterpret_cast<int*>(s_sx + NT);   // [own token][source CTA][128 channels]
    __shared__ int s_failed;
    __shared__ int s_issued;

    const uint32_t warp = warp_id(), lane = lane_id();
    // the cluster is the whole x extent, a power of two
    const int split = (int)gridDim.x, rank = (int)blockIdx.x, log_split = 31 - __clz(split);
    const int n0 = (int)blockIdx.y * a.tile_n, m0 = (int)blockIdx.z * NT;
    const int c0 = (int)((int64_t)a.chunks * rank / split), c1 = (int)((int64_t)a.chunks * (rank + 1) / split);

    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(&full[s], kPer + 1);   // the loading warps that fill it
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 2);       // both MMA warps
        s_failed = 0;
        s_issued = 0;
        fence_barrier_init();
    }
    if (warp == kWarpW0 && lane == 0) prefetch_tensormap(&tm_w);
    if (warp == kWarpX && lane == 0) prefetch_tensormap(&tm_x);
    if (warp == kWarpMma0) {
        tmem_alloc(tmem_slot, TCOLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // Decode: the ring's worth of weights on its way into the L2 while the
    // previous kernel ends (only into the L2: that kernel may have written
    // them).  Quantizer and GEMM of one token: 20.5 -> 19.8 us at N = 10240,
    // K = 8192; with more tokens (37, N = 11008, K = 2080) 9.9 -> 10.7 us.
    if (NT == 16 && warp >= (uint32_t)kEpiWarp0 && lane == 0)
        for (int c = c0 + (int)warp - kEpiWarp0; c < min(c1, c0 + a.stages * kPer); c += kEpiWarps)
            tma_prefetch_l2_2d(&tm_w, c * BK, n0);
    griddep_wait();
    griddep_launch_dependents();
    if (split > 1) cluster_arrive();   // waited for before the first remote store: every CTA has started by then

    float sw = 0.0f, bias = 0.0f;
    using T = typename OutType<OUT>::type;
    const int q = (int)(warp & 3u), part = ((int)warp - kEpiWarp0) >> 2;   // an epilogue warp's lane quarter, its turn
    // an epilogue thread's output channel; lanes past the tile hold what the
    // tensor core made of stale shared memory
    const int n = 32 * q + (int)lane < a.tile_n ? n0 + 32 * q + (int)lane : a.N;
    const int tokens = min(NT, a.M - m0);
    // A stage is kPer chunks of the weight tile, then kPer of the token tile.
    if (warp <= kWarpX) {
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 1u;
            for (int c = c0, it = 0; c < c1; c += kPer, ++it) {
                // with one chunk per stage the weight warps take alternate
                // stages (always the same ones: the ring's length is even)
                const bool mine = kPer == 2 || warp == kWarpX || (it & 1) == (int)warp;
                if (mine && !bounded_wait(&empty[s], ph, kSiteW8NarrowEmpty)) {
                    s_failed = 1;
                    break;
                }
                uint8_t* dst = smem + (size_t)s * STAGE;
                if (warp == kWarpX) {
                    const bool both = kPer == 2 && c + 1 < c1;
                    mbar_arrive_expect_tx(&full[s], (uint32_t)(NT * BK) * (both ? 2u : 1u));
                    tma_load_2d(dst + kPer * W_BYTES, &tm_x, &full[s], c * BK, m0);
                    if (both) tma_load_2d(dst + kPer * W_BYTES + NT * BK, &tm_x, &full[s], (c + 1) * BK, m0);
                    s_issued = s_issued + 1;
                } else if (mine) {
                    const int k = kPer == 2 ? (int)warp : 0;   // the chunk of the stage
                    if (c + k < c1) {
                        mbar_arrive_expect_tx(&full[s], (uint32_t)(a.tile_n * BK));
                        tma_load_2d(dst + k * W_BYTES, &tm_w, &full[s], (c + k) * BK, n0);
                    } else {
                        mbar_arrive(&full[s]);   // a last stage of one chunk
                    }
                }
                if (++s == a.stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        __syncwarp();
        if (split > 1) cluster_wait();
    } else if (warp <= kWarpMma1) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_s8_s32(NT);
            const uint32_t smem0 = smem_u32(smem);
            const int me = (int)warp - kWarpMma0;
            const uint32_t acc = tmem + (uint32_t)(me * NT);
            bool ok = true;
            int s = me;
            uint32_t ph = 0u;
            for (int c = c0 + me * kPer; c < c1; c += 2 * kPer, s += 2) {
                for (; s >= a.stages; s -= a.stages) ph ^= 1u;
                if (!bounded_wait(&full[s], ph, kSiteW8NarrowFull)) {
                    s_failed = 1;
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sa = smem0 + (uint32_t)s * (uint32_t)STAGE;
                const uint64_t da = desc_sw128(sa), db = desc_sw128(sa + (uint32_t)(kPer * W_BYTES));
                constexpr uint64_t kNextW = W_BYTES >> 4, kNextX = (NT * BK) >> 4;   // descriptor units per chunk
                const uint32_t more = c > c0 + me * kPer ? 1u : 0u;
                const auto mma = [&](int j) {   // K-step j of the stage
                    mma_s8(acc, da + (uint64_t)(j >> 2) * kNextW + 2u * (j & 3),
                           db + (uint64_t)(j >> 2) * kNextX + 2u * (j & 3), idesc, j == 0 ? more : 1u);
                };
                const int here = min(kPer, c1 - c);
                if (here == kPer && (c + kPer < a.chunks || a.last_steps == 4)) {
#pragma unroll
                    for (int j = 0; j < 4 * kPer; ++j) mma(j);
                } else {   // a stage that is not full, or that ends K inside a chunk
                    const int n_steps = 4 * here - (c + here == a.chunks ? 4 - a.last_steps : 0);
                    for (int j = 0; j < n_steps; ++j) mma(j);
                }
                tc_commit(&empty[s]);
            }
            if (ok) tc_commit(acc_full);
        }
        __syncwarp();
        if (split > 1) cluster_wait();
    } else {
        const int t = (int)threadIdx.x - 32 * kEpiWarp0;
        for (int i = t; i < NT; i += 32 * kEpiWarps) s_sx[i] = i < tokens ? a.x_scales[m0 + i] : 0.0f;
        if (n < a.N) {
            sw = a.w_scales[n];
            bias = bias_at(a.bias, OUT, n);
        }
        named_bar_sync(1, 32 * kEpiWarps);   // the token scales are in shared memory
        if (split > 1) cluster_wait();
        if (!bounded_wait(acc_full, 0u, kSiteW8NarrowAcc)) s_failed = 1;
        tc_fence_after();
        __syncwarp();
        const uint32_t acc = tmem + ((32u * (uint32_t)q) << 16);
#pragma unroll 1
        for (int c = 16 * part; c < tokens; c += 32) {
            uint32_t v[16];
            tmem_ld_32x32b_x16(acc + (uint32_t)c, v);
            if (c1 - c0 > kPer) {   // the second MMA warp had stages too
                uint32_t u[16];
                tmem_ld_32x32b_x16(acc + (uint32_t)(NT + c), u);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] += u[i];
            }
            tmem_ld_wait();
            if (split == 1) {
                if (n < a.N) {
                    T* y = reinterpret_cast<T*>(a.y) + (int64_t)(m0 + c) * a.N + n;
                    T o[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        o[i] = OutType<OUT>::of(fmaf(__fmul_rn((float)(int)v[i], s_sx[c + i]), sw, bias));
                    if (c + 16 <= tokens) {
#pragma unroll
                        for (int i = 0; i < 16; ++i, y += a.N) *y = o[i];
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i, y += a.N)
                            if (c + i < tokens) *y = o[i];
                    }
                }
            } else {
                const uint32_t mine = smem_u32(s_part) + (uint32_t)(rank * BN + 32 * q + (int)lane) * 4u;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int tok = c + i;
                    if (tok < tokens)
                        st_cluster_s32(cluster_addr_u32(mine + (uint32_t)((tok >> log_split) << log_split) * BN * 4u,
                                                        (uint32_t)(tok & (split - 1))),
                                       (int)v[i]);
                }
            }
        }
    }
    __syncwarp();
    if (split > 1) {
        cluster_sync_all();   // every partial sum has arrived
        if (warp >= (uint32_t)kEpiWarp0 && n < a.N) {
            // own token j (token rank + j split of the tile): [j][source CTA][channel]
            const int* mine = s_part + 32 * q + (int)lane;
            T* y = reinterpret_cast<T*>(a.y) + (int64_t)(m0 + rank) * a.N + n;
            const int own = tokens > rank ? ((tokens - rank - 1) >> log_split) + 1 : 0;
#pragma unroll 2
            for (int j = part; j < own; j += 2) {
                int sum = 0;
#pragma unroll
                for (int r = 0; r < kMaxSplit; ++r)
                    if (r < split) sum += mine[((j << log_split) + r) * BN];
                y[(int64_t)(j << log_split) * a.N] =
                    OutType<OUT>::of(fmaf(__fmul_rn((float)sum, s_sx[rank + (j << log_split)]), sw, bias));
            }
        }
    }
    __syncthreads();
    if (s_failed && warp == 0 && lane == 0) {
        // after a timeout, let the loads already issued land (best effort: each wait is bounded)
        for (int s = 0; s < a.stages; ++s) {
            const int issued = *reinterpret_cast<volatile int*>(&s_issued);
            if (issued > s) bounded_wait(&full[s], (uint32_t)((issued - 1 - s) / a.stages) & 1u, kSiteW8NarrowDrain);
        }
    }
    __syncthreads();
    tc_fence_before();
    if (warp == kWarpMma0) {
        tc_fence_after();
        tmem_dealloc(tmem, TCOLS);
    }
}

}  // namespace svdq
