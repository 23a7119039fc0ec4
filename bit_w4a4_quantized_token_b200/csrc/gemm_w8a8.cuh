// gemm_w8a8.cuh -- the 8-bit integer GEMM of the W8A8 linear layer (sm_100a):
//     y[m, n] = round( float(sum_k qx[m, k] qw[n, k]) sx[m] sw[n] + b[n] )
// with signed 8-bit codes, one fp32 scale per token and per output channel,
// and the sum exact in int32 (K < 2^17, so that even codes of -128 cannot
// overflow it).  The scales are common to whole rows and columns of the
// product, so they stay out of the main loop: tcgen05.mma kind::i8 multiplies
// the codes as they lie in memory (K-major rows, 128-byte swizzled TMA boxes)
// and the epilogue scales once per output.
//
// Two kernels compute it:
//  * gemm_w8a8_pair_kernel: 256 x 256 output tiles on two-CTA clusters, for
//    problems that fill the chip with such tiles;
//  * gemm_w8a8_narrow_kernel: 128 output channels x 16..256 tokens on single
//    CTAs with the K range split over a cluster, for few tokens or few tiles.
#pragma once
#include "gelu_mlp.cuh"        // st_shared_v4
#include "quantize_w8a8.cuh"   // the element types, pack2

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
    int stages;              // narrow kernel: ring depth
    int out;                 // type of y and bias: kBf16, kF16 or kF32
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
    kSiteW8Empty = 40,
    kSiteW8Full = 41,
    kSiteW8Acc = 42,
    kSiteW8AccEmpty = 43,
    kSiteW8Drain = 44,
    kSiteW8NarrowEmpty = 45,
    kSiteW8NarrowFull = 46,
    kSiteW8NarrowAcc = 47,
    kSiteW8NarrowDrain = 48
};

// ------------------------------------------------------------ CTA-pair kernel
namespace w8p {
constexpr int BM = 256;                       // tokens of a tile (128 per CTA)
constexpr int BN = 256;                       // output channels of a tile (128 weight rows loaded per CTA)
constexpr int BK = 128;                       // bytes of K per stage
constexpr int kStages = 6;
constexpr int A_BYTES = 128 * BK;
constexpr int B_BYTES = 128 * BK;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
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
constexpr int kGroupM = 8;                    // row tiles that are walked together (below)
}  // namespace w8p

// Tile of a running index: groups of kGroupM row tiles, the row tile fastest,
// so that the ~74 tiles in flight form a block of about 8 x 9 and share their
// operands in the L2 (a row-major walk keeps 74 different weight tiles in
// flight and re-reads the whole weight for every row tile).
__device__ __forceinline__ void w8_tile(int id, int m_tiles, int n_tiles, int& m, int& n) {
    const int per_group = w8p::kGroupM * n_tiles;
    const int g = id / per_group, in = id - g * per_group;
    const int gm = min(w8p::kGroupM, m_tiles - g * w8p::kGroupM);
    n = in / gm;
    m = g * w8p::kGroupM + (in - n * gm);
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
    griddep_wait();   // everything above overlaps the end of the previous kernel

    if (warp == kWarpX || warp == kWarpW) {
        // ---------------------------------------------------------- producers
        // Each CTA loads its own 128 token rows and 128 weight rows of every
        // stage; all loads complete on CTA 0's barrier.
        if (lane == 0) {
            const bool is_x = warp == kWarpX;
            const CUtensorMap* map = is_x ? &tm_x : &tm_w;
            int it = 0;
            bool ok = true;
            for (int id = cluster; id < total && ok; id += n_clusters) {
                int m, n;
                w8_tile(id, a.m_tiles, a.n_tiles, m, n);
                const int row0 = (is_x ? m * BM : n * BN) + 128 * (int)rank;
                for (int c = 0; c < a.chunks; ++c, ++it) {
                    const int s = it % kStages;
                    if (!mbar_wait(&empty[s], ((uint32_t)(it / kStages) & 1u) ^ 1u, kSiteW8Empty)) {
                        s_failed = 1;
                        ok = false;
                        break;
                    }
                    uint8_t* dst = smem + (size_t)s * STAGE_BYTES + (is_x ? 0 : A_BYTES);
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2u * A_BYTES);
                    tma_load_2d_pair(dst, map, cluster_addr(&full[s], 0), c * BK, row0);
                    if (is_x) s_issued[s] = s_issued[s] + 1;
                }
            }
        }
    } else if (warp == kWarpMma) {
        // ------------------------------------------------- MMAs (CTA 0 only)
        if (rank == 0 && lane == 0) {
            const uint32_t idesc = idesc_m(idesc_s8_s32(BN), BM);
            const uint32_t smem0 = smem_u32(smem);
            int it = 0, local = 0;
            bool ok = true;
            for (int id = cluster; id < total && ok; id += n_clusters, ++local) {
                const uint32_t acc = tmem + (uint32_t)(local & 1) * ACC_COLS;
                if (!mbar_wait(&acc_empty[local & 1], ((uint32_t)(local >> 1) & 1u) ^ 1u, kSiteW8AccEmpty)) {
                    s_failed = 1;
                    break;
                }
                for (int c = 0; c < a.chunks; ++c, ++it) {
                    const int s = it % kStages;
                    if (!mbar_wait(&full[s], (uint32_t)(it / kStages) & 1u, kSiteW8Full)) {
                        s_failed = 1;
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem0 + (uint32_t)s * STAGE_BYTES;
                    const uint64_t da = desc_sw128(sa), db = desc_sw128(sa + A_BYTES);   // + 2 per 32-byte K-step
                    const int steps = c + 1 < a.chunks ? 4 : a.last_steps;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < steps) mma_s8_pair(acc, da + 2u * j, db + 2u * j, idesc, (c > 0 || j > 0) ? 1u : 0u);
                    tc_commit_pair(&empty[s], 0x3);
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
        const uint32_t box = smem_u32(smem + BOX_OFF) + e * (uint32_t)kBoxBytes;
        constexpr int kBoxCols = OUT == kF32 ? 16 : 32;
        int local = 0;
        for (int id = cluster; id < total; id += n_clusters, ++local) {
            int mt, nt;
            w8_tile(id, a.m_tiles, a.n_tiles, mt, nt);
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
            if (!mbar_wait(&acc_full[local & 1], (uint32_t)(local >> 1) & 1u, kSiteW8Acc)) {
                s_failed = 1;
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + ((32u * q) << 16) + (uint32_t)(local & 1) * ACC_COLS + 128u * (uint32_t)half;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(acc + 32u * c, v);
                tmem_ld_wait();
                if (c == 3) {   // drained: the accumulator may be overwritten
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(cluster_addr(&acc_empty[local & 1], 0));
                }
                if (n0 + 32 * c >= a.N) continue;   // warp-uniform
                float o[32];
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 s4 = *reinterpret_cast<const float4*>(col_s + 32 * c + i);
                    const float4 b4 = *reinterpret_cast<const float4*>(col_b + 32 * c + i);
                    float f0 = (float)(int)v[i], f1 = (float)(int)v[i + 1];
                    float f2 = (float)(int)v[i + 2], f3 = (float)(int)v[i + 3];
                    fmul2_rn(f0, f1, sx, sx, f0, f1);
                    fmul2_rn(f2, f3, sx, sx, f2, f3);
                    ffma2_rn(f0, f1, s4.x, s4.y, b4.x, b4.y, o[i], o[i + 1]);
                    ffma2_rn(f2, f3, s4.z, s4.w, b4.z, b4.w, o[i + 2], o[i + 3]);
                }
#pragma unroll
                for (int p = 0; p < 32 / kBoxCols; ++p) {
                    // 32 rows x 64 bytes through the warp's box (64-byte swizzle), stored with TMA
                    if (lane == 0) bulk_wait_group_read<0>();
                    __syncwarp();
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
            if (n > 0) mbar_wait(&full[s], (uint32_t)(n - 1) & 1u, kSiteW8Drain);
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
constexpr int BN = 128;                       // output channels of a tile: the MMA's M
constexpr int BK = 128;
constexpr int W_BYTES = BN * BK;
constexpr int kMaxStages = 16;
constexpr int kMaxSplit = 8;                  // CTAs of a cluster that share a tile's K range
constexpr int kThreads = 192;                 // warp 0: loads, warp 1: MMAs, warps 2..5: epilogue
constexpr int kBarBytes = 512;
static_assert((2 * kMaxStages + 1) * 8 + 4 <= kBarBytes, "barriers do not fit");
__host__ __device__ constexpr int stage_bytes(int nt) { return W_BYTES + nt * BK; }
// barriers, token scales, alignment slack
__host__ __device__ constexpr int fixed_bytes(int nt) { return 1024 + kBarBytes + nt * 4; }
// int32 partial sums of a tile, kept in the ring once it has been drained
__host__ __device__ constexpr int partial_bytes(int nt) { return BN * nt * 4; }
}  // namespace w8n

__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void store_out(void* y, int out, int64_t i, float v) {
    if (out == kF32)
        reinterpret_cast<float*>(y)[i] = v;
    else if (out == kF16)
        reinterpret_cast<__half*>(y)[i] = __float2half_rn(v);
    else
        reinterpret_cast<__nv_bfloat16*>(y)[i] = __float2bfloat16_rn(v);
}

// The product transposed: the MMA's A operand (M = 128) holds weight rows, its
// B operand NT token rows, so that few tokens cost few tensor-core columns and
// few bytes of TMEM, and the weight streams through a ring as deep as shared
// memory allows.  The cluster's CTAs split the K range; their int32 partial
// sums meet in shared memory (exact, so the split does not change y), and each
// CTA finishes a share of the tile's tokens.
template <int NT>
__global__ void __launch_bounds__(w8n::kThreads)
    gemm_w8a8_narrow_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                            GemmW8Args a) {
    using namespace w8n;
    constexpr int STAGE = stage_bytes(NT);
    constexpr uint32_t TCOLS = NT < 32 ? 32 : NT;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + (size_t)a.stages * STAGE);
    uint64_t* empty = full + kMaxStages;
    uint64_t* acc_full = empty + kMaxStages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
    float* s_sx = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(full) + kBarBytes);
    int* s_part = reinterpret_cast<int*>(smem);
    __shared__ int s_failed;
    __shared__ int s_issued;

    const uint32_t warp = warp_id(), lane = lane_id();
    const int split = (int)gridDim.x, rank = (int)blockIdx.x;   // the cluster is the whole x extent
    const int n0 = (int)blockIdx.y * BN, m0 = (int)blockIdx.z * NT;
    const int c0 = (int)((int64_t)a.chunks * rank / split), c1 = (int)((int64_t)a.chunks * (rank + 1) / split);

    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        s_failed = 0;
        s_issued = 0;
        fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&tm_x);
        prefetch_tensormap(&tm_w);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, TCOLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();

    float sw = 0.0f, bias = 0.0f;
    const int q = (int)(warp & 3u);
    const int n = n0 + 32 * q + (int)lane;   // an epilogue thread's output channel
    if (warp == 0) {
        if (lane == 0) {
            for (int c = c0; c < c1; ++c) {
                const int it = c - c0, s = it % a.stages;
                if (!mbar_wait(&empty[s], ((uint32_t)(it / a.stages) & 1u) ^ 1u, kSiteW8NarrowEmpty)) {
                    s_failed = 1;
                    break;
                }
                uint8_t* dst = smem + (size_t)s * STAGE;
                mbar_arrive_expect_tx(&full[s], (uint32_t)STAGE);
                tma_load_2d(dst, &tm_w, &full[s], c * BK, n0);
                tma_load_2d(dst + W_BYTES, &tm_x, &full[s], c * BK, m0);
                s_issued = it + 1;
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_s8_s32(NT);
            const uint32_t smem0 = smem_u32(smem);
            bool ok = true;
            for (int c = c0; c < c1; ++c) {
                const int it = c - c0, s = it % a.stages;
                if (!mbar_wait(&full[s], (uint32_t)(it / a.stages) & 1u, kSiteW8NarrowFull)) {
                    s_failed = 1;
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sa = smem0 + (uint32_t)s * (uint32_t)STAGE;
                const uint64_t da = desc_sw128(sa), db = desc_sw128(sa + W_BYTES);
                const int steps = c + 1 < a.chunks ? 4 : a.last_steps;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < steps) mma_s8(tmem, da + 2u * j, db + 2u * j, idesc, (it > 0 || j > 0) ? 1u : 0u);
                tc_commit(&empty[s]);
            }
            if (ok) tc_commit(acc_full);
        }
    } else {
        const int t = (int)threadIdx.x - 64;
        for (int i = t; i < NT; i += 128) s_sx[i] = m0 + i < a.M ? a.x_scales[m0 + i] : 0.0f;
        if (n < a.N) {
            sw = a.w_scales[n];
            bias = bias_at(a.bias, a.out, n);
        }
        named_bar_sync(1, 128);   // the token scales are in shared memory
        if (!mbar_wait(acc_full, 0u, kSiteW8NarrowAcc)) s_failed = 1;
        tc_fence_after();
        const uint32_t acc = tmem + ((32u * (uint32_t)q) << 16);
        if (split == 1) {
            if (!*reinterpret_cast<volatile int*>(&s_failed)) {
#pragma unroll 1
                for (int c = 0; c < NT; c += 16) {
                    if (m0 + c >= a.M) break;
                    uint32_t v[16];
                    __syncwarp();
                    tmem_ld_32x32b_x16(acc + (uint32_t)c, v);
                    tmem_ld_wait();
                    if (n < a.N) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (m0 + c + i < a.M)
                                store_out(a.y, a.out, (int64_t)(m0 + c + i) * a.N + n,
                                          fmaf(__fmul_rn((float)(int)v[i], s_sx[c + i]), sw, bias));
                    }
                }
            }
        } else {
            // the ring is drained: every load has been consumed by an MMA that acc_full waited for
#pragma unroll 1
            for (int c = 0; c < NT; c += 16) {
                if (m0 + c >= a.M) break;
                uint32_t v[16];
                __syncwarp();
                tmem_ld_32x32b_x16(acc + (uint32_t)c, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) s_part[(c + i) * BN + 32 * q + (int)lane] = (int)v[i];
            }
        }
    }
    __syncwarp();
    if (split > 1) {
        cluster_sync_all();   // every CTA's partial sums are in its shared memory
        if (warp >= 2 && n < a.N) {
            const int tokens = min(NT, a.M - m0);
            const uint32_t mine = (uint32_t)(32 * q + (int)lane) * 4u;
            for (int i = rank; i < tokens; i += split) {
                int sum = 0;
                for (int r = 0; r < split; ++r)
                    sum += ld_cluster_s32(cluster_addr(s_part, (uint32_t)r) + (uint32_t)(i * BN) * 4u + mine);
                store_out(a.y, a.out, (int64_t)(m0 + i) * a.N + n, fmaf(__fmul_rn((float)sum, s_sx[i]), sw, bias));
            }
        }
        __syncwarp();
        cluster_sync_all();   // no CTA's partial sums go away while another reads them
    }
    __syncthreads();
    if (s_failed && warp == 0 && lane == 0) {
        // after a timeout, let the loads already issued land (best effort: each wait is bounded)
        for (int s = 0; s < a.stages; ++s) {
            const int issued = *reinterpret_cast<volatile int*>(&s_issued);
            if (issued > s) mbar_wait(&full[s], (uint32_t)((issued - 1 - s) / a.stages) & 1u, kSiteW8NarrowDrain);
        }
    }
    __syncthreads();
    tc_fence_before();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TCOLS);
    }
}

}  // namespace svdq
