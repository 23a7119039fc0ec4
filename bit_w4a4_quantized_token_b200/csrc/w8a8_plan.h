// w8a8_plan.h -- arithmetic of the W8A8 kernels that needs no GPU: plain C++,
// shared by the kernels and their host side, and compiled alone by the tests.
#pragma once
#include <algorithm>
#include <cstdint>

#ifdef __CUDACC__
#define SVDQ_HD __host__ __device__
#else
#define SVDQ_HD
#endif

namespace svdq {

// The ring of the row quantizer.  A block takes rows first, first + step, ...;
// the copy of its i-th row goes to place i % stages, where it is phase
// i / stages of that place's barrier.  When the wait for `lost` has run out,
// the copies still in flight are those of the rows from lost on that were
// fetched, that is below `ahead` (the next row to fetch, or the number of rows).
// wait(place, parity) is called for each of them and for nothing else: a wait
// for another phase would return at once, or run out without a copy to wait for.
template <typename Wait>
SVDQ_HD inline void drain_ring(int first, int step, int lost, int ahead, int stages, Wait wait) {
    const int64_t begin = ((int64_t)lost - first) / step, end = ((int64_t)ahead - first + step - 1) / step;
    for (int64_t i = begin; i < end; ++i) wait((int)(i % stages), (uint32_t)(i / stages) & 1u);
}

// ------------------------------------------------------------------ the GEMM
constexpr int kW8SmemBudget = 224 * 1024;     // dynamic shared memory of a block, with room for its static one

namespace w8p {   // the CTA-pair kernel
constexpr int BM = 256;                       // tokens of a tile (128 per CTA)
constexpr int BN = 256;                       // output channels of a tile (128 weight rows loaded per CTA)
constexpr int BK = 128;                       // bytes of K of a chunk: the rows of a swizzled box
}  // namespace w8p

namespace w8n {   // the narrow kernel
constexpr int BN = 128;                       // output channels of a tile: the MMA's M
constexpr int BK = 128;
// Chunks of K per stage: two where the tokens add little to a stage's bytes
// (one barrier round trip for both), one where two would leave the ring with
// two stages.
SVDQ_HD constexpr int per(int nt) { return nt <= 64 ? 2 : 1; }
constexpr int W_BYTES = BN * BK;              // of one chunk
constexpr int kMaxStages = 8;
constexpr int kMaxSplit = 8;                  // CTAs of a cluster that share a tile's K range
constexpr int kBarBytes = 512;
SVDQ_HD constexpr int stage_bytes(int nt) { return per(nt) * (W_BYTES + nt * BK); }
// int32 partial sums that a CTA receives: for each of its tokens (every
// split-th of the tile) 128 channels from every CTA of the cluster
SVDQ_HD constexpr int partial_bytes(int nt, int split) {
    return split == 1 ? 0 : (nt + split - 1) / split * split * BN * 4;
}
// alignment slack, barriers, token scales, partial sums
SVDQ_HD constexpr int fixed_bytes(int nt, int split) { return 1024 + kBarBytes + nt * 4 + partial_bytes(nt, split); }
}  // namespace w8n

// What the plan depends on of a GPU: how many clusters of 1, 2, 4 and 8 of the
// narrow kernel's CTAs are resident at once, one CTA on an SM (148, 74, 33, 15
// on a B200 of 148 SMs: clusters of 4 and 8 leave SMs of a GPC unused).
struct W8Chip {
    int clusters[4];
};

// How svdq_gemm_w8a8 runs a shape.
struct W8Plan {
    bool pair;
    int nt, split, stages;   // narrow kernel: tokens of a tile, CTAs sharing its K range, ring depth
    int tile_n;              // and its output channels
};
// Stages of the narrow kernel's ring: as many as shared memory holds, one when
// a CTA has no more to do, else an even number, so that each place in the ring
// belongs to one of the two MMA warps (a warp must see every phase of a
// barrier that it waits on: parities repeat).
inline int w8_ring(int nt, int split, int64_t chunks) {
    const int64_t most = ((chunks + split - 1) / split + w8n::per(nt) - 1) / w8n::per(nt);
    const int64_t room = (kW8SmemBudget - w8n::fixed_bytes(nt, split)) / w8n::stage_bytes(nt);
    if (most == 1) return 1;
    return (int)(std::min<int64_t>({(int64_t)w8n::kMaxStages, room, most + 1}) / 2 * 2);
}
// Output channels of a narrow tile: as few as `tiles` tiles still cover N with
// (64 at least), so that every SM of the last wave has its share.  Tiles of 128
// against these, us: one token, N = 10240, K = 8192 (80 tiles; 143 of 72) 18.6,
// 16.8; N = 12288, K = 4096 11.9, 11.2; 24 tokens, N = 20480, K = 2560 16.5, 15.6.
inline int w8_tile_n(int64_t N, int64_t tiles) {
    const int64_t rows = ((N + tiles - 1) / tiles + 7) / 8 * 8;
    return (int)std::clamp<int64_t>(rows, 64, w8n::BN);
}
// The kernel and tile whose estimated time is least, in nanoseconds:
//   pair:   5950 + load(waves x 290 per chunk of 128 bytes of K)
//   narrow: 2650 + load(waves x chunks of a CTA x t) + (split: 1050 + 96 per token that a CTA finishes)
// with t = 150, 150, 224, 316 for tiles of 16, 32, 64, 128 tokens and load(x) =
// the larger of x and the weight's time from HBM (5.7 TB/s) plus a quarter of
// the smaller.  The constants are fitted to 500 timings at 74 shapes (1 to 2200
// tokens, N 1024 to 28672, K 1024 to 13824, weights from HBM), before narrower
// tiles and the limit on splits.  As it is now, every candidate timed at 170
// shapes (1 to 16384 tokens, N 8 to 28672, K 256 to 13824): the choice is the
// best one at 135, within 10 % of it at 154, 3.6 % slower on average.  The
// others are mostly of K <= 1040, where what the estimate leaves out is most of
// the time: the start and end of a narrow tile in each wave (1000 tokens, N =
// 2560, K = 1040: 128-token tiles 14.4 us, pairs 10.1) and the bytes of x and y
// (16384 tokens, N = K = 512: 19.3 and 12.0, the worst).  Examples of both
// sides: 256 tokens, N = K = 4096: 64-token tiles 9.7 us, pairs 15.7; 1000
// tokens: 128-token tiles 24.6, pairs 16.9; one token, N = K = 4096: split in
// four 6.5, not split 7.8.  mode: 0 both kernels, 1 the narrow one
// (where its grid holds the shape), 2 the pair kernel.
inline W8Plan w8_plan(int64_t M, int64_t N, int64_t K, const W8Chip& chip, int mode) {
    const int64_t chunks = (K + w8n::BK - 1) / w8n::BK;
    const int64_t weights_ns = N * K / 5700;
    const auto load = [&](int64_t x) { return std::max(x, weights_ns) + std::min(x, weights_ns) / 4; };
    W8Plan best = {true, 0, 0, 0, 0};
    int64_t best_ns = INT64_MAX;
    if (mode != 1) {
        const int64_t tiles = ((M + w8p::BM - 1) / w8p::BM) * ((N + w8p::BN - 1) / w8p::BN);
        const int64_t waves = (tiles + chip.clusters[1] - 1) / chip.clusters[1];
        best_ns = 5950 + load(waves * chunks * 290);
    }
    if (mode == 2) return best;
    constexpr int kNt[4] = {16, 32, 64, 128}, kChunkNs[4] = {150, 150, 224, 316};
    // CTAs of a split that are resident at once.  16 tokens, N = 2560, K =
    // 13824: 20 tiles split in four 11.2 us, in eight (160 CTAs) 14.8.
    int slots[4];
    for (int l = 0; l < 4; ++l) slots[l] = chip.clusters[l] << l;
    for (int i = 0; i < 4; ++i) {
        const int nt = kNt[i];
        const int64_t mt = (M + nt - 1) / nt, ntl = (N + w8n::BN - 1) / w8n::BN;
        if (mt > 65535 || ntl > 65535) continue;   // the grid's limits
        for (int l = 0; l < 4 && (1 << l) <= chunks; ++l) {
            const int64_t ctas = (mt * ntl) << l, waves = (ctas + slots[l] - 1) / slots[l];
            if (l > 0 && waves > 1) break;   // a second wave of clusters costs more than a split saves
            const int64_t of_cta = (chunks + (1 << l) - 1) >> l;
            int64_t ns = 2650 + load(waves * of_cta * kChunkNs[i]);
            if (l > 0) ns += 1050 + 96 * ((std::min<int64_t>(M, nt) + (1 << l) - 1) >> l);
            if (ns < best_ns) {
                best_ns = ns;
                const int64_t tiles = std::min<int64_t>(waves * slots[l] / (mt << l), 65535);
                best = {false, nt, 1 << l, w8_ring(nt, 1 << l, chunks), w8_tile_n(N, tiles)};
            }
        }
    }
    return best;
}

}  // namespace svdq
