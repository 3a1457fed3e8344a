// gemm_fp4.cu -- products of MXFP4 operands with BF16 output: dense, the experts' products, their weight gradients.
//
//   y[m, n] = sum_k (qa[m, k] 2^ea[m, k/32]) (qb[n, k] 2^eb[n, k/32])
//
// tcgen05.mma.kind::mxf4.block_scale: packed E2M1 operands from shared memory, two E8M0 scales a row and
// instruction from tensor memory, 64 K elements an instruction, FP32 accumulators in tensor memory.  A pipeline stage is
// 256 K elements: 128 bytes of payload and two 512-byte scale atoms for 128 rows of an operand.
//
// Two kernels.  gemm_mxfp4_pair_kernel: 256 x 256 tiles on CTA pairs, for products that fill the device with such
// tiles.  gemm_mxfp4_rows_kernel: 128 columns of B by up to 128 rows of A on a single CTA, B in the place of the
// instruction's 128-row operand, so that few rows of A cost few instructions; K split over a cluster where
// there are few tiles.  Every mbarrier wait is bounded (see mxq_device.cuh).

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "mxq_elem.cuh"
#include "mxq_internal.h"

namespace mxq {
namespace {

constexpr int kBK = 256;              // K elements of a stage (128 bytes of payload)
constexpr int kBandBytes = 128 * 128; // payload of 128 rows of a stage
constexpr int kAtom = 512;            // scales of 128 rows and 4 groups
constexpr int kMaxExperts = 1024;

struct Args {
    const uint8_t *a_s, *b_s;
    uint16_t* y;
    int64_t M, N, ldy;
    int64_t k_atoms;           // scale atoms of a 128-row band
    int64_t k_padded;          // K up to a multiple of 32
    int m_tiles, n_tiles;      // dense
    int items;                 // grouped: work items of a launch at most
    int64_t b_bands;           // 128-row bands of an expert's (of B's) scales
    const int64_t* offsets;    // grouped: [G + 1] on the device
    int64_t offset_limit;      // rows that they may point to
    int G;
    int64_t bands_cap;         // grouped: bands of A's scales
    int y_tma, y_vec;          // the output has a map; its rows hold whole vectors (16 bytes, rows kernel 8)
    int tok_cap, stages, split, log_split, chunked;   // rows kernel: rows of A in a slot, slots, CTAs along K, see RowsMaps
    unsigned int* status;
    uint64_t wait_limit_ns;
};

// Offset g, inside [0, offset_limit] whatever it holds.
__device__ __forceinline__ int64_t offset_at(const Args& p, int g) {
    const int64_t o = p.offsets[g];
    return o < 0 ? int64_t(0) : (o > p.offset_limit ? p.offset_limit : o);
}

// A wait by one lane, its verdict as a vote: the compiler sees that a vote is the same in all lanes, so that the loops of
// the issuing warps keep counters, addresses and descriptors in uniform registers, where the
// instructions want them.
template <typename Wait>
__device__ __forceinline__ bool warp_waits(int lane, Wait wait) {
    return __all_sync(0xFFFFFFFFu, lane != 0 || wait()) != 0;
}

// First 128-row band of expert g's scales; its bands end before the next expert's.
__device__ __forceinline__ int64_t first_band(int64_t first_row, int g) { return first_row / 128 + g; }

// Grouped: prefix[g] = work items of the experts before g; `rows` rows of A an item.  All threads of the block.
// Sums stop at p.items, which offsets that keep the rule never pass.  Others may have one row in the ranges of many experts:
// their items past that are left out, or the sums would leave 32 bits and a cluster of a split product meet a second tile.
__device__ __forceinline__ void build_prefix(const Args& p, int rows, int* prefix) {
    const uint32_t most = static_cast<uint32_t>(p.items);   // below 2^31: the sum of two of them fits
    for (int g = threadIdx.x; g < p.G; g += blockDim.x) {
        const int64_t lo = offset_at(p, g), hi = offset_at(p, g + 1);
        int64_t n = hi > lo ? (hi - lo + rows - 1) / rows : 0;
        if (first_band(lo, g) + (hi - lo + 127) / 128 > p.bands_cap) n = 0;   // offsets that break the rule
        prefix[g + 1] = static_cast<int>(min(n * p.n_tiles, static_cast<int64_t>(most)));
    }
    if (threadIdx.x == 0) prefix[0] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {
        uint32_t carry = 0;
        for (int base = 0; base < p.G; base += 32) {
            const int g = base + static_cast<int>(threadIdx.x);
            uint32_t v = g < p.G ? static_cast<uint32_t>(prefix[g + 1]) : 0u;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const uint32_t up = __shfl_up_sync(0xFFFFFFFFu, v, d);
                if (static_cast<int>(threadIdx.x) >= d) v = min(v + up, most);
            }
            if (g < p.G) prefix[g + 1] = static_cast<int>(min(carry + v, most));
            carry = min(carry + __shfl_sync(0xFFFFFFFFu, v, 31), most);
        }
    }
    __syncthreads();
}

// The expert of item t.
__device__ __forceinline__ int expert_of(const int* prefix, int G, int t) {
    int lo = 0, hi = G;   // the last g with prefix[g] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// Instructions (64 K elements each) that block kb of `block` K elements needs.
template <int kBlock>
__device__ __forceinline__ int mmas_of(int64_t k_padded, int64_t kb) {
    const int64_t left = k_padded - kb * kBlock;
    return left >= kBlock ? kBlock / 64 : static_cast<int>((left + 63) / 64);
}

// ---- CTA pairs -------------------------------------------------------------------------------
//
// Output tiles of 256 x 256 per pair of SMs (cta_group::2).  CTA r of the pair loads 128 rows of A, its 128-row half
// of B, its two A scale atoms, and multicasts the two scale atoms of its half of B to both (each tensor
// core needs the scales of all 256 B rows).  One thread of the even CTA issues, per stage, six scale copies and four
// 256 x 256 x 64 instructions of 128 cycles each; it asks for the next stage's bytes before them and reads the answer
// behind them.
//
// Measured: 16384^3 1160 us (7.58 PFLOP/s), 16384 x 7168 x 7168 223 us, 8192 x 4096 x 4096 45 us, 2048 x 4096 x 4096
// 16.8 us; experts' products of 131072 rows (128 experts of 4096 x 4096, unequal loads) 746 us, their weight gradients
// 1248 us.
//
// What bounds it: a stage takes about 660 cycles (1.9 GHz) instead of the 512 of its instructions.  With five stages
// it took 690 (16384^3: 1256 us; 8192 x 4096 x 4096: 48.4 us); there the same kernel without the operands' loads
// took 984 us, without the instructions 1004 us (35 KB a stage and SM, 64 bytes a cycle), without the scale copies
// 1207 us: loads and instructions meet in shared memory, and bytes in flight are part of it.  Tried without gain, with five
// stages: scale copies by a second warp (1490 us), scale copies a stage ahead (1278 us), clusters of two pairs that
// share B's loads (1280 to 1380 us; 8192 x 4096 x 4096 47.4 us against 47.7 us); with six: operands and scales
// loaded by two warps (1225 us).
//
// Tensor memory (512 columns): two accumulators of 256 columns, at 0 and 96, that share 160 of them, and a slot of 24
// columns of scales for each stage.  The epilogue of a tile reads the shared columns first and hands them back,
// so the next tile's instructions wait for these only.
struct PairCfg {
    static constexpr int kStages = 6;
    static constexpr int kEpiWarps = 8;
    static constexpr int kThreads = 64 + 32 * kEpiWarps;
    static constexpr int kSfaBytes = 2 * kAtom, kSfbBytes = 4 * kAtom;
    static constexpr int kStageBytes = 2 * kBandBytes + kSfaBytes + kSfbBytes;
    static constexpr int kOffB = 0;
    static constexpr int kOffA = kOffB + kStages * kBandBytes;
    static constexpr int kOffSfa = kOffA + kStages * kBandBytes;
    static constexpr int kOffSfb = kOffSfa + kStages * kSfaBytes;
    static constexpr int kOffStage = kOffSfb + kStages * kSfbBytes;   // 1024-byte aligned
    static constexpr int kStageWarpBytes = 32 * 16 * 2;               // a BF16 chunk of 32 rows
    static constexpr int kOffBar = kOffStage + kEpiWarps * kStageWarpBytes;
    static constexpr int kNumBars = 2 * kStages + 3;   // full, empty, accumulator full / handed back, drain
    static constexpr int kOffTmemSlot = kOffBar + 8 * kNumBars;
    static constexpr int kOffAbort = kOffTmemSlot + 4;
    static constexpr int kOffPrefix = kOffAbort + 4;
    static constexpr int kBytes = kOffPrefix + 4 * (kMaxExperts + 1);
    static constexpr int kAlloc = kBytes + 1024;
    static constexpr int kTmemCols = 512;
    static constexpr int kAcc1 = 96;                  // second accumulator
    static constexpr int kShared = 256 - kAcc1;       // columns of both
    static constexpr int kTmemScales = kAcc1 + 256, kScaleCols = 24;
    static_assert(kTmemScales + kScaleCols * kStages <= kTmemCols, "tensor memory budget");
    static_assert(kShared % 32 == 0, "chunks of 16 columns of two halves");
    static_assert(kAlloc <= 227 * 1024, "shared memory budget");
    static_assert(kOffStage % 1024 == 0, "swizzle atoms");
};

struct PairMaps {
    CUtensorMap a, b, sfa, sfb, y;
};

// What a launch computes: one product; the experts' products, their rows of A by offsets; the experts' weight gradients,
// the contraction by offsets and a full grid of tiles each.
constexpr int kDense = 0, kExperts = 1, kGradients = 2;

struct PairTile {
    int64_t m0;              // this CTA's first A row (may lie past the matrix)
    int64_t a_band;          // its A scale band
    int64_t y_row;           // the output row of m0
    int64_t row_lo, row_hi;  // output rows that are stored (empty: none)
    int64_t n0;              // first output column
    int64_t b_row, b_band;   // first B row of the pair's tile and its scale band
    int k_atom;              // where the contraction starts, in 128 K elements
    int num_kb;              // its K blocks (0: the tile is zero) and K elements
    int64_t k_padded;
};

template <int kMode>
__device__ __forceinline__ PairTile pair_tile(const Args& p, const int* prefix, int t, uint32_t rank) {
    PairTile ti;
    ti.k_atom = 0;
    ti.k_padded = p.k_padded;
    if constexpr (kMode != kExperts) {
        int g = 0;
        if constexpr (kMode == kGradients) {
            const int per = p.m_tiles * p.n_tiles;
            g = t / per;
            t -= g * per;
            const int64_t lo = offset_at(p, g), hi = offset_at(p, g + 1);
            ti.k_atom = static_cast<int>(first_band(lo, g));
            ti.k_padded = hi > lo && ti.k_atom + (hi - lo + 127) / 128 <= p.k_atoms ? (hi - lo + 31) / 32 * 32 : 0;
        }
        constexpr int kBand = 4;   // raster: bands of 1024 rows, columns inside a band
        const int per_band = kBand * p.n_tiles, band = t / per_band, within = t - band * per_band;
        const int height = min(kBand, p.m_tiles - band * kBand), n = within / height;
        ti.m0 = static_cast<int64_t>(band * kBand + within - n * height) * 256 + 128 * rank;
        ti.n0 = static_cast<int64_t>(n) * 256;
        ti.a_band = ti.m0 / 128;
        ti.y_row = ti.row_lo = g * p.M + ti.m0;
        ti.row_hi = g * p.M + min(ti.m0 + 128, p.M);
        ti.b_row = ti.n0;
        ti.b_band = ti.n0 / 128;
    } else {
        const int g = expert_of(prefix, p.G, t);
        const int64_t lo = offset_at(p, g), hi = offset_at(p, g + 1);
        const int local = t - prefix[g], row = local / p.n_tiles;
        ti.n0 = static_cast<int64_t>(local - row * p.n_tiles) * 256;
        const int64_t i = 2 * static_cast<int64_t>(row) + rank;
        const bool any = lo + 128 * i < hi;   // an odd number of row tiles leaves the last odd CTA without rows
        ti.m0 = any ? lo + 128 * i : lo;
        ti.a_band = first_band(lo, g) + (any ? i : 0);
        ti.y_row = ti.row_lo = ti.m0;
        ti.row_hi = any ? min(ti.m0 + 128, hi) : ti.m0;
        ti.b_row = static_cast<int64_t>(g) * p.N + ti.n0;
        ti.b_band = static_cast<int64_t>(g) * p.b_bands + ti.n0 / 128;
    }
    ti.num_kb = static_cast<int>((ti.k_padded + kBK - 1) / kBK);
    return ti;
}

// 32 x 16 results of a warp (lane l: output row row0 + l, columns n .. n + 15) through its staging buffer of 1 KB: 16-byte
// chunk j of row r sits at position j ^ ((r >> 2) & 1), the 32-byte swizzle of a tiled bulk copy.  Rows that are all
// stored leave with one such copy; otherwise by rows, in vectors or, where rows start
// anywhere, in words on the memory's 4-byte grid: where that starts at a row's second column, the row's words hold the
// columns -1 and 0, 1 and 2, ..; column -1 is the last one of the chunk before (*carry).  Single columns are left at the
// ends of a run of chunks (start, last) only: a store of one column of 32 rows costs as much as four of words
// (15143 x 3615 x 77: 71 us with such ends at every chunk, 46 us).  The buffer is small so that the ring is large.
template <bool kAny>
__device__ __forceinline__ void store_chunk(const Args& p, const uint32_t* v, uint32_t stage, int64_t row0, int64_t row_lo,
                                            int64_t row_hi, int64_t n, int lane, const CUtensorMap* map, bool start, bool last,
                                            uint32_t* carry) {
    if (n >= p.N) return;
    // not across N: the copy leaves out columns past it by 16 bytes only, and what follows them in a row is the caller's
    const bool tiled = !kAny && p.y_tma && row0 >= row_lo && row0 + 32 <= row_hi && n + 16 <= p.N;
    uint4 o[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        o[j].x = cvt_bf16x2(__uint_as_float(v[8 * j + 0]), __uint_as_float(v[8 * j + 1]));
        o[j].y = cvt_bf16x2(__uint_as_float(v[8 * j + 2]), __uint_as_float(v[8 * j + 3]));
        o[j].z = cvt_bf16x2(__uint_as_float(v[8 * j + 4]), __uint_as_float(v[8 * j + 5]));
        o[j].w = cvt_bf16x2(__uint_as_float(v[8 * j + 6]), __uint_as_float(v[8 * j + 7]));
    }
    uint16_t* to = p.y + row0 * p.ldy + n;
    const int first = static_cast<int>(reinterpret_cast<uintptr_t>(to) >> 1) & 1, step = static_cast<int>(p.ldy & 1);
    const int odd = kAny ? first ^ (step & lane) : 0;   // of this lane's row
    const uint32_t column0 = o[0].x, before = *carry;
    *carry = o[1].w >> 16;
    if (kAny && odd) {
        const uint32_t w[8] = {o[0].x, o[0].y, o[0].z, o[0].w, o[1].x, o[1].y, o[1].z, o[1].w};
        o[0] = make_uint4(before | (w[0] << 16), __funnelshift_r(w[0], w[1], 16), __funnelshift_r(w[1], w[2], 16), __funnelshift_r(w[2], w[3], 16));
        o[1] = make_uint4(__funnelshift_r(w[3], w[4], 16), __funnelshift_r(w[4], w[5], 16), __funnelshift_r(w[5], w[6], 16),
                          __funnelshift_r(w[6], w[7], 16));
    }
    if (lane == 0) bulk_wait_read_all();   // the copy before has read the buffer
    __syncwarp();
    const uint32_t swz = static_cast<uint32_t>((lane >> 2) & 1);
#pragma unroll
    for (int j = 0; j < 2; ++j) sts128(stage + 32u * static_cast<uint32_t>(lane) + 16u * (static_cast<uint32_t>(j) ^ swz), o[j]);
    if (tiled) {
        fence_proxy_async_smem();   // the buffer is read by the bulk copy (async proxy)
        __syncwarp();
        if (lane == 0) {
            tma_store_2d(map, static_cast<int32_t>(n), static_cast<int32_t>(row0), stage);
            bulk_commit_group();
        }
        return;
    }
    __syncwarp();
    const int lo = static_cast<int>(max(row_lo - row0, int64_t(0))), hi = static_cast<int>(min(row_hi - row0, int64_t(32)));
    const int cols = static_cast<int>(min(p.N - n, int64_t(16)));
    if constexpr (!kAny) {
        const int jj = lane & 1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 16 * i + (lane >> 1);
            const uint4 x = lds128_ordered(stage + 32u * static_cast<uint32_t>(r) + 16u * static_cast<uint32_t>(jj ^ ((r >> 2) & 1)));
            if (r < lo || r >= hi) continue;
            uint16_t* at = to + r * p.ldy + 8 * jj;
            if (8 * jj + 8 <= cols) {
                *reinterpret_cast<uint4*>(at) = x;
            } else {
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                for (int c = 0; c < 8 && 8 * jj + c < cols; ++c) at[c] = static_cast<uint16_t>(w[c >> 1] >> (16 * (c & 1)));
            }
        }
    } else {
        auto word = [&](int r, int w) {
            return lds32(stage + 32u * static_cast<uint32_t>(r) + 16u * static_cast<uint32_t>((w >> 2) ^ ((r >> 2) & 1)) +
                         4u * static_cast<uint32_t>(w & 3));
        };
        const int w = lane & 7;
#pragma unroll
        for (int i = 0; i < 8; ++i) {   // four rows at a time
            const int r = 4 * i + (lane >> 3), at = 2 * w - (first ^ (step & r));   // the word's first column
            const uint32_t x = word(r, w);
            if (r >= lo && r < hi && at + 2 <= cols && (at >= 0 || !start)) *reinterpret_cast<uint32_t*>(to + r * p.ldy + at) = x;
        }
        if (lane >= lo && lane < hi) {
            uint16_t* row = to + lane * p.ldy;
            if (odd && start) row[0] = static_cast<uint16_t>(column0);
            // the last column where it has no partner: the first one of a word, or of the one behind the last
            if (last && ((cols - odd) & 1))
                row[cols - 1] = static_cast<uint16_t>(cols == 16 ? *carry : word(lane, cols >> 1));
        }
    }
    __syncwarp();
}

// kAny: output rows that do not start on 16 bytes.
template <int kMode, bool kAny>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PairCfg::kThreads, 1)
    gemm_mxfp4_pair_kernel(const __grid_constant__ PairMaps maps, const Args p) {
    using L = PairCfg;
    constexpr int STAGES = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = blockIdx.x & 1u;
    const bool leader = rank == 0;
    const uint32_t bar0 = sbase + L::kOffBar;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    const uint32_t tfull_bar = bar0 + 8u * (2 * STAGES), tempty_bar = tfull_bar + 8u, drain_bar = tfull_bar + 16u;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffAbort);
    int* prefix = reinterpret_cast<int*>(smem + L::kOffPrefix);
    const WaitGuard guard{abort_flag, p.status, p.wait_limit_ns};

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);    // the even CTA's producer (with both CTAs' bytes)
            mbar_init(empty_bar(s), 1);   // the even CTA's commit
        }
        mbar_init(tfull_bar, 1);
        mbar_init(tempty_bar, 2 * L::kEpiWarps);   // every epilogue warp of both CTAs
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&maps.a);
        prefetch_tensormap(&maps.b);
        prefetch_tensormap(&maps.sfa);
        prefetch_tensormap(&maps.sfb);
    }
    __syncwarp();
    if (warp == 1) {
        tmem_alloc_pair(sbase + L::kOffTmemSlot, L::kTmemCols);
        tmem_relinquish_pair();
    }
    wait_for_previous();
    int total = p.m_tiles * p.n_tiles;
    if constexpr (kMode == kExperts) {
        build_prefix(p, 256, prefix);
        total = prefix[p.G];
    }
    if constexpr (kMode == kGradients) total *= p.G;
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();   // both CTAs' barriers initialised and tensor memory allocated
    tc_fence_after();
    const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(smem + L::kOffTmemSlot);
    const int pair_id = static_cast<int>(blockIdx.x >> 1), n_pairs = static_cast<int>(gridDim.x >> 1);

    if (warp == 0) {
        // ---- producer (both CTAs) --------------------------------------------------
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            const uint32_t full0 = leader ? full_bar(0) : mapa_shared(full_bar(0), 0);
            bool stop = false;
            for (int t = pair_id; t < total && !stop && !*abort_flag; t += n_pairs) {
                const PairTile ti = pair_tile<kMode>(p, prefix, t, rank);
                const int32_t ma = static_cast<int32_t>(ti.m0), nb = static_cast<int32_t>(ti.b_row + 128 * rank);
                const int32_t sfa_row = static_cast<int32_t>(2 * (ti.a_band * p.k_atoms + ti.k_atom));
                const int32_t sfb_row = static_cast<int32_t>(2 * ((ti.b_band + rank) * p.k_atoms + ti.k_atom));
                for (int kb = 0; kb < ti.num_kb; ++kb) {
                    if (!wait_phase(empty_bar(stage), phase ^ 1u, guard)) { stop = true; break; }
                    const uint32_t fb = full0 + 8u * stage;
                    if (leader) mbar_arrive_expect_tx(fb, 2u * L::kStageBytes);
                    const int32_t kx = 64 * ti.k_atom + 128 * kb, ks = 4 * kb;
                    tma_load_2d_pair(sbase + L::kOffA + stage * kBandBytes, &maps.a, kx, ma, fb);
                    tma_load_2d_pair(sbase + L::kOffB + stage * kBandBytes, &maps.b, kx, nb, fb);
                    tma_load_2d_pair(sbase + L::kOffSfa + stage * L::kSfaBytes, &maps.sfa, 0, sfa_row + ks, fb);
                    tma_load_2d_pair_mc(sbase + L::kOffSfb + stage * L::kSfbBytes + 2 * kAtom * rank, &maps.sfb, 0,
                                        sfb_row + ks, fb, 0x3);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            if (*abort_flag) {
                // Loads in flight complete on the even CTA's barrier, which the odd
                // CTA cannot wait on: give them a bounded while to land.
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 200000ull) __nanosleep(1000);
            }
        }
    } else if (warp == 1) {
        // ---- MMA issuer (even CTA; warp-uniform loops, one elected lane issues) -----------
        if (leader) {
            const uint64_t a_desc0 = make_smem_desc(sbase + L::kOffA, 16, 1024, 2);
            const uint64_t b_desc0 = make_smem_desc(sbase + L::kOffB, 16, 1024, 2);
            const uint64_t sfa_desc0 = make_smem_desc(sbase + L::kOffSfa, 0, 128, 0);
            const uint64_t sfb_desc0 = make_smem_desc(sbase + L::kOffSfb, 0, 128, 0);
            int stage = 0;
            uint32_t phase = 0, acc = 0, acc_phase = 0;
            bool ok = true, landed = false;   // the stage's bytes, seen already
            for (int t = pair_id; t < total && ok; t += n_pairs) {
                if (!warp_waits(lane, [&] { return spin_phase(tempty_bar, acc_phase ^ 1u, guard); })) { ok = false; break; }
                tc_fence_after();
                const PairTile ti = pair_tile<kMode>(p, prefix, t, 0u);
                const uint32_t d_tmem = tmem_base + acc * L::kAcc1;
                for (int kb = 0; kb < ti.num_kb; ++kb) {
                    if (!landed && !warp_waits(lane, [&] { return wait_phase(full_bar(stage), phase, guard); })) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sfa_t = tmem_base + L::kTmemScales + L::kScaleCols * stage, sfb_t = sfa_t + 8;
                    const uint64_t a_desc = a_desc0 + static_cast<uint64_t>((stage * kBandBytes) >> 4);
                    const uint64_t b_desc = b_desc0 + static_cast<uint64_t>((stage * kBandBytes) >> 4);
                    const uint64_t sfa_d = sfa_desc0 + static_cast<uint64_t>((stage * L::kSfaBytes) >> 4);
                    const uint64_t sfb_d = sfb_desc0 + static_cast<uint64_t>((stage * L::kSfbBytes) >> 4);
                    const int mmas = mmas_of<kBK>(ti.k_padded, kb);
                    const uint32_t this_empty = empty_bar(stage);
                    // ask for the next stage now and look at the answer behind the instructions
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    const bool next = mbar_test_wait(full_bar(stage), phase);
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {   // atom i: K elements 128 i .. of the stage
                            tc_cp_32x128b_warpx4_pair(sfa_t + 4 * i, sfa_d + static_cast<uint64_t>((i * kAtom) >> 4));
                            tc_cp_32x128b_warpx4_pair(sfb_t + 8 * i, sfb_d + static_cast<uint64_t>((i * kAtom) >> 4));
                            tc_cp_32x128b_warpx4_pair(sfb_t + 8 * i + 4, sfb_d + static_cast<uint64_t>(((i + 2) * kAtom) >> 4));
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k < mmas)
                                tc_mma_mxf4_pair(d_tmem, a_desc + 2 * k, b_desc + 2 * k,
                                                 make_idesc_mxf4(256, 256, 2 * (k & 1)), sfa_t + 4 * (k >> 1),
                                                 sfb_t + 8 * (k >> 1), (kb > 0 || k > 0) ? 1u : 0u);
                        tc_commit_pair_multicast(this_empty, 0x3);   // frees the slot in both CTAs
                    }
                    __syncwarp();
                    landed = __all_sync(0xFFFFFFFFu, next) != 0;
                }
                if (!ok) break;
                if (elect_one()) tc_commit_pair_multicast(tfull_bar, 0x3);
                __syncwarp();
                acc ^= 1u;
                acc_phase ^= 1u;
            }
            // Drain: every MMA issued above completes before teardown.
            if (lane == 0) {
                tc_commit_pair(drain_bar);
                WaitGuard g2 = guard;
                volatile int never = 0;
                g2.abort_flag = &never;
                (void)mbar_wait(drain_bar, 0, g2);
            }
            __syncwarp();
        }
    } else {
        // ---- epilogue (both CTAs; warps 2..9) ----------------------------------------
        const int quad = warp & 3, half = (warp - 2) >> 2;
        const uint32_t tempty_leader = leader ? tempty_bar : mapa_shared(tempty_bar, 0);
        const uint32_t buffer = sbase + L::kOffStage + (warp - 2) * L::kStageWarpBytes;
        // chunks of 16 columns of a half: of the columns that the other accumulator shares, the upper ones of the first
        // accumulator and the lower ones of the second, and of the others
        constexpr int kFirst = L::kShared / 32, kRest = 8 - kFirst;
        uint32_t acc = 0, acc_phase = 0;
        for (int t = pair_id; t < total; t += n_pairs) {
            const PairTile ti = pair_tile<kMode>(p, prefix, t, rank);
            if (!warp_waits(lane, [&] { return wait_phase(tfull_bar, acc_phase, guard); })) break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * quad) << 16) + acc * L::kAcc1;
            const int64_t row0 = ti.y_row + 32 * quad;
            uint32_t carry = 0u;
            auto store = [&](uint32_t* v, int col, bool start, bool last) {
                if (kMode == kGradients && ti.num_kb == 0) {   // an expert without rows
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = 0u;
                }
                store_chunk<kAny>(p, v, buffer, row0, ti.row_lo, ti.row_hi, ti.n0 + col, lane, &maps.y, start, last || ti.n0 + col + 16 >= p.N, &carry);
            };
            {
                const int col = (acc ? 0 : L::kAcc1) + 16 * kFirst * half;
                uint32_t v[kFirst][16];
#pragma unroll
                for (int c = 0; c < kFirst; ++c) tmem_ld_32x32b_x16(taddr + col + 16 * c, v[c]);
                tmem_ld_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (leader) mbar_arrive(tempty_bar);
                    else mbar_arrive_cluster(tempty_leader);
                }
#pragma unroll
                for (int c = 0; c < kFirst; ++c) store(v[c], col + 16 * c, c == 0, c == kFirst - 1);
            }
            {
                const int col = (acc ? L::kShared : 0) + 16 * kRest * half;
                uint32_t v[kRest][16];
#pragma unroll
                for (int c = 0; c < kRest; ++c) tmem_ld_32x32b_x16(taddr + col + 16 * c, v[c]);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < kRest; ++c) store(v[c], col + 16 * c, c == 0, c == kRest - 1);
            }
            acc ^= 1u;
            acc_phase ^= 1u;
        }
        if (lane == 0) bulk_wait_all();   // this warp's tiled stores complete before the CTA ends
        __syncwarp();
    }

    // ---- teardown: nothing may still target the peer when either CTA leaves ----
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc_pair(tmem_base, L::kTmemCols);
    }
}

// ---- few rows ----------------------------------------------------------------------------------
//
// A tile: 128 columns of y (rows of B) by up to 128 rows of A, transposed in tensor memory: lane n, column m.  The
// instruction's N is the number of rows of A, rounded up to 16, so few rows cost little beside B's bytes.
// What bounds such a product is the stream of B's bytes, and next to that the single threads that issue it: a copy takes
// its thread about 90 cycles, a scale copy or an instruction of the tensor core about 50.  So a slot is 512 K elements
// (of B 32 KB), loaded by four copies where a row's payload is a multiple of 128 bytes: B, A, and the four scale
// atoms of each; as many slots as shared memory holds.  A comes in boxes of 16 rows or of tok_cap.
// Measured: 16 x 16384 x 16384 26 us (B at 5.5 TB/s), 1 x 7168 x 7168 9.2 us, 8 x 4096 x 4096 5.5 us.  Tried without
// gain: sums sent to the CTA that adds them, each counted on a barrier there, instead of fetched between two
// barriers of the cluster (8 x 4096 x 4096 5.6 us to 7.0 us, 64 rows 6.9 us to 11.9 us).
//
// split > 1 (a cluster, one tile): CTA r takes the r-th part of K; the parts' sums are joined through
// distributed shared memory in the order of the parts.  split == 1: persistent over tiles, two accumulators.
struct RowsCfg {
    static constexpr int kThreads = 192;      // producer, MMA issuer, four epilogue warps
    static constexpr int kBlockK = 2 * kBK;   // K elements of a slot
    static constexpr int kMaxStages = 6;
    static constexpr int kNumBars = 2 * kMaxStages + 5;
    static constexpr int kTail = 8 * kNumBars + 16 + 4 * (kMaxExperts + 1);   // behind the ring
    static constexpr int kAlloc = 227 * 1024;   // at most
    static constexpr int kRing = (kAlloc - 1024 - kTail) / 1024 * 1024;
    static constexpr int kTmemCols = 512;
    static constexpr int kTmemScales = 256, kScaleCols = 32;   // after two accumulators of 128 columns, of a slot
    static_assert(kTmemScales + kScaleCols * kMaxStages <= kTmemCols, "tensor memory budget");
};

// Payloads as [chunk of 128 bytes][row][byte] with boxes of two chunks (Args::chunked), or as [row][byte] with boxes of
// one; a16: boxes of 16 rows of A, a: of tok_cap.
struct RowsMaps {
    CUtensorMap a, a16, b;
};

struct RowsTile {
    int64_t m0, a_band, n0, b_row, b_band;
    int rows;   // of A
};

template <bool kGrouped>
__device__ __forceinline__ RowsTile rows_tile(const Args& p, const int* prefix, int t) {
    RowsTile ti;
    if constexpr (!kGrouped) {   // the row tiles of a column tile follow each other: B's tile is in L2
        const int n = p.m_tiles == 1 ? t : t / p.m_tiles, i = t - n * p.m_tiles;
        ti.n0 = static_cast<int64_t>(n) * 128;
        ti.m0 = static_cast<int64_t>(i) * 128;
        ti.a_band = i;
        ti.rows = static_cast<int>(min(static_cast<int64_t>(128), p.M - ti.m0));
        ti.b_row = ti.n0;
        ti.b_band = ti.n0 / 128;
    } else {
        const int g = expert_of(prefix, p.G, t);
        const int64_t lo = offset_at(p, g), hi = offset_at(p, g + 1);
        const int tiles = static_cast<int>((hi - lo + 127) / 128), local = t - prefix[g], n = local / tiles;
        const int64_t i = local - n * tiles;
        ti.n0 = static_cast<int64_t>(n) * 128;
        ti.m0 = lo + 128 * i;
        ti.a_band = first_band(lo, g) + i;
        ti.rows = static_cast<int>(min(static_cast<int64_t>(128), hi - ti.m0));
        ti.b_row = static_cast<int64_t>(g) * p.N + ti.n0;
        ti.b_band = static_cast<int64_t>(g) * p.b_bands + ti.n0 / 128;
    }
    return ti;
}

template <bool kGrouped>
__global__ void __launch_bounds__(RowsCfg::kThreads, 1)
    gemm_mxfp4_rows_kernel(const __grid_constant__ RowsMaps maps, const Args p) {
    using L = RowsCfg;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = p.split, stages = p.stages;
    const int rank = static_cast<int>(blockIdx.x) & (split - 1);
    const int tok_bytes = p.tok_cap * 256, stage_bytes = 2 * kBandBytes + tok_bytes + 8 * kAtom;
    const int ring = stages * stage_bytes;
    const uint32_t bar0 = sbase + ring;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (L::kMaxStages + s); };
    auto tfull_bar = [&](uint32_t a) { return bar0 + 8u * (2 * L::kMaxStages) + 8u * a; };
    auto tempty_bar = [&](uint32_t a) { return bar0 + 8u * (2 * L::kMaxStages + 2) + 8u * a; };
    const uint32_t drain_bar = bar0 + 8u * (2 * L::kMaxStages + 4);
    uint8_t* tail = smem + ring + 8 * L::kNumBars;
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(tail);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tail + 4);
    int* prefix = reinterpret_cast<int*>(tail + 16);
    const WaitGuard guard{abort_flag, p.status, p.wait_limit_ns};

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (uint32_t a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), 4);   // the epilogue warps
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&maps.a);
        prefetch_tensormap(&maps.a16);
        prefetch_tensormap(&maps.b);
    }
    __syncwarp();
    if (warp == 1) {
        tmem_alloc(smem_u32(tail), L::kTmemCols);
        tmem_relinquish();
    }
    int total = p.m_tiles * p.n_tiles;
    if constexpr (kGrouped) {
        wait_for_previous();
        build_prefix(p, 128, prefix);
        total = prefix[p.G];
    }
    // The producer goes on: it needs the barriers, which are its own, and not the tensor memory.
    tc_fence_before();
    if (warp == 0) named_bar_arrive(1, L::kThreads);
    else named_bar_sync(1, L::kThreads);
    tc_fence_after();
    const uint32_t tmem_base = warp == 0 ? 0u : *tmem_slot;
    // split is a power of two; 64-bit divisions here would cost more than a slot's load
    const int num_kb = static_cast<int>((p.k_padded + L::kBlockK - 1) / L::kBlockK);
    const int kb_lo = static_cast<int>(static_cast<uint64_t>(num_kb) * rank >> p.log_split);
    const int kb_hi = static_cast<int>(static_cast<uint64_t>(num_kb) * (rank + 1) >> p.log_split);
    const int first = static_cast<int>(blockIdx.x >> p.log_split), step = static_cast<int>(gridDim.x >> p.log_split);

    if (warp == 0) {
        // ---- producer (warp-uniform loops, one elected lane issues) ------------------------------
        int stage = 0, issued = 0;
        uint32_t phase = 0;
        bool stop = false, waited = kGrouped;
        for (int t = first; t < total && !stop; t += step) {
            const RowsTile ti = rows_tile<kGrouped>(p, prefix, t);
            const bool few = ti.rows <= 16;
            const CUtensorMap* map_a = few ? &maps.a16 : &maps.a;
            const int box = few ? 16 * 128 : p.tok_cap * 128;   // bytes of a chunk of A
            const int32_t row_a = static_cast<int32_t>(ti.m0), row_b = static_cast<int32_t>(ti.b_row);
            const uint8_t* sfa = p.a_s + (ti.a_band * p.k_atoms + 4 * kb_lo) * kAtom;
            const uint8_t* sfb = p.b_s + (ti.b_band * p.k_atoms + 4 * kb_lo) * kAtom;
            int32_t chunk = 2 * kb_lo;
            int atoms = static_cast<int>(p.k_atoms) - 4 * kb_lo;   // that are left
            if (!waited) wait_for_previous();   // nothing above reads what the kernel before wrote
            waited = true;
            for (int kb = kb_lo; kb < kb_hi; ++kb) {
                if (issued >= stages &&   // the slots are free at first
                    !warp_waits(lane, [&] { return wait_phase(empty_bar(stage), phase ^ 1u, guard); })) { stop = true; break; }
                const uint32_t fb = full_bar(stage), at = sbase + stage * stage_bytes, at_a = at + 2 * kBandBytes;
                const uint32_t scales = atoms >= 4 ? 4 * kAtom : kAtom * static_cast<uint32_t>(atoms);
                if (elect_one()) {
                    mbar_arrive_expect_tx(fb, 2u * (kBandBytes + box + scales));
                    if (p.chunked) {
                        tma_load_3d(at, &maps.b, 0, row_b, chunk, fb);
                        tma_load_3d(at_a, map_a, 0, row_a, chunk, fb);
                    } else {
                        tma_load_2d(at, &maps.b, 128 * chunk, row_b, fb);
                        tma_load_2d(at + kBandBytes, &maps.b, 128 * chunk + 128, row_b, fb);
                        tma_load_2d(at_a, map_a, 128 * chunk, row_a, fb);
                        tma_load_2d(at_a + box, map_a, 128 * chunk + 128, row_a, fb);
                    }
                    bulk_load(at_a + tok_bytes, sfb, scales, fb);
                    bulk_load(at_a + tok_bytes + 4 * kAtom, sfa, scales, fb);
                }
                __syncwarp();
                sfa += 4 * kAtom, sfb += 4 * kAtom, chunk += 2, atoms -= 4;
                ++issued;
                if (++stage == stages) { stage = 0; phase ^= 1u; }
            }
        }
        if (lane == 0 && *abort_flag) {
            // Let copies already in flight land before the CTA exits.
            for (int i = issued < stages ? issued : stages; i > 0; --i) {
                if (--stage < 0) { stage = stages - 1; phase ^= 1u; }
                WaitGuard g2 = guard;
                volatile int never = 0;
                g2.abort_flag = &never;
                (void)mbar_wait(full_bar(stage), phase, g2);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- MMA issuer ----------------------------------------------------------------
        if (!kGrouped) wait_for_previous();
        int stage = 0;
        uint32_t phase = 0, acc = 0, acc_phase = 0;
        bool ok = true;
        for (int t = first; t < total && ok; t += step) {
            const RowsTile ti = rows_tile<kGrouped>(p, prefix, t);
            const uint32_t N = static_cast<uint32_t>((ti.rows + 15) & ~15);
            if (!warp_waits(lane, [&] { return spin_phase(tempty_bar(acc), acc_phase ^ 1u, guard); })) { ok = false; break; }
            tc_fence_after();
            const uint32_t d_tmem = tmem_base + acc * 128;
            const uint32_t idesc = make_idesc_mxf4(128, N, 0), idesc2 = make_idesc_mxf4(128, N, 2);
            const uint64_t a_chunk = static_cast<uint64_t>((ti.rows <= 16 ? 16 * 128 : p.tok_cap * 128) >> 4);
            for (int kb = kb_lo; kb < kb_hi; ++kb) {
                if (!warp_waits(lane, [&] { return wait_phase(full_bar(stage), phase, guard); })) { ok = false; break; }
                tc_fence_after();
                const uint32_t at = sbase + stage * stage_bytes, sc = at + 2 * kBandBytes + tok_bytes;
                const uint32_t sfb_t = tmem_base + L::kTmemScales + L::kScaleCols * stage, sfa_t = sfb_t + 16;
                const uint64_t b_desc = make_smem_desc(at, 16, 1024, 2), a_desc = make_smem_desc(at + 2 * kBandBytes, 16, 1024, 2);
                const uint64_t s_desc = make_smem_desc(sc, 0, 128, 0);
                const int mmas = mmas_of<L::kBlockK>(p.k_padded, kb);
                if (elect_one()) {
                    // atom i: K elements 128 i .. of the slot, two instructions; chunk i / 2
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (2 * i < mmas) {
                            tc_cp_32x128b_warpx4(sfb_t + 4 * i, s_desc + static_cast<uint64_t>((i * kAtom) >> 4));
                            tc_cp_32x128b_warpx4(sfa_t + 4 * i, s_desc + static_cast<uint64_t>(((i + 4) * kAtom) >> 4));
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < mmas)
                            tc_mma_mxf4(d_tmem, b_desc + static_cast<uint64_t>(((k >> 2) * kBandBytes) >> 4) + 2 * (k & 3),
                                        a_desc + (k >= 4 ? a_chunk : 0) + 2 * (k & 3), k & 1 ? idesc2 : idesc,
                                        sfb_t + 4 * (k >> 1), sfa_t + 4 * (k >> 1), (kb > kb_lo || k > 0) ? 1u : 0u);
                    tc_commit(empty_bar(stage));
                }
                __syncwarp();
                if (++stage == stages) { stage = 0; phase ^= 1u; }
            }
            if (!ok) break;
            if (elect_one()) tc_commit(tfull_bar(acc));
            __syncwarp();
            if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        }
        // Drain: every MMA and copy issued above completes before teardown.
        if (lane == 0) {
            tc_commit(drain_bar);
            WaitGuard g2 = guard;
            volatile int never = 0;
            g2.abort_flag = &never;
            (void)mbar_wait(drain_bar, 0, g2);
        }
        __syncwarp();
    } else {
        // ---- epilogue: lane l of the warp on quarter q holds column n0 + 32 q + l of y ----------------
        if (!kGrouped) wait_for_previous();
        const int quad = warp & 3, n = 32 * quad + lane;
        uint32_t acc = 0, acc_phase = 0;
        for (int t = first; t < total; t += step) {
            const RowsTile ti = rows_tile<kGrouped>(p, prefix, t);
            if (!warp_waits(lane, [&] { return wait_phase(tfull_bar(acc), acc_phase, guard); })) break;
            tc_fence_after();
            const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * quad) << 16) + acc * 128;
            const bool in = ti.n0 + n < p.N;
            uint16_t* out = p.y + ti.m0 * p.ldy + ti.n0 + n;
#pragma unroll 1
            for (int c = 0; c < ti.rows; c += 16) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(taddr + c, v);
                tmem_ld_wait();
                if (split > 1) {   // the ring is free: every copy has been consumed
                    float* part = reinterpret_cast<float*>(smem) + c * 128 + n;
#pragma unroll
                    for (int i = 0; i < 16; ++i) part[i * 128] = __uint_as_float(v[i]);
                } else if (in) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c + i < ti.rows) out[(c + i) * p.ldy] = from_float<bf16_bits>(__uint_as_float(v[i]));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty_bar(acc));
            if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (split > 1) {
        cluster_sync_all();   // every part is written
        if (first < total) {
            // a warp joins a row of 128 columns at a time, four a lane
            const RowsTile ti = rows_tile<kGrouped>(p, prefix, first);
            const int64_t n = ti.n0 + 4 * lane;
#pragma unroll 2
            for (int m = rank + split * warp; m < ti.rows; m += split * (L::kThreads / 32)) {
                const uint32_t at = sbase + 16u * static_cast<uint32_t>(m * 32 + lane);
                float4 part[8];
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    if (s < split) part[s] = ld_cluster(mapa_shared(at, static_cast<uint32_t>(s)));
                float4 sum = part[0];
#pragma unroll
                for (int s = 1; s < 8; ++s)
                    if (s < split) sum.x += part[s].x, sum.y += part[s].y, sum.z += part[s].z, sum.w += part[s].w;
                const uint32_t lo = cvt_bf16x2(sum.x, sum.y), hi = cvt_bf16x2(sum.z, sum.w);
                uint16_t* out = p.y + (ti.m0 + m) * p.ldy + n;
                if (p.y_vec && n + 4 <= p.N) {
                    *reinterpret_cast<uint2*>(out) = make_uint2(lo, hi);
                } else {
                    if (n < p.N) out[0] = static_cast<uint16_t>(lo);
                    if (n + 1 < p.N) out[1] = static_cast<uint16_t>(lo >> 16);
                    if (n + 2 < p.N) out[2] = static_cast<uint16_t>(hi);
                    if (n + 3 < p.N) out[3] = static_cast<uint16_t>(hi >> 16);
                }
            }
        }
        cluster_sync_relaxed();   // nobody leaves while its part is read
    }
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc(tmem_base, L::kTmemCols);
    }
}

// ---- host --------------------------------------------------------------------------------------

// Output rows that start on 16 bytes.
bool whole_rows(const Gemm4Args& g) { return (reinterpret_cast<uintptr_t>(g.y) & 15u) == 0 && g.ldy % 8 == 0; }

constexpr int64_t kMostItems = (int64_t(1) << 31) - 4096;   // tiles of a launch: 32-bit counters step past the last one

// Payload [rows, row_bytes], boxes of box_rows x 128 bytes, 128-byte swizzle.
bool payload_map(CUtensorMap* map, const void* q, int64_t rows, int64_t row_bytes, uint32_t box_rows) {
    return encode_tensor_map_2d(map, q, false, static_cast<uint64_t>(row_bytes), static_cast<uint64_t>(rows),
                                static_cast<uint64_t>(row_bytes), 128u, box_rows, true);
}

// The same by chunks of 128 bytes (row_bytes a multiple of it), boxes of box_rows rows of two chunks, chunk by chunk.
bool chunk_map(CUtensorMap* map, const void* q, int64_t rows, int64_t row_bytes, uint32_t box_rows) {
    return encode_tensor_map_chunks(map, q, static_cast<uint64_t>(rows), static_cast<uint64_t>(row_bytes), box_rows, 2u);
}

// MMA-tiled scales as rows of 256 bytes, boxes of two atoms.
bool scale_map(CUtensorMap* map, const void* s, int64_t bands, int64_t k_atoms) {
    if ((bands + 2) * k_atoms * 2 >= (int64_t(1) << 31)) return false;
    return encode_tensor_map_2d(map, s, false, 256u, static_cast<uint64_t>(bands * k_atoms * 2), 256u, 256u, 4u, false);
}

// One launch of `grid` CTAs in clusters of `cluster` (0: as the kernel says), whose start overlaps the end of the
// kernel before it on the stream.
template <typename Maps>
cudaError_t launch(void (*kernel)(const Maps, const Args), int64_t grid, int threads, int smem, int cluster,
                   cudaStream_t stream, const Maps& maps, const Args& args) {
    cudaLaunchAttribute attrs[2] = {};
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = static_cast<unsigned>(cluster > 0 ? cluster : 1);
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = dim3(static_cast<unsigned>(grid));
    config.blockDim = dim3(static_cast<unsigned>(threads));
    config.dynamicSmemBytes = static_cast<size_t>(smem);
    config.stream = stream;
    config.attrs = attrs;
    config.numAttrs = cluster > 0 ? 2 : 1;
    void* addresses[] = {const_cast<Maps*>(&maps), const_cast<Args*>(&args)};
    return cudaLaunchKernelExC(&config, reinterpret_cast<const void*>(kernel), addresses);
}

// The kernel's shared-memory limit, once per device and thread.
template <typename Kernel>
cudaError_t allow_smem(Kernel* kernel, int bytes, int device, int* configured) {
    if (*configured == device) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) *configured = device;
    return e;
}

template <int kMode, bool kAny>
cudaError_t launch_pair_of(const DeviceInfo& dev, const Gemm4Args& g, Args args, cudaStream_t stream) {
    using L = PairCfg;
    static thread_local int configured = -1;
    const cudaError_t e = allow_smem(gemm_mxfp4_pair_kernel<kMode, kAny>, L::kAlloc, dev.device, &configured);
    if (e != cudaSuccess) return e;
    const int64_t row_bytes = args.k_padded / 2, experts = kMode == kExperts ? g.G : 1;
    PairMaps maps;
    if (!payload_map(&maps.a, g.a_q, g.M, row_bytes, 128) || !payload_map(&maps.b, g.b_q, experts * g.N, row_bytes, 128) ||
        !scale_map(&maps.sfa, g.a_s, kMode == kExperts ? g.bands_cap : (g.M + 127) / 128, args.k_atoms) ||
        !scale_map(&maps.sfb, g.b_s, experts * args.b_bands, args.k_atoms))
        return cudaErrorInvalidValue;
    const int64_t m_tiles = (g.M + 255) / 256, n_tiles = (g.N + 255) / 256;
    const int64_t y_rows = kMode == kGradients ? g.G * g.M : g.M;
    const int64_t items = kMode == kDense ? m_tiles * n_tiles : kMode == kExperts ? (m_tiles + g.G) * n_tiles : g.G * m_tiles * n_tiles;
    if (items > kMostItems) return cudaErrorInvalidValue;
    args.items = static_cast<int>(items);
    args.m_tiles = static_cast<int>(m_tiles);
    args.n_tiles = static_cast<int>(n_tiles);
    args.y_tma = !kAny && encode_tensor_map_bf16_store16(&maps.y, g.y, static_cast<uint64_t>(g.N),
                                                              static_cast<uint64_t>(y_rows), static_cast<uint64_t>(g.ldy));
    const int64_t pairs = items < dev.sm_count / 2 ? items : dev.sm_count / 2;
    return launch(gemm_mxfp4_pair_kernel<kMode, kAny>, 2 * pairs, L::kThreads, L::kAlloc, 0, stream, maps, args);
}

template <int kMode>
cudaError_t launch_pair(const DeviceInfo& dev, const Gemm4Args& g, const Args& args, cudaStream_t stream) {
    return whole_rows(g) ? launch_pair_of<kMode, false>(dev, g, args, stream) : launch_pair_of<kMode, true>(dev, g, args, stream);
}

// Clusters of 1 << log_split CTAs of the rows kernel that the device holds at once (looked up once per device and thread).
template <bool kGrouped>
int64_t clusters_of(const DeviceInfo& dev, int log_split) {
    static thread_local int known_device = -1;
    static thread_local int known[4];
    if (known_device != dev.device) {
        for (int i = 0; i < 4; ++i) {
            cudaLaunchAttribute attr{};
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = 1u << i;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cudaLaunchConfig_t config{};
            config.gridDim = dim3(static_cast<unsigned>(dev.sm_count >> i << i));
            config.blockDim = dim3(RowsCfg::kThreads);
            config.dynamicSmemBytes = RowsCfg::kAlloc;
            config.attrs = &attr;
            config.numAttrs = 1;
            known[i] = 0;
            if (cudaOccupancyMaxActiveClusters(&known[i], gemm_mxfp4_rows_kernel<kGrouped>, &config) != cudaSuccess)
                (void)cudaGetLastError();
        }
        known_device = dev.device;
    }
    return known[log_split];
}

// Grouped: tiles of the rows kernel at most, of the experts with rows, each with one partly filled tile.
int64_t most_tiles(const Gemm4Args& g) { return ((g.M < g.G ? g.M : g.G) + g.M / 128) * ((g.N + 127) / 128); }

template <bool kGrouped>
cudaError_t launch_rows(const DeviceInfo& dev, const Gemm4Args& g, Args args, cudaStream_t stream) {
    using L = RowsCfg;
    static thread_local int configured = -1;
    const cudaError_t e = allow_smem(gemm_mxfp4_rows_kernel<kGrouped>, L::kAlloc, dev.device, &configured);
    if (e != cudaSuccess) return e;
    const int64_t row_bytes = args.k_padded / 2, experts = kGrouped ? g.G : 1;
    RowsMaps maps;
    const int64_t m_tiles = (g.M + 127) / 128, n_tiles = (g.N + 127) / 128;
    const int64_t tiles = kGrouped ? most_tiles(g) : m_tiles * n_tiles;
    if (tiles > kMostItems) return cudaErrorInvalidValue;
    args.items = static_cast<int>(tiles);
    args.m_tiles = static_cast<int>(m_tiles);
    args.n_tiles = static_cast<int>(n_tiles);
    args.y_vec = (reinterpret_cast<uintptr_t>(g.y) & 7u) == 0 && g.ldy % 4 == 0;
    args.tok_cap = static_cast<int>(g.M < 128 ? (g.M + 15) / 16 * 16 : 128);
    args.chunked = row_bytes % 128 == 0;
    const auto map = [&](CUtensorMap* m, const void* q, int64_t rows, int box) {
        return args.chunked ? chunk_map(m, q, rows, row_bytes, static_cast<uint32_t>(box))
                            : payload_map(m, q, rows, row_bytes, static_cast<uint32_t>(box));
    };
    if (!map(&maps.a, g.a_q, g.M, args.tok_cap) || !map(&maps.a16, g.a_q, g.M, 16) || !map(&maps.b, g.b_q, experts * g.N, 128))
        return cudaErrorInvalidValue;
    const int stage_bytes = 2 * kBandBytes + args.tok_cap * 256 + 8 * kAtom;
    args.stages = L::kRing / stage_bytes < L::kMaxStages ? L::kRing / stage_bytes : L::kMaxStages;
    const int smem = 1024 + args.stages * stage_bytes + L::kTail;
    const int64_t num_kb = (args.k_padded + L::kBlockK - 1) / L::kBlockK;
    int log_split = 0;
    while (log_split < 3 && tiles << (log_split + 1) <= dev.sm_count && num_kb >> (log_split + 1) >= 1) ++log_split;
    // as many clusters as the device holds at once: 8 CTAs have to lie in one GPC, whose other SMs stay idle
    while (log_split > 1 && tiles > clusters_of<kGrouped>(dev, log_split)) --log_split;
    const int split = 1 << log_split;
    args.split = split;
    args.log_split = log_split;
    const int64_t grid = split > 1 ? tiles * split : (tiles < dev.sm_count ? tiles : dev.sm_count);
    return launch(gemm_mxfp4_rows_kernel<kGrouped>, grid, L::kThreads, smem, split > 1 ? split : 0, stream, maps, args);
}

// Which kernel.  Few rows leave most of a 256-row tile's instructions idle; where there are few tiles, a cluster of the
// rows kernel splits K of each and more SMs work than there are pairs.  Measured, rows kernel / pairs (us, in a graph):
//   N x K           M = 16      64            128           256           512           1024
//   4096 x 1024     4.9 / 7.1   6.1 / 7.3     7.9 / 7.5     8.1 / 7.3     8.1 / 7.5     12.2 / 7.7
//   2048 x 2048     4.9 / 8.3   5.9 / 8.2     7.2 / 8.5     7.6 / 8.4     8.9 / 8.4     9.1 / 8.5
//   1024 x 7168     5.7 / 13.5  6.7 / 13.5    8.0 / 13.7    8.8 / 13.6    9.3 / 13.7    11.4 / 13.9
//   4096 x 4096     5.8 / 10.8  6.8 / 10.8    8.2 / 10.9    9.9 / 10.8    11.7 / 11.1   16.6 / 12.0
//   7168 x 7168     9.7 / 15.2  11.3 / 15.2   13.8 / 15.5   17.0 / 15.3   24.6 / 16.2   33.1 / 24.6
//   16384 x 16384   25.9 / 31.1 28.6 / 31.3   33.9 / 31.9   50.3 / 32.4   85.7 / 48.8   139 / 86.6
// Output rows that do not start on 16 bytes cost the pairs up to 1 us more and the rows kernel nothing: 777 x 2085 (K 1003)
// 7.8 / 8.2, 300 x 4099 (K 4096) 10.5 / 11.3, 777 x 1003 (K 300) 7.3 / 7.4, (K 2085) 9.5 / 9.2, but 2000 x 2085 (K 1003), two
// waves of tiles, 11.9 / 8.4.
// Grouped, up to 48 rows an expert the rows kernel, past that as for a dense product, of the most tiles that the rows can make.
// Rows an expert, experts of equal loads:
//   experts of N x K      64             128            256            512
//   1 of 4096 x 4096      7.4 / 13.4     10.1 / 13.6    11.2 / 10.6    11.3 / 10.7
//   1 of 2048 x 2048      6.5 / 8.3      7.8 / 8.4      9.1 / 8.4      9.3 / 8.5
//   1 of 1024 x 7168      7.2 / 13.8     9.3 / 13.9     9.4 / 14.4     11.4 / 14.0
//   4 of 1024 x 7168      9.9 / 13.7     11.7 / 13.9    14.2 / 13.9    14.5 / 14.1
//   4 of 768 x 4096       7.5 / 10.5     10.2 / 10.6    10.4 / 10.6    11.3 / 10.7
//   8 of 4096 x 4096      14.2 / 16.8    17.6 / 17.3    28.7 / 17.8    48.3 / 31.1
//   16 of 2048 x 2048     10.4 / 12.0    14.2 / 12.1    23.1 / 12.2    37.3 / 19.3
//   128 of 4096 x 4096    193 / 209      209 / 220      343 / 232      633 / 394
//   128 of 4096 x 1024    80 / 72        131 / 76       255 / 103      505 / 145
// and with loads as 1, 2^-1.1, 3^-1.1, ..:
//   128 of 4096 x 4096    225 / 227      278 / 257      398 / 326      657 / 475
//   32 of 4096 x 4096     61 / 61        74 / 68        106 / 82       173 / 115
//   8 of 1024 x 7168      14.1 / 14.1    14.2 / 14.2    14.5 / 14.3    22.4 / 15.2
// 48 rows: between 10% for the rows kernel (equal loads) and 10% for pairs (unequal ones of 128 x 4096 x 1024).
template <bool kGrouped>
bool fills_pairs(const DeviceInfo& dev, const Gemm4Args& g) {
    if (g.M <= (kGrouped ? 48 * static_cast<int64_t>(g.G) : 64)) return false;
    const int64_t tiles = kGrouped ? most_tiles(g) : ((g.M + 127) / 128) * ((g.N + 127) / 128);
    if (!kGrouped && !whole_rows(g)) return tiles > dev.sm_count;
    if (g.K >= 4096) return 2 * tiles > dev.sm_count;
    return g.K < 2048 || 4 * tiles > dev.sm_count;
}

}  // namespace

namespace {

Args args_of(const DeviceInfo& dev, const Gemm4Args& g) {
    Args a{};
    a.a_s = static_cast<const uint8_t*>(g.a_s);
    a.b_s = static_cast<const uint8_t*>(g.b_s);
    a.y = static_cast<uint16_t*>(g.y);
    a.M = g.M, a.N = g.N, a.ldy = g.ldy;
    a.k_padded = (g.K + 31) / 32 * 32;
    a.k_atoms = (a.k_padded + 127) / 128;
    a.b_bands = (g.N + 127) / 128;
    a.offsets = g.offsets;
    a.offset_limit = g.M;
    a.G = g.G;
    a.bands_cap = g.bands_cap;
    a.split = 1;
    a.status = dev.status;
    // The epilogue waits for a tile's whole contraction, 0.27 to 0.35 us a stage: of an expert's 2^31 rows 2.2 s, where the
    // default limit alone, 2 s, would run out on work that goes on.
    a.wait_limit_ns = kDefaultWaitLimitNs + static_cast<uint64_t>(a.k_padded / kBK) * 1000u;
    return a;
}

}  // namespace

cudaError_t launch_gemm_mxfp4(const DeviceInfo& dev, const Gemm4Args& g, cudaStream_t stream) {
    const Args a = args_of(dev, g);
    return g.offsets != nullptr ? (fills_pairs<true>(dev, g) ? launch_pair<kExperts>(dev, g, a, stream) : launch_rows<true>(dev, g, a, stream))
                                : (fills_pairs<false>(dev, g) ? launch_pair<kDense>(dev, g, a, stream) : launch_rows<false>(dev, g, a, stream));
}

cudaError_t launch_grouped_wgrad_mxfp4(const DeviceInfo& dev, const Gemm4Args& g, int64_t rows, cudaStream_t stream) {
    Args a = args_of(dev, g);
    a.offset_limit = rows;
    return launch_pair<kGradients>(dev, g, a, stream);
}

}  // namespace mxq
