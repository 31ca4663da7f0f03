// One-query attention over the paged cache with a sliding window, a few first
// tokens that stay visible, and grouped heads, for 16-bit caches and for the
// 8-bit cache with one scale per (block, head).
//
// Mathematics: the query at p = L - 1 sees t < L with t >= ws = max(0, L -
// window) or t < sinks; out = sum_t w_t V_t / sum_t w_t with w_t =
// 2^(c s_t - m), taken in one pass over the visible tokens.  The reference m
// is moved only when a score passes it by more than 2^8, so most tiles need
// one vote and no reduction; numerator and denominator always share it.
//
// What bounds it: reading K and V once, 4 D bytes a token and K/V head (2 D
// in 8 bits) for about 4 D flops a query head and token, so memory as long as
// a tile costs few instructions.  Both products are warp matrix products with
// the tokens (K Q^T) or the dims (V^T P^T) as their 16 rows and the query
// heads of the K/V head as their 8 columns: for up to 8 heads that is half the
// products, sums and accumulators of the other order, and K and V are read
// once per group.  (tcgen05 needs 64 rows and more and its operands through
// one more hop; at these sizes the copies would wait for it.)
// Measured (kernel alone, one B200): 32 sequences of 256 to 2048, window 1024,
// 40 heads, fp16: 89 us, 6.4 TB/s; 256 of 1000 to 32768, window 4096, 8 K/V
// heads, bf16: 629 us, 6.6 TB/s; 128 of 1024 to 16384, 8 K/V heads, e4m3:
// 370 us (405 on some runs), 6.2 TB/s, the same at 1530 and 1965 MHz, with the
// ALU 37 % and the matrix unit 26 % busy.  Small calls are bound by latency:
// lengths, table, tiles, then the join, 14.5 us for one sequence and a window
// of 4100.
//
// Layout of the work: a "unit" is (sequence, K/V head, kHeads query heads);
// its visible tokens are cut into tiles of 4 KB of K and 4 KB of V (16 tokens
// at D = 128 in 16 bits).  The kernel's blocks count the tiles and choose, all
// alike, one of three ways to share them out:
//   * as many units as CTAs or fewer: each unit is cut into even parts of at
//     least 16 tiles, one a CTA, whose four warps take its tiles in turn and
//     merge in shared memory;
//   * as many units as warps or fewer: the same with parts for single warps;
//   * else the tiles of all units, unit after unit, are cut into equal
//     contiguous ranges, one a warp, which needs nobody else until the end of
//     a unit that straddles ranges.  Cuts within 2 tiles of a unit's end move
//     there.
// A cut unit's parts go to the workspace and the last one to arrive merges
// them in order, so the result does not depend on the order of arrival.
// Ranges also take over from parts when there is much work (16 tiles a warp)
// of unlike lengths: when parts of up to 1.75 (8 bits: 1.25) times a worker's
// share do not give each worker one at most, or the longest is more than 1.3
// times their mean.  Memory does not mind that a third of the warps have no
// part, as long as the others end together, and a second segment or a
// straddling unit costs a warp 4 us or more; the conversions of 8-bit codes
// do mind.  Measured, parts against ranges (us, D = 128, 16 bits; units of up
// to 8 heads): 8 units of 4100 tokens 14.3 / 88; 128 of 4100 50 / 60; 256 of
// 4100 102 / 98; 1280 of 1028 108 / 115; 1280 of 256 to 1028 80 / 77; 1280 of
// 256 to 1028, window 1024 (the 32 windows) 93 / 100; 384 of 512 to 4100 82 / 85.
// Parts of up to 1.75 times a share in 8 bits against ranges (int8, e4m3): 1024
// units of 1024 to 16384 584, 486 / 379, 375; like lengths, 1088 of 4000 256, 213
// / 179, 186; 1088 of 9000 601, 521 / 386, 399; 1280 of 6000 415, 352 / 324, 325;
// 320 of 8000 135, 116 / 113, 117; 1120 of 2000 131, 108 / 99, 105; 1280 of 1028
// 71, 62 / 65, 64: hence 1.25 there.
//
// kHeads: groups of more than 8 heads take 16 columns at a time, which reads K
// and V half as often (128 such units of 8000 tokens: 94 us against 131, 64 to
// 71 against 77 to 88 in 8 bits), but 8 at a time when there are 32 such units
// or fewer, twice the parts to run side by side (8 units of 8000: 18.2 us
// against 23.3, 32: 31.9 against 34.0; in 8 bits 17.7 and 28.3 against 25.9 and
// 31.7).
//
// Each warp keeps a ring of kStages tiles full, across units: one lane per
// block run issues TMA boxes (K and V) that complete an mbarrier, with the
// 128-byte swizzle that keeps matrix loads free of bank conflicts.  The block
// ids of the next tile are looked up one tile ahead.  Rows of a loaded run
// that the mask hides are zeroed in V and masked in the scores.  Waits are
// bounded; one that runs out records PA_DEVERR_TIMEOUT.
//
// Choices of fewer bits: the weights enter the product with V as the sum of
// two 16-bit numbers, within 2^-15 (bf16) or 2^-20 (fp16) of fp32 ones.  With up
// to 4 heads the second ones stand in columns 4 to 7, which the heads of
// columns 0 to 3 take once more; with up to 8 they are a second matrix product.
// One number alone rounds weights by 2^-8 or 2^-11, for this much less time
// (us): 32 windows of 40 heads 90.4 against 90.6, 256 windows in groups of 8
// 620 against 626; in 8 bits, 4 contexts of 40 heads 19.3 against 19.7, groups
// of 8 19.2 against 20.3 (200 contexts of 300 to 900) and 369 against 372 (the
// 128).  With 16 heads there is one number: two would take 32 contexts of
// 8000 in 8 bits from 65 to 77 us, and groups of 128 from 128 to 153.
// fp16 weights are 2^7 times larger than the softmax's (numerator and
// denominator alike; below 2^15 with the stale reference), which keeps those
// down to 2^-31 of the largest.  bf16: small enough for the largest V
// (weight_shift in window_host.cuh).  With 8-bit codes the products are fp16
// (codes are exact in it): the query row is scaled by a power of two so that
// its largest component is near 2^14, exact for every component above 2^-28 of
// it; a block's s_v is folded into its weights relative to a running power of
// two at or above the largest s_v so far (a block's values count down to 2^-31
// of the largest s_v times the largest weight).
#pragma once

#include <cuda.h>
#include <climits>
#include <cstdint>

#include "../../include/pa_window.h"
#include "half_types.cuh"
#include "mma_sync.cuh"
#include "ptx.cuh"
#include "tcgen05_window.cuh"

namespace pa {

enum class KvStore { kF16, kBf16, kInt8, kE4m3 };

struct WindowDecodeParams {
    void *out;                  // [B, H, D]
    const void *q;              // [B, H, D]
    const float2 *scales;       // [NB, scale_heads] (8-bit)
    const int32_t *tables;      // [B, max_blocks]
    const int32_t *lens;        // [B]
    int max_blocks, max_len, window, sinks;
    int num_seqs, heads, kv_heads, group, row_tiles;  // row_tiles = ceil(group / kHeads)
    int log2_bs, num_blocks, scale_heads;
    int bf16;                   // type of q and out
    float scale_log2;           // softmax scale * log2(e)
    float shift;                // weights are 2^shift times the softmax's
    float4 *part_o;             // [kWdSlots][kNq][D / 16][32 lanes]
    float4 *part_ml;            // [kWdSlots][kNq][4] (m, l) of two query heads
    unsigned *tickets;          // [units]
    unsigned *err;
};

constexpr int kWdWarps = 4;
constexpr int kWdThreads = kWdWarps * 32;
constexpr int kWdMaxCtas = 512;
constexpr int kWdMaxRanges = kWdMaxCtas * kWdWarps;
constexpr float kWdRescale = 8.0f;   // move the reference only past this growth
constexpr int kWdSnap = 2;           // cuts of ranges this close to a unit's end move there
constexpr int kWdMuchWork = 16;      // tiles a warp below which ranges are not worth it
constexpr int kWdCuts = 2;           // lengths of parts that are tried
constexpr int kWdCuts8 = 1;          // of them, those that a large 8-bit batch may use
constexpr float kWdAlike = 1.3f;     // longest part of a large batch, times their mean
// least tiles of a part: one for a CTA (4 a warp), one for a warp
constexpr int kWdTeamTiles = 16, kWdWarpTiles = 8;
constexpr int kWdSlots = 2 * kWdMaxRanges;  // partial results: 2 a range, or 1 a part

template <KvStore kStore, int D>
struct WindowTraits {
    static constexpr bool kEight = kStore == KvStore::kInt8 || kStore == KvStore::kE4m3;
    static constexpr bool kBf16 = kStore == KvStore::kBf16;
    static constexpr int kStages = 2;
    static constexpr int kRowBytes = D * (kEight ? 1 : 2);
    static constexpr int kTile = 4096 / kRowBytes;        // tokens per tile
    static constexpr int kMt = kTile / 16;                // 16-token rows of products per tile
    static constexpr int kStageBytes = 8192;
    static constexpr int kOffMerge = kWdWarps * kStages * kStageBytes;
    static constexpr int kOffMl = kOffMerge + kWdWarps * 4 * 32 * 16;  // 4 fragments a warp
    static constexpr int kSmem = kOffMl + kWdWarps * 8 * 8;

    // Byte offset of a 16-byte chunk of a token's row in a tile: 128-byte
    // lines, the chunk's place XORed with the line's number mod 8.
    static __device__ __forceinline__ uint32_t at(int token, int chunk)
    {
        if constexpr (!kEight) {          // [8-token group][64-dim half][8 tokens]
            const int r = token & 7;
            return uint32_t(((token >> 3) * (D / 64) + (chunk >> 3)) * 1024 + r * 128 +
                            (((chunk & 7) ^ r) << 4));
        } else if constexpr (D == 128) {  // a token a line
            return uint32_t(token * 128 + ((chunk ^ (token & 7)) << 4));
        } else {                          // two tokens a line
            const int line = token >> 1;
            return uint32_t(line * 128 + (((((token & 1) << 2) | chunk) ^ (line & 7)) << 4));
        }
    }

    // Token of product row g (+ 8 when `high`) within 16 tokens: for 8-bit
    // rows in the order in which the transposing load gives V, four tokens to
    // a lane.
    static __device__ __forceinline__ int token_of(int g, int high)
    {
        return kEight ? 4 * (g >> 1) + (g & 1) + 2 * high : g + 8 * high;
    }
};

// What one sequence's query sees, in tiles of kTile tokens: the tiles that
// hold its first tokens, then those of the window.
struct WindowView {
    int L, ws, sink_tiles, first, tiles;

    template <int kTile>
    __device__ __forceinline__ void set(int len, int max_len, int window, int sinks)
    {
        L = max(0, min(len, max_len));
        ws = max(0, L - window);
        first = ws / kTile;
        sink_tiles = min((min(sinks, ws) + kTile - 1) / kTile, first);
        tiles = L > 0 ? sink_tiles + (L + kTile - 1) / kTile - first : 0;
    }
    // First token of visible tile i.
    template <int kTile>
    __device__ __forceinline__ int token(int i) const
    {
        return (i < sink_tiles ? i : i - sink_tiles + first) * kTile;
    }
    __device__ __forceinline__ bool sees(int t, int sinks) const
    {
        return t < L && (t >= ws || t < sinks);
    }
};

// How the tiles are shared out (in shared memory, looked at between segments).
struct WindowPlan {
    long long items, total;   // parts; tiles
    long long workers;        // warps (or CTAs)
    const long long *before;  // tiles (or parts) before each thread's sequences [kWdThreads]
    bool ranges;              // contiguous ranges, or parts
    int chunk;                // most tiles of a part
    int units;                // units of a sequence
    int per;                  // sequences per thread in `before`
};

// A stretch [begin, end) of one unit's tiles for one worker.
struct WindowSegment {
    int b, r;              // sequence, unit within the sequence
    int begin, end;
    long long item;        // ranges: number of the unit's first tile; else of the part
    long long left;        // ranges: tiles of the range behind this segment
    int part, parts;       // not ranges: place among the unit's parts
    WindowView view;

    // Number of parts of a unit of `tiles` tiles.
    static __device__ __forceinline__ int cut(int tiles, int chunk)
    {
        return int((unsigned(tiles) + unsigned(chunk) - 1) / unsigned(chunk));
    }

    // The part `item` (its number is set); false behind the last one.
    template <int kTile>
    __device__ __forceinline__ bool locate(const WindowDecodeParams &p, const WindowPlan &plan)
    {
        if (item >= plan.items)
            return false;
        int t = 0;         // last thread whose sequences begin at or before the part
#pragma unroll
        for (int half = kWdThreads / 2; half >= 1; half >>= 1)
            if (plan.before[t + half] <= item)
                t += half;
        long long at = plan.before[t];
        for (b = t * plan.per;; ++b) {
            view.set<kTile>(p.lens[b], p.max_len, p.window, p.sinks);
            parts = cut(view.tiles, plan.chunk);
            const long long n = (long long)parts * plan.units;
            if (item < at + n)
                break;
            at += n;
        }
        const unsigned in = unsigned(item - at);  // parts are fewer than the slots
        r = int(in / unsigned(parts));
        part = int(in % unsigned(parts));
        begin = int((long long)part * view.tiles / parts);
        end = int((long long)(part + 1) * view.tiles / parts);
        return true;
    }

    template <int kTile>
    __device__ __forceinline__ bool next(const WindowDecodeParams &p, const WindowPlan &plan)
    {
        if (!plan.ranges) {
            item += plan.workers;
            return locate<kTile>(p, plan);
        }
        if (left <= 0)
            return false;
        item += view.tiles;
        if (++r == plan.units) {
            r = 0;
            do {
                ++b;
                view.set<kTile>(p.lens[b], p.max_len, p.window, p.sinks);
            } while (view.tiles == 0);
        }
        begin = 0;
        end = int(min((long long)view.tiles, left));
        left -= end;
        return true;
    }
};

// Four int8 or e4m3 codes of a word as two fp16 pairs (exact).
template <bool kE4m3>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    if constexpr (kE4m3) {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        // a byte under the exponent of 1024 is the number 1024 + byte; with
        // the sign bit flipped the byte is code + 128
        const uint32_t u = w ^ 0x80808080u;
        const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140);
        const uint32_t b = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), bias);
        const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), bias);
        lo = *reinterpret_cast<const uint32_t *>(&x);
        hi = *reinterpret_cast<const uint32_t *>(&y);
    }
}

__device__ __forceinline__ long long ceil_div(long long a, long long b)
{
    return (a + b - 1) / b;
}

// Smallest power of two >= x (x >= 0; infinity stays, NaN gives 0).
__device__ __forceinline__ float pow2_at_least(float x)
{
    return __uint_as_float((__float_as_uint(x) + 0x7fffffu) & 0x7f800000u);
}


// The larger one of the two 16-bit numbers that stand for a weight.  Of 8-bit
// codes, which are finite, the nearest; else less than the weight, so that the
// rest is not zero or negative and an infinite V row stays infinite: bf16, the
// number at or below the next smaller fp32 one (the rest is rounded by 2^-15 of
// the weight); fp16, a little less than the nearest one (2^-20; weights below
// 2^-23 have one part only).
template <KvStore kStore>
__device__ __forceinline__ uint32_t most_of(float w0, float w1)
{
    if constexpr (kStore == KvStore::kBf16)
        return __byte_perm(max(__float_as_uint(w0), 1u) - 1u, max(__float_as_uint(w1), 1u) - 1u, 0x7632);
    else if constexpr (kStore == KvStore::kF16)
        return Half16<false>::pack(fmaxf(fmaf(w0, 1.0f - 0x1p-10f, -0x1p-24f), 0.0f),
                                   fmaxf(fmaf(w1, 1.0f - 0x1p-10f, -0x1p-24f), 0.0f));
    else
        return Half16<false>::pack(w0, w1);
}

// Joins a unit's parts, in order: for each 8 query heads the fragments n0,
// n0 + kStride, ... (kCount of them), kAhead parts' loads in flight.
template <int kCount, int kStride, typename Slot, typename Ml, typename Part, typename Store>
__device__ __forceinline__ void merge_parts(int parts, Slot slot_of, Ml part_ml, Part part_o, Store store,
                                            int columns8, int n0, int c, int rows)
{
    constexpr int kAhead = kCount >= 8 ? 2 : kCount >= 4 ? 4 : 8;
    const float4 none = make_float4(-INFINITY, 0.0f, -INFINITY, 0.0f);
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
    for (int nq = 0; nq < columns8; ++nq) {
        const int most = 8 * nq + 2 * c < rows ? parts : 0;
        float M0 = -INFINITY, M1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
        float4 acc[kCount];
#pragma unroll
        for (int n = 0; n < kCount; ++n)
            acc[n] = zero;
#pragma unroll 1
        for (int k = 0; k < most; k += kAhead) {
            float4 e[kAhead], x[kAhead][kCount];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const size_t slot = slot_of(k + j);
                e[j] = k + j < most ? __ldcg(part_ml(slot, nq)) : none;
#pragma unroll
                for (int n = 0; n < kCount; ++n)
                    x[j][n] = k + j < most ? __ldcg(part_o(slot, nq, n0 + kStride * n)) : zero;
            }
            float x0 = M0, x1 = M1;
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                x0 = fmaxf(x0, e[j].x), x1 = fmaxf(x1, e[j].z);
            const float z0 = x0 == -INFINITY ? 0.0f : x0, z1 = x1 == -INFINITY ? 0.0f : x1;
            const float d0 = exp2_sfu(M0 - z0), d1 = exp2_sfu(M1 - z1);
            M0 = x0, M1 = x1;
            l0 *= d0, l1 *= d1;
#pragma unroll
            for (int n = 0; n < kCount; ++n)
                acc[n].x *= d0, acc[n].y *= d1, acc[n].z *= d0, acc[n].w *= d1;
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const float f0 = exp2_sfu(e[j].x - z0), f1 = exp2_sfu(e[j].z - z1);
                l0 += f0 * e[j].y, l1 += f1 * e[j].w;
#pragma unroll
                for (int n = 0; n < kCount; ++n) {
                    acc[n].x += f0 * x[j][n].x, acc[n].y += f1 * x[j][n].y;
                    acc[n].z += f0 * x[j][n].z, acc[n].w += f1 * x[j][n].w;
                }
            }
        }
        __syncwarp();
        const float i0 = 1.0f / l0, i1 = 1.0f / l1;
#pragma unroll
        for (int n = 0; n < kCount; ++n)
            store(nq, n0 + kStride * n,
                  make_float4(acc[n].x * i0, acc[n].y * i1, acc[n].z * i0, acc[n].w * i1));
    }
}

template <KvStore kStore, int D, int kHeads>
__global__ void __launch_bounds__(kWdThreads, 3)
    window_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ WindowDecodeParams p)
{
    using W = WindowTraits<kStore, D>;
    constexpr int kTile = W::kTile, kMt = W::kMt, kStages = W::kStages, kDt = D / 16;
    constexpr int kNq = kHeads > 8 ? 2 : 1;      // eights of columns
    constexpr bool kTwice = kHeads == 4;         // columns 4 .. 7 are heads 0 .. 3 once more
    constexpr bool kPair = kHeads == 8;          // two products for the two parts of the weights
    constexpr bool kEight = W::kEight, kE4m3 = kStore == KvStore::kE4m3;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ uint64_t s_full[kWdWarps][kStages];
    __shared__ long long s_scan[kWdWarps], s_before[kWdThreads];
    __shared__ int s_live[kWdWarps], s_parts[kWdWarps][kWdCuts], s_last;
    __shared__ WindowPlan plan;
    // of each warp, the segment it works on and the one it fetches; what every
    // tile needs of them is kept in registers
    __shared__ WindowSegment s_seg[kWdWarps], s_fetch[kWdWarps];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;
    if (lane == 0) {
        for (int i = 0; i < kStages; ++i)
            mbar_init(smem_u32(&s_full[warp][i]), 1);
        fence_mbar_init();
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
    }
    grid_dependency_wait();
    allow_dependent_launch();

    // ---- the list of tiles and this CTA's ranges of it --------------------
    // Each thread counts the tiles of a contiguous chunk of the sequences.
    const int units = p.kv_heads * p.row_tiles;
    const int per = (p.num_seqs + kWdThreads - 1) / kWdThreads;
    const int sb0 = min(p.num_seqs, tid * per), sb1 = min(p.num_seqs, sb0 + per);
    long long mine = 0;
    int live = 0;
    for (int b = sb0; b < sb1; ++b) {
        const int len = p.lens[b];
        if ((len < 0 || len > p.max_len) && blockIdx.x == 0)
            atomicOr(p.err, PA_DEVERR_CONTEXT_LEN);
        WindowView v{};
        v.set<kTile>(len, p.max_len, p.window, p.sinks);
        mine += (long long)v.tiles * units;
        live += v.tiles > 0;
    }
    long long incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(kFullMask, incl, off);
        incl += lane >= off ? o : 0;
    }
    live = __reduce_add_sync(kFullMask, live);
    if (lane == 31)
        s_scan[warp] = incl, s_live[warp] = live;
    __syncthreads();
    long long excl = incl - mine, total = 0, all_units = 0;
#pragma unroll
    for (int w = 0; w < kWdWarps; ++w) {
        excl += w < warp ? s_scan[w] : 0;
        total += s_scan[w];
        all_units += (long long)s_live[w] * units;
    }
    if (all_units < (long long)p.num_seqs * units)  // empty contexts: their rows of out are zero
        for (int b = blockIdx.x; b < p.num_seqs; b += gridDim.x)
            if (p.lens[b] <= 0)
                for (int e = tid; e < p.heads * D / 8; e += kWdThreads)
                    reinterpret_cast<uint4 *>(p.out)[size_t(b) * p.heads * D / 8 + e] =
                        make_uint4(0, 0, 0, 0);
    if (total == 0)
        return;
    const long long ctas = gridDim.x, warps = ctas * kWdWarps;
    const bool few = all_units <= ctas / 4, little = total < kWdMuchWork * warps;
    const bool for_ctas = all_units <= ctas;
    bool ranges = all_units > warps;
    long long items = 0;
    int chunk = 0;
    if (!ranges) {                 // how long the longest part must be for one part a worker
        const long long workers = for_ctas ? ctas : warps;
        int longest[kWdCuts], sum[kWdCuts] = {};
#pragma unroll
        for (int j = 0; j < kWdCuts; ++j) {
            constexpr float kTimes[kWdCuts] = {1.25f, 1.75f};
            const float even = few ? float(total) / float(ctas - all_units)  // (always long enough)
                                   : kTimes[j] * float(total) / float(workers);
            longest[j] = max(for_ctas ? kWdTeamTiles : kWdWarpTiles, int(fminf(even, 1e9f)) + 1);
        }
        for (int b = sb0; b < sb1; ++b) {
            WindowView v{};
            v.set<kTile>(p.lens[b], p.max_len, p.window, p.sinks);
#pragma unroll
            for (int j = 0; j < kWdCuts; ++j)
                sum[j] += WindowSegment::cut(v.tiles, longest[j]) * units;
        }
        int own[kWdCuts];
#pragma unroll
        for (int j = 0; j < kWdCuts; ++j) {
            own[j] = sum[j];
            sum[j] = __reduce_add_sync(kFullMask, sum[j]);
            if (lane == 0)
                s_parts[warp][j] = sum[j];
        }
        __syncthreads();
        int pick = 0, parts = 0;
        bool fits = false;
#pragma unroll
        for (int j = kWdCuts - 1; j >= 0; --j) {
            int all = 0;
#pragma unroll
            for (int w = 0; w < kWdWarps; ++w)
                all += s_parts[w][j];
            if (j == kWdCuts - 1 || all <= workers)
                pick = j, parts = own[j], chunk = longest[j], items = all, fits = all <= workers;
        }
        const bool alike = float(chunk) * float(items) <= kWdAlike * float(total);
        ranges = !(few || little || (fits && alike && (!kEight || pick < kWdCuts8)));
        if (!ranges) {             // the same scan for the parts
            int upto = parts;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(kFullMask, upto, off);
                upto += lane >= off ? o : 0;
            }
            excl = upto - parts;
#pragma unroll
            for (int w = 0; w < kWdWarps; ++w)
                excl += w < warp ? s_parts[w][pick] : 0;
        }
    }
    const bool team = for_ctas && !ranges;
    s_before[tid] = excl;
    if (tid == 0)
        plan = WindowPlan{items, total, team ? ctas : warps, s_before, ranges, chunk, units, per};
    __syncthreads();
    const long long worker = team ? (long long)blockIdx.x : (long long)warp * ctas + blockIdx.x;

    WindowSegment seg;
    if (!ranges) {
        seg.item = worker;
        seg.left = 0;
        if (!seg.locate<kTile>(p, plan))
            return;                // (for a CTA's part, all warps)
    } else {
        // the range's two cuts: lane 0 its begin, lane 1 its end
        long long cut_x = (worker + (lane & 1)) * total / warps, cut_u0 = 0;
        int cut_b = 0, cut_r = 0;
        if (lane < 2 && cut_x < total) {
            int t = 0;             // last thread whose sequences begin at or before the cut
#pragma unroll
            for (int half = kWdThreads / 2; half >= 1; half >>= 1)
                if (s_before[t + half] <= cut_x)
                    t += half;
            long long at = s_before[t];
            int b = t * per;
            WindowView v{};
            for (;; ++b) {
                v.set<kTile>(p.lens[b], p.max_len, p.window, p.sinks);
                const long long n = (long long)v.tiles * units;
                if (cut_x < at + n)
                    break;
                at += n;
            }
            int r = int((cut_x - at) / v.tiles);
            cut_u0 = at + (long long)r * v.tiles;
            const long long before = cut_x - cut_u0, behind = v.tiles - before;
            if (before <= kWdSnap && before <= behind) {
                cut_x = cut_u0;
            } else if (behind <= kWdSnap) {
                cut_x = cut_u0 = cut_u0 + v.tiles;
                if (++r == units) {
                    r = 0;
                    do {
                        ++b;
                        if (b < p.num_seqs)
                            v.set<kTile>(p.lens[b], p.max_len, p.window, p.sinks);
                    } while (b < p.num_seqs && v.tiles == 0);
                }
            } else if (before <= kWdSnap) {
                cut_x = cut_u0;
            }
            cut_b = b, cut_r = r;
        }
        const long long lo = __shfl_sync(kFullMask, cut_x, 0), hi = __shfl_sync(kFullMask, cut_x, 1);
        if (lo >= hi)
            return;
        seg.b = __shfl_sync(kFullMask, cut_b, 0);
        seg.r = __shfl_sync(kFullMask, cut_r, 0);
        seg.item = __shfl_sync(kFullMask, cut_u0, 0);
        seg.view.set<kTile>(p.lens[seg.b], p.max_len, p.window, p.sinks);
        seg.begin = int(lo - seg.item);
        seg.end = int(min((long long)seg.view.tiles, seg.begin + hi - lo));
        seg.left = hi - lo - (seg.end - seg.begin);
        seg.part = seg.parts = 0;
    }

    // ---- the warp's stream of tiles --------------------------------------
    const uint32_t ring = smem_u32(smem) + uint32_t(warp * kStages) * W::kStageBytes;
    const uint64_t policy = l2_policy_evict_first();
    const int step = team ? kWdWarps : 1, sub = team ? warp : 0;
    const int bs = 1 << p.log2_bs;
    const int log2_run = min(p.log2_bs, __ffs(kTile) - 1), run = 1 << log2_run;  // rows of one box
    const int runs = kTile >> log2_run;

    int ii = seg.begin + sub;      // the next tile to fetch, of a unit of head fh of sequence fb
    int f_end = seg.end, fb = seg.b, fh = seg.r / p.row_tiles;
    WindowView fv = seg.view;
    bool more = true, dead = false;
    if (lane == 0)
        s_seg[warp] = s_fetch[warp] = seg;
    __syncwarp();
    int id = -2;                   // lane j: block of the tile's run j; -2: nothing of it is seen
    auto settle = [&]() {          // move to the warp's next tile and look up its blocks
        while (more && ii >= f_end) {
            WindowSegment next = s_fetch[warp];
            more = next.next<kTile>(p, plan);
            __syncwarp();
            if (lane == 0)
                s_fetch[warp] = next;
            __syncwarp();
            ii = next.begin + sub;
            f_end = next.end, fb = next.b, fh = next.r / p.row_tiles;
            fv = next.view;
        }
        id = -2;
        if (more && lane < runs) {
            const int t = fv.token<kTile>(ii) + (lane << log2_run);
            if (t < fv.L && (t + run > fv.ws || t < p.sinks))
                id = __ldg(p.tables + size_t(fb) * p.max_blocks + (t >> p.log2_bs));
        }
    };
    float2 coming = make_float2(0.0f, 0.0f);  // lane j: scales of run j of the tile fetched last
    auto issue = [&](int stage) {
        if (!more || dead)
            return;
        const int t = fv.token<kTile>(ii) + (lane << log2_run);
        const bool ok = unsigned(id) < unsigned(p.num_blocks);
        if (id != -2 && !ok)
            atomicOr(p.err, PA_DEVERR_BLOCK_ID);
        const uint32_t bar = smem_u32(&s_full[warp][stage]);
        const unsigned there = __ballot_sync(kFullMask, ok);
        if (lane == 0)
            mbar_arrive_expect_tx(bar, uint32_t(__popc(there)) * uint32_t(2 * W::kRowBytes) << log2_run);
        __syncwarp();
        if (ok) {
            const long long row = (((long long)id * p.kv_heads + fh) << p.log2_bs) + (t & (bs - 1));
            const uint32_t dst = ring + uint32_t(stage) * W::kStageBytes +
                                 (uint32_t(lane) << log2_run) * uint32_t(W::kRowBytes);
            if constexpr (kEight) {      // 128-byte lines
                const int y = int(row * W::kRowBytes / 128);
                tma_load_2d_hint(dst, &tm_k, 0, y, bar, policy);
                tma_load_2d_hint(dst + 4096u, &tm_v, 0, y, bar, policy);
            } else {                     // groups of 8 rows
                tma_load_4d_hint(dst, &tm_k, 0, 0, 0, int(row >> 3), bar, policy);
                tma_load_4d_hint(dst + 4096u, &tm_v, 0, 0, 0, int(row >> 3), bar, policy);
            }
        }
        if constexpr (kEight)
            coming = ok ? __ldg(p.scales + (long long)id * p.scale_heads + fh) : make_float2(0.0f, 0.0f);
        ii += step;
        settle();
    };
    settle();
    issue(0);

    int stage = 0;
    uint32_t phase = 0;
    bool have = true;
    while (have) {
        const int h = s_seg[warp].r / p.row_tiles, row0 = (s_seg[warp].r % p.row_tiles) * kHeads;
        const int rows = min(kHeads, p.group - row0);
        const size_t out_row = size_t(s_seg[warp].b) * p.heads + size_t(h) * p.group + row0;

        // ---- query heads as the columns (B operand) ----------------------
        uint32_t qb[kNq][kDt][2];
        float f[kNq][2];           // what the scores of columns 2c, 2c + 1 are multiplied by
#pragma unroll
        for (int nq = 0; nq < kNq; ++nq) {
            const int mine = 8 * nq + (kTwice ? g & 3 : g);
            const bool there = mine < rows;
            const uint16_t *src = static_cast<const uint16_t *>(p.q) + (out_row + (there ? mine : 0)) * D;
            if constexpr (!kEight) {
                const uint32_t *w = reinterpret_cast<const uint32_t *>(src) + c;
#pragma unroll
                for (int k = 0; k < kDt; ++k) {
                    qb[nq][k][0] = there ? __ldg(w + 8 * k) : 0u;
                    qb[nq][k][1] = there ? __ldg(w + 8 * k + 4) : 0u;
                }
                f[nq][0] = f[nq][1] = p.scale_log2;
            } else {
                // 16 dims from each 16-byte chunk of codes that the lane reads
                float x[D / 4];
                float m = 0.0f;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint4 v = there ? __ldg(reinterpret_cast<const uint4 *>(
                                                src + (c + 4 * (i >> 1)) * 16 + 8 * (i & 1)))
                                          : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 y = p.bf16 ? Half16<true>::unpack(w[e]) : Half16<false>::unpack(w[e]);
                        x[8 * i + 2 * e] = y.x;
                        x[8 * i + 2 * e + 1] = y.y;
                        m = fmaxf(m, fmaxf(fabsf(y.x), fabsf(y.y)));
                    }
                }
                m = fmaxf(m, __shfl_xor_sync(kFullMask, m, 1));
                m = fmaxf(m, __shfl_xor_sync(kFullMask, m, 2));
                // power of two that brings the largest component to [2^14, 2^15)
                const int e2 = m > 0.0f ? min(max(141 - int(__float_as_uint(m) >> 23), -100), 100) : 0;
                const float up = __uint_as_float(uint32_t(127 + e2) << 23);
                const float down = p.scale_log2 * __uint_as_float(uint32_t(127 - e2) << 23);
#pragma unroll
                for (int k = 0; k < kDt; ++k) {
                    qb[nq][k][0] = Half16<false>::pack(x[4 * k] * up, x[4 * k + 1] * up);
                    qb[nq][k][1] = Half16<false>::pack(x[4 * k + 2] * up, x[4 * k + 3] * up);
                }
                f[nq][0] = __shfl_sync(kFullMask, down, 8 * c);
                f[nq][1] = __shfl_sync(kFullMask, down, 8 * c + 4);
            }
        }

        // o[.][dt]: dims of 16-row dt, rows g (x, y) and g + 8 (z, w), columns
        // 2c (x, z) and 2c + 1 (y, w); m and l of the same columns
        float o[kNq][kDt][4], m[kNq][2], l[kNq][2];
#pragma unroll
        for (int nq = 0; nq < kNq; ++nq) {
#pragma unroll
            for (int i = 0; i < kDt; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[nq][i][e] = 0.0f;
            m[nq][0] = m[nq][1] = -INFINITY;
            l[nq][0] = l[nq][1] = 0.0f;
        }
        float sv_ref = 0.0f, sv_inv = 0.0f;

        const WindowView view = s_seg[warp].view;
        const int end = s_seg[warp].end;
        for (int i = s_seg[warp].begin + sub; i < end; i += step) {
            const float2 sc = coming;
            issue(stage ^ 1);
            if (!dead && !mbar_wait_bounded(smem_u32(&s_full[warp][stage]), phase)) {
                atomicOr(p.err, PA_DEVERR_TIMEOUT);
                // once more for the copies in flight, which must not land
                // after the block has ended
                mbar_wait_bounded(smem_u32(&s_full[warp][stage]), phase);
                mbar_wait_bounded(smem_u32(&s_full[warp][stage ^ 1]), phase ^ uint32_t(stage));
                dead = true;
            }
            dead = __any_sync(kFullMask, dead);
            const uint32_t kt = ring + uint32_t(stage) * W::kStageBytes, vt = kt + 4096u;
            const int t0 = view.token<kTile>(i);
            const bool edge = t0 + kTile > view.L || (t0 < view.ws && t0 + kTile > p.sinks);
            if (edge) {            // hidden rows of V must not reach the product
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    constexpr int kChunks = W::kRowBytes / 16;
                    const int row = (e * 32 + lane) / kChunks, chunk = (e * 32 + lane) % kChunks;
                    if (!view.sees(t0 + row, p.sinks))
                        sts128_zero(vt + W::at(row, chunk));
                }
                fence_proxy_async_smem();
                __syncwarp();
            }

            // ---- scores: tokens x query heads -----------------------------
            float s[kMt][kNq][4];
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt) {
#pragma unroll
                for (int nq = 0; nq < kNq; ++nq)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[mt][nq][e] = 0.0f;
                if constexpr (!kEight) {
                    const uint32_t base = kt + W::at(16 * mt + (lane & 15), lane >> 4);
#pragma unroll
                    for (int k = 0; k < kDt; ++k) {
                        uint32_t a[4];
                        ldmatrix_x4((base ^ uint32_t((k & 3) * 32)) + uint32_t(k >> 2) * 1024u, a);
#pragma unroll
                        for (int nq = 0; nq < kNq; ++nq)
                            mma16816<W::kBf16>(s[mt][nq], a, qb[nq][k][0], qb[nq][k][1]);
                    }
                } else {
                    uint32_t w[2][kDt];
#pragma unroll
                    for (int high = 0; high < 2; ++high)
#pragma unroll
                        for (int k = 0; k < D / 64; ++k) {
                            const uint4 v = lds128(kt + W::at(16 * mt + W::token_of(g, high), c + 4 * k));
                            w[high][4 * k] = v.x, w[high][4 * k + 1] = v.y;
                            w[high][4 * k + 2] = v.z, w[high][4 * k + 3] = v.w;
                        }
#pragma unroll
                    for (int k = 0; k < kDt; ++k) {
                        uint32_t a[4];
                        widen4<kE4m3>(w[0][k], a[0], a[2]);
                        widen4<kE4m3>(w[1][k], a[1], a[3]);
#pragma unroll
                        for (int nq = 0; nq < kNq; ++nq)
                            mma16816<false>(s[mt][nq], a, qb[nq][k][0], qb[nq][k][1]);
                    }
                }
            }
            float ratio[kMt][2];   // s_v of rows g, g + 8 over the running reference
            if constexpr (kEight) {
                const float top = pow2_at_least(
                    __uint_as_float(__reduce_max_sync(kFullMask, __float_as_uint(fmaxf(sc.y, 0.0f)))));
                if (top > sv_ref) {
                    const float down = sv_ref / top;
#pragma unroll
                    for (int nq = 0; nq < kNq; ++nq)
#pragma unroll
                        for (int n = 0; n < kDt; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                o[nq][n][e] *= down;
                    sv_ref = top;
                    sv_inv = 1.0f / top;
                }
#pragma unroll
                for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
                    for (int high = 0; high < 2; ++high) {
                        const int from = (16 * mt + W::token_of(g, high)) >> log2_run;
                        const float sk = __shfl_sync(kFullMask, sc.x, from);
                        ratio[mt][high] = __shfl_sync(kFullMask, sc.y, from) * sv_inv;
#pragma unroll
                        for (int nq = 0; nq < kNq; ++nq) {
                            s[mt][nq][2 * high] *= f[nq][0] * sk;
                            s[mt][nq][2 * high + 1] *= f[nq][1] * sk;
                        }
                    }
            } else {
#pragma unroll
                for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
                    for (int nq = 0; nq < kNq; ++nq)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s[mt][nq][e] *= p.scale_log2;
            }
            if (edge) {
#pragma unroll
                for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
                    for (int high = 0; high < 2; ++high)
                        if (!view.sees(t0 + 16 * mt + W::token_of(g, high), p.sinks))
#pragma unroll
                            for (int nq = 0; nq < kNq; ++nq)
                                s[mt][nq][2 * high] = s[mt][nq][2 * high + 1] = -INFINITY;
            }

            // ---- reference of the softmax ---------------------------------
            bool grows = false;
#pragma unroll
            for (int nq = 0; nq < kNq; ++nq)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = -INFINITY;
#pragma unroll
                    for (int mt = 0; mt < kMt; ++mt)
                        x = fmaxf(x, fmaxf(s[mt][nq][e], s[mt][nq][e + 2]));
                    grows |= x > m[nq][e] + kWdRescale;
                }
            if (__any_sync(kFullMask, grows)) {
#pragma unroll
                for (int nq = 0; nq < kNq; ++nq)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = m[nq][e];
#pragma unroll
                        for (int mt = 0; mt < kMt; ++mt)
                            x = fmaxf(x, fmaxf(s[mt][nq][e], s[mt][nq][e + 2]));
                        x = fmaxf(x, __shfl_xor_sync(kFullMask, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(kFullMask, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(kFullMask, x, 16));
                        const float down = x > m[nq][e] ? exp2_sfu(m[nq][e] - x) : 1.0f;
                        m[nq][e] = x;
                        l[nq][e] *= down;
#pragma unroll
                        for (int n = 0; n < kDt; ++n) {
                            o[nq][n][e] *= down;
                            o[nq][n][e + 2] *= down;
                        }
                    }
            }

            // ---- weights and the product with V: dims x query heads --------
            // a column whose scores are all -inf so far keeps weights of zero
            float z[kNq][2];
#pragma unroll
            for (int nq = 0; nq < kNq; ++nq)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    z[nq][e] = (m[nq][e] == -INFINITY ? 0.0f : m[nq][e]) - p.shift;
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt) {
                uint32_t pb[kNq][2], pr[kNq][2];  // most of the weights, and the rest
#pragma unroll
                for (int nq = 0; nq < kNq; ++nq)
#pragma unroll
                    for (int high = 0; high < 2; ++high) {
                        float w0 = exp2_sfu(s[mt][nq][2 * high] - z[nq][0]);
                        float w1 = exp2_sfu(s[mt][nq][2 * high + 1] - z[nq][1]);
                        l[nq][0] += w0;
                        l[nq][1] += w1;
                        if constexpr (kEight) {
                            w0 *= ratio[mt][high];
                            w1 *= ratio[mt][high];
                        }
                        if constexpr (kNq == 2) {
                            pb[nq][high] = movmatrix_trans(Half16<W::kBf16>::pack(w0, w1));
                        } else {
                            const uint32_t most = most_of<kStore>(w0, w1);
                            const float2 x = Half16<W::kBf16>::unpack(most);
                            const uint32_t rest = Half16<W::kBf16>::pack(w0 - x.x, w1 - x.y);
                            pb[nq][high] = movmatrix_trans(kTwice && c >= 2 ? rest : most);
                            if constexpr (kPair)
                                pr[nq][high] = movmatrix_trans(rest);
                        }
                    }
                if constexpr (!kEight) {
                    const uint32_t base = vt + W::at(16 * mt + (lane & 7) + 8 * (lane >> 4), (lane >> 3) & 1);
#pragma unroll
                    for (int n = 0; n < kDt; ++n) {
                        uint32_t a[4];
                        ldmatrix_x4_trans((base ^ uint32_t((n & 3) * 32)) + uint32_t(n >> 2) * 1024u, a);
#pragma unroll
                        for (int nq = 0; nq < kNq; ++nq) {
                            mma16816<W::kBf16>(o[nq][n], a, pb[nq][0], pb[nq][1]);
                            if constexpr (kPair)
                                mma16816<W::kBf16>(o[nq][n], a, pr[nq][0], pr[nq][1]);
                        }
                    }
                } else {
                    // lane (g, c): codes of tokens 4c .. 4c + 3 of dims g and g + 8
                    // of 16-dim chunks 2n, 2n + 1
                    const int row = 16 * mt + (lane & 15), high = lane >> 4;
#pragma unroll
                    for (int n = 0; n < kDt / 2; ++n) {
                        uint32_t w[4];
                        ldmatrix_x2_trans8(vt + W::at(row, 2 * n + high), w);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            uint32_t a[4];
                            widen4<kE4m3>(w[2 * e], a[0], a[2]);
                            widen4<kE4m3>(w[2 * e + 1], a[1], a[3]);
#pragma unroll
                            for (int nq = 0; nq < kNq; ++nq) {
                                mma16816<false>(o[nq][2 * n + e], a, pb[nq][0], pb[nq][1]);
                                if constexpr (kPair)
                                    mma16816<false>(o[nq][2 * n + e], a, pr[nq][0], pr[nq][1]);
                            }
                        }
                    }
                }
            }
            __syncwarp();  // the stage may be filled again
            stage ^= 1;
            phase ^= stage == 0 ? 1u : 0u;
        }

        // ---- the end of the unit, or of the range's part of it --------------
        WindowSegment seg = s_seg[warp];
        const bool whole = seg.begin == 0 && seg.end == seg.view.tiles;
#pragma unroll
        for (int nq = 0; nq < kNq; ++nq) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int off = 4; off < 32; off <<= 1)
                    l[nq][e] += __shfl_xor_sync(kFullMask, l[nq][e], off);
            if constexpr (kEight) {
                // up to 2^30 weights of up to 2^15: a large s_v finds room for
                // their sum under a reference that is larger by as much
                const bool huge = sv_ref > 0x1p64f;
                const float down = huge ? 0x1p-45f : 1.0f;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    l[nq][e] *= down;
                    m[nq][e] += huge ? 45.0f : 0.0f;
                }
#pragma unroll
                for (int n = 0; n < kDt; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[nq][n][e] *= down * sv_ref;
            }
        }
        if constexpr (kTwice)
#pragma unroll
            for (int n = 0; n < kDt; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[0][n][e] += __shfl_xor_sync(kFullMask, o[0][n][e], 2);
        // 16 dims of 8 query heads, from fragment to rows of out
        const bool bf = kEight ? p.bf16 != 0 : W::kBf16;
        auto store = [&](int nq, int n, const float4 &v) {
            uint32_t lo2 = bf ? Half16<true>::pack(v.x, v.y) : Half16<false>::pack(v.x, v.y);
            uint32_t hi2 = bf ? Half16<true>::pack(v.z, v.w) : Half16<false>::pack(v.z, v.w);
            lo2 = movmatrix_trans(lo2);
            hi2 = movmatrix_trans(hi2);
            if (8 * nq + g < rows) {
                uint16_t *dst = static_cast<uint16_t *>(p.out) + (out_row + 8 * nq + g) * D;
                *reinterpret_cast<uint32_t *>(dst + 16 * n + 2 * c) = lo2;
                *reinterpret_cast<uint32_t *>(dst + 16 * n + 8 + 2 * c) = hi2;
            }
        };
        // Parts of the unit, and their slots.  With ranges, the parts lie
        // between the cuts that stayed inside the unit; the first is its
        // range's last segment, the others are their ranges' first.
        long long first = seg.item - seg.part;
        int parts = seg.parts, part = seg.part;
        if (ranges && !whole) {
            first = ceil_div((seg.item + kWdSnap + 1) * plan.workers, plan.total) - 1;
            parts = int(ceil_div((seg.item + seg.view.tiles - kWdSnap) * plan.workers, plan.total) - 1 -
                        first) + 1;
            part = int((long long)warp * gridDim.x + blockIdx.x - first);
        }
        auto slot_of = [&](int k) {
            return size_t(ranges ? 2 * (first + k) + (k == 0 ? 1 : 0) : first + k);
        };
        const size_t slot = slot_of(part);
        auto part_o = [&](size_t sl, int nq, int n) {
            return p.part_o + ((sl * kNq + nq) * kDt + n) * 32 + lane;
        };
        auto part_ml = [&](size_t sl, int nq) { return p.part_ml + (sl * kNq + nq) * 4 + c; };

        if (!team) {
#pragma unroll
            for (int nq = 0; nq < kNq; ++nq) {
                if (whole) {
                    const float i0 = 1.0f / l[nq][0], i1 = 1.0f / l[nq][1];
#pragma unroll
                    for (int n = 0; n < kDt; ++n)
                        store(nq, n, make_float4(o[nq][n][0] * i0, o[nq][n][1] * i1, o[nq][n][2] * i0,
                                                 o[nq][n][3] * i1));
                } else if (8 * nq + 2 * c < rows) {
#pragma unroll
                    for (int n = 0; n < kDt; ++n)
                        __stcg(part_o(slot, nq, n),
                               make_float4(o[nq][n][0], o[nq][n][1], o[nq][n][2], o[nq][n][3]));
                    if (g == 0)
                        __stcg(part_ml(slot, nq), make_float4(m[nq][0], l[nq][0], m[nq][1], l[nq][1]));
                }
            }
        } else {
            float4 *mo = reinterpret_cast<float4 *>(smem + W::kOffMerge);
            float2 *ml = reinterpret_cast<float2 *>(smem + W::kOffMl);
#pragma unroll
            for (int nq = 0; nq < kNq; ++nq)
#pragma unroll
                for (int pass = 0; pass < kDt / 4; ++pass) {
                    __syncthreads();  // the merge buffer is free
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float(&x)[4] = o[nq][4 * pass + i];
                        mo[(warp * 4 + i) * 32 + lane] = make_float4(x[0], x[1], x[2], x[3]);
                    }
                    if (g == 0) {
                        ml[warp * 8 + 2 * c] = make_float2(m[nq][0], l[nq][0]);
                        ml[warp * 8 + 2 * c + 1] = make_float2(m[nq][1], l[nq][1]);
                    }
                    __syncthreads();
                    float M0 = -INFINITY, M1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
#pragma unroll
                    for (int w = 0; w < kWdWarps; ++w) {
                        M0 = fmaxf(M0, ml[w * 8 + 2 * c].x);
                        M1 = fmaxf(M1, ml[w * 8 + 2 * c + 1].x);
                    }
                    const float z0 = M0 == -INFINITY ? 0.0f : M0, z1 = M1 == -INFINITY ? 0.0f : M1;
                    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int w = 0; w < kWdWarps; ++w) {
                        const float2 a = ml[w * 8 + 2 * c], b = ml[w * 8 + 2 * c + 1];
                        const float f0 = exp2_sfu(a.x - z0), f1 = exp2_sfu(b.x - z1);
                        const float4 x = mo[(w * 4 + warp) * 32 + lane];
                        l0 += f0 * a.y, l1 += f1 * b.y;
                        acc.x += f0 * x.x, acc.y += f1 * x.y, acc.z += f0 * x.z, acc.w += f1 * x.w;
                    }
                    const int n = 4 * pass + warp;
                    if (whole) {
                        const float i0 = 1.0f / l0, i1 = 1.0f / l1;
                        store(nq, n, make_float4(acc.x * i0, acc.y * i1, acc.z * i0, acc.w * i1));
                    } else if (8 * nq + 2 * c < rows) {
                        __stcg(part_o(slot, nq, n), acc);
                        if (warp == 0 && pass == 0 && g == 0)
                            __stcg(part_ml(slot, nq), make_float4(M0, l0, M1, l1));
                    }
                }
        }

        // ---- the last of a straddling unit's parts merges them ---------------
        if (!whole) {
            unsigned *ticket = p.tickets + (size_t(seg.b) * plan.units + seg.r);
            bool last;
            __threadfence();
            if (team) {
                __syncthreads();
                if (tid == 0)
                    s_last = atomicInc(ticket, unsigned(parts - 1)) == unsigned(parts - 1);
                __syncthreads();
                last = s_last;
            } else {
                __syncwarp();
                last = lane == 0 && atomicInc(ticket, unsigned(parts - 1)) == unsigned(parts - 1);
                last = __shfl_sync(kFullMask, int(last), 0) != 0;
            }
            if (last) {
                __threadfence();
                // a CTA's warps take every fourth 16 dims each
                if (team)
                    merge_parts<kDt / 4, 4>(parts, slot_of, part_ml, part_o, store, kNq, warp, c, rows);
                else
                    merge_parts<kDt, 1>(parts, slot_of, part_ml, part_o, store, kNq, 0, c, rows);
            }
        }
        have = seg.next<kTile>(p, plan);
        __syncwarp();
        if (lane == 0)
            s_seg[warp] = seg;
        __syncwarp();
    }
}

} // namespace pa
