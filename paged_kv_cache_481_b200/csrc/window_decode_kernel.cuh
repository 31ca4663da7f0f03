// One-query attention over the paged cache with a sliding window, a few first
// tokens that stay visible, and grouped heads, for 16-bit caches and for the
// 8-bit cache with one scale per (block, head).
//
// Mathematics: the query at p = L - 1 sees t < L with t >= ws = max(0, L -
// window) or t < sinks; out = sum_t w_t V_t / sum_t w_t with w_t =
// 2^(c s_t - m), taken in one pass over the visible tokens with the running
// maximum m (online softmax in base 2).
//
// What bounds it: reading K and V once, 4 D bytes a token and K/V head for
// about 4 D flops a query head and token, so memory as long as the matrix
// work is not done on scalar units.  The G query heads of a K/V head are the
// rows of a 16-row warp matrix product, so K and V are read once per group
// and a tile costs the same few instructions for any G <= 16.
//
// Layout of the work: a "unit" is (sequence, K/V head, 16 query heads); its
// visible tokens are cut into tiles of 4 KB of K and 4 KB of V (16 tokens at
// D = 128 in 16 bits).  The tiles of all units, unit after unit, are cut into
// equal contiguous ranges, one per CTA; within a range the tiles of a unit go
// to the CTA's warps in turn.  Each warp has its own ring of kStages tiles,
// filled by 16-byte asynchronous copies (rows that are not seen are written
// as zeros and not read) and keeps it full across units.  Rows of 128 bytes
// and more are XOR-swizzled in shared memory, so matrix loads have no bank
// conflicts.  The warps' results of a unit are merged in shared memory; a
// unit that straddles CTAs leaves partial results in the workspace, and the
// last CTA to arrive merges them in CTA order, so that the result does not
// depend on the order of arrival.
//
// Choices of fewer bits: the weights enter the product with V in 16 bits.
// They are taken 2^14 times larger than the softmax's (numerator and
// denominator alike), which keeps weights down to 2^-38 of the largest in
// fp16 instead of losing those under 2^-24.  With 8-bit codes the products
// are fp16 (codes are exact in it): the query row is scaled by a power of two
// so that its largest component is near 2^14, exact for every component above
// 2^-28 of it; a block's s_v is folded into its weights relative to a running
// power of two at or above the largest s_v so far.
#pragma once

#include <cstdint>

#include "../../include/pa_window.h"
#include "half_types.cuh"
#include "mma_sync.cuh"
#include "ptx.cuh"

namespace pa {

enum class KvStore { kF16, kBf16, kInt8, kE4m3 };

struct WindowDecodeParams {
    void *out;                  // [B, H, D]
    const void *q;              // [B, H, D]
    const void *k, *v;          // caches or codes [NB, KVH, bs, D]
    const float2 *scales;       // [NB, scale_heads] (8-bit)
    const int32_t *tables;      // [B, max_blocks]
    const int32_t *lens;        // [B]
    int max_blocks, max_len, window, sinks;
    int num_seqs, heads, kv_heads, group, row_tiles;  // row_tiles = ceil(group / 16)
    int log2_bs, num_blocks, scale_heads;
    int bf16;                   // type of q and out
    float scale_log2;           // softmax scale * log2(e)
    int min_tiles;              // least tiles per CTA
    float *part_o;              // [2 * CTAs, 16, D]
    float2 *part_ml;            // [2 * CTAs, 16] (m, l)
    unsigned *tickets;          // [units]
    unsigned *err;
};

constexpr int kWdWarps = 4;
constexpr int kWdThreads = kWdWarps * 32;
constexpr int kWdMaxCtas = 512;
constexpr float kWdShift = 14.0f;   // weights are 2^14 times the softmax's

template <KvStore kStore, int D>
struct WindowTraits {
    static constexpr bool kEight = kStore == KvStore::kInt8 || kStore == KvStore::kE4m3;
    static constexpr bool kBf16 = kStore == KvStore::kBf16;
    static constexpr int kStages = 3;
    static constexpr int kRowBytes = D * (kEight ? 1 : 2);
    static constexpr int kTile = 4096 / kRowBytes;        // tokens per tile
    static constexpr int kGroups = kTile / 8;             // 8-token groups: one block each
    static constexpr int kChunks = kRowBytes / 16;        // 16-byte chunks per row
    static constexpr int kRowsPerCopy = 32 / kChunks;     // rows one warp-wide copy covers
    static constexpr int kScaleBytes = kEight ? kGroups * 8 : 0;
    static constexpr int kStageBytes = 8192;
    static constexpr int kPitch = 64 + 8;                 // merge rows of 64 dims, no bank conflicts
    static constexpr int kOffMerge = kWdWarps * kStages * kStageBytes;
    static constexpr int kOffMl = kOffMerge + kWdWarps * 8 * kPitch * 4;
    static constexpr int kOffScales = kOffMl + kWdWarps * 16 * 8;
    static constexpr int kSmem = kOffScales + kWdWarps * kStages * kScaleBytes;

    // Byte offset of a 16-byte chunk of a row in a swizzled tile.
    static __device__ __forceinline__ uint32_t at(int row, int chunk)
    {
        if constexpr (kRowBytes >= 128) {
            return uint32_t(row * kRowBytes + ((chunk ^ (row & 7)) << 4));
        } else {  // two 64-byte rows share a 128-byte line
            const int line = row >> 1;
            return uint32_t(line * 128 + (((((row & 1) << 2) | chunk) ^ ((line & 3) << 1)) << 4));
        }
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

// A stretch [i, end) of one unit's tiles that belongs to this CTA, and what
// of the CTA's range is left behind it.
struct WindowSegment {
    int b, r;              // sequence, unit within the sequence
    int begin, end;
    long long left;
    WindowView view;

    template <int kTile>
    __device__ __forceinline__ bool next(const WindowDecodeParams &p, int units)
    {
        if (left <= 0)
            return false;
        if (++r == units) {
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
        const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w & 0xffffu), __NV_E4M3);
        const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w >> 16), __NV_E4M3);
        lo = uint32_t(a.x) | (uint32_t(a.y) << 16);
        hi = uint32_t(b.x) | (uint32_t(b.y) << 16);
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

// Smallest power of two >= x (x >= 0; infinity stays, NaN gives 0).
__device__ __forceinline__ float pow2_at_least(float x)
{
    return __uint_as_float((__float_as_uint(x) + 0x7fffffu) & 0x7f800000u);
}

template <KvStore kStore, int D>
__global__ void __launch_bounds__(kWdThreads, 2) window_decode_kernel(const WindowDecodeParams p)
{
    using W = WindowTraits<kStore, D>;
    constexpr int kTile = W::kTile, kNT = W::kGroups, kStages = W::kStages;
    constexpr bool kEight = W::kEight, kE4m3 = kStore == KvStore::kE4m3;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long s_scan[kWdWarps];
    __shared__ long long s_start;    // first tile of the unit the range begins in
    __shared__ int s_b, s_r, s_last;

    grid_dependency_wait();
    allow_dependent_launch();

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;
    const int units = p.kv_heads * p.row_tiles;

    // ---- this CTA's range of the tile list -------------------------------
    // Each thread counts the tiles of a contiguous chunk of the sequences; a
    // block scan gives the total and the chunk the range begins in.
    const int per = (p.num_seqs + kWdThreads - 1) / kWdThreads;
    const int sb0 = min(p.num_seqs, tid * per), sb1 = min(p.num_seqs, sb0 + per);
    long long mine = 0;
    for (int b = sb0; b < sb1; ++b) {
        const int len = p.lens[b];
        if ((len < 0 || len > p.max_len) && blockIdx.x == 0)
            atomicOr(p.err, PA_DEVERR_CONTEXT_LEN);
        WindowView v{};
        v.set<kTile>(len, p.max_len, p.window, p.sinks);
        mine += (long long)v.tiles * units;
    }
    long long incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(kFullMask, incl, off);
        if (lane >= off)
            incl += o;
    }
    if (lane == 31)
        s_scan[warp] = incl;
    __syncthreads();
    long long base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kWdWarps; ++w) {
        base += w < warp ? s_scan[w] : 0;
        total += s_scan[w];
    }
    // empty contexts: their rows of out are zero
    for (int b = blockIdx.x; b < p.num_seqs; b += gridDim.x)
        if (p.lens[b] <= 0)
            for (int e = tid; e < p.heads * D / 8; e += kWdThreads)
                reinterpret_cast<uint4 *>(p.out)[size_t(b) * p.heads * D / 8 + e] = make_uint4(0, 0, 0, 0);
    const long long ctas = max(1ll, min((long long)gridDim.x, total / p.min_tiles));
    if (blockIdx.x >= ctas || total == 0)
        return;
    const long long lo = blockIdx.x * total / ctas, hi = (blockIdx.x + 1) * total / ctas;
    const long long excl = base + incl - mine;
    if (excl <= lo && lo < excl + mine) {
        long long at = excl;
        for (int b = sb0; b < sb1; ++b) {
            WindowView v{};
            v.set<kTile>(p.lens[b], p.max_len, p.window, p.sinks);
            const long long n = (long long)v.tiles * units;
            if (lo < at + n) {
                s_b = b;
                s_r = int((lo - at) / v.tiles);
                s_start = at + (long long)s_r * v.tiles;
                break;
            }
            at += n;
        }
    }
    __syncthreads();

    WindowSegment seg;
    seg.b = s_b;
    seg.r = s_r;
    seg.view.set<kTile>(p.lens[seg.b], p.max_len, p.window, p.sinks);
    seg.begin = int(lo - s_start);
    seg.end = int(min((long long)seg.view.tiles, seg.begin + hi - lo));
    seg.left = hi - lo - (seg.end - seg.begin);

    // ---- the warp's stream of tiles --------------------------------------
    const uint32_t sbase = smem_u32(smem);
    const uint32_t ring = sbase + uint32_t(warp * kStages) * W::kStageBytes;
    const uint32_t sring = sbase + W::kOffScales + uint32_t(warp * kStages) * W::kScaleBytes;
    const uint64_t policy = l2_policy_evict_first();
    const int bs = 1 << p.log2_bs;
    const unsigned char *kbase = static_cast<const unsigned char *>(p.k);
    const unsigned char *vbase = static_cast<const unsigned char *>(p.v);

    WindowSegment is = seg;        // where the next tile to fetch lies
    int ii = is.begin + warp;
    bool more = true;
    int id = -1;                   // lane j: block of the tile's 8-token group j, if it is seen
    auto settle = [&]() {          // move to the warp's next tile and look up its blocks
        while (more && ii >= is.end) {
            more = is.next<kTile>(p, units);
            ii = is.begin + warp;
        }
        id = -2;                   // -2: nothing of the group is seen
        if (more && lane < kNT) {
            const int t = is.view.token<kTile>(ii) + 8 * lane;
            if (t < is.view.L && (t + 7 >= is.view.ws || t < p.sinks))
                id = __ldg(p.tables + size_t(is.b) * p.max_blocks + (t >> p.log2_bs));
        }
    };
    auto issue = [&](int stage) {
        if (more) {
            const int t0 = is.view.token<kTile>(ii);
            const int h = is.r / p.row_tiles;
            const bool ok = unsigned(id) < unsigned(p.num_blocks);
            if (id != -2 && !ok)
                atomicOr(p.err, PA_DEVERR_BLOCK_ID);
            const int in_block = (t0 + 8 * lane) & (bs - 1);
            const long long off =
                ok ? ((((long long)id * p.kv_heads + h) << p.log2_bs) + in_block) * W::kRowBytes : -1;
            const uint32_t dst = ring + uint32_t(stage) * W::kStageBytes;
            const int chunk = lane % W::kChunks;
#pragma unroll
            for (int it = 0; it < 8; ++it) {
                const int row = it * W::kRowsPerCopy + lane / W::kChunks;
                const long long o = __shfl_sync(kFullMask, off, it * W::kGroups / 8);
                const bool seen = o >= 0 && is.view.sees(t0 + row, p.sinks);
                const long long from = seen ? o + (row & 7) * W::kRowBytes + chunk * 16 : 0;
                const uint32_t to = dst + W::at(row, chunk);
                cp_async16(to, kbase + from, seen ? 16u : 0u, policy);
                cp_async16(to + 4096u, vbase + from, seen ? 16u : 0u, policy);
            }
            if constexpr (kEight) {
                if (lane < kNT)
                    cp_async8(sring + uint32_t(stage) * W::kScaleBytes + uint32_t(lane) * 8u,
                              p.scales + (ok ? (long long)id * p.scale_heads + h : 0), ok ? 8u : 0u);
            }
            ii += kWdWarps;
            settle();
        }
        cp_async_commit();
    };
    settle();
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s)
        issue(s);

    int stage = 0;
    int nseg = 0;
    bool have = true;
    while (have) {
        const int h = seg.r / p.row_tiles, row0 = (seg.r % p.row_tiles) * 16;
        const int rows = min(16, p.group - row0);
        const size_t out_row = size_t(seg.b) * p.heads + size_t(h) * p.group + row0;
        const bool two = rows > 8;

        // ---- query rows as the A operand ---------------------------------
        // a[0], a[2]: row g; a[1], a[3]: row g + 8
        uint32_t qa[D / 16][4];
        float f0 = p.scale_log2, f1 = p.scale_log2;
        {
            const uint32_t *q0 = reinterpret_cast<const uint32_t *>(
                static_cast<const uint16_t *>(p.q) + (out_row + g) * D);
            const uint32_t *q1 = q0 + 8 * D / 2;
            if constexpr (!kEight) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    qa[k][0] = g < rows ? __ldg(q0 + 8 * k + c) : 0u;
                    qa[k][1] = g + 8 < rows ? __ldg(q1 + 8 * k + c) : 0u;
                    qa[k][2] = g < rows ? __ldg(q0 + 8 * k + c + 4) : 0u;
                    qa[k][3] = g + 8 < rows ? __ldg(q1 + 8 * k + c + 4) : 0u;
                }
            } else {
                // dims [c D/4, (c + 1) D/4) of a row, 4 per step of the product,
                // in the order in which the codes are read
                auto load = [&](const uint32_t *src, bool there, int half, float &f) {
                    float x[D / 4];
                    float m = 0.0f;
#pragma unroll
                    for (int e = 0; e < D / 8; ++e) {
                        const uint32_t w = there ? __ldg(src + c * (D / 8) + e) : 0u;
                        const float2 y = p.bf16 ? Half16<true>::unpack(w) : Half16<false>::unpack(w);
                        x[2 * e] = y.x;
                        x[2 * e + 1] = y.y;
                        m = fmaxf(m, fmaxf(fabsf(y.x), fabsf(y.y)));
                    }
                    m = fmaxf(m, __shfl_xor_sync(kFullMask, m, 1));
                    m = fmaxf(m, __shfl_xor_sync(kFullMask, m, 2));
                    // power of two that brings the largest component to [2^14, 2^15)
                    const int e2 = m > 0.0f ? min(max(141 - int(__float_as_uint(m) >> 23), -100), 100) : 0;
                    const float up = __uint_as_float(uint32_t(127 + e2) << 23);
                    f = p.scale_log2 * __uint_as_float(uint32_t(127 - e2) << 23);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        qa[k][half] = Half16<false>::pack(x[4 * k] * up, x[4 * k + 1] * up);
                        qa[k][half + 2] = Half16<false>::pack(x[4 * k + 2] * up, x[4 * k + 3] * up);
                    }
                };
                load(q0, g < rows, 0, f0);
                load(q1, g + 8 < rows, 1, f1);
            }
        }

        float o[D / 8][4];
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[i][e] = 0.0f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
        float sv_ref = 0.0f, sv_inv = 0.0f;

        for (int i = seg.begin + warp; i < seg.end; i += kWdWarps) {
            cp_async_wait<kStages - 2>();
            __syncwarp();
            const uint32_t kt = ring + uint32_t(stage) * W::kStageBytes, vt = kt + 4096u;
            const uint32_t sc = sring + uint32_t(stage) * W::kScaleBytes;
            issue(stage == 0 ? kStages - 1 : stage - 1);
            stage = stage == kStages - 1 ? 0 : stage + 1;

            // ---- scores -----------------------------------------------------
            float s[kNT][4];
#pragma unroll
            for (int j = 0; j < kNT; ++j) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s[j][e] = 0.0f;
                if constexpr (!kEight) {
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        uint32_t b[4];
                        ldmatrix_x4(kt + W::at(8 * j + (lane & 7), 4 * k + (lane >> 3)), b);
                        mma16816<W::kBf16>(s[j], qa[2 * k], b[0], b[1]);
                        mma16816<W::kBf16>(s[j], qa[2 * k + 1], b[2], b[3]);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < D / 64; ++k) {
                        const uint4 w = lds128(kt + W::at(8 * j + g, c * (D / 64) + k));
                        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t b0, b1;
                            widen4<kE4m3>(ww[e], b0, b1);
                            mma16816<false>(s[j], qa[4 * k + e], b0, b1);
                        }
                    }
                }
            }
            float ratio[kNT];      // s_v of each 8-token group over the running reference
            if constexpr (kEight) {
                float top = 0.0f;
#pragma unroll
                for (int j = 0; j < kNT; ++j) {
                    const uint2 w = lds64(sc + uint32_t(j) * 8u);
                    const float sk = __uint_as_float(w.x);
                    ratio[j] = __uint_as_float(w.y);
                    top = fmaxf(top, ratio[j]);
                    s[j][0] *= f0 * sk;
                    s[j][1] *= f0 * sk;
                    s[j][2] *= f1 * sk;
                    s[j][3] *= f1 * sk;
                }
                top = pow2_at_least(top);
                if (top > sv_ref) {
                    const float down = sv_ref / top;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[n][e] *= down;
                    sv_ref = top;
                    sv_inv = 1.0f / top;
                }
#pragma unroll
                for (int j = 0; j < kNT; ++j)
                    ratio[j] *= sv_inv;
            } else {
#pragma unroll
                for (int j = 0; j < kNT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[j][e] *= f0;
            }
            const int t0 = seg.view.token<kTile>(i);
            if (t0 + kTile > seg.view.L || (t0 < seg.view.ws && t0 + kTile > p.sinks)) {
#pragma unroll
                for (int j = 0; j < kNT; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (!seg.view.sees(t0 + 8 * j + 2 * c + e, p.sinks)) {
                            s[j][e] = -INFINITY;
                            s[j][e + 2] = -INFINITY;
                        }
            }

            // ---- running maximum ------------------------------------------
            float n0 = m0, n1 = m1;
#pragma unroll
            for (int j = 0; j < kNT; ++j) {
                n0 = fmaxf(n0, fmaxf(s[j][0], s[j][1]));
                n1 = fmaxf(n1, fmaxf(s[j][2], s[j][3]));
            }
            n0 = fmaxf(n0, __shfl_xor_sync(kFullMask, n0, 1));
            n0 = fmaxf(n0, __shfl_xor_sync(kFullMask, n0, 2));
            if (two) {
                n1 = fmaxf(n1, __shfl_xor_sync(kFullMask, n1, 1));
                n1 = fmaxf(n1, __shfl_xor_sync(kFullMask, n1, 2));
            } else {
                n1 = 0.0f;
            }
            if (__any_sync(kFullMask, n0 > m0 || n1 > m1)) {
                const float a0 = n0 > m0 ? exp2_sfu(m0 - n0) : 1.0f;
                const float a1 = n1 > m1 ? exp2_sfu(m1 - n1) : 1.0f;
                l0 *= a0;
                l1 *= a1;
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    o[n][0] *= a0;
                    o[n][1] *= a0;
                    o[n][2] *= a1;
                    o[n][3] *= a1;
                }
                m0 = n0;
                m1 = n1;
            }
            // a row whose scores are all -inf so far keeps weights of zero
            const float z0 = (m0 == -INFINITY ? 0.0f : m0) - kWdShift;
            const float z1 = (m1 == -INFINITY ? 0.0f : m1) - kWdShift;

            // ---- weights and the product with V ---------------------------
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k) {
                uint32_t pa[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int j = 2 * k + e;
                    float w0 = exp2_sfu(s[j][0] - z0), w1 = exp2_sfu(s[j][1] - z0);
                    l0 += w0 + w1;
                    float w2 = 0.0f, w3 = 0.0f;
                    if (two) {
                        w2 = exp2_sfu(s[j][2] - z1);
                        w3 = exp2_sfu(s[j][3] - z1);
                        l1 += w2 + w3;
                    }
                    if constexpr (kEight) {
                        w0 *= ratio[j];
                        w1 *= ratio[j];
                        w2 *= ratio[j];
                        w3 *= ratio[j];
                    }
                    pa[2 * e] = Half16<W::kBf16>::pack(w0, w1);
                    pa[2 * e + 1] = Half16<W::kBf16>::pack(w2, w3);
                }
                if constexpr (!kEight) {
#pragma unroll
                    for (int n = 0; n < D / 16; ++n) {
                        uint32_t b[4];
                        ldmatrix_x4_trans(vt + W::at(16 * k + (lane & 15), 2 * n + (lane >> 4)), b);
                        mma16816<W::kBf16>(o[2 * n], pa, b[0], b[1]);
                        mma16816<W::kBf16>(o[2 * n + 1], pa, b[2], b[3]);
                    }
                } else {
                    // codes of dims [g D/8, (g + 1) D/8) of tokens 2c, 2c + 1 and
                    // 2c + 8, 2c + 9; pairs of tokens are interleaved bytewise
                    constexpr int kWords = D / 32;
                    uint32_t w[4][kWords];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int row = 16 * k + 2 * c + (e & 1) + 8 * (e >> 1);
                        if constexpr (D == 128) {
                            const uint4 x = lds128(vt + W::at(row, g));
                            w[e][0] = x.x, w[e][1] = x.y, w[e][2] = x.z, w[e][3] = x.w;
                        } else {
                            const uint2 x = lds64(vt + W::at(row, g >> 1) + uint32_t(g & 1) * 8u);
                            w[e][0] = x.x, w[e][1] = x.y;
                        }
                    }
#pragma unroll
                    for (int n = 0; n < kWords; ++n) {
                        const uint32_t x0 = __byte_perm(w[0][n], w[1][n], 0x5140);
                        const uint32_t x1 = __byte_perm(w[0][n], w[1][n], 0x7362);
                        const uint32_t y0 = __byte_perm(w[2][n], w[3][n], 0x5140);
                        const uint32_t y1 = __byte_perm(w[2][n], w[3][n], 0x7362);
                        uint32_t b0[4], b1[4];
                        widen4<kE4m3>(x0, b0[0], b0[1]);
                        widen4<kE4m3>(x1, b0[2], b0[3]);
                        widen4<kE4m3>(y0, b1[0], b1[1]);
                        widen4<kE4m3>(y1, b1[2], b1[3]);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            mma16816<false>(o[4 * n + e], pa, b0[e], b1[e]);
                    }
                }
            }
            __syncwarp();  // the stage may be filled again
        }

        // ---- merge the warps' parts of the unit ---------------------------
        l0 += __shfl_xor_sync(kFullMask, l0, 1);
        l0 += __shfl_xor_sync(kFullMask, l0, 2);
        l1 += __shfl_xor_sync(kFullMask, l1, 1);
        l1 += __shfl_xor_sync(kFullMask, l1, 2);
        if constexpr (kEight) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[n][e] *= sv_ref;
        }
        float2 *ml = reinterpret_cast<float2 *>(smem + W::kOffMl);
        float *mo = reinterpret_cast<float *>(smem + W::kOffMerge);
        const bool whole = seg.begin == 0 && seg.end == seg.view.tiles;
        const int slot = 2 * blockIdx.x + (nseg == 0 ? 0 : 1);
        constexpr int kPerRow = D / 8;                 // threads per row, 8 dims each
        // 8 rows and 64 dims at a time
        for (int pass = 0; pass < (two ? 2 : 1) * (D / 64); ++pass) {
            const int half = pass / (D / 64), part = pass % (D / 64);
            __syncthreads();  // the merge buffer is free
            if (c == 0)
                ml[warp * 8 + g] = half ? make_float2(m1, l1) : make_float2(m0, l0);
            float *row = mo + (warp * 8 + g) * W::kPitch;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
                const float a = half ? o[n][2] : o[n][0], b = half ? o[n][3] : o[n][1];
                if constexpr (kEight) {
                    if (D == 64 || (c >> 1) == part) {
                        const int d = (2 * c * (D / 8) + n) & 63;
                        row[d] = a;
                        row[d + D / 8] = b;
                    }
                } else if (n / 8 == part) {
                    *reinterpret_cast<float2 *>(row + 8 * (n & 7) + 2 * c) = make_float2(a, b);
                }
            }
            __syncthreads();
            const int rr = tid / 8, dd = (tid % 8) * 8, d0 = part * 64 + dd;
            if (rr < 8 && half * 8 + rr < rows) {
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWdWarps; ++w)
                    M = fmaxf(M, ml[w * 8 + rr].x);
                const float z = M == -INFINITY ? 0.0f : M;
                float l = 0.0f, acc[8] = {};
#pragma unroll
                for (int w = 0; w < kWdWarps; ++w) {
                    const float2 e = ml[w * 8 + rr];
                    const float f = exp2_sfu(e.x - z);
                    l += f * e.y;
                    const float4 *src = reinterpret_cast<const float4 *>(mo + (w * 8 + rr) * W::kPitch + dd);
                    const float4 x = src[0], y = src[1];
                    acc[0] += f * x.x, acc[1] += f * x.y, acc[2] += f * x.z, acc[3] += f * x.w;
                    acc[4] += f * y.x, acc[5] += f * y.y, acc[6] += f * y.z, acc[7] += f * y.w;
                }
                if (whole) {
                    const float inv = 1.0f / l;
                    const bool bf = kEight ? p.bf16 != 0 : W::kBf16;
                    uint32_t v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = bf ? Half16<true>::pack(acc[2 * e] * inv, acc[2 * e + 1] * inv)
                                  : Half16<false>::pack(acc[2 * e] * inv, acc[2 * e + 1] * inv);
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) +
                                               (out_row + half * 8 + rr) * D + d0) =
                        make_uint4(v[0], v[1], v[2], v[3]);
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(
                        p.part_o + (size_t(slot) * 16 + half * 8 + rr) * D + d0);
                    __stcg(dst, make_float4(acc[0], acc[1], acc[2], acc[3]));
                    __stcg(dst + 1, make_float4(acc[4], acc[5], acc[6], acc[7]));
                    if (d0 == 0)
                        __stcg(p.part_ml + size_t(slot) * 16 + half * 8 + rr, make_float2(M, l));
                }
            }
        }

        // ---- a unit shared with other CTAs --------------------------------
        if (!whole) {
            // tiles [u0, u0 + tiles) of the list belong to CTAs first .. last
            const long long u0 = hi - seg.left - seg.end;
            const int first = int(((u0 + 1) * ctas - 1) / total);
            const int last = int(((u0 + seg.view.tiles) * ctas - 1) / total);
            const int n = last - first + 1;
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                unsigned *ticket = p.tickets + (size_t(seg.b) * units + seg.r);
                s_last = atomicInc(ticket, unsigned(n - 1)) == unsigned(n - 1);
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                // the first CTA's part is its last segment, unless its range
                // begins with the unit; the others' is their first
                const bool head = (long long)first * total / ctas == u0;
                for (int item = tid; item < rows * kPerRow; item += kWdThreads) {
                    const int rr = item / kPerRow, d0 = (item % kPerRow) * 8;
                    auto part = [&](int k) { return size_t(2 * (first + k) + (k == 0 && !head ? 1 : 0)) * 16 + rr; };
                    float M = -INFINITY;
#pragma unroll 4
                    for (int k = 0; k < n; ++k)
                        M = fmaxf(M, __ldcg(p.part_ml + part(k)).x);
                    const float z = M == -INFINITY ? 0.0f : M;
                    float l = 0.0f, acc[8] = {};
#pragma unroll 4
                    for (int k = 0; k < n; ++k) {
                        const float2 e = __ldcg(p.part_ml + part(k));
                        const float4 *src = reinterpret_cast<const float4 *>(p.part_o + part(k) * D + d0);
                        const float4 x = __ldcg(src), y = __ldcg(src + 1);
                        const float f = exp2_sfu(e.x - z);
                        l += f * e.y;
                        acc[0] += f * x.x, acc[1] += f * x.y, acc[2] += f * x.z, acc[3] += f * x.w;
                        acc[4] += f * y.x, acc[5] += f * y.y, acc[6] += f * y.z, acc[7] += f * y.w;
                    }
                    const float inv = 1.0f / l;
                    const bool bf = kEight ? p.bf16 != 0 : W::kBf16;
                    uint32_t v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[e] = bf ? Half16<true>::pack(acc[2 * e] * inv, acc[2 * e + 1] * inv)
                                  : Half16<false>::pack(acc[2 * e] * inv, acc[2 * e + 1] * inv);
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + (out_row + rr) * D + d0) =
                        make_uint4(v[0], v[1], v[2], v[3]);
                }
            }
        }
        ++nseg;
        have = seg.next<kTile>(p, units);
    }
    cp_async_wait<0>();
}

} // namespace pa
