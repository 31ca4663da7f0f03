// Position rotation fused with the write into the paged cache, for the 16-bit
// cache and for the 8-bit cache with one scale per (block, head).
//
// Mathematics: component pairs (a, b) of a head row are turned by the
// position's angle, y_a = x_a c - x_b s, y_b = x_b c + x_a s.  Each product
// and sum is rounded to fp32 by itself (no contraction), so that the value
// that is quantized does not depend on how the compiler groups them.
//
// Both kernels are bound by memory: every row is read once and written once,
// and a token's angles are loaded once per thread and used for several heads.
// A thread works on a "unit" of 16 elements of a row, two 16-byte pieces that
// hold whole pairs: elements [8u, 8u + 8) and [r/2 + 8u, ...) of a
// half-split rotation of r dims, else 16 neighbouring elements.
//
// Measured (kernel alone in a graph of four, one B200 at 1965 MHz): 9 packed
// prompts, H 32, KVH 8, bf16: 42.2 us, 5.8 TB/s, 88 % of a plain copy's rate
// (the rest is the first and the last wave); 32 tokens of 40 heads: 2.1 us,
// three dependent loads.  The 8-bit write: 12 chunks, H 32, KVH 8, e4m3: 37.4
// us, 3.8 TB/s, bound by the chain slot -> rows -> angles -> maximum -> codes
// with 64 registers a thread, which are too few: all instances spill 84 to 100
// bytes and read back 220 to 316; 256 single tokens of 40 heads: 6.2 us.
#pragma once

#include <cstdint>

#include "../../include/pa_window.h"
#include "half_types.cuh"
#include "ptx.cuh"

namespace pa {

struct RopeParams {
    void *q_out;
    const void *q, *key, *value;
    int64_t q_out_stride, q_stride, key_stride, value_stride;  // elements between tokens
    void *k_cache, *v_cache;        // 16-bit values, or 8-bit codes
    float2 *kv_scales;              // 8-bit cache only
    const float *cos_sin;
    const int64_t *positions, *slots;
    int num_tokens, num_heads, num_kv_heads;
    int rotary, max_position;
    int block_size, num_blocks;
    int scale_heads;                // heads of a block's scale row (kv heads rounded up to even)
    int groups;                     // 8-bit kernel: CTAs per token
    int scan_ctas, scan_blocks;     // 8-bit kernel: CTAs that look for blocks with two runs, blocks of each
    unsigned int *err;
};

// Angles of one unit: cosines and sines of its 8 pairs.
struct UnitAngles {
    float c[8], s[8];
};

__device__ __forceinline__ void load_angles(UnitAngles &a, const float *row, int half, int u)
{
    const float4 *c = reinterpret_cast<const float4 *>(row + 8 * u);
    const float4 *s = reinterpret_cast<const float4 *>(row + half + 8 * u);
    const float4 c0 = __ldg(c), c1 = __ldg(c + 1), s0 = __ldg(s), s1 = __ldg(s + 1);
    a.c[0] = c0.x, a.c[1] = c0.y, a.c[2] = c0.z, a.c[3] = c0.w;
    a.c[4] = c1.x, a.c[5] = c1.y, a.c[6] = c1.z, a.c[7] = c1.w;
    a.s[0] = s0.x, a.s[1] = s0.y, a.s[2] = s0.z, a.s[3] = s0.w;
    a.s[4] = s1.x, a.s[5] = s1.y, a.s[6] = s1.z, a.s[7] = s1.w;
}

__device__ __forceinline__ void turn(float &a, float &b, float c, float s)
{
    const float x = a, y = b;
    a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
    b = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
}

// Element offsets of a unit's two 16-byte pieces within a row.
template <bool kInterleaved>
__device__ __forceinline__ void unit_pieces(int u, int rotary, int &p0, int &p1)
{
    if (!kInterleaved && u < rotary / 16) {
        p0 = 8 * u;
        p1 = rotary / 2 + 8 * u;
    } else {
        p0 = 16 * u;
        p1 = p0 + 8;
    }
}

// The 16 values of a unit in fp32, rotated.
template <bool kBf16, bool kInterleaved>
__device__ __forceinline__ void rotate_unit(const uint4 &v0, const uint4 &v1, const UnitAngles &a,
                                            float (&x)[16])
{
    using H = Half16<kBf16>;
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = H::unpack(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (kInterleaved)
            turn(x[2 * i], x[2 * i + 1], a.c[i], a.s[i]);
        else
            turn(x[i], x[8 + i], a.c[i], a.s[i]);
    }
}

template <bool kBf16, bool kInterleaved>
__device__ __forceinline__ void rotate_pieces(uint4 &v0, uint4 &v1, const UnitAngles &a)
{
    using H = Half16<kBf16>;
    float x[16];
    rotate_unit<kBf16, kInterleaved>(v0, v1, a, x);
    v0 = make_uint4(H::pack(x[0], x[1]), H::pack(x[2], x[3]), H::pack(x[4], x[5]), H::pack(x[6], x[7]));
    v1 = make_uint4(H::pack(x[8], x[9]), H::pack(x[10], x[11]), H::pack(x[12], x[13]),
                    H::pack(x[14], x[15]));
}

// Whether a token's slot and position are to be worked on; false (with the
// reason recorded by one thread) when it is padding or they are outside the
// pool or the table.
__device__ __forceinline__ bool token_is_live(const RopeParams &p, bool report, int64_t slot, int64_t pos)
{
    if (slot < 0)
        return false;
    unsigned bad = 0;
    if (slot >= int64_t(p.num_blocks) * p.block_size)
        bad |= PA_DEVERR_SLOT;
    if (p.rotary > 0 && (pos < 0 || pos >= p.max_position))
        bad |= PA_DEVERR_POSITION;
    if (bad && report)
        atomicOr(p.err, bad);
    return bad == 0;
}

constexpr int kRopeThreads = 128;
constexpr int kRopePasses = 2;     // rows of a token that a thread works on

// Rows [row0, row0 + kRopePasses * rows per pass) of one token: row r < H is
// query head r, then the K heads, then the V heads.  The rows are fetched
// together with the token's slot and position, so that only the angles wait
// for another load.
template <int D, bool kBf16, bool kInterleaved, bool kQueriesOnly>
__device__ __forceinline__ void rope_rows(const RopeParams &p, int i, int row0)
{
    constexpr int kUnits = D / 16, kRows = kRopeThreads / kUnits;
    const int u = threadIdx.x % kUnits, r0 = row0 + threadIdx.x / kUnits;
    const int H = p.num_heads, KVH = p.num_kv_heads;
    const int rows = kQueriesOnly ? H : H + 2 * KVH;
    const bool turned = u < p.rotary / 16;
    int p0, p1;
    unit_pieces<kInterleaved>(u, p.rotary, p0, p1);
    const int64_t slot = p.slots[i], pos = p.rotary > 0 ? p.positions[i] : 0;
    uint4 v0[kRopePasses], v1[kRopePasses];
#pragma unroll
    for (int k = 0; k < kRopePasses; ++k) {
        const int r = r0 + k * kRows;
        if (r >= rows)
            continue;
        const uint16_t *src;
        if (kQueriesOnly || r < H)
            src = static_cast<const uint16_t *>(p.q) + i * p.q_stride + int64_t(r) * D;
        else if (r < H + KVH)
            src = static_cast<const uint16_t *>(p.key) + i * p.key_stride + int64_t(r - H) * D;
        else
            src = static_cast<const uint16_t *>(p.value) + i * p.value_stride + int64_t(r - H - KVH) * D;
        v0[k] = *reinterpret_cast<const uint4 *>(src + p0);
        v1[k] = *reinterpret_cast<const uint4 *>(src + p1);
    }
    if (!token_is_live(p, threadIdx.x == 0 && row0 == 0, slot, pos))
        return;
    UnitAngles a;
    if (turned)
        load_angles(a, p.cos_sin + pos * p.rotary, p.rotary / 2, u);
    const int64_t block = slot / p.block_size, offset = slot % p.block_size;
#pragma unroll
    for (int k = 0; k < kRopePasses; ++k) {
        const int r = r0 + k * kRows;
        if (r >= rows)
            continue;
        uint16_t *dst;
        if (kQueriesOnly || r < H) {
            dst = static_cast<uint16_t *>(p.q_out) + i * p.q_out_stride + int64_t(r) * D;
        } else {
            const bool is_v = r >= H + KVH;
            const int h = r - H - (is_v ? KVH : 0);
            dst = static_cast<uint16_t *>(is_v ? p.v_cache : p.k_cache) +
                  ((block * KVH + h) * p.block_size + offset) * D;
        }
        if (turned && (kQueriesOnly || r < H + KVH))
            rotate_pieces<kBf16, kInterleaved>(v0[k], v1[k], a);
        *reinterpret_cast<uint4 *>(dst + p0) = v0[k];
        *reinterpret_cast<uint4 *>(dst + p1) = v1[k];
    }
}

// Grid (num_tokens, ceil(rows / (kRopePasses * rows per pass))).
template <int D, bool kBf16, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_and_cache_kernel(const RopeParams p)
{
    grid_dependency_wait();
    allow_dependent_launch();
    constexpr int kRows = kRopeThreads / (D / 16) * kRopePasses;
    rope_rows<D, kBf16, kInterleaved, false>(p, blockIdx.x, blockIdx.y * kRows);
}

// ------------------------------------------------------- 8-bit block cache

// How a row's values become codes: code = round(x a / d).  With a new scale
// s = m / top that is x top / m, one rounding instead of two (a value exactly
// between two codes stays there; bf16 rows hold many); else x / s.
//
// The quotient is the product with the rounded reciprocal, corrected by its
// own remainder (Markstein): 4 operations, and correctly rounded as long as
// nothing underflows, which factors of 2^40 see to.
struct CodeScale {
    float a, d, r;
    float scale;           // what the block's scale becomes
    bool grown;            // it is not what it was

    __device__ __forceinline__ CodeScale(float m, float old, int first, float top)
    {
        scale = __fdiv_rn(m, top);
        grown = first == 0 || scale > old;
        scale = grown ? scale : old;
        // (a scale below the normal numbers may be rounded so far down that
        // x / s passes the top: such rows take x top / m too)
        const bool by_max = grown || (old < 0x1p-126f && m > __fmul_rn(old, top));
        d = by_max ? m : old;
        const float by = d > 1e30f ? 0x1p-40f : d < 1e-30f ? 0x1p40f : 1.0f;
        a = by_max ? top * by : by;
        d *= by;
        r = d > 0.0f ? __frcp_rn(d) : 0.0f;   // all codes are 0 where the scale is
    }
    __device__ __forceinline__ float code(float x) const
    {
        const float n = __fmul_rn(x, a), q = __fmul_rn(n, r);
        return __fmaf_rn(__fmaf_rn(-q, d, n), r, q);
    }
    template <bool kE4m3>
    __device__ __forceinline__ uint2 encode8(const float *x) const
    {
        uint2 w;
        w.x = encode4<kE4m3>(code(x[0]), code(x[1]), code(x[2]), code(x[3]));
        w.y = encode4<kE4m3>(code(x[4]), code(x[5]), code(x[6]), code(x[7]));
        return w;
    }
};

// Codes of older rows [0, first) of a block whose scale grew, taken to the new
// scale; this thread's 16 codes of rows r0, r0 + stride, ..., four at a time.
template <int D, bool kE4m3>
__device__ __forceinline__ void rescale_rows(uint8_t *codes, int first, float ratio, int r0, int stride,
                                             int u)
{
#pragma unroll 1
    for (int r = r0; r < first; r += 4 * stride) {
        uint4 c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (r + j * stride < first)
                c[j] = *reinterpret_cast<const uint4 *>(codes + (r + j * stride) * D + 16 * u);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (r + j * stride >= first)
                break;
            const uint32_t w[4] = {c[j].x, c[j].y, c[j].z, c[j].w};
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 x = decode2<kE4m3>(w[e]), y = decode2<kE4m3>(w[e] >> 16);
                o[e] = encode4<kE4m3>(__fmul_rn(x.x, ratio), __fmul_rn(x.y, ratio),
                                      __fmul_rn(y.x, ratio), __fmul_rn(y.y, ratio));
            }
            *reinterpret_cast<uint4 *>(codes + (r + j * stride) * D + 16 * u) =
                make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

// The K or V rows of one run (new tokens i0 .. i0 + n - 1, consecutive slots
// of one block) of one K/V head, by kLanes lanes (part of a warp, or the two
// warps that share `both`), D / 16 to a row: a first sweep finds the largest
// magnitude, a second one writes the codes.  The first kKept rows of a lane
// stay in registers in between (as they came, rotated twice rather than kept
// in fp32), the others are read again.
template <int D, bool kBf16, bool kInterleaved, bool kE4m3, int kLanes, int kKept>
__device__ __forceinline__ void quantize_run(const RopeParams &p, int i0, int n, int64_t block, int first,
                                             int h, bool is_v, int lane, float *both)
{
    constexpr int kUnits = D / 16, kRows = kLanes / kUnits;
    constexpr float kTop = code_top<kE4m3>();
    const int u = lane % kUnits, r0 = lane / kUnits % kRows;
    const bool turned = !is_v && u < p.rotary / 16;
    int p0 = 16 * u, p1 = 16 * u + 8;
    if (!is_v)
        unit_pieces<kInterleaved>(u, p.rotary, p0, p1);
    const int64_t stride = is_v ? p.value_stride : p.key_stride;
    const uint16_t *src = static_cast<const uint16_t *>(is_v ? p.value : p.key) + i0 * stride + int64_t(h) * D;
    uint8_t *codes = static_cast<uint8_t *>(is_v ? p.v_cache : p.k_cache) +
                     (block * p.num_kv_heads + h) * p.block_size * D;
    float *my_scale = reinterpret_cast<float *>(p.kv_scales + block * p.scale_heads + h) + is_v;
    const float old = *my_scale;

    auto load = [&](int r, uint4 (&v)[2]) {
        v[0] = *reinterpret_cast<const uint4 *>(src + r * stride + p0);
        v[1] = *reinterpret_cast<const uint4 *>(src + r * stride + p1);
    };
    auto values = [&](int r, const uint4 (&v)[2], float (&x)[16]) {
        if (turned) {
            int64_t pos = p.positions[i0 + r];
            if (pos < 0 || pos >= p.max_position) {
                if (u == 0 && h == 0)
                    atomicOr(p.err, PA_DEVERR_POSITION);
                pos = 0;
            }
            UnitAngles a;
            load_angles(a, p.cos_sin + pos * p.rotary, p.rotary / 2, u);
            rotate_unit<kBf16, kInterleaved>(v[0], v[1], a, x);
        } else {
            using H = Half16<kBf16>;
            const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 f = H::unpack(w[e]);
                x[2 * e] = f.x;
                x[2 * e + 1] = f.y;
            }
        }
    };

    uint4 kept[kKept][2];
#pragma unroll
    for (int k = 0; k < kKept; ++k)
        if (r0 + k * kRows < n)
            load(r0 + k * kRows, kept[k]);
    float m = 0.0f;
    auto largest = [&](int r, const uint4 (&v)[2]) {
        if (turned) {
            float x[16];
            values(r, v, x);
#pragma unroll
            for (int e = 0; e < 16; ++e)
                m = fmaxf(m, fabsf(x[e]));
        } else {
            const float2 x = Half16<kBf16>::unpack(abs_max_pairs<typename Half16<kBf16>::T2>(v[0], v[1]));
            m = fmaxf(m, fmaxf(x.x, x.y));
        }
    };
#pragma unroll
    for (int k = 0; k < kKept; ++k)
        if (r0 + k * kRows < n)
            largest(r0 + k * kRows, kept[k]);
#pragma unroll 1
    for (int r = r0 + kKept * kRows; r < n; r += kRows) {
        uint4 v[2];
        load(r, v);
        largest(r, v);
    }
    // (within this run's lanes: the lanes of a group agree on their way here)
    constexpr int kIn = kLanes < 32 ? kLanes : 32;
    const unsigned group = kIn == 32 ? kFullMask : ((1u << (kIn & 31)) - 1u) << ((lane & 31) / kIn * kIn);
#pragma unroll
    for (int off = kIn / 2; off >= 1; off >>= 1)
        m = fmaxf(m, __shfl_xor_sync(group, m, off));
    if constexpr (kLanes == 64) {  // (the whole CTA comes here)
        __syncthreads();           // the last run's maxima have been read
        if ((lane & 31) == 0)
            both[lane / 32] = m;
        __syncthreads();           // also: the old scale has been read
        m = fmaxf(both[0], both[1]);
    }
    const CodeScale scale(m, old, first, kTop);

    auto put = [&](int r, const float (&x)[16]) {
        uint8_t *dst = codes + (first + r) * D;
        *reinterpret_cast<uint2 *>(dst + p0) = scale.encode8<kE4m3>(x);
        *reinterpret_cast<uint2 *>(dst + p1) = scale.encode8<kE4m3>(x + 8);
    };
#pragma unroll
    for (int k = 0; k < kKept; ++k)
        if (r0 + k * kRows < n) {
            float x[16];
            values(r0 + k * kRows, kept[k], x);
            put(r0 + k * kRows, x);
        }
#pragma unroll 1
    for (int r = r0 + kKept * kRows; r < n; r += kRows) {
        uint4 v[2];
        float x[16];
        load(r, v);
        values(r, v, x);
        put(r, x);
    }
    if (first > 0 && scale.grown)
        rescale_rows<D, kE4m3>(codes, first, __fdiv_rn(old, scale.scale), r0, kRows, u);
    if (lane % kLanes == 0 && scale.grown)
        *my_scale = scale.scale;
}

// Records blocks from `first` on, p.scan_blocks of them, that the call's tokens
// enter more than once: a block's rows, older ones and scale are one run's to
// write.  A bit a block, set by the first token of each run.  (A second one
// whose position is outside the table is recorded for that.)
// The bit map takes 512 bytes (4096 blocks a CTA) for pools up to 64 such
// parts, else 4 KB: next to 4 KB a CTA the L1 holds fewer of the rows that long
// runs read twice (20 runs of 100 to 300 tokens, one K/V head: 25.6 us, with
// 512 bytes or none 24.5), but every one of these CTAs passes over all slots,
// and hundreds of them would be in the others' way.  (10000 tokens of 7 heads
// and one K/V head of 64, the most that this can weigh: 17.5 us without, 17.9
// with 2000 blocks, 18.7 with 260,000, 18.3 with a million.)
constexpr int kScanFew = 4096, kScanMany = 32768, kScanParts = 64;

__device__ __forceinline__ void scan_runs(const RopeParams &p, int64_t first, uint32_t *seen)
{
    const int log2_bs = __ffs(p.block_size) - 1;
    const int64_t blocks = min(int64_t(p.scan_blocks), p.num_blocks - first);
    for (int i = threadIdx.x; i < (blocks + 31) / 32; i += kRopeThreads)
        seen[i] = 0;
    __syncthreads();
    constexpr int kAhead = 4;      // loads in flight: one CTA passes over all the call's slots
    for (int i0 = threadIdx.x; i0 < p.num_tokens; i0 += kAhead * kRopeThreads) {
        int64_t slot[kAhead], before[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = i0 + j * kRopeThreads;
            slot[j] = i < p.num_tokens ? p.slots[i] : -1;
            before[j] = i > 0 && i < p.num_tokens ? p.slots[i - 1] : -1;
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int64_t at = (slot[j] >> log2_bs) - first;
            if (slot[j] < 0 || at < 0 || at >= blocks ||
                (before[j] == slot[j] - 1 && (slot[j] & (p.block_size - 1)) != 0))
                continue;
            const uint32_t bit = 1u << (at & 31);
            if (!(atomicOr(&seen[at >> 5], bit) & bit))
                continue;
            const int64_t pos = p.rotary > 0 ? p.positions[i0 + j * kRopeThreads] : 0;
            if (pos >= 0 && (p.rotary == 0 || pos < p.max_position))
                atomicOr(p.err, PA_DEVERR_SLOT);
        }
    }
}

// Grid: p.scan_ctas CTAs, which look for blocks that two runs write (0 to 2 % of
// a call), then p.groups CTAs a token.  CTA g of them rotates the token's g-th
// 32 query rows (64 at D = 64) and looks after its g-th kSpan K/V heads.  A
// token alone in its run (a decode step) has its heads done side by side, D / 16
// lanes each for K and for V.  The heads of a longer run are shared out over the
// CTAs of its first kSpan tokens, a CTA a head (64 threads K, 64 threads V).
// The q rows are rotated by the same CTAs: with CTAs of their own the streaming
// part waited behind the dependent one (55 us against 39 on 12 chunks).
template <int D, bool kBf16, bool kInterleaved, bool kE4m3>
__global__ void __launch_bounds__(kRopeThreads, 8) rope_and_cache_q8_kernel(const RopeParams p)
{
    __shared__ float both[2][2];
    extern __shared__ uint32_t seen[];
    grid_dependency_wait();
    allow_dependent_launch();
    if (int(blockIdx.x) < p.scan_ctas) {
        scan_runs(p, int64_t(blockIdx.x) * p.scan_blocks, seen);
        return;
    }
    const int cta = int(blockIdx.x) - p.scan_ctas;
    constexpr int kUnits = D / 16, kHeads = 32 / kUnits, kSpan = 2 * kHeads;
    constexpr int kRows = kRopeThreads / kUnits * kRopePasses;
    const int i = cta / p.groups, g = cta % p.groups;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    // slots of the kSpan tokens before this one and of those from it on
    const int j = i - kSpan + lane;
    const int64_t near = j >= 0 && j < p.num_tokens ? p.slots[j] : -1;
    if (g * kRows < p.num_heads)
        rope_rows<D, kBf16, kInterleaved, true>(p, i, g * kRows);
    const int h0 = g * kSpan;
    if (h0 >= p.num_kv_heads)
        return;
    const int64_t slot = __shfl_sync(kFullMask, near, kSpan);
    const int bs = p.block_size;
    if (slot < 0 || slot >= int64_t(p.num_blocks) * bs)
        return;                    // padding, or recorded with the query rows
    const int64_t block = slot / bs;
    const int at = int(slot % bs);
    const unsigned same =
        __ballot_sync(kFullMask, near == slot + (lane - kSpan) && near >= block * bs && near < (block + 1) * bs);
    const int before = __clz(~(same << (32 - kSpan)));  // of the tokens before it, those of its run
    if (before >= kSpan)
        return;
    int n = before + __ffs(~(same >> kSpan)) - 1;
    if (n - before == 32 - kSpan) {  // the run goes on behind the tokens looked at
        const int most = before + min(bs - at, p.num_tokens - i);
        while (n < most) {
            const int k = n + lane;
            const unsigned more =
                __ballot_sync(kFullMask, k < most && p.slots[i - before + k] == slot - before + k);
            if (more != kFullMask) {
                n += __ffs(~more) - 1;
                break;
            }
            n += 32;
        }
    }
    if (n == 1) {
        const int h = h0 + warp / 2 * kHeads + lane / kUnits;
        if (h < p.num_kv_heads)
            quantize_run<D, kBf16, kInterleaved, kE4m3, kUnits, 1>(p, i, 1, block, at, h, warp & 1, lane,
                                                                   nullptr);
    } else {
        const int end = min(h0 + kSpan, p.num_kv_heads), half = threadIdx.x / 64;
        for (int h = h0 + before; h < end; h += n)
            quantize_run<D, kBf16, kInterleaved, kE4m3, 64, 2>(p, i - before, n, block, at - before, h, half,
                                                               threadIdx.x % 64, both[half]);
    }
}

} // namespace pa
