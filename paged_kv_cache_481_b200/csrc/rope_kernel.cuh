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
    int tokens_per_cta;             // 8-bit kernel: tokens whose runs one CTA looks after
    int64_t kv_ctas;                // 8-bit kernel: CTAs of the K/V part (the rest rotate q)
    int q_row_groups;               // 8-bit kernel: CTAs per token of the q part
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

// A token's slot and position; false (with the reason recorded once) when the
// token is padding or its indices are outside the pool or the table.
__device__ __forceinline__ bool token_place(const RopeParams &p, int i, bool report, int64_t &slot,
                                            int64_t &pos)
{
    slot = p.slots[i];
    if (slot < 0)
        return false;
    pos = p.rotary > 0 ? p.positions[i] : 0;
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

// Rows [row0, row0 + kPasses * rows per pass) of one token: row r < H is
// query head r, then the K heads, then the V heads.  All loads of a thread's
// passes are issued before the first result is stored.
template <int D, bool kBf16, bool kInterleaved, int kPasses, bool kQueriesOnly, int kThreads>
__device__ __forceinline__ void rope_rows(const RopeParams &p, int i, int row0, int64_t slot,
                                          int64_t pos)
{
    constexpr int kUnits = D / 16, kRows = kThreads / kUnits;
    const int u = threadIdx.x % kUnits, r0 = row0 + threadIdx.x / kUnits;
    const int H = p.num_heads, KVH = p.num_kv_heads;
    const int rows = kQueriesOnly ? H : H + 2 * KVH;
    const bool turned = u < p.rotary / 16;
    int p0, p1;
    unit_pieces<kInterleaved>(u, p.rotary, p0, p1);
    uint4 v0[kPasses], v1[kPasses];
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
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
    UnitAngles a;
    if (turned)
        load_angles(a, p.cos_sin + pos * p.rotary, p.rotary / 2, u);
    const int64_t block = slot / p.block_size, offset = slot % p.block_size;
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
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

// Grid (num_tokens, ceil(rows / (kPasses * rows per pass))).
template <int D, bool kBf16, bool kInterleaved, int kPasses>
__global__ void __launch_bounds__(kRopeThreads) rope_and_cache_kernel(const RopeParams p)
{
    grid_dependency_wait();
    allow_dependent_launch();
    constexpr int kRows = kRopeThreads / (D / 16) * kPasses;
    int64_t slot, pos;
    const int i = blockIdx.x;
    if (!token_place(p, i, threadIdx.x == 0 && blockIdx.y == 0, slot, pos))
        return;
    rope_rows<D, kBf16, kInterleaved, kPasses, false, kRopeThreads>(p, i, blockIdx.y * kRows, slot, pos);
}

// ------------------------------------------------------- 8-bit block cache

// One run (new tokens i0 .. i0 + n - 1 of one block, consecutive slots from
// `slot`) and one K/V head: the first half of the CTA's warps does K, the
// second V.  A first sweep over the rows finds the largest magnitude, a
// second one writes the codes; the first kKept rows of a thread stay in
// registers in between, the others are read again (from the caches).
template <int D, bool kBf16, bool kInterleaved, bool kE4m3, int kThreads>
__device__ __forceinline__ void quantize_run(const RopeParams &p, int i0, int n, int64_t slot, int h,
                                             float (&amax_sm)[2][kThreads / 64])
{
    constexpr int kUnits = D / 16, kHalf = kThreads / 2, kRows = kHalf / kUnits, kWarps = kHalf / 32;
    constexpr int kKept = 2;
    constexpr float kTop = code_top<kE4m3>();
    const int is_v = threadIdx.x / kHalf, ht = threadIdx.x % kHalf;
    const int u = ht % kUnits, r0 = ht / kUnits;
    const int KVH = p.num_kv_heads;
    const bool turned = !is_v && u < p.rotary / 16;
    int p0 = 16 * u, p1 = 16 * u + 8;
    if (!is_v)
        unit_pieces<kInterleaved>(u, p.rotary, p0, p1);
    const int64_t block = slot / p.block_size;
    const int first = int(slot % p.block_size);
    const uint16_t *src = static_cast<const uint16_t *>(is_v ? p.value : p.key) + int64_t(h) * D;
    const int64_t stride = is_v ? p.value_stride : p.key_stride;
    uint8_t *codes = static_cast<uint8_t *>(is_v ? p.v_cache : p.k_cache) +
                     (block * KVH + h) * p.block_size * D;
    float2 *scales = p.kv_scales + block * p.scale_heads + h;
    float *my_scale = reinterpret_cast<float *>(scales) + is_v;
    const float old = *my_scale;

    auto fetch = [&](int r, float(&x)[16]) {
        const int64_t i = i0 + r;
        const uint4 v0 = *reinterpret_cast<const uint4 *>(src + i * stride + p0);
        const uint4 v1 = *reinterpret_cast<const uint4 *>(src + i * stride + p1);
        UnitAngles a;
        if (turned) {
            int64_t pos = p.positions[i];
            if (pos < 0 || pos >= p.max_position) {
                if (u == 0 && h == 0)
                    atomicOr(p.err, PA_DEVERR_POSITION);
                pos = 0;
            }
            load_angles(a, p.cos_sin + pos * p.rotary, p.rotary / 2, u);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                a.c[e] = 1.0f, a.s[e] = 0.0f;
        }
        if (turned) {
            rotate_unit<kBf16, kInterleaved>(v0, v1, a, x);
        } else {
            using H = Half16<kBf16>;
            const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 f = H::unpack(w[e]);
                x[2 * e] = f.x;
                x[2 * e + 1] = f.y;
            }
        }
    };
    auto largest = [](const float(&x)[16]) {
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            m = fmaxf(m, fabsf(x[e]));
        return m;
    };

    float kept[kKept][16];
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < kKept; ++k)
        if (r0 + k * kRows < n) {
            fetch(r0 + k * kRows, kept[k]);
            m = fmaxf(m, largest(kept[k]));
        }
    for (int r = r0 + kKept * kRows; r < n; r += kRows) {
        float x[16];
        fetch(r, x);
        m = fmaxf(m, largest(x));
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1)
        m = fmaxf(m, __shfl_xor_sync(kFullMask, m, off));
    __syncthreads();  // the shared maxima of the previous run have been read
    if ((threadIdx.x & 31) == 0)
        amax_sm[is_v][ht / 32] = m;
    __syncthreads();  // also: every thread has read the old scale
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        m = fmaxf(m, amax_sm[is_v][w]);
    float scale = __fdiv_rn(m, kTop);
    if (first > 0)
        scale = fmaxf(old, scale);

    auto put = [&](int r, const float(&x)[16]) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float y[4];
#pragma unroll
            for (int f = 0; f < 4; ++f)
                y[f] = scale > 0.0f ? __fdiv_rn(x[4 * e + f], scale) : 0.0f;
            w[e] = encode2<kE4m3>(y[0], y[1]) | (encode2<kE4m3>(y[2], y[3]) << 16);
        }
        uint8_t *dst = codes + int64_t(first + r) * D;
        *reinterpret_cast<uint2 *>(dst + p0) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2 *>(dst + p1) = make_uint2(w[2], w[3]);
    };
#pragma unroll
    for (int k = 0; k < kKept; ++k)
        if (r0 + k * kRows < n)
            put(r0 + k * kRows, kept[k]);
    for (int r = r0 + kKept * kRows; r < n; r += kRows) {
        float x[16];
        fetch(r, x);
        put(r, x);
    }
    if (first > 0 && scale > old) {
        const float ratio = __fdiv_rn(old, scale);
        for (int r = r0; r < first; r += kRows) {
            uint4 *row = reinterpret_cast<uint4 *>(codes + int64_t(r) * D + 16 * u);
            const uint4 c = *row;
            const uint32_t w[4] = {c.x, c.y, c.z, c.w};
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 a = decode2<kE4m3>(w[e]), b = decode2<kE4m3>(w[e] >> 16);
                o[e] = encode2<kE4m3>(__fmul_rn(a.x, ratio), __fmul_rn(a.y, ratio)) |
                       (encode2<kE4m3>(__fmul_rn(b.x, ratio), __fmul_rn(b.y, ratio)) << 16);
            }
            *row = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    if (ht == 0 && (first == 0 || scale > old))
        *my_scale = scale;
}

// Grid: p.kv_ctas CTAs, each (a stretch of tokens_per_cta tokens, one K/V
// head) for the runs that begin in the stretch, then num_tokens *
// q_row_groups CTAs that rotate query rows.
template <int D, bool kBf16, bool kInterleaved, bool kE4m3, int kThreads>
__global__ void __launch_bounds__(kThreads) rope_and_cache_q8_kernel(const RopeParams p)
{
    grid_dependency_wait();
    allow_dependent_launch();
    __shared__ float amax_sm[2][kThreads / 64];
    const int64_t cta = blockIdx.x;
    if (cta >= p.kv_ctas) {
        constexpr int kPasses = 2, kRows = kThreads / (D / 16) * kPasses;
        const int64_t k = cta - p.kv_ctas;
        const int i = int(k / p.q_row_groups), g = int(k % p.q_row_groups);
        int64_t slot, pos;
        if (token_place(p, i, threadIdx.x == 0 && g == 0, slot, pos))
            rope_rows<D, kBf16, kInterleaved, kPasses, true, kThreads>(p, i, g * kRows, slot, pos);
        return;
    }
    const int h = int(cta % p.num_kv_heads);
    const int t0 = int(cta / p.num_kv_heads) * p.tokens_per_cta;
    const int t1 = min(p.num_tokens, t0 + p.tokens_per_cta);
    const int lane = threadIdx.x & 31, bs = p.block_size;
    const int64_t slots = int64_t(p.num_blocks) * bs;
    // every warp finds the same runs: token i begins one unless its slot
    // follows its neighbour's inside the same block
    for (int base = t0; base < t1; base += 32) {
        const int mine = base + lane;
        int64_t s = -1;
        bool begins = false;
        if (mine < t1) {
            s = p.slots[mine];
            begins = s >= 0 && s < slots &&
                     (mine == 0 || s % bs == 0 || p.slots[mine - 1] != s - 1);
        }
        unsigned heads = __ballot_sync(kFullMask, begins);
        while (heads) {
            const int l = __ffs(heads) - 1;
            heads &= heads - 1;
            const int i0 = base + l;
            const int64_t slot = __shfl_sync(kFullMask, s, l);
            const int most = min(bs - int(slot % bs), p.num_tokens - i0);
            int n = 0;
            while (n < most) {  // the run's length, 32 tokens at a time
                const int j = n + lane;
                const unsigned same =
                    __ballot_sync(kFullMask, j < most && p.slots[i0 + j] == slot + j);
                if (same != kFullMask) {
                    n += __ffs(~same) - 1;
                    break;
                }
                n += 32;
            }
            quantize_run<D, kBf16, kInterleaved, kE4m3, kThreads>(p, i0, n, slot, h, amax_sm);
        }
    }
}

} // namespace pa
