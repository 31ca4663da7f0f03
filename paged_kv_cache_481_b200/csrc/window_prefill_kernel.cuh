// Multi-query window attention over the paged cache on the sm_100a tensor
// cores: fp16 or bf16, head_dim 64 or 128, grouped heads, a sliding window
// and a few first tokens that stay visible.
//
// Mathematics: the query at position p sees t <= p with t > p - window or
// t < sinks; out = sum_t w_t V_t / sum_t w_t, w_t = 2^(c s_t - m), in one pass
// over the visible tokens (online softmax in base 2).  The reference m is
// moved only when a row's maximum grows by more than 2^8, so that the
// accumulator is rarely rescaled; numerator and denominator always share it.
//
// What bounds it: 4 D flops a visible (query, token) pair on the matrix unit
// and one exponential a pair on the special-function unit (16 a clock and
// SM: as long as the matrix work at D = 128, twice as long at D = 64); for a
// few queries a sequence, the read of K and V.
//
// Layout of the work: the 128 rows of a query tile are tq = floor(128 / G)
// tokens times the G query heads of one K/V head, so K and V are read once
// per group and few tokens still fill rows.  An item is two query tiles of one
// (sequence, K/V head); the items of a sequence run latest (heaviest) first.
// One CTA per SM; a CTA takes its first item from its index and then the
// items of CTAs that have not started (clusterlaunchcontrol), so the work
// balances itself without a counter in memory.  An item walks the 128-token
// context tiles that some row of it sees: the tile in which its first row's
// window begins, the tiles of the first tokens, the window's others.  The
// second query tile skips the first one where its window has left it.
//
// Roles in a CTA (10 warps), as pipelines over mbarriers:
//   * warp 8 loads: TMA boxes of Q rows (64 dims x G heads x tq tokens), then
//     K and V, one box per block run, into a ring of four 128-byte-swizzled
//     tiles; runs that no row sees are not looked up or read;
//   * warp 9, one thread: S_t = Q_t K^T into TMEM, O_t += P_t V with P_t read
//     from TMEM, in the order S_0 PV_0 S_0' PV_1 S_1' so that the matrix unit
//     works on one tile while the other's softmax runs;
//   * warps 0-3 / 4-7: softmax of tile 0 / 1, one row per thread (TMEM lane).
//     Only tiles that cross an edge of the mask pay for it.  Warps without
//     rows only keep the pipeline's count.
// TMEM: S0, S1 at columns 0 and 128 (P over S), O0, O1 from column 256.
// Every wait is bounded; one that runs out records PA_DEVERR_TIMEOUT and ends
// all roles, after which copies and matrix work in flight are drained.
//
// Choices of fewer bits: P enters the product with V in the cache's 16-bit
// type, 2^7 times larger than the softmax's weights (below 2^15 with the
// stale reference), which keeps weights down to 2^-31 of the largest in fp16.
// The row sums are taken from the unrounded weights.
#pragma once

#include <cuda.h>
#include <cstdint>

#include "../../include/pa_window.h"
#include "half_types.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"
#include "tile_softmax.cuh"

namespace pa {

struct WindowPrefillParams {
    void *out;                    // [num_rows, heads, D]
    const int32_t *tables;        // [B, max_blocks]
    const int32_t *lens;          // [B]
    const int32_t *starts;        // [B + 1]
    int max_blocks, max_len, max_new, window, sinks;
    int num_seqs, heads, kv_heads, group, tq;
    int log2_bs, num_blocks, num_rows;
    float scale_log2;             // softmax scale * log2(e), > 0
    unsigned int *err;
};

namespace wp {

constexpr int kM = 128;               // rows per query tile
constexpr int kN = 128;               // context tokens per tile
constexpr int kTiles = 2;             // query tiles per item
constexpr int kRing = 4;              // K / V tile slots
constexpr int kItemRing = 2;
constexpr int kItemConsumers = 1 + 8; // the MMA thread and the eight softmax warps
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 10 * 32;
constexpr uint32_t kTmemCols = 512, kTmemO = 2 * kN;
constexpr float kRescaleLog2 = 8.0f;  // move the reference only past this growth
constexpr float kShift = 7.0f;        // weights are 2^7 times the softmax's
constexpr float kFloor = -1e30f;      // reference of a row that has seen nothing yet

template <int D>
struct Shape {
    static constexpr int kHalves = D / 64;                     // 64-wide halves of a row
    static constexpr uint32_t kSub = kM * 128;                 // one half of a Q tile
    static constexpr uint32_t kTileBytes = kHalves * kSub;     // a Q, K or V tile
    static constexpr uint32_t kGroupBytes = 8 * D * 2;         // 8 context rows
    static constexpr uint32_t kOffRing = kTiles * kTileBytes;
    static constexpr uint32_t kSmem = kOffRing + kRing * kTileBytes + 1024;  // + alignment slack
};

// Two query tiles (up to 2 tq new tokens) of one (sequence, K/V head).
struct Item {
    int b, h, L, token;        // token: row of q of the item's first query
    int rows[kTiles];          // new tokens in query tile t (0: absent)
    int pos0[kTiles];          // position of the tile's first token
    int lo;                    // first position of the first token's window
    int first, sink_tiles;     // context tile of lo; tiles of first tokens before it
    int begin[kTiles], end[kTiles];  // steps of the walk that tile t takes part in
    int steps;                 // 0: no more items

    // Context tile of step j: the window's first, the first tokens', the rest.
    __device__ __forceinline__ int tile(int j) const
    {
        return j == 0 ? first : j <= sink_tiles ? j - 1 : first + j - sink_tiles;
    }
};

struct Shared {
    uint64_t item_full[kItemRing], item_empty[kItemRing];
    uint64_t q_full, q_empty, drain, next_full;
    uint64_t kv_full[kRing], kv_empty[kRing];
    uint64_t s_full[kTiles], p_full[kTiles], o_full[kTiles], o_empty[kTiles];
    alignas(16) uint64_t next[2];  // answer about a CTA that has not started
    Item item[kItemRing];
    uint32_t tmem;
    int abort;
};

// Bounded wait that also gives up as soon as another role raised the abort flag.
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int *abort,
                                              unsigned int *err)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort)
            return false;
        if (global_timer_ns() - t0 > kWaitLimitNs) {
            atomicOr(err, PA_DEVERR_TIMEOUT);
            *abort = 1;
            return false;
        }
    }
    return true;
}

// New tokens of sequence b that can be worked on (0 where its arguments are
// wrong: more new tokens than context or than announced, rows outside q).
__device__ __forceinline__ int new_tokens(const WindowPrefillParams &p, int b, int &first, int &L,
                                          unsigned &bad)
{
    first = p.starts[b];
    const long long n = (long long)p.starts[b + 1] - first;
    L = p.lens[b];
    bad = L < 0 || L > p.max_len ? PA_DEVERR_CONTEXT_LEN : 0u;
    L = max(0, min(L, p.max_len));
    if (n <= 0)
        return 0;
    if (first < 0 || n > p.num_rows - first || n > L || n > p.max_new) {
        bad = PA_DEVERR_CONTEXT_LEN;
        return 0;
    }
    return int(n);
}

// Finds items by number: the items of sequence 0, then 1, ...  A whole warp
// works on it, 32 sequences at a time; numbers mostly come in rising order.
struct Cursor {
    int base_b = 0;
    long long base_k = 0;

    __device__ __forceinline__ bool find(const WindowPrefillParams &p, int k, int lane, Item &it)
    {
        if (k < base_k)
            base_b = 0, base_k = 0;
        const int per_item = kTiles * p.tq;
        for (; base_b < p.num_seqs; base_b += 32) {
            int n = 0, first = 0, L = 0;
            unsigned bad = 0;
            if (base_b + lane < p.num_seqs)
                n = new_tokens(p, base_b + lane, first, L, bad);
            const long long mine = (long long)((n + per_item - 1) / per_item) * p.kv_heads;
            long long incl = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const long long o = __shfl_up_sync(kFullMask, incl, off);
                incl += lane >= off ? o : 0;
            }
            const unsigned past = __ballot_sync(kFullMask, base_k + incl > k);
            if (past) {
                const int src = __ffs(past) - 1;
                n = __shfl_sync(kFullMask, n, src);
                first = __shfl_sync(kFullMask, first, src);
                L = __shfl_sync(kFullMask, L, src);
                const int r = int(k - base_k - __shfl_sync(kFullMask, incl - mine, src));
                fill(p, base_b + src, n, first, L, r, it);
                return true;
            }
            base_k += __shfl_sync(kFullMask, incl, 31);
        }
        return false;
    }

    // Item r of sequence b: the latest tokens first, all K/V heads of them.
    static __device__ __forceinline__ void fill(const WindowPrefillParams &p, int b, int n,
                                                int q_first, int L, int r, Item &it)
    {
        const int per_item = kTiles * p.tq;
        const int pair = (n + per_item - 1) / per_item - 1 - r / p.kv_heads;
        const int row0 = pair * per_item;
        it.b = b;
        it.h = r % p.kv_heads;
        it.L = L;
        it.token = q_first + row0;
        const int pos = L - n + row0;                      // position of the item's first token
        it.lo = pos - p.window + 1 > 0 ? pos - p.window + 1 : 0;
        it.first = it.lo / kN;
        it.sink_tiles = min((min(p.sinks, it.lo) + kN - 1) / kN, it.first);
        it.steps = 0;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            it.rows[t] = max(0, min(p.tq, n - row0 - t * p.tq));
            it.pos0[t] = pos + t * p.tq;
            const int last = it.pos0[t] + it.rows[t] - 1;
            const int lo_t = max(0, it.pos0[t] - p.window + 1);
            // the window's first tile is left out where it lies wholly
            // before the tile's own window and holds no first token
            it.begin[t] = lo_t >= (it.first + 1) * kN && p.sinks <= it.first * kN ? 1 : 0;
            it.end[t] = it.rows[t] > 0 ? it.sink_tiles + last / kN + 1 - it.first : 0;
            it.steps = max(it.steps, it.end[t]);
        }
    }
};

// ---- work of CTAs that have not started ------------------------------------

__device__ __forceinline__ void ask_next(Shared &sh)
{
    mbar_arrive_expect_tx(smem_u32(&sh.next_full), 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
                 "[%0], [%1];" ::"r"(smem_u32(sh.next)),
                 "r"(smem_u32(&sh.next_full))
                 : "memory");
}

// Index of the CTA whose work was taken over, or -1.
__device__ __forceinline__ int next_cta(Shared &sh)
{
    int x;
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
                 "ld.shared.b128 r, [%1];\n\t"
                 "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
                 "mov.b32 %0, -1;\n\t"
                 "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n\t}"
                 : "=r"(x)
                 : "r"(smem_u32(sh.next))
                 : "memory");
    fence_proxy_async_smem();  // the answer has been read before it is overwritten
    return x;
}

// ---------------------------------------------------------------- loads
template <int D>
__device__ __forceinline__ void load_role(const CUtensorMap *tm_q, const CUtensorMap *tm_k,
                                          const CUtensorMap *tm_v, const WindowPrefillParams &p,
                                          Shared &sh, uint32_t sbase, int lane)
{
    using S = Shape<D>;
    volatile int *abort = &sh.abort;
    const int bs = 1 << p.log2_bs, box = min(bs, kN);
    const uint32_t q_bytes = uint32_t(p.tq * p.group) * 128u * S::kHalves;
    int last_use[kRing];
#pragma unroll
    for (int i = 0; i < kRing; ++i)
        last_use[i] = -1;
    Cursor cursor;
    int ring = 0, items = 0, asked = 0;
    int k = blockIdx.x;
    bool go = true;
    while (go) {
        Item it;
        it.steps = 0;
        const bool found = k >= 0 && cursor.find(p, k, lane, it);
        const int slot = items % kItemRing, use = items / kItemRing;
        bool ok = true;
        if (lane == 0) {
            if (use > 0)
                ok = wait_or_abort(smem_u32(&sh.item_empty[slot]), uint32_t(use - 1) & 1u, abort, p.err);
            if (ok) {
                sh.item[slot] = it;
                mbar_arrive(smem_u32(&sh.item_full[slot]));  // release: the item is visible
                if (found)
                    ask_next(sh);
            }
        }
        if (!__shfl_sync(kFullMask, int(ok), 0) || !found)
            break;
        ++asked;
        // Q once the previous item's score products are done
        if (lane == 0) {
            if (items > 0)
                ok = wait_or_abort(smem_u32(&sh.q_empty), uint32_t(items - 1) & 1u, abort, p.err);
            if (ok) {
                const uint32_t full = smem_u32(&sh.q_full);
                mbar_arrive_expect_tx(full, (it.rows[1] > 0 ? 2u : 1u) * q_bytes);
                for (int t = 0; t < kTiles; ++t)
                    for (int hf = 0; hf < S::kHalves && it.rows[t] > 0; ++hf)
                        tma_load_3d(sbase + uint32_t(t) * S::kTileBytes + uint32_t(hf) * S::kSub, tm_q,
                                    hf * 64, it.h * p.group, it.token + t * p.tq, full);
            }
        }
        if (!__shfl_sync(kFullMask, int(ok), 0))
            break;
        ++items;
        const int32_t *trow = p.tables + size_t(it.b) * p.max_blocks;
        for (int j = 0; go && j < it.steps; ++j) {
            // one run of up to a block per lane
            const int tok = it.tile(j) * kN + lane * box;
            const bool seen = lane * box < kN && tok < it.L && (tok + box > it.lo || tok < p.sinks);
            bool ok_id = false;
            int y = 0;
            if (seen) {
                const int id = trow[tok >> p.log2_bs];
                ok_id = unsigned(id) < unsigned(p.num_blocks);
                if (!ok_id)
                    atomicOr(p.err, PA_DEVERR_BLOCK_ID);
                // in groups of 8 rows
                y = ok_id ? int((((long long)id * p.kv_heads + it.h) * bs + (tok & (bs - 1))) >> 3) : 0;
            }
            const uint32_t bytes = uint32_t(__popc(__ballot_sync(kFullMask, ok_id))) * uint32_t(box) *
                                   uint32_t(D * 2);
#pragma unroll
            for (int kind = 0; kind < 2; ++kind) {  // K, then V
                const int i = ring + 2 * j + kind, slot_kv = i % kRing, use_kv = i / kRing;
                const uint32_t full = smem_u32(&sh.kv_full[slot_kv]);
                if (lane == 0) {
                    if (use_kv > 0)
                        ok = wait_or_abort(smem_u32(&sh.kv_empty[slot_kv]), uint32_t(use_kv - 1) & 1u,
                                           abort, p.err);
                    if (ok)
                        mbar_arrive_expect_tx(full, bytes);
                }
                if (!(go = __shfl_sync(kFullMask, int(ok), 0) != 0))
                    break;
                last_use[slot_kv] = use_kv;
                if (ok_id)
                    tma_load_4d(sbase + S::kOffRing + uint32_t(slot_kv) * S::kTileBytes +
                                    uint32_t(lane * box / 8) * S::kGroupBytes,
                                kind == 0 ? tm_k : tm_v, 0, 0, 0, y, full);
            }
        }
        ring += 2 * it.steps;
        if (!go)
            break;
        if (lane == 0)
            ok = wait_or_abort(smem_u32(&sh.next_full), uint32_t(asked - 1) & 1u, abort, p.err);
        if (!__shfl_sync(kFullMask, int(ok), 0))
            break;
        k = __shfl_sync(kFullMask, lane == 0 ? next_cta(sh) : 0, 0);
    }
    // After an abort, let what was asked for land before the shared memory goes away.
    if (*abort && lane == 0) {
        for (int i = 0; i < kRing; ++i)
            if (last_use[i] >= 0)
                mbar_wait_bounded(smem_u32(&sh.kv_full[i]), uint32_t(last_use[i]) & 1u);
        if (items > 0)
            mbar_wait_bounded(smem_u32(&sh.q_full), uint32_t(items - 1) & 1u);
        if (asked > 0)
            mbar_wait_bounded(smem_u32(&sh.next_full), uint32_t(asked - 1) & 1u);
    }
}

// ------------------------------------------------------------ matrix unit
template <int D, bool kBf16>
__device__ __forceinline__ void mma_role(const WindowPrefillParams &p, Shared &sh, uint32_t sbase)
{
    using S = Shape<D>;
    constexpr uint32_t kIdescS = idesc_16_f32(kM, kN, false, kBf16);
    constexpr uint32_t kIdescO = idesc_16_f32(kM, D, true, kBf16);
    volatile int *abort = &sh.abort;
    const uint32_t tmem = sh.tmem;
    auto slot_addr = [&](int i) { return sbase + S::kOffRing + uint32_t(i % kRing) * S::kTileBytes; };
    auto wait_full = [&](int i) {
        const bool ok = wait_or_abort(smem_u32(&sh.kv_full[i % kRing]), uint32_t(i / kRing) & 1u, abort,
                                      p.err);
        tc_fence_after_sync();
        return ok;
    };
    // K: rows of 8-row groups kGroupBytes apart, halves 1 KB apart
    auto issue_s = [&](int t, uint32_t k_addr) {
        const uint32_t q_addr = sbase + uint32_t(t) * S::kTileBytes;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            const uint32_t hf = uint32_t(k >> 2), kk = uint32_t(k & 3) * 32u;
            umma_f16(tmem + uint32_t(t) * kN, smem_desc_sw128(q_addr + hf * S::kSub + kk, 16, 1024),
                     smem_desc_sw128(k_addr + hf * 1024u + kk, 16, S::kGroupBytes), kIdescS, k > 0);
        }
        umma_commit(smem_u32(&sh.s_full[t]));
    };
    auto issue_pv = [&](int t, uint32_t v_addr, bool accumulate) {
        const uint32_t p_tmem = tmem + uint32_t(t) * kN;  // P aliases S
        const uint32_t o_tmem = tmem + kTmemO + uint32_t(t) * D;
#pragma unroll
        for (int k = 0; k < kN / 16; ++k)
            umma_f16_ts(o_tmem, p_tmem + uint32_t(k) * 8u,
                        smem_desc_sw128(v_addr + uint32_t(k) * 2u * S::kGroupBytes, 1024, S::kGroupBytes),
                        kIdescO, accumulate || k > 0);
        umma_commit(smem_u32(&sh.o_full[t]));
    };

    int ring = 0;
    int cnt[kTiles] = {0, 0};       // steps taken per query tile (all items)
    int t_items[kTiles] = {0, 0};   // items in which query tile t took part
    bool ok = true;
    for (int u = 0; ok; ++u) {
        const int slot = u % kItemRing;
        if (!wait_or_abort(smem_u32(&sh.item_full[slot]), uint32_t(u / kItemRing) & 1u, abort, p.err))
            break;
        const int steps = sh.item[slot].steps;
        const int b0 = sh.item[slot].begin[0], b1 = sh.item[slot].begin[1];
        const int e0 = sh.item[slot].end[0], e1 = sh.item[slot].end[1];
        mbar_arrive(smem_u32(&sh.item_empty[slot]));
        if (steps == 0)
            break;
        auto in0 = [&](int j) { return j >= b0 && j < e0; };
        auto in1 = [&](int j) { return j >= b1 && j < e1; };
        // P V of tile t at step j: the softmax has written P_t, and, at the
        // tile's first step, the previous item's epilogue has read O_t
        auto pv = [&](int t, int j, int begin, uint32_t v_addr) {
            if (j == begin && t_items[t] > 0 &&
                !wait_or_abort(smem_u32(&sh.o_empty[t]), uint32_t(t_items[t] - 1) & 1u, abort, p.err))
                return false;
            if (!wait_or_abort(smem_u32(&sh.p_full[t]), uint32_t(cnt[t] + j - begin) & 1u, abort, p.err))
                return false;
            tc_fence_after_sync();
            issue_pv(t, v_addr, j > begin);
            return true;
        };
        if (!(ok = wait_or_abort(smem_u32(&sh.q_full), uint32_t(u) & 1u, abort, p.err) &&
                   wait_full(ring)))
            break;
        if (in0(0))
            issue_s(0, slot_addr(ring));
        if (in1(0))
            issue_s(1, slot_addr(ring));
        umma_commit(smem_u32(&sh.kv_empty[ring % kRing]));
        if (steps == 1)
            umma_commit(smem_u32(&sh.q_empty));  // last score product of the item issued
        for (int j = 0; j < steps; ++j) {
            const int iv = ring + 2 * j + 1, ik = ring + 2 * j + 2;
            const bool next = j + 1 < steps;
            if (!(ok = wait_full(iv)))
                break;
            if (in0(j) && !(ok = pv(0, j, b0, slot_addr(iv))))
                break;
            if (next) {
                if (!(ok = wait_full(ik)))
                    break;
                if (in0(j + 1))
                    issue_s(0, slot_addr(ik));
            }
            if (in1(j) && !(ok = pv(1, j, b1, slot_addr(iv))))
                break;
            umma_commit(smem_u32(&sh.kv_empty[iv % kRing]));
            if (next) {
                if (in1(j + 1))
                    issue_s(1, slot_addr(ik));
                umma_commit(smem_u32(&sh.kv_empty[ik % kRing]));
                if (j + 2 == steps)
                    umma_commit(smem_u32(&sh.q_empty));
            }
        }
        if (e0 > 0)
            cnt[0] += e0 - b0, ++t_items[0];
        if (e1 > 0)
            cnt[1] += e1 - b1, ++t_items[1];
        ring += 2 * steps;
    }
    // every matrix operation issued has finished before TMEM and the shared
    // tiles are released
    umma_commit(smem_u32(&sh.drain));
    mbar_wait_bounded(smem_u32(&sh.drain), 0u);
}

// ---------------------------------------------------------------- softmax

// Bits [a, b) of a 32-bit word (a, b anywhere).
__device__ __forceinline__ uint32_t bits_between(int a, int b)
{
    const uint32_t up = b >= 32 ? ~0u : b <= 0 ? 0u : (1u << b) - 1u;
    const uint32_t down = a >= 32 ? ~0u : a <= 0 ? 0u : (1u << a) - 1u;
    return up & ~down;
}

// Columns the row does not see become -inf: it sees [lo, lim) and [0, sinks).
__device__ __forceinline__ void mask_row(ScoreRow &r, int lo, int lim, int sinks)
{
    const int s = min(sinks, lim);
#pragma unroll
    for (int w = 0; w < kN / 32; ++w) {
        const uint32_t m = bits_between(lo - 32 * w, lim - 32 * w) | bits_between(0, s - 32 * w);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (!((m >> i) & 1u))
                r.s[32 * w + i] = 0xff800000u;
    }
}

// P = 2^(c * s - m) of the row, as 16-bit pairs over the first 64 columns of
// S; returns the row sum of the unrounded P.
template <bool kBf16>
__device__ __forceinline__ float write_weights(uint32_t tS, const ScoreRow &r, float c, float m)
{
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int cc = 0; cc < kN / 32; ++cc) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int i = cc * 32 + 2 * e;
            const float p0 = ex2_approx(fmaf(__uint_as_float(r.s[i]), c, -m));
            const float p1 = ex2_approx(fmaf(__uint_as_float(r.s[i + 1]), c, -m));
            sum[(e & 1) * 2] += p0;
            sum[(e & 1) * 2 + 1] += p1;
            pk[e] = Half16<kBf16>::pack(p0, p1);
        }
        tmem_store16(tS + uint32_t(cc * 16), pk);
    }
    return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

template <int D, bool kBf16>
__device__ __forceinline__ void softmax_role(const WindowPrefillParams &p, Shared &sh,
                                             unsigned char *smem, int warp, int lane)
{
    using S = Shape<D>;
    volatile int *abort = &sh.abort;
    const int t = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const int r_token = r / p.group, r_head = r % p.group;
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tS = sh.tmem + uint32_t(t) * kN + lane_base;
    const uint32_t tO = sh.tmem + kTmemO + uint32_t(t) * D + lane_base;
    const float c = p.scale_log2;
    int ring = 0, cnt = 0;
    for (int u = 0;; ++u) {
        const int slot = u % kItemRing;
        if (!__all_sync(kFullMask, wait_or_abort(smem_u32(&sh.item_full[slot]),
                                                 uint32_t(u / kItemRing) & 1u, abort, p.err)))
            break;
        const Item it = sh.item[slot];
        __syncwarp();
        if (lane == 0)
            mbar_arrive(smem_u32(&sh.item_empty[slot]));
        if (it.steps == 0)
            break;
        const int item_ring = ring;
        ring += 2 * it.steps;
        if (it.rows[t] <= 0)
            continue;
        const bool live = (warp & 3) * 32 < it.rows[t] * p.group;  // the warp holds rows
        const int my_pos = it.pos0[t] + r_token;
        const int my_lo = max(0, my_pos - p.window + 1), my_end = min(my_pos + 1, it.L);
        const int begin = it.begin[t], end = it.end[t];
        float m_ref = kFloor, l = 0.f;
        bool ok = true;
        for (int j = begin; j < end; ++j) {
            ok = __all_sync(kFullMask, wait_or_abort(smem_u32(&sh.s_full[t]),
                                                     uint32_t(cnt + j - begin) & 1u, abort, p.err));
            if (!ok)
                break;
            tc_fence_after_sync();
            const int t0 = it.tile(j) * kN;
            if (live) {
                ScoreRow row;
                load_score_row(tS, row);
                const int lo = my_lo - t0, lim = my_end - t0, sinks = p.sinks - t0;
                if (__any_sync(kFullMask, lim < kN || (lo > 0 && sinks < kN)))
                    mask_row(row, lo, lim, sinks);
                const float m_new = fmaxf(m_ref, score_row_max<false>(row, kN) * c);
                if (j == begin) {
                    m_ref = m_new;
                } else if (__any_sync(kFullMask, m_new > m_ref + kRescaleLog2)) {
                    // move this warp's reference: rescale O and l
                    ok = __all_sync(kFullMask, wait_or_abort(smem_u32(&sh.o_full[t]),
                                                             uint32_t(cnt + j - begin - 1) & 1u, abort,
                                                             p.err));
                    if (!ok)
                        break;
                    tc_fence_after_sync();
                    const float alpha = ex2_approx(m_ref - m_new);
#pragma unroll 1
                    for (int cc = 0; cc < D / 16; ++cc) {  // 16 columns at a time: the score row is live
                        uint32_t o[16];
                        tmem_load16_async(tO + uint32_t(cc * 16), o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tmem_store16(tO + uint32_t(cc * 16), o);
                    }
                    l *= alpha;
                    m_ref = m_new;
                }
                l += write_weights<kBf16>(tS, row, c, m_ref - kShift);
                tmem_wait_st();
            }
            // V rows that no row of the item sees (behind the context, before
            // the window, stale ring contents) are zeroed, so that 0 * garbage
            // cannot reach O.  Done by the first tile that uses the step.
            if ((t0 + kN > it.L || (t0 < it.lo && t0 + kN > p.sinks)) && t == (j < it.end[0] ? 0 : 1)) {
                const int iv = item_ring + 2 * j + 1;
                ok = __all_sync(kFullMask, wait_or_abort(smem_u32(&sh.kv_full[iv % kRing]),
                                                         uint32_t(iv / kRing) & 1u, abort, p.err));
                if (!ok)
                    break;
                const int tok = t0 + r;
                if (!(tok < it.L && (tok >= it.lo || tok < p.sinks))) {
                    unsigned char *at = smem + S::kOffRing + uint32_t(iv % kRing) * S::kTileBytes +
                                        uint32_t(r >> 3) * S::kGroupBytes + uint32_t(r & 7) * 128u;
#pragma unroll
                    for (int hf = 0; hf < S::kHalves; ++hf)
#pragma unroll
                        for (int q16 = 0; q16 < 8; ++q16)
                            *reinterpret_cast<uint4 *>(at + hf * 1024 + q16 * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&sh.p_full[t]));
        }
        if (!ok)
            break;
        // epilogue: out = O / l, then O_t is free for the next item
        ok = __all_sync(kFullMask, wait_or_abort(smem_u32(&sh.o_full[t]),
                                                 uint32_t(cnt + end - begin - 1) & 1u, abort, p.err));
        if (!ok)
            break;
        cnt += end - begin;
        if (live) {
            tc_fence_after_sync();
            const float inv = 1.f / l;
            const bool store = r < it.rows[t] * p.group;
            const size_t token = size_t(it.token) + t * p.tq + r_token;
            uint4 *dst = reinterpret_cast<uint4 *>(
                static_cast<uint16_t *>(p.out) + (token * p.heads + it.h * p.group + r_head) * D);
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
                uint32_t o[32];
                tmem_load32_async(tO + uint32_t(cc * 32), o);
                tmem_wait_ld();
                if (store) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        uint32_t v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = Half16<kBf16>::pack(__uint_as_float(o[g * 8 + 2 * e]) * inv,
                                                       __uint_as_float(o[g * 8 + 2 * e + 1]) * inv);
                        dst[cc * 4 + g] = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                }
            }
            tc_fence_before_sync();
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(smem_u32(&sh.o_empty[t]));
    }
}

} // namespace wp

template <int D, bool kBf16>
__global__ void __launch_bounds__(wp::kThreads, 1)
    window_prefill_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const WindowPrefillParams p)
{
    using namespace wp;
    using S = Shape<D>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    grid_dependency_wait();
    allow_dependent_launch();

    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    unsigned char *smem = smem_raw + (sbase - raw);
    if (tid == 0) {
        for (int i = 0; i < kItemRing; ++i) {
            mbar_init(smem_u32(&sh.item_full[i]), 1);
            mbar_init(smem_u32(&sh.item_empty[i]), kItemConsumers);
        }
        mbar_init(smem_u32(&sh.q_full), 1);
        mbar_init(smem_u32(&sh.q_empty), 1);
        mbar_init(smem_u32(&sh.drain), 1);
        mbar_init(smem_u32(&sh.next_full), 1);
        for (int i = 0; i < kRing; ++i) {
            mbar_init(smem_u32(&sh.kv_full[i]), 1);
            mbar_init(smem_u32(&sh.kv_empty[i]), 1);
        }
        for (int t = 0; t < kTiles; ++t) {
            mbar_init(smem_u32(&sh.s_full[t]), 1);
            mbar_init(smem_u32(&sh.p_full[t]), 4);   // one arrival per softmax warp
            mbar_init(smem_u32(&sh.o_full[t]), 1);
            mbar_init(smem_u32(&sh.o_empty[t]), 4);
        }
        sh.abort = 0;
        fence_mbar_init();
    }
    // rows of a query tile that the boxes do not fill (128 is no multiple of G)
    for (int i = tid; i < kTiles * S::kHalves * (kM - p.tq * p.group) * 8; i += kThreads) {
        const int sub = i / ((kM - p.tq * p.group) * 8), at = i % ((kM - p.tq * p.group) * 8);
        *reinterpret_cast<uint4 *>(smem + uint32_t(sub) * S::kSub + uint32_t(p.tq * p.group) * 128u +
                                   uint32_t(at) * 16u) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    if (warp == kMmaWarp)
        tmem_alloc(smem_u32(&sh.tmem), kTmemCols);
    if (blockIdx.x == 0)  // one CTA records wrong arguments
        for (int b = tid; b < p.num_seqs; b += kThreads) {
            int first, L;
            unsigned bad;
            new_tokens(p, b, first, L, bad);
            if (bad)
                atomicOr(p.err, bad);
        }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();

    if (warp == kLoadWarp) {
        load_role<D>(&tm_q, &tm_k, &tm_v, p, sh, sbase, lane);
    } else if (warp == kMmaWarp) {
        if (lane == 0)
            mma_role<D, kBf16>(p, sh, sbase);
        __syncwarp();
    } else {
        softmax_role<D, kBf16>(p, sh, smem, warp, lane);
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after_sync();
        tmem_free(sh.tmem, kTmemCols);
    }
}

} // namespace pa
