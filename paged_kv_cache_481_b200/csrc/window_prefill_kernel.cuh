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
// Measured (one B200; long runs, where the power limit holds the clock near
// 1725 MHz, and in brackets bursts at 1965 MHz): one prompt of 8192, window
// 4096, H 32, KVH 8, bf16: 422 us (373), 0.98 PFLOP/s of visible pairs (1.10), 59
// % of the library product's rate (67 %); 8 chunks of 100 to 512 queries, 40
// heads, fp16: 112 us (100), 560 items where 396 would hold all rows, 4 to 5 us
// between items; 16 sequences of 1 to 7 queries: 21.4 us, one wave of dependent
// steps of 0.9 us with 4 to 28 of 256 rows in use.
//
// Layout of the work: the 128 rows of a query tile are tq = floor(128 / G)
// tokens times the G query heads of one K/V head, so K and V are read once
// per group and few tokens still fill rows.  An item is two query tiles of one
// (sequence, K/V head); the items of a sequence run latest (heaviest) first.
// One CTA per SM; a CTA takes its first item from its index and then the
// items of CTAs that have not started (clusterlaunchcontrol), so the work
// balances itself without a counter in memory.  An item walks the 128-token
// context tiles that some row of it sees, half a tile (64 tokens) a step: the
// tile in which its first row's window begins, the tiles of the first tokens,
// the window's others.  Steps at either end that a query tile does not see
// are left out for it.
//
// Roles in a CTA (11 warps), as pipelines over mbarriers:
//   * warp 8 loads: TMA boxes of Q rows (64 dims x G heads x tq tokens), then
//     K and V, one box per block run, into a ring of five 128-byte-swizzled
//     tiles; runs that no row sees are not looked up or read;
//   * warps 9 and 10, tile 0 and 1: S_t = Q_t K^T of 64 tokens into one of two
//     TMEM buffers a query tile, one step ahead, and O_t += P_t V with P_t read
//     from TMEM, so that the softmax warps do not wait for the matrix unit.
//     The issue of a product takes about 130 clocks next to busy softmax
//     warps, twice what the product takes: hence a warp for each tile;
//   * warps 0-3 / 4-7: softmax of tile 0 / 1, one row per thread (TMEM lane).
//     Only steps that cross an edge of the mask pay for it.  Warps without
//     rows, and steps a tile does not take part in, only keep the count.
// TMEM: S_t buffers at columns 128 t and 128 t + 64 (P over S), O_t from
// column 256.  Every wait is bounded; one that runs out records
// PA_DEVERR_TIMEOUT and ends all roles, after which copies and matrix work in
// flight are drained.
//
// Choices of fewer bits: P enters the product with V in the cache's 16-bit
// type.  fp16: 2^7 times larger than the softmax's weights (below 2^15 with
// the stale reference), which keeps weights down to 2^-31 of the largest.
// bf16: small enough for the largest V (weight_shift in window_host.cuh).
// The row sums are taken from the unrounded weights.  (Two 16-bit numbers a
// weight took 549 us against 438 on the prompt, 138 against 109 on the chunks.)
#pragma once

#include <cuda.h>
#include <cstdint>

#include "../../include/pa_window.h"
#include "half_types.cuh"
#include "mma_sync.cuh"
#include "ptx.cuh"
#include "tcgen05_window.cuh"

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
    float shift;                  // weights are 2^shift times the softmax's
    unsigned int *err;
};

namespace wp {

constexpr int kM = 128;               // rows per query tile
constexpr int kN = 128;               // context tokens per K / V tile
constexpr int kHalf = 64;             // context tokens per step
constexpr int kTiles = 2;             // query tiles per item
constexpr int kRing = 5;              // K / V tile slots
constexpr int kItemRing = 2;
constexpr int kItemConsumers = 2 + 8; // the matrix warps and the softmax warps
constexpr int kLoadWarp = 8, kMmaWarp = 9;
constexpr int kThreads = (kMmaWarp + kTiles) * 32;
constexpr uint32_t kTmemCols = 512, kTmemO = 2 * kN;
constexpr float kRescaleLog2 = 8.0f;  // move the reference only past this growth
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
    int begin[kTiles], end[kTiles];  // steps (half tiles) of the walk that tile t takes part in
    int tiles;                 // context tiles of the walk; 0: no more items

    // Context tile j of the walk: the window's first, the first tokens', the rest.
    static __device__ __forceinline__ int tile(int j, int first, int sink_tiles)
    {
        return j == 0 ? first : j <= sink_tiles ? j - 1 : first + j - sink_tiles;
    }
};

struct Shared {
    uint64_t item_full[kItemRing], item_empty[kItemRing];
    uint64_t q_full, q_empty, next_full;
    uint64_t kv_full[kRing], kv_empty[kRing];
    uint64_t s_full[kTiles][2], p_full[kTiles][2];
    uint64_t o_mid[kTiles], o_full[kTiles];  // an item's products but the last step's; all of them
    uint64_t o_empty[kTiles], drain[kTiles];
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
    if (n <= 0) {
        bad |= n < 0 ? PA_DEVERR_CONTEXT_LEN : 0u;
        return 0;
    }
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
        it.tiles = 0;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            it.rows[t] = max(0, min(p.tq, n - row0 - t * p.tq));
            it.pos0[t] = pos + t * p.tq;
            const int last = it.pos0[t] + it.rows[t] - 1;
            const int lo_t = max(0, it.pos0[t] - p.window + 1);
            // halves of the window's first tile are left out where they lie
            // wholly before the tile's own window and hold no first token
            const int skip = min(lo_t / kHalf - 2 * it.first, 2);
            it.begin[t] = p.sinks <= it.first * kN ? skip : 0;
            // (behind the first tokens' tiles the walk goes on with tile first + 1)
            const int halves = last / kHalf + 1 - 2 * it.first;
            it.end[t] = it.rows[t] <= 0        ? 0
                        : it.sink_tiles > 0 ? 2 * it.sink_tiles + max(halves, 2)
                                            : halves;
            it.tiles = max(it.tiles, (it.end[t] + 1) / 2);
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
        it.tiles = 0;
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
        // one run of up to a block per lane; the ids of the next tile's blocks
        // are on their way while this one's boxes wait for their places
        auto look_up = [&](int j) {
            const int tok = Item::tile(j, it.first, it.sink_tiles) * kN + lane * box;
            const bool seen = j < it.tiles && lane * box < kN && tok < it.L && (tok + box > it.lo || tok < p.sinks);
            return seen ? trow[tok >> p.log2_bs] : -2;  // -2: nothing of the run is seen
        };
        int ahead = look_up(0);
        for (int j = 0; go && j < it.tiles; ++j) {
            const int id = ahead;
            ahead = look_up(j + 1);
            const bool ok_id = unsigned(id) < unsigned(p.num_blocks);
            if (id != -2 && !ok_id)
                atomicOr(p.err, PA_DEVERR_BLOCK_ID);
            // in groups of 8 rows
            const int in_block = (Item::tile(j, it.first, it.sink_tiles) * kN + lane * box) & (bs - 1);
            const int y = ok_id ? int((((long long)id * p.kv_heads + it.h) * bs + in_block) >> 3) : 0;
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
        ring += 2 * it.tiles;
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

// The products of query tile t; the whole warp comes along, one lane issues.
template <int D, bool kBf16, int t>
__device__ __forceinline__ void mma_role(const WindowPrefillParams &p, Shared &sh, uint32_t sbase)
{
    using S = Shape<D>;
    constexpr uint32_t kIdescS = idesc_16_f32(kM, kHalf, false, kBf16);
    constexpr uint32_t kIdescO = idesc_16_f32(kM, D, true, kBf16);
    volatile int *abort = &sh.abort;
    const uint32_t tmem = sh.tmem;
    const uint32_t leader = elect_one();
    auto wait = [&](uint64_t &bar, int phase) {
        const bool ok = __all_sync(kFullMask, wait_or_abort(smem_u32(&bar), uint32_t(phase) & 1u, abort, p.err));
        tc_fence_after_sync();
        return ok;
    };
    auto commit = [&](uint64_t &bar) { umma_commit_if(leader, smem_u32(&bar)); };
    // half `h` of tile i of the ring
    auto half_addr = [&](int i, int h) {
        return sbase + S::kOffRing + uint32_t(i % kRing) * S::kTileBytes + uint32_t(h) * (S::kTileBytes / 2);
    };
    const uint64_t q_desc = smem_desc_sw128(sbase + uint32_t(t) * S::kTileBytes, 16, 1024);
    // K: rows of 8-row groups kGroupBytes apart, 64-dim halves 1 KB apart.
    // The scores overwrite the weights of the product before the last, which
    // the matrix unit takes up first: it works in the order of issue.
    auto issue_s = [&](int buf, uint32_t k_addr) {
        const uint32_t d = tmem + uint32_t(2 * t + buf) * kHalf;
        const uint64_t kd = smem_desc_sw128(k_addr, 16, S::kGroupBytes);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
            umma_f16_if(leader, d, q_desc + ((uint32_t(k >> 2) * S::kSub + uint32_t(k & 3) * 32u) >> 4),
                        kd + ((uint32_t(k >> 2) * 1024u + uint32_t(k & 3) * 32u) >> 4), kIdescS, k > 0);
        commit(sh.s_full[t][buf]);
    };
    auto issue_pv = [&](int buf, uint32_t v_addr, bool accumulate) {
        const uint32_t a = tmem + uint32_t(2 * t + buf) * kHalf;  // P aliases S
        const uint32_t d = tmem + kTmemO + uint32_t(t) * D;
        const uint64_t vd = smem_desc_sw128(v_addr, 1024, S::kGroupBytes);
#pragma unroll
        for (int k = 0; k < kHalf / 16; ++k)
            umma_f16_ts_if(leader, d, a + uint32_t(k) * 8u, vd + (uint32_t(k) * 2u * S::kGroupBytes >> 4),
                           kIdescO, accumulate || k > 0);
    };

    int ring = 0, s_cnt = 0, pv_cnt = 0, items = 0;  // (of this tile)
    bool ok = true;
    for (int u = 0; ok; ++u) {
        const int slot = u % kItemRing;
        if (!wait(sh.item_full[slot], u / kItemRing))
            break;
        const int tiles = sh.item[slot].tiles, begin = sh.item[slot].begin[t], end = sh.item[slot].end[t];
        __syncwarp();
        if (leader)
            mbar_arrive(smem_u32(&sh.item_empty[slot]));
        if (tiles == 0)
            break;
        // score product of step y, if the tile takes part in it
        auto scores = [&](int y) {
            const int i = ring + (y & ~1);
            if (!(y & 1) && !wait(sh.kv_full[i % kRing], i / kRing))
                return false;
            if (y >= begin && y < end)
                issue_s(s_cnt++ & 1, half_addr(i, y & 1));
            if (y & 1)
                commit(sh.kv_empty[i % kRing]);
            if (y == 2 * tiles - 1)
                commit(sh.q_empty);
            return true;
        };
        ok = wait(sh.q_full, u) && scores(0);
        for (int y = 0; ok && y < 2 * tiles; ++y) {
            const int iv = ring + (y & ~1) + 1;
            const bool mine = y >= begin && y < end;
            ok = (y + 1 >= 2 * tiles || scores(y + 1)) && ((y & 1) || wait(sh.kv_full[iv % kRing], iv / kRing));
            if (ok && mine) {
                // the previous item's epilogue has read O, the softmax has written P
                const int x = pv_cnt++;
                ok = (y > begin || items == 0 || wait(sh.o_empty[t], items - 1)) &&
                     wait(sh.p_full[t][x & 1], x >> 1);
                if (!ok)
                    break;
                issue_pv(x & 1, half_addr(iv, y & 1), y > begin);
                if (y == end - 2)
                    commit(sh.o_mid[t]);
                if (y == end - 1)
                    commit(sh.o_full[t]);
            }
            if (ok && (y & 1))
                commit(sh.kv_empty[iv % kRing]);
        }
        items += end > 0;
        ring += 2 * tiles;
    }
    // every matrix operation issued has finished before TMEM and the shared
    // tiles are released
    commit(sh.drain[t]);
    mbar_wait_bounded(smem_u32(&sh.drain[t]), 0u);
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
__device__ __forceinline__ void mask_row(uint32_t (&r)[kHalf], int lo, int lim, int sinks)
{
    const int s = min(sinks, lim);
#pragma unroll
    for (int w = 0; w < kHalf / 32; ++w) {
        const uint32_t m = bits_between(lo - 32 * w, lim - 32 * w) | bits_between(0, s - 32 * w);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (!((m >> i) & 1u))
                r[32 * w + i] = 0xff800000u;
    }
}

__device__ __forceinline__ float row_max(const uint32_t (&r)[kHalf])
{
    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < kHalf; i += 8)
#pragma unroll
        for (int a = 0; a < 4; ++a)
            m[a] = max3_f32(m[a], __uint_as_float(r[i + 2 * a]), __uint_as_float(r[i + 2 * a + 1]));
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// P = 2^(c * s - m) of the row as 16-bit pairs over the first 32 columns of its
// buffer; also the row sum of the unrounded P and the row maximum of s, which
// nothing here waits for.
template <bool kBf16>
__device__ __forceinline__ void write_weights(uint32_t tS, const uint32_t (&r)[kHalf], float c, float m,
                                              float &sum, float &largest)
{
    const uint64_t cc = pack_f32x2(c, c), mm = pack_f32x2(-m, -m);
    uint64_t total[2] = {0, 0};
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        uint32_t pk[kHalf / 4];
#pragma unroll
        for (int i = 0; i < kHalf / 4; ++i) {
            const int e = part * (kHalf / 4) + i;
            const uint64_t x = fma_f32x2(uint64_t(r[2 * e]) | uint64_t(r[2 * e + 1]) << 32, cc, mm);
            const float2 v = unpack_f32x2(x);
            const float p0 = exp2_sfu(v.x), p1 = exp2_sfu(v.y);
            total[e & 1] = add_f32x2(total[e & 1], pack_f32x2(p0, p1));
            pk[i] = Half16<kBf16>::pack(p0, p1);
            top[e & 1] = max3_f32(top[e & 1], __uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
        }
        tmem_store16(tS + uint32_t(part * (kHalf / 4)), pk);
    }
    const float2 v = unpack_f32x2(add_f32x2(total[0], total[1]));
    sum = v.x + v.y;
    largest = fmaxf(top[0], top[1]);
}

__device__ __forceinline__ uint16_t *shfl_pointer(uint16_t *v, int lane)
{
    return reinterpret_cast<uint16_t *>(__shfl_sync(kFullMask, reinterpret_cast<unsigned long long>(v), lane));
}

// Word i of four lanes (c = 0 .. 3) becomes the words of lane i, in order.
__device__ __forceinline__ uint4 transpose_quad(const uint32_t (&w)[4], int c)
{
    // with the neighbour: two words of column c & 1, two of 2 + (c & 1)
    const bool odd = c & 1, upper = c & 2;
    const uint32_t x = __shfl_xor_sync(kFullMask, odd ? w[0] : w[1], 1);
    const uint32_t y = __shfl_xor_sync(kFullMask, odd ? w[2] : w[3], 1);
    const uint32_t a0 = odd ? x : w[0], a1 = odd ? w[1] : x, b0 = odd ? y : w[2], b1 = odd ? w[3] : y;
    // with the other pair
    const uint32_t u = __shfl_xor_sync(kFullMask, upper ? a0 : b0, 2);
    const uint32_t v = __shfl_xor_sync(kFullMask, upper ? a1 : b1, 2);
    return upper ? make_uint4(u, v, b0, b1) : make_uint4(a0, a1, u, v);
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
    const uint32_t tS = sh.tmem + uint32_t(t) * 2u * kHalf + lane_base;
    const uint32_t tO = sh.tmem + kTmemO + uint32_t(t) * D + lane_base;
    const float c = p.scale_log2;
    int ring = 0, cnt = 0, mid = 0, items = 0;  // steps, items of two steps and more, items (of this tile)
    for (int u = 0;; ++u) {
        const int slot = u % kItemRing;
        if (!__all_sync(kFullMask, wait_or_abort(smem_u32(&sh.item_full[slot]),
                                                 uint32_t(u / kItemRing) & 1u, abort, p.err)))
            break;
        // (field by field: a copy would lie in local memory)
        const Item &it = sh.item[slot];
        const int tiles = it.tiles, first = it.first, sink_tiles = it.sink_tiles, L = it.L, lo = it.lo;
        const int head = it.h * p.group + r_head, token = it.token + t * p.tq + r_token;
        const int rows = it.rows[t], my_pos = it.pos0[t] + r_token, begin = it.begin[t], end = it.end[t];
        __syncwarp();
        if (lane == 0)
            mbar_arrive(smem_u32(&sh.item_empty[slot]));
        if (tiles == 0)
            break;
        const int item_ring = ring;
        ring += 2 * tiles;
        if (rows <= 0)
            continue;
        const bool live = (warp & 3) * 32 < rows * p.group;  // the warp holds rows
        const int my_lo = max(0, my_pos - p.window + 1), my_end = min(my_pos + 1, L);
        // no row of the warp needs a mask for tokens in [warp_lo, warp_end)
        const int warp_lo = __reduce_max_sync(kFullMask, my_lo), warp_end = __reduce_min_sync(kFullMask, my_end);
        float m_ref = kFloor, l = 0.f;
        bool ok = true;
        for (int y = begin; y < end; ++y) {
            const int x = cnt + y - begin, buf = x & 1;
            ok = __all_sync(kFullMask, wait_or_abort(smem_u32(&sh.s_full[t][buf]), uint32_t(x >> 1) & 1u,
                                                     abort, p.err));
            if (!ok)
                break;
            tc_fence_after_sync();
            const int t0 = Item::tile(y >> 1, first, sink_tiles) * kN + (y & 1) * kHalf;
            if (live) {
                uint32_t row[kHalf];
                tmem_load32_into(tS + uint32_t(buf) * kHalf, row);
                tmem_load32_into(tS + uint32_t(buf) * kHalf + 32u, row + 32);
                tmem_wait_ld();
                if (t0 + kHalf > warp_end || (t0 < warp_lo && t0 + kHalf > p.sinks))
                    mask_row(row, my_lo - t0, my_end - t0, p.sinks - t0);
                if (y == begin)
                    m_ref = fmaxf(m_ref, row_max(row) * c);
                // The weights are taken against the reference as it is; where a
                // score turns out to be too far above it, which is rare, it is
                // moved and they are taken again.
                float sum, largest;
                for (;;) {
                    write_weights<kBf16>(tS + uint32_t(buf) * kHalf, row, c, m_ref - p.shift, sum, largest);
                    const float m_new = fmaxf(m_ref, largest * c);
                    if (!__any_sync(kFullMask, m_new > m_ref + kRescaleLog2))
                        break;
                    // move this warp's reference: rescale O and l, once the
                    // last step's product is done, which the next scores or
                    // the end of the item tell
                    ok = __all_sync(kFullMask,
                                    y + 1 < end
                                        ? wait_or_abort(smem_u32(&sh.s_full[t][buf ^ 1]),
                                                        uint32_t((x + 1) >> 1) & 1u, abort, p.err)
                                        : wait_or_abort(smem_u32(&sh.o_mid[t]), uint32_t(mid) & 1u, abort,
                                                        p.err));
                    if (!ok)
                        break;
                    tc_fence_after_sync();
                    const float alpha = exp2_sfu(m_ref - m_new);
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
                    // stores to one place have no order of their own: the
                    // weights written first must not land on the next ones
                    tmem_wait_st();
                    l *= alpha;
                    m_ref = m_new;
                }
                if (!ok)
                    break;
                l += sum;
                tmem_wait_st();
            }
            // V rows that no row of the item sees (behind the context, before
            // the window, stale ring contents) are zeroed, so that 0 * garbage
            // cannot reach O: by each tile that takes part in the step, since
            // either may be first, two threads a row.
            if (t0 + kHalf > L || (t0 < lo && t0 + kHalf > p.sinks)) {
                const int iv = item_ring + (y & ~1) + 1;
                ok = __all_sync(kFullMask, wait_or_abort(smem_u32(&sh.kv_full[iv % kRing]),
                                                         uint32_t(iv / kRing) & 1u, abort, p.err));
                if (!ok)
                    break;
                const int vr = r >> 1, tok = t0 + vr;
                if (!(tok < L && (tok >= lo || tok < p.sinks))) {
                    unsigned char *at = smem + S::kOffRing + uint32_t(iv % kRing) * S::kTileBytes +
                                        uint32_t(y & 1) * (S::kTileBytes / 2) +
                                        uint32_t(vr >> 3) * S::kGroupBytes + uint32_t(vr & 7) * 128u;
#pragma unroll
                    for (int hf = 0; hf < S::kHalves; ++hf)
#pragma unroll
                        for (int q16 = 0; q16 < 4; ++q16)
                            *reinterpret_cast<uint4 *>(at + hf * 1024 + (r & 1) * 64 + q16 * 16) =
                                make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_u32(&sh.p_full[t][buf]));
        }
        if (!ok)
            break;
        // epilogue: out = O / l, then O_t is free for the next item
        ok = __all_sync(kFullMask, wait_or_abort(smem_u32(&sh.o_full[t]), uint32_t(items) & 1u, abort, p.err));
        if (!ok)
            break;
        cnt += end - begin;
        mid += end - begin > 1;
        ++items;
        if (live) {
            tc_fence_after_sync();
            // O comes in the layout of a matrix fragment (lane: row lane / 4 of 8,
            // two columns of every eight); the four lanes of a row exchange
            // until each holds 16 bytes, so that a store covers 64 bytes of 8
            // rows instead of 16 bytes of 32.
            const float inv = 1.f / l;
            uint16_t *my_dst = r < rows * p.group ? static_cast<uint16_t *>(p.out) +
                                                        (size_t(token) * p.heads + head) * D
                                                  : nullptr;
            const int g = lane >> 2, c4 = lane & 3;
#pragma unroll 1
            for (int part = 0; part < 2; ++part) {  // rows 16 part .. 16 part + 15 of the warp
                const float inv0 = __shfl_sync(kFullMask, inv, 16 * part + g);
                const float inv1 = __shfl_sync(kFullMask, inv, 16 * part + g + 8);
                uint16_t *dst0 = shfl_pointer(my_dst, 16 * part + g), *dst1 = shfl_pointer(my_dst, 16 * part + g + 8);
#pragma unroll
                for (int cc = 0; cc < D / 32; ++cc) {
                    uint32_t o[16], w[2][4];
                    tmem_load_16x256b_x4(tO + (uint32_t(16 * part) << 16) + uint32_t(cc * 32), o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        w[0][i] = Half16<kBf16>::pack(__uint_as_float(o[4 * i]) * inv0,
                                                      __uint_as_float(o[4 * i + 1]) * inv0);
                        w[1][i] = Half16<kBf16>::pack(__uint_as_float(o[4 * i + 2]) * inv1,
                                                      __uint_as_float(o[4 * i + 3]) * inv1);
                    }
                    const uint4 v0 = transpose_quad(w[0], c4), v1 = transpose_quad(w[1], c4);
                    if (dst0)
                        *reinterpret_cast<uint4 *>(dst0 + cc * 32 + c4 * 8) = v0;
                    if (dst1)
                        *reinterpret_cast<uint4 *>(dst1 + cc * 32 + c4 * 8) = v1;
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
        mbar_init(smem_u32(&sh.q_empty), kTiles);
        mbar_init(smem_u32(&sh.next_full), 1);
        for (int i = 0; i < kRing; ++i) {
            mbar_init(smem_u32(&sh.kv_full[i]), 1);
            mbar_init(smem_u32(&sh.kv_empty[i]), kTiles);
        }
        for (int t = 0; t < kTiles; ++t) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(smem_u32(&sh.s_full[t][i]), 1);
                mbar_init(smem_u32(&sh.p_full[t][i]), 4);  // one arrival per softmax warp
            }
            mbar_init(smem_u32(&sh.o_mid[t]), 1);
            mbar_init(smem_u32(&sh.o_full[t]), 1);
            mbar_init(smem_u32(&sh.o_empty[t]), 4);
            mbar_init(smem_u32(&sh.drain[t]), 1);
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
        mma_role<D, kBf16, 0>(p, sh, sbase);
    } else if (warp == kMmaWarp + 1) {
        mma_role<D, kBf16, 1>(p, sh, sbase);
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
