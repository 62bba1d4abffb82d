// Attention of rows to all keys of their sequence (no causal mask) over a paged cache, on the tensor
// cores: tokens or beams to an encoder's states, and a batch's single tokens to a prefix they share.
//
// Tiles, items, key blocks and the two products are those of the causal kernel
// (tpmlp_attn_prompt.cuh): a tile is up to 128 rows (row = token * G + head of the group), an item two
// tiles of one kv head, K and V come in blocks of 128 keys, and the tiles step through them (e4m3: half a
// block at a time): S = Q K^T in tensor memory, P = 2^(S c - m) over S in 16 bits, O += P V. Without a mask
// all rows of an item see the same keys, which is what this kernel is made of:
//  - every item of a sequence has the same number of blocks, so that a CTA finds its share of the work
//    by arithmetic, for any number of items;
//  - values that are not finite need no second way: no row has a weight of 0 for a key that another
//    sees, and the last block's rows behind the keys are cleared.
//
// Warps: 0-3 softmax of tile 0, 4-7 of tile 1, 8 and 10 issue the MMAs of tile 0 and 1, 9 loads K, V and
// Q, 11 makes the work list; e4m3 caches: further ones convert the loaded bytes to fp16.
//
// A step of a whole block (bf16) reads Q once for its scores, and a product of 128 columns takes the tensor
// core 64 cycles where two of 64 take 96. All 128 scores stay in a thread's registers; the weights of the
// first 96 keys are handed over before those of the last 32, whose product with V is the shorter wait. With
// half a block a step: 4 x 1024 rows on 4096 keys x 96 heads of 128 550 us (now 510), 95 x 256 rows on 2048
// keys x 8 heads of 64 126 (now 115); 64 rows there 93 (now 97), and 256 rows on 64 keys 19.7 (now 23). In
// e4m3, whose threads have registers for 64 scores, whole blocks with the first half's scores read once
// more: 2 x 1000 rows on 24000 keys x 32 heads of 128 701 us (half a block a step: 650).
// What bounds it, per block of 128 keys and 256 rows: with heads of 128 in bf16 2900 cycles, of which the
// products take 2050; the rest is the chain of a tile's scores, maximum, weights and products, which the
// other tile's fill in part; items whose keys come from DRAM 1.67 us (5.8 TB/s). With an e4m3 cache 1.9 us:
// shared memory moves 384 KB a block at 128 bytes a cycle. With heads of 64 1.2 us (e4m3 1.45): the chain
// of a tile. Items of one tile's rows: 1.4 (DRAM, 5.9 TB/s), 1.0 us with heads of 64. An item costs about
// 2 us beside its blocks, e4m3 ones 5: Q, the first scores and the result.
// Tried, with steps of 64 keys (1.35 us a block with heads of 64): no search for a step's maximum while its
// weights' sum stays small (1.41 us, the sum's check costs what the search did); softmax warps and
// accumulators of their own for even and odd steps (1.25 us, but 1 us more an item; 66 us for 24 ragged
// sequences of 20 heads of 64, against 56); every second block for an idle second tile (0.83 us, 1 us more
// an item, and 0.03 us more where it is not idle); the next step's scores loaded beside the hand-over
// (registers spill); four pieces ahead in the work list (items are dealt too early: 66 us, against 56 with
// two).
#pragma once

#include "tpmlp_attn_prompt.cuh"

namespace tpmlp {

constexpr int kOpenCode = 0x4000;  // wait sites: kOpenCode | role
constexpr int kOpenRuns = 512;     // entries of the table of sequences
constexpr int kOpenPieces = 2;     // pieces between the work list's warp and the others

struct OpenArgs {
    KvView kv;
    const __nv_bfloat16* q;
    int64_t ldq;
    __nv_bfloat16* out;
    int64_t ldo;
    float* lse;
    const int32_t* cu_q;  // null: one row of each sequence (T = B)
    int32_t T, Hq, G, tpt;  // tpt: tokens per tile
    float scale_log2;
    float* partial;   // [CTAs][2 pieces][2 tiles] slots of kPromptSlotFloats
    uint32_t* count;  // [CTAs][2 tiles] arrivals, then items dealt and CTAs done; 0 between launches
    // where results go instead of out (null: they go to out), for join_parts_kernel: fp32 [T][Hq][D]
    // and what they are [T][Hq]; those of split items stay in their contributors' slots of `partial`
    float* part;
    RowOf* part_of;
    int32_t rows_of_none;  // place of the rows of no sequence in part_of
    int32_t few;  // above 0: as RowArgs', whose kernel has computed all rows if no sequence has more
};

template <int D, bool FP8>
struct OpenShape {
    static constexpr int kConvert = FP8 ? (D == 64 ? 4 : 8) : 0;  // warps that convert
    static constexpr int kThreads = 32 * (12 + kConvert);
    // Registers of a softmax thread and of the others: together at most what the block is launched with
    // (65536 over its threads, a multiple of 8 each: 168, 128, 96).
    static constexpr int kLaunch = 65536 / kThreads / 8 * 8;
    static constexpr int kSoftmaxRegs = FP8 ? (D == 64 ? 168 : 144) : 184;
    static constexpr int kOtherRegs = FP8 ? (D == 64 ? 88 : 64) : 136;
    static_assert(256 * kSoftmaxRegs + (kThreads - 256) * kOtherRegs <= kThreads * kLaunch,
                  "the register split draws on what the block was launched with");

    static constexpr uint32_t kTile = kPB * D * 2;  // a Q, K or V tile of 16-bit values
    static constexpr uint32_t kRaw = FP8 ? kPB * D : 0;
    static constexpr int kStages = D == 128 ? (FP8 ? 3 : 4) : 8;
    static constexpr int kRaws = FP8 ? (D == 128 ? 2 : 4) : 0;
    static constexpr uint32_t kStage0 = 2 * kTile;
    static constexpr uint32_t kRaw0 = kStage0 + kStages * kTile;
    static constexpr uint32_t kBars = kRaw0 + kRaws * kRaw;
    static constexpr int kNumBars = 2 * kStages + 2 * kRaws + 48;
    static constexpr uint32_t kCtl = kBars + 8 * kNumBars;  // TMEM address, abort, s_last [2], groups [8]
    static constexpr uint32_t kPieces0 = kCtl + 64;
    static constexpr uint32_t kUp = kPieces0 + kOpenPieces * 64;  // [2 tiles][128] fp32, e4m3
    static constexpr uint32_t kStore0 = (kUp + (FP8 ? 2 * 128 * 4 : 0) + 127) / 128 * 128;
    static constexpr uint32_t kTables = kStore0 + 8 * 2048;  // 2 KB of output staging per softmax warp
    static constexpr uint32_t kTotal = 1024 + kTables + 2 * kOpenRuns * 4 + 64;
    static_assert(kTotal <= 232448, "dynamic shared memory per CTA");
    static_assert((kStages + kRaws) / 2 + 1 < 8, "blocks in flight, against the ring of loaded groups");
};

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        :
        : "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
          "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// A sequence's rows: [first, first + n) of Q, all of which see its first `len` keys.
struct OpenSeq {
    int first, n, len;
};
__device__ __forceinline__ OpenSeq open_seq(const OpenArgs& a, int b) {
    OpenSeq s;
    s.first = a.cu_q ? max(0, min(a.cu_q[b], a.T)) : b;
    s.n = a.cu_q ? max(0, min(a.cu_q[b + 1], a.T) - s.first) : 1;
    s.len = kv_length(a.kv, b);
    return s;
}

// An item, or the part of its key blocks [b0, b1) that one CTA computes.
struct OpenPiece {
    int valid;
    int h, b;            // kv head, sequence
    int len;             // its keys
    int row0;            // row of Q of tile 0's first token
    int tokens[2];       // of each tile
    int b0, b1;          // blocks
    int first, last;     // contributing CTAs
    int starts;          // 1: the item's first blocks are in this piece
    __device__ __forceinline__ int begin() const { return 2 * b0; }
    __device__ __forceinline__ int end(int t) const {
        return tokens[t] > 0 ? min((len + kSB - 1) / kSB, 2 * b1) : 2 * b0;
    }
};
static_assert(sizeof(OpenPiece) <= 64, "piece slots");

// The CTA's work list. A sequence's items are numbered by kv head and then by tile, so that those that
// share keys are at work together. An item's work is a unit for its start and its blocks. The numbers of
// items and of split lists' units stay below 2^31 (32-bit divisions: a first piece 5000 cycles earlier).
struct OpenWork {
    const uint32_t *items_at, *units_at;  // items and work before each run of `run` sequences
    int runs, run;
    uint32_t items;
    bool split;            // equal runs of work instead of whole items
    bool dealt;            // whole items: this CTA has had its first
    uint32_t at, end, per;  // split: this CTA's run of work, the length of every run

    __device__ __forceinline__ static uint32_t tiles(const OpenArgs& a, const OpenSeq& s) {
        return (static_cast<uint32_t>(s.n) + 2u * a.tpt - 1u) / (2u * a.tpt);
    }
    __device__ __forceinline__ static uint32_t blocks(const OpenSeq& s) {
        return (static_cast<uint32_t>(s.len) + kPB - 1u) / kPB;
    }

    // The sequence of the k-th item (UNITS: unit); k becomes its number within the sequence. For a whole
    // warp.
    template <bool UNITS>
    __device__ __forceinline__ int locate(const OpenArgs& a, uint32_t& k, OpenSeq& s) const {
        const uint32_t* const table = UNITS ? units_at : items_at;
        int lo = 0, hi = runs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (table[mid] <= k) lo = mid;
            else hi = mid;
        }
        k -= table[lo];
        // within the run, 32 sequences at a time
        const int lane = threadIdx.x & 31, upto = min(a.kv.B, (lo + 1) * run);
        for (int b0 = lo * run;; b0 += 32) {
            OpenSeq mine{0, 0, 0};
            if (b0 + lane < upto) mine = open_seq(a, b0 + lane);
            const uint32_t n = tiles(a, mine) * a.kv.Hkv * (UNITS ? 1 + blocks(mine) : 1);
            uint32_t sum = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(~0u, sum, o);
                if (lane >= o) sum += v;
            }
            const uint32_t past = __ballot_sync(~0u, k < sum);
            // (none only if the lengths changed during the launch)
            if (!past && b0 + 32 < upto) {
                k -= __shfl_sync(~0u, sum, 31);
                continue;
            }
            const int at = past ? __ffs(past) - 1 : min(31, upto - 1 - b0);
            k -= __shfl_sync(~0u, sum - n, at);
            s.first = __shfl_sync(~0u, mine.first, at);
            s.n = __shfl_sync(~0u, mine.n, at);
            s.len = __shfl_sync(~0u, mine.len, at);
            return b0 + at;
        }
    }
    __device__ __forceinline__ static void item(const OpenArgs& a, int b, const OpenSeq& s, uint32_t k, OpenPiece& p) {
        const uint32_t nt = max(1u, tiles(a, s)), h = k / nt, j = k - h * nt;
        p.valid = 1;
        p.b = b;
        p.h = static_cast<int>(min(h, static_cast<uint32_t>(a.kv.Hkv - 1)));
        p.len = s.len;
        const int tok0 = static_cast<int>(j) * 2 * a.tpt;
        p.row0 = s.first + tok0;
#pragma unroll
        for (int t = 0; t < 2; ++t) p.tokens[t] = max(0, min(s.n - tok0 - t * a.tpt, a.tpt));
        p.b0 = 0;
        p.b1 = static_cast<int>(blocks(s));
        p.first = p.last = 0;
        p.starts = 1;
    }
    __device__ __forceinline__ OpenPiece next(const OpenArgs& a) {
        OpenPiece p;
        p.valid = 0;
        OpenSeq s;
        if (!split) {
            // the first item goes by the CTA's number, the others are dealt to whichever CTA asks next
            // (who computes an item does not change its result); one lane asks
            uint32_t k = blockIdx.x;
            if (dealt) {
                if ((threadIdx.x & 31) == 0) k = gridDim.x + atomicAdd(a.count + 2 * gridDim.x, 1u);
                k = __shfl_sync(~0u, k, 0);
            }
            dealt = true;
            if (k >= items) return p;
            const int b = locate<false>(a, k, s);
            item(a, b, s, k, p);
            return p;
        }
        while (at < end) {
            uint32_t r = at;
            const int b = locate<true>(a, r, s);
            const uint32_t each = 1 + blocks(s), k = r / each, u0 = at - (r - k * each), u1 = u0 + each;
            item(a, b, s, k, p);
            const int from = max(static_cast<int>(at - u0) - 1, 0);
            at = min(end, u1);
            const int upto = static_cast<int>(at - u0) - 1;
            if (upto == 0 && each > 1) {  // the start alone: its blocks are the next CTA's
                p.valid = 0;
                continue;
            }
            p.first = static_cast<int>((u0 + (each > 1)) / per);
            p.last = static_cast<int>((u1 - 1) / per);
            p.starts = from == 0;
            p.b0 = from;
            p.b1 = upto;
            return p;
        }
        return p;
    }
};

// The logs of a row's sum of weights: of its sum l by the maximum m.
__device__ __forceinline__ float log2_of(float m, float l, bool fp8) {
    return l == 0.0f ? -CUDART_INF_F : m + log2f(l) - (fp8 ? kRaiseLog2 : 0.0f);
}
__device__ __forceinline__ float natural_log(float m, float l, bool fp8) { return log2_of(m, l, fp8) * 0.69314718055994531f; }

// Rows of V past the item's last key or in a page that is not there, in a group of 16 that the product
// reads: their weights are 0, but 0 times what they hold may be NaN; they are cleared first (by both
// tiles' warps alike).
template <int D>
__device__ __noinline__ void clear_rows(uint8_t* block, int in, uint32_t have, int lane) {
    constexpr int kLanes = D / 8;  // to a row, 16 bytes each per 64 columns
    const int upto = min(kPB, (in + 15) & ~15), piece = lane % kLanes;
    for (int r = (have == 0xFFu ? in : 0) + lane / kLanes; r < upto; r += 32 / kLanes)
        if (r >= in || !((have >> (r >> 4)) & 1u))
            *reinterpret_cast<uint4*>(block + (piece >> 3) * 16384 + r * 128 + (piece & 7) * 16) = make_uint4(0, 0, 0, 0);
}

// The result of the first `count` rows of tile t of a split item, from its contributors' slots, first
// to last. The tile's 128 threads call it (row: the thread's number), P to a row of the result, each
// with an equal part of the columns: 16 loads of 16 bytes in flight, however few the rows.
template <int D, bool FP8, int P>
__device__ __forceinline__ void join_open(const OpenArgs& a, const OpenPiece& p, int t, int row, int count,
                                          const float* slots, float v_scale) {
    constexpr int kRows = 128 / P, kCols = D / P;    // a thread's columns
    constexpr int kChunk = kCols < 64 ? kCols : 64;  // of which it sums so many at a time,
    constexpr int kAtOnce = 64 / kChunk;             // of so many contributors
    const int r = row % kRows, part = row / kRows;
    const int from = p.first, upto = p.last;
    if (r >= count) return;
    auto slot_of = [&](int cta) {
        return slots + (static_cast<int64_t>(cta) * 2 + (cta == from)) * 2 * kPromptSlotFloats;
    };
    float mm = -CUDART_INF_F, ll = 0.0f;
    for (int x0 = from; x0 <= upto; x0 += kJoinLoads) {
        float mx[kJoinLoads], lx[kJoinLoads], top = mm;
#pragma unroll
        for (int u = 0; u < kJoinLoads; ++u) {
            const float* src = slot_of(min(x0 + u, upto)) + 128 * 128 + r;
            mx[u] = __ldcg(src);
            lx[u] = x0 + u <= upto ? __ldcg(src + 128) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kJoinLoads; ++u) top = fmaxf(top, mx[u]);
        const float safe = top == -CUDART_INF_F ? 0.0f : top;
        ll *= exp2_approx(mm - safe);
        mm = top;
#pragma unroll
        for (int u = 0; u < kJoinLoads; ++u) ll += exp2_approx(mx[u] - safe) * lx[u];
    }
    const float safe = mm == -CUDART_INF_F ? 0.0f : mm;
    const float scale = ll == 0.0f ? 0.0f : v_scale / ll;
    const int64_t to = p.row0 + t * a.tpt + r / a.G;
    const int64_t to_head = static_cast<int64_t>(p.h) * a.G + r % a.G;
    __nv_bfloat16* const dst = a.out + to * a.ldo + to_head * D;
#pragma unroll 1
    for (int col = part * kCols; col < (part + 1) * kCols; col += kChunk) {
        float v[kChunk];
#pragma unroll
        for (int k = 0; k < kChunk; ++k) v[k] = 0.0f;
#pragma unroll 1
        for (int x0 = from; x0 <= upto; x0 += kAtOnce) {
            float4 y[kAtOnce][kChunk / 4];
            float w[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const float* src = slot_of(min(x0 + u, upto));
#pragma unroll
                for (int k = 0; k < kChunk / 4; ++k)
                    y[u][k] = __ldcg(reinterpret_cast<const float4*>(src + (col + 4 * k) * 128 + r * 4));
                w[u] = __ldcg(src + 128 * 128 + r);
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                // past the last one, sums of 0 as well (see the row kernel)
                const bool on = x0 + u <= upto;
                const float f = on ? exp2_approx(w[u] - safe) : 0.0f;
#pragma unroll
                for (int k = 0; k < kChunk / 4; ++k) {
                    v[4 * k] += f * (on ? y[u][k].x : 0.0f);
                    v[4 * k + 1] += f * (on ? y[u][k].y : 0.0f);
                    v[4 * k + 2] += f * (on ? y[u][k].z : 0.0f);
                    v[4 * k + 3] += f * (on ? y[u][k].w : 0.0f);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kChunk; k += 8) {
            float z[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = ll == 0.0f ? 0.0f : v[k + e] * scale;
            *reinterpret_cast<uint4*>(dst + col + k) = pack8_bf16(z);
        }
    }
    if (a.lse && part == 0) a.lse[to * a.Hq + to_head] = natural_log(mm, ll, FP8);
}

template <int D, bool FP8>
__global__ void __launch_bounds__(OpenShape<D, FP8>::kThreads, 1)
attn_open_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const __grid_constant__ OpenArgs a) {
    using L = OpenShape<D, FP8>;
    constexpr int NST = L::kStages, NRAW = L::kRaws, W0 = 8;
    constexpr bool kBlockStep = !FP8;              // a softmax step is a whole block
    constexpr int kKeys = kBlockStep ? kPB : kSB;  // of a softmax step
    constexpr int kFirst = kBlockStep ? 96 : kSB;  // of a block's first product with V
    constexpr uint32_t kIdescS = prompt_idesc(kKeys, FP8, false);
    constexpr uint32_t kIdescO = prompt_idesc(D, FP8, true);
    constexpr uint32_t kHalf = 16384;  // bytes of 64 columns x 128 rows

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* const base_ptr = smem_raw + (base - raw);
    const uint32_t bars = base + L::kBars;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (NST + s); };
    auto raw_full = [&](int s) { return bars + 8u * (2 * NST + s); };
    auto raw_empty = [&](int s) { return bars + 8u * (2 * NST + NRAW + s); };
    const uint32_t more = bars + 8u * (2 * NST + 2 * NRAW);
    auto q_full = [&](int t) { return more + 8u * t; };
    const uint32_t q_empty = more + 16u;
    const uint32_t drain = more + 24u;
    auto join_in = [&](int t) { return more + 32u + 8u * t; };
    auto join_out = [&](int t) { return more + 48u + 8u * t; };
    auto s_full = [&](int t, int buf) { return more + 80u + 16u * t + 8u * buf; };
    auto p_full = [&](int t, int buf) { return more + 112u + 16u * t + 8u * buf; };
    auto o_full = [&](int t) { return more + 144u + 8u * t; };
    auto o_empty = [&](int t) { return more + 160u + 8u * t; };
    auto pv_done = [&](int t) { return more + 176u + 8u * t; };
    auto piece_full = [&](int s) { return more + 240u + 8u * s; };
    auto piece_empty = [&](int s) { return more + 272u + 8u * s; };
    static_assert(304 <= 48 * 8, "barriers");
    uint32_t* const ctl = reinterpret_cast<uint32_t*>(base_ptr + L::kCtl);
    volatile uint32_t* const abort_flag = ctl + 1;
    uint32_t* const s_last = ctl + 2;           // [2]
    volatile uint32_t* const groups = ctl + 4;  // [8] loaded groups of 16 keys of the last 8 blocks
    auto piece_of = [&](uint32_t k) {
        return reinterpret_cast<const OpenPiece*>(base_ptr + L::kPieces0 + (k % kOpenPieces) * 64);
    };
    uint32_t* const items_at = reinterpret_cast<uint32_t*>(base_ptr + L::kTables);
    uint32_t* const units_at = items_at + kOpenRuns;
    uint32_t* const found = units_at + kOpenRuns;  // items, units (at most 2^31), longest item

    const int warp = __shfl_sync(~0u, static_cast<int>(threadIdx.x) >> 5, 0);
    const int lane = threadIdx.x & 31;

    if (a.few > 0) {
        // The row kernel, the launch before, let this one start when everything before itself was done:
        // cu_q can be read (from L2). Where there is nothing left to do, only the order of launches is kept:
        // what comes next may start beside the row kernel, and is done after it.
        bool many = false;
        for (int b = threadIdx.x; b < a.kv.B; b += L::kThreads) many |= is_many(row_span<true>(a.cu_q, a.T, b), a.G, a.few);
        if (!__syncthreads_or(many)) {
            ptx::griddep_launch_dependents();
            return ptx::griddep_wait();
        }
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            ptx::mbar_init(full(s), FP8 ? L::kConvert : 1);
            ptx::mbar_init(empty(s), 2);
        }
        for (int s = 0; s < NRAW; ++s) {
            ptx::mbar_init(raw_full(s), 1);
            ptx::mbar_init(raw_empty(s), L::kConvert);
        }
        for (int t = 0; t < 2; ++t) {
            ptx::mbar_init(q_full(t), FP8 ? 4 : 1);
            for (int buf = 0; buf < 2; ++buf) {
                ptx::mbar_init(s_full(t, buf), 1);
                ptx::mbar_init(p_full(t, buf), 4);
            }
            ptx::mbar_init(o_full(t), 1);
            ptx::mbar_init(o_empty(t), 4);
            ptx::mbar_init(pv_done(t), 1);
            ptx::mbar_init(join_in(t), 4);
            ptx::mbar_init(join_out(t), 1);
        }
        for (int s = 0; s < kOpenPieces; ++s) {
            ptx::mbar_init(piece_full(s), 1);
            ptx::mbar_init(piece_empty(s), W0 + 3 + L::kConvert);
        }
        ptx::mbar_init(q_empty, 2);
        ptx::mbar_init(drain, 2);
        *abort_flag = 0u;
        ptx::fence_barrier_init();
    }
    if (!FP8 && warp == W0 + 1 && lane == 0) {
        ptx::prefetch_tensormap(&tmQ);
        ptx::prefetch_tensormap(&tmK);
        ptx::prefetch_tensormap(&tmV);
    }
    if (warp == W0) {
        ptx::tmem_alloc(ptx::smem_addr(ctl), 512);
        ptx::tmem_relinquish();
    }
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    // (rows of no sequence have no keys; the kernel that joins their results has to know)
    if (a.part && a.cu_q) clear_rows_of_none(a.part_of, a.cu_q, a.kv.B, a.T, a.Hq, a.rows_of_none);

    // ---------------------------------------------------------------- the work list
    OpenWork work;
    work.items_at = items_at;
    work.units_at = units_at;
    work.run = (a.kv.B + kOpenRuns - 1) / kOpenRuns;
    work.runs = (a.kv.B + work.run - 1) / work.run;
    if (threadIdx.x == 0) found[2] = 0;
    __syncthreads();
    constexpr uint32_t kMost = 1u << 31;
    for (int e = threadIdx.x; e < work.runs; e += L::kThreads) {
        uint64_t items = 0, units = 0;
        uint32_t most = 0;
        for (int b = e * work.run; b < min(a.kv.B, (e + 1) * work.run); ++b) {
            const OpenSeq s = open_seq(a, b);
            const uint64_t n = static_cast<uint64_t>(OpenWork::tiles(a, s)) * a.kv.Hkv;
            const uint32_t each = 1 + OpenWork::blocks(s);
            items += n;
            units += n * each;
            if (n) most = max(most, each);
        }
        items_at[e] = static_cast<uint32_t>(min(items, static_cast<uint64_t>(kMost)));
        units_at[e] = static_cast<uint32_t>(min(units, static_cast<uint64_t>(kMost)));
        if (most) atomicMax(found + 2, most);
    }
    __syncthreads();
    if (warp < 2) {
        // running sums, a table to a warp
        uint32_t* const table = warp ? units_at : items_at;
        const int each = (work.runs + 31) / 32;
        uint64_t sum = 0;
        for (int i = 0; i < each; ++i)
            if (lane * each + i < work.runs) sum += table[lane * each + i];
        uint64_t before = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t v = __shfl_up_sync(~0u, before, o);
            if (lane >= o) before += v;
        }
        if (lane == 31) found[warp] = static_cast<uint32_t>(min(before, static_cast<uint64_t>(kMost)));
        before -= sum;
        for (int i = 0; i < each; ++i)
            if (lane * each + i < work.runs) {
                const uint32_t n = table[lane * each + i];
                table[lane * each + i] = static_cast<uint32_t>(min(before, static_cast<uint64_t>(kMost)));
                before += n;
            }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    work.items = found[0];
    work.split = work.dealt = false;
    work.at = work.end = 0;
    work.per = 1;
    {
        // Work is split evenly where the longest item, or about half of it in the last round, would keep
        // the GPU waiting for more than a tenth over what the split's partial sums and joins cost:
        // kJoinFew blocks of time where there is no more than an item for a CTA, kJoinMany where there
        // are more (every CTA then has two pieces to hand over, and what was dealt would have filled
        // the gaps).
        constexpr uint32_t kJoinFew = 8, kJoinMany = 16;
        const uint32_t total = found[1], g = gridDim.x, most = found[2];
        const uint32_t share = max((total + g - 1) / g, 1u);
        const uint32_t whole = work.items <= g ? most : share + most / 2;
        const uint32_t join = work.items <= g ? kJoinFew : kJoinMany;
        if (total < kMost && 10ull * whole > 11ull * (share + join)) {
            work.split = true;
            work.per = share;
            work.at = min(share * blockIdx.x, total);
            work.end = min(work.at + share, total);
        }
    }
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(ctl);
    auto tmem_s = [&](int t, int buf) { return tmem + 256u + 128u * t + kSB * buf; };
    auto tmem_o = [&](int t) { return tmem + static_cast<uint32_t>(D * t); };
    // (polls for a while before the bounded wait, which reads the global timer)
    auto wait = [&](uint32_t bar, uint32_t parity, int role, uint64_t limit_ns = ptx::kWaitLimitNs) {
        bool done = false;
        for (int n = 0; n < 64 && !done; ++n) done = ptx::mbar_try_wait(bar, parity);
        return __all_sync(~0u, done || ptx::mbar_wait(bar, parity, abort_flag, a.kv.status, kOpenCode | role, limit_ns));
    };

    if (warp < W0) regs_up<L::kSoftmaxRegs>();
    else regs_down<L::kOtherRegs>();

    // The pieces, in the order that every role goes through them. next_piece() waits for one (null:
    // no more, or a wait gave up); release_piece() hands its slot back.
    uint32_t piece_at = 0;
    auto next_piece = [&]() -> const OpenPiece* {
        if (!wait(piece_full(piece_at % kOpenPieces), (piece_at / kOpenPieces) & 1u, 15, kPieceWaitNs)) return nullptr;
        const OpenPiece* p = piece_of(piece_at);
        return p->valid ? p : nullptr;
    };
    auto release_piece = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(piece_empty(piece_at % kOpenPieces));
        ++piece_at;
    };

    if (warp < W0) {
        // ------------------------------------------------------------ softmax of one tile
        const int t = warp >> 2;
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        uint32_t s_phase = 0, o_phase = 0, q_empty_phase = 0, j_phase = 0, blocks = 0;
        uint32_t pv_count = 0;  // products P V of this tile so far
        const int token = row / a.G, head = row - token * a.G;
        while (const OpenPiece* p = next_piece()) {
            const int tokens = p->tokens[t];
            const bool mine = token < tokens;
            // the row and head of Q that this thread has
            auto qrow = [&] { return static_cast<int64_t>(p->row0) + t * a.tpt + token; };
            auto qhead = [&] { return static_cast<int64_t>(p->h) * a.G + head; };
            const int len = p->len, b0 = p->b0, b1 = p->b1;
            const int begin = p->begin(), end = p->end(t);
            float c = a.scale_log2;
            if constexpr (FP8) {
                if (b1 > b0) {
                    if (tokens > 0) {
                        // Q in fp16, scaled (query_exponent). A row's D / 8 lanes load 16 bytes each,
                        // neighbours side by side, all in flight together (a thread to a row, 16 bytes of
                        // 32 rows to a load: 7 us for 256 rows of 128). The factor that the row was
                        // divided by goes to the thread that has the row.
                        constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kLoads = 32 / kAtOnce;
                        float* const up = reinterpret_cast<float*>(base_ptr + L::kUp) + t * 128;
                        const __nv_bfloat16* mine_at = mine ? a.q + qrow() * a.ldq + qhead() * D : nullptr;
                        if (!wait(q_empty, q_empty_phase ^ 1u, 1, kPieceWaitNs)) break;
                        uint4 v[kLoads];
#pragma unroll
                        for (int x = 0; x < kLoads; ++x) {
                            const int r = x * kAtOnce + lane / kLanes;
                            const auto at = __shfl_sync(~0u, reinterpret_cast<unsigned long long>(mine_at), r);
                            v[x] = make_uint4(0, 0, 0, 0);
                            if (at) v[x] = load16(reinterpret_cast<const uint8_t*>(at) + 16 * (lane % kLanes));
                        }
#pragma unroll
                        for (int x = 0; x < kLoads; ++x) {
                            const int r = x * kAtOnce + lane / kLanes, piece = lane % kLanes;
                            float f[8], big = 0.0f;
                            unpack8(v[x], f);
#pragma unroll
                            for (int k = 0; k < 8; ++k) big = fmaxf(big, fabsf(f[k]));
#pragma unroll
                            for (int o = 1; o < kLanes; o <<= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, o));
                            const int e = query_exponent(big), in_tile = (warp & 3) * 32 + r;
                            const float down = power_of_two(-e);
                            uint8_t* const dst = base_ptr + t * L::kTile + in_tile * 128;
                            *reinterpret_cast<uint4*>(dst + (piece >> 3) * kHalf + (((piece & 7) ^ (in_tile & 7)) << 4)) =
                                make_uint4(pack_half2(f[0] * down, f[1] * down), pack_half2(f[2] * down, f[3] * down),
                                           pack_half2(f[4] * down, f[5] * down), pack_half2(f[6] * down, f[7] * down));
                            if (piece == 0) up[in_tile] = power_of_two(e);
                        }
                        fence_async_shared();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(q_full(t));
                        c = c * a.kv.scales[p->h] * up[row];
                        if (c == 0.0f) c = FLT_MIN;  // 0 times a masked score of -infinity would be NaN
                    }
                    q_empty_phase ^= 1u;
                }
            }
            float m = -CUDART_INF_F, l = 0.0f;  // reference (log2 units), sum
            const uint32_t block0 = blocks - b0;
            blocks += b1 - b0;
            bool ok = true;
            for (int j = begin; j < end; j += kKeys / kSB) {
                const int buf = kBlockStep ? 0 : j & 1;
                // (a tile that had no rows in the piece before is here while the other goes through that one)
                if (!(ok = wait(s_full(t, buf), (s_phase >> buf) & 1u, 2, j == begin ? kPieceWaitNs : ptx::kWaitLimitNs))) break;
                s_phase ^= 1u << buf;
                constexpr uint32_t kHave = (1u << (kKeys / 16)) - 1u;
                const uint32_t have = (groups[(block0 + (j >> 1)) & 7] >> (4 * buf)) & kHave;
                ptx::tc_fence_after();
                const uint32_t ts = tmem_s(t, buf) + lanes;
                uint32_t s[kKeys];
#pragma unroll
                for (int x0 = 0; x0 < kKeys; x0 += 64) {
#pragma unroll
                    for (int x = x0; x < x0 + 64; x += 32) ptx::tmem_ld_32x32b_x32(ts + x, *reinterpret_cast<uint32_t(*)[32]>(s + x));
#pragma unroll
                    for (int x = x0; x < x0 + 64; x += 32) ptx::tmem_wait_ld(*reinterpret_cast<uint32_t(*)[32]>(s + x));
                }
                const int below = len - j * kSB;
                if (below < kKeys || have != kHave) {
#pragma unroll
                    for (int x = 0; x < kKeys; x += 16) {
                        const int n = (have >> (x >> 4)) & 1u ? below - x : 0;
                        if (n < 16) {
#pragma unroll
                            for (int k = 0; k < 16; ++k) s[x + k] = k < n ? s[x + k] : 0xFF800000u;
                        }
                    }
                }
                float top[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    top[x] = __uint_as_float(s[x]);
#pragma unroll
                    for (int k = 4; k < kKeys - 4; k += 8)
                        top[x] = max3(top[x], __uint_as_float(s[k + x]), __uint_as_float(s[k + 4 + x]));
                    top[x] = fmaxf(top[x], __uint_as_float(s[kKeys - 4 + x]));
                }
                const float now = fmaxf(max3(top[0], top[1], top[2]), top[3]) * c;
                const bool move = now > m + kLazyLog2;
                if (__any_sync(~0u, move)) {
                    const float f = move ? exp2_approx(m - now) : 1.0f;
                    if (move) m = now;
                    l *= f;
                    // O of the steps before is scaled, once the last of their products is done (with whole
                    // blocks it was before these scores)
                    if (j > begin) {
                        if (!kBlockStep && !(ok = wait(pv_done(t), (pv_count - 1) & 1u, 17))) break;
                        ptx::tc_fence_after();
                        constexpr int kAtOnce = kBlockStep ? 16 : 32;
#pragma unroll 1
                        for (int x = 0; x < D; x += kAtOnce) {
                            uint32_t o[kAtOnce];
                            if constexpr (kBlockStep) {
                                ptx::tmem_ld_32x32b_x16_wait(tmem_o(t) + lanes + x, o);
                            } else {
                                ptx::tmem_ld_32x32b_x32(tmem_o(t) + lanes + x, o);
                                ptx::tmem_wait_ld(o);
                            }
#pragma unroll
                            for (int k = 0; k < kAtOnce; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            if constexpr (kBlockStep) tmem_st_x16(tmem_o(t) + lanes + x, o);
                            else tmem_st_x32(tmem_o(t) + lanes + x, o);
                        }
                    }
                }
                ++pv_count;
                // P = 2^(S c - m), two values to an instruction where there is one; rounded to 16 bits for
                // the product with V, of V's type (both operands of these instructions have one type):
                // half a step of a weight is 2^-8 of it in bf16, 2^-11 in fp16; its sum is taken before
                const float shift = (FP8 ? kRaiseLog2 : 0.0f) - (m == -CUDART_INF_F ? 0.0f : m);
                const float2 c2 = make_float2(c, c), shift2 = make_float2(shift, shift);
                float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                for (int part = 0; part < (kBlockStep ? 2 : 1); ++part) {
                    if (part > 0 && below <= kFirst) break;
                    const int from = part * kFirst, upto = part ? kKeys : kFirst;
                    uint32_t w[kFirst / 2];
#pragma unroll
                    for (int k = 0; k < kFirst / 2; ++k) {
                        if (k >= (upto - from) / 2) break;
                        const uint32_t* const x = s + from + 2 * k;
                        float2 e = fma2(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), c2, shift2);
                        e.x = exp2_approx(e.x);
                        e.y = exp2_approx(e.y);
                        sum[k & 1] = add2(sum[k & 1], e);
                        w[k] = FP8 ? pack_half2(e.x, e.y) : pack_bf162(e.x, e.y);
                    }
                    if (part == 0) tmem_st_x32(ts, w);
                    if (kBlockStep) tmem_st_x16(ts + (part ? 48 : 32), w + (part ? 0 : 32));
                    tmem_wait_st();
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full(t, buf + part));
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            }
            if (!ok) break;
            // -------------------------------------------------------- the tile's result
            if (tokens == 0) {
                release_piece();
                continue;
            }
            const bool whole = p->first == p->last, any = end > begin;
            float* const slots = a.partial + static_cast<int64_t>(t) * kPromptSlotFloats;
            float* const slot = slots + (static_cast<int64_t>(blockIdx.x) * 2 + p->starts) * 2 * kPromptSlotFloats;
            const float v_scale = FP8 ? a.kv.scales[a.kv.Hkv + p->h] : 1.0f;
            const float inv = l == 0.0f ? 0.0f : v_scale / l;  // no keys: zeros
            const int64_t at = qrow() * a.Hq + qhead();
            __nv_bfloat16* const dst = mine ? a.out + qrow() * a.ldo + qhead() * D : nullptr;
            if (any) {
                if (!wait(o_full(t), o_phase, 3)) break;
                o_phase ^= 1u;
                ptx::tc_fence_after();
            }
            uint8_t* const stage = base_ptr + L::kStore0 + warp * 2048;
            __nv_bfloat16* rows_to[4];  // rows 8k + lane / 4, from their lanes
#pragma unroll
            for (int k = 0; k < 4; ++k)
                rows_to[k] = reinterpret_cast<__nv_bfloat16*>(
                    __shfl_sync(~0u, reinterpret_cast<unsigned long long>(dst), 8 * k + (lane >> 2)));
#pragma unroll 1
            for (int col = 0; col < D; col += 32) {
                __syncwarp();
                uint32_t o[32];
                if (any) {
                    ptx::tmem_ld_32x32b_x32(tmem_o(t) + lanes + col, o);
                    ptx::tmem_wait_ld(o);
                    if (col + 32 == D) {
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(o_empty(t));
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0u;
                }
                if (!whole) {
                    if (mine) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            __stcg(reinterpret_cast<float4*>(slot + (col + k) * 128 + row * 4),
                                   make_float4(__uint_as_float(o[k]), __uint_as_float(o[k + 1]),
                                               __uint_as_float(o[k + 2]), __uint_as_float(o[k + 3])));
                    }
                    continue;
                }
                float v[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] = l == 0.0f ? 0.0f : __uint_as_float(o[k]) * inv;
                if (a.part) {
                    if (mine) {
                        float* const part = a.part + at * D + col;
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *reinterpret_cast<float4*>(part + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                    }
                    continue;
                }
                // through shared memory, so that four lanes write 64 contiguous bytes of a row (a line of
                // a store takes the SM a cycle, however few of its bytes are written)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = v[8 * k + e];
                    *reinterpret_cast<uint4*>(stage + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) = pack8_bf16(x);
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = 8 * k + (lane >> 2), x = lane & 3;
                    const uint4 y = *reinterpret_cast<const uint4*>(stage + r * 64 + ((x ^ ((r >> 1) & 3)) << 4));
                    if (rows_to[k]) *reinterpret_cast<uint4*>(rows_to[k] + col + 8 * x) = y;
                }
            }
            if (whole) {
                if (a.part && mine) a.part_of[at] = RowOf{log2_of(m, l, FP8), 0, 0, -1};
                else if (a.lse && mine) a.lse[at] = natural_log(m, l, FP8);
            } else if (a.part) {
                // (a join by the last contributor alone took 20 us of 10 contributors' sums of 256 rows)
                if (mine) {
                    __stcg(slot + 128 * 128 + row, m);
                    __stcg(slot + 128 * 128 + 128 + row, l);
                    if (p->starts) a.part_of[at] = RowOf{0.0f, p->first, p->last, t * 128 + row};
                }
            } else {
                // The last contributor to arrive sums all of them, first to last (see the row kernel);
                // each tile's 128 threads count and join on their own.
                if (mine) {
                    __stcg(slot + 128 * 128 + row, m);
                    __stcg(slot + 128 * 128 + 128 + row, l);
                }
                __threadfence();
                __syncwarp();
                if (lane == 0) mbar_arrive(join_in(t));
                if (warp == 4 * t) {
                    if (!wait(join_in(t), j_phase, 13)) break;
                    if (lane == 0) {
                        __threadfence();
                        const uint32_t n = atomicAdd(a.count + 2 * p->first + t, 1u);
                        s_last[t] = n == static_cast<uint32_t>(p->last - p->first);
                        if (s_last[t]) a.count[2 * p->first + t] = 0;
                        __threadfence();
                        mbar_arrive(join_out(t));
                    }
                    __syncwarp();
                }
                if (!wait(join_out(t), j_phase, 14)) break;
                j_phase ^= 1u;
                if (*reinterpret_cast<volatile uint32_t*>(s_last + t)) {
                    __threadfence();
                    const int count = tokens * a.G;
                    if (count > 64) join_open<D, FP8, 1>(a, *p, t, row, count, slots, v_scale);
                    else if (count > 32) join_open<D, FP8, 2>(a, *p, t, row, count, slots, v_scale);
                    else if (count > 16) join_open<D, FP8, 4>(a, *p, t, row, count, slots, v_scale);
                    else join_open<D, FP8, 8>(a, *p, t, row, count, slots, v_scale);
                }
            }
            release_piece();
        }
    } else if (warp == W0 || warp == W0 + 2) {
        // ------------------------------------------------------------ MMAs of one tile
        const int t = (warp - W0) >> 1;
        const uint64_t dq = sdesc_k128(base + t * L::kTile);
        uint32_t stage = 0, phase = 0, q_phase = 0, p_phase = 0, o_phase = 0, blocks = 0;
        bool ok = true;
        while (ok) {
            const OpenPiece* p = next_piece();
            if (!p) break;
            const int b0 = p->b0, b1 = p->b1, begin = p->begin(), end = p->end(t), len = p->len;
            if (b1 > b0) {
                // (a tile without rows waits for the other's: its word that Q is free must not come
                // before that of the piece before is complete)
                const int x = p->tokens[t] > 0 ? t : 0;
                if (!(ok = wait(q_full(x), (q_phase >> x) & 1u, 4))) break;
                q_phase ^= p->tokens[1] > 0 ? 3u : 1u;
                ptx::tc_fence_after();
            }
            // Round i: O += P V for both parts of block i - 1, and S of block i, which may overwrite those P
            // once their products have been issued: after the second (whole blocks), or half by half.
            for (int i = b0; i <= b1; ++i) {
                const uint32_t vs = stage, vph = phase;
                uint32_t ks = vs, kph = vph;
                if (i > b0 && ++ks == NST) {
                    ks = 0;
                    kph ^= 1u;
                }
                const uint32_t sv = L::kStage0 + vs * L::kTile;
                const uint64_t dv = sdesc_v(base + sv), dk = sdesc_k128(base + L::kStage0 + ks * L::kTile);
                if (i > b0) {
                    if (!(ok = wait(full(vs), vph, 5))) break;
                    const uint32_t have = groups[(blocks + i - 1 - b0) & 7];
                    if (len < i * kPB || have != 0xFFu) {
                        clear_rows<D>(base_ptr + sv, len - (i - 1) * kPB, have, lane);
                        fence_async_shared();
                        __syncwarp();
                    }
                }
                if (i < b1) {
                    if (!(ok = wait(full(ks), kph, 8))) break;
                    ptx::tc_fence_after();
                }
#pragma unroll
                for (int par = 0; par < 2; ++par) {
                    const int jk = 2 * i + par;
                    const uint32_t ts = tmem_s(t, par), to = tmem_o(t);
                    // groups of 16 keys [k0, k1) of the block
                    const int in16 = (len - (i - 1) * kPB + 15) / 16;
                    const int k0 = par ? kFirst / 16 : 0, k1 = min(par ? kPB / 16 : kFirst / 16, in16);
                    if (i > b0 && begin < end && k1 > k0) {
                        const bool fresh = par == 0 && i == b0 + 1;
                        if (fresh) {  // the tile's result before this one has been read
                            if (!(ok = wait(o_empty(t), o_phase ^ 1u, 6))) break;
                            o_phase ^= 1u;
                        }
                        if (!(ok = wait(p_full(t, par), (p_phase >> par) & 1u, 7))) break;
                        p_phase ^= 1u << par;
                        ptx::tc_fence_after();
                        if (elect_one()) {
                            const uint32_t p0 = kBlockStep ? tmem_s(t, 0) : ts - 8 * k0;
                            if (k1 == (par ? kPB / 16 : kFirst / 16)) {
#pragma unroll
                                for (int k = 0; k < (par ? kPB - kFirst : kFirst) / 16; ++k)
                                    mma_ts(to, p0 + 8 * (k0 + k), dv + 128 * (k0 + k), kIdescO, k == 0 ? !fresh : 1u);
                            } else {
                                for (int k = k0; k < k1; ++k) mma_ts(to, p0 + 8 * k, dv + 128 * k, kIdescO, k == k0 ? !fresh : 1u);
                            }
                            if (!kBlockStep) ptx::mma_commit(pv_done(t));
                            if (i == b1 && (par == 1 || in16 <= kFirst / 16)) ptx::mma_commit(o_full(t));
                        }
                        __syncwarp();
                    }
                    if (i < b1 && (kBlockStep ? par == 1 && jk - 1 < end : jk < end)) {
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < D / 16; ++k) {
                                const uint32_t off = (k >> 2) * (kHalf >> 4) + 2 * (k & 3);
                                ptx::mma_bf16_ss(kBlockStep ? tmem_s(t, 0) : ts, dq + off, dk + (kBlockStep ? 0 : 512 * par) + off,
                                                 kIdescS, k ? 1u : 0u);
                            }
                            ptx::mma_commit(s_full(t, kBlockStep ? 0 : par));
                        }
                        __syncwarp();
                    }
                }
                if (!ok) break;
                if (elect_one()) {
                    if (i > b0) ptx::mma_commit(empty(vs));
                    if (i < b1) ptx::mma_commit(empty(ks));
                    if (i + 1 == b1) ptx::mma_commit(q_empty);  // the last use of Q
                }
                __syncwarp();
                stage = ks;
                phase = kph;
                if (i < b1 && ++stage == NST) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
            blocks += b1 - b0;
            release_piece();
        }
        __syncwarp();
        if (elect_one()) {
            // every product has completed before tensor memory is released
            ptx::mma_commit(drain);
            ptx::mbar_wait_drain(drain, 0);
        }
        __syncwarp();
    } else if (warp == W0 + 1) {
        // ------------------------------------------------------------ TMA producer
        const int rows = min(1 << a.kv.page_shift, kPB);  // of a copy
        const int copies = kPB / rows;
        uint32_t stage = 0, phase = 0, issued = 0, q_phase = 0, q_loads[2] = {0, 0}, blocks = 0;
        constexpr int NR = FP8 ? NRAW : NST;
        bool ok = true;
        while (ok) {
            const OpenPiece* p = next_piece();
            if (!p) break;
            const int b0 = p->b0, b1 = p->b1, h = p->h, b = p->b, len = p->len;
            // whether this lane copies a part of block i (not past the last key)
            auto wanted = [&](int i) { return lane < copies && i < b1 && i * kPB + lane * rows < len; };
            // the table's entry for this lane's copy of a block, looked up a block ahead
            auto entry = [&](int i) { return wanted(i) ? kv_entry(a.kv, b, i * kPB + lane * rows) : 0; };
            int next = entry(b0);
            for (int i = b0; ok && i < b1; ++i) {
                const int key = i * kPB + lane * rows;
                const bool in = wanted(i);
                const int found_page = next;
                next = entry(i + 1);
                const int64_t page = in ? kv_checked(a.kv, found_page) : -1;
                const uint32_t there = __ballot_sync(~0u, page >= 0);
                // groups of 16 keys that are there; those outside the item's keys count as such
                uint32_t have = 0xFFu;
                const uint32_t missing = __ballot_sync(~0u, in && page < 0);
                if (missing) {
                    for (int x = 0; x < copies; ++x)
                        if ((missing >> x) & 1u) have &= ~(((1u << (rows / 16)) - 1u) << (x * (rows / 16)));
                }
                const int slot = key & ((1 << a.kv.page_shift) - 1);
                for (int kv = 0; kv < 2; ++kv) {
                    const uint32_t bar_full = FP8 ? raw_full(stage) : full(stage);
                    if (!(ok = wait(FP8 ? raw_empty(stage) : empty(stage), phase ^ 1u, 10))) break;
#ifdef TPMLP_TEST_SKIP_STAGE
                    // a stage that is never filled: the waits for it run out
                    const bool fill = issued != TPMLP_TEST_SKIP_STAGE;
#else
                    constexpr bool fill = true;
#endif
                    if (lane == 0 && fill) {
                        if (kv == 0) groups[(blocks + i - b0) & 7] = have;
                        ptx::mbar_arrive_expect_tx(bar_full, static_cast<uint32_t>(__popc(there) * rows) * D * (FP8 ? 1 : 2));
                    }
                    __syncwarp();
                    if (page >= 0 && fill) {
                        if constexpr (FP8) {
                            bulk_load(base + L::kRaw0 + stage * L::kRaw + lane * rows * D,
                                      (kv ? a.kv.V : a.kv.K) + page * a.kv.page_bytes + h * a.kv.head_bytes +
                                          static_cast<int64_t>(slot) * D,
                                      static_cast<uint32_t>(rows) * D, bar_full);
                        } else {
                            const uint32_t dst = base + L::kStage0 + stage * L::kTile + lane * rows * 128;
#pragma unroll
                            for (int x = 0; x < D / 64; ++x)
                                ptx::tma_load_3d(dst + x * kHalf, kv ? &tmV : &tmK, bar_full, 64 * x,
                                                 (h << a.kv.page_shift) + slot, static_cast<int>(page));
                        }
                    }
                    __syncwarp();
                    ++issued;
                    if (++stage == NR) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (!FP8 && i == b0 && kv == 0) {
                        // Q after the first keys, which need not wait for the piece before
                        if (!(ok = wait(q_empty, q_phase ^ 1u, 9, kPieceWaitNs))) break;
                        q_phase ^= 1u;
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (p->tokens[t] == 0) continue;
                            if (lane == 0) {
                                ptx::mbar_arrive_expect_tx(q_full(t), static_cast<uint32_t>(a.tpt * a.G) * D * 2);
                                for (int x = 0; x < D / 64; ++x)
                                    ptx::tma_load_3d(base + t * L::kTile + x * kHalf, &tmQ, q_full(t), 64 * x, h * a.G,
                                                     p->row0 + t * a.tpt);
                            }
                            ++q_loads[t];
                        }
                        __syncwarp();
                    }
                }
            }
            if (!ok) break;
            blocks += b1 - b0;
            release_piece();
        }
        if ((!ok || *abort_flag) && lane == 0) {
            // wait for the copies still in flight before the CTA may exit (also when another role
            // gave up, and no piece came after the last one)
            for (uint32_t s = 0; s < NR && s < issued; ++s) {
                const uint32_t last = s + ((issued - 1 - s) / NR) * NR;
                ptx::mbar_wait_drain(FP8 ? raw_full(s) : full(s), (last / NR) & 1u);
            }
            for (int t = 0; t < 2; ++t)
                if (q_loads[t]) ptx::mbar_wait_drain(q_full(t), (q_loads[t] - 1) & 1u);
        }
        __syncwarp();
    } else if (warp == W0 + 3) {
        // ------------------------------------------------------------ work list
        for (;; ++piece_at) {
            if (!wait(piece_empty(piece_at % kOpenPieces), ((piece_at / kOpenPieces) & 1u) ^ 1u, 16, kPieceWaitNs)) break;
            const OpenPiece p = work.next(a);
            if (lane == 0) {
                if (p.valid) *const_cast<OpenPiece*>(piece_of(piece_at)) = p;
                else const_cast<OpenPiece*>(piece_of(piece_at))->valid = 0;
                mbar_arrive(piece_full(piece_at % kOpenPieces));
            }
            __syncwarp();
            if (!p.valid) break;
        }
        if (!work.split && lane == 0) {
            // the last CTA to have asked in vain leaves the counters at 0 for the next launch
            uint32_t* const done = a.count + 2 * gridDim.x + 1;
            if (atomicAdd(done, 1u) == gridDim.x - 1) {
                done[-1] = 0;
                done[0] = 0;
            }
        }
    } else if (FP8) {
        // ------------------------------------------------------------ e4m3 -> fp16
        uint32_t rs = 0, rph = 0, stage = 0, phase = 0;
        bool ok = true;
        const int tid = (warp - W0 - 4) * 32 + lane;
        while (ok) {
            const OpenPiece* p = next_piece();
            if (!p) break;
            const int n = 2 * (p->b1 - p->b0);
            release_piece();
            for (int x0 = 0; x0 < n; ++x0) {
                if (!(ok = wait(raw_full(rs), rph, 11))) break;
                if (!(ok = wait(empty(stage), phase ^ 1u, 12))) break;
                const uint8_t* src = base_ptr + L::kRaw0 + rs * L::kRaw;
                uint8_t* dst = base_ptr + L::kStage0 + stage * L::kTile;
                constexpr int kAll = 32 * (FP8 ? L::kConvert : 1);
                constexpr int kParts = kPB * D / 16 / kAll;  // 16-byte parts per thread
                uint4 v[kParts];
#pragma unroll
                for (int x = 0; x < kParts; ++x) v[x] = *reinterpret_cast<const uint4*>(src + (x * kAll + tid) * 16);
#pragma unroll
                for (int x = 0; x < kParts; ++x) {
                    const int part = x * kAll + tid;
                    const int r = part / (D / 16), j = part % (D / 16);
                    uint4 lo, hi;
                    e4m3x4_to_half2(v[x].x, lo.x, lo.y);
                    e4m3x4_to_half2(v[x].y, lo.z, lo.w);
                    e4m3x4_to_half2(v[x].z, hi.x, hi.y);
                    e4m3x4_to_half2(v[x].w, hi.z, hi.w);
                    // the two 16-byte chunks in an order that spreads a row's writes over all banks
                    uint8_t* const d = dst + (j >> 2) * kHalf + r * 128;
                    const int c0 = 2 * (j & 3), swap = (j >> 2) & 1;
                    *reinterpret_cast<uint4*>(d + (((c0 + swap) ^ (r & 7)) << 4)) = swap ? hi : lo;
                    *reinterpret_cast<uint4*>(d + (((c0 + 1 - swap) ^ (r & 7)) << 4)) = swap ? lo : hi;
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(full(stage));
                    mbar_arrive(raw_empty(rs));
                }
                if (++rs == NRAW) {
                    rs = 0;
                    rph ^= 1u;
                }
                if (++stage == NST) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    }

    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == W0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ two parts of a row's keys
// A row's results over two parts of its keys (or one), with one softmax over both.
struct JoinPartsArgs {
    struct Side {
        const float* part;  // as OpenArgs' part, part_of (null: there is no such part) and partial
        const RowOf* of;
        const float* slots;
    } side[2];
    __nv_bfloat16* out;
    int64_t ldo;
    float* lse;
    int64_t heads;  // rows * Hq
    int32_t Hq, G;
    int32_t ctas;          // of the kernel that made split rows' sums
    const float* v_scale;  // e4m3: [Hkv]
};
constexpr int kJoinThreads = 128;
constexpr int kPartLoads = 4;  // contributors whose sums a thread loads at once

// D / 4 lanes to each of kSlices slices of a head's contributors, four columns each; the slices' sums meet
// in shared memory. Bound by latency: where the results lie, then the contributors' maxima, sums and
// columns, kPartLoads contributors of a slice at a time. 4 slices against 1, the whole decode_shared: 64
// sequences x 8 heads of one kv head, 59 contributors 35, 48 us; 192 x 12 heads of 64, 13 contributors 65, 72;
// 128 x 32 on 8 kv heads, 10 contributors 204, 206; 96 x 96 on 8 kv heads, 3 contributors 94, 88.
template <int D, bool FP8, int kSlices>
__global__ void __launch_bounds__(kJoinThreads) join_parts_kernel(const __grid_constant__ JoinPartsArgs a) {
    constexpr int kLanes = D / 4, kHeads = kJoinThreads / (kLanes * kSlices);  // of a block
    __shared__ float4 s_o[2][kHeads][kSlices][kLanes];
    __shared__ float2 s_ml[2][kHeads][kSlices];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int lane = threadIdx.x % kLanes, slice = threadIdx.x / kLanes % kSlices, mine = threadIdx.x / (kLanes * kSlices);
    const int64_t at = static_cast<int64_t>(blockIdx.x) * kHeads + mine;
    const bool on = at < a.heads;
    const int d = lane * 4;
    const int64_t row = at / a.Hq;
    const int head = static_cast<int>(at - row * a.Hq);
    float log[2];
    float4 o[2];
    uint4 where[2];
    bool split[2];
#pragma unroll
    for (int x = 0; x < 2; ++x)
        where[x] = on && a.side[x].of ? load16(reinterpret_cast<const uint8_t*>(a.side[x].of + at)) : make_uint4(0xFF800000u, 0, 0, ~0u);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        // (held to the slots there are: a launch that gave up may have left another call's)
        const uint32_t most = a.ctas - 1;
        const int first = static_cast<int>(min(where[x].y, most)), last = static_cast<int>(min(where[x].z, most));
        const int place = min(static_cast<int>(where[x].w), 255);
        o[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        log[x] = __uint_as_float(where[x].x);
        split[x] = place >= 0;
        if (!split[x]) {
            if (slice == 0 && log[x] != -CUDART_INF_F) o[x] = __ldcg(reinterpret_cast<const float4*>(a.side[x].part + at * D + d));
            continue;
        }
        // a split row: every kSlices-th of its contributors (one pass with a running maximum)
        const int r = place & 127;
        const float* const slots = a.side[x].slots + static_cast<int64_t>(place >> 7) * kPromptSlotFloats;
        float m = -CUDART_INF_F, l = 0.0f;
        for (int c0 = first + slice; c0 <= last; c0 += kPartLoads * kSlices) {
            float mx[kPartLoads], lx[kPartLoads], top = m;
            float4 v[kPartLoads];
#pragma unroll
            for (int u = 0; u < kPartLoads; ++u) {
                const int c = c0 + u * kSlices;
                const bool in = c <= last;
                const float* p = slots + (static_cast<int64_t>(c) * 2 + (c == first)) * 2 * kPromptSlotFloats;
                mx[u] = in ? __ldcg(p + 128 * 128 + r) : -CUDART_INF_F;
                lx[u] = in ? __ldcg(p + 128 * 128 + 128 + r) : 0.0f;
                v[u] = in ? __ldcg(reinterpret_cast<const float4*>(p + d * 128 + r * 4)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
            for (int u = 0; u < kPartLoads; ++u) top = fmaxf(top, mx[u]);
            const float safe = top == -CUDART_INF_F ? 0.0f : top;
            const float f = exp2_approx(m - safe);
            m = top;
            l *= f;
            o[x] = make_float4(o[x].x * f, o[x].y * f, o[x].z * f, o[x].w * f);
#pragma unroll
            for (int u = 0; u < kPartLoads; ++u) {
                const float w = exp2_approx(mx[u] - safe);
                l += w * lx[u];
                o[x].x += w * v[u].x;
                o[x].y += w * v[u].y;
                o[x].z += w * v[u].z;
                o[x].w += w * v[u].w;
            }
        }
        s_o[x][mine][slice][lane] = o[x];
        if (lane == 0) s_ml[x][mine][slice] = make_float2(m, l);
    }
    __syncthreads();
    if (!on || slice > 0 || static_cast<int>(where[0].w) == -2) return;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        if (!split[x]) continue;
        float m = -CUDART_INF_F, l = 0.0f;
#pragma unroll
        for (int k = 0; k < kSlices; ++k) m = fmaxf(m, s_ml[x][mine][k].x);
        const float safe = m == -CUDART_INF_F ? 0.0f : m;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kSlices; ++k) {
            // (a slice without contributors has sums of 0)
            const float2 ml = s_ml[x][mine][k];
            const float4 v = s_o[x][mine][k][lane];
            const float w = exp2_approx(ml.x - safe);
            l += w * ml.y;
            sum = make_float4(sum.x + w * v.x, sum.y + w * v.y, sum.z + w * v.z, sum.w + w * v.w);
        }
        const float by = l == 0.0f ? 0.0f : (FP8 ? a.v_scale[head / a.G] : 1.0f) / l;
        o[x] = make_float4(sum.x * by, sum.y * by, sum.z * by, sum.w * by);
        log[x] = log2_of(m, l, FP8);
    }
    const float top = fmaxf(log[0], log[1]), safe = top == -CUDART_INF_F ? 0.0f : top;
    float w[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) w[x] = exp2f(log[x] - safe);
    const float sum = w[0] + w[1], inv = sum == 0.0f ? 0.0f : 1.0f / sum;  // no keys at all: zeros
    // (a part without keys has no say: 0 times its result would do but for what is not finite)
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        if (log[x] == -CUDART_INF_F) continue;
        const float f = w[x] * inv;
        y = make_float4(y.x + o[x].x * f, y.y + o[x].y * f, y.z + o[x].z * f, y.w + o[x].w * f);
    }
    *reinterpret_cast<uint2*>(a.out + row * a.ldo + static_cast<int64_t>(head) * D + d) =
        make_uint2(pack_bf162(y.x, y.y), pack_bf162(y.z, y.w));
    if (a.lse && d == 0) a.lse[at] = sum == 0.0f ? -CUDART_INF_F : (top + log2f(sum)) * 0.69314718055994531f;
}

}  // namespace tpmlp
