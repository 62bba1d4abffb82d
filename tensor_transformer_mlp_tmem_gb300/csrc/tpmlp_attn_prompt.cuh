// Causal attention of chunks of new tokens over a paged cache, on the tensor cores.
//
// For one kv head, G query heads and TPT = floor(128 / G) consecutive tokens make a tile of up to
// 128 rows (row = token * G + head of the group), so that grouped heads share each K and V tile.
// A CTA works on an item of two tiles (2 TPT tokens of one kv head). K and V come in blocks of
// 128 keys; the tiles step through them 64 keys at a time:
//   S_t = Q_t K^T      tcgen05.mma, both operands in shared memory, S fp32 in tensor memory
//   P_t = 2^(S c - m)  one thread per row, written back over S in 16 bits
//   O_t += P_t V       tcgen05.mma, P from tensor memory, V from shared memory (keys are the
//                      reduction, so V is read as it lies, D contiguous)
// While the softmax warps of one tile work, the tensor core runs the other tile's two products.
//
// Warps: 0-3 softmax of tile 0, 4-7 of tile 1 (a warp may read the 32 tensor-memory lanes of its
// rank mod 4), 8 and 10 issue the MMAs of tile 0 and 1, 9 loads K and V (and Q) by TMA, page by
// page, 11 makes the work list; e4m3 caches: 12-19 convert the loaded bytes to fp16. One warp
// per tile issues MMAs because each waits for several barriers a step: with one warp for both
// tiles the tensor core idled during those waits.
//
// What bounds it (GPT-3-shaped prompt, 4096 tokens x 96 heads of 128: 305-324 us, 1.3 PFLOP/s,
// about two thirds of the measured bf16 rate, at the board's power limit): two bounds lie close
// together. A softmax step takes a warp about 1300 cycles, so 128 keys of both tiles take 2600.
// That is a chain of latencies (load of S, maximum, weights, store, one after the other) more than
// of issue slots: two such warps share a scheduler, which issues 0.4 instructions a cycle over a
// launch. And their products take 2048 cycles of the tensor core, which S's 64 columns stretch (Q
// is read again for every 64 keys, and shared memory feeds the tensor core at 128 bytes a cycle).
// Leaving out all exponentials, half of Q K^T or half of P V changed the time by 3 to 4 % each.
// Steps of 64 keys with two buffers of S per tile let a softmax follow the one before it at once;
// with steps of 128 and one buffer (S, P and both O fill tensor memory) every softmax waited for
// the two products before it: 416 against 486 us. Two groups of softmax warps to a tile, for even
// and odd steps or for halves of a block, gained nothing (361 against 340; 439).
#pragma once

#include <cfloat>

#include "tpmlp_attn.cuh"
#include "tpmlp_gemm.cuh"

namespace tpmlp {

constexpr int kPB = 128;          // keys per block (a stage) = rows per tile
constexpr int kSB = 64;           // keys per step: S has two buffers of 64 columns per tile
constexpr int kPromptItems = 1024;  // items whose sizes a CTA tabulates
constexpr int kCoarse = 512;        // entries of the table of sequences
constexpr int kPromptCode = 0x2000;  // wait sites: kPromptCode | role
// Limit of the waits that last as long as another role's piece (2^24 blocks of keys at 2 us each, at
// most). The roles that such a wait is for have the usual limit for every step of theirs, and end
// this one at once when they give up.
constexpr uint64_t kPieceWaitNs = 60ull * 1000 * 1000 * 1000;
// fp32 values of a tile's partial sums: O in groups of 4 columns [D/4][128][4], m [128], l [128].
constexpr int kPromptSlotFloats = 128 * 128 + 256;
// A row's reference maximum follows its running maximum only when that has grown by more than
// 2^8: weights then stay below 2^8 (no loss in fp32, bf16 or fp16) and O is rarely rescaled.
constexpr float kLazyLog2 = 8.0f;
constexpr float kRaiseLog2 = 6.0f;  // e4m3 caches: fp16 weights are raised by 2^6 (see the rows)

struct PromptArgs {
    KvView kv;
    const __nv_bfloat16* q;
    int64_t ldq;
    __nv_bfloat16* out;
    int64_t ldo;
    float* lse;
    const int32_t* cu_q;  // null: one token of each sequence (T = B)
    int32_t T, Hq, G, tpt;  // tpt: tokens per tile
    float scale_log2;
    int32_t window;
    float* partial;   // [CTAs][2 pieces][2 tiles] slots
    uint32_t* count;  // [CTAs][2 tiles] arrivals, then items dealt and CTAs done; 0 between launches
};

template <int D, bool FP8>
struct PromptSmem {
    static constexpr uint32_t kTile = kPB * D * 2;   // a Q, K or V tile of 16-bit values
    static constexpr uint32_t kRaw = FP8 ? kPB * D : 0;
    static constexpr int kStages = D == 128 ? (FP8 ? 3 : 4) : 6;
    static constexpr int kRaws = FP8 ? (D == 128 ? 2 : 3) : 0;
    static constexpr uint32_t kStage0 = 2 * kTile;
    static constexpr uint32_t kRaw0 = kStage0 + kStages * kTile;
    static constexpr uint32_t kBars = kRaw0 + kRaws * kRaw;
    static constexpr int kNumBars = 2 * kStages + 2 * kRaws + 32;
    static constexpr uint32_t kStore0 = kBars + (8 * kNumBars + 64 + 2 * 96 + 127) / 128 * 128;
    static constexpr uint32_t kTables = kStore0 + 8 * 2048;  // 2 KB of output staging per softmax warp
    static constexpr uint32_t kTotal = 1024 + kTables + (kCoarse + 1) * 8 + (kPromptItems + 1) * 4 + 256;
    static_assert(kTotal <= 232448, "dynamic shared memory per CTA");
    static constexpr int kThreads = FP8 ? 640 : 384;
};

// D[tmem] (+)= A[tmem] * B[smem]: the 16-bit A operand lies in tensor memory, two values to a
// column.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
          "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
          "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
          "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
          "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_async_shared() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
        : "memory");
}
// One lane of the (converged) warp, the same one every time: the MMAs of a warp are issued and
// committed by one thread.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}
template <int R>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// Packed fp32 pairs and the three-operand maximum.
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return d;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(x), "f"(y), "f"(z));
    return d;
}

// B operand with the reduction (keys) along rows: blocks of 64 columns of D, each 128 keys x 128
// bytes with the 128-byte swizzle; 16 KB from block to block, 1 KB from 8 keys to 8 keys.
__device__ __forceinline__ uint64_t sdesc_v(uint32_t saddr) {
    return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(16384 >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}

// Instruction descriptor: fp32 accumulators, bf16 or fp16 operands, A K-major, B K- or N-major.
__host__ __device__ constexpr uint32_t prompt_idesc(int N, bool half, bool b_mn) {
    return (1u << 4) | (half ? 0u : (1u << 7) | (1u << 10)) | (b_mn ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

// A sequence's new tokens: rows [first, first + n) of Q, at positions len - n ...
struct PromptSeq {
    int first, n, len;
    __device__ __forceinline__ int hi(int token) const {  // keys that the token may see end here
        return max(0, min(len, len - n + token + 1));
    }
};
__device__ __forceinline__ PromptSeq prompt_seq(const PromptArgs& a, int b) {
    PromptSeq s;
    s.first = a.cu_q ? max(0, min(a.cu_q[b], a.T)) : b;
    s.n = a.cu_q ? max(0, min(a.cu_q[b + 1], a.T) - s.first) : 1;
    s.len = kv_length(a.kv, b);
    return s;
}

// An item, or the part of its key blocks [b0, b1) that one CTA computes.
struct Piece {
    int valid;
    int h, tok0;           // kv head, first token of tile 0
    int b;                 // sequence
    PromptSeq seq;
    int tokens[2];         // of each tile
    int lo[2], hi[2];      // each tile's steps
    int last_hi[2];        // end of the keys of each tile's last token
    int lo_key;            // first key that any of the item's tokens sees
    int b0, b1;            // blocks
    int first, last;       // contributing CTAs
    int starts;            // 1: the item's first blocks are in this piece
    int redo;              // tiles (bits) found to need the careful way, 0 at first
    int careful;           // 0, or the tiles whose results are made again, the careful way
    __device__ __forceinline__ int begin(int t) const { return max(lo[t], 2 * b0); }
    __device__ __forceinline__ int end(int t) const { return min(hi[t], 2 * b1); }
};
static_assert(sizeof(Piece) <= 96, "piece slots");
constexpr int kPieces = 2;  // pieces between the work list's warp and the others: one ahead

__device__ __forceinline__ int prompt_lo_key(const PromptArgs& a, int hi) {
    return a.window > 0 ? max(0, hi - a.window) : 0;
}

// The steps and blocks of tokens [tok0, tok0 + 2 tpt) of a sequence.
__device__ __forceinline__ void item_blocks(const PromptArgs& a, Piece& p) {
    p.b0 = 0x7FFFFFFF;
    p.b1 = 0;
    p.lo_key = prompt_lo_key(a, p.seq.hi(p.tok0));
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int k0 = p.tok0 + t * a.tpt;
        p.tokens[t] = max(0, min(p.seq.n - k0, a.tpt));
        p.lo[t] = p.hi[t] = p.last_hi[t] = 0;
        if (p.tokens[t] > 0) {
            p.last_hi[t] = p.seq.hi(k0 + p.tokens[t] - 1);
            p.hi[t] = (p.last_hi[t] + kSB - 1) / kSB;
            p.lo[t] = min(p.hi[t], prompt_lo_key(a, p.seq.hi(k0)) / kSB);
        }
        if (p.hi[t] > p.lo[t]) {
            p.b0 = min(p.b0, p.lo[t] / 2);
            p.b1 = max(p.b1, (p.hi[t] + 1) / 2);
        }
    }
    if (p.b1 == 0) p.b0 = 0;
    p.redo = p.careful = 0;
}

// The CTA's work list. Items are numbered sequence by sequence; within a sequence in groups of
// kv heads, so that the heads in flight keep their K and V in L2, and within a group from the last
// tokens (most keys) to the first. A group has two items or more for each CTA: with one, a last
// group's largest items were started when little else was left (GPT-3-shaped prompt: 326 us, so 302,
// both in one session; 305-324 over all).
struct PromptWork {
    const int64_t* coarse;  // items before each run of `run` sequences
    const int* units;       // work before each item (split lists)
    int runs, run;          // entries of coarse, sequences per entry
    int64_t items;
    bool split;             // equal runs of work instead of whole items
    int64_t at, end, per;   // split: this CTA's run of work, the length of every run

    __device__ __forceinline__ static int tiles(const PromptArgs& a, const PromptSeq& s) {
        return (s.n + 2 * a.tpt - 1) / (2 * a.tpt);
    }
    __device__ __forceinline__ void item(const PromptArgs& a, int64_t k, Piece& p) const {
        int lo = 0, hi = runs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (coarse[mid] <= k) lo = mid;
            else hi = mid;
        }
        int64_t r = k - coarse[lo];
        int b = lo * run;
        PromptSeq s = prompt_seq(a, b);
        int nt = tiles(a, s);
        while (r >= static_cast<int64_t>(nt) * a.kv.Hkv && b + 1 < a.kv.B) {
            r -= static_cast<int64_t>(nt) * a.kv.Hkv;
            s = prompt_seq(a, ++b);
            nt = tiles(a, s);
        }
        nt = max(nt, 1);
        const int groups = max(1, static_cast<int>(min(static_cast<int64_t>(nt) * a.kv.Hkv / (2 * gridDim.x),
                                                       static_cast<int64_t>(a.kv.Hkv))));
        const int group = (a.kv.Hkv + groups - 1) / groups;
        const int64_t per_group = static_cast<int64_t>(nt) * group;
        const int h0 = static_cast<int>(r / per_group) * group;
        const int j = static_cast<int>(r % per_group);
        const int heads = max(1, min(group, a.kv.Hkv - h0));
        p.b = b;
        p.seq = s;
        p.h = min(h0 + j % heads, a.kv.Hkv - 1);
        p.tok0 = (nt - 1 - j / heads) * 2 * a.tpt;
        item_blocks(a, p);
    }
    __device__ __forceinline__ Piece next(const PromptArgs& a) {
        Piece p;
        p.valid = 0;
        if (!split) {
            // items are dealt to whichever CTA asks next (who computes an item does not change
            // its result); one lane asks
            uint32_t k = 0;
            if ((threadIdx.x & 31) == 0) k = atomicAdd(a.count + 2 * gridDim.x, 1u);
            k = __shfl_sync(~0u, k, 0);
            if (k >= items) return p;
            item(a, k, p);
            p.valid = 1;
            p.first = p.last = 0;
            p.starts = 1;
            return p;
        }
        while (at < end) {
            int lo = 0, hi = static_cast<int>(items);
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (units[mid] <= at) lo = mid;
                else hi = mid;
            }
            // an item's units: one for its start, then its blocks
            const int u0 = units[lo], u1 = units[lo + 1];
            const int from = max(static_cast<int>(at) - u0 - 1, 0);
            at = min(end, static_cast<int64_t>(u1));
            const int upto = static_cast<int>(at) - u0 - 1;
            if (upto == 0 && u1 > u0 + 1) continue;  // the start alone: its blocks are the next CTA's
            item(a, lo, p);
            p.valid = 1;
            p.first = (u0 + (u1 > u0 + 1)) / static_cast<int>(per);
            p.last = (u1 - 1) / static_cast<int>(per);
            p.starts = from == 0;
            const int base = p.b0;
            p.b0 = base + from;
            p.b1 = base + upto;
            return p;
        }
        return p;
    }
};

// A value (V) that is not finite, at a key that some of an item's tokens see and others do not: the
// product P V carries it to the others too (its weight is 0 there, and 0 times it is NaN). An item is
// therefore computed as if there were none; a tile whose sums are not finite though its weights' are is
// computed once more, the careful way: the MMA warps clear such values of such keys in the loaded
// tile, and add_cleared adds them to the rows that see them (a weight above 0 times them is what
// they are). Without such values that costs next to nothing (before and after, us: GPT-3-shaped
// prompt 321, 321; ragged batch 94.4, 94.2; e4m3 chunks 657, 657; 61 tokens 7.7, 7.9-8.0).
// Keys [lo, hi) that all of the item's tokens see.
struct SeenByAll {
    int lo, hi;
    __device__ __forceinline__ SeenByAll(const PromptArgs& a, const Piece& p)
        : lo(prompt_lo_key(a, max(p.last_hi[0], p.last_hi[1]))), hi(p.seq.hi(p.tok0)) {}
    __device__ __forceinline__ bool operator()(int key) const { return key >= lo && key < hi; }
};
template <bool FP8>
__device__ __forceinline__ void clear_not_finite(uint4& v) {
    constexpr uint32_t kExponent = FP8 ? 0x7C00u : 0x7F80u;  // fp16, bf16
    uint32_t w[4] = {v.x, v.y, v.z, v.w}, found = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t lo = (w[e] & kExponent) == kExponent ? 0xFFFFu : 0u;
        const uint32_t hi = ((w[e] >> 16) & kExponent) == kExponent ? 0xFFFF0000u : 0u;
        w[e] &= ~(lo | hi);
        found |= lo | hi;
    }
    if (found) v = make_uint4(w[0], w[1], w[2], w[3]);
}
// Rows of V that no query of the item may see, in a group of 16 that the product reads: past the
// item's last key, before its first (a window's), or in a page that is not there. Their weights are
// 0, but 0 times what they hold may be NaN; they are cleared first (by both tiles' warps alike). The
// careful way, so are values that are not finite, of keys that some tokens do not see.
template <int D, bool FP8>
__device__ __forceinline__ void clear_values(const PromptArgs& a, const Piece& p, uint8_t* block, int key0,
                                             uint32_t have, int lane) {
    constexpr int kLanes = D / 8;  // to a row, 16 bytes each per 64 columns
    const int in = max(p.last_hi[0], p.last_hi[1]) - key0, low = p.lo_key - key0;
    const bool careful = p.careful != 0;
    const SeenByAll all(a, p);
    const int upto = min(kPB, (in + 15) & ~15), piece = lane % kLanes;
    for (int r = (have == 0xFFu && low <= 0 && !careful ? in : 0) + lane / kLanes; r < upto; r += 32 / kLanes) {
        uint4& v = *reinterpret_cast<uint4*>(block + (piece >> 3) * 16384 + r * 128 + (piece & 7) * 16);
        if (r >= in || r < low || !((have >> (r >> 4)) & 1u)) v = make_uint4(0, 0, 0, 0);
        else if (careful && !all(key0 + r)) clear_not_finite<FP8>(v);
    }
}
// (out of line for e4m3 caches, whose MMA warps have few registers)
template <int D>
__device__ __noinline__ void clear_values_e4m3(const PromptArgs& a, const Piece& p, uint8_t* block, int key0,
                                               uint32_t have, int lane) {
    clear_values<D, true>(a, p, block, key0, have, lane);
}
// The warp's 32 rows of O, at `to` in tensor memory; the lane's row sees keys [lo, hi).
template <int D, bool FP8>
__device__ __noinline__ void add_cleared(const PromptArgs& a, const Piece& p, int lo, int hi, uint32_t to) {
    const int from = max(lo, p.b0 * kPB), upto = min(hi, p.b1 * kPB);
    const SeenByAll all(a, p);
#pragma unroll 1
    for (int x = 0; x < D; x += 32) {
        uint32_t o[32];
        ptx::tmem_ld_32x32b_x32(to + x, o);
        ptx::tmem_wait_ld(o);
#pragma unroll 1
        for (int key = from; key < upto; ++key) {
            if (all(key)) key = all.hi;
            if (key >= upto) break;
            const int page = kv_page(a.kv, p.b, key);
            if (page < 0) continue;
            const int64_t slot = key & ((1 << a.kv.page_shift) - 1);
            const uint8_t* src = a.kv.V + page * a.kv.page_bytes + p.h * a.kv.head_bytes + (slot * D + x) * (FP8 ? 1 : 2);
#pragma unroll
            for (int k = 0; k < (FP8 ? 2 : 4); ++k) {
                const uint4 v = load16(src + 16 * k);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (FP8) {
#pragma unroll
                        for (int b = 0; b < 4; ++b)  // e4m3 has NaN and no infinity
                            if (((w[e] >> (8 * b)) & 0x7Fu) == 0x7Fu) o[16 * k + 4 * e + b] = 0x7FFFFFFFu;
                    } else {
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const uint32_t f = b ? w[e] & 0xFFFF0000u : w[e] << 16;
                            if ((f & 0x7F800000u) == 0x7F800000u) {
                                uint32_t& y = o[8 * k + 2 * e + b];
                                y = __float_as_uint(__uint_as_float(y) + __uint_as_float(f));
                            }
                        }
                    }
                }
            }
        }
        __syncwarp();
        tmem_st_x32(to + x, o);
    }
    tmem_wait_st();
}

// The result of the first `count` rows of tile t of a split item, from its contributors' slots, first
// to last. The tile's 128 threads call it (row: the thread's number), P to a row of the result, each
// with an equal part of the columns: 16 loads of 16 bytes in flight, however few the rows. One token of
// 16 heads over 131072 keys, 51 contributors: 56 us (with one thread to a row: 113).
template <int D, bool FP8, int P>
__device__ __forceinline__ void join_rows(const PromptArgs& a, const Piece& p, int t, int row, int count,
                                          const float* slots, float v_scale) {
    constexpr int kRows = 128 / P, kCols = D / P;       // a thread's columns
    constexpr int kChunk = kCols < 64 ? kCols : 64;     // of which it sums so many at a time,
    constexpr int kAtOnce = 64 / kChunk;                // of so many contributors
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
    const int64_t to = p.seq.first + p.tok0 + t * a.tpt + r / a.G;
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
    if (a.lse && part == 0)
        a.lse[to * a.Hq + to_head] =
            ll == 0.0f ? -CUDART_INF_F : (mm + log2f(ll) - (FP8 ? kRaiseLog2 : 0.0f)) * 0.69314718055994531f;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(PromptSmem<D, FP8>::kThreads, 1)
attn_prompt_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PromptArgs a) {
    using L = PromptSmem<D, FP8>;
    constexpr int NST = L::kStages, NRAW = L::kRaws;
    constexpr uint32_t kIdescS = prompt_idesc(kSB, FP8, false);
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
    auto o_full = [&](int t) { return more + 32u + 8u * t; };
    auto o_empty = [&](int t) { return more + 48u + 8u * t; };
    auto join_in = [&](int t) { return more + 64u + 8u * t; };
    auto join_out = [&](int t) { return more + 80u + 8u * t; };
    auto s_full = [&](int t, int buf) { return more + 96u + 16u * t + 8u * buf; };
    auto p_full = [&](int t, int buf) { return more + 128u + 16u * t + 8u * buf; };
    auto piece_full = [&](int s) { return more + 160u + 8u * s; };
    auto piece_empty = [&](int s) { return more + 192u + 8u * s; };
    auto pv_done = [&](int t) { return more + 224u + 8u * t; };
    auto checked = [&](int s) { return more + 240u + 8u * s; };  // both tiles' sums of a piece
    uint32_t* const ctl = reinterpret_cast<uint32_t*>(base_ptr + L::kBars + 8 * L::kNumBars);
    volatile uint32_t* const abort_flag = ctl + 1;
    uint32_t* const s_last = ctl + 2;      // [2]
    volatile uint32_t* const groups = ctl + 4;  // [8] loaded groups of 16 keys of the last 8 blocks
    const Piece* const pieces = reinterpret_cast<const Piece*>(base_ptr + L::kBars + 8 * L::kNumBars + 64);
    int64_t* const coarse = reinterpret_cast<int64_t*>(base_ptr + L::kTables);
    int* const units = reinterpret_cast<int*>(coarse + kCoarse + 1);
    int64_t* const found = reinterpret_cast<int64_t*>(base_ptr + L::kTables + (kCoarse + 1) * 8 +
                                                      ((kPromptItems + 2) * 4 + 7) / 8 * 8);

    const int warp = __shfl_sync(~0u, static_cast<int>(threadIdx.x) >> 5, 0);
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            ptx::mbar_init(full(s), FP8 ? 8 : 1);
            ptx::mbar_init(empty(s), 2);
        }
        for (int s = 0; s < NRAW; ++s) {
            ptx::mbar_init(raw_full(s), 1);
            ptx::mbar_init(raw_empty(s), 8);
        }
        for (int t = 0; t < 2; ++t) {
            ptx::mbar_init(q_full(t), FP8 ? 4 : 1);
            for (int buf = 0; buf < 2; ++buf) {
                ptx::mbar_init(s_full(t, buf), 1);
                ptx::mbar_init(p_full(t, buf), 4);
            }
            ptx::mbar_init(o_full(t), 1);
            ptx::mbar_init(pv_done(t), 1);
            ptx::mbar_init(o_empty(t), 4);
            ptx::mbar_init(join_in(t), 4);
            ptx::mbar_init(join_out(t), 1);
        }
        for (int s = 0; s < kPieces; ++s) {
            ptx::mbar_init(piece_full(s), 1);
            ptx::mbar_init(piece_empty(s), FP8 ? 19 : 11);
            ptx::mbar_init(checked(s), 8);
        }
        ptx::mbar_init(q_empty, 2);
        ptx::mbar_init(drain, 2);
        *abort_flag = 0u;
        ptx::fence_barrier_init();
    }
    if (!FP8 && warp == 9 && lane == 0) {
        ptx::prefetch_tensormap(&tmQ);
        ptx::prefetch_tensormap(&tmK);
        ptx::prefetch_tensormap(&tmV);
    }
    if (warp == 8) {
        ptx::tmem_alloc(ptx::smem_addr(ctl), 512);
        ptx::tmem_relinquish();
    }
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    // ---------------------------------------------------------------- the work list
    PromptWork work;
    work.coarse = coarse;
    work.units = units;
    work.run = (a.kv.B + kCoarse - 1) / kCoarse;
    work.runs = (a.kv.B + work.run - 1) / work.run;
    for (int e = threadIdx.x; e < work.runs; e += L::kThreads) {
        int64_t n = 0;
        for (int b = e * work.run; b < min(a.kv.B, (e + 1) * work.run); ++b)
            n += static_cast<int64_t>(PromptWork::tiles(a, prompt_seq(a, b))) * a.kv.Hkv;
        coarse[e] = n;
    }
    __syncthreads();
    if (warp == 0) {
        const int each = (work.runs + 31) / 32;
        int64_t sum = 0;
        for (int i = 0; i < each; ++i)
            if (lane * each + i < work.runs) sum += coarse[lane * each + i];
        int64_t before = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(~0u, before, o);
            if (lane >= o) before += v;
        }
        if (lane == 31) found[0] = before;
        before -= sum;
        for (int i = 0; i < each; ++i)
            if (lane * each + i < work.runs) {
                const int64_t n = coarse[lane * each + i];
                coarse[lane * each + i] = before;
                before += n;
            }
    }
    __syncthreads();
    work.items = found[0];
    work.split = false;
    work.at = work.end = 0;
    work.per = 1;
    if (work.items <= kPromptItems) {
        // Few items: tabulate their work (a block of time each for an item's start and its
        // result, and its blocks), and split it evenly where the longest item, or about half of
        // it in the last round, would keep the GPU waiting for more than a tenth over what the
        // split's partial sums and joins cost: kJoinFew blocks of time where there is no more
        // than an item for a CTA, kJoinMany where there are more (every CTA then has two pieces
        // to hand over, and what was dealt would have filled the gaps). Whole items against a
        // split, us: 4096 tokens of 32 heads 105, 123; 2048 of 32 heads with 8 kv heads 44, 50; 256
        // of them on 8192 keys 99, 48; two chunks of 1000 on 24000 e4m3 keys 786, 655; of no more
        // items than CTAs, 8 times 4 tokens on 4000 keys 45, 37; 2048 tokens of 12 heads of 64 30,
        // 26; 3 times 700 on 3000 e4m3 keys 60, 67.
        constexpr int kJoinFew = 8, kJoinMany = 16;
        const int n = static_cast<int>(work.items);
        for (int i = threadIdx.x; i < n; i += L::kThreads) {
            Piece p;
            work.item(a, i, p);
            units[i] = 1 + p.b1 - p.b0;
        }
        __syncthreads();
        if (warp == 0) {
            const int each = (n + 31) / 32;
            int sum = 0, most = 0;
            for (int i = 0; i < each; ++i)
                if (lane * each + i < n) {
                    sum += units[lane * each + i];
                    most = max(most, units[lane * each + i]);
                }
            // in 64 bits: 1024 items of 2^24 blocks (a lane's 32 items stay below 2^31)
            int64_t before = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(~0u, before, o);
                if (lane >= o) before += v;
                most = max(most, __shfl_xor_sync(~0u, most, o));
            }
            if (lane == 31) found[0] = before;
            if (lane == 0) found[1] = most;
            before -= sum;
            for (int i = 0; i < each; ++i)
                if (lane * each + i < n) {
                    const int u = units[lane * each + i];
                    units[lane * each + i] = static_cast<int>(before);
                    before += u;
                }
        }
        __syncthreads();
        const int64_t all = found[0];
        const int total = static_cast<int>(min(all, static_cast<int64_t>(INT_MAX)));
        const int most = static_cast<int>(found[1]);
        if (threadIdx.x == 0) units[n] = total;
        const int g = static_cast<int>(gridDim.x);
        const int share = max((total + g - 1) / g, 1);
        const int whole = n <= g ? most : share + most / 2;
        const int join = n <= g ? kJoinFew : kJoinMany;
        if (all == total && 10 * whole > 11 * (share + join)) {
            work.split = true;
            work.per = share;
            work.at = static_cast<int64_t>(share) * blockIdx.x;
            work.end = min(work.at + share, static_cast<int64_t>(total));
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(ctl);
    auto tmem_s = [&](int t) { return tmem + 256u + 128u * t; };
    auto tmem_o = [&](int t) { return tmem + 128u * t; };
    // The bounded wait reads the global timer, which takes longer than most waits here last: poll
    // for a while first.
    auto wait = [&](uint32_t bar, uint32_t parity, int role, uint64_t limit_ns = ptx::kWaitLimitNs) {
        bool done = false;
        for (int n = 0; n < 64 && !done; ++n) done = ptx::mbar_try_wait(bar, parity);
        return __all_sync(~0u, done || ptx::mbar_wait(bar, parity, abort_flag, a.kv.status, kPromptCode | role, limit_ns));
    };

    // The register split sums to what the block was launched with (384 x 168, 640 x 96).
    if (warp < 8) regs_up<FP8 ? 144 : 184>();
    else regs_down<FP8 ? 64 : 136>();

    // The pieces, in the order that every role goes through them. next_piece() waits for one (null:
    // no more, or a wait gave up); release_piece() hands its slot back.
    uint32_t piece_at = 0;
    auto piece_of = [&](uint32_t k) {
        return reinterpret_cast<const Piece*>(reinterpret_cast<const uint8_t*>(pieces) + (k % kPieces) * 96);
    };
    auto next_piece = [&]() -> const Piece* {
        if (!wait(piece_full(piece_at % kPieces), (piece_at / kPieces) & 1u, 15, kPieceWaitNs)) return nullptr;
        const Piece* p = piece_of(piece_at);
        return p->valid ? p : nullptr;
    };
    auto release_piece = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(piece_empty(piece_at % kPieces));
        ++piece_at;
    };

    if (warp < 8) {
        // ------------------------------------------------------------ softmax of one tile
        const int t = warp >> 2;
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        uint32_t s_phase = 0, o_phase = 0, q_phase = 0, j_phase = 0, blocks = 0;
        uint32_t pv_count = 0;  // products P V of this tile so far
        const int token = row / a.G, head = row - token * a.G;
        while (const Piece* p = next_piece()) {
            const bool mine = token < p->tokens[t];
            const int tok = p->tok0 + t * a.tpt + token;
            float c = a.scale_log2;
            if constexpr (FP8) {
                // Q in fp16, scaled (query_exponent); one thread converts its own row
                // (a tile without rows gets here while the other one is at the piece before)
                if (!wait(q_empty, q_phase ^ 1u, 1, kPieceWaitNs)) break;
                q_phase ^= 1u;
                const __nv_bfloat16* src = a.q + static_cast<int64_t>(p->seq.first + tok) * a.ldq +
                                           (static_cast<int64_t>(p->h) * a.G + head) * D;
                uint4 v[D / 8];
                float big = 0.0f;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    v[i] = mine ? load16(reinterpret_cast<const uint8_t*>(src + 8 * i)) : make_uint4(0, 0, 0, 0);
                    float f[8];
                    unpack8(v[i], f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) big = fmaxf(big, fabsf(f[j]));
                }
                const int e = query_exponent(big);
                const float down = power_of_two(-e);
                c = c * a.kv.scales[p->h] * power_of_two(e);
                if (c == 0.0f) c = FLT_MIN;  // 0 times a masked score of -infinity would be NaN
                uint8_t* const dst = base_ptr + t * L::kTile + row * 128;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    float f[8];
                    unpack8(v[i], f);
                    *reinterpret_cast<uint4*>(dst + (i >> 3) * kHalf + (((i & 7) ^ (row & 7)) << 4)) =
                        make_uint4(pack_half2(f[0] * down, f[1] * down), pack_half2(f[2] * down, f[3] * down),
                                   pack_half2(f[4] * down, f[5] * down), pack_half2(f[6] * down, f[7] * down));
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full(t));
            }
            float m = -CUDART_INF_F, l = 0.0f;  // reference maximum (log2 units), sum
            const int begin = p->begin(t), end = p->end(t);
            // keys that this row sees: [lo, hi); that every row of the tile sees: [last_lo, first_hi)
            const int hi = p->seq.hi(mine ? tok : p->seq.n - 1);
            const int lo = prompt_lo_key(a, hi);
            const int first_hi = p->seq.hi(p->tok0 + t * a.tpt);
            const int last_lo = prompt_lo_key(a, p->last_hi[t]);
            const uint32_t block0 = blocks - p->b0;
            blocks += p->b1 - p->b0;
            bool ok = true;
            for (int j = begin; j < end; ++j) {
                const int buf = j & 1;
                if (!(ok = wait(s_full(t, buf), (s_phase >> buf) & 1u, 2))) break;
                s_phase ^= 1u << buf;
                const uint32_t have = (groups[(block0 + (j >> 1)) & 7] >> (4 * buf)) & 0xFu;
                ptx::tc_fence_after();
                const uint32_t ts = tmem_s(t) + lanes + kSB * buf;
                uint32_t s[kSB];
                ptx::tmem_ld_32x32b_x32(ts, *reinterpret_cast<uint32_t(*)[32]>(s));
                ptx::tmem_ld_32x32b_x32(ts + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
                ptx::tmem_wait_ld(*reinterpret_cast<uint32_t(*)[32]>(s));
                ptx::tmem_wait_ld(*reinterpret_cast<uint32_t(*)[32]>(s + 32));
                const int key0 = j * kSB;
                if (last_lo > key0 || have != 0xFu) {
                    const int below = hi - key0, from = lo - key0;
#pragma unroll
                    for (int k = 0; k < kSB; ++k) {
                        const bool on = k < below && k >= from && ((have >> (k >> 4)) & 1u);
                        s[k] = on ? s[k] : 0xFF800000u;
                    }
                } else if (first_hi < key0 + kSB) {
                    const int below = hi - key0;
#pragma unroll
                    for (int k = 0; k < kSB; ++k) s[k] = k < below ? s[k] : 0xFF800000u;
                }
                float top[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    top[x] = __uint_as_float(s[x]);
#pragma unroll
                    for (int k = 4; k < kSB - 4; k += 8)
                        top[x] = max3(top[x], __uint_as_float(s[k + x]), __uint_as_float(s[k + 4 + x]));
                    top[x] = fmaxf(top[x], __uint_as_float(s[kSB - 4 + x]));
                }
                const float now = fmaxf(max3(top[0], top[1], top[2]), top[3]) * c;
                const bool move = now > m + kLazyLog2;
                if (__any_sync(~0u, move)) {
                    const float f = move ? exp2_approx(m - now) : 1.0f;
                    if (move) m = now;
                    l *= f;
                    // O of the steps before is scaled, once the last of their products (of the
                    // other buffer) is done
                    if (j > begin) {
                        if (!(ok = wait(pv_done(t), (pv_count - 1) & 1u, 17))) break;
                        ptx::tc_fence_after();
#pragma unroll 1
                        for (int x = 0; x < D; x += 32) {
                            uint32_t o[32];
                            ptx::tmem_ld_32x32b_x32(tmem_o(t) + lanes + x, o);
                            ptx::tmem_wait_ld(o);
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            tmem_st_x32(tmem_o(t) + lanes + x, o);
                        }
                    }
                }
                ++pv_count;
                // P = 2^(S c - m), two values to an instruction where there is one
                const float shift = (FP8 ? kRaiseLog2 : 0.0f) - (m == -CUDART_INF_F ? 0.0f : m);
                const float2 c2 = make_float2(c, c), shift2 = make_float2(shift, shift);
                float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                uint32_t w[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    float2 e = fma2(make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), c2, shift2);
                    e.x = exp2_approx(e.x);
                    e.y = exp2_approx(e.y);
                    sum[k & 1] = add2(sum[k & 1], e);
                    // rounded to 16 bits for the product with V, of V's type (both operands of these
                    // instructions have one type): half a step of a weight is 2^-8 of it in bf16,
                    // 2^-11 in fp16; its sum is taken before
                    w[k] = FP8 ? pack_half2(e.x, e.y) : pack_bf162(e.x, e.y);
                }
                tmem_st_x32(ts, w);
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(t, buf));
            }
            if (!ok) break;
            // -------------------------------------------------------- the tile's result
            const int64_t qrow = p->seq.first + tok;
            const int64_t qhead = static_cast<int64_t>(p->h) * a.G + head;
            const int from = p->first, upto = p->last;
            const bool whole = from == upto;
            float* const slots = a.partial + static_cast<int64_t>(t) * kPromptSlotFloats;
            float* const slot = slots + (static_cast<int64_t>(blockIdx.x) * 2 + p->starts) * 2 * kPromptSlotFloats;
            const float v_scale = FP8 ? a.kv.scales[a.kv.Hkv + p->h] : 1.0f;
            __nv_bfloat16* const dst = mine ? a.out + qrow * a.ldo + qhead * D : nullptr;
            uint8_t* const stage = base_ptr + L::kStore0 + warp * 2048;
            __nv_bfloat16* rows_to[4];  // rows 8k + lane / 4, from their lanes
#pragma unroll
            for (int k = 0; k < 4; ++k)
                rows_to[k] = reinterpret_cast<__nv_bfloat16*>(
                    __shfl_sync(~0u, reinterpret_cast<unsigned long long>(dst), 8 * k + (lane >> 2)));
            // 32 columns of the warp's 32 rows: through shared memory, so that four lanes write 64
            // contiguous bytes of a row
            auto put = [&](int col, const float* v, float inv) {
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = v[8 * k + e] * inv;
                    *reinterpret_cast<uint4*>(stage + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) = pack8_bf16(x);
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = 8 * k + (lane >> 2), x = lane & 3;
                    const uint4 w = *reinterpret_cast<const uint4*>(stage + r * 64 + ((x ^ ((r >> 1) & 3)) << 4));
                    if (rows_to[k]) *reinterpret_cast<uint4*>(rows_to[k] + col + 8 * x) = w;
                }
            };
            auto put_lse = [&](float mm, float ll) {
                if (a.lse && mine)
                    a.lse[qrow * a.Hq + qhead] =
                        ll == 0.0f ? -CUDART_INF_F
                                   : (mm + log2f(ll) - (FP8 ? kRaiseLog2 : 0.0f)) * 0.69314718055994531f;
            };
            const float inv = l == 0.0f ? 0.0f : v_scale / l;  // no keys: zeros
            const bool any = end > begin;
            // The tile has to be done again if a row's sums are not finite though its weights' is
            // (one token to an item: all rows see the same keys).
            const int careful = p->careful;
            const bool suspect = any && mine && a.cu_q && !careful && l - l == 0.0f;
            // (the other tile's result may stand already)
            const bool give = p->tokens[t] > 0 && (!careful || ((careful >> t) & 1));
            if (any) {
                if (!wait(o_full(t), o_phase, 3)) break;
                o_phase ^= 1u;
                ptx::tc_fence_after();
                if (careful) add_cleared<D, FP8>(a, *p, lo, mine ? hi : 0, tmem_o(t) + lanes);
            }
            float2 not_finite[4] = {};  // NaN once a sum is not finite
            auto check = [&] {
                const float2 x = add2(add2(not_finite[0], not_finite[1]), add2(not_finite[2], not_finite[3]));
                if (suspect && !(x.x + x.y == 0.0f)) atomicOr(&const_cast<Piece*>(p)->redo, 1 << t);
                __syncwarp();
                if (lane == 0) mbar_arrive(checked(piece_at % kPieces));
            };
            if (p->tokens[t] == 0) {
                check();
            } else {
#pragma unroll 1
                for (int col = 0; col < D; col += 64) {
                    uint32_t o[2][32];
                    if (any) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) ptx::tmem_ld_32x32b_x32(tmem_o(t) + lanes + col + 32 * x, o[x]);
#pragma unroll
                        for (int x = 0; x < 2; ++x) ptx::tmem_wait_ld(o[x]);
                        if (col + 64 == D) {
                            ptx::tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(o_empty(t));
                        }
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int k = 0; k < 32; k += 2)
                                not_finite[k / 2 & 3] = fma2(make_float2(__uint_as_float(o[x][k]), __uint_as_float(o[x][k + 1])),
                                                             make_float2(0.0f, 0.0f), not_finite[k / 2 & 3]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[0][k] = o[1][k] = 0u;
                    }
                    if (col + 64 == D) check();
                    if (!give) continue;
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if (whole) {
                            float v[32];
#pragma unroll
                            for (int k = 0; k < 32; ++k) v[k] = l == 0.0f ? 0.0f : __uint_as_float(o[x][k]);
                            put(col + 32 * x, v, inv);
                        } else if (mine) {
#pragma unroll
                            for (int k = 0; k < 32; k += 4)
                                __stcg(reinterpret_cast<float4*>(slot + (col + 32 * x + k) * 128 + row * 4),
                                       make_float4(__uint_as_float(o[x][k]), __uint_as_float(o[x][k + 1]),
                                                   __uint_as_float(o[x][k + 2]), __uint_as_float(o[x][k + 3])));
                        }
                    }
                }
            }
            if (whole) {
                if (give) put_lse(m, l);
            } else if (give) {
                // The last contributor to arrive sums all of them, first to last (see the row
                // kernel); each tile's 128 threads count and join on their own.
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
                        s_last[t] = 0;
                        if (!((*const_cast<const volatile int*>(&p->redo) >> t) & 1)) {
                            __threadfence();
                            const uint32_t n = atomicAdd(a.count + 2 * from + t, 1u);
                            s_last[t] = n == static_cast<uint32_t>(upto - from);
                            if (s_last[t]) a.count[2 * from + t] = 0;
                            __threadfence();
                        }
                        mbar_arrive(join_out(t));
                    }
                    __syncwarp();
                }
                if (!wait(join_out(t), j_phase, 14)) break;
                j_phase ^= 1u;
                if (*reinterpret_cast<volatile uint32_t*>(s_last + t)) {
                    __threadfence();
                    const int count = p->tokens[t] * a.G;
                    if (count > 64) join_rows<D, FP8, 1>(a, *p, t, row, count, slots, v_scale);
                    else if (count > 32) join_rows<D, FP8, 2>(a, *p, t, row, count, slots, v_scale);
                    else if (count > 16) join_rows<D, FP8, 4>(a, *p, t, row, count, slots, v_scale);
                    else join_rows<D, FP8, 8>(a, *p, t, row, count, slots, v_scale);
                }
            }
            release_piece();
        }
    } else if (warp == 8 || warp == 10) {
        // ------------------------------------------------------------ MMAs of one tile
        const int t = (warp - 8) >> 1;
        const uint32_t ts = tmem_s(t), to = tmem_o(t);
        const uint64_t dq = sdesc_k128(base + t * L::kTile);
        uint32_t stage = 0, phase = 0, q_phase = 0, p_phase[2] = {0, 0}, o_phase = 0, blocks = 0;
        bool ok = true;
        while (ok) {
            const Piece* p = next_piece();
            if (!p) break;
            const int b0 = p->b0, b1 = p->b1, begin = p->begin(t), end = p->end(t), last_hi = p->last_hi[t];
            const int item_hi = max(p->last_hi[0], p->last_hi[1]);
            const int item_lo = p->careful ? INT_MAX : p->lo_key;  // (the careful way looks at every block)
            if (b1 > b0 || FP8) {
                if (!(ok = wait(q_full(t), q_phase, 4))) break;
                q_phase ^= 1u;
                ptx::tc_fence_after();
            }
            // Round i: O += P V for the two steps of block i - 1, each followed by S of the step
            // two later (block i), which may overwrite that P once its product has been issued.
            // So a step's S is ready before the softmax of the step before it has ended.
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
                    if (item_hi < i * kPB || item_lo > (i - 1) * kPB || have != 0xFFu) {
                        const Piece& q = *piece_of(piece_at);
                        if constexpr (FP8) clear_values_e4m3<D>(a, q, base_ptr + sv, (i - 1) * kPB, have, lane);
                        else clear_values<D, false>(a, q, base_ptr + sv, (i - 1) * kPB, have, lane);
                        fence_async_shared();
                        __syncwarp();
                    }
                }
                if (i < b1) {
                    if (!(ok = wait(full(ks), kph, 8))) break;
                    ptx::tc_fence_after();
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int jv = 2 * (i - 1) + u, jk = 2 * i + u;
                    if (jv >= begin && jv < end) {
                        const bool fresh = jv == begin;
                        if (fresh) {  // the tile's result before this one has been read
                            if (!(ok = wait(o_empty(t), o_phase ^ 1u, 6))) break;
                            o_phase ^= 1u;
                        }
                        if (!(ok = wait(p_full(t, u), p_phase[u], 7))) break;
                        p_phase[u] ^= 1u;
                        ptx::tc_fence_after();
                        const int groups16 = min(kSB, last_hi - jv * kSB + 15) / 16;
                        if (elect_one()) {
                            if (groups16 == kSB / 16) {
#pragma unroll
                                for (int k = 0; k < kSB / 16; ++k)
                                    mma_ts(to, ts + kSB * u + 8 * k, dv + 512 * u + 128 * k, kIdescO, k == 0 ? !fresh : 1u);
                            } else {
                                for (int k = 0; k < groups16; ++k)
                                    mma_ts(to, ts + kSB * u + 8 * k, dv + 512 * u + 128 * k, kIdescO, k == 0 ? !fresh : 1u);
                            }
                            ptx::mma_commit(pv_done(t));
                            if (jv + 1 == end) ptx::mma_commit(o_full(t));
                        }
                        __syncwarp();
                    }
                    if (jk >= begin && jk < end && i < b1) {
                        if (elect_one()) {
#pragma unroll
                            for (int k = 0; k < D / 16; ++k) {
                                const uint32_t off = (k >> 2) * (kHalf >> 4) + 2 * (k & 3);
                                ptx::mma_bf16_ss(ts + kSB * u, dq + off, dk + 512 * u + off, kIdescS, k ? 1u : 0u);
                            }
                            ptx::mma_commit(s_full(t, u));
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
            if (FP8 && b1 == b0 && elect_one()) ptx::mma_commit(q_empty);
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
    } else if (warp == 9) {
        // ------------------------------------------------------------ TMA producer
        const int rows = min(1 << a.kv.page_shift, kPB);  // of a copy
        const int copies = kPB / rows;
        uint32_t stage = 0, phase = 0, issued = 0, q_phase = 0, q_loads = 0, blocks = 0;
        constexpr int NR = FP8 ? NRAW : NST;
        bool ok = true;
        while (ok) {
            const Piece* p = next_piece();
            if (!p) break;
            const int b0 = p->b0, b1 = p->b1, h = p->h, b = p->b;
            const int top = max(p->last_hi[0], p->last_hi[1]), low = p->lo_key;
            if (!FP8 && b1 > b0) {
                if (!(ok = wait(q_empty, q_phase ^ 1u, 9))) break;
                q_phase ^= 1u;
                if (lane == 0) {
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        ptx::mbar_arrive_expect_tx(q_full(t), static_cast<uint32_t>(a.tpt * a.G) * D * 2);
                        for (int x = 0; x < D / 64; ++x)
                            ptx::tma_load_3d(base + t * L::kTile + x * kHalf, &tmQ, q_full(t), 64 * x, h * a.G,
                                             p->seq.first + p->tok0 + t * a.tpt);
                    }
                }
                ++q_loads;
            }
            // whether this lane copies a part of block i: not past the item's last key, and no page
            // that lies before its first (a window's user may have given that page away)
            auto wanted = [&](int i) {
                const int key = i * kPB + lane * rows;
                return lane < copies && i < b1 && key < top && key + rows > low;
            };
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
            if (q_loads)
                for (int t = 0; t < 2; ++t) ptx::mbar_wait_drain(q_full(t), (q_loads - 1) & 1u);
        }
        __syncwarp();
    } else if (warp == 11) {
        // ------------------------------------------------------------ work list
        bool ended = false;
        uint32_t next_redo = 0;  // the piece after the last one to be done again
        for (;; ++piece_at) {
            // (an item is asked for only when there is room for it)
            if (!wait(piece_empty(piece_at % kPieces), ((piece_at / kPieces) & 1u) ^ 1u, 16, kPieceWaitNs)) break;
            // A piece that has to be done again, the careful way, is the next one: the one that was
            // in this slot, or, with no more items, the one before, once its sums are known.
            Piece p;
            p.valid = 0;
            auto redone = [&](uint32_t k) {
                const Piece* const old = piece_of(k);
                if (!old->redo || k + 1 == next_redo) return false;
                p = *old;
                p.careful = old->redo;
                p.redo = 0;
                next_redo = k + 1;
                return true;
            };
            if (piece_at < kPieces || !redone(piece_at - kPieces)) {
                if (!ended) p = work.next(a);
                if (!p.valid) {
                    ended = true;
                    if (piece_at > 0) {
                        if (!wait(checked((piece_at - 1) % kPieces), ((piece_at - 1) / kPieces) & 1u, 16, kPieceWaitNs)) break;
                        redone(piece_at - 1);
                    }
                }
            }
            if (lane == 0) {
                if (p.valid) *const_cast<Piece*>(piece_of(piece_at)) = p;
                else const_cast<Piece*>(piece_of(piece_at))->valid = 0;
                mbar_arrive(piece_full(piece_at % kPieces));
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
        const int tid = (warp - 12) * 32 + lane;
        while (ok) {
            const Piece* p = next_piece();
            if (!p) break;
            const int n = 2 * (p->b1 - p->b0);
            release_piece();
            for (int x0 = 0; x0 < n; ++x0) {
                if (!(ok = wait(raw_full(rs), rph, 11))) break;
                if (!(ok = wait(empty(stage), phase ^ 1u, 12))) break;
                const uint8_t* src = base_ptr + L::kRaw0 + rs * L::kRaw;
                uint8_t* dst = base_ptr + L::kStage0 + stage * L::kTile;
                constexpr int kParts = kPB * D / 16 / 256;  // 16-byte parts per thread
                uint4 v[kParts];
#pragma unroll
                for (int x = 0; x < kParts; ++x) v[x] = *reinterpret_cast<const uint4*>(src + (x * 256 + tid) * 16);
#pragma unroll
                for (int x = 0; x < kParts; ++x) {
                    const int part = x * 256 + tid;
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
    if (warp == 8) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

}  // namespace tpmlp
