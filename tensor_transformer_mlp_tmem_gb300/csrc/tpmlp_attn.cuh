// Attention over a paged key-value cache: the append kernel (rotation, page writes) and the
// row kernel (decode: attention of one token's query heads over its sequence's keys).
//
// A pool is [num_pages][Hkv][page][D]: the keys of one head in one page are contiguous, so a
// warp that walks a head's keys reads whole 16-byte pieces of whole rows, whatever the page size.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math_constants.h>

#include "sm103_ptx.cuh"
#include "tpmlp_context.h"

namespace tpmlp {

// The caller's cache and the context's head layout, as the kernels read them.
struct KvView {
    uint8_t* K;
    uint8_t* V;
    int64_t page_bytes;   // from page to page of a pool
    int64_t head_bytes;   // from head to head of a page
    const int32_t* table;
    int64_t table_stride;
    int32_t table_pages;
    int32_t page_shift;   // log2 of the keys per page
    int32_t num_pages;
    const int32_t* lens;
    int32_t B;
    int32_t Hkv;
    const float* scales;  // e4m3: [2][Hkv] k and v scales
    int* status;          // kStatusWords
};

__device__ __forceinline__ void report_bad_page(int* status) {
    *reinterpret_cast<volatile int*>(status + kBadPageWord) = 1;
}

// Keys of sequence b: its length held to [0, the table's capacity].
__device__ __forceinline__ int kv_length(const KvView& kv, int b) {
    int len = kv.lens[b];
    const int64_t most = static_cast<int64_t>(kv.table_pages) << kv.page_shift;
    if (len > most) {
        report_bad_page(kv.status);
        len = static_cast<int>(most);
    }
    return max(len, 0);
}

// The table's entry for key `key` (inside the table) of sequence b.
__device__ __forceinline__ int kv_entry(const KvView& kv, int b, int key) {
    return kv.table[b * kv.table_stride + (key >> kv.page_shift)];
}

// A table entry as a page of the pool; -1, reported, if it names none.
__device__ __forceinline__ int kv_checked(const KvView& kv, int p) {
    if (p >= 0 && p < kv.num_pages) return p;
    report_bad_page(kv.status);
    return -1;
}

__device__ __forceinline__ int kv_page(const KvView& kv, int b, int key) {
    return kv_checked(kv, kv_entry(kv, b, key));
}

// ------------------------------------------------------------------ append
struct AppendArgs {
    KvView kv;
    const __nv_bfloat16 *q, *k, *v;
    int64_t ldq, ldk, ldv;
    __nv_bfloat16* q_out;
    int64_t ldqo;
    const int32_t *pos, *seq;
    int32_t Hq;         // 0: no queries
    int32_t rot;        // rotated dimensions, a multiple of 16
    int32_t interleaved;
    int32_t parts;      // blocks per token
    int32_t part_units; // units of each
    int32_t T;
    int32_t tokens;     // tokens per block (more than one: parts is 1)
    uint32_t per_unit;  // 2^32 / units of a token, rounded up
    double turns[64];   // whole turns per position of each pair
};

// Loads of what another kernel of the stream may have just written: through L2 (the read-only
// path must not be used while this kernel may overlap the writer's end).
__device__ __forceinline__ uint4 load16(const uint8_t* p) {
    return __ldcg(reinterpret_cast<const uint4*>(p));
}
constexpr int kAppendThreads = 128;
constexpr int kAppendUnits = 3;  // units of 16 elements that a thread has in flight
// Blocks an SM, which hold a thread to 64 registers. 16384 tokens of 32 query and 8 kv heads: 6, 7, 8, 9
// blocks 74, 70, 66, 69 us; 8 blocks and units of 2, 4: 71, 79 us.
constexpr int kAppendBlocks = 8;
constexpr int kAppendTokens = 8;  // tokens of a block, at most

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8_bf16(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// x / scale to e4m3, to nearest even, held to +-448 (NaN stays NaN).
__device__ __forceinline__ uint2 pack8_e4m3(const float (&f)[8], float scale) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_fp8x2_storage_t h = __nv_cvt_float2_to_fp8x2(
            make_float2(f[2 * i] / scale, f[2 * i + 1] / scale), __NV_SATFINITE, __NV_E4M3);
        w[i >> 1] |= static_cast<uint32_t>(h) << (16 * (i & 1));
    }
    return make_uint2(w[0], w[1]);
}

// A block takes a token, one of `parts` equal parts of it where there are few tokens, or (MANY)
// several tokens where a token has so few heads that its units would leave threads idle. The
// rotation's sines and cosines are the same for all heads: the block computes the token's rot / 2
// of them once, in shared memory, while its first loads are under way. The angle is taken in whole
// turns in fp64 and reduced to [-1/2, 1/2] there, so its error is that of the fp32 result however
// far the position (an fp32 product would be off by whole radians at position 10^7). A thread
// takes units of 16 elements: 8 dimensions of the lower half of a head's rotated (or other)
// dimensions and the 8 of the upper half that lie as far on, so that neighbouring threads read and
// write neighbouring 16 bytes; where halves are rotated they are the partners. Bound by DRAM: 16384
// tokens of 32 query and 8 kv heads of 128 in 67 us, 6.0 TB/s, 89 % of a copy's rate (256 threads a
// block, each loading a unit when it had the sines: 87 us).
template <int D, bool FP8, bool MANY>
__global__ void __launch_bounds__(kAppendThreads, kAppendBlocks) append_kernel(const __grid_constant__ AppendArgs a) {
    constexpr int kTokens = MANY ? kAppendTokens : 1;
    __shared__ float2 trig[kTokens * (D / 2)];
    __shared__ int2 places[kTokens];  // MANY: position and page of each token
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    constexpr int kUnits = D / 16;  // units per head
    const int64_t t0 = MANY ? static_cast<int64_t>(blockIdx.x) * a.tokens : blockIdx.x / a.parts;
    const int tokens = MANY ? static_cast<int>(min(static_cast<int64_t>(a.tokens), a.T - t0)) : 1;
    const int units = (a.Hq + 2 * a.kv.Hkv) * kUnits;
    const int begin = MANY ? 0 : static_cast<int>(blockIdx.x % a.parts) * a.part_units;
    const int end = MANY ? tokens * units : min(begin + a.part_units, units);
    const int half = a.rot >> 1;
    // the position and sequence of this thread's token (MANY: of the block's thread-th)
    const bool own = !MANY || static_cast<int>(threadIdx.x) < tokens;
    const int64_t t_own = t0 + (MANY ? threadIdx.x : 0);
    int pos = own ? a.pos[t_own] : -1, page = -1;
    const int b = !own ? -1 : a.seq ? a.seq[t_own] : static_cast<int>(t_own);
    for (int first = begin; first < end; first += kAppendThreads * kAppendUnits) {
        uint4 raw[kAppendUnits][2];
        // unit i: its token of the block, part of the token, head, whether it is rotated, its two
        // pieces of 8 dimensions
        struct Unit {
            int token, kind, h, d0, d1;  // kind: 0 q, 1 k, 2 v
            bool rotate;
        };
        auto unit = [&](int i) {
            Unit x;
            x.token = MANY ? static_cast<int>(__umulhi(static_cast<uint32_t>(i), a.per_unit)) : 0;
            if (MANY) i -= x.token * units;
            const int head = i / kUnits, u = i % kUnits;
            x.kind = head < a.Hq ? 0 : head < a.Hq + a.kv.Hkv ? 1 : 2;
            x.h = x.kind == 0 ? head : x.kind == 1 ? head - a.Hq : head - a.Hq - a.kv.Hkv;
            x.rotate = x.kind != 2 && 16 * u < a.rot;
            const int first = x.kind == 2 || x.rotate ? 0 : a.rot;
            const int dims = x.kind == 2 ? D : x.rotate ? a.rot : D - a.rot;
            x.d0 = first + 8 * (u - first / 16);
            x.d1 = x.d0 + dims / 2;
            return x;
        };
#pragma unroll
        for (int y = 0; y < kAppendUnits; ++y) {
            const int i = first + y * kAppendThreads + static_cast<int>(threadIdx.x);
            if (i >= end) break;
            const Unit x = unit(i);
            const int64_t t = t0 + x.token;
            const __nv_bfloat16* src = (x.kind == 0 ? a.q + t * a.ldq : x.kind == 1 ? a.k + t * a.ldk : a.v + t * a.ldv) +
                                       static_cast<int64_t>(x.h) * D;
            raw[y][0] = load16(reinterpret_cast<const uint8_t*>(src + x.d0));
            raw[y][1] = load16(reinterpret_cast<const uint8_t*>(src + x.d1));
        }
        if (first == begin) {
            if (!MANY && pos < 0) return;
            // the table's entry, asked for before the sines of many tokens and after those of one
            // (16384 tokens of 12 + 12 heads of 64: 30 against 35 us; of 32 + 8 heads of 128: 70 against 67)
            auto look_up = [&] {
                const bool inside = b >= 0 && b < a.kv.B && pos >= 0 && (pos >> a.kv.page_shift) < a.kv.table_pages;
                return inside ? kv_entry(a.kv, b, pos) : -1;
            };
            int entry = MANY ? look_up() : -1;
            for (int i = threadIdx.x; i < (MANY ? tokens * (D / 2) : half); i += kAppendThreads) {
                const int d = i % (D / 2);
                if (MANY && d >= half) continue;
                const double turn = (MANY ? a.pos[t0 + i / (D / 2)] : pos) * a.turns[d];
                float s, c;
                sincospif(2.0f * static_cast<float>(turn - rint(turn)), &s, &c);
                trig[i] = make_float2(c, s);
            }
            if (!MANY) entry = look_up();
            if (pos >= 0) page = kv_checked(a.kv, entry);  // -1: the token's k and v are dropped
            if (MANY && own) places[threadIdx.x] = make_int2(pos, page);
            __syncthreads();
        }
#pragma unroll
        for (int y = 0; y < kAppendUnits; ++y) {
            const int i = first + y * kAppendThreads + static_cast<int>(threadIdx.x);
            if (i >= end) break;
            const Unit w = unit(i);
            if constexpr (MANY) {
                pos = places[w.token].x;
                page = places[w.token].y;
                if (pos < 0) continue;
            }
            const int64_t t = t0 + w.token;
            const int slot = pos & ((1 << a.kv.page_shift) - 1);
            const float2* const turns = trig + w.token * (D / 2);
            float x0[8], x1[8];
            unpack8(raw[y][0], x0);
            unpack8(raw[y][1], x1);
            if (w.rotate) {
                if (a.interleaved) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 r0 = turns[w.d0 / 2 + j], r1 = turns[w.d1 / 2 + j];
                        const float p0 = x0[2 * j], p1 = x1[2 * j];
                        x0[2 * j] = p0 * r0.x - x0[2 * j + 1] * r0.y;
                        x0[2 * j + 1] = x0[2 * j + 1] * r0.x + p0 * r0.y;
                        x1[2 * j] = p1 * r1.x - x1[2 * j + 1] * r1.y;
                        x1[2 * j + 1] = x1[2 * j + 1] * r1.x + p1 * r1.y;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 r0 = turns[w.d0 + j];
                        const float p0 = x0[j];
                        x0[j] = p0 * r0.x - x1[j] * r0.y;
                        x1[j] = x1[j] * r0.x + p0 * r0.y;
                    }
                }
            }
            if (w.kind == 0) {
                __nv_bfloat16* const dst = a.q_out + t * a.ldqo + static_cast<int64_t>(w.h) * D;
                *reinterpret_cast<uint4*>(dst + w.d0) = pack8_bf16(x0);
                *reinterpret_cast<uint4*>(dst + w.d1) = pack8_bf16(x1);
                continue;
            }
            if (page < 0) continue;
            uint8_t* const at = (w.kind == 2 ? a.kv.V : a.kv.K) + page * a.kv.page_bytes + w.h * a.kv.head_bytes +
                                static_cast<int64_t>(slot) * (D * (FP8 ? 1 : 2));
            if constexpr (FP8) {
                const float scale = a.kv.scales[(w.kind == 2 ? a.kv.Hkv : 0) + w.h];
                *reinterpret_cast<uint2*>(at + w.d0) = pack8_e4m3(x0, scale);
                *reinterpret_cast<uint2*>(at + w.d1) = pack8_e4m3(x1, scale);
            } else {
                *reinterpret_cast<uint4*>(at + 2 * w.d0) = pack8_bf16(x0);
                *reinterpret_cast<uint4*>(at + 2 * w.d1) = pack8_bf16(x1);
            }
        }
    }
}

// ------------------------------------------------------------------ rows
// Attention of one token of each sequence: row b has G query heads to each kv head, and attends to
// keys [lo, hi) of sequence b.
struct RowArgs {
    KvView kv;
    const __nv_bfloat16* q;
    int64_t ldq;
    __nv_bfloat16* out;
    int64_t ldo;
    float* lse;             // [rows][Hq] or null
    int32_t rows;           // sequences
    int32_t Hq, G;
    float scale_log2;         // softmax scale * log2(e)
    int32_t window;
    float* partial;         // [CTAs][2] slots of RowSlot floats
    uint32_t* count;        // [CTAs] arrivals, 0 between launches
};

// Query heads to a kv head that this kernel takes, at most; decode of wider groups goes to the prompt
// kernel, whose products' tiles they fill and which takes the same time for any G, while this
// kernel's time grows with every 8 heads, and from 17 on it takes its keys twice (PASSES; the second
// time from L2). 64 sequences of 4096 keys, 8 kv heads, this kernel against the prompt kernel, us:
//   D = 128, bf16: G = 8: 165, 188; 9: 215, 190; 16: 216, 187; 24: 417, 192
//   D = 128, e4m3: G = 16: 130, 223; 17: 244, 212; 32: 249, 214
//   D = 64, bf16:  G = 16: 112, 147; 17: 208, 147; 32: 210, 146
//   D = 64, e4m3:  G = 16: 77, 194; 17: 125, 191; 32: 129, 191; from G = 33 on three times and more
constexpr int row_heads(int D, bool fp8) { return D == 128 ? (fp8 ? 16 : 8) : (fp8 ? 32 : 16); }

constexpr int kRowWarps = 8;
// A segment's fixed time (its start, merge and result) in steps, as it counts in the CTAs' shares. 0, 1,
// 2, 3: 64 sequences of 8192 keys at most x 32 heads 617, 590, 591, 595 us; 48 sequences in e4m3, 12
// heads to a kv head 118, 104, 100, 101; one sequence of 131072 keys 88, 87, 85, 88.
constexpr int kSegmentStart = 2;
constexpr int kRowThreads = 32 * kRowWarps;
constexpr int kJoinLoads = 8;  // contributors of a split range whose sums a thread loads at once
// e4m3 caches: fp16 weights are raised by 2^10, so that the small ones of a long cache stay clear of
// fp16's smallest steps; it cancels against the sum.
constexpr float kRowRaise = 10.0f;
// fp32 values of a partial sum: O [16][128], m [16], l [16].
constexpr int kRowSlotFloats = 16 * 128 + 32;

__device__ __forceinline__ void mma_16816_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_16816_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit values spread over the warp (lane 4 r + c holds row r,
// columns 2 c and 2 c + 1).
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// Four e4m3 values as two pairs of fp16 (exact). The halves of the register are named, not
// masked and shifted out: that would cost as much again as the conversions.
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t v, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf162(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// e4m3 caches: the power of two by which a query row is divided before it is rounded to fp16, from
// the row's largest magnitude: that one comes to [2^14, 2^15), so that no bf16 value overflows and
// only what is 2^-28 of it and less meets fp16's smallest steps. The scores are multiplied by it
// again; it is held above 2^-100 so that it does not vanish with them. (Infinities stay infinite.)
__device__ __forceinline__ int query_exponent(float largest) {
    const int e = static_cast<int>(__float_as_uint(largest) >> 23) - 127 - 14;
    return largest == 0.0f ? 0 : max(-100, min(e, 113));
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// Keys of a row: [lo, hi) of its sequence.
struct RowRange {
    int lo, hi;
};

__device__ __forceinline__ RowRange row_range(const RowArgs& a, int b) {
    RowRange x{0, kv_length(a.kv, b)};
    if (a.window > 0) x.lo = max(0, x.hi - a.window);
    return x;
}

// The kernel's shape. A warp takes KT keys at a time and holds all their K and V in registers (8 KB
// of cache per warp and iteration): K rows are the A operand of S^T = K Q^T (16 keys x 8 query
// heads a matrix instruction), so the loads are whole 16-byte pieces of the rows as they lie in
// memory, in an order of the reduction index that Q's registers share; V is the A operand of
// O^T = V^T P^T, its pairs of keys put together with byte permutes. No shared memory, no barriers
// and no copies are needed on the way: 16 warps an SM keep 128 KB of loads in flight, and the
// bound is DRAM (64 sequences of 4096 keys x 32 heads in bf16: 6.6 TB/s, 97 % of a copy's rate).
// Tried and slower by a fifth to a third: the same tiles copied to shared memory ahead of use
// (cp.async), also for the wide head groups alone, and loading the next tile's K and V in
// registers while this one is in use (spills), also each only once the registers of this one's are
// free (591 against 690 us; 12 heads to a kv head in e4m3 100 against 101). A warp holds NT = 1 or 2 blocks of
// 8 query heads (2: one CTA an SM). e4m3 values are converted to fp16 in registers (the 8-bit forms
// of these matrix instructions take three times as long as the fp16 ones on this GPU).
template <int D, bool FP8, int NT>
struct RowShape {
    static constexpr int kElem = FP8 ? 1 : 2;
    static constexpr int kSub = 256 / (D * kElem);   // subtiles of 16 keys
    static constexpr int KT = 16 * kSub;
    static constexpr int kStep = KT * kRowWarps;     // keys of a CTA's step
    static constexpr int kRows = 8 * NT;             // query heads
    static constexpr int kCtasPerSm = NT == 1 ? 2 : 1;
    static constexpr int NK = D * kElem / 64;        // 16-byte pieces of a K row per thread
    static constexpr int NV = D / 8;                 // V dimensions per thread
    static constexpr int kVPieces = NV * kElem >= 16 ? NV * kElem / 16 : 1;  // 16-byte pieces of a V row
    static constexpr int kQRegs = D / 8;             // Q registers of 8 query heads
    static constexpr int kPitch = D + 4;             // fp32 row of the merge buffer
    static constexpr int kSmem = kRowWarps * 8 * NT * (kPitch + 2) * 4;
};

// The dimension that element e of lane group g's V registers stands for.
template <int D, bool FP8>
__device__ __forceinline__ int v_dim(int g, int e) {
    if constexpr (D == 128 && !FP8) return e < 8 ? 8 * g + e : 64 + 8 * g + (e - 8);
    else return (D / 8) * g + e;
}

template <int D, bool FP8, int NT, int PASSES>
__global__ void __launch_bounds__(kRowThreads, RowShape<D, FP8, NT>::kCtasPerSm)
attn_row_kernel(const __grid_constant__ RowArgs a) {
    using S = RowShape<D, FP8, NT>;
    extern __shared__ __align__(16) float smem[];  // (read and written in float4)
    float* const sO = smem;                                       // [parts][rows][pitch]
    float* const sM = sO + kRowWarps * S::kRows * S::kPitch;      // [parts][rows]
    float* const sL = sM + kRowWarps * S::kRows;                  // [parts][rows]
    __shared__ int64_t s_scan[kRowWarps + 1];
    __shared__ int64_t s_found[2];
    __shared__ uint32_t s_last;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;

    ptx::griddep_wait();
    ptx::griddep_launch_dependents();

    auto steps_of = [&](const RowRange& x) {
        return max(1, (x.hi - (x.lo & ~15) + S::kStep - 1) / S::kStep);
    };
    // Sum of the rows' work: a (row, kv head, pass) segment's is its row's steps and kSegmentStart, and
    // each CTA takes an equal run of all segments' work. Then the row that holds this CTA's first unit.
    const int64_t per_row = static_cast<int64_t>(a.kv.Hkv) * PASSES;
    int64_t per_cta, at, end;
    int row = -1;
    int64_t row_start = 0;  // first unit of that row
    auto share = [&](int64_t total) {
        per_cta = (total + gridDim.x - 1) / gridDim.x;
        at = per_cta * blockIdx.x;
        end = min(at + per_cta, total);
    };
    if (a.rows <= 32) {
        // every warp for itself, a row to a lane: no barrier in a small call's way
        const uint32_t c = lane < a.rows ? kSegmentStart + steps_of(row_range(a, lane)) : 0;
        uint32_t sum = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(~0u, sum, o);
            if (lane >= o) sum += v;
        }
        share(__shfl_sync(~0u, sum, 31) * per_row);
        if (at >= end) return;
        row = __ffs(__ballot_sync(~0u, at < sum * per_row)) - 1;
        row_start = __shfl_sync(~0u, sum - c, row) * per_row;
    } else {
        int64_t mine = 0;
        for (int r = tid; r < a.rows; r += kRowThreads) mine += kSegmentStart + steps_of(row_range(a, r));
#pragma unroll
        for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(~0u, mine, o);
        if (lane == 0) s_scan[warp] = mine;
        __syncthreads();
        int64_t total = 0;
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) total += s_scan[w];
        share(total * per_row);
        if (at >= end) return;
        int64_t before = 0;
        for (int r0 = 0; r0 < a.rows; r0 += kRowThreads) {
            const int r = r0 + tid;
            const int64_t c = r < a.rows ? kSegmentStart + steps_of(row_range(a, r)) : 0;
            int64_t sum = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(~0u, sum, o);
                if (lane >= o) sum += v;
            }
            __syncthreads();
            if (lane == 31) s_scan[warp] = sum;
            if (tid == 0) s_found[0] = -1;
            __syncthreads();
            int64_t base = before;
            for (int w = 0; w < warp; ++w) base += s_scan[w];
            const int64_t first = (base + sum - c) * per_row;
            if (r < a.rows && at >= first && at < first + c * per_row) {
                s_found[0] = r;
                s_found[1] = first;
            }
            for (int w = 0; w < kRowWarps; ++w) before += s_scan[w];
            __syncthreads();
            if (s_found[0] >= 0) break;
        }
        row = static_cast<int>(s_found[0]);
        row_start = s_found[1];
        if (row < 0) return;  // only if the lengths changed during the launch
    }
    RowRange range = row_range(a, row);
    int steps = steps_of(range);
    int64_t segment_start;  // first unit of the current segment
    int part;               // kv head * PASSES + pass
    {
        const int64_t into = at - row_start;
        part = static_cast<int>(into / (steps + kSegmentStart));
        segment_start = row_start + static_cast<int64_t>(part) * (steps + kSegmentStart);
    }

    while (at < end) {
        const int step0 = max(static_cast<int>(at - segment_start) - kSegmentStart, 0);
        at = min(end, segment_start + steps + kSegmentStart);
        const int n = static_cast<int>(at - segment_start) - kSegmentStart - step0;
        if (n <= 0) return;  // the start alone: the segment's steps are the next CTA's
        const int h = part / PASSES;
        const int q0 = part % PASSES * S::kRows;  // the pass's query heads of the group
        auto heads = [&] { return PASSES > 1 ? min(a.G - q0, S::kRows) : a.G; };  // of them

        // Q in the reduction order of the K pieces; for an 8-bit cache's products in fp16, scaled
        // (query_exponent), and the scores scaled back.
        uint32_t qr[NT][S::kQRegs];
        float c_log2[NT][2];  // score -> log2 units, for the lane's query columns 2 t, 2 t + 1
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int qi = nt * 8 + g;
            const __nv_bfloat16* src = a.q + row * a.ldq + (static_cast<int64_t>(h) * a.G + q0 + qi) * D;
            const bool on = qi < heads();
            if constexpr (!FP8) {
#pragma unroll
                for (int j = 0; j < S::NK; ++j) {
                    const uint4 v = on ? load16(reinterpret_cast<const uint8_t*>(src + 8 * (t + 4 * j)))
                                       : make_uint4(0, 0, 0, 0);
                    qr[nt][4 * j] = v.x;
                    qr[nt][4 * j + 1] = v.y;
                    qr[nt][4 * j + 2] = v.z;
                    qr[nt][4 * j + 3] = v.w;
                }
                c_log2[nt][0] = c_log2[nt][1] = a.scale_log2;
            } else {
                float x[S::NK][2][8];
                float big = 0.0f;
#pragma unroll
                for (int j = 0; j < S::NK; ++j)
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const uint4 v = on ? load16(reinterpret_cast<const uint8_t*>(src + 16 * (t + 4 * j) + 8 * p))
                                           : make_uint4(0, 0, 0, 0);
                        unpack8(v, x[j][p]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(x[j][p][i]));
                    }
                big = fmaxf(big, __shfl_xor_sync(~0u, big, 1));
                big = fmaxf(big, __shfl_xor_sync(~0u, big, 2));
                const int e = query_exponent(big);
                const float down = power_of_two(-e), up = power_of_two(e);
#pragma unroll
                for (int j = 0; j < S::NK; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        qr[nt][8 * j + i] = pack_half2(x[j][i >> 2][2 * (i & 3)] * down, x[j][i >> 2][2 * (i & 3) + 1] * down);
                const float ks = a.scale_log2 * a.kv.scales[h];
                c_log2[nt][0] = ks * __shfl_sync(~0u, up, 8 * t);
                c_log2[nt][1] = ks * __shfl_sync(~0u, up, 8 * t + 4);
            }
        }

        float o[NT][S::NV / 2][4];  // O^T: (dim e, q 2t), (dim e, q 2t+1), (dim e + NV/2, ...)
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -CUDART_INF_F;
            l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
            for (int i = 0; i < S::NV / 2; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.0f;
        }

        const int64_t head_off = h * a.kv.head_bytes;
        const int lo16 = range.lo & ~15;
        for (int it = 0; it < n; ++it) {
            const int key0 = lo16 + ((step0 + it) * kRowWarps + warp) * S::KT;
            if (key0 >= range.hi) break;  // the warp's keys only grow
            int page[S::kSub];
            bool ok[S::kSub];
#pragma unroll
            for (int u = 0; u < S::kSub; ++u) {
                const int kb = key0 + 16 * u;
                page[u] = -1;
                if (kb < range.hi) page[u] = kv_page(a.kv, row, kb);
                ok[u] = page[u] >= 0;
            }
            uint4 kr[S::kSub][2][S::NK];
            uint4 vr[S::kSub][4][S::kVPieces];
#pragma unroll
            for (int u = 0; u < S::kSub; ++u) {
                const int kb = key0 + 16 * u;
                const int64_t off = page[u] * a.kv.page_bytes + head_off +
                                    static_cast<int64_t>(kb & ((1 << a.kv.page_shift) - 1)) * (D * S::kElem);
                const uint8_t* kp = a.kv.K + off;
                const uint8_t* vp = a.kv.V + off;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int key = kb + g + 8 * r;
                    const bool on = ok[u] && key >= range.lo && key < range.hi;
#pragma unroll
                    for (int j = 0; j < S::NK; ++j)
                        kr[u][r][j] = on ? load16(kp + (g + 8 * r) * (D * S::kElem) + 16 * (t + 4 * j))
                                         : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int kk = 2 * t + (x & 1) + 8 * (x >> 1);
                    const int key = kb + kk;
                    const bool on = ok[u] && key >= range.lo && key < range.hi;
                    const uint8_t* src = vp + kk * (D * S::kElem);
                    if constexpr (S::NV * S::kElem == 8) {
                        const uint2 w = on ? __ldcg(reinterpret_cast<const uint2*>(src + 8 * g)) : make_uint2(0, 0);
                        vr[u][x][0] = make_uint4(w.x, w.y, 0, 0);
                    } else {
#pragma unroll
                        for (int y = 0; y < S::kVPieces; ++y)
                            vr[u][x][y] = on ? load16(src + 128 * y + 16 * g) : make_uint4(0, 0, 0, 0);
                    }
                }
            }
            // S^T = K Q^T, in log2 units
            float s[S::kSub][NT][4];
            float top[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = -CUDART_INF_F;
#pragma unroll
            for (int u = 0; u < S::kSub; ++u) {
                const int kb = key0 + 16 * u;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s[u][nt][0] = s[u][nt][1] = s[u][nt][2] = s[u][nt][3] = 0.0f;
#pragma unroll
                for (int j = 0; j < S::NK; ++j) {
                    const uint4 x = kr[u][0][j], y = kr[u][1][j];
                    if constexpr (!FP8) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_16816_bf16(s[u][nt], x.x, y.x, x.y, y.y, qr[nt][4 * j], qr[nt][4 * j + 1]);
                            mma_16816_bf16(s[u][nt], x.z, y.z, x.w, y.w, qr[nt][4 * j + 2], qr[nt][4 * j + 3]);
                        }
                    } else {
                        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            uint32_t f[4];
                            e4m3x4_to_half2(xs[w], f[0], f[2]);
                            e4m3x4_to_half2(ys[w], f[1], f[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_16816_f16(s[u][nt], f[0], f[1], f[2], f[3], qr[nt][8 * j + 2 * w], qr[nt][8 * j + 2 * w + 1]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = kb + g + 8 * (i >> 1);
                    const bool on = ok[u] && key >= range.lo && key < range.hi;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        s[u][nt][i] = on ? s[u][nt][i] * c_log2[nt][i & 1] : -CUDART_INF_F;
                        top[nt][i & 1] = fmaxf(top[nt][i & 1], s[u][nt][i]);
                    }
                }
            }
            // running maximum and sum
            float base[NT][2];  // what a score's exponent is taken from
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float f[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float v = top[nt][i];
                    v = fmaxf(v, __shfl_xor_sync(~0u, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(~0u, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(~0u, v, 16));
                    const float now = fmaxf(m[nt][i], v);
                    f[i] = now == m[nt][i] ? 1.0f : exp2_approx(m[nt][i] - now);
                    m[nt][i] = now;
                    l[nt][i] *= f[i];
                    base[nt][i] = (now == -CUDART_INF_F ? 0.0f : now) - (FP8 ? kRowRaise : 0.0f);
                }
                if (__any_sync(~0u, f[0] != 1.0f || f[1] != 1.0f)) {
#pragma unroll
                    for (int i = 0; i < S::NV / 2; ++i) {
                        o[nt][i][0] *= f[0];
                        o[nt][i][1] *= f[1];
                        o[nt][i][2] *= f[0];
                        o[nt][i][3] *= f[1];
                    }
                }
            }
            // P^T, rounded to 16 bits for the product with V, of V's type: half a step of a weight is
            // 2^-8 of it in bf16, 2^-11 in fp16. Its sum is taken before the rounding, in fp32.
            uint32_t pb[S::kSub][NT][2];
#pragma unroll
            for (int u = 0; u < S::kSub; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        p[i] = exp2_approx(s[u][nt][i] - base[nt][i & 1]);
                        l[nt][i & 1] += p[i];
                    }
                    pb[u][nt][0] = transpose_8x8(FP8 ? pack_half2(p[0], p[1]) : pack_bf162(p[0], p[1]));
                    pb[u][nt][1] = transpose_8x8(FP8 ? pack_half2(p[2], p[3]) : pack_bf162(p[2], p[3]));
                }
            // O^T += V^T P^T
            // word w of the dimensions of the lane's key x
            auto word = [&](int u, int x, int w) {
                const uint4& y = vr[u][x][w >> 2];
                return (w & 3) == 0 ? y.x : (w & 3) == 1 ? y.y : (w & 3) == 2 ? y.z : y.w;
            };
#pragma unroll
            for (int u = 0; u < S::kSub; ++u)
#pragma unroll
                for (int i = 0; i < S::NV / 2; i += 2) {
                    // fragments of two instructions: dimensions i, i + 1 and those NV/2 further on
                    // (x & 1); keys 2t, 2t+1 and 2t+8, 2t+9 (x >> 1)
                    uint32_t av[2][4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int e = i + (x & 1) * (S::NV / 2), ka = 2 * (x >> 1);
                        if constexpr (!FP8) {
                            av[0][x] = __byte_perm(word(u, ka, e >> 1), word(u, ka + 1, e >> 1), 0x5410);
                            av[1][x] = __byte_perm(word(u, ka, e >> 1), word(u, ka + 1, e >> 1), 0x7632);
                        } else {
                            const uint32_t both =
                                __byte_perm(word(u, ka, e >> 2), word(u, ka + 1, e >> 2), (e & 2) ? 0x7362 : 0x5140);
                            e4m3x4_to_half2(both, av[0][x], av[1][x]);
                        }
                    }
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if constexpr (FP8)
                                mma_16816_f16(o[nt][i + y], av[y][0], av[y][1], av[y][2], av[y][3], pb[u][nt][0], pb[u][nt][1]);
                            else
                                mma_16816_bf16(o[nt][i + y], av[y][0], av[y][1], av[y][2], av[y][3], pb[u][nt][0], pb[u][nt][1]);
                        }
                }
        }

        // The warps' sums of this segment, joined in shared memory.
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float v = l[nt][i];
                v += __shfl_xor_sync(~0u, v, 4);
                v += __shfl_xor_sync(~0u, v, 8);
                v += __shfl_xor_sync(~0u, v, 16);
                l[nt][i] = v;
            }
        __syncthreads();  // the segment before has been read
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = warp * S::kRows + nt * 8 + 2 * t + i;
                if (g == 0) {
                    sM[r] = m[nt][i];
                    sL[r] = l[nt][i];
                }
                float* dst = sO + r * S::kPitch;
#pragma unroll
                for (int e = 0; e < S::NV; e += 4) {
                    const int k = e % (S::NV / 2), hi = e >= S::NV / 2 ? 2 : 0;
                    *reinterpret_cast<float4*>(dst + v_dim<D, FP8>(g, e)) =
                        make_float4(o[nt][k][hi + i], o[nt][k + 1][hi + i], o[nt][k + 2][hi + i], o[nt][k + 3][hi + i]);
                }
            }
        __syncthreads();

        // Contributors of the segment: the CTAs whose runs meet its steps.
        const int first = static_cast<int>((segment_start + kSegmentStart) / per_cta);
        const int last = static_cast<int>((segment_start + kSegmentStart + steps - 1) / per_cta);
        const bool whole = first == last;
        float* const slot = a.partial + (static_cast<int64_t>(blockIdx.x) * 2 + (step0 == 0)) * kRowSlotFloats;
        const float v_scale = FP8 ? a.kv.scales[a.kv.Hkv + h] : 1.0f;

        auto finish = [&](int r, int d, float4 v, float mm, float ll) {
            const int64_t head = static_cast<int64_t>(h) * a.G + q0 + r;
            const float inv = ll == 0.0f ? 0.0f : v_scale / ll;  // no keys: zeros
            uint2 w;
            w.x = pack_bf162(v.x * inv, v.y * inv);
            w.y = pack_bf162(v.z * inv, v.w * inv);
            *reinterpret_cast<uint2*>(a.out + row * a.ldo + head * D + d) = w;
            if (a.lse && d == 0)
                a.lse[static_cast<int64_t>(row) * a.Hq + head] =
                    ll == 0.0f ? -CUDART_INF_F
                               : (mm + log2f(ll) - (FP8 ? kRowRaise : 0.0f)) * 0.69314718055994531f;
        };
        for (int i = tid; i < heads() * (D / 4); i += kRowThreads) {
            const int r = i / (D / 4), d = (i % (D / 4)) * 4;
            float mm = -CUDART_INF_F;
#pragma unroll
            for (int w = 0; w < kRowWarps; ++w) mm = fmaxf(mm, sM[w * S::kRows + r]);
            const float safe = mm == -CUDART_INF_F ? 0.0f : mm;
            float ll = 0.0f;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kRowWarps; ++w) {
                const float f = exp2_approx(sM[w * S::kRows + r] - safe);
                const float4 x = *reinterpret_cast<const float4*>(sO + (w * S::kRows + r) * S::kPitch + d);
                ll += f * sL[w * S::kRows + r];
                v.x += f * x.x;
                v.y += f * x.y;
                v.z += f * x.z;
                v.w += f * x.w;
            }
            if (whole) {
                finish(r, d, v, mm, ll);
            } else {
                __stcg(reinterpret_cast<float4*>(slot + r * D + d), v);
                if (d == 0) {
                    __stcg(slot + 16 * 128 + r, mm);
                    __stcg(slot + 16 * 128 + 16 + r, ll);
                }
            }
        }
        if (!whole) {
            // The last contributor to arrive sums all of them, first to last. The counter
            // belongs to the first contributor, which starts one split segment at most.
            __threadfence();
            __syncthreads();
            if (tid == 0) s_last = atomicAdd(a.count + first, 1u) == static_cast<uint32_t>(last - first);
            __syncthreads();
            if (s_last) {
                __threadfence();
                if (tid == 0) a.count[first] = 0;
                for (int i = tid; i < heads() * (D / 4); i += kRowThreads) {
                    const int r = i / (D / 4), d = (i % (D / 4)) * 4;
                    // (one pass with a running maximum, the loads of eight contributors in flight)
                    float mm = -CUDART_INF_F, ll = 0.0f;
                    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    for (int c0 = first; c0 <= last; c0 += kJoinLoads) {
                        float mx[kJoinLoads], lx[kJoinLoads], top = mm;
                        float4 x[kJoinLoads];
#pragma unroll
                        for (int u = 0; u < kJoinLoads; ++u) {
                            const int c = min(c0 + u, last);
                            const float* p = a.partial + (static_cast<int64_t>(c) * 2 + (c == first)) * kRowSlotFloats;
                            mx[u] = __ldcg(p + 16 * 128 + r);
                            lx[u] = __ldcg(p + 16 * 128 + 16 + r);
                            x[u] = __ldcg(reinterpret_cast<const float4*>(p + r * D + d));
                        }
#pragma unroll
                        for (int u = 0; u < kJoinLoads; ++u) top = fmaxf(top, mx[u]);
                        const float safe = top == -CUDART_INF_F ? 0.0f : top;
                        const float f = exp2_approx(mm - safe);
                        mm = top;
                        ll *= f;
                        v = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
#pragma unroll
                        for (int u = 0; u < kJoinLoads; ++u) {
                            // past the last one, sums of 0 as well: a weight of 0 alone would make
                            // NaN of an infinite sum (and a branch here would hold up the loads)
                            const bool on = c0 + u <= last;
                            const float w = on ? exp2_approx(mx[u] - safe) : 0.0f;
                            ll += w * lx[u];
                            v.x += w * (on ? x[u].x : 0.0f);
                            v.y += w * (on ? x[u].y : 0.0f);
                            v.z += w * (on ? x[u].z : 0.0f);
                            v.w += w * (on ? x[u].w : 0.0f);
                        }
                    }
                    finish(r, d, v, mm, ll);
                }
            }
        }

        // the next segment
        segment_start += steps + kSegmentStart;
        if (++part == a.kv.Hkv * PASSES) {
            part = 0;
            if (++row < a.rows) {
                range = row_range(a, row);
                steps = steps_of(range);
            }
        }
    }
}

}  // namespace tpmlp
