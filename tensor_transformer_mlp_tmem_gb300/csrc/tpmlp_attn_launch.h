// Argument checks and launches that the attention entry points share (tpmlp_attn.cu,
// tpmlp_attn_open.cu).
#pragma once

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <string>

#include "tpmlp_attn.cuh"
#include "tpmlp_attn_prompt.cuh"
#include "tpmlp_context.h"

namespace tpmlp {

inline bool is_e4m3(const tpmlp_ctx* c) { return (c->flags & TPMLP_FLAG_KV_E4M3) != 0; }

// Items of cross attention that about so many SMs or more share leave their parts to a join of its own, by
// all SMs, where a sequence's table has room for so many keys (its length is on the device: short ones
// behind wide tables pay the launch, 2 x 100 rows on 577 keys x 16 heads of 64 14.2 us, 11.3 without). With
// and without, us, at so many SMs to an item:
//   D = 128, bf16: 4: 2 x 300 rows on 9000 keys x 12 heads 59.2, 59.5, 1 x 256 on 4096 x 32 39.0, 38.2;
//     6: 1 x 256 on 2304 x 24 28.8, 31.9; 19: 1 x 256 on 4096 x 8 24.7, 41.1
//   D = 128, e4m3: 4: the first 74.4, 75.6, the second 45.2, 46.9; 6: 34.0, 39.2; 19: 27.0, 48.0
//   D = 64, bf16: 4: 2 x 300 on 9000 x 12 43.4, 43.8, 1 x 40 on 16384 x 32 45.1, 45.1; 6: 3 x 200 on 5000 x 8
//     25.3, 26.0; 9: 1 x 256 on 4096 x 16 19.6, 22.7; 76: 64 x 8 heads on 30000 keys of one kv head 27.7, 45.4
//   D = 64, e4m3: 4: the first 54.6, 52.5, the second 58.0, 52.9; 6: 34.4, 30.1; 9: 25.6, 28.2; 12: 1 x 40 on
//     4096 x 12 18.4, 17.9, 2 x 200 on 4096 x 6 20.6, 23.5; 76: 40.3, 58.3
inline int join_apart(const tpmlp_ctx* c) { return c->head_dim == 64 && is_e4m3(c) ? 9 : 4; }
constexpr int kJoinApartKeys = 2048;
// Rows x heads of such a call at most: two tiles to an item, and an item to join_apart SMs.
inline int64_t cross_part_heads(const tpmlp_ctx* c) {
    return static_cast<int64_t>(c->num_sms) / join_apart(c) * 2 * kPB;
}

// Rows of `width` bf16 elements at pitch ld that 16-byte loads may read.
inline int check_rows(tpmlp_ctx* c, const void* p, int64_t ld, int64_t width) {
    if (!p) return TPMLP_ERR_INVALID_ARG;
    if (ld < width || ld > (int64_t(1) << 40)) {
        c->last_error = "a row pitch is smaller than its row";
        return TPMLP_ERR_INVALID_ARG;
    }
    if (!aligned16(p) || ld % 8) return TPMLP_ERR_MISALIGNED;
    return TPMLP_OK;
}

inline int check_kv(tpmlp_ctx* c, const tpmlp_kv* kv, bool lens) {
    if (!kv || !kv->K || !kv->V || !kv->page_table || (lens && !kv->lens)) return TPMLP_ERR_INVALID_ARG;
    if (kv->num_pages <= 0 || kv->table_pages <= 0 || kv->B < 0) return TPMLP_ERR_INVALID_ARG;
    if (kv->num_pages > INT_MAX) return TPMLP_ERR_UNSUPPORTED_SHAPE;
    if (kv->table_stride != 0 && kv->table_stride < kv->table_pages) return TPMLP_ERR_INVALID_ARG;
    const int64_t page = static_cast<int64_t>(c->heads_kv) * c->page_size * c->head_dim;
    if (kv->page_stride != 0 && kv->page_stride < page) return TPMLP_ERR_INVALID_ARG;
    // key numbers stay below 2^31 with a step of every kernel past the end
    if (static_cast<int64_t>(kv->table_pages) * c->page_size > (int64_t(1) << 31) - (1 << 16)) {
        c->last_error = "a sequence's table holds more than 2^31 - 2^16 keys";
        return TPMLP_ERR_UNSUPPORTED_SHAPE;
    }
    const int elem = is_e4m3(c) ? 1 : 2;
    if (!aligned16(kv->K) || !aligned16(kv->V) || kv->page_stride * elem % 16) return TPMLP_ERR_MISALIGNED;
    if ((reinterpret_cast<uintptr_t>(kv->page_table) | reinterpret_cast<uintptr_t>(kv->lens)) & 3)
        return TPMLP_ERR_MISALIGNED;
    return TPMLP_OK;
}

inline KvView view_of(const tpmlp_ctx* c, const tpmlp_kv* kv) {
    const int elem = is_e4m3(c) ? 1 : 2;
    const int64_t head = static_cast<int64_t>(c->page_size) * c->head_dim;
    KvView v{};
    v.K = static_cast<uint8_t*>(kv->K);
    v.V = static_cast<uint8_t*>(kv->V);
    v.page_bytes = (kv->page_stride ? kv->page_stride : head * c->heads_kv) * elem;
    v.head_bytes = head * elem;
    v.table = kv->page_table;
    v.table_stride = kv->table_stride ? kv->table_stride : kv->table_pages;
    v.table_pages = kv->table_pages;
    while ((1 << v.page_shift) < c->page_size) ++v.page_shift;
    v.num_pages = static_cast<int32_t>(kv->num_pages);
    v.lens = kv->lens;
    v.B = kv->B;
    v.Hkv = c->heads_kv;
    v.scales = c->kv_scale;
    v.status = c->status;
    return v;
}

// What a call that would have to allocate answers while its stream is being captured (`first`: the
// call to be made before the capture).
inline int refuse_allocation(tpmlp_ctx* c, cudaStream_t s, const char* first) {
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    TPMLP_CUDA(c, cudaStreamIsCapturing(s, &st));
    if (st == cudaStreamCaptureStatusNone) return TPMLP_OK;
    c->last_error = std::string("no allocation under stream capture: call ") + first;
    return TPMLP_ERR_INVALID_ARG;
}

inline int allocate(tpmlp_ctx* c, void** p, size_t bytes) {
    const cudaError_t e = cudaMalloc(p, bytes);
    if (e == cudaSuccess) return TPMLP_OK;
    *p = nullptr;
    if (e != cudaErrorMemoryAllocation) return fail_cuda(c, e, "cudaMalloc");
    cudaGetLastError();
    return TPMLP_ERR_OOM;
}

// Launch with programmatic stream serialisation. The kernels wait in griddep_wait before they touch global
// memory, but for two that come behind another launch of their own call, whose CTAs let them start only
// after a griddep_wait of theirs: the row kernel of kRowsPart (behind run_all_keys), and the tile kernel's
// look at cu_q (behind the row kernel).
template <typename Kernel, typename... Args>
int launch(tpmlp_ctx* c, Kernel kern, int64_t grid, int threads, uint32_t smem, cudaStream_t s,
           const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    TPMLP_CUDA(c, cudaLaunchKernelEx(&cfg, kern, args...));
    ++c->launches;
    return TPMLP_OK;
}

template <typename Kernel>
int allow_smem(tpmlp_ctx* c, Kernel kern, uint32_t smem, std::atomic<uint64_t>& done, int carveout = -1) {
    const uint64_t bit = uint64_t(1) << (c->device & 63);
    if (done.load(std::memory_order_acquire) & bit) return TPMLP_OK;
    TPMLP_CUDA(c, cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    if (carveout >= 0)
        TPMLP_CUDA(c, cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, carveout));
    done.fetch_or(bit, std::memory_order_acq_rel);
    return TPMLP_OK;
}

template <int D, bool FP8, int NT, int PASSES, int MODE>
int launch_rows(tpmlp_ctx* c, const RowArgs& a, cudaStream_t s) {
    using S = RowShape<D, FP8, NT, row_warps(MODE)>;
    auto kern = attn_row_kernel<D, FP8, NT, PASSES, MODE>;
    static std::atomic<uint64_t> done{0};
    // Loads in flight lie in what shared memory leaves of an SM's 256 KB. Without this an SM keeps the split
    // of the launch before it while that has room enough: behind a prompt kernel 28 KB of loads, and 64
    // sequences of at most 1024 keys x 32 heads take 150 us instead of 98.
    constexpr int kCarveout = static_cast<int>((S::kCtasPerSm * (S::kSmem + 2048) * 100 + 233471) / 233472);
    if (int rc = allow_smem(c, kern, S::kSmem, done, kCarveout)) return rc;
    const int grid = c->num_sms * S::kCtasPerSm;
    return launch(c, kern, grid, S::kThreads, S::kSmem, s, a);
}

template <int D, bool FP8, int MODE>
int run_rows_of(tpmlp_ctx* c, const RowArgs& a, cudaStream_t s, int64_t heads) {
    if constexpr (row_heads(D, FP8) > 16 && MODE < kRowsCross)
        if (heads > 16) return launch_rows<D, FP8, 2, 2, MODE>(c, a, s);
    if constexpr (row_heads(D, FP8) > 8)
        if (heads > 8) return launch_rows<D, FP8, 2, 1, MODE>(c, a, s);
    return launch_rows<D, FP8, 1, 1, MODE>(c, a, s);
}

// heads: query heads to a kv head (kRowsCross, kRowsCrossPart: of a sequence's rows, about).
template <int MODE>
int run_rows(tpmlp_ctx* c, const RowArgs& a, cudaStream_t s, int64_t heads) {
    if (c->head_dim == 128) return is_e4m3(c) ? run_rows_of<128, true, MODE>(c, a, s, heads) : run_rows_of<128, false, MODE>(c, a, s, heads);
    return is_e4m3(c) ? run_rows_of<64, true, MODE>(c, a, s, heads) : run_rows_of<64, false, MODE>(c, a, s, heads);
}

// The pool as [page][Hkv * page size][D], in boxes of 64 columns and one page's (at most a
// block's) rows.
inline int pool_map(tpmlp_ctx* c, CUtensorMap* map, const void* pool, const KvView& kv) {
    const uint64_t dims[3] = {static_cast<uint64_t>(c->head_dim),
                              static_cast<uint64_t>(c->heads_kv) * c->page_size,
                              static_cast<uint64_t>(kv.num_pages)};
    const uint64_t strides[2] = {static_cast<uint64_t>(c->head_dim) * 2, static_cast<uint64_t>(kv.page_bytes)};
    const uint32_t box[3] = {64, static_cast<uint32_t>(std::min(c->page_size, kPB)), 1};
    return encode_map_typed(c, map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, pool, 3, dims, strides, box);
}

// The tensor maps of a bf16 cache's pools and of T rows of queries in boxes of G heads x `tokens`.
inline int prompt_maps(tpmlp_ctx* c, const RowArgs& r, int64_t T, int tokens, CUtensorMap* q, CUtensorMap* k,
                       CUtensorMap* v) {
    if (is_e4m3(c)) return TPMLP_OK;
    const uint64_t dims[3] = {static_cast<uint64_t>(c->head_dim), static_cast<uint64_t>(c->heads_q),
                              static_cast<uint64_t>(T)};
    const uint64_t strides[2] = {static_cast<uint64_t>(c->head_dim) * 2, static_cast<uint64_t>(r.ldq) * 2};
    const uint32_t box[3] = {64, static_cast<uint32_t>(r.G), static_cast<uint32_t>(tokens)};
    if (int rc = encode_map_typed(c, q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, r.q, 3, dims, strides, box)) return rc;
    if (int rc = pool_map(c, k, r.kv.K, r.kv)) return rc;
    return pool_map(c, v, r.kv.V, r.kv);
}

// What decode and prompt check alike; rows: rows of Q and Out.
inline int check_attend(tpmlp_ctx* c, const void* Q, int64_t ldq, const tpmlp_kv* kv, float scale,
                 const void* Out, int64_t ldo, const float* Lse) {
    if (int rc = check_kv(c, kv, true)) return rc;
    if (!(scale > 0.0f) || !std::isfinite(scale)) return TPMLP_ERR_INVALID_ARG;
    const int64_t width = static_cast<int64_t>(c->heads_q) * c->head_dim;
    if (int rc = check_rows(c, Q, ldq, width)) return rc;
    if (int rc = check_rows(c, Out, ldo, width)) return rc;
    if (reinterpret_cast<uintptr_t>(Lse) & 3) return TPMLP_ERR_MISALIGNED;
    return TPMLP_OK;
}

inline RowArgs row_args(const tpmlp_ctx* c, const void* Q, int64_t ldq, const tpmlp_kv* kv,
                        float scale, int32_t window, void* Out, int64_t ldo, float* Lse) {
    RowArgs a{};
    a.kv = view_of(c, kv);
    a.q = static_cast<const __nv_bfloat16*>(Q);
    a.ldq = ldq;
    a.out = static_cast<__nv_bfloat16*>(Out);
    a.ldo = ldo;
    a.lse = Lse;
    a.Hq = c->heads_q;
    a.G = c->heads_q / c->heads_kv;
    a.scale_log2 = scale * 1.44269504088896341f;
    a.window = window;
    a.partial = c->attn_partial;
    a.count = c->attn_count;
    return a;
}

inline int check_attention(tpmlp_ctx* c) {
    if (!c || c->kind != kKindAttention) return TPMLP_ERR_INVALID_ARG;
    return check_device(c);
}

}  // namespace tpmlp
