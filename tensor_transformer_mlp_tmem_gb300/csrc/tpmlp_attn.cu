// Entry points of the attention over a paged cache (include/tpmlp.h): argument checks and
// launches. As in tpmlp_api.cu, every entry point returns a tpmlp_status and no C++ exception
// crosses this boundary.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstring>
#include <new>

#include "tpmlp_attn.cuh"
#include "tpmlp_attn_prompt.cuh"
#include "tpmlp_context.h"

using tpmlp::aligned16;
using tpmlp::check_device;

namespace {

constexpr int kRowCtasPerSm = 2;

bool is_e4m3(const tpmlp_ctx* c) { return (c->flags & TPMLP_FLAG_KV_E4M3) != 0; }

// Rows of `width` bf16 elements at pitch ld that 16-byte loads may read.
int check_rows(tpmlp_ctx* c, const void* p, int64_t ld, int64_t width) {
    if (!p) return TPMLP_ERR_INVALID_ARG;
    if (ld < width || ld > (int64_t(1) << 40)) {
        c->last_error = "a row pitch is smaller than its row";
        return TPMLP_ERR_INVALID_ARG;
    }
    if (!aligned16(p) || ld % 8) return TPMLP_ERR_MISALIGNED;
    return TPMLP_OK;
}

int check_kv(tpmlp_ctx* c, const tpmlp_kv* kv, bool lens) {
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

tpmlp::KvView view_of(const tpmlp_ctx* c, const tpmlp_kv* kv) {
    const int elem = is_e4m3(c) ? 1 : 2;
    const int64_t head = static_cast<int64_t>(c->page_size) * c->head_dim;
    tpmlp::KvView v{};
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

// Launch with programmatic stream serialisation (the kernels wait in griddep_wait before they
// touch global memory).
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
int allow_smem(tpmlp_ctx* c, Kernel kern, uint32_t smem, std::atomic<uint64_t>& done) {
    const uint64_t bit = uint64_t(1) << (c->device & 63);
    if (done.load(std::memory_order_acquire) & bit) return TPMLP_OK;
    TPMLP_CUDA(c, cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    done.fetch_or(bit, std::memory_order_acq_rel);
    return TPMLP_OK;
}

template <int D, bool FP8, int NT, int PASSES>
int launch_rows(tpmlp_ctx* c, const tpmlp::RowArgs& a, cudaStream_t s) {
    using S = tpmlp::RowShape<D, FP8, NT>;
    auto kern = tpmlp::attn_row_kernel<D, FP8, NT, PASSES>;
    static std::atomic<uint64_t> done{0};
    if (int rc = allow_smem(c, kern, S::kSmem, done)) return rc;
    const int grid = c->num_sms * S::kCtasPerSm;
    return launch(c, kern, grid, tpmlp::kRowThreads, S::kSmem, s, a);
}

template <int D, bool FP8>
int run_rows_of(tpmlp_ctx* c, const tpmlp::RowArgs& a, cudaStream_t s) {
    if constexpr (tpmlp::row_heads(D, FP8) > 16)
        if (a.G > 16) return launch_rows<D, FP8, 2, 2>(c, a, s);
    if constexpr (tpmlp::row_heads(D, FP8) > 8)
        if (a.G > 8) return launch_rows<D, FP8, 2, 1>(c, a, s);
    return launch_rows<D, FP8, 1, 1>(c, a, s);
}

int run_rows(tpmlp_ctx* c, const tpmlp::RowArgs& a, cudaStream_t s) {
    if (c->head_dim == 128) return is_e4m3(c) ? run_rows_of<128, true>(c, a, s) : run_rows_of<128, false>(c, a, s);
    return is_e4m3(c) ? run_rows_of<64, true>(c, a, s) : run_rows_of<64, false>(c, a, s);
}

template <int D, bool FP8>
int launch_prompt(tpmlp_ctx* c, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                  const tpmlp::PromptArgs& a, cudaStream_t s) {
    using S = tpmlp::PromptSmem<D, FP8>;
    auto kern = tpmlp::attn_prompt_kernel<D, FP8>;
    static std::atomic<uint64_t> done{0};
    if (int rc = allow_smem(c, kern, S::kTotal, done)) return rc;
    return launch(c, kern, c->num_sms, S::kThreads, S::kTotal, s, q, k, v, a);
}

// The pool as [page][Hkv * page size][D], in boxes of 64 columns and one page's (at most a
// block's) rows.
int pool_map(tpmlp_ctx* c, CUtensorMap* map, const void* pool, const tpmlp::KvView& kv) {
    const uint64_t dims[3] = {static_cast<uint64_t>(c->head_dim),
                              static_cast<uint64_t>(c->heads_kv) * c->page_size,
                              static_cast<uint64_t>(kv.num_pages)};
    const uint64_t strides[2] = {static_cast<uint64_t>(c->head_dim) * 2, static_cast<uint64_t>(kv.page_bytes)};
    const uint32_t box[3] = {64, static_cast<uint32_t>(std::min(c->page_size, tpmlp::kPB)), 1};
    return tpmlp::encode_map_typed(c, map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, pool, 3, dims, strides, box);
}

int run_prompt(tpmlp_ctx* c, const tpmlp::RowArgs& r, const int32_t* cu_q, int64_t T, cudaStream_t s) {
    tpmlp::PromptArgs a{};
    a.kv = r.kv;
    a.q = r.q;
    a.ldq = r.ldq;
    a.out = r.out;
    a.ldo = r.ldo;
    a.lse = r.lse;
    a.cu_q = cu_q;
    a.T = static_cast<int32_t>(T);
    a.Hq = r.Hq;
    a.G = r.G;
    a.tpt = tpmlp::kPB / r.G;
    a.scale_log2 = r.scale_log2;
    a.window = r.window;
    a.partial = c->attn_partial;
    a.count = c->attn_count;
    CUtensorMap q{}, k{}, v{};
    if (!is_e4m3(c)) {
        const uint64_t dims[3] = {static_cast<uint64_t>(c->head_dim), static_cast<uint64_t>(c->heads_q),
                                  static_cast<uint64_t>(T)};
        const uint64_t strides[2] = {static_cast<uint64_t>(c->head_dim) * 2, static_cast<uint64_t>(a.ldq) * 2};
        const uint32_t box[3] = {64, static_cast<uint32_t>(a.G), static_cast<uint32_t>(a.tpt)};
        int rc = tpmlp::encode_map_typed(c, &q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, 3, dims, strides, box);
        if (rc || (rc = pool_map(c, &k, a.kv.K, a.kv)) || (rc = pool_map(c, &v, a.kv.V, a.kv))) return rc;
    }
    if (c->head_dim == 128)
        return is_e4m3(c) ? launch_prompt<128, true>(c, q, k, v, a, s) : launch_prompt<128, false>(c, q, k, v, a, s);
    return is_e4m3(c) ? launch_prompt<64, true>(c, q, k, v, a, s) : launch_prompt<64, false>(c, q, k, v, a, s);
}

// Tokens of an append block: as many as its threads' units hold, but no fewer blocks than run at
// once. 16384 tokens of 12 + 12 heads of 64, 16 + 2 of 64, 8 + 1 of 128 in e4m3, 1 + 1 of 64: 30, 16, 23,
// 9 us (a block for each token: 37, 27, 34, 25).
int64_t append_tokens(const tpmlp_ctx* c, int64_t units, int64_t T) {
    const int64_t hold = tpmlp::kAppendThreads * tpmlp::kAppendUnits / units;
    const int64_t fill = T / (static_cast<int64_t>(tpmlp::kAppendBlocks) * c->num_sms);
    return std::max<int64_t>(1, std::min({hold, fill, static_cast<int64_t>(tpmlp::kAppendTokens)}));
}

template <int D, bool FP8>
int run_append(tpmlp_ctx* c, const tpmlp::AppendArgs& a, cudaStream_t s) {
    if (a.tokens > 1)
        return launch(c, tpmlp::append_kernel<D, FP8, true>, (a.T + int64_t(a.tokens) - 1) / a.tokens,
                      tpmlp::kAppendThreads, 0, s, a);
    return launch(c, tpmlp::append_kernel<D, FP8, false>, int64_t(a.T) * a.parts, tpmlp::kAppendThreads, 0, s, a);
}

// What decode and prompt check alike; rows: rows of Q and Out.
int check_attend(tpmlp_ctx* c, const void* Q, int64_t ldq, const tpmlp_kv* kv, float scale,
                 const void* Out, int64_t ldo, const float* Lse) {
    if (int rc = check_kv(c, kv, true)) return rc;
    if (!(scale > 0.0f) || !std::isfinite(scale)) return TPMLP_ERR_INVALID_ARG;
    const int64_t width = static_cast<int64_t>(c->heads_q) * c->head_dim;
    if (int rc = check_rows(c, Q, ldq, width)) return rc;
    if (int rc = check_rows(c, Out, ldo, width)) return rc;
    if (reinterpret_cast<uintptr_t>(Lse) & 3) return TPMLP_ERR_MISALIGNED;
    return TPMLP_OK;
}

tpmlp::RowArgs row_args(const tpmlp_ctx* c, const void* Q, int64_t ldq, const tpmlp_kv* kv,
                        float scale, int32_t window, void* Out, int64_t ldo, float* Lse) {
    tpmlp::RowArgs a{};
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

int check_attention(tpmlp_ctx* c) {
    if (!c || c->kind != kKindAttention) return TPMLP_ERR_INVALID_ARG;
    return check_device(c);
}

}  // namespace

extern "C" {

int tpmlp_attn_create(tpmlp_ctx** out, int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size,
                      uint32_t flags) {
    if (!out) return TPMLP_ERR_INVALID_ARG;
    *out = nullptr;
    if (Hq <= 0 || Hkv <= 0 || D <= 0 || page_size <= 0) return TPMLP_ERR_INVALID_ARG;
    if (flags & ~TPMLP_FLAG_KV_E4M3) return TPMLP_ERR_INVALID_ARG;
    if (Hq % Hkv || Hq / Hkv > 128 || Hq > (1 << 16) || (D != 64 && D != 128))
        return TPMLP_ERR_UNSUPPORTED_SHAPE;
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
        return TPMLP_ERR_UNSUPPORTED_SHAPE;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return TPMLP_ERR_CUDA;
    cudaDeviceProp prop;
    if (cudaGetDeviceProperties(&prop, dev) != cudaSuccess) return TPMLP_ERR_CUDA;
    if (prop.major != 10 || prop.minor != 3) return TPMLP_ERR_ARCH;
    tpmlp_ctx* c = new (std::nothrow) tpmlp_ctx();
    if (!c) return TPMLP_ERR_OOM;
    c->device = dev;
    c->num_sms = prop.multiProcessorCount;
    c->kind = kKindAttention;
    c->flags = flags;
    c->heads_q = Hq;
    c->heads_kv = Hkv;
    c->head_dim = D;
    c->page_size = page_size;
    const size_t ctas = static_cast<size_t>(c->num_sms) * kRowCtasPerSm;
    // two slots per CTA of either kernel (the prompt kernel's hold two tiles each)
    const size_t partial = std::max(ctas * 2 * tpmlp::kRowSlotFloats,
                                    static_cast<size_t>(c->num_sms) * 4 * tpmlp::kPromptSlotFloats);
    const size_t counters = ctas + 2;  // a counter per CTA (prompt: per tile), the deal's two
    c->attn_counters = counters;
    const size_t scales = static_cast<size_t>(Hkv) * 2;
    cudaError_t e;
    float* ones = new (std::nothrow) float[scales];
    if (!ones) {
        tpmlp_destroy(c);
        return TPMLP_ERR_OOM;
    }
    std::fill(ones, ones + scales, 1.0f);
    if ((e = cudaMalloc(&c->kv_scale, scales * sizeof(float))) != cudaSuccess ||
        (e = cudaMalloc(&c->attn_partial, partial * sizeof(float))) != cudaSuccess ||
        (e = cudaMalloc(&c->attn_count, counters * sizeof(uint32_t))) != cudaSuccess ||
        (e = cudaMalloc(&c->status, kStatusWords * sizeof(int))) != cudaSuccess ||
        (e = cudaMemset(c->attn_count, 0, counters * sizeof(uint32_t))) != cudaSuccess ||
        (e = cudaMemset(c->status, 0, kStatusWords * sizeof(int))) != cudaSuccess ||
        (e = cudaMemcpy(c->kv_scale, ones, scales * sizeof(float), cudaMemcpyHostToDevice)) != cudaSuccess ||
        // streams made without blocking do not wait for the default stream, where these run
        (e = cudaStreamSynchronize(nullptr)) != cudaSuccess) {
        delete[] ones;
        tpmlp_destroy(c);
        cudaGetLastError();
        return e == cudaErrorMemoryAllocation ? TPMLP_ERR_OOM : TPMLP_ERR_CUDA;
    }
    delete[] ones;
    *out = c;
    return TPMLP_OK;
}

int tpmlp_attn_set_rope(tpmlp_ctx* c, int32_t rot_dim, int32_t interleaved, const double* freq) {
    if (!c || c->kind != kKindAttention || rot_dim < 0 || (rot_dim > 0 && !freq)) return TPMLP_ERR_INVALID_ARG;
    if (interleaved != 0 && interleaved != 1) return TPMLP_ERR_INVALID_ARG;
    if (rot_dim % 16 || rot_dim > c->head_dim) return TPMLP_ERR_UNSUPPORTED_SHAPE;
    for (int i = 0; i < rot_dim / 2; ++i)
        if (!std::isfinite(freq[i])) return TPMLP_ERR_INVALID_ARG;
    for (int i = 0; i < rot_dim / 2; ++i) c->rope_turns[i] = freq[i] / 6.283185307179586476925;
    c->rot_dim = rot_dim;
    c->rope_interleaved = interleaved != 0;
    return TPMLP_OK;
}

int tpmlp_attn_set_scales(tpmlp_ctx* c, const void* k_scale, const void* v_scale, void* stream) {
    if (!c || c->kind != kKindAttention || !is_e4m3(c) || !k_scale || !v_scale) return TPMLP_ERR_INVALID_ARG;
    if (int rc = check_device(c)) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t n = static_cast<size_t>(c->heads_kv) * sizeof(float);
    TPMLP_CUDA(c, cudaMemcpyAsync(c->kv_scale, k_scale, n, cudaMemcpyDeviceToDevice, s));
    TPMLP_CUDA(c, cudaMemcpyAsync(c->kv_scale + c->heads_kv, v_scale, n, cudaMemcpyDeviceToDevice, s));
    return TPMLP_OK;
}

int tpmlp_attn_append(tpmlp_ctx* c, const void* Q, int64_t ldq, const void* K, int64_t ldk,
                      const void* V, int64_t ldv, int64_t T, const int32_t* pos,
                      const int32_t* seq, const tpmlp_kv* kv, void* Qout, int64_t ldqo,
                      void* stream) {
    if (int rc = check_attention(c)) return rc;
    if (T < 0) return TPMLP_ERR_INVALID_ARG;
    if (T == 0) return TPMLP_OK;
    if (T > INT_MAX) return TPMLP_ERR_UNSUPPORTED_SHAPE;
    if (int rc = check_kv(c, kv, false)) return rc;
    if (!pos || (Q != nullptr) != (Qout != nullptr)) return TPMLP_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(pos) | reinterpret_cast<uintptr_t>(seq)) & 3) return TPMLP_ERR_MISALIGNED;
    const int64_t wq = static_cast<int64_t>(c->heads_q) * c->head_dim;
    const int64_t wk = static_cast<int64_t>(c->heads_kv) * c->head_dim;
    int rc;
    if (Q && ((rc = check_rows(c, Q, ldq, wq)) || (rc = check_rows(c, Qout, ldqo, wq)))) return rc;
    if ((rc = check_rows(c, K, ldk, wk)) || (rc = check_rows(c, V, ldv, wk))) return rc;
    tpmlp::AppendArgs a{};
    a.kv = view_of(c, kv);
    a.q = static_cast<const __nv_bfloat16*>(Q);
    a.k = static_cast<const __nv_bfloat16*>(K);
    a.v = static_cast<const __nv_bfloat16*>(V);
    a.ldq = ldq;
    a.ldk = ldk;
    a.ldv = ldv;
    a.q_out = static_cast<__nv_bfloat16*>(Qout);
    a.ldqo = ldqo;
    a.pos = pos;
    a.seq = seq;
    a.Hq = Q ? c->heads_q : 0;
    a.rot = c->rot_dim;
    a.interleaved = c->rope_interleaved;
    std::memcpy(a.turns, c->rope_turns, sizeof(a.turns));
    // Parts of a token: as many blocks as run at once where there are few tokens, each thread with
    // a unit at least. One token of 32 + 32 heads of 128: 2.4 us (one block: 3.5 us); 256 tokens of 96
    // + 8 heads into e4m3: 4.5 us (two, four blocks an SM: 5.7, 4.8).
    const int64_t units = static_cast<int64_t>(a.Hq + 2 * c->heads_kv) * (c->head_dim / 16);
    const int64_t most = (units + tpmlp::kAppendThreads - 1) / tpmlp::kAppendThreads;
    a.parts = static_cast<int32_t>(std::min(most, std::max<int64_t>(1, tpmlp::kAppendBlocks * c->num_sms / T)));
    a.part_units = static_cast<int32_t>((units + a.parts - 1) / a.parts);
    a.T = static_cast<int32_t>(T);
    a.tokens = static_cast<int32_t>(append_tokens(c, units, T));
    a.per_unit = static_cast<uint32_t>((uint64_t(1) << 32) / units + 1);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (c->head_dim == 128) return is_e4m3(c) ? run_append<128, true>(c, a, s) : run_append<128, false>(c, a, s);
    return is_e4m3(c) ? run_append<64, true>(c, a, s) : run_append<64, false>(c, a, s);
}

int tpmlp_attn_decode(tpmlp_ctx* c, const void* Q, int64_t ldq, const tpmlp_kv* kv, float scale,
                      int32_t window, void* Out, int64_t ldo, float* Lse, void* stream) {
    if (int rc = check_attention(c)) return rc;
    if (!kv) return TPMLP_ERR_INVALID_ARG;
    if (kv->B == 0) return TPMLP_OK;
    if (int rc = check_attend(c, Q, ldq, kv, scale, Out, ldo, Lse)) return rc;
    tpmlp::RowArgs a = row_args(c, Q, ldq, kv, scale, window, Out, ldo, Lse);
    a.rows = kv->B;
    if (a.G > tpmlp::row_heads(c->head_dim, is_e4m3(c)))
        return run_prompt(c, a, nullptr, kv->B, static_cast<cudaStream_t>(stream));
    return run_rows(c, a, static_cast<cudaStream_t>(stream));
}

int tpmlp_attn_prompt(tpmlp_ctx* c, const void* Q, int64_t ldq, int64_t T, const int32_t* cu_q,
                      const tpmlp_kv* kv, float scale, int32_t window, void* Out, int64_t ldo,
                      float* Lse, void* stream) {
    if (int rc = check_attention(c)) return rc;
    if (!kv || T < 0) return TPMLP_ERR_INVALID_ARG;
    if (T == 0 || kv->B == 0) return TPMLP_OK;
    if (T > INT_MAX / 2) return TPMLP_ERR_UNSUPPORTED_SHAPE;
    if (int rc = check_attend(c, Q, ldq, kv, scale, Out, ldo, Lse)) return rc;
    if (!cu_q) return TPMLP_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(cu_q) & 3) return TPMLP_ERR_MISALIGNED;
    const tpmlp::RowArgs a = row_args(c, Q, ldq, kv, scale, window, Out, ldo, Lse);
    return run_prompt(c, a, cu_q, T, static_cast<cudaStream_t>(stream));
}

int tpmlp_attn_append_packed(const tpmlp_append_args* a) {
    if (!a) return TPMLP_ERR_INVALID_ARG;
    return tpmlp_attn_append(a->ctx, a->Q, a->ldq, a->K, a->ldk, a->V, a->ldv, a->T, a->pos, a->seq, a->kv, a->Qout,
                             a->ldqo, a->stream);
}

int tpmlp_attn_decode_packed(const tpmlp_attend_args* a) {
    if (!a || a->window > INT_MAX || a->window < INT_MIN) return TPMLP_ERR_INVALID_ARG;
    return tpmlp_attn_decode(a->ctx, a->Q, a->ldq, a->kv, static_cast<float>(a->scale),
                             static_cast<int32_t>(a->window), a->Out, a->ldo, a->Lse, a->stream);
}

int tpmlp_attn_prompt_packed(const tpmlp_attend_args* a) {
    if (!a || a->window > INT_MAX || a->window < INT_MIN) return TPMLP_ERR_INVALID_ARG;
    return tpmlp_attn_prompt(a->ctx, a->Q, a->ldq, a->T, a->cu_q, a->kv, static_cast<float>(a->scale),
                             static_cast<int32_t>(a->window), a->Out, a->ldo, a->Lse, a->stream);
}

}  // extern "C"

#ifdef TPMLP_TEST_HOOKS
// Test builds only: an attention context that holds no device memory (tpmlp_test_host_context).
extern "C" TPMLP_API tpmlp_ctx* tpmlp_test_attn_context(int32_t Hq, int32_t Hkv, int32_t D,
                                                        int32_t page_size, int32_t device,
                                                        uint32_t flags) {
    tpmlp_ctx* c = new (std::nothrow) tpmlp_ctx();
    if (!c) return nullptr;
    c->kind = kKindAttention;
    c->flags = flags;
    c->device = device;
    c->num_sms = 152;
    c->heads_q = Hq;
    c->heads_kv = Hkv;
    c->head_dim = D;
    c->page_size = page_size;
    return c;
}

// Test builds only: whether decode of G heads to a kv head takes the row kernel.
extern "C" TPMLP_API int tpmlp_test_decode_on_rows(int32_t G, int32_t D, uint32_t flags) {
    return G <= tpmlp::row_heads(D, (flags & TPMLP_FLAG_KV_E4M3) != 0);
}
#endif
