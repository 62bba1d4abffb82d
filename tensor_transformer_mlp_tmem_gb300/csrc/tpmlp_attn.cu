// Entry points of the attention over a paged cache (include/tpmlp.h): argument checks and
// launches. As in tpmlp_api.cu, every entry point returns a tpmlp_status and no C++ exception
// crosses this boundary.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <new>

#include "tpmlp_attn_launch.h"

using namespace tpmlp;

namespace {

constexpr int kRowCtasPerSm = 2;

template <int D, bool FP8>
int launch_prompt(tpmlp_ctx* c, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                  const PromptArgs& a, cudaStream_t s) {
    using S = PromptSmem<D, FP8>;
    auto kern = attn_prompt_kernel<D, FP8>;
    static std::atomic<uint64_t> done{0};
    if (int rc = allow_smem(c, kern, S::kTotal, done)) return rc;
    return launch(c, kern, c->num_sms, S::kThreads, S::kTotal, s, q, k, v, a);
}

int run_prompt(tpmlp_ctx* c, const RowArgs& r, const int32_t* cu_q, int64_t T, cudaStream_t s) {
    PromptArgs a{};
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
    a.tpt = kPB / r.G;
    a.scale_log2 = r.scale_log2;
    a.window = r.window;
    a.partial = c->attn_partial;
    a.count = c->attn_count;
    CUtensorMap q{}, k{}, v{};
    if (int rc = prompt_maps(c, r, T, a.tpt, &q, &k, &v)) return rc;
    if (c->head_dim == 128)
        return is_e4m3(c) ? launch_prompt<128, true>(c, q, k, v, a, s) : launch_prompt<128, false>(c, q, k, v, a, s);
    return is_e4m3(c) ? launch_prompt<64, true>(c, q, k, v, a, s) : launch_prompt<64, false>(c, q, k, v, a, s);
}

// Tokens of an append block: as many as its threads' units hold, but no fewer blocks than run at
// once. 16384 tokens of 12 + 12 heads of 64, 16 + 2 of 64, 8 + 1 of 128 in e4m3, 1 + 1 of 64: 30, 16, 23,
// 9 us (a block for each token: 37, 27, 34, 25).
int64_t append_tokens(const tpmlp_ctx* c, int64_t units, int64_t T) {
    const int64_t hold = kAppendThreads * kAppendUnits / units;
    const int64_t fill = T / (static_cast<int64_t>(kAppendBlocks) * c->num_sms);
    return std::max<int64_t>(1, std::min({hold, fill, static_cast<int64_t>(kAppendTokens)}));
}

// Where the norms' weights of either kind lie.
struct NormWeights {
    uint16_t *q, *k;
};
NormWeights norm_weights(const tpmlp_ctx* c, bool per_head) {
    const int64_t D = c->head_dim;
    if (per_head) return {c->norm_w, c->norm_w + c->heads_q * D};
    uint16_t* const shared = c->norm_w + (static_cast<int64_t>(c->heads_q) + c->heads_kv) * D;
    return {shared, shared + D};
}

template <int D, bool FP8, int NORM>
int launch_append(tpmlp_ctx* c, const AppendArgs& a, cudaStream_t s) {
    if (a.tokens > 1)
        return launch(c, append_kernel<D, FP8, true, NORM>, (a.T + int64_t(a.tokens) - 1) / a.tokens,
                      kAppendThreads, 0, s, a);
    return launch(c, append_kernel<D, FP8, false, NORM>, int64_t(a.T) * a.parts, kAppendThreads, 0, s, a);
}

template <int D, bool FP8>
int run_append(tpmlp_ctx* c, const AppendArgs& a, cudaStream_t s) {
    if (!c->norm_on) return launch_append<D, FP8, kNormNone>(c, a, s);
    return c->norm_per_head ? launch_append<D, FP8, kNormHeads>(c, a, s) : launch_append<D, FP8, kNormShared>(c, a, s);
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
    const size_t partial = std::max(ctas * 2 * kRowSlotFloats,
                                    static_cast<size_t>(c->num_sms) * 4 * kPromptSlotFloats);
    // (cross attention's results that are joined apart)
    const size_t behind = static_cast<size_t>(cross_part_heads(c)) * (D * sizeof(float) + sizeof(RowOf));
    const size_t counters = ctas + 2;  // a counter per CTA (prompt: per tile), the deal's two
    c->attn_counters = counters;
    c->attn_partial_floats = partial;
    const size_t scales = static_cast<size_t>(Hkv) * 2;
    cudaError_t e;
    float* ones = new (std::nothrow) float[scales];
    if (!ones) {
        tpmlp_destroy(c);
        return TPMLP_ERR_OOM;
    }
    std::fill(ones, ones + scales, 1.0f);
    if ((e = cudaMalloc(&c->kv_scale, scales * sizeof(float))) != cudaSuccess ||
        (e = cudaMalloc(&c->attn_partial, partial * sizeof(float) + behind)) != cudaSuccess ||
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

int tpmlp_attn_set_norms(tpmlp_ctx* c, const void* q_weight, const void* k_weight, int32_t per_head,
                         float eps, void* stream) {
    if (!c || c->kind != kKindAttention || (q_weight != nullptr) != (k_weight != nullptr))
        return TPMLP_ERR_INVALID_ARG;
    if (!q_weight) {
        c->norm_on = false;
        return TPMLP_OK;
    }
    if (per_head != 0 && per_head != 1) return TPMLP_ERR_INVALID_ARG;
    if (!(eps >= 0x1p-40f && eps <= 1.0f)) return TPMLP_ERR_INVALID_ARG;
    if (int rc = check_device(c)) return rc;
    if (!aligned16(q_weight) || !aligned16(k_weight)) return TPMLP_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // Weights per head and shared ones have places of their own, so that a captured append finds its kind's.
    const size_t head = static_cast<size_t>(c->head_dim) * sizeof(uint16_t);
    if (!c->norm_w) {
        if (int rc = refuse_allocation(c, s, "tpmlp_attn_set_norms before the capture")) return rc;
        if (int rc = allocate(c, reinterpret_cast<void**>(&c->norm_w), (c->heads_q + c->heads_kv + 2) * head)) return rc;
    }
    const size_t nq = per_head ? c->heads_q : 1, nk = per_head ? c->heads_kv : 1;
    const NormWeights to = norm_weights(c, per_head != 0);
    TPMLP_CUDA(c, cudaMemcpyAsync(to.q, q_weight, nq * head, cudaMemcpyDeviceToDevice, s));
    TPMLP_CUDA(c, cudaMemcpyAsync(to.k, k_weight, nk * head, cudaMemcpyDeviceToDevice, s));
    c->norm_on = true;
    c->norm_per_head = per_head != 0;
    c->norm_eps = eps;
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
    AppendArgs a{};
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
    const int64_t most = (units + kAppendThreads - 1) / kAppendThreads;
    a.parts = static_cast<int32_t>(std::min(most, std::max<int64_t>(1, kAppendBlocks * c->num_sms / T)));
    a.part_units = static_cast<int32_t>((units + a.parts - 1) / a.parts);
    if (c->norm_on) {
        // whole heads to a block: their units' threads add up the squares
        const int32_t per_head = c->head_dim / 16;
        a.part_units = (a.part_units + per_head - 1) / per_head * per_head;
        a.parts = static_cast<int32_t>((units + a.part_units - 1) / a.part_units);
        const NormWeights w = norm_weights(c, c->norm_per_head);
        a.wq = reinterpret_cast<const __nv_bfloat16*>(w.q);
        a.wk = reinterpret_cast<const __nv_bfloat16*>(w.k);
        a.eps = c->norm_eps;
    }
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
    RowArgs a = row_args(c, Q, ldq, kv, scale, window, Out, ldo, Lse);
    a.rows = kv->B;
    if (a.G > row_heads(c->head_dim, is_e4m3(c)))
        return run_prompt(c, a, nullptr, kv->B, static_cast<cudaStream_t>(stream));
    return run_rows<kRowsDecode>(c, a, static_cast<cudaStream_t>(stream), a.G);
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
    const RowArgs a = row_args(c, Q, ldq, kv, scale, window, Out, ldo, Lse);
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
    return G <= row_heads(D, (flags & TPMLP_FLAG_KV_E4M3) != 0);
}
#endif
