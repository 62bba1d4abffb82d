// The context behind every entry point and the helpers that the translation units share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <string>

#include "tpmlp.h"
#include "tpmlp_plan.h"

// Row chunks of tpmlp_forward_host's pipeline at most (sizes the context's event arrays).
#ifndef TPMLP_HOST_CHUNKS_MAX
#define TPMLP_HOST_CHUNKS_MAX 4
#endif
static_assert(TPMLP_HOST_CHUNKS_MAX >= 1 && TPMLP_HOST_CHUNKS_MAX <= 16, "host chunk limit");

// tpmlp_ctx::kind
constexpr int kKindBlock = 0, kKindColumn = 1, kKindRow = 2, kKindAttention = 3;

struct tpmlp_ctx {
    int device = -1;
    int num_sms = 0;
    int64_t H = 0, F = 0, f = 0;
    int32_t k = 0;
    uint32_t flags = 0;
    int bn1 = 0, bn2 = 0;  // output tile widths of GEMM1 / GEMM2

    uint16_t* W1p = nullptr;  // [k][f][H]  (gated: [k][2f][H])
    uint16_t* W2p = nullptr;  // [k][H][f]
    float* b1 = nullptr;      // [F]        (gated: [2F])
    float* b2 = nullptr;      // [H]
    bool packed = false;
    CUtensorMap tmW1{}, tmW2{};            // B boxes for the single-SM kernel (BN rows)
    CUtensorMap tmW1_pair{}, tmW2_pair{};  // B boxes for the CTA-pair kernel (128 rows)
    bool pair1 = false, pair2 = false;     // GEMM1 / GEMM2 run on CTA pairs
    int kind = 0;        // kKindBlock, ...
    bool gated = false;  // SwiGLU block: W1p holds gate and up rows interleaved
    int gate_block = 0;  // G: gate/up interleave block (output columns per half-tile)

    uint16_t* Y = nullptr;  // [y_rows][F] intermediate activations
    int64_t y_rows = 0;
    void* Xs = nullptr;  // staging for tpmlp_forward_host
    void* Zs = nullptr;
    int64_t stage_rows = 0;
    cudaStream_t s_in = nullptr, s_out = nullptr;  // its copy streams (created on first use)
    cudaEvent_t host_ev[TPMLP_HOST_CHUNKS_MAX + 1] = {}, in_ev[TPMLP_HOST_CHUNKS_MAX] = {},
                out_ev[TPMLP_HOST_CHUNKS_MAX] = {};
    // row chunks of the last tpmlp_forward_host call (re-planned when M changes)
    int64_t plan_M = -1;
    int plan_n = 0;
    int64_t plan_rows[TPMLP_HOST_CHUNKS_MAX] = {};
    // tpmlp_forward_host_async: two staging slots used in turn, so that a call's copies in and
    // out overlap the kernels of the calls before and after it
    void* Xa[2] = {};
    void* Za[2] = {};
    int64_t async_rows = 0;
    cudaEvent_t a_in[2] = {}, a_xfree[2] = {}, a_zready[2] = {}, a_zfree[2] = {};
    bool a_used[2] = {};
    uint32_t a_calls = 0;

    // activation tensor maps of the last call (re-encoded only when pointer or rows change)
    const void* x_map_ptr = nullptr;
    int64_t x_map_rows = -1;
    CUtensorMap tmX{};
    const void* y_map_ptr = nullptr;
    int64_t y_map_rows = -1;
    CUtensorMap tmY{};

    // LayerNorm in front of the block (tpmlp_set_layernorm / tpmlp_block_forward)
    float* ln_gamma = nullptr;  // [H] fp32
    float* ln_beta = nullptr;   // [H] fp32
    float ln_eps = 0.0f;
    bool ln_set = false;
    uint16_t* Xn = nullptr;  // [xn_rows][H] normalised block input
    int64_t xn_rows = 0;

    // backward pass
    float* zeros = nullptr;        // [max(H, F)] fp32 zeros: the "no bias" of dX
    float* colsum = nullptr;       // partial column sums for the bias gradients
    int64_t colsum_floats = 0;
    uint16_t* dgu = nullptr;       // gated backward: dG and dU, [rows][2F] bf16
    int64_t dgu_elems = 0;

    // split reduction of the last tiles on CTA pairs (absent with TPMLP_FLAG_FIXED_ORDER)
    float* sk_partial = nullptr;  // [num_sms / 2 pairs][2 units][2 CTAs][128 x 256] fp32 partials
    uint32_t* sk_count = nullptr; // [num_sms split tiles][2 CTAs][epilogue warps] arrivals
    uint32_t sk_epoch = 0;

    tpmlp::DeviceRates rates{};  // the planners' rates (device_rates, or tpmlp_set_device_rates)
    // row group of the tall units' sweep, for the last (512-row blocks, column blocks, pairs)
    int tall_group = 8, tall_group_m = -1, tall_group_n = -1, tall_group_pairs = -1;

    // attention over a paged cache (kKindAttention; tpmlp_attn.cu)
    int32_t heads_q = 0, heads_kv = 0, head_dim = 0, page_size = 0;
    int32_t rot_dim = 0;             // rotated leading dimensions of each head (0: no rotation)
    bool rope_interleaved = false;   // pairs are neighbours instead of halves
    double rope_turns[64] = {};      // whole turns per position of each rotated pair
    float* kv_scale = nullptr;       // [2][heads_kv] fp32: the k scales, then the v scales
    float* attn_partial = nullptr;   // partial sums of split key ranges (tpmlp_attn.cuh)
    uint32_t* attn_count = nullptr;  // arrivals at a split key range, one counter per CTA
    size_t attn_counters = 0;        // entries of attn_count
    // tpmlp_attn_set_norms, bf16: weights per head [heads_q + heads_kv][head_dim], then shared ones [2][head_dim]
    uint16_t* norm_w = nullptr;
    bool norm_on = false, norm_per_head = false;
    float norm_eps = 0.0f;
    size_t attn_partial_floats = 0;  // values of attn_partial
    // tpmlp_attn_decode_shared: results over prefixes (tpmlp_attn_open.cu) of shared_rows sequences.
    // Captured graphs hold a buffer's address, so the smaller ones before the last stay until the context
    // goes; each is at least twice the one before. tail_partial: a second attn_partial.
    float* tail_partial = nullptr;
    uint32_t* tail_count = nullptr;  // behind tail_partial
    float* shared[40] = {};
    int shared_n = 0;
    int64_t shared_rows = 0;

    int* status = nullptr;  // device status: kStatusWords
    int64_t launches = 0;
    std::string last_error;
};

// The device status: word 0 names the first wait that gave up, word kBadPageWord is 1 after a bad
// entry of a page table. Each is recorded whatever the other holds. tpmlp_get_status hands them out
// as one number, word 0 with the bit kStatusBadPage.
constexpr int kStatusWords = 2, kBadPageWord = 1;
constexpr int kStatusBadPage = 0x10000;

namespace tpmlp {

int fail_cuda(tpmlp_ctx* c, cudaError_t e, const char* what);
int check_device(tpmlp_ctx* c);  // the context's device is current, or INVALID_ARG
int get_encoder(tpmlp_ctx* c);   // looks up cuTensorMapEncodeTiled once
// A tensor map with the 128-byte swizzle: dims and box innermost first, strides in bytes for
// dims 1..rank-1.
int encode_map_typed(tpmlp_ctx* c, CUtensorMap* map, CUtensorMapDataType type, const void* ptr,
                     int rank, const uint64_t* dims, const uint64_t* strides,
                     const uint32_t* box);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace tpmlp

#define TPMLP_CUDA(ctx, call)                                           \
    do {                                                                \
        cudaError_t e_ = (call);                                        \
        if (e_ != cudaSuccess) return tpmlp::fail_cuda(ctx, e_, #call); \
    } while (0)
