// Entry points of attention without a causal mask (include/tpmlp.h): to all keys of another sequence,
// and of one token of each sequence to a prefix that several share and to its own keys. In a
// translation unit of its own: its kernels compile beside those of tpmlp_attn.cu.
#include <climits>

#include "tpmlp_attn_launch.h"
#include "tpmlp_attn_open.cuh"

using namespace tpmlp;

namespace {

template <int D, bool FP8>
int launch_open(tpmlp_ctx* c, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                const OpenArgs& a, cudaStream_t s) {
    using S = OpenShape<D, FP8>;
    auto kern = attn_open_kernel<D, FP8>;
    static std::atomic<uint64_t> done{0};
    if (int rc = allow_smem(c, kern, S::kTotal, done)) return rc;
    return launch(c, kern, c->num_sms, S::kThreads, S::kTotal, s, q, k, v, a);
}

int run_open(tpmlp_ctx* c, const RowArgs& r, const int32_t* cu_q, int64_t T, cudaStream_t s,
             int32_t rows_of_none = -1) {
    OpenArgs a{};
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
    a.partial = r.partial;
    a.count = c->attn_count;
    a.part = r.part;
    a.part_of = r.part_of;
    a.rows_of_none = rows_of_none;
    a.few = r.few;
    CUtensorMap q{}, k{}, v{};
    if (int rc = prompt_maps(c, r, T, a.tpt, &q, &k, &v)) return rc;
    if (c->head_dim == 128)
        return is_e4m3(c) ? launch_open<128, true>(c, q, k, v, a, s) : launch_open<128, false>(c, q, k, v, a, s);
    return is_e4m3(c) ? launch_open<64, true>(c, q, k, v, a, s) : launch_open<64, false>(c, q, k, v, a, s);
}

// The workspace of decode_shared: results over prefixes and over own keys, each fp32 [rows][Hq][D] and what
// they are [rows][Hq]. Own keys' split ranges have partial sums of their own, since the prefixes' are read
// with them.
struct SharedPart {
    float* part;
    RowOf* of;
};
size_t part_bytes(const tpmlp_ctx* c, int64_t rows) {
    return static_cast<size_t>(rows) * c->heads_q * (c->head_dim * sizeof(float) + sizeof(RowOf));
}
SharedPart shared_part(const tpmlp_ctx* c, int which) {
    char* const p = reinterpret_cast<char*>(c->shared[c->shared_n - 1]) + which * part_bytes(c, c->shared_rows);
    const int64_t values = c->shared_rows * c->heads_q * c->head_dim;
    return {reinterpret_cast<float*>(p), reinterpret_cast<RowOf*>(reinterpret_cast<float*>(p) + values)};
}

template <int D, bool FP8, int SLICES>
int launch_join(tpmlp_ctx* c, const JoinPartsArgs& a, cudaStream_t s) {
    constexpr int64_t kHeads = kJoinThreads / (D / 4 * SLICES);  // of a block
    return launch(c, join_parts_kernel<D, FP8, SLICES>, (a.heads + kHeads - 1) / kHeads, kJoinThreads, 0, s, a);
}

// CTAs that an item of `heads` rows x heads of B sequences is split over, about, if their keys are many.
int64_t split_over(const tpmlp_ctx* c, int64_t B, int64_t heads) {
    const int64_t tiles = std::max(B, (heads / c->heads_kv + 2 * kPB - 1) / (2 * kPB));
    return c->num_sms / (tiles * c->heads_kv);
}

// Joins the parts of `rows` rows of Q over keys of B sequences.
int run_join(tpmlp_ctx* c, JoinPartsArgs a, int64_t B, int64_t rows, cudaStream_t s) {
    a.heads = rows * c->heads_q;
    a.Hq = c->heads_q;
    a.G = c->heads_q / c->heads_kv;
    a.ctas = c->num_sms;
    a.v_scale = c->kv_scale + c->heads_kv;
    const bool many = split_over(c, B, a.heads) >= 8;
    if (c->head_dim == 128) {
        if (is_e4m3(c)) return many ? launch_join<128, true, 4>(c, a, s) : launch_join<128, true, 1>(c, a, s);
        return many ? launch_join<128, false, 4>(c, a, s) : launch_join<128, false, 1>(c, a, s);
    }
    if (is_e4m3(c)) return many ? launch_join<64, true, 4>(c, a, s) : launch_join<64, true, 1>(c, a, s);
    return many ? launch_join<64, false, 4>(c, a, s) : launch_join<64, false, 1>(c, a, s);
}

// The memory behind attn_partial for a call of tpmlp_attn_cross whose items are split over join_apart
// CTAs or more, and so are few.
SharedPart cross_part(const tpmlp_ctx* c) {
    float* const p = c->attn_partial + c->attn_partial_floats;
    return {p, reinterpret_cast<RowOf*>(p + static_cast<size_t>(cross_part_heads(c)) * c->head_dim)};
}

// Which launches take T rows of Q over the keys of B sequences, whose tables hold `keys` each. Few rows to a
// sequence on average: the row kernel, if it finds that no sequence has many, and then the open one, if there
// is one that has (the other ends at once). Both against the open kernel alone, us: 16 x 4 rows on 577 keys x
// 12 heads of 64 13, 19 (e4m3 10, 22); 64 x 4 on 1500 x 20 of 64 84, 126 (63, 157); 8 x 8 on 1500 x 32 of 128
// 41, 42 (30, 48); 16 x 3 on 577 x 24 of 64, 6 to a kv head 12.1, 11.5 (8, 13). Where all rows together are
// few the open kernel is left out (decode of 5 sequences x 12 heads of 64 behind 511 keys 9.3, with it 12.9).
struct AllKeysPath {
    int64_t heads;  // rows x heads of a kv head to a sequence, on average
    bool rows, open, apart;  // the row kernel, the open one, a join of the open one's parts
    int few;        // rows x heads of a sequence that the row kernel takes
};
AllKeysPath all_keys_path(const tpmlp_ctx* c, int64_t B, int64_t T, int64_t keys) {
    AllKeysPath x{};
    const int64_t G = c->heads_q / c->heads_kv;
    x.heads = (T * G + B - 1) / B;
    x.rows = x.heads <= row_heads(c->head_dim, is_e4m3(c));
    x.few = x.heads <= 8 ? 16 : 32;
    x.open = !x.rows || T * G > x.few;  // (else no sequence can have more)
    x.apart = !x.rows && keys >= kJoinApartKeys && split_over(c, B, T * c->heads_q) >= join_apart(c);
    return x;
}

// Each sequence's rows over all of its keys (MODE: kRowsCross, kRowsCrossPart).
template <int MODE>
int run_all_keys(tpmlp_ctx* c, RowArgs a, const int32_t* cu_q, int64_t T, cudaStream_t s) {
    const AllKeysPath x = all_keys_path(c, a.kv.B, T, static_cast<int64_t>(a.kv.table_pages) << a.kv.page_shift);
    if (x.rows) {
        a.rows = a.kv.B;
        a.cu_q = cu_q;
        a.T = static_cast<int32_t>(T);
        a.few = x.few;
        if (int rc = run_rows<MODE>(c, a, s, x.heads)) return rc;
        if (!x.open) return TPMLP_OK;
    }
    if (MODE == kRowsCross && x.apart) {
        JoinPartsArgs j{};
        const SharedPart part = cross_part(c);
        j.side[0] = {part.part, part.of, c->attn_partial};
        j.out = a.out;
        j.ldo = a.ldo;
        j.lse = a.lse;
        a.part = part.part;
        a.part_of = part.of;
        if (int rc = run_open(c, a, cu_q, T, s, -2)) return rc;  // (rows of no sequence stay as they are)
        return run_join(c, j, a.kv.B, T, s);
    }
    return run_open(c, a, cu_q, T, s);
}

// Clears new memory, before any stream's work may meet it (streams made without blocking do not wait for
// the default stream, where this runs); frees it if that fails.
int clear_new(tpmlp_ctx* c, void* p, size_t bytes) {
    cudaError_t e = cudaMemset(p, 0, bytes);
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    if (e == cudaSuccess) return TPMLP_OK;
    cudaFree(p);
    return fail_cuda(c, e, "clearing the workspace of decode_shared");
}

// It holds `rows` sequences (s: the stream that a call is on; null: tpmlp_attn_reserve).
int reserve_shared(tpmlp_ctx* c, int64_t rows, const cudaStream_t* s) {
    if (rows <= c->shared_rows) return TPMLP_OK;
    if (s)
        if (int rc = refuse_allocation(c, *s, "tpmlp_attn_reserve before the capture")) return rc;
    if (!c->tail_partial) {
        // two slots and a counter to a CTA of either kernel (the open kernel's counters are the context's)
        const size_t ctas = static_cast<size_t>(c->num_sms) * 16 / row_warps(kRowsPart);
        const size_t floats = std::max(c->attn_partial_floats, ctas * 2 * kRowSlotFloats);
        void* p = nullptr;
        if (int rc = allocate(c, &p, floats * sizeof(float) + ctas * sizeof(uint32_t))) return rc;
        uint32_t* const count = reinterpret_cast<uint32_t*>(static_cast<float*>(p) + floats);
        if (int rc = clear_new(c, p, floats * sizeof(float) + ctas * sizeof(uint32_t))) return rc;
        c->tail_partial = static_cast<float*>(p);
        c->tail_count = count;
    }
    const int64_t now = std::max(rows, 2 * c->shared_rows);
    void* p = nullptr;
    if (int rc = allocate(c, &p, 2 * part_bytes(c, now))) return rc;
    if (int rc = clear_new(c, p, 2 * part_bytes(c, now))) return rc;
    c->shared[c->shared_n++] = static_cast<float*>(p);
    c->shared_rows = now;
    return TPMLP_OK;
}

}  // namespace

extern "C" {

int tpmlp_attn_cross(tpmlp_ctx* c, const void* Q, int64_t ldq, int64_t T, const int32_t* cu_q,
                     const tpmlp_kv* kv, float scale, void* Out, int64_t ldo, float* Lse, void* stream) {
    if (int rc = check_attention(c)) return rc;
    if (!kv || T < 0) return TPMLP_ERR_INVALID_ARG;
    if (T == 0 || kv->B == 0) return TPMLP_OK;
    if (T > INT_MAX / 2) return TPMLP_ERR_UNSUPPORTED_SHAPE;
    if (int rc = check_attend(c, Q, ldq, kv, scale, Out, ldo, Lse)) return rc;
    if (!cu_q) return TPMLP_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(cu_q) & 3) return TPMLP_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    RowArgs a = row_args(c, Q, ldq, kv, scale, 0, Out, ldo, Lse);
    return run_all_keys<kRowsCross>(c, a, cu_q, T, s);
}

int tpmlp_attn_reserve(tpmlp_ctx* c, int64_t max_sequences) {
    if (int rc = check_attention(c)) return rc;
    if (max_sequences < 0) return TPMLP_ERR_INVALID_ARG;
    if (max_sequences > INT_MAX / 2) return TPMLP_ERR_UNSUPPORTED_SHAPE;
    return reserve_shared(c, max_sequences, nullptr);
}

int tpmlp_attn_decode_shared(tpmlp_ctx* c, const void* Q, int64_t ldq, const tpmlp_kv* prefix,
                             const int32_t* cu, const tpmlp_kv* kv, float scale, void* Out,
                             int64_t ldo, float* Lse, void* stream) {
    if (int rc = check_attention(c)) return rc;
    if (!kv || !prefix) return TPMLP_ERR_INVALID_ARG;
    if (kv->B == 0) return TPMLP_OK;
    if (prefix->B == 0) return tpmlp_attn_decode(c, Q, ldq, kv, scale, 0, Out, ldo, Lse, stream);
    if (kv->B > INT_MAX / 2) return TPMLP_ERR_UNSUPPORTED_SHAPE;
    if (int rc = check_attend(c, Q, ldq, kv, scale, Out, ldo, Lse)) return rc;
    if (int rc = check_kv(c, prefix, true)) return rc;
    if (!cu) return TPMLP_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(cu) & 3) return TPMLP_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (int rc = reserve_shared(c, kv->B, &s)) return rc;
    const SharedPart common = shared_part(c, 0), own = shared_part(c, 1);
    RowArgs p = row_args(c, Q, ldq, prefix, scale, 0, Out, ldo, nullptr);
    p.part = common.part;
    p.part_of = common.of;
    if (int rc = run_all_keys<kRowsCrossPart>(c, p, cu, kv->B, s)) return rc;
    RowArgs a = row_args(c, Q, ldq, kv, scale, 0, Out, ldo, nullptr);
    a.rows = kv->B;
    a.partial = c->tail_partial;
    a.part = own.part;
    a.part_of = own.of;
    const bool wide = a.G > row_heads(c->head_dim, is_e4m3(c));
    if (!wide) a.count = c->tail_count;
    if (int rc = wide ? run_open(c, a, nullptr, kv->B, s) : run_rows<kRowsPart>(c, a, s, a.G)) return rc;
    JoinPartsArgs j{};
    j.side[0] = {common.part, common.of, c->attn_partial};
    j.side[1] = {own.part, own.of, c->tail_partial};
    j.out = a.out;
    j.ldo = ldo;
    j.lse = Lse;
    return run_join(c, j, prefix->B, kv->B, s);
}

int tpmlp_attn_cross_packed(const tpmlp_attend_args* a) {
    if (!a || a->window != 0) return TPMLP_ERR_INVALID_ARG;
    return tpmlp_attn_cross(a->ctx, a->Q, a->ldq, a->T, a->cu_q, a->kv, static_cast<float>(a->scale), a->Out,
                            a->ldo, a->Lse, a->stream);
}

int tpmlp_attn_decode_shared_packed(const tpmlp_shared_args* a) {
    if (!a) return TPMLP_ERR_INVALID_ARG;
    return tpmlp_attn_decode_shared(a->ctx, a->Q, a->ldq, a->prefix, a->cu, a->kv, static_cast<float>(a->scale),
                                    a->Out, a->ldo, a->Lse, a->stream);
}

}  // extern "C"

#ifdef TPMLP_TEST_HOOKS
// Test builds only: the launches of cross attention of T rows over the keys of B sequences (bit 0: the row
// kernel, 1: the open one, 2: the join of its parts), and the rows x heads that such a join has room for.
extern "C" TPMLP_API int tpmlp_test_cross_path(const tpmlp_ctx* c, int64_t B, int64_t T, int64_t keys) {
    const AllKeysPath x = all_keys_path(c, B, T, keys);
    return x.rows | x.open << 1 | x.apart << 2;
}
extern "C" TPMLP_API int64_t tpmlp_test_cross_room(const tpmlp_ctx* c) { return cross_part_heads(c); }
#endif
