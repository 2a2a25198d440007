// C ABI of the paged cache's entry points: argument validation, the tensor
// maps of the cache, workspace layout and dispatch. As in api.cu every call
// validates on the host, returns before any launch on a host-detectable error
// and otherwise enqueues one kernel without synchronising.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "paged.h"

namespace {

using sv::check_device;
using sv::fail_cuda;

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0 && s < (int64_t(1) << 38); }

// Entries of their own: what is broadcast cannot be written.
bool apart(int64_t stride, int extent) { return stride > 0 || extent <= 1; }

sv_status check_cache(const sv_kv_cache& c) {
    if (!c.k || !c.v || !c.page_table || !c.ctx_lens) return SV_ERR_NULL;
    if (c.dtype != SV_BF16 && c.dtype != SV_F16) return SV_ERR_DTYPE;
    if (c.n_pages < 1 || c.n_pages == INT32_MAX || c.page_size < 8 || c.page_size > 65536 || c.page_size % 8 != 0 || c.Hkv < 1 ||
        c.Hkv > 65535 || (c.D != 64 && c.D != 128) || c.B < 1 || c.max_pages < 1 || c.page_table_stride < c.max_pages)
        return SV_ERR_SHAPE;
    // slot numbers are int32, with room for a tile past the last one
    if ((int64_t)c.max_pages * c.page_size > INT32_MAX - 1024) return SV_ERR_SHAPE;
    if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.page_table, 4) || !aligned(c.ctx_lens, 4)) return SV_ERR_ALIGN;
    if (!stride_ok(c.k_page_stride) || !stride_ok(c.k_token_stride) || !stride_ok(c.k_head_stride) ||
        !stride_ok(c.v_page_stride) || !stride_ok(c.v_token_stride) || !stride_ok(c.v_head_stride))
        return SV_ERR_ALIGN;
    if (!apart(c.k_page_stride, c.n_pages) || !apart(c.k_token_stride, c.page_size) || !apart(c.k_head_stride, c.Hkv) ||
        !apart(c.v_page_stride, c.n_pages) || !apart(c.v_token_stride, c.page_size) || !apart(c.v_head_stride, c.Hkv))
        return SV_ERR_SHAPE;
    return SV_OK;
}

sv_status check_tree(const int32_t* parents, int N) {
    if (!parents) return SV_OK;
    if (N < 1 || N > sv::KV_MAX_TREE) return SV_ERR_SHAPE;
    return aligned(parents, 4) ? SV_OK : SV_ERR_ALIGN;
}

sv::ChunkParams chunk_of(const sv_kv_cache& c, const int32_t* cu, int T, const int32_t* parents, int N, uint32_t* status) {
    sv::ChunkParams p = {};
    p.cu = cu;
    p.ctx = c.ctx_lens;
    p.table = c.page_table;
    p.table_stride = c.page_table_stride;
    p.max_pages = c.max_pages;
    p.page_size = c.page_size;
    p.n_pages = c.n_pages;
    p.B = c.B;
    p.T = T;
    p.Hkv = c.Hkv;
    p.parents = parents;
    p.N = N;
    p.status = status;
    return p;
}

template <class P>
void put_cache(P& p, const sv_kv_cache& c) {
    p.kc = static_cast<char*>(c.k);
    p.vc = static_cast<char*>(c.v);
    p.kc_ps = c.k_page_stride * 2, p.kc_ts = c.k_token_stride * 2, p.kc_hs = c.k_head_stride * 2;
    p.vc_ps = c.v_page_stride * 2, p.vc_ts = c.v_token_stride * 2, p.vc_hs = c.v_head_stride * 2;
}

PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
    static std::atomic<void*> fn{nullptr};
    void* f = fn.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(f, std::memory_order_release);
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
}

// A tensor map of the cache's type, 128-byte swizzled, in boxes of 64 columns.
// A stride of an extent of 1 is never used, but has to be a valid one.
bool encode(CUtensorMap* map, sv_dtype dtype, const void* base, int rank, const int64_t* extents, const int64_t* strides,
            const int* box) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = get_encode();
    if (!fn) return false;
    cuuint64_t dims[4], bytes[3];
    cuuint32_t boxes[4];
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    for (int i = 0; i < rank; ++i) {
        dims[i] = (cuuint64_t)extents[i];
        boxes[i] = (cuuint32_t)box[i];
        if (i > 0) bytes[i - 1] = extents[i] == 1 && strides[i] == 0 ? 16 : (cuuint64_t)strides[i] * 2;
    }
    return fn(map, dtype == SV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank,
              const_cast<void*>(base), dims, bytes, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One half of the cache as (D, entry of the page, head, page); a box is `box`
// entries of one head.
bool encode_cache(CUtensorMap* map, const sv_kv_cache& c, const void* base, int64_t page, int64_t token, int64_t head, int box) {
    const int64_t extents[4] = {c.D, c.page_size, c.Hkv, c.n_pages}, strides[4] = {1, token, head, page};
    const int boxes[4] = {64, box, 1, 1};
    return encode(map, c.dtype, base, 4, extents, strides, boxes);
}

// The queries as (D, head, token); a box is `tokens` tokens of one kv head's
// `group` query heads, in the order of a tile's rows.
bool encode_queries(CUtensorMap* map, const sv_paged_attention_args& a, int tokens, int group) {
    const int64_t extents[3] = {a.cache.D, a.Hq, a.T}, strides[3] = {1, a.q_head_stride, a.q_token_stride};
    const int boxes[3] = {64, group, tokens};
    return encode(map, a.cache.dtype, a.q, 3, extents, strides, boxes);
}

// 2^64 times the fraction of a turn that t turns are, modulo 2^64.
uint64_t fixed_turns(double t) {
    const double whole = std::fabs(t), x = (whole - std::floor(whole)) * 18446744073709551616.0;  // below 2^64, exact
    return t < 0.0 ? 0 - (uint64_t)x : (uint64_t)x;
}

// The same of w radians. A position multiplies the error by up to 2^31, so 1 /
// 2 pi is taken in two parts and the product with what its rounding dropped:
// with one double each, 2^31 positions were off by 2^-24 turns at w = 1 and by
// 2^-18 at w = 100.
uint64_t turn_fraction(double w) {
    constexpr double high = 0x1.45f306dc9c883p-3, low = -0x1.6b01ec5417056p-57;  // 1 / 2 pi
    const double t = std::fma(w, high, 0.0);  // the product, rounded, and not contracted with what follows
    const double rest = std::fma(w, high, -t) + w * low;
    return fixed_turns(t) + (std::fabs(rest) < 0.25 ? (uint64_t)(int64_t)(rest * 18446744073709551616.0) : fixed_turns(rest));
}

// Rows of one piece: a tile of 128 or, when a sequence may have more rows, a
// pair of them; fewer when all packed rows together have fewer.
int piece_rows(long long T, int G) {
    const long long rows = T * G;
    if (T > 128 / G) return 256;
    return (int)((rows + 31) / 32 * 32);
}

bool heads_ok(int Hq, int Hkv) { return Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0 && Hq / Hkv <= 128; }

constexpr size_t kPieces = 2 * SV_PAGED_MAX_CTAS;
size_t stats_bytes(int rows) { return kPieces * (size_t)rows * sizeof(float2); }

}  // namespace

extern "C" sv_status spec_kv_append(const sv_kv_append_args* a) {
    if (!a) return SV_ERR_NULL;
    sv_status st = check_cache(a->cache);
    if (st != SV_OK) return st;
    const sv_kv_cache& c = a->cache;
    if (!a->cu_new || (a->T > 0 && (!a->k || !a->v)) || (a->q && !a->q_out)) return SV_ERR_NULL;
    if (a->T < 0 || (a->q && (a->Hq < 1 || a->Hq > 65535))) return SV_ERR_SHAPE;
    if (a->rotary < 0 || a->rotary > c.D || a->rotary % 16 != 0) return SV_ERR_SHAPE;
    if (a->rotary > 0 && !a->inv_freq) return SV_ERR_NULL;
    if ((st = check_tree(a->tree_parents, a->N)) != SV_OK) return st;
    if (!aligned(a->cu_new, 4) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->q, 16) || !aligned(a->q_out, 16) ||
        !aligned(a->positions, 4) || !aligned(a->status_word, 4) || !aligned(a->inv_freq, 8))
        return SV_ERR_ALIGN;
    if (!stride_ok(a->k_token_stride) || !stride_ok(a->k_head_stride) || !stride_ok(a->v_token_stride) ||
        !stride_ok(a->v_head_stride) ||
        (a->q && (!stride_ok(a->q_token_stride) || !stride_ok(a->q_head_stride) || !stride_ok(a->q_out_token_stride) ||
                  !stride_ok(a->q_out_head_stride))))
        return SV_ERR_ALIGN;
    if (a->q && (!apart(a->q_out_token_stride, a->T) || !apart(a->q_out_head_stride, a->Hq))) return SV_ERR_SHAPE;
    for (int i = 0; i < a->rotary / 2; ++i)
        if (!std::isfinite(a->inv_freq[i])) return SV_ERR_CONFIG;
    int sms = 0;
    if ((st = check_device(&sms)) != SV_OK) return st;
    if (a->T == 0) return SV_OK;

    sv::KvAppendParams p = {};
    p.ch = chunk_of(c, a->cu_new, a->T, a->tree_parents, a->N, a->status_word);
    put_cache(p, c);
    p.k = static_cast<const char*>(a->k);
    p.v = static_cast<const char*>(a->v);
    p.q = static_cast<const char*>(a->q);
    p.q_out = static_cast<char*>(a->q_out);
    p.k_ts = a->k_token_stride * 2, p.k_hs = a->k_head_stride * 2;
    p.v_ts = a->v_token_stride * 2, p.v_hs = a->v_head_stride * 2;
    p.q_ts = a->q_token_stride * 2, p.q_hs = a->q_head_stride * 2;
    p.qo_ts = a->q_out_token_stride * 2, p.qo_hs = a->q_out_head_stride * 2;
    p.Hq = a->Hq;
    p.D = c.D;
    p.rotary = a->rotary;
    p.interleaved = a->interleaved != 0;
    p.positions = a->positions;
    for (int i = 0; i < a->rotary / 2; ++i) p.turns[i] = turn_fraction(a->inv_freq[i]);
    const cudaError_t e = sv::launch_kv_append(p, c.dtype == SV_F16, sms, (cudaStream_t)a->stream);
    return e == cudaSuccess ? SV_OK : fail_cuda(e);
}

extern "C" size_t spec_paged_attention_workspace_bytes(int T, int Hq, int Hkv, int D) {
    if (T < 0 || !heads_ok(Hq, Hkv) || (D != 64 && D != 128)) return 0;
    const int rows = piece_rows(T, Hq / Hkv);
    return SV_PAGED_WORKSPACE_HEAD + stats_bytes(rows) + kPieces * (size_t)rows * D * sizeof(float);
}

extern "C" sv_status spec_paged_attention(const sv_paged_attention_args* a) {
    if (!a) return SV_ERR_NULL;
    sv_status st = check_cache(a->cache);
    if (st != SV_OK) return st;
    const sv_kv_cache& c = a->cache;
    if (!a->cu_new || (a->T > 0 && (!a->q || !a->out))) return SV_ERR_NULL;
    if (a->T < 0 || !heads_ok(a->Hq, c.Hkv)) return SV_ERR_SHAPE;
    const int G = a->Hq / c.Hkv, TT = sv::PA_TILE / G;
    // the kernel counts key tiles of (sequence, head, row tile) items in int32
    const double items = (std::ceil(a->T / (2.0 * TT)) + c.B) * c.Hkv;
    if (items * (std::ceil((double)c.max_pages * c.page_size / sv::PA_TILE) + sv::PA_ITEM_COST) > 2147483647.0) return SV_ERR_SHAPE;
    if (!std::isfinite(a->scale) || !(a->scale > 0.0f) || !std::isfinite(a->scale * 1.4426950408889634f)) return SV_ERR_CONFIG;
    if (a->flags & ~SV_ARG_TEST_WAIT_TIMEOUT) return SV_ERR_CONFIG;
    if ((st = check_tree(a->tree_parents, a->N)) != SV_OK) return st;
    if (!aligned(a->cu_new, 4) || !aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->out_lse, 4) ||
        !aligned(a->status_word, 4) || !aligned(a->workspace, 256))
        return SV_ERR_ALIGN;
    if (!stride_ok(a->q_token_stride) || !stride_ok(a->q_head_stride) || !stride_ok(a->out_token_stride) ||
        !stride_ok(a->out_head_stride))
        return SV_ERR_ALIGN;
    // (queries: a tensor map has no stride of 0)
    if (!apart(a->q_token_stride, a->T) || !apart(a->q_head_stride, a->Hq) || !apart(a->out_token_stride, a->T) ||
        !apart(a->out_head_stride, a->Hq))
        return SV_ERR_SHAPE;
    if (a->T > 0 &&
        (!a->workspace || a->workspace_bytes < spec_paged_attention_workspace_bytes(a->T, a->Hq, c.Hkv, c.D)))
        return SV_ERR_WORKSPACE;
    int sms = 0;
    if ((st = check_device(&sms)) != SV_OK) return st;
    if (a->T == 0) return SV_OK;

    sv::PagedAttnParams p = {};
    p.ch = chunk_of(c, a->cu_new, a->T, a->tree_parents, a->N, a->status_word);
    p.out = static_cast<char*>(a->out);
    p.o_ts = a->out_token_stride * 2, p.o_hs = a->out_head_stride * 2;
    p.lse = a->out_lse;
    p.vc = static_cast<const char*>(c.v);
    p.vc_ps = c.v_page_stride * 2, p.vc_ts = c.v_token_stride * 2, p.vc_hs = c.v_head_stride * 2;
    p.Hq = a->Hq;
    p.G = G;
    p.TT = TT;
    while (p.box_shift < 7 && c.page_size % (2 << p.box_shift) == 0) ++p.box_shift;
    p.c = a->scale * 1.4426950408889634f;
    p.rows_cap = piece_rows(a->T, G);
    char* ws = static_cast<char*>(a->workspace);
    p.counters = reinterpret_cast<uint32_t*>(ws);
    p.part_ml = reinterpret_cast<float2*>(ws + SV_PAGED_WORKSPACE_HEAD);
    p.part_o = reinterpret_cast<float*>(ws + SV_PAGED_WORKSPACE_HEAD + stats_bytes(p.rows_cap));
    p.test_wait_timeout = (a->flags & SV_ARG_TEST_WAIT_TIMEOUT) != 0;
    // queries come in boxes of about as many tokens as a sequence has: one box
    // for a token or a tile, and few rows of other sequences with them
    const int mean = (int)(((int64_t)a->T + c.B - 1) / c.B);
    for (p.q_box = mean < TT ? mean : TT; TT % p.q_box != 0;) --p.q_box;
    CUtensorMap tm_q, tm_k, tm_v;
    if (!encode_queries(&tm_q, *a, p.q_box, G) || !encode_cache(&tm_k, c, c.k, c.k_page_stride, c.k_token_stride, c.k_head_stride, 1 << p.box_shift) ||
        !encode_cache(&tm_v, c, c.v, c.v_page_stride, c.v_token_stride, c.v_head_stride, 1 << p.box_shift))
        return fail_cuda(cudaErrorInvalidValue);
    const cudaError_t e = sv::launch_paged_attention(tm_q, tm_k, tm_v, p, c.D, c.dtype == SV_F16, sms, (cudaStream_t)a->stream);
    return e == cudaSuccess ? SV_OK : fail_cuda(e);
}

extern "C" sv_status spec_kv_commit(const sv_kv_cache* cache, const int32_t* n_accepted, const int32_t* tree_parents, int N,
                                    const int32_t* last_node, int32_t* out_lens, uint32_t* status_word, sv_stream_t stream) {
    if (!cache) return SV_ERR_NULL;
    sv_status st = check_cache(*cache);
    if (st != SV_OK) return st;
    if (!n_accepted || !out_lens || (tree_parents && !last_node)) return SV_ERR_NULL;
    if ((st = check_tree(tree_parents, N)) != SV_OK) return st;
    if (!aligned(n_accepted, 4) || !aligned(last_node, 4) || !aligned(out_lens, 4) || !aligned(status_word, 4)) return SV_ERR_ALIGN;
    int sms = 0;
    if ((st = check_device(&sms)) != SV_OK) return st;
    sv::KvCommitParams p = {};
    p.ch = chunk_of(*cache, nullptr, 0, tree_parents, N, status_word);
    put_cache(p, *cache);
    p.D = cache->D;
    p.n_accepted = n_accepted;
    p.last_node = last_node;
    p.out_lens = out_lens;
    const cudaError_t e = sv::launch_kv_commit(p, (cudaStream_t)stream);
    return e == cudaSuccess ? SV_OK : fail_cuda(e);
}

extern "C" size_t sv_kv_cache_size(void) { return sizeof(sv_kv_cache); }
extern "C" size_t sv_kv_append_args_size(void) { return sizeof(sv_kv_append_args); }
extern "C" size_t sv_paged_attention_args_size(void) { return sizeof(sv_paged_attention_args); }
