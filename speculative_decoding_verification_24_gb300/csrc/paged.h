// Internal interface between the paged cache's C-ABI layer (paged_api.cu) and
// its kernels (kv_cache.cu, paged_attention.cu).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "specverify.h"

namespace sv {

constexpr int KV_MAX_TREE = 32;       // nodes of a tree: one warp lane, one mask bit each
constexpr int KV_MAX_ROTARY = 128;    // rotary size: 64 frequencies in the kernel's parameters
constexpr int PA_TILE = 128;          // keys per tile (MMA N), rows per tile (MMA M)
constexpr int PA_MAX_CTAS = SV_PAGED_MAX_CTAS;
constexpr int PA_ITEM_COST = 2;       // units of work of an item besides its key tiles

// The chunk of a batch: which packed rows belong to which sequence, and where
// its tokens lie in the cache.
struct ChunkParams {
    const int32_t* cu;       // [B+1]
    const int32_t* ctx;      // [B]
    const int32_t* table;    // [B, max_pages], rows table_stride apart
    int64_t table_stride;
    int max_pages, page_size, n_pages;
    int B, T, Hkv;
    const int32_t* parents;  // [B, N] or nullptr
    int N;
    uint32_t* status;        // or nullptr
};

struct KvAppendParams {
    ChunkParams ch;
    char *kc, *vc;                              // cache bases
    int64_t kc_ps, kc_ts, kc_hs, vc_ps, vc_ts, vc_hs;  // bytes
    const char *k, *v, *q;                      // q may be nullptr
    int64_t k_ts, k_hs, v_ts, v_hs, q_ts, q_hs, qo_ts, qo_hs;  // bytes
    char* q_out;
    int Hq, D, rotary, interleaved;
    const int32_t* positions;                   // [T] or nullptr
    int tokens_per_cta;
    uint64_t turns[KV_MAX_ROTARY / 2];          // inverse frequencies in 2^-64 turns per position
};

struct KvCommitParams {
    ChunkParams ch;          // cu unused
    char *kc, *vc;
    int64_t kc_ps, kc_ts, kc_hs, vc_ps, vc_ts, vc_hs;
    int D;
    const int32_t *n_accepted, *last_node;
    int32_t* out_lens;
};

struct PagedAttnParams {
    ChunkParams ch;
    char* out;
    int64_t o_ts, o_hs;      // bytes
    float* lse;              // [T, Hq] or nullptr
    const char* vc;          // the values, for the few read by address (add_not_finite)
    int64_t vc_ps, vc_ts, vc_hs;  // bytes
    int Hq, G, TT;           // G = Hq / Hkv; TT = tokens per 128-row tile
    int q_box;               // tokens of one copy of queries, a divisor of TT
    int box_shift;           // log2 of the rows of one copy (page_size's power of two, at most 128)
    float c;                 // scale * log2(e)
    int rows_cap;            // rows of one partial in the workspace
    uint32_t* counters;      // [PA_MAX_CTAS], zero between calls
    float2* part_ml;         // [2 * PA_MAX_CTAS, rows_cap]
    float* part_o;           // [2 * PA_MAX_CTAS, D / 4, rows_cap, 4]
    int test_wait_timeout;
};

cudaError_t launch_kv_append(const KvAppendParams& p, int f16, int sms, cudaStream_t stream);
cudaError_t launch_kv_commit(const KvCommitParams& p, cudaStream_t stream);
cudaError_t launch_paged_attention(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                   const PagedAttnParams& p, int D, int f16, int sms, cudaStream_t stream);

// The library's record of a failed CUDA call on this host thread, and the
// check that the current device is one it was built for (api.cu).
sv_status fail_cuda(cudaError_t e);
sv_status check_device(int* sms);

}  // namespace sv
