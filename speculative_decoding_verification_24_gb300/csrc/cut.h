// Internal interface between the C-ABI layer of the operators that cut rows of
// logits (cut_api.cu) and their kernel (cut_logits.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "specverify.h"

namespace sv {

constexpr int CUT_MAX_V = 1 << 18;  // an index takes 18 bits of a place in a row's order

struct CutParams {
    const char* logits;
    int64_t seq_bytes, row_bytes;  // strides
    int B, R, V;
    float temperature, top_p, min_p;
    int top_k;
    const float *temperatures, *top_ps, *min_ps;  // [B] or nullptr
    const int32_t* top_ks;                        // [B] or nullptr
    // drawing
    const float* uniforms;   // [B, R]
    int32_t* tokens;         // [B, R]
    float* logprobs;         // [B, R] or nullptr
    // cutting
    char* out;
    int64_t out_seq_bytes, out_row_bytes;
    int32_t* n_kept;         // [B, R] or nullptr
    uint32_t* status;        // or nullptr
    int slice_vecs;          // 16-byte pieces of a row per CTA at most
    int longest_first;       // the rows' order
};

cudaError_t launch_cut_logits(CutParams p, int dtype, bool draw, int sms, cudaStream_t stream);

// The library's record of a failed CUDA call on this host thread, and the
// check that the current device is one it was built for (api.cu).
sv_status fail_cuda(cudaError_t e);
sv_status check_device(int* sms);

}  // namespace sv
