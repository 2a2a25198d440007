// C ABI of the operators that cut rows of logits: argument validation and
// dispatch. As in api.cu every call validates on the host, returns before any
// launch on a host-detectable error and otherwise enqueues one kernel without
// synchronising.
#include <cmath>
#include <cstdint>

#include "cut.h"

namespace {

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool stride_ok(int64_t s) { return s >= 0 && s < (int64_t(1) << 40); }

sv_status check(const sv_logits_cut* c) {
    if (!c) return SV_ERR_NULL;
    if (!c->logits) return SV_ERR_NULL;
    if (c->dtype != SV_F32 && c->dtype != SV_BF16) return SV_ERR_DTYPE;
    if (c->B < 1 || c->R < 1 || c->V < 2 || c->V > sv::CUT_MAX_V || (int64_t)c->B * c->R > (int64_t(1) << 28)) return SV_ERR_SHAPE;
    if (!stride_ok(c->seq_stride) || !stride_ok(c->row_stride)) return SV_ERR_SHAPE;
    if (!c->temperatures && !(c->temperature == 0.0f || (c->temperature >= 0x1p-64f && c->temperature <= 0x1p64f)))
        return SV_ERR_TEMPERATURE;
    if ((!c->top_ks && c->top_k < 0) || (!c->top_ps && !(c->top_p >= 0.0f && c->top_p <= 1.0f)) ||
        (!c->min_ps && !(c->min_p >= 0.0f && c->min_p <= 1.0f)))
        return SV_ERR_CONFIG;
    const size_t e = c->dtype == SV_F32 ? 4 : 2;
    if (!aligned(c->logits, e) || !aligned(c->temperatures, 4) || !aligned(c->top_ks, 4) || !aligned(c->top_ps, 4) ||
        !aligned(c->min_ps, 4) || !aligned(c->status_word, 4))
        return SV_ERR_ALIGN;
    return SV_OK;
}

sv::CutParams params(const sv_logits_cut& c) {
    const int64_t e = c.dtype == SV_F32 ? 4 : 2;
    sv::CutParams p = {};
    p.logits = static_cast<const char*>(c.logits);
    p.seq_bytes = c.seq_stride * e;
    p.row_bytes = c.row_stride * e;
    p.B = c.B, p.R = c.R, p.V = c.V;
    p.temperature = c.temperature, p.top_p = c.top_p, p.min_p = c.min_p, p.top_k = c.top_k;
    p.temperatures = c.temperatures, p.top_ks = c.top_ks, p.top_ps = c.top_ps, p.min_ps = c.min_ps;
    p.status = c.status_word;
    return p;
}

sv_status enqueue(const sv::CutParams& p, const sv_logits_cut& c, bool draw) {
    int sms = 0;
    const sv_status st = sv::check_device(&sms);
    if (st != SV_OK) return st;
    const cudaError_t e = sv::launch_cut_logits(p, c.dtype, draw, sms, (cudaStream_t)c.stream);
    return e == cudaSuccess ? SV_OK : sv::fail_cuda(e);
}

// Rows of the output that share memory cannot be written by two.
bool rows_apart(int64_t seq, int64_t row, const sv_logits_cut& c) {
    if (c.R > 1 && row < c.V) return false;
    if (c.B == 1) return true;
    if (seq < c.V) return false;
    return c.R == 1 || seq >= (c.R - 1) * row + c.V || row >= (c.B - 1) * seq + c.V;
}

}  // namespace

extern "C" sv_status spec_sample(const sv_logits_cut* cut, const float* uniforms, int32_t* out_tokens, float* out_logprobs) {
    const sv_status st = check(cut);
    if (st != SV_OK) return st;
    if (!uniforms || !out_tokens) return SV_ERR_NULL;
    if (!aligned(uniforms, 4) || !aligned(out_tokens, 4) || !aligned(out_logprobs, 4)) return SV_ERR_ALIGN;
    sv::CutParams p = params(*cut);
    p.uniforms = uniforms;
    p.tokens = out_tokens;
    p.logprobs = out_logprobs;
    return enqueue(p, *cut, true);
}

extern "C" sv_status spec_truncate_logits(const sv_logits_cut* cut, void* out, int64_t out_seq_stride, int64_t out_row_stride,
                                          int32_t* out_n_kept) {
    const sv_status st = check(cut);
    if (st != SV_OK) return st;
    if (!out) return SV_ERR_NULL;
    if (!stride_ok(out_seq_stride) || !stride_ok(out_row_stride) || !rows_apart(out_seq_stride, out_row_stride, *cut)) return SV_ERR_SHAPE;
    const size_t e = cut->dtype == SV_F32 ? 4 : 2;
    if (!aligned(out, e) || !aligned(out_n_kept, 4)) return SV_ERR_ALIGN;
    sv::CutParams p = params(*cut);
    p.out = static_cast<char*>(out);
    p.out_seq_bytes = out_seq_stride * (int64_t)e;
    p.out_row_bytes = out_row_stride * (int64_t)e;
    p.n_kept = out_n_kept;
    return enqueue(p, *cut, false);
}

extern "C" size_t sv_logits_cut_size(void) { return sizeof(sv_logits_cut); }
