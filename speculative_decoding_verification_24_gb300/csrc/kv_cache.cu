// Writing and rearranging a paged key/value cache: appending a chunk's keys
// and values with the rotary rotation applied on the way, and keeping the
// path of a verified tree.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged_device.cuh"

namespace sv {

// ---------------------------------------------------------------------------
// Append. For a token at position t and frequency f_i the pair (a, b) becomes
//   (a cos(t f_i) - b sin(t f_i), b cos(t f_i) + a sin(t f_i)),
// with (a, b) = (x_i, x_{i + R/2}) or (x_2i, x_2i+1); elements past R stay.
// The angle is formed in turns as a 64-bit fixed-point fraction: position
// times f_i / 2 pi modulo 2^64 drops whole turns exactly, so a position of
// 2^20 has the same angle error (2^-25 turns, the fp32 argument of sincospif)
// as position 1. A float product would lose 2^-4 turns there.
//
// Every input byte is read once and every output byte written once, so HBM
// bounds it; a small call is bound by its chain of dependent loads (token ->
// sequence -> page). A CTA takes a few tokens: one warp per token finds its
// sequence and page, the angles of a token are formed once for all heads, and
// then D/16 lanes move one head, each two 16-byte pieces that hold whole pairs
// (pieces i and i + R/16, or neighbours), so that a rotation needs no exchange
// between lanes.
// ---------------------------------------------------------------------------
constexpr int KA_THREADS = 256;
constexpr int KA_MAX_TOKENS = 8;    // a warp each
constexpr int KA_MANY = 16;         // tokens per SM from which on there are many
constexpr int KA_BATCH = 3;         // pairs of pieces per thread whose loads are in flight together

struct TokenPlace {
    int64_t k_off, v_off;  // byte offsets of the slot in the caches, -1: not stored
    int row;               // packed row, -1: no sequence claims it
};

template <bool F16>
__device__ __forceinline__ void unpack8(uint4 w, float (&x)[8]) {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (F16) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r[i]));
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        } else {
            x[2 * i] = bf16_lo(r[i]), x[2 * i + 1] = bf16_hi(r[i]);
        }
    }
}

// Rounded once, to nearest even: the cache's own type.
template <bool F16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (F16) {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            r[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            r[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// The last sequence b with cu[b] <= t, by a warp that tests 32 places at once.
// Whatever cu holds, the answer lies in [0, B).
__device__ __forceinline__ int find_sequence(const int32_t* cu, int B, int t, int lane) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + lane * step;
        const uint32_t le = __ballot_sync(0xFFFFFFFFu, at < hi && cu[at] <= t);
        const int k = le ? 31 - __clz(le) : 0;
        const int nlo = lo + k * step;
        hi = min(hi, nlo + step);
        lo = nlo;
    }
    return lo;
}

// Read once, so not kept in L1; not the read-only path, since q_out may be q.
__device__ __forceinline__ uint4 ld_once(const char* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// What a lane moves: two pieces of one head of one of the CTA's tokens.
// Heads count keys first, then values, then queries.
template <int D>
struct Pieces {
    int token, head, c;  // c: which pair of pieces
    __device__ __forceinline__ Pieces(int x, int heads) {
        constexpr int L = D / 16;  // lanes per head
        const int y = x / L;
        c = x % L;
        token = y / heads;
        head = y - token * heads;
    }
    __device__ __forceinline__ bool apart(const KvAppendParams& p) const { return !p.interleaved && c < p.rotary / 16; }
    __device__ __forceinline__ int first(const KvAppendParams& p) const { return apart(p) ? c : 2 * c; }
    __device__ __forceinline__ int second(const KvAppendParams& p) const { return apart(p) ? c + p.rotary / 16 : 2 * c + 1; }
    __device__ __forceinline__ const char* from(const KvAppendParams& p, int row) const {
        const int Hkv = p.ch.Hkv;
        if (head < Hkv) return p.k + row * p.k_ts + head * p.k_hs;
        if (head < 2 * Hkv) return p.v + row * p.v_ts + (head - Hkv) * p.v_hs;
        return p.q + row * p.q_ts + (head - 2 * Hkv) * p.q_hs;
    }
    // nullptr: not stored
    __device__ __forceinline__ char* to(const KvAppendParams& p, const TokenPlace& pl) const {
        const int Hkv = p.ch.Hkv;
        if (head < Hkv) return pl.k_off < 0 ? nullptr : p.kc + pl.k_off + head * p.kc_hs;
        if (head < 2 * Hkv) return pl.v_off < 0 ? nullptr : p.vc + pl.v_off + (head - Hkv) * p.vc_hs;
        return pl.row < 0 ? nullptr : p.q_out + pl.row * p.qo_ts + (head - 2 * Hkv) * p.qo_hs;
    }
    __device__ __forceinline__ bool rotates(const KvAppendParams& p) const {
        return c < p.rotary / 16 && (head < p.ch.Hkv || head >= 2 * p.ch.Hkv);
    }
};

template <int D, bool F16, int BATCH>
__global__ void __launch_bounds__(KA_THREADS, BATCH > 1 ? 4 : 6) kv_append_kernel(const __grid_constant__ KvAppendParams p) {
    __shared__ TokenPlace place[KA_MAX_TOKENS];
    __shared__ int pos_s[KA_MAX_TOKENS];
    __shared__ __align__(16) float2 cs[KA_MAX_TOKENS][KV_MAX_ROTARY / 2];  // (cos, sin)
    const ChunkParams& ch = p.ch;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    launch_dependents();
    const int t0 = blockIdx.x * p.tokens_per_cta;
    const int nt = min(p.tokens_per_cta, ch.T - t0);
    const int heads = (p.q ? p.Hq : 0) + 2 * ch.Hkv, all = nt * heads * (D / 16);

    uint4 w0[BATCH], w1[BATCH];
    const auto load = [&](int x0) {
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int x = x0 + u * KA_THREADS;
            if (x >= all) continue;
            const Pieces<D> m(x, heads);
            const char* src = m.from(p, t0 + m.token);
            w0[u] = ld_once(src + 16 * m.first(p));
            w1[u] = ld_once(src + 16 * m.second(p));
        }
    };
    // The rows are known before their places are: with few tokens the first
    // loads fly while the places are found.
    constexpr bool EARLY = BATCH > 1;
    if (EARLY) load(threadIdx.x);

    if (warp < nt) {
        const int t = t0 + warp;
        const int b = find_sequence(ch.cu, ch.B, t, lane);
        const Chunk s = load_chunk(ch, b);
        const int i = t - s.q0;
        const bool mine = s.rows_ok && i >= 0 && i < s.n;
        int pos = s.ctx + i;
        if (mine && s.ok && ch.parents) {
            const uint32_t set = __shfl_sync(0xFFFFFFFFu, tree_sets(ch, b, s.n, lane), i);
            pos = s.ctx + (set ? __popc(set) - 1 : 0);
        }
        if (lane == 0) {
            TokenPlace pl{-1, -1, mine ? t : -1};
            if (mine && !s.ok) raise_flag(ch.status, SV_FLAG_BAD_LENGTH);
            if (mine && s.ok) {
                const int slot = s.ctx + i;
                const int page = page_of(ch, b, slot);
                if (page >= 0) {
                    const int at = slot % ch.page_size;
                    pl.k_off = page * p.kc_ps + at * p.kc_ts;
                    pl.v_off = page * p.vc_ps + at * p.vc_ts;
                }
            }
            place[warp] = pl;
            pos_s[warp] = p.positions && mine ? p.positions[t] : pos;
        }
    }
    // A sequence whose rows are not where rows can be is flagged, whether or not
    // a token has led to it: the grid's threads look at one each, the last first,
    // whose warps find no places when tokens are few.
    for (int64_t b = (int64_t)blockIdx.x * KA_THREADS + (KA_THREADS - 1 - threadIdx.x); b < ch.B; b += (int64_t)gridDim.x * KA_THREADS)
        if (!load_chunk(ch, (int)b).rows_ok) raise_flag(ch.status, SV_FLAG_BAD_LENGTH);
    __syncthreads();
    const int half = p.rotary / 2;
    for (int x = threadIdx.x; x < nt * (KV_MAX_ROTARY / 2); x += KA_THREADS) {
        const int tk = x / (KV_MAX_ROTARY / 2), i = x % (KV_MAX_ROTARY / 2);
        if (i < half) {
            const uint64_t turns = (uint64_t)(int64_t)pos_s[tk] * p.turns[i];
            float sn, cn;
            sincospif((float)(int32_t)(turns >> 32) * 4.656612873077393e-10f, &sn, &cn);  // 2^-31 half turns
            cs[tk][i] = make_float2(cn, sn);
        }
    }
    __syncthreads();

    for (int x0 = threadIdx.x; x0 < all; x0 += BATCH * KA_THREADS) {
        if (!EARLY || x0 != threadIdx.x) load(x0);
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int x = x0 + u * KA_THREADS;
            if (x >= all) continue;
            const Pieces<D> m(x, heads);
            char* dst = m.to(p, place[m.token]);
            if (!dst) continue;
            uint4 o0 = w0[u], o1 = w1[u];
            if (m.rotates(p)) {
                float a[8], b[8];
                unpack8<F16>(o0, a);
                unpack8<F16>(o1, b);
                const float2* t = cs[m.token] + 8 * m.c;
                if (p.interleaved) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 f = t[i], g = t[4 + i];
                        const float a0 = a[2 * i], a1 = a[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
                        a[2 * i] = a0 * f.x - a1 * f.y, a[2 * i + 1] = a1 * f.x + a0 * f.y;
                        b[2 * i] = b0 * g.x - b1 * g.y, b[2 * i + 1] = b1 * g.x + b0 * g.y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 f = t[i];
                        const float a0 = a[i], b0 = b[i];
                        a[i] = a0 * f.x - b0 * f.y;
                        b[i] = b0 * f.x + a0 * f.y;
                    }
                }
                o0 = pack8<F16>(a);
                o1 = pack8<F16>(b);
            }
            reinterpret_cast<uint4*>(dst)[m.first(p)] = o0;
            reinterpret_cast<uint4*>(dst)[m.second(p)] = o1;
        }
    }
}

template <class K, class P>
static cudaError_t launch_early(K kernel, int grid, int threads, const P& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int BATCH>
static cudaError_t launch_append(const KvAppendParams& p, int f16, cudaStream_t stream) {
    const int grid = (p.ch.T - 1) / p.tokens_per_cta + 1;  // T >= 1, and may be near 2^31
    auto kernel = p.D == 128 ? (f16 ? kv_append_kernel<128, true, BATCH> : kv_append_kernel<128, false, BATCH>)
                             : (f16 ? kv_append_kernel<64, true, BATCH> : kv_append_kernel<64, false, BATCH>);
    return launch_early(kernel, grid, KA_THREADS, p, stream);
}

// Many tokens: several per CTA and one pair of loads per thread at a time, in
// few registers, so that 6 CTAs per SM cover one another's searches. Fewer: as
// many tokens as one batch of loads holds, which then fly while the places are
// found. Measured with 48 heads of 128, the first and the second way, in us:
// 512 tokens 6.5 and 5.4, 1024 11.5 and 7.5, 2560 16.7 and 16.8, 6400 32.3 and
// 35.1, 32000 131 and 140 (6.0 and 5.6 TB/s).
cudaError_t launch_kv_append(const KvAppendParams& in, int f16, int sms, cudaStream_t stream) {
    KvAppendParams p = in;
    const int per_token = ((p.q ? p.Hq : 0) + 2 * p.ch.Hkv) * (p.D / 16);
    const int fit = KA_BATCH * KA_THREADS / per_token;
    if (p.ch.T > KA_MANY * sms) {
        p.tokens_per_cta = KA_MAX_TOKENS / 2;
        return launch_append<1>(p, f16, stream);
    }
    p.tokens_per_cta = p.ch.T <= 4 * sms || fit < 1 ? 1 : fit > KA_MAX_TOKENS ? KA_MAX_TOKENS : fit;
    return launch_append<KA_BATCH>(p, f16, stream);
}

// ---------------------------------------------------------------------------
// Commit. A tree's nodes were appended at slots ctx + node; the kept path
// 0 = p_0 < p_1 < ... < p_n moves to slots ctx + 1 .. ctx + n (keys carry the
// rotation of ctx + depth already). Node p_j >= j, so a place j is never the
// source of a later node: a thread that reads some nodes of its 16 bytes in
// ascending order before it writes them, and then goes on to the next, moves
// the path in place. One CTA per sequence; the bytes are few (2 n Hkv D per
// cache) and the call is bound by its launch and its dependent loads.
// ---------------------------------------------------------------------------
constexpr int KC_THREADS = 256;
constexpr int KC_BATCH = 8;  // 16-byte loads in flight per thread

__global__ void __launch_bounds__(KC_THREADS) kv_commit_kernel(const __grid_constant__ KvCommitParams p) {
    __shared__ int64_t k_from[KV_MAX_TREE], k_to[KV_MAX_TREE], v_from[KV_MAX_TREE], v_to[KV_MAX_TREE];
    __shared__ int moves_s;
    const ChunkParams& ch = p.ch;
    const int lane = threadIdx.x & 31;
    grid_dependency_wait();
    launch_dependents();
    const int b = blockIdx.x;
    if (threadIdx.x < 32) {
        const int ctx = ch.ctx[b], n = p.n_accepted[b];
        const long long room = (long long)ch.max_pages * ch.page_size;
        bool ok = ctx >= 0 && n >= 0 && (long long)ctx + 1 + n <= room && (!ch.parents || n < ch.N);
        if (lane == 0 && n >= 0 && !ok) raise_flag(ch.status, SV_FLAG_BAD_LENGTH);
        int moves = 0;
        if (ok && ch.parents) {
            const int last = p.last_node[b];
            const bool in_tree = last >= 0 && last < ch.N && (long long)ctx + last < room;
            // nodes past the last one are not needed, and may be padding
            const uint32_t set = __shfl_sync(0xFFFFFFFFu, tree_sets(ch, b, in_tree ? last + 1 : 0, lane), in_tree ? last : 0);
            ok = in_tree && __popc(set) == n + 1;
            if (lane == 0 && !ok) raise_flag(ch.status, SV_FLAG_BAD_TREE);
            const int to = __popc(set & ((1u << lane) - 1u));
            bool move = ok && ((set >> lane) & 1u) && to != lane;
            int from_page = 0, to_page = 0;
            if (move) {
                from_page = page_of(ch, b, ctx + lane);
                to_page = page_of(ch, b, ctx + to);
                move = from_page >= 0 && to_page >= 0;
            }
            const uint32_t all = __ballot_sync(0xFFFFFFFFu, move);
            moves = __popc(all);
            if (move) {
                const int at = __popc(all & ((1u << lane) - 1u));
                const int f = (ctx + lane) % ch.page_size, d = (ctx + to) % ch.page_size;
                k_from[at] = from_page * p.kc_ps + f * p.kc_ts;
                k_to[at] = to_page * p.kc_ps + d * p.kc_ts;
                v_from[at] = from_page * p.vc_ps + f * p.vc_ts;
                v_to[at] = to_page * p.vc_ps + d * p.vc_ts;
            }
        }
        if (lane == 0) {
            moves_s = moves;
            p.out_lens[b] = ok ? ctx + 1 + n : ctx;
        }
    }
    __syncthreads();
    const int moves = moves_s;
    const int pieces = p.D / 8, per_cache = ch.Hkv * pieces;
    for (int x = threadIdx.x; moves > 0 && x < 2 * per_cache; x += KC_THREADS) {
        const bool is_v = x >= per_cache;
        const int y = is_v ? x - per_cache : x;
        const int h = y / pieces, c = y % pieces;
        char* base = is_v ? p.vc + h * p.vc_hs + c * 16 : p.kc + h * p.kc_hs + c * 16;
        const int64_t* from = is_v ? v_from : k_from;
        const int64_t* to = is_v ? v_to : k_to;
        for (int j0 = 0; j0 < moves; j0 += KC_BATCH) {
            uint4 w[KC_BATCH];
#pragma unroll
            for (int j = 0; j < KC_BATCH; ++j)
                if (j0 + j < moves) w[j] = *reinterpret_cast<const uint4*>(base + from[j0 + j]);
#pragma unroll
            for (int j = 0; j < KC_BATCH; ++j)
                if (j0 + j < moves) *reinterpret_cast<uint4*>(base + to[j0 + j]) = w[j];
        }
    }
}

cudaError_t launch_kv_commit(const KvCommitParams& p, cudaStream_t stream) {
    return launch_early(kv_commit_kernel, p.ch.B, KC_THREADS, p, stream);
}

}  // namespace sv
