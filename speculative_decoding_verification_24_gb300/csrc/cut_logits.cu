// Rows of logits cut by temperature, top-k, top-p and min-p: a token drawn from
// what is kept, or the row with everything else at -inf.
//
// A row's order is descending by logit, equal ones ascending by index. Each cut
// keeps a beginning of it, so what is kept together is the shortest of the
// three, and one number says what that is: the place of the last kept element,
// (key of its logit, reversed index) as one integer that grows towards the
// row's top. Places are unique, so ties need no care of their own.
//
// Weights w_j = exp((z_j - max) / T) are whole numbers in units of 2^-44, right
// to about 2^-33 of themselves (weight()). Whole numbers add up to the same sum
// in any order, so results do not depend on how a row is split over threads and
// CTAs or on the order of atomics, and a token is the one that the definition
// gives unless its u lies within about 1e-11 of an edge between two tokens. In
// fp32 a sum of 150,000 weights is off by 1e-6, as much as flat rows' edges lie
// apart.
//
// One cluster of CTAs per row; a row lies in their shared memory, read from HBM
// once. Steps, of which a row takes those that its settings need:
//   1. the maximum, and a bound on the k-th largest from the largest of each
//      warp's (or lane group's) part: k parts' maxima lie at or above it;
//   2. the sum of all weights, for top-p without top-k;
//   3. what lies at or above the bound goes to a list in the first CTA, which
//      ranks it by comparing all pairs and applies the cuts there;
//   4. where that is more than the list takes, the place is found by histograms:
//      2048 bins over the places that are possible, the bin in which the count
//      or the weight is reached becomes the next range, until it fits the list;
//   5. the draw, over the list or over the rows' parts by their sums, or the
//      row's output.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <atomic>

#include "cut.h"
#include "paged_device.cuh"

namespace cg = cooperative_groups;

namespace sv {

typedef unsigned long long u64;

constexpr int CL_THREADS = 512;
constexpr int CL_WARPS = CL_THREADS / 32;
constexpr int CL_MAX_CS = 8;
constexpr int CL_BINS = 2048;
constexpr int CL_LIST = 1024;
constexpr int CL_ROUNDS = 5;  // of 11 bits each; a place has 50
constexpr int CL_INDEX_BITS = 18;
constexpr uint32_t CL_INDEX_MASK = (1u << CL_INDEX_BITS) - 1;
constexpr int CL_EXP_BITS = 8;
constexpr int CL_EXP = 1 << CL_EXP_BITS;  // entries of the table of 2^(i / 256)
constexpr int CL_UNIT = 44;               // weights are in units of 2^-44
static_assert((1 << CL_INDEX_BITS) == CUT_MAX_V, "an index per place");

// 2^(i / 256), in weight units and as a float in units of 2^-39.
struct alignas(16) ExpEntry {
    u64 q;
    float f;
    float unused;
};
struct ExpTable {
    ExpEntry e[CL_EXP];
};
constexpr double exp_series(double x) {
    double sum = 1.0, term = 1.0;
    for (int i = 1; i < 30; ++i) {
        term *= x / i;
        sum += term;
    }
    return sum;
}
constexpr ExpTable make_exp_table() {
    ExpTable t = {};
    for (int i = 0; i < CL_EXP; ++i) {
        const double v = exp_series(0.69314718055994530942 * i / CL_EXP);
        t.e[i].q = (u64)(v * (double)(1ull << CL_UNIT) + 0.5);
        t.e[i].f = (float)(v * (double)(1ull << 39));
        t.e[i].unused = 0.0f;
    }
    return t;
}
__device__ const ExpTable g_exp_table = make_exp_table();

// What one row's cluster shares; every CTA has its own copy, written by all.
struct CutShared {
    ExpEntry exp[CL_EXP];
    // histogram; after its rounds the first CTA's list: places in mass, weights in list_w
    u64 mass[CL_BINS];
    union {
        uint32_t count[CL_BINS];
        u64 list_w[CL_LIST];
    };
    float warp_max[CL_MAX_CS * CL_WARPS];
    float group_min[CL_MAX_CS * CL_WARPS];
    u64 cta_mass[2][CL_MAX_CS];      // sums over the cluster's CTAs, two in turn
    uint32_t cta_count[2][CL_MAX_CS];
    u64 warp_mass[CL_WARPS];
    uint32_t warp_count[CL_WARPS];
    u64 seg_mass[CL_MAX_CS];
    uint32_t seg_count[CL_MAX_CS];
    // the bin found by a round, or the place found in the list
    u64 found_mass, found_place;
    uint32_t found_bin, found_above, found_count;
    uint32_t list_n;
    u64 block_mass;
    float bound;
};

struct RowScale {
    float top;       // the row's maximum
    float ch, cl;    // 256 log2(e) / T in two floats
};

__device__ __forceinline__ float elem_of(uint32_t w, int half) { return half ? bf16_hi(w) : bf16_lo(w); }

// Order of floats as unsigned integers; -0 counts as 0.
__device__ __forceinline__ uint32_t key32(float z) {
    const uint32_t b = __float_as_uint(__fadd_rn(z, 0.0f));
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_key32(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
template <bool BF16>
__device__ __forceinline__ uint32_t key_of(float z) { return BF16 ? key32(z) >> 16 : key32(z); }
template <bool BF16>
__device__ __forceinline__ float key_value(uint32_t k) { return from_key32(BF16 ? (k << 16) | ((k >> 15) ? 0u : 0xFFFFu) : k); }
// A place in the row's order. A padding element has key 0 (a negative NaN),
// which no place that is kept has.
__device__ __forceinline__ u64 place_of(uint32_t key, int index) {
    return (u64)key << CL_INDEX_BITS | (CL_INDEX_MASK - (uint32_t)index);
}
constexpr u64 CL_LOWEST = 1ull << CL_INDEX_BITS;  // at or below every real element's place
__device__ __forceinline__ int place_index(u64 p) { return (int)(CL_INDEX_MASK - ((uint32_t)p & CL_INDEX_MASK)); }
__device__ __forceinline__ uint32_t place_key(u64 p) { return (uint32_t)(p >> CL_INDEX_BITS); }

// exp((z - top) / T) in units of 2^-44. With d = z - top in two floats, exactly,
// y = 256 d log2(e) / T = n + x, n whole and |x| <= 1/2: 2^(n / 256) comes from the
// table and a shift, and 2^(x / 256) - 1, below 2^-9, from three terms of its
// series. x is off by 2^-26 and the series by 2^-24 of itself: 2^-33 of w.
__device__ __forceinline__ u64 weight(float z, const RowScale& s, const ExpEntry* table) {
    const float dh = __fsub_rn(z, s.top);
    const float bb = __fsub_rn(dh, z);
    const float dl = __fsub_rn(__fsub_rn(z, __fsub_rn(dh, bb)), __fadd_rn(s.top, bb));
    constexpr float MAGIC = 12582912.0f;  // 1.5 * 2^23: adding it rounds to whole numbers
    const float t = __fmaf_rn(dh, s.ch, MAGIC);
    const float n = __fsub_rn(t, MAGIC);
    const float x = __fadd_rn(__fmaf_rn(dh, s.ch, -n), __fmaf_rn(dh, s.cl, __fmul_rn(dl, s.ch)));
    constexpr float L1 = 2.7076061740622863e-3f;   // ln 2 / 256
    constexpr float L2 = 3.6655655969053526e-6f;   // its square / 2
    constexpr float L3 = 3.3083027270131e-9f;      // its cube / 6
    const float e = __fmul_rn(x, __fmaf_rn(x, __fmaf_rn(x, L3, L2), L1));
    const int ni = __float_as_int(t) - 0x4B400000;
    const ExpEntry en = table[ni & (CL_EXP - 1)];
    const int tail = __float2int_rn(__fmul_rn(en.f, e));  // below 2^30.5
    const u64 q = en.q + (u64)((long long)tail * 32);
    const int sh = -(ni >> CL_EXP_BITS);
    const u64 w = (q + ((1ull << (sh & 63)) >> 1)) >> (sh & 63);
    return t > MAGIC - 46.0f * CL_EXP ? w : 0ull;  // (and where d is -inf)
}

// The elements of one CTA's part of a row, in 16-byte pieces of which a warp has
// a run; lane l has its pieces l, l + 32, ...
template <bool BF16>
struct Part {
    static constexpr int E = BF16 ? 8 : 4;
    const uint4* data;   // shared memory
    int v0, v1;          // this warp's pieces of the part
    int first;           // index in the row of the part's first element (negative: padding)
    __device__ __forceinline__ int index(int v) const { return first + v * E; }
};

template <bool BF16>
__device__ __forceinline__ float piece_elem(const uint4& x, int e) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    return BF16 ? elem_of(w[e >> 1], e & 1) : __uint_as_float(w[e]);
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 t = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += t;
    }
    return v;
}

// Sum of weights and number of elements at or above `cut`, per warp into
// sh.warp_mass / warp_count, and over the cluster.
template <bool BF16>
__device__ __forceinline__ void sum_kept(const Part<BF16>& part, CutShared& sh, const RowScale& s, u64 cut, int lane, int warp,
                                         bool weights, cg::cluster_group& cluster, int CS, int rank, int slot, u64& mass, uint32_t& count) {
    u64 m = 0;
    uint32_t n = 0;
    const uint32_t cut_key = place_key(cut);
    for (int v = part.v0 + lane; v < part.v1; v += 32) {
        const uint4 x = part.data[v];
        const int i0 = part.index(v);
#pragma unroll
        for (int e = 0; e < Part<BF16>::E; ++e) {
            const float z = piece_elem<BF16>(x, e);
            const uint32_t key = key_of<BF16>(z);
            if (key > cut_key || (key == cut_key && place_of(key, i0 + e) >= cut)) {
                ++n;
                if (weights) m += weight(z, s, sh.exp);
            }
        }
    }
    m = warp_sum(m);
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if (lane == 0) {
        sh.warp_mass[warp] = m;
        sh.warp_count[warp] = n;
    }
    __syncthreads();
    if (warp == 0) {
        u64 a = warp_sum(lane < CL_WARPS ? sh.warp_mass[lane] : 0);
        uint32_t c = __reduce_add_sync(0xFFFFFFFFu, lane < CL_WARPS ? sh.warp_count[lane] : 0);
        if (lane < CS) {
            *cluster.map_shared_rank(&sh.cta_mass[slot][rank], lane) = a;
            *cluster.map_shared_rank(&sh.cta_count[slot][rank], lane) = c;
        }
    }
    cluster.sync();
    mass = 0;
    count = 0;
    for (int c = 0; c < CS; ++c) {
        mass += sh.cta_mass[slot][c];
        count += sh.cta_count[slot][c];
    }
}

// Appends the places in [lo, hi] of all parts to the first CTA's list. What does
// not fit is counted only. The list's places lie where the histogram was.
template <bool BF16>
__device__ __forceinline__ uint32_t gather(const Part<BF16>& part, CutShared& sh, u64 lo, u64 hi, int lane, cg::cluster_group& cluster) {
    CutShared* head = cluster.map_shared_rank(&sh, 0);
    const uint32_t lo_key = place_key(lo);
    for (int v = part.v0 + lane; v < part.v1; v += 32) {
        const uint4 x = part.data[v];
        const int i0 = part.index(v);
#pragma unroll
        for (int e = 0; e < Part<BF16>::E; ++e) {
            const uint32_t key = key_of<BF16>(piece_elem<BF16>(x, e));
            if (key < lo_key) continue;
            const u64 p = place_of(key, i0 + e);
            if (p < lo || p > hi) continue;
            const uint32_t at = atomicAdd(&head->list_n, 1u);
            if (at < CL_LIST) head->mass[at] = p;
        }
    }
    cluster.sync();
    return head->list_n;
}

// One round of the search in [lo, hi]: the bin in which the count `k` (by_mass
// false) or the weight `goal` is reached from above, given what lies above hi.
// The range becomes that bin.
template <bool BF16, bool BY_MASS>
__device__ __forceinline__ uint32_t narrow(const Part<BF16>& part, CutShared& sh, const RowScale& s, u64& lo, u64& hi, uint32_t& above,
                                           u64& mass_above, uint32_t k, double goal, int lane, int warp, cg::cluster_group& cluster,
                                           int CS, int rank) {
    const int tid = threadIdx.x;
    const u64 width = hi - lo;  // one less than the places
    const int bits = 64 - __clzll((long long)width);
    const int shift = width == 0 ? 0 : max(0, bits - 11);
    for (int i = tid; i < CL_BINS; i += CL_THREADS) {
        sh.count[i] = 0;
        if (BY_MASS) sh.mass[i] = 0;
    }
    __syncthreads();
    const uint32_t lo_key = place_key(lo);
    for (int v = part.v0 + lane; v < part.v1; v += 32) {
        const uint4 x = part.data[v];
        const int i0 = part.index(v);
#pragma unroll
        for (int e = 0; e < Part<BF16>::E; ++e) {
            const float z = piece_elem<BF16>(x, e);
            const uint32_t key = key_of<BF16>(z);
            if (key < lo_key) continue;
            const u64 p = place_of(key, i0 + e);
            if (p < lo || p > hi) continue;
            const int bin = (int)((p - lo) >> shift);
            atomicAdd(&sh.count[bin], 1u);
            if (BY_MASS) atomicAdd(&sh.mass[bin], weight(z, s, sh.exp));
        }
    }
    cluster.sync();
    // A CTA adds up its share of the bins over all CTAs; a thread has `per`
    // neighbouring ones.
    const int seg = CL_BINS / CS, per = max(1, seg / CL_THREADS);
    const int b0 = rank * seg + tid * per;
    const bool on = tid * per < seg;
    uint32_t c_of[4] = {0, 0, 0, 0}, c_sum = 0;  // seg / 512 <= 4
    u64 m_of[4] = {0, 0, 0, 0}, m_sum = 0;
    if (on) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= per) break;
            for (int c = 0; c < CS; ++c) {
                const CutShared* o = cluster.map_shared_rank(&sh, c);
                c_of[i] += o->count[b0 + i];
                if (BY_MASS) m_of[i] += o->mass[b0 + i];
            }
            c_sum += c_of[i];
            m_sum += m_of[i];
        }
    }
    // inclusive sums from this thread's bins upwards within the share
    uint32_t c_in = c_sum;
    u64 m_in = m_sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t ct = __shfl_down_sync(0xFFFFFFFFu, c_in, o);
        const u64 mt = BY_MASS ? __shfl_down_sync(0xFFFFFFFFu, m_in, o) : 0;
        if (lane + o < 32) {
            c_in += ct;
            m_in += mt;
        }
    }
    if (lane == 0) {
        sh.warp_count[warp] = c_in;
        sh.warp_mass[warp] = m_in;
    }
    __syncthreads();
    for (int w = warp + 1; w < CL_WARPS; ++w) {
        c_in += sh.warp_count[w];
        m_in += sh.warp_mass[w];
    }
    if (tid == 0) {
        for (int c = 0; c < CS; ++c) {
            *cluster.map_shared_rank(&sh.seg_count[rank], c) = c_in;
            *cluster.map_shared_rank(&sh.seg_mass[rank], c) = m_in;
        }
    }
    cluster.sync();
    uint32_t c_up = above;
    u64 m_up = mass_above;
    for (int c = rank + 1; c < CS; ++c) {
        c_up += sh.seg_count[c];
        m_up += sh.seg_mass[c];
    }
    if (on) {
        // what lies above this thread's bins
        uint32_t c = c_up + c_in - c_sum;
        u64 m = m_up + m_in - m_sum;
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            if (i >= per) continue;
            const bool reached = BY_MASS ? (double)(m + m_of[i]) >= goal : c + c_of[i] >= k;
            const bool before = BY_MASS ? (c != 0 && (double)m >= goal) : c >= k;
            if (c_of[i] != 0 && reached && !before) {
                for (int d = 0; d < CS; ++d) {
                    CutShared* o = cluster.map_shared_rank(&sh, d);
                    o->found_bin = (uint32_t)(b0 + i);
                    o->found_above = c;
                    o->found_mass = m;
                    o->found_count = c_of[i];
                }
            }
            c += c_of[i];
            m += m_of[i];
        }
    }
    cluster.sync();
    above = sh.found_above;
    mass_above = sh.found_mass;
    const u64 bin = sh.found_bin;
    const u64 new_lo = lo + (bin << shift);
    hi = min(hi, new_lo + ((1ull << shift) - 1));
    lo = new_lo;
    return sh.found_count;
}

// The place of the last element that a cut keeps: the search narrows [lo, hi]
// until what is left fits the list, and the first CTA picks it there.
template <bool BF16, bool BY_MASS>
__device__ __noinline__ u64 find_cut(const Part<BF16>& part, CutShared& sh, const RowScale& s, u64 lo, u64 hi, uint32_t k, double goal,
                                     int lane, int warp, int CS, int rank, uint32_t& kept) {
    cg::cluster_group cluster = cg::this_cluster();
    uint32_t above = 0, left = CL_LIST + 1;
    u64 mass_above = 0;
    for (int round = 0; round < CL_ROUNDS && left > CL_LIST; ++round)
        left = narrow<BF16, BY_MASS>(part, sh, s, lo, hi, above, mass_above, k, goal, lane, warp, cluster, CS, rank);
    if (threadIdx.x == 0) {
        sh.list_n = 0;
        sh.found_place = lo;
    }
    cluster.sync();  // (also: every CTA has read the histograms, on which the list goes)
    const uint32_t n = min(gather<BF16>(part, sh, lo, hi, lane, cluster), (uint32_t)CL_LIST);
    if (rank == 0) {
        if (BY_MASS) {
            for (int i = threadIdx.x; i < (int)n; i += CL_THREADS) sh.list_w[i] = weight(key_value<BF16>(place_key(sh.mass[i])), s, sh.exp);
            __syncthreads();
        }
        for (int i = threadIdx.x; i < (int)n; i += CL_THREADS) {
            const u64 mine = sh.mass[i];
            uint32_t c = above;
            u64 m = mass_above;
            for (int j = 0; j < (int)n; ++j) {
                if (sh.mass[j] > mine) {
                    ++c;
                    if (BY_MASS) m += sh.list_w[j];
                }
            }
            const bool reached = BY_MASS ? (double)(m + sh.list_w[i]) >= goal : c + 1 == k;
            const bool before = BY_MASS ? (c != 0 && (double)m >= goal) : false;
            if (reached && !before) {
                for (int d = 0; d < CS; ++d) {
                    CutShared* o = cluster.map_shared_rank(&sh, d);
                    o->found_place = mine;
                    o->found_count = c + 1;
                }
            }
        }
    }
    cluster.sync();
    kept = sh.found_count;
    return sh.found_place;
}

__device__ __forceinline__ u64 block_sum(u64 v, CutShared& sh, int lane, int warp) {
    v = warp_sum(v);
    __syncthreads();
    if (lane == 0) sh.warp_mass[warp] = v;
    __syncthreads();
    u64 t = 0;
#pragma unroll
    for (int w = 0; w < CL_WARPS; ++w) t += sh.warp_mass[w];
    return t;
}

// The largest whole number below or at u of `total`, below total.
__device__ __forceinline__ u64 draw_target(float u, u64 total) {
    const double x = (u > 0.0f ? (double)fminf(u, 1.0f) : 0.0) * (double)total;
    const u64 t = (u64)x;
    return t < total ? t : total - 1;
}

__device__ __forceinline__ void put_token(const CutParams& P, int64_t row, int index, float z, const RowScale& s, double inv_t, u64 total) {
    P.tokens[row] = index;
    if (P.logprobs)
        P.logprobs[row] = (float)(((double)z - (double)s.top) * inv_t - log((double)total * (1.0 / (double)(1ull << CL_UNIT))));
}

template <bool BF16, bool DRAW>
__global__ void __launch_bounds__(CL_THREADS, 2) cut_logits_kernel(const __grid_constant__ CutParams P) {
    cluster_arrive_started();
    cg::cluster_group cluster = cg::this_cluster();
    const int CS = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    extern __shared__ __align__(16) char smem[];
    CutShared& sh = *reinterpret_cast<CutShared*>(smem);
    uint4* data = reinterpret_cast<uint4*>(smem + sizeof(CutShared));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    using Pt = Part<BF16>;
    constexpr int ES = BF16 ? 2 : 4;

    const int64_t row = blockIdx.x / CS;
    const int b = (int)(row / P.R), r = (int)(row - (int64_t)b * P.R);
    const char* src = P.logits + b * P.seq_bytes + r * P.row_bytes;
    const int lead = (int)(reinterpret_cast<uintptr_t>(src) & 15) / ES;  // elements before the row in its first piece
    const char* base = src - lead * ES;
    const int pieces = (lead + P.V + Pt::E - 1) / Pt::E;
    const int begin = min(rank * P.slice_vecs, pieces), n_vecs = min(P.slice_vecs, pieces - begin);
    Pt part;
    part.data = data;
    part.v0 = min(warp * P.warp_vecs, n_vecs);
    part.v1 = min(part.v0 + P.warp_vecs, n_vecs);
    part.first = begin * Pt::E - lead;
    if (tid == 0) sh.list_n = 0;

    grid_dependency_wait();
    launch_dependents();

    // 1. This lane's pieces on their way to shared memory; a piece that the row
    // fills in part goes by elements, with -inf beside them for now.
    const auto partial = [&](int i0) { return i0 < 0 || i0 + Pt::E > P.V; };
    for (int v = part.v0 + lane; v < part.v1; v += 32) {
        const int i0 = part.index(v);
        if (!partial(i0)) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(data + v)), "l"(base + (int64_t)(begin + v) * 16) : "memory");
        } else {
#pragma unroll
            for (int e = 0; e < Pt::E; ++e) {
                const bool in = i0 + e >= 0 && i0 + e < P.V;
                if constexpr (BF16) {
                    reinterpret_cast<uint16_t*>(data + v)[e] = in ? *reinterpret_cast<const uint16_t*>(src + (int64_t)(i0 + e) * 2) : (uint16_t)0xFF80u;
                } else {
                    reinterpret_cast<uint32_t*>(data + v)[e] = in ? *reinterpret_cast<const uint32_t*>(src + (int64_t)(i0 + e) * 4) : 0xFF800000u;
                }
            }
        }
    }
    if (tid < CL_EXP)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(&sh.exp[tid])), "l"(&g_exp_table.e[tid]) : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");

    const float T = P.temperatures ? P.temperatures[b] : P.temperature;
    const int top_k = P.top_ks ? P.top_ks[b] : P.top_k;
    const float top_p = P.top_ps ? P.top_ps[b] : P.top_p, min_p = P.min_ps ? P.min_ps[b] : P.min_p;
    const bool settings_ok = (T == 0.0f || (T >= 0x1p-64f && T <= 0x1p64f)) && top_k >= 0 && top_p >= 0.0f && top_p <= 1.0f &&
                             min_p >= 0.0f && min_p <= 1.0f;
    const int k = T == 0.0f ? 1 : top_k > 0 && top_k < P.V ? top_k : P.V;
    const double inv_t = T == 0.0f ? 1.0 : 1.0 / (double)T;

    asm volatile("cp.async.wait_group 0;" ::: "memory");
    float top = -INFINITY;
    for (int v = part.v0 + lane; v < part.v1; v += 32) {
        const uint4 x = data[v];
        if constexpr (BF16) {
            const uint32_t m = max_nan_bf16x2(max_nan_bf16x2(x.x, x.y), max_nan_bf16x2(x.z, x.w));
            top = max_nan(top, max_nan(bf16_lo(m), bf16_hi(m)));
        } else {
            top = max_nan(top, max_nan(max_nan(__uint_as_float(x.x), __uint_as_float(x.y)), max_nan(__uint_as_float(x.z), __uint_as_float(x.w))));
        }
    }
    for (int v = part.v0 + lane; v < part.v1; v += 32) {  // padding leaves the order
        const int i0 = part.index(v);
        if (!partial(i0)) continue;
        for (int e = 0; e < Pt::E; ++e) {
            if (i0 + e >= 0 && i0 + e < P.V) continue;
            if constexpr (BF16) reinterpret_cast<uint16_t*>(data + v)[e] = 0xFFFFu;
            else reinterpret_cast<uint32_t*>(data + v)[e] = 0xFFFFFFFFu;
        }
    }
    // groups of 32 or fewer lanes, at least k of them where there are as many lanes
    const int warps = CS * CL_WARPS;
    int group = 32;
    while (group > 1 && warps * (32 / group) < k) group >>= 1;
    float gmin = top;
    float wmax = top;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        if (o == group) gmin = wmax;
        wmax = max_nan(wmax, __shfl_xor_sync(0xFFFFFFFFu, wmax, o));
    }
    if (group == 32) gmin = wmax;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) gmin = fminf(gmin, __shfl_xor_sync(0xFFFFFFFFu, gmin, o));
    cluster_wait_started();
    if (lane < CS) {
        cluster.map_shared_rank(sh.warp_max, lane)[rank * CL_WARPS + warp] = wmax;
        cluster.map_shared_rank(sh.group_min, lane)[rank * CL_WARPS + warp] = gmin;
    }
    cluster.sync();
    RowScale s;
    s.top = -INFINITY;
    float least = INFINITY;
    for (int w = lane; w < warps; w += 32) {
        s.top = max_nan(s.top, sh.warp_max[w]);
        least = fminf(least, sh.group_min[w]);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        s.top = max_nan(s.top, __shfl_xor_sync(0xFFFFFFFFu, s.top, o));
        least = fminf(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
    }
    const bool row_ok = s.top < INFINITY && s.top > -INFINITY;
    const int64_t out_row = row;
    u64 cut = CL_LOWEST;  // what is kept lies at or above it
    uint32_t kept = 0;
    if (!row_ok || !settings_ok) {
        if (rank == 0 && tid == 0) {
            raise_flag(P.status, (row_ok ? 0u : (uint32_t)SV_FLAG_BAD_ROW) | (settings_ok ? 0u : (uint32_t)SV_FLAG_BAD_SETTING));
            if constexpr (DRAW) {
                P.tokens[out_row] = -1;
                if (P.logprobs) P.logprobs[out_row] = __int_as_float(0x7fc00000);
            }
        }
        if constexpr (DRAW) return;
        if (!DRAW && rank == 0 && tid == 0 && P.n_kept) P.n_kept[out_row] = -1;
    } else {
        const double c = 1.4426950408889634 * CL_EXP * inv_t;
        s.ch = (float)c;
        s.cl = (float)(c - (double)s.ch);
        const u64 highest = (u64)key_of<BF16>(s.top) << CL_INDEX_BITS | CL_INDEX_MASK;
        // min-p: z >= max + T ln(min_p)
        if (min_p > 0.0f && T != 0.0f) {
            const float z = __double2float_ru((double)s.top + (double)T * log((double)min_p));
            // bf16 keys of negative values end in ones, those of others in zeros
            const uint32_t kz = key32(z), key = !BF16 ? kz : (kz >> 31) ? (uint32_t)(((u64)kz + 0xFFFFu) >> 16) : kz >> 16;
            cut = max(cut, (u64)key << CL_INDEX_BITS);
        }
        const bool by_k = k < P.V, by_p = T != 0.0f && top_p < 1.0f;
        bool listed = false;   // the first CTA's list holds what may be kept
        if (by_k) {
            // 3. the list, if it takes everything at or above the bound
            u64 bound = CL_LOWEST;
            if (k <= warps) {
                // the k-th largest of the warps' maxima
                if (tid < warps) {
                    const float mine = sh.warp_max[tid];
                    int before = 0;
                    for (int w = 0; w < warps; ++w) {
                        const float other = sh.warp_max[w];
                        before += other > mine || (other == mine && w < tid);
                    }
                    if (before == k - 1) sh.bound = mine;
                }
                __syncthreads();
                least = sh.bound;
            }
            if (k <= warps * 32) bound = max(bound, (u64)key_of<BF16>(least) << CL_INDEX_BITS);
            // (what min-p drops counts too: it is among the k)
            const uint32_t n = gather<BF16>(part, sh, bound, highest, lane, cluster);
            listed = n <= CL_LIST;
            if (!listed) {
                uint32_t n_k;
                const u64 cut_k = find_cut<BF16, false>(part, sh, s, bound, highest, (uint32_t)k, 0.0, lane, warp, CS, rank, n_k);
                if (k <= CL_LIST) {
                    if (tid == 0) sh.list_n = 0;  // (every CTA has read it)
                    cluster.sync();
                    gather<BF16>(part, sh, cut_k, highest, lane, cluster);
                    listed = true;
                } else {
                    if (by_p) {
                        u64 mass;
                        uint32_t n_all;
                        sum_kept<BF16>(part, sh, s, cut_k, lane, warp, true, cluster, CS, rank, 0, mass, n_all);
                        uint32_t n_p;
                        cut = max(cut, find_cut<BF16, true>(part, sh, s, cut_k, highest, 0, (double)top_p * (double)mass, lane, warp, CS, rank, n_p));
                    }
                    cut = max(cut, cut_k);
                }
            }
        } else if (by_p) {
            u64 mass;
            uint32_t n_all;
            sum_kept<BF16>(part, sh, s, CL_LOWEST, lane, warp, true, cluster, CS, rank, 0, mass, n_all);
            // weights below (1 - p) / V of the sum cannot be among the kept:
            // all of them together are less than what may be left out
            const double share = (1.0 - (double)top_p) * (double)mass / ((double)P.V * (double)(1ull << CL_UNIT));
            const float z = __double2float_rd((double)s.top + (double)(T == 0.0f ? 1.0f : T) * (log(share) * 1.000001 - 0.001));
            const u64 lo = max(CL_LOWEST, (u64)key_of<BF16>(z) << CL_INDEX_BITS);
            uint32_t n_p;
            cut = max(cut, find_cut<BF16, true>(part, sh, s, min(lo, highest), highest, 0, (double)top_p * (double)mass, lane, warp, CS, rank, n_p));
        }
        if (listed) {
            // The cuts, in the list: an element's rank and the weights before it.
            cluster.sync();  // every CTA has read the list's length
            if (rank == 0) {
                const int n = (int)min(sh.list_n, (uint32_t)CL_LIST);
                for (int i = tid; i < n; i += CL_THREADS) sh.list_w[i] = weight(key_value<BF16>(place_key(sh.mass[i])), s, sh.exp);
                __syncthreads();
                uint32_t before[CL_LIST / CL_THREADS];
                u64 mass_before[CL_LIST / CL_THREADS];
                u64 of_k = 0;
#pragma unroll
                for (int q = 0; q < CL_LIST / CL_THREADS; ++q) {
                    const int i = tid + q * CL_THREADS;
                    before[q] = 0;
                    mass_before[q] = 0;
                    if (i >= n) continue;
                    const u64 mine = sh.mass[i];
                    for (int j = 0; j < n; ++j) {
                        if (sh.mass[j] > mine) {
                            ++before[q];
                            mass_before[q] += sh.list_w[j];
                        }
                    }
                    if (before[q] < (uint32_t)k) of_k += sh.list_w[i];
                }
                of_k = block_sum(of_k, sh, lane, warp);
                const double goal = (double)top_p * (double)of_k;
                u64 lowest = ~0ull;
                bool keep[CL_LIST / CL_THREADS];
#pragma unroll
                for (int q = 0; q < CL_LIST / CL_THREADS; ++q) {
                    const int i = tid + q * CL_THREADS;
                    keep[q] = i < n && before[q] < (uint32_t)k && sh.mass[i] >= cut &&
                              (!by_p || before[q] == 0 || (double)mass_before[q] < goal);
                    if (keep[q]) lowest = min(lowest, sh.mass[i]);
                }
                // the last kept place
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) lowest = min(lowest, __shfl_xor_sync(0xFFFFFFFFu, lowest, o));
                __syncthreads();
                if (lane == 0) sh.warp_mass[warp] = lowest;
                __syncthreads();
                for (int w = 0; w < CL_WARPS; ++w) lowest = min(lowest, sh.warp_mass[w]);
                if constexpr (DRAW) {
                    u64 total = 0;
#pragma unroll
                    for (int q = 0; q < CL_LIST / CL_THREADS; ++q)
                        if (keep[q]) total += sh.list_w[tid + q * CL_THREADS];
                    total = block_sum(total, sh, lane, warp);
                    const u64 target = draw_target(P.uniforms[out_row], total);
#pragma unroll
                    for (int q = 0; q < CL_LIST / CL_THREADS; ++q) {
                        if (!keep[q]) continue;
                        const int i = tid + q * CL_THREADS;
                        const u64 mine = sh.mass[i];
                        const int index = place_index(mine);
                        u64 m = 0;
                        for (int j = 0; j < n; ++j)
                            if (sh.mass[j] >= lowest && place_index(sh.mass[j]) < index) m += sh.list_w[j];
                        if (m <= target && target < m + sh.list_w[i])
                            put_token(P, out_row, index, key_value<BF16>(place_key(mine)), s, inv_t, total);
                    }
                } else if (tid < CS) {
                    *cluster.map_shared_rank(&sh.found_place, tid) = lowest;
                }
            }
            if constexpr (DRAW) return;
            cluster.sync();
            cut = sh.found_place;
        }
        if constexpr (DRAW) {
            // 5. the draw over the parts: their sums, then the warps', then the elements
            u64 total;
            uint32_t n_all;
            sum_kept<BF16>(part, sh, s, cut, lane, warp, true, cluster, CS, rank, 1, total, n_all);
            u64 target = draw_target(P.uniforms[out_row], total);
            u64 before = 0;
            for (int c2 = 0; c2 < rank; ++c2) before += sh.cta_mass[1][c2];
            if (before > target || target >= before + sh.cta_mass[1][rank]) return;
            for (int w = 0; w < warp; ++w) before += sh.warp_mass[w];
            if (before > target || target >= before + sh.warp_mass[warp]) return;
            const uint32_t cut_key = place_key(cut);
            for (int v0 = part.v0; v0 < part.v1; v0 += 32) {
                const int v = v0 + lane;
                u64 w_of[Pt::E], mine = 0;
                uint4 x = make_uint4(0, 0, 0, 0);
                if (v < part.v1) x = data[v];
#pragma unroll
                for (int e = 0; e < Pt::E; ++e) {
                    const float z = piece_elem<BF16>(x, e);
                    const uint32_t key = key_of<BF16>(z);
                    const bool in = v < part.v1 && (key > cut_key || (key == cut_key && place_of(key, part.index(v) + e) >= cut));
                    w_of[e] = in ? weight(z, s, sh.exp) : 0;
                    mine += w_of[e];
                }
                const u64 incl = warp_scan(mine, lane);
                u64 at = before + incl - mine;
                before += __shfl_sync(0xFFFFFFFFu, incl, 31);
                if (target >= before) continue;
                if (at <= target && target < at + mine) {
#pragma unroll
                    for (int e = 0; e < Pt::E; ++e) {
                        if (at <= target && target < at + w_of[e]) put_token(P, out_row, part.index(v) + e, piece_elem<BF16>(x, e), s, inv_t, total);
                        at += w_of[e];
                    }
                }
                return;
            }
            return;
        }
    }
    if constexpr (!DRAW) {
        // 5. the row's output
        const bool valid = row_ok && settings_ok;
        char* out = P.out + b * P.out_seq_bytes + r * P.out_row_bytes;
        const bool same = (reinterpret_cast<uintptr_t>(out) & 15) == (uintptr_t)(lead * ES);
        const uint32_t cut_key = valid ? place_key(cut) : 1u;
        if (!valid) cut = CL_LOWEST;
        for (int v = part.v0 + lane; v < part.v1; v += 32) {
            uint4 x = data[v];
            const int i0 = part.index(v);
            uint32_t keep = 0;
#pragma unroll
            for (int e = 0; e < Pt::E; ++e) {
                const uint32_t key = key_of<BF16>(piece_elem<BF16>(x, e));
                if (!valid || key > cut_key || (key == cut_key && place_of(key, i0 + e) >= cut)) keep |= 1u << e;
            }
            const bool whole = !partial(i0);
            if (!whole) {  // padding is nobody's
                for (int e = 0; e < Pt::E; ++e)
                    if (i0 + e < 0 || i0 + e >= P.V) keep &= ~(1u << e);
            }
            kept += __popc(keep);
            uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
            for (int e = 0; e < Pt::E; ++e) {
                if (keep >> e & 1u) continue;
                if constexpr (BF16) w[e / 2] = e % 2 ? (w[e / 2] & 0xFFFFu) | 0xFF800000u : (w[e / 2] & 0xFFFF0000u) | 0xFF80u;
                else w[e] = 0xFF800000u;
            }
            if (whole && same) {
                *reinterpret_cast<uint4*>(out + (int64_t)i0 * ES) = x;
            } else {
#pragma unroll
                for (int e = 0; e < Pt::E; ++e) {
                    if (i0 + e < 0 || i0 + e >= P.V) continue;
                    if constexpr (BF16) reinterpret_cast<uint16_t*>(out)[i0 + e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
                    else reinterpret_cast<uint32_t*>(out)[i0 + e] = w[e];
                }
            }
        }
        if (P.n_kept && valid) {
            kept = __reduce_add_sync(0xFFFFFFFFu, kept);
            __syncthreads();
            if (lane == 0) sh.warp_count[warp] = kept;
            __syncthreads();
            if (tid == 0) {
                uint32_t n = 0;
                for (int w = 0; w < CL_WARPS; ++w) n += sh.warp_count[w];
                *cluster.map_shared_rank(&sh.cta_count[1][rank], 0) = n;
            }
            cluster.sync();
            if (rank == 0 && tid == 0) {
                uint32_t n = 0;
                for (int c = 0; c < CS; ++c) n += sh.cta_count[1][c];
                P.n_kept[out_row] = (int32_t)n;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Launch.
// ---------------------------------------------------------------------------
// Shared memory per CTA up to which two are resident per SM.
constexpr int CL_TWO = 112 * 1024;
constexpr int CL_ONE = 226 * 1024;

template <bool BF16, bool DRAW>
static cudaError_t launch(CutParams p, int sms, cudaStream_t stream) {
    auto kernel = cut_logits_kernel<BF16, DRAW>;
    static std::atomic<int> attr_done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_done[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, CL_ONE);
        if (e != cudaSuccess) return e;
        attr_done[dev].store(1, std::memory_order_release);
    }
    constexpr int E = BF16 ? 8 : 4;
    const int64_t rows = (int64_t)p.B * p.R;
    const int vecs = (p.V + E - 1) / E + 1;  // (a row may begin inside a piece)
    const auto smem_of = [&](int cs) { return (int)sizeof(CutShared) + (vecs + cs - 1) / cs * 16; };
    int cs = 1;
    while (cs < CL_MAX_CS && smem_of(cs) > CL_TWO) cs *= 2;
    // few rows are spread over more SMs, down to 4 pieces per thread
    while (cs < CL_MAX_CS && rows * cs * 2 <= sms && vecs / cs > 4 * CL_THREADS) cs *= 2;
    p.slice_vecs = (vecs + cs - 1) / cs;
    p.warp_vecs = (p.slice_vecs + CL_WARPS - 1) / CL_WARPS;
    const int smem = smem_of(cs);
    if (smem > CL_ONE || rows * cs > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3((unsigned)(rows * cs), 1, 1);
    cfg.blockDim = dim3(CL_THREADS, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cs;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

cudaError_t launch_cut_logits(CutParams p, int dtype, bool draw, int sms, cudaStream_t stream) {
    if (dtype == SV_BF16) return draw ? launch<true, true>(p, sms, stream) : launch<true, false>(p, sms, stream);
    return draw ? launch<false, true>(p, sms, stream) : launch<false, false>(p, sms, stream);
}

}  // namespace sv
