// Rows of logits cut by temperature, top-k, top-p and min-p: a token drawn from
// what is kept, or the row with everything else at -inf.
//
// A row's order is descending by logit, equal ones ascending by index. Each cut
// keeps a beginning of it, so what is kept together is the shortest of the
// three, and one number says what that is: the place of the last kept element,
// (key of its logit, reversed index) as one integer that grows towards the
// row's top. Places are unique, so ties need no care of their own.
//
// Weights w_j = exp((z_j - max) / T) are whole numbers (weight()) wherever a place is
// decided, in the finest unit that the row's sum leaves room for: right to 2^-40 of
// themselves. Whole numbers add up to the same sum in any order, whatever the order of
// atomics. Sums over whole rows are first formed in floats with their rounding errors
// kept (WeightSum), in an order that the row's split over threads alone gives, and
// decide where what they may be off by leaves no doubt; a row in thousands is summed
// once more in whole numbers. So a call's results do not depend on timing, and a token
// is the one that the definition gives unless its u lies within 1e-11 of an edge
// between two tokens. In plain fp32 a sum of 150,000 weights is off by 1e-6, as much as
// flat rows' edges lie apart.
//
// A row goes to one CTA, or, where rows are few, to a cluster of up to 8. It is
// read from HBM once, and of every 16 bytes the largest logit's key (16 bits) is
// kept in shared memory: whatever looks for large elements afterwards reads those
// keys, and from L2 only the pieces that hold some. Steps, of which a row takes
// those that its settings need:
//   1. the maximum and the pieces' keys;
//   2. top-k: a bound on the k-th largest element (k pieces' maxima lie at or
//      above it, by ranking the warps' maxima or a histogram of the pieces'); what
//      lies at or above it goes to the first CTA's list, which sorts it and
//      applies all cuts there;
//   3. top-p alone: the list gets a few hundred of the row's largest, and the sum of
//      all weights in fp32 often shows already where among them p of it is reached.
//      Else a histogram of log weights says nearly where; then the sum above that
//      region, whose elements go to the list, where the place is found;
//   4. where a list overflows (thousands of equal logits, k in the thousands) the
//      place is found by exact histograms over shrinking ranges of places;
//   5. the draw, over the sorted list or over the warps' parts by their sums and
//      then in one of them, once more by exact sums next to an edge; or the row's
//      output: pieces whose key lies below the cut are written as -inf without another
//      look.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <atomic>
#include <cstddef>

#include "cut.h"
#include "paged_device.cuh"
#include "cut_weights.cuh"

namespace cg = cooperative_groups;

namespace sv {

constexpr int CL_THREADS = 512;
constexpr int CL_WARPS = CL_THREADS / 32;
constexpr int CL_MAX_CS = 8;
constexpr int CL_BINS = 2048;
constexpr int CL_LIST = 2048;
constexpr int CL_GROUPS = 256;
constexpr uint32_t CL_NEAR = 150;  // elements on either side of where a histogram finds a border
constexpr int CL_HITS = 2048;  // pieces of one CTA that gather() reads in one step
constexpr int CL_ROUNDS = 5;   // of 11 bits each; a place has 50
constexpr int CL_INDEX_BITS = 18;
constexpr uint32_t CL_INDEX_MASK = (1u << CL_INDEX_BITS) - 1;
static_assert((1 << CL_INDEX_BITS) == CUT_MAX_V, "an index per place");

__device__ const ExpTable g_exp_table = make_exp_table();

// Order of floats as unsigned integers; -0 counts as 0.
__device__ __forceinline__ uint32_t key32(float z) {
    const uint32_t u = __float_as_uint(z), b = u == 0x80000000u ? 0u : u;
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
    return (u64)key << CL_INDEX_BITS | ((CL_INDEX_MASK - (uint32_t)index) & CL_INDEX_MASK);
}
constexpr u64 CL_LOWEST = 1ull << CL_INDEX_BITS;  // at or below every real element's place
__device__ __forceinline__ int place_index(u64 p) { return (int)(CL_INDEX_MASK - ((uint32_t)p & CL_INDEX_MASK)); }
__device__ __forceinline__ uint32_t place_key(u64 p) { return (uint32_t)(p >> CL_INDEX_BITS); }

// What one row's cluster shares; every CTA has its own copy.
struct alignas(16) CutShared {
    ExpEntry exp[CL_EXP];
    ExpEntry copies[CL_EXP * CL_COPIES];  // of it, where a row's weights are summed
    u64 list[CL_LIST];               // the first CTA's: places, sorted later; or the exact histogram's weights
    union {
        uint32_t count[CL_BINS];     // histogram
        uint32_t hits[CL_HITS];      // pieces to read
    };
    u64 part_mass[CL_MAX_CS * CL_WARPS];  // weights of every warp's part, in the first CTA
    u64 part_all[CL_MAX_CS * CL_WARPS];
    float group_max[CL_GROUPS];  // of lanes, whose pieces' maxima they are
    float lane_min[CL_MAX_CS * CL_WARPS];
    u64 warp_mass[CL_WARPS];
    uint32_t warp_count[CL_WARPS];
    float warp_value[CL_WARPS];
    u64 seg_mass[CL_MAX_CS];
    uint32_t seg_count[CL_MAX_CS];
    // what a search has found, told to every CTA
    u64 found_mass, found_place, draw_at, draw_before;
    uint32_t found_bin, found_from, found_to, found_above, found_count, draw_warp, drawn;
    uint32_t list_n, hits_n, counts[CL_MAX_CS];
    float bound;
    int first_largest, firsts[CL_MAX_CS], sequence;
    // This CTA's part of the row. (Here and not in every thread's registers: 64 are
    // what two CTAs per SM leave a thread, and the sums' loops need them.)
    const char* src;       // the row's first element
    const uint4* base;     // the part's pieces in memory
    int V, first;          // index in the row of the part's first element (negative: padding)
    int n_vecs, slice, run;  // pieces of the part; per CTA and per warp
    int full0, full1;      // those that lie in the row as a whole
    int CS, rank;
    RowScale s;
    // of the row's settings (formed by one thread: the units for doubles are few)
    double inv_t, log_sum;
    float ch, cl, low_by, min_hi, min_lo;
};
// (read and cleared 16 bytes at a time, like the pieces' keys behind the struct)
static_assert(sizeof(CutShared) % 16 == 0 && offsetof(CutShared, list) % 16 == 0 && offsetof(CutShared, count) % 16 == 0 &&
                  offsetof(CutShared, group_max) % 16 == 0, "alignment");

template <bool BF16>
__device__ __forceinline__ float piece_elem(const uint4& x, int e) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    return BF16 ? (e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1])) : __uint_as_float(w[e]);
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
template <class N>
__device__ __forceinline__ N warp_scan(N v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const N t = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += t;
    }
    return v;
}

// A piece that the row src[0..V) fills in part, from index i0 on, `pad` (an
// element's bits) beside it.
template <bool BF16>
__device__ __noinline__ uint4 load_part(const char* src, int V, int i0, uint32_t pad) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < (BF16 ? 8 : 4); ++e) {
        uint32_t b = pad;
        if (i0 + e >= 0 && i0 + e < V)
            b = BF16 ? *reinterpret_cast<const uint16_t*>(src + (int64_t)(i0 + e) * 2) : *reinterpret_cast<const uint32_t*>(src + (int64_t)(i0 + e) * 4);
        if (BF16) w[e / 2] |= b << (16 * (e % 2));
        else w[e] = b;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One CTA's part of a row, in 16-byte pieces of which a warp has a run; lane l
// has its pieces l, l + 32, ...
template <bool BF16>
struct Row {
    static constexpr int E = BF16 ? 8 : 4;
    static constexpr int ES = BF16 ? 2 : 4;
    CutShared* sh;
    int lane, warp;

    __device__ __forceinline__ int CS() const { return sh->CS; }
    __device__ __forceinline__ int rank() const { return sh->rank; }
    __device__ __forceinline__ int n_vecs() const { return sh->n_vecs; }
    __device__ __forceinline__ int v0() const { return min(warp * sh->run, sh->n_vecs); }
    __device__ __forceinline__ int v1() const { return min((warp + 1) * sh->run, sh->n_vecs); }
    __device__ __forceinline__ const RowScale& s() const { return sh->s; }
    // shared memory: a piece's largest key, upper 16 bits
    __device__ __forceinline__ uint16_t* keys() const { return reinterpret_cast<uint16_t*>(sh + 1); }
    __device__ __forceinline__ int index(int v) const { return sh->first + v * E; }
    __device__ __forceinline__ bool partial(int v) const { return v < sh->full0 || v >= sh->full1; }
    static __device__ __forceinline__ uint4 load_whole(const uint4* at) {
        uint4 x;
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                     : "l"(at)
                     : "memory");
        return x;
    }
    __device__ __forceinline__ uint4 load(int v) const {
        return partial(v) ? load_part<BF16>(sh->src, sh->V, index(v), NOBODY) : load_whole(sh->base + v);
    }
    // padding that has no place in the order (a negative NaN, key 0)
    static constexpr uint32_t NOBODY = BF16 ? 0xFFFFu : 0xFFFFFFFFu;
    static constexpr uint32_t MINUS_INF = BF16 ? 0xFF80u : 0xFF800000u;

    // Every thread of the row's CTAs has got here, and what they wrote is seen.
    __device__ __forceinline__ void sync() const {
        if (CS() == 1) __syncthreads();
        else cg::this_cluster().sync();
    }
    template <class X>
    __device__ __forceinline__ X* of(X* mine, int cta) const { return CS() == 1 ? mine : cg::this_cluster().map_shared_rank(mine, cta); }
    template <class F>
    __device__ __forceinline__ void each_cta(F&& f) const {
        for (int c = 0; c < CS(); ++c) f(of(sh, c));
    }

    // f(x, v) for this lane's pieces whose key is at least that of `lo`; the next
    // one is on its way meanwhile.
    template <class F>
    __device__ __forceinline__ void each_piece(u64 lo, F&& f) const {
        const uint32_t lo16 = lo16_of(lo);
        const uint16_t* k = keys();
        const uint4* from = sh->base;
        const int end = v1(), whole0 = sh->full0, whole1 = sh->full1;
        const auto next = [&](int at) {
            while (at < end && k[at] < lo16) at += 32;
            return at;
        };
        const auto get = [&](int v) { return v < whole0 || v >= whole1 ? load_part<BF16>(sh->src, sh->V, index(v), NOBODY) : load_whole(from + v); };
        int v = next(v0() + lane);
        uint4 x = make_uint4(0, 0, 0, 0);
        if (v < end) x = get(v);
        while (v < end) {
            const int n = next(v + 32);
            uint4 y = x;
            if (n < end) y = get(n);
            f(x, v);
            x = y;
            v = n;
        }
    }
    // The same for passes that do little with a piece: U loads at a time. (One ahead,
    // as above, leaves them waiting for L2.)
    template <class F>
    __device__ __forceinline__ void each_piece_quick(u64 lo, F&& f) const {
        constexpr int U = 8;
        const uint32_t lo16 = lo16_of(lo);
        const uint16_t* k = keys();
        const int end = v1();
        for (int v = v0() + lane; v < end; v += 32 * U) {
            uint4 x[U];
            bool on[U];
#pragma unroll
            for (int q = 0; q < U; ++q) {
                on[q] = v + 32 * q < end && k[v + 32 * q] >= lo16;
                if (on[q]) x[q] = load(v + 32 * q);
            }
#pragma unroll
            for (int q = 0; q < U; ++q)
                if (on[q]) f(x[q], v + 32 * q);
        }
    }
    // What a piece's key is compared with. (The pieces' keys are of the bits as they
    // are: -0 has the one below that of 0.)
    static __device__ __forceinline__ uint32_t lo16_of(u64 place) {
        const uint32_t k = BF16 ? place_key(place) : place_key(place) >> 16;
        return k == 0x8000u ? 0x7FFFu : k;
    }
    // The key of a piece, and its maximum taken into `most` (of two halves in bf16).
    static __device__ __forceinline__ uint16_t piece_key(const uint4& x, uint32_t& most) {
        uint32_t m, b;
        if constexpr (BF16) {
            m = max_nan_bf16x2(max_nan_bf16x2(x.x, x.y), max_nan_bf16x2(x.z, x.w));
            most = max_nan_bf16x2(most, m);
            b = max_nan_bf16x2(m, m >> 16) << 16;
        } else {
            m = __float_as_uint(max_nan(max_nan(__uint_as_float(x.x), __uint_as_float(x.y)), max_nan(__uint_as_float(x.z), __uint_as_float(x.w))));
            most = __float_as_uint(max_nan(__uint_as_float(most), __uint_as_float(m)));
            b = m;
        }
        return (uint16_t)((b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u)) >> 16);
    }
};

// A CTA's part of the row at sh.src: `slice` pieces from piece `begin` on, of CS parts.
template <bool BF16>
__device__ __forceinline__ void set_part(CutShared& sh, int lead, int V, int begin, int slice, int CS, int rank) {
    using R = Row<BF16>;
    const int pieces = (lead + V + R::E - 1) / R::E;
    begin = min(begin, pieces);
    sh.base = reinterpret_cast<const uint4*>(sh.src - lead * R::ES) + begin;
    sh.V = V;
    sh.first = begin * R::E - lead;
    sh.n_vecs = min(slice, pieces - begin);
    sh.slice = slice;
    sh.run = (slice + CL_WARPS - 1) / CL_WARPS;
    sh.full0 = sh.first < 0 ? 1 : 0;
    sh.full1 = sh.first + sh.n_vecs * R::E > V ? sh.n_vecs - 1 : sh.n_vecs;
    sh.CS = CS;
    sh.rank = rank;
}

// The list. Every CTA appends to its own (atomics on another CTA's memory took a
// microsecond each) after begin_list, collect brings them to the first CTA's and
// returns how many there are: with more than CL_LIST nothing is moved. What does
// not fit is counted only.
__device__ __forceinline__ void begin_list(CutShared& sh) {
    if (threadIdx.x == 0) sh.list_n = 0;
    __syncthreads();
}
__device__ __forceinline__ void append(CutShared& sh, u64 place) {
    const uint32_t at = atomicAdd(&sh.list_n, 1u);
    if (at < CL_LIST) sh.list[at] = place;
}
// Places for this lane's `mine` entries of a counted array, the warp's by one atomic.
__device__ __forceinline__ uint32_t take_places(uint32_t* n, uint32_t mine, int lane) {
    const uint32_t incl = warp_scan(mine, lane);
    uint32_t first = 0;
    if (lane == 31 && incl) first = atomicAdd(n, incl);
    return __shfl_sync(0xFFFFFFFFu, first, 31) + incl - mine;
}
template <bool BF16>
__device__ __forceinline__ uint32_t collect(const Row<BF16>& row) {
    CutShared& sh = *row.sh;
    __syncthreads();
    uint32_t n = sh.list_n;
    if (row.CS() == 1) return n;
    if (threadIdx.x < row.CS()) row.of(sh.counts, threadIdx.x)[row.rank()] = n;
    row.sync();
    uint32_t before = 0, all = 0;
    for (int c = 0; c < row.CS(); ++c) {
        if (c < row.rank()) before += sh.counts[c];
        all += sh.counts[c];
    }
    if (all <= CL_LIST && row.rank() > 0) {
        CutShared* head = row.of(&sh, 0);
        for (uint32_t i = threadIdx.x; i < n; i += CL_THREADS) head->list[before + i] = sh.list[i];
    }
    row.sync();
    return all;
}

// f(v, piece, on) for this CTA's pieces that hold places from `lo` on, by whole
// warps, a lane without a piece not `on`: the CTA collects them,
// then its threads take one each. Too many to collect: each lane its own, four loads
// at a time.
template <bool BF16, class F>
__device__ __forceinline__ void each_hit(const Row<BF16>& row, u64 lo, F&& f) {
    CutShared& sh = *row.sh;
    const uint32_t lo16 = Row<BF16>::lo16_of(lo);
    if (threadIdx.x == 0) sh.hits_n = 0;
    __syncthreads();
    // 8 keys at a time; the keys behind the part's last are 0
    const uint4* keys = reinterpret_cast<const uint4*>(row.keys());
    const int n_vecs = row.n_vecs();
    for (int g0 = row.warp * 32; g0 * 8 < n_vecs; g0 += CL_THREADS) {
        const int g = g0 + row.lane;
        uint32_t hit = 0;
        if (g * 8 < n_vecs) {
            const uint4 k8 = keys[g];
            const uint32_t w[4] = {k8.x, k8.y, k8.z, k8.w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (((w[i / 2] >> (16 * (i % 2))) & 0xFFFFu) >= lo16 && g * 8 + i < n_vecs) hit |= 1u << i;
        }
        if (!__any_sync(0xFFFFFFFFu, hit != 0)) continue;
        for (uint32_t at = take_places(&sh.hits_n, __popc(hit), row.lane); hit; hit &= hit - 1, ++at)
            if (at < CL_HITS) sh.hits[at] = (uint32_t)(g * 8 + __ffs(hit) - 1);
    }
    __syncthreads();
    if (sh.hits_n <= CL_HITS) {
        const int n = (int)sh.hits_n;
        for (int i0 = row.warp * 32; i0 < n; i0 += CL_THREADS) {
            const bool on = i0 + row.lane < n;
            const int v = on ? (int)sh.hits[i0 + row.lane] : 0;
            f(v, on ? row.load(v) : make_uint4(0, 0, 0, 0), on);
        }
    } else {
        constexpr int U = 4;
        const int end = row.v1();
        for (int v0 = row.v0(); v0 < end; v0 += 32 * U) {
            uint4 x[U];
            bool on[U];
#pragma unroll
            for (int q = 0; q < U; ++q) {
                const int v = v0 + row.lane + 32 * q;
                on[q] = v < end && row.keys()[v] >= lo16;
                x[q] = on[q] ? row.load(v) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int q = 0; q < U; ++q)
                if (__any_sync(0xFFFFFFFFu, on[q])) f(v0 + row.lane + 32 * q, x[q], on[q]);
        }
    }
}

// The places in [lo, hi] of all parts, to the list. Returns how many there are.
template <bool BF16>
__device__ __forceinline__ uint32_t gather(const Row<BF16>& row, u64 lo, u64 hi) {
    using R = Row<BF16>;
    CutShared& sh = *row.sh;
    begin_list(sh);
    each_hit(row, lo, [&](int v, const uint4& x, bool on) {
        const int i0 = row.index(v);
        uint32_t in = 0;
#pragma unroll
        for (int e = 0; e < R::E; ++e) {
            const u64 p = place_of(key_of<BF16>(piece_elem<BF16>(x, e)), i0 + e);
            if (on && p >= lo && p <= hi) in |= 1u << e;
        }
        uint32_t at = take_places(&sh.list_n, __popc(in), row.lane);
#pragma unroll
        for (int e = 0; e < R::E; ++e) {
            if (!(in >> e & 1u)) continue;
            if (at < CL_LIST) sh.list[at] = place_of(key_of<BF16>(piece_elem<BF16>(x, e)), i0 + e);
            ++at;
        }
    });
    return collect(row);
}

// The first index of the row's largest element, whose key is lo's.
template <bool BF16>
__device__ __forceinline__ int first_largest(const Row<BF16>& row, u64 lo) {
    using R = Row<BF16>;
    CutShared& sh = *row.sh;
    each_hit(row, lo, [&](int v, const uint4& x, bool on) {
        int first = INT32_MAX;
#pragma unroll
        for (int e = R::E - 1; e >= 0; --e)
            if (key_of<BF16>(piece_elem<BF16>(x, e)) == place_key(lo)) first = row.index(v) + e;
        if (on) atomicMin(&sh.first_largest, first);
    });
    __syncthreads();
    if (threadIdx.x < row.CS()) row.of(sh.firsts, threadIdx.x)[row.rank()] = sh.first_largest;
    row.sync();
    int first = INT32_MAX;
    for (int c = 0; c < row.CS(); ++c) first = min(first, sh.firsts[c]);
    return first;
}

// Inclusive sums over the CTA's threads.
template <class N>
__device__ __forceinline__ N block_scan(N v, N* warp_sums, int lane, int warp, N& total) {
    v = warp_scan(v, lane);
    __syncthreads();
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < CL_WARPS; ++w) {
        const N t = warp_sums[w];
        if (w < warp) v += t;
        total += t;
    }
    return v;
}

// Sorts the first n entries of the list, descending, by this CTA; they lie in [lo,
// hi]. Few: by counting what is larger, 4 lanes per entry. More: into 1024 buckets
// of equal width, and within a bucket by counting. Where that leaves many in a
// bucket (equal logits, say): by a bitonic network in shared memory, whose steps
// over up to 64 neighbours stay within a warp.
__device__ __noinline__ void sort_list(CutShared& sh, int n, u64 lo, u64 hi) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    u64* list = sh.list;
    if (n <= CL_THREADS / 4) {
        const int i = tid >> 2;
        u64 mine = 0;
        int before = 0;
        if (i < n) {
            mine = list[i];
            for (int j = tid & 3; j < n; j += 4) before += list[j] > mine;
        }
        before += __shfl_xor_sync(0xFFFFFFFFu, before, 1);
        before += __shfl_xor_sync(0xFFFFFFFFu, before, 2);
        __syncthreads();
        if (i < n && (tid & 3) == 0) list[before] = mine;
        __syncthreads();
        return;
    }
    constexpr int PER = CL_LIST / CL_THREADS, BUCKETS = 2 * CL_THREADS, MOST = 64;
    const int shift = max(0, 54 - __clzll((long long)(hi - lo)));
    const auto bucket = [&](u64 x) { return BUCKETS - 1 - (int)min((max(x, lo) - lo) >> shift, (u64)(BUCKETS - 1)); };
    uint2* counts = reinterpret_cast<uint2*>(sh.count);
    counts[tid] = make_uint2(0, 0);
    __syncthreads();
    u64 x[PER];
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int i = tid + q * CL_THREADS;
        if (i >= n) continue;
        x[q] = list[i];
        atomicAdd(&sh.count[bucket(x[q])], 1u);
    }
    __syncthreads();
    const uint2 mine = counts[tid];
    uint32_t all;
    const uint32_t before = block_scan(mine.x + mine.y, sh.warp_count, lane, warp, all) - mine.x - mine.y;
    if (!__syncthreads_or(mine.x > MOST || mine.y > MOST)) {
        counts[tid] = make_uint2(before, before + mine.x);
        __syncthreads();
#pragma unroll
        for (int q = 0; q < PER; ++q)
            if (tid + q * CL_THREADS < n) list[atomicAdd(&sh.count[bucket(x[q])], 1u)] = x[q];
        __syncthreads();
        // a bucket's count is now where it ends
        uint32_t to[PER];
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            if (tid + q * CL_THREADS >= n) continue;
            const int b = bucket(x[q]);
            const uint32_t first = b > 0 ? sh.count[b - 1] : 0;
            to[q] = first;
            for (uint32_t j = first; j < sh.count[b]; ++j) to[q] += list[j] > x[q];
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < PER; ++q)
            if (tid + q * CL_THREADS < n) list[to[q]] = x[q];
        __syncthreads();
        return;
    }
    int size = 256;
    while (size < n) size <<= 1;
    for (int i = n + tid; i < size; i += CL_THREADS) list[i] = 0;
    for (int block = 2; block <= size; block <<= 1) {
        for (int stride = block >> 1; stride > 0; stride >>= 1) {
            if (stride >= 32 || stride == block >> 1) __syncthreads();
            else __syncwarp();
            for (int p = tid; p < size / 2; p += CL_THREADS) {
                const int a = 2 * p - (p & (stride - 1)), b = a + stride;
                const u64 y = list[a], z = list[b];
                const bool down = (a & block) == 0;
                if ((y < z) == down) {
                    list[a] = z;
                    list[b] = y;
                }
            }
        }
    }
    __syncthreads();
}

// The first bin, from 0 on, in which the sum over the bins of all CTAs reaches
// `goal` (the last one if none does), told to every CTA as found_bin. A bin's value
// is its count, or with `decay` count / CL_SHARE times 2^(-decay * bin). With `near`
// also the bins around it, found_from to found_to, that hold up to `near` elements
// on either side and one bin at least.
constexpr uint32_t CL_SHARE = 8192;  // counts per element where bins hold weights
template <bool BF16>
__device__ __forceinline__ void find_bin(const Row<BF16>& row, float goal, float decay, uint32_t near) {
    CutShared& sh = *row.sh;
    row.sync();
    if (row.rank() == 0) {
        static_assert(CL_BINS == 4 * CL_THREADS, "four bins per thread");
        const int tid = threadIdx.x;
        if (tid == 0) {
            sh.found_bin = sh.found_from = CL_BINS - 1;
            sh.found_to = 0;
        }
        uint32_t n[4] = {0, 0, 0, 0};
        for (int c = 0; c < row.CS(); ++c) {
            const uint4 k = reinterpret_cast<const uint4*>(row.of(&sh, c)->count)[tid];
            n[0] += k.x, n[1] += k.y, n[2] += k.z, n[3] += k.w;
        }
        const float unit = decay == 0.0f ? 1.0f : 1.0f / (float)CL_SHARE;
        float v[4], sum = 0.0f, total;
        uint32_t number = 0, all;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = (float)n[i] * unit * (decay == 0.0f ? 1.0f : ex2(-decay * (float)(4 * tid + i)));
            sum += v[i];
            number += n[i];
        }
        const float before = block_scan(sum, sh.warp_value, row.lane, row.warp, total) - sum;
        if (before < goal && before + sum >= goal) {
            int b = 4 * tid + 3;
#pragma unroll
            for (int i = 3; i >= 0; --i) {
                float upto = before;
                for (int q = 0; q <= i; ++q) upto += v[q];
                if (upto >= goal) b = 4 * tid + i;
            }
            atomicMin(&sh.found_bin, (uint32_t)b);  // (sums of floats need not ascend to the last bit)
        }
        if (near) {
            const uint32_t upto = block_scan(number, sh.warp_count, row.lane, row.warp, all);
            const uint32_t bin = sh.found_bin;
            if ((bin >> 2) == (uint32_t)tid) {
                uint32_t c = upto - number;
                for (uint32_t i = 0; i < (bin & 3); ++i) c += n[i];
                sh.found_above = c;  // (counts before the bin, and with it)
                sh.found_count = c + n[bin & 3];
            }
            __syncthreads();
            const uint32_t first = sh.found_above, past = sh.found_count;
            uint32_t c = upto - number;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t at = 4 * tid + i;
                if (at <= bin && (first - c <= near * CL_SHARE || at + 1 >= bin)) atomicMin(&sh.found_from, at);
                c += n[i];
                if (at >= bin && (c - past <= near * CL_SHARE || at <= bin + 1)) atomicMax(&sh.found_to, at);
            }
        }
        __syncthreads();
        if (tid > 0 && tid < row.CS()) {
            CutShared* o = row.of(&sh, tid);
            o->found_bin = sh.found_bin;
            o->found_from = sh.found_from;
            o->found_to = sh.found_to;
        }
    }
    row.sync();
}

template <bool BF16>
__device__ __forceinline__ void clear_bins(const Row<BF16>& row) {
    reinterpret_cast<uint4*>(row.sh->count)[threadIdx.x] = make_uint4(0, 0, 0, 0);
    __syncthreads();
}

// This lane's copy of the table, all of them written first.
template <bool BF16>
__device__ __forceinline__ const ExpEntry* copy_table(const Row<BF16>& row) {
    CutShared& sh = *row.sh;
    __syncthreads();
    for (int i = threadIdx.x; i < CL_EXP * CL_COPIES; i += CL_THREADS) sh.copies[i] = sh.exp[i / CL_COPIES];
    __syncthreads();
    return sh.copies + (threadIdx.x & (CL_COPIES - 1));
}

// Sums of the weights at or above `cut`, this warp's into the first CTA's
// part_mass and the total to every thread.
template <bool BF16>
__device__ __forceinline__ u64 sum_above(const Row<BF16>& row, u64 cut) {
    using R = Row<BF16>;
    CutShared& sh = *row.sh;
    u64 m = 0;
    const ExpEntry* copy = copy_table(row);
    if (row.s().low == row.s().low) {
        // At or above the cut is z >= its logit before its index and z > it behind.
        const float z_cut = key_value<BF16>(place_key(cut)), z_from = fmaxf(z_cut, row.s().low);
        const int i_cut = place_index(cut);
        const float z_over = cut == CL_LOWEST ? z_from : fmaxf(key_value<BF16>(place_key(cut) + 1), row.s().low);
        WeightSum sum;
        row.each_piece(cut, [&](const uint4& x, int v) {
            const int i0 = row.index(v);
            if (i0 <= i_cut && i_cut < i0 + R::E - 1) {  // the one piece that the index divides
#pragma unroll
                for (int e = 0; e < R::E; ++e) {
                    const float z = piece_elem<BF16>(x, e);
                    if (place_of(key_of<BF16>(z), i0 + e) >= cut) m += weight(z, row.s(), row.sh->exp);
                }
            } else {
                const float from = i0 + R::E - 1 <= i_cut ? z_from : z_over;
#pragma unroll
                for (int e = 0; e < R::E; e += 2) {
                    const float z0 = piece_elem<BF16>(x, e), z1 = piece_elem<BF16>(x, e + 1);
                    sum.add(z0 >= from ? z0 : row.s().low, z1 >= from ? z1 : row.s().low, row.s(), copy, e == 0);
                }
                sum.end_piece();
            }
        });
        m += sum.total(row.s().unit);
    } else {
        row.each_piece(cut, [&](const uint4& x, int v) {
            const int i0 = row.index(v);
#pragma unroll 1
            for (int e = 0; e < R::E; ++e) {
                const float z = piece_elem<BF16>(x, e);
                if (place_of(key_of<BF16>(z), i0 + e) >= cut) m += weight(z, row.s(), row.sh->exp);
            }
        });
    }
    m = warp_sum(m);
    if (row.lane == 0) row.of(&sh, 0)->part_mass[row.rank() * CL_WARPS + row.warp] = m;
    row.sync();
    u64 total = 0;
    const u64* parts = row.of(&sh, 0)->part_mass;
    for (int w = row.lane; w < row.CS() * CL_WARPS; w += 32) total += parts[w];
    return warp_sum(total);
}

// The row's unit from then on, its sum being `total` in the present one (to 2^-27).
template <bool BF16>
__device__ __forceinline__ void refine_unit(const Row<BF16>& row, u64 total) {
    CutShared& sh = *row.sh;
    __syncthreads();  // everyone has used the present one
    if (threadIdx.x == 0) set_unit(sh.s, unit_of((float)total * 0x1.0008p0f * __uint_as_float((uint32_t)(127 - sh.s.unit) << 23)));
    __syncthreads();
}

// The whole part of u total, 0 <= u <= 1, and whether there is more: by whole
// numbers, in every thread (one thread's doubles kept the others waiting).
__device__ __forceinline__ u64 share_of(float u, u64 total, bool& more) {
    const uint32_t b = __float_as_uint(u) & 0x7FFFFFFFu, exponent = max(b >> 23, 1u);
    const u64 m = b >> 23 ? (b & 0x7FFFFFu) | 0x800000u : b;  // u = m 2^-shift
    const int shift = 150 - (int)exponent;                    // 23 to 149
    const u64 low = m * total, high = __umul64hi(m, total);   // (below 2^22)
    if (shift < 64) {
        more = (low << (64 - shift)) != 0;
        return high << (64 - shift) | low >> shift;
    }
    const int rest = shift - 64;
    more = low != 0 || (rest < 32 ? (uint32_t)high << 1 << (31 - rest) : (uint32_t)high) != 0;
    return rest < 32 ? high >> rest : 0;
}

// The fewest units that are p of `total`.
__device__ __forceinline__ u64 goal_of(float p, u64 total) {
    bool more;
    const u64 goal = share_of(p, total, more);
    return goal + more;
}

// One round of the exact search in [lo, hi]: the bin in which the count `k`
// (BY_MASS false) or the weight `goal` is reached from above, given what lies
// above hi. The range becomes that bin. The first round's GOAL_OF_ALL becomes p of all
// weights in the range: a share of the same whole numbers that are searched.
constexpr u64 GOAL_OF_ALL = ~0ull;
template <bool BF16, bool BY_MASS>
__device__ __forceinline__ uint32_t narrow(const Row<BF16>& row, u64& lo, u64& hi, uint32_t& above, u64& mass_above, uint32_t k, u64& goal,
                                           float p) {
    using R = Row<BF16>;
    CutShared& sh = *row.sh;
    u64* mass = sh.list;
    const int tid = threadIdx.x, lane = row.lane, warp = row.warp, CS = row.CS();
    const u64 width = hi - lo;  // one less than the places
    const int bits = 64 - __clzll((long long)width);
    const int shift = width == 0 ? 0 : max(0, bits - 11);
    for (int i = tid; i < CL_BINS; i += CL_THREADS) {
        sh.count[i] = 0;
        mass[i] = 0;
    }
    if (tid == 0) {
        sh.found_bin = 0;
        sh.found_above = above;
        sh.found_mass = mass_above;
        sh.found_count = 0;
    }
    row.sync();
    row.each_piece(lo, [&](const uint4& x, int v) {
        const int i0 = row.index(v);
#pragma unroll 1
        for (int e = 0; e < R::E; ++e) {
            const float z = piece_elem<BF16>(x, e);
            const u64 place = place_of(key_of<BF16>(z), i0 + e);
            if (place < lo || place > hi) continue;
            const int bin = (int)((place - lo) >> shift);
            atomicAdd(&sh.count[bin], 1u);
            if (BY_MASS) atomicAdd(&mass[bin], weight(z, row.s(), row.sh->exp));
        }
    });
    row.sync();
    // A CTA adds up its share of the bins over all CTAs; a thread has `per`
    // neighbouring ones.
    const int seg = CL_BINS / CS, per = max(1, seg / CL_THREADS);
    const int b0 = row.rank() * seg + tid * per;
    const bool on = tid * per < seg;
    uint32_t c_of[4] = {0, 0, 0, 0}, c_sum = 0;  // seg / 512 <= 4
    u64 m_of[4] = {0, 0, 0, 0}, m_sum = 0;
    if (on) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= per) break;
            for (int c = 0; c < CS; ++c) {
                const CutShared* o = row.of(&sh, c);
                c_of[i] += o->count[b0 + i];
                if (BY_MASS) m_of[i] += o->list[b0 + i];
            }
            c_sum += c_of[i];
            m_sum += m_of[i];
        }
    }
    // inclusive sums from the share's first bin on, turned into those from above
    uint32_t c_total;
    u64 m_total;
    const uint32_t c_in = block_scan(c_sum, sh.warp_count, lane, warp, c_total);
    const u64 m_in = block_scan(m_sum, sh.warp_mass, lane, warp, m_total);
    if (tid == 0) {
        row.each_cta([&](CutShared* o) {
            o->seg_count[row.rank()] = c_total;
            o->seg_mass[row.rank()] = m_total;
        });
    }
    row.sync();
    if (BY_MASS && goal == GOAL_OF_ALL) {
        u64 all = 0;
        for (int q = 0; q < CS; ++q) all += sh.seg_mass[q];
        goal = goal_of(p, all);
    }
    uint32_t c = above + c_total - c_in;
    u64 m = mass_above + m_total - m_in;
    for (int q = row.rank() + 1; q < CS; ++q) {
        c += sh.seg_count[q];
        m += sh.seg_mass[q];
    }
    if (on) {
        // c and m: what lies above the bin
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            if (i >= per) continue;
            const bool reached = BY_MASS ? m + m_of[i] >= goal : c + c_of[i] >= k;
            const bool before = BY_MASS ? (c != 0 && m >= goal) : c >= k;
            if (c_of[i] != 0 && reached && !before) {
                row.each_cta([&](CutShared* o) {
                    o->found_bin = (uint32_t)(b0 + i);
                    o->found_above = c;
                    o->found_mass = m;
                    o->found_count = c_of[i];
                });
            }
            c += c_of[i];
            m += m_of[i];
        }
    }
    row.sync();
    above = sh.found_above;
    mass_above = sh.found_mass;
    const uint32_t n = sh.found_count;
    const u64 new_lo = lo + ((u64)sh.found_bin << shift);
    hi = min(hi, new_lo + ((1ull << shift) - 1));
    lo = new_lo;
    row.sync();  // everyone has read what was found
    return n;
}

// In the sorted list of n places, below others (if `any`) of weight mass_above: the
// one with which the weight is reached, or 0. A goal known to lie from `goal` to
// goal_hi only has to be reached by the same place throughout. This CTA's threads.
template <bool BF16>
__device__ __forceinline__ u64 reach_in_list(const Row<BF16>& row, int n, bool any, u64 mass_above, u64 goal, u64 goal_hi) {
    CutShared& sh = *row.sh;
    const int tid = threadIdx.x;
    if (any && mass_above >= goal) return 0;
    if (tid == 0) sh.found_place = 0;
    u64 carry = mass_above;
    for (int base = 0; base < n; base += CL_THREADS) {
        const int i = base + tid;
        const u64 p = i < n ? sh.list[i] : 0, w = i < n ? weight(key_value<BF16>(place_key(p)), row.s(), row.sh->exp) : 0;
        u64 total;
        const u64 incl = carry + block_scan(w, sh.warp_mass, row.lane, row.warp, total);
        const bool first = !any && i == 0;
        if (i < n && incl >= goal_hi && (first || incl - w < goal)) sh.found_place = p;
        carry += total;
    }
    __syncthreads();
    return sh.found_place;
}

// The groups' n-th largest maximum, from 0 on: each is compared with all others, by
// as many lanes as there are for it.
__device__ __forceinline__ float nth_group(CutShared& sh, int groups, int n) {
    const int lanes = min(CL_THREADS / groups, 32), i = (int)threadIdx.x / lanes, from = (int)threadIdx.x % lanes;
    const float mine = i < groups ? sh.group_max[i] : 0.0f;
    int before = 0;
    if (i < groups) {
        for (int w = 4 * from; w < groups; w += 4 * lanes) {
            const float4 o = *reinterpret_cast<const float4*>(sh.group_max + w);
            before += (o.x > mine || (o.x == mine && w < i)) + (o.y > mine || (o.y == mine && w + 1 < i)) +
                      (o.z > mine || (o.z == mine && w + 2 < i)) + (o.w > mine || (o.w == mine && w + 3 < i));
        }
    }
    for (int o = 1; o < lanes; o <<= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
    if (i < groups && before == n) sh.bound = mine;
    __syncthreads();
    return sh.bound;
}

// 4. The place of the last element that a cut keeps, exactly, in [lo, hi], the k-th or
// (BY_MASS) the one with which p of all weights there is reached: the range narrows
// until what is left fits the list, where it is picked.
template <bool BF16, bool BY_MASS>
__device__ __noinline__ u64 find_cut(const Row<BF16> row, u64 lo, u64 hi, uint32_t k, float p) {
    CutShared& sh = *row.sh;
    uint32_t above = 0, left = CL_LIST + 1;
    u64 mass_above = 0, goal = GOAL_OF_ALL;
    for (int round = 0; round < CL_ROUNDS && left > CL_LIST; ++round) left = narrow<BF16, BY_MASS>(row, lo, hi, above, mass_above, k, goal, p);
    const int n = (int)min(gather(row, lo, hi), (uint32_t)CL_LIST);
    if (row.rank() == 0) {
        sort_list(sh, n, lo, hi);
        u64 place = 0;
        if constexpr (BY_MASS) {
            place = reach_in_list(row, n, above != 0, mass_above, goal, goal);
        } else {
            const int at = (int)k - 1 - (int)above;
            place = at >= 0 && at < n ? sh.list[at] : 0;
        }
        place = place ? place : lo;
        __syncthreads();
        if (threadIdx.x == 0) row.each_cta([&](CutShared* o) { o->found_place = place; });
    }
    row.sync();
    const u64 place = sh.found_place;
    row.sync();  // everyone has read it
    return place;
}

// The largest whole number below or at u of `total`, below total.
__device__ __forceinline__ u64 draw_target(float u, u64 total) {
    bool more;
    const u64 t = share_of(u > 0.0f ? fminf(u, 1.0f) : 0.0f, total, more);
    return t < total ? t : total - 1;
}

// ln(total / 2^unit) for a total of one or more: total = 2^(k + i / 256) (1 + d) with
// the table's factor, and ln(1 + d) by its series, d < 2^-8; to about 2^-36.
__device__ __forceinline__ double log_total(u64 total, int unit, const ExpEntry* table) {
    const int k = 63 - __clzll((long long)total);
    const double m = (double)total * __longlong_as_double((long long)(1023 - k) << 52);  // [1, 2)
    const int i = min((int)(log2f((float)m) * (float)CL_EXP), CL_EXP - 1);
    // 2^(-i / 256) = 2^((256 - i) / 256) / 2
    const ExpEntry e = table[(CL_EXP - i) & (CL_EXP - 1)];
    const double d = m * (((double)e.hi + (double)e.lo) * (i == 0 ? 1.0 : 0.5)) - 1.0;
    const float f = (float)d, tail = f * f * (f * (1.0f / 3.0f) - 0.5f - f * f * 0.25f);
    return ((double)(k - unit) + (double)i * (1.0 / CL_EXP)) * 0.69314718055994530942 + (d + (double)tail);
}

__device__ __forceinline__ void put_token(const CutParams& P, int64_t row, int index, float z, const CutShared& sh, float top, double log_sum) {
    P.tokens[row] = index;
    if (P.logprobs) P.logprobs[row] = (float)(((double)z - (double)top) * sh.inv_t - log_sum);
}

// Draws from the first n of the sorted list, by this CTA.
template <bool BF16>
__device__ __forceinline__ void draw_list(const CutParams& P, const Row<BF16>& row, int64_t at_row, float u, int n) {
    CutShared& sh = *row.sh;
    const int tid = threadIdx.x;
    if (n <= CL_THREADS / 4) {
        // Few: 4 lanes per entry add up those before it in the order of indices, and
        // all; the sum's logarithm is formed meanwhile. (A row of 32,000, top-k 50 and
        // top-p: 12.9 us with a sort and two scans, 10.2 so.) Entries become (reversed
        // index, weight), 18 and 45 bits: 128 halves of that unit are 2^-38.
        constexpr int UNIT = 44;
        constexpr u64 W = (2ull << UNIT) - 1;
        const int i = tid >> 2;
        float z = 0.0f;
        if (i < n && (tid & 3) == 0) {
            const u64 p = sh.list[i];
            z = key_value<BF16>(place_key(p));
            sh.list[i] = (p & CL_INDEX_MASK) << (UNIT + 1) | weight(z, row.s(), row.sh->exp, UNIT, none_of(UNIT));
        }
        __syncthreads();
        const u64 mine = i < n ? sh.list[i] : 0;
        u64 before = 0, all = 0;
        if (i < n) {
            for (int j = tid & 3; j < n; j += 4) {
                const u64 e = sh.list[j];
                all += e & W;
                before += e > mine ? e & W : 0;  // (descending reversed index)
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
            all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
        }
        if (tid == 3 && P.logprobs) sh.log_sum = log_total(all, UNIT, sh.exp);
        __syncthreads();
        if (i < n && (tid & 3) == 0) {
            const u64 target = draw_target(u, all);
            if (before <= target && target < before + (mine & W))
                put_token(P, at_row, (int)(CL_INDEX_MASK - (uint32_t)(mine >> (UNIT + 1))), z, sh, row.s().top, sh.log_sum);
        }
        return;
    }
    // entries become (reversed index, key) and are sorted by index
    for (int i = tid; i < n; i += CL_THREADS) {
        const u64 p = sh.list[i];
        sh.list[i] = (p & CL_INDEX_MASK) << 32 | place_key(p);
    }
    __syncthreads();
    sort_list(sh, n, 0, (1ull << (CL_INDEX_BITS + 32)) - 1);  // (descending reversed index)
    const auto weight_of = [&](u64 e) { return weight(key_value<BF16>((uint32_t)e), row.s(), row.sh->exp); };
    u64 total = 0;
    for (int i = tid; i < n; i += CL_THREADS) total += weight_of(sh.list[i]);
    u64 all;
    block_scan(total, sh.warp_mass, row.lane, row.warp, all);
    const u64 target = draw_target(u, all);
    u64 carry = 0;
    for (int base = 0; base < n; base += CL_THREADS) {
        const int i = base + tid;
        const u64 e = i < n ? sh.list[i] : 0, w = i < n ? weight_of(e) : 0;
        u64 sum;
        const u64 incl = carry + block_scan(w, sh.warp_mass, row.lane, row.warp, sum);
        if (i < n && incl - w <= target && target < incl)
            put_token(P, at_row, (int)(CL_INDEX_MASK - (uint32_t)(e >> 32)), key_value<BF16>((uint32_t)e), sh, row.s().top,
                      log_total(all, row.s().unit, sh.exp));
        carry += sum;
    }
}

// Draws over the warps' parts, whose sums at or above `cut` lie in the first
// CTA's part_mass: that finds the warp, and its CTA the element, by weight(). Where
// the sums are in floats (not `precise`) and the target comes as near to the element's
// edges as they may be off by, nothing is drawn, and that CTA gets false: a row in some
// thousands, whose sums it then forms anew (the others have ended: with a barrier that
// kept them 256 rows under min-p took 63 us, not 54).
template <bool BF16>
__device__ __forceinline__ bool draw_parts(const CutParams& P, const Row<BF16>& row, int64_t at_row, float u, u64 cut, bool precise) {
    using R = Row<BF16>;
    CutShared& sh = *row.sh;
    const int lane = row.lane;
    if (row.rank() == 0 && row.warp == 0) {
        constexpr int N = CL_MAX_CS * CL_WARPS / 32;  // neighbouring parts per lane
        u64 m[N], sum = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            m[i] = N * lane + i < row.CS() * CL_WARPS ? sh.part_mass[N * lane + i] : 0;
            sum += m[i];
        }
        const u64 incl = warp_scan(sum, lane), total = __shfl_sync(0xFFFFFFFFu, incl, 31);
        const u64 target = draw_target(u, total);
        u64 before = incl - sum;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (before <= target && target < before + m[i]) {
                row.each_cta([&](CutShared* o) {
                    o->draw_warp = (uint32_t)(N * lane + i);
                    o->draw_before = before;
                    o->draw_at = target - before;
                    o->found_mass = total;
                });
            }
            before += m[i];
        }
    }
    if (threadIdx.x == 0) sh.drawn = 0;
    row.sync();
    // The part's pieces, a run of neighbours for each thread of its CTA.
    const int part = (int)sh.draw_warp - row.rank() * CL_WARPS;
    if (part < 0 || part >= CL_WARPS) return true;
    const u64 target = sh.draw_at, total = sh.found_mass, before = sh.draw_before;
    const uint32_t lo16 = R::lo16_of(cut);
    const int p0 = min(part * row.sh->run, row.n_vecs()), p1 = min(p0 + row.sh->run, row.n_vecs());
    const int per = (row.sh->run + CL_THREADS - 1) / CL_THREADS, v0 = min(p0 + (int)threadIdx.x * per, p1), v1 = min(v0 + per, p1);
    const auto each_weight = [&](auto&& f) {
        for (int v = v0; v < v1; ++v) {
            if (!precise && row.keys()[v] < lo16) continue;
            const uint4 x = row.load(v);
#pragma unroll
            for (int e = 0; e < R::E; ++e) {
                const float z = piece_elem<BF16>(x, e);
                if (place_of(key_of<BF16>(z), row.index(v) + e) >= cut) f(weight(z, row.s(), sh.exp), row.index(v) + e, z);
            }
        }
    };
    u64 mine = 0, all;
    each_weight([&](u64 w, int, float) { mine += w; });
    u64 at = block_scan(mine, sh.warp_mass, lane, row.warp, all) - mine;
    if (at <= target && target < at + mine) {
        u64 slack = 0;
        if (!precise) {
            // (of the weights' own errors those before the part count 1 - u, the others u)
            const float ft = (float)total, fb = (float)before, share = __saturatef(u);
            slack = (u64)(CL_PAIR_ERROR * (share * (ft - fb) + (1.0f - share) * fb) + sum_error(share * ft + fb, sh.V, row.s().unit));
            if (!(row.s().low == row.s().low)) slack += (u64)sh.V;  // (weight()'s halves of a unit)
        }
        each_weight([&](u64 w, int index, float z) {
            if (at <= target && target < at + w && (target - at >= slack || before + at == 0) && at + w - target > slack) {
                put_token(P, at_row, index, z, sh, row.s().top, log_total(total, row.s().unit, sh.exp));
                sh.drawn = 1;
            }
            at += w;
        });
    }
    __syncthreads();
    return sh.drawn != 0;
}

// After a draw that came too near to an edge: the CTA that looked for the element takes
// the whole row for its part, the unit from its sum, and forms the warps' parts' sums
// by weight(). (It has no keys of most of these pieces.)
template <bool BF16>
__device__ __noinline__ void sum_alone(const Row<BF16> row, u64 cut) {
    using R = Row<BF16>;
    CutShared& sh = *row.sh;
    refine_unit(row, sh.found_mass);
    if (threadIdx.x == 0) {
        const int lead = (int)(reinterpret_cast<uintptr_t>(sh.src) & 15) / R::ES;
        set_part<BF16>(sh, lead, sh.V, 0, (lead + sh.V + R::E - 1) / R::E, 1, 0);
    }
    __syncthreads();
    u64 m = 0;
    const int end = row.v1();
    for (int v = row.v0() + row.lane; v < end; v += 32) {
        const uint4 x = row.load(v);
        const int i0 = row.index(v);
#pragma unroll 1
        for (int e = 0; e < R::E; ++e) {
            const float z = piece_elem<BF16>(x, e);
            if (place_of(key_of<BF16>(z), i0 + e) >= cut) m += weight(z, row.s(), sh.exp);
        }
    }
    m = warp_sum(m);
    if (row.lane == 0) sh.part_mass[row.warp] = m;
    __syncthreads();
}

// 3. Top-p alone. Returns the place of the last kept element and leaves the sums
// of the warps' parts at or above it in the first CTA's part_mass.
template <bool BF16>
__device__ __noinline__ u64 cut_by_mass(const Row<BF16> row, float top_p, float T, u64 highest, float about) {
    using R = Row<BF16>;
    CutShared& sh = *row.sh;
    const RowScale& s = row.s();
    const int tid = threadIdx.x;
    // The last kept element has at least (1 - p) / V of the sum of all weights
    // (all smaller ones together hold less than 1 - p of it), which is at least 1:
    // the bins span what can be kept, evenly in log weights.
    const float span_log = __logf((float)row.sh->V / fmaxf(1.0f - top_p, 1e-9f)) + 0.01f;
    const float span = span_log * T, to_bin = (float)CL_BINS / span, bin_log = span_log / (float)CL_BINS;
    clear_bins(row);
    // The histogram: CL_SHARE per element at a bin's upper edge, less towards its
    // lower one as the weight falls. A logit's bin and its place in it come from the
    // low bits of a float that 2^23 was added to.
    const float fine = 128.0f * to_bin, shifted = __fmaf_rn(s.top, fine, 8388608.0f), last = 8388608.0f + 128.0f * CL_BINS - 1.0f;
    const uint32_t fall = (uint32_t)(bin_log * (float)CL_SHARE * 2.0f + 0.5f);
    const bool flat = !(fabsf(s.top * fine) < 4194304.0f);  // (then shifted has no room)
    const float least = __fsub_rn(s.top, span * 1.0001f);
    row.each_piece_quick(max(CL_LOWEST, (u64)key_of<BF16>(least) << CL_INDEX_BITS), [&](const uint4& x, int) {
#pragma unroll
        for (int e = 0; e < R::E; ++e) {
            const float z = piece_elem<BF16>(x, e);
            const float y = flat ? __fmaf_rn(__fsub_rn(s.top, z), fine, 8388608.0f) : __fmaf_rn(-z, fine, shifted);
            if (!(y <= last)) continue;
            const uint32_t at = __float_as_uint(fmaxf(y, 8388608.0f)) & 0x7FFFFFu;
            atomicAdd(&sh.count[at >> 7], CL_SHARE - (((at & 127u) * fall + 128u) >> 8));
        }
    });
    find_bin(row, about * top_p * 0x1p-44f, bin_log * 1.4426950408889634f, CL_NEAR);
    const int bin0 = (int)sh.found_from, bin1 = (int)sh.found_to;
    u64 place = 0;
    bool any_above = false;
    // The sum of all weights and of those above the first of these bins, and what
    // lies in them to the list. Where the goal comes so near to a border that the
    // sums in floats may err (a flat row in thousands), or is not in the list, once more
    // with every weight formed by weight().
    for (bool precise = !(s.low == s.low);; precise = true) {
        const float z_hi = bin0 > 0 ? __fsub_rn(s.top, (float)bin0 / to_bin) : INFINITY;
        const float z_lo = key_value<BF16>(key_of<BF16>(__fsub_rn(s.top, (float)(bin1 + 1) / to_bin)));
        const u64 over = bin0 > 0 ? (u64)(key_of<BF16>(z_hi) + 1) << CL_INDEX_BITS : ~0ull;  // above z_hi
        const u64 lo = max(CL_LOWEST, (u64)key_of<BF16>(z_lo) << CL_INDEX_BITS);
        CutShared* head = row.of(&sh, 0);
        any_above = over <= highest;
        begin_list(sh);
        const ExpEntry* copy = copy_table(row);
        const float from = bin0 > 0 ? fmaxf(key_value<BF16>(key_of<BF16>(z_hi) + 1), precise ? -INFINITY : s.low) : INFINITY;
        u64 all = 0, above = 0;
        const auto to_list = [&](float z, int i) {
            if (z >= z_lo && z < from) append(sh, place_of(key_of<BF16>(z), i));
        };
        if (!precise) {
            WeightSum upper, lower;
            const f32x2 minus = pack2(-1.0f, -1.0f);
            row.each_piece(CL_LOWEST, [&](const uint4& x, int v) {
                const int i0 = row.index(v);
#pragma unroll
                for (int e = 0; e < R::E; e += 2) {
                    const float z0 = piece_elem<BF16>(x, e), z1 = piece_elem<BF16>(x, e + 1);
                    f32x2 a, rest;
                    WeightSum::pair(z0 >= s.low ? z0 : s.low, z1 >= s.low ? z1 : s.low, s, copy, a, rest);
                    float a0, a1, r0, r1;
                    unpack2(a, a0, a1);
                    unpack2(rest, r0, r1);
                    const bool up0 = z0 >= from, up1 = z1 >= from;
                    const f32x2 a_up = pack2(up0 ? a0 : 0.0f, up1 ? a1 : 0.0f), rest_up = pack2(up0 ? r0 : 0.0f, up1 ? r1 : 0.0f);
                    upper.add(a_up, rest_up, e == 0);
                    lower.add(fma2(a_up, minus, a), fma2(rest_up, minus, rest), e == 0);
                    to_list(z0, i0 + e);
                    to_list(z1, i0 + e + 1);
                }
                upper.end_piece();
                lower.end_piece();
            });
            above = upper.total(s.unit);
            all = above + lower.total(s.unit);
        } else {
            row.each_piece(CL_LOWEST, [&](const uint4& x, int v) {
                const int i0 = row.index(v);
#pragma unroll 1
                for (int e = 0; e < R::E; ++e) {
                    const float z = piece_elem<BF16>(x, e);
                    const u64 w = weight(z, s, sh.exp);
                    all += w;
                    above += z >= from ? w : 0;
                    to_list(z, i0 + e);
                }
            });
        }
        all = warp_sum(all);
        above = warp_sum(above);
        if (row.lane == 0) {
            head->part_mass[row.rank() * CL_WARPS + row.warp] = above;
            head->part_all[row.rank() * CL_WARPS + row.warp] = all;
        }
        const int n = (int)collect(row);
        if (row.CS() == 1) __syncthreads();
        all = 0;
        for (int w = row.lane; w < row.CS() * CL_WARPS; w += 32) all += head->part_all[w];
        all = warp_sum(all);
        const u64 goal = goal_of(top_p, all);
        if (row.rank() == 0) {
            u64 mass_above = 0, place = 0;
            for (int w = row.lane; w < row.CS() * CL_WARPS; w += 32) mass_above += sh.part_mass[w];
            mass_above = warp_sum(mass_above);
            if (n <= CL_LIST) {
                sort_list(sh, n, lo, min(highest, over - 1));
                // (p of all less what is above: errors above count 1 - p, the others' p)
                const float off = top_p * (float)(all - mass_above) + (1.0f - top_p) * (float)mass_above;
                const u64 unsure = precise ? 0 : (u64)(CL_PAIR_ERROR * off + sum_error(off, sh.V, s.unit));
                place = reach_in_list(row, n, any_above, mass_above, goal - min(goal, unsure), goal + unsure);
                // what of the list is kept joins its warps' sums
                if (place) {
                    const int lead = (int)((reinterpret_cast<uintptr_t>(row.sh->src) & 15) / R::ES);
                    for (int i = tid; i < n; i += CL_THREADS) {
                        const u64 p = sh.list[i];
                        if (p < place) continue;
                        const int piece = (place_index(p) + lead) / R::E, cta = piece / row.sh->slice, in_cta = piece - cta * row.sh->slice;
                        atomicAdd(&sh.part_mass[cta * CL_WARPS + in_cta / row.sh->run], weight(key_value<BF16>(place_key(p)), s, row.sh->exp));
                    }
                }
            }
            __syncthreads();
            if (tid == 0) row.each_cta([&](CutShared* o) { o->found_place = place; });
        }
        row.sync();
        place = sh.found_place;
        row.sync();
        if (place || precise || n > CL_LIST) break;
    }
    if (place == 0) {
        // more equal logits than the list takes, or a border that the histogram missed
        place = find_cut<BF16, true>(row, CL_LOWEST, highest, 0, top_p);
        sum_above(row, place);
    }
    return place;
}

// 3a. Top-p alone, first try: a few hundred of the row's largest go to the list with
// their exact weights, the others' are summed in fp32, to 2^-15 of their sum (an
// exponent is off by 2^-23 of itself, at most 2^-17 for weights that matter, a
// thread's sums of at most 132 terms by 2^-17). Where the place is the same whatever that error, it is
// found: so for rows whose mass lies with few tokens, in one cheap pass instead of
// the exact ones. Else 0, and the list is empty. about: the sum of all weights in
// units of 2^-44; from here on it gives the row's unit.
template <bool BF16>
__device__ __noinline__ u64 cut_near_top(const Row<BF16> row, float top_p, int groups, u64 highest, float& about, uint32_t& n) {
    using R = Row<BF16>;
    CutShared& sh = *row.sh;
    const float edge = nth_group(sh, groups, groups * 3 / 4);
    // (what is -inf has no weight)
    const u64 lo = (u64)max(key_of<BF16>(edge), key_of<BF16>(-INFINITY) + 1) << CL_INDEX_BITS;
    const float c = row.s().ch * (1.0f / (float)CL_EXP), top = row.s().top;
    const uint32_t lo16 = R::lo16_of(lo);
    f32x2 sum = pack2(0.0f, 0.0f), large = sum;
    const f32x2 cc = pack2(c, c), minus_top = pack2(-top, -top);
    row.each_piece_quick(CL_LOWEST, [&](const uint4& x, int v) {
        const bool some = row.keys()[v] >= lo16 || row.partial(v);  // (padding is not below the edge either)
        f32x2 part = pack2(0.0f, 0.0f);
#pragma unroll
        for (int e = 0; e < R::E; e += 2) {
            const float z0 = piece_elem<BF16>(x, e), z1 = piece_elem<BF16>(x, e + 1);
            const f32x2 w = ex2x2(mul2(add2(pack2(z0, z1), minus_top), cc));
            if (some) {
                float w0, w1;
                unpack2(w, w0, w1);
                part = add2(part, pack2(z0 < edge ? w0 : 0.0f, z1 < edge ? w1 : 0.0f));
                large = add2(large, pack2(z0 >= edge ? w0 : 0.0f, z1 >= edge ? w1 : 0.0f));
            } else {
                part = add2(part, w);
            }
        }
        sum = add2(sum, part);
    });
    float s0, s1, l0, l1;
    unpack2(sum, s0, s1);
    unpack2(large, l0, l1);
    u64 others = warp_sum((u64)__float2ll_rn((s0 + s1) * 0x1p44f)), listed = warp_sum((u64)__float2ll_rn((l0 + l1) * 0x1p44f));
    if (row.lane < row.CS()) {
        CutShared* o = row.of(&sh, row.lane);
        o->part_mass[row.rank() * CL_WARPS + row.warp] = others;
        o->part_all[row.rank() * CL_WARPS + row.warp] = listed;
    }
    row.sync();
    others = listed = 0;
    for (int w = row.lane; w < row.CS() * CL_WARPS; w += 32) {
        others += sh.part_mass[w];
        listed += sh.part_all[w];
    }
    others = warp_sum(others);
    listed = warp_sum(listed);
    about = (float)(others + listed);
    // (the sum is right to 2^-15)
    if (threadIdx.x == 0) set_unit(sh.s, unit_of(about * 0x1.0008p-44f));
    __syncthreads();
    if ((float)listed < about * top_p) return 0;  // (what is near is left to the exact passes)
    n = gather(row, lo, highest);
    if (row.rank() == 0) {
        u64 place = 0;
        if (n <= CL_LIST) {
            sort_list(sh, (int)n, lo, highest);
            u64 m = 0;
            for (int i = threadIdx.x; i < (int)n; i += CL_THREADS) m += weight(key_value<BF16>(place_key(sh.list[i])), row.s(), sh.exp);
            block_scan(m, sh.warp_mass, row.lane, row.warp, listed);
            // (2^18: the units to which the warps' sums were rounded, and more)
            const int up = row.s().unit - 44;
            const u64 error = ((others >> 15) + (1ull << 18)) << up;
            others <<= up;
            const u64 goal = goal_of(top_p, listed + others - min(others, error)), goal_hi = goal_of(top_p, listed + others + error);
            place = reach_in_list(row, (int)n, false, 0, goal, goal_hi);
        }
        __syncthreads();
        if (threadIdx.x == 0) row.each_cta([&](CutShared* o) { o->found_place = place; });
    }
    row.sync();
    const u64 place = sh.found_place;
    if (place == 0) row.sync();  // everyone has read it
    return place;
}

// The n-th sequence when those whose rows may need all their weights summed come
// first: top-p without a short top-k, or a draw from a row that no top-k cuts short.
// (256 rows of 151936 bf16, drawn with no cut or top-k 50 by sequence: 70 us with top-p's
// alone first, 62 so; 700 of 128256 fp32: 159, 120.)
constexpr int CL_ORDERED = 4 * CL_THREADS;  // sequences at most
template <bool DRAW>
__device__ __forceinline__ int longest_first(const CutParams& P, CutShared& sh, int n, int lane, int warp) {
    constexpr int PER = CL_ORDERED / CL_THREADS;
    const int first = PER * threadIdx.x;
    uint32_t slow = 0, all;
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int i = first + q;
        if (i >= P.B) continue;
        const float T = P.temperatures ? P.temperatures[i] : P.temperature, p = P.top_ps ? P.top_ps[i] : P.top_p;
        const int k = P.top_ks ? P.top_ks[i] : P.top_k;
        if (T != 0.0f && (DRAW || p < 1.0f) && (k <= 0 || k >= P.V || k > CL_LIST)) slow |= 1u << q;
    }
    const uint32_t mine = __popc(slow);
    int before = (int)(block_scan(mine, sh.warp_count, lane, warp, all) - mine);
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int i = first + q;
        const bool s = slow >> q & 1u;
        if (i < P.B && n == (s ? before : (int)all + i - before)) sh.sequence = i;
        before += s;
    }
    __syncthreads();
    return sh.sequence;
}

template <bool BF16, bool DRAW>
__global__ void __launch_bounds__(CL_THREADS, 2) cut_logits_kernel(const __grid_constant__ CutParams P) {
    cluster_arrive_started();
    using R = Row<BF16>;
    extern __shared__ __align__(16) char smem[];
    CutShared& sh = *reinterpret_cast<CutShared*>(smem);
    const int tid = threadIdx.x;
    R row;
    row.lane = tid & 31;
    row.warp = tid >> 5;
    row.sh = &sh;
    const int CS = (int)cg::this_cluster().num_blocks(), rank = (int)cg::this_cluster().block_rank(), lane = row.lane, warp = row.warp;

    if (tid < CL_EXP) sh.exp[tid] = g_exp_table.e[tid];
    grid_dependency_wait();
    launch_dependents();

    // Which row. Where there are more than run at once, those that take longest come
    // first, lest one begins when the others are done.
    int b = blockIdx.x / CS / P.R;
    const int r = blockIdx.x / CS - b * P.R;
    if (P.longest_first) b = longest_first<DRAW>(P, sh, b, lane, warp);
    const int64_t at_row = (int64_t)b * P.R + r;
    const char* src = P.logits + b * P.seq_bytes + r * P.row_bytes;
    const int lead = (int)(reinterpret_cast<uintptr_t>(src) & 15) / R::ES;  // elements before the row in its first piece
    if (tid == 0) {
        sh.src = src;
        set_part<BF16>(sh, lead, P.V, rank * P.slice_vecs, P.slice_vecs, CS, rank);
    }
    if (tid == 0) sh.first_largest = INT32_MAX;
    __syncthreads();
    // behind the last key up to whole 16 bytes
    if (tid < (-row.n_vecs() & 7)) row.keys()[row.n_vecs() + tid] = 0;

    const float T = P.temperatures ? P.temperatures[b] : P.temperature;
    const int top_k = P.top_ks ? P.top_ks[b] : P.top_k;
    const float top_p = P.top_ps ? P.top_ps[b] : P.top_p, min_p = P.min_ps ? P.min_ps[b] : P.min_p;
    const bool settings_ok = (T == 0.0f || (T >= 0x1p-64f && T <= 0x1p64f)) && top_k >= 0 && top_p >= 0.0f && top_p <= 1.0f &&
                             min_p >= 0.0f && min_p <= 1.0f;
    const int k = T == 0.0f ? 1 : top_k > 0 && top_k < P.V ? top_k : P.V;
    const float u = DRAW ? P.uniforms[at_row] : 0.0f;
    if (tid == CL_THREADS - 1) {
        const double inv_t = T == 0.0f ? 1.0 : 1.0 / (double)T, c = 1.4426950408889634 * CL_EXP * inv_t;
        sh.inv_t = inv_t;
        sh.ch = (float)c;
        sh.cl = (float)(c - (double)sh.ch);
        sh.low_by = (float)(100.0 * CL_EXP / 1.4426950408889634 / CL_EXP) * (T == 0.0f ? 1.0f : T);
        const double d = min_p > 0.0f && T != 0.0f ? (double)T * log((double)min_p) : 0.0;
        sh.min_hi = (float)d;
        sh.min_lo = (float)(d - (double)sh.min_hi);
    }

    // A row that nothing cuts is written as it is read.
    char* out = nullptr;
    bool same = false, through = false;
    uint4* copy_to = nullptr;
    if constexpr (!DRAW) {
        out = P.out + b * P.out_seq_bytes + r * P.out_row_bytes;
        same = (reinterpret_cast<uintptr_t>(out) & 15) == (uintptr_t)(lead * R::ES);
        through = same && k >= P.V && top_p >= 1.0f && min_p == 0.0f;
        if (through && out != src) copy_to = reinterpret_cast<uint4*>(out + (int64_t)sh.first * R::ES);
    }

    // 1. The maximum and the pieces' keys.
    float top;
    {
        constexpr int U = 8;
        uint32_t most = BF16 ? 0xFF80FF80u : 0xFF800000u;
        int v = row.v0() + lane;
        const int end = min(row.v1(), row.sh->full1);
        if (v < row.sh->full0 && v < row.v1()) {
            row.keys()[v] = R::piece_key(load_part<BF16>(row.sh->src, P.V, row.index(v), R::MINUS_INF), most);
            v += 32;
        }
        for (; v + 32 * (U - 1) < end; v += 32 * U) {
            uint4 x[U];
#pragma unroll
            for (int q = 0; q < U; ++q) x[q] = R::load_whole(sh.base + v + 32 * q);
#pragma unroll
            for (int q = 0; q < U; ++q) row.keys()[v + 32 * q] = R::piece_key(x[q], most);
            if (!DRAW && copy_to) {
#pragma unroll
                for (int q = 0; q < U; ++q) __stcs(copy_to + v + 32 * q, x[q]);
            }
        }
        {
            uint4 x[U];
#pragma unroll
            for (int q = 0; q < U; ++q)
                if (v + 32 * q < end) x[q] = R::load_whole(sh.base + v + 32 * q);
#pragma unroll
            for (int q = 0; q < U; ++q)
                if (v + 32 * q < end) row.keys()[v + 32 * q] = R::piece_key(x[q], most);
            if (!DRAW && copy_to) {
#pragma unroll
                for (int q = 0; q < U; ++q)
                    if (v + 32 * q < end) __stcs(copy_to + v + 32 * q, x[q]);
            }
        }
        const int last = row.v1() - 1;
        if (last >= max(row.sh->full1, row.v0()) && last >= row.sh->full0 && ((last - row.v0()) & 31) == lane)
            row.keys()[last] = R::piece_key(load_part<BF16>(row.sh->src, P.V, row.index(last), R::MINUS_INF), most);
        top = BF16 ? max_nan(bf16_lo(most), bf16_hi(most)) : __uint_as_float(most);
    }
    // The maxima of groups of lanes: so many that enough lie above what is looked for
    // and the smallest part of a row is between (a quarter more groups than k, all
    // that there is room for in top-p's first try).
    const int warps = CS * CL_WARPS, wanted = k == 1 ? 1 : k < P.V ? (k < CL_GROUPS ? k + k / 4 : CL_GROUPS) : CL_GROUPS / 2;
    int per_warp = 1;
    while (warps * per_warp < wanted && warps * per_warp < CL_GROUPS) per_warp *= 2;
    const int groups = warps * per_warp, width = 32 / per_warp;
    float least = top > -INFINITY ? top : INFINITY, group = top;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        if (o < width) group = max_nan(group, __shfl_xor_sync(0xFFFFFFFFu, group, o));
        least = fminf(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
    }
    cluster_wait_started();
    if (lane < CS) row.of(sh.lane_min, lane)[rank * CL_WARPS + warp] = least;
    if (lane % width == 0)
        for (int c = 0; c < CS; ++c) row.of(sh.group_max, c)[(rank * CL_WARPS + warp) * per_warp + lane / width] = group;
    row.sync();
    float row_top = -INFINITY;
    least = INFINITY;
    for (int w = lane; w < groups; w += 32) row_top = max_nan(row_top, sh.group_max[w]);
    for (int w = lane; w < warps; w += 32) least = fminf(least, sh.lane_min[w]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        row_top = max_nan(row_top, __shfl_xor_sync(0xFFFFFFFFu, row_top, o));
        least = fminf(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
    }
    const bool row_ok = row_top < INFINITY && row_top > -INFINITY;
    u64 cut = CL_LOWEST;  // what is kept lies at or above it
    if (!row_ok || !settings_ok) {
        if (rank == 0 && tid == 0) {
            raise_flag(P.status, (row_ok ? 0u : (uint32_t)SV_FLAG_BAD_ROW) | (settings_ok ? 0u : (uint32_t)SV_FLAG_BAD_SETTING));
            if constexpr (DRAW) {
                P.tokens[at_row] = -1;
                if (P.logprobs) P.logprobs[at_row] = __int_as_float(0x7fc00000);
            } else {
                if (P.n_kept) P.n_kept[at_row] = -1;
            }
        }
        if constexpr (DRAW) return;
    } else {
        const RowScale& s = sh.s;
        if (tid == 0) {
            set_scale(sh.s, row_top, sh.ch, sh.cl, sh.low_by);
            set_unit(sh.s, unit_of((float)k));  // (the sum is not above that)
        }
        __syncthreads();
        const u64 highest = (u64)key_of<BF16>(s.top) << CL_INDEX_BITS | CL_INDEX_MASK;
        // min-p: z >= max + T ln(min_p)
        if (min_p > 0.0f && T != 0.0f) {
            // the smallest float that is not below the sum of three
            const ff sum = two_sum(s.top, sh.min_hi);
            const float rest = __fadd_rn(sum.lo, sh.min_lo);
            const float z = rest > 0.0f ? from_key32(key32(sum.hi) + 1) : sum.hi;
            // bf16 keys of negative values end in ones, those of others in zeros
            const uint32_t kz = key32(z), key = !BF16 ? kz : (kz >> 31) ? (uint32_t)(((u64)kz + 0xFFFFu) >> 16) : kz >> 16;
            cut = max(cut, (u64)key << CL_INDEX_BITS);
        }
        const bool by_k = k < P.V, by_p = T != 0.0f && top_p < 1.0f;
        bool summed = false;  // part_mass holds the sums at or above the cut
        if (k == 1) {
            // the first of the largest
            const int first = first_largest(row, highest & ~(u64)CL_INDEX_MASK);
            if constexpr (DRAW) {
                if (rank == 0 && tid == 0) {
                    P.tokens[at_row] = first;
                    if (P.logprobs) P.logprobs[at_row] = 0.0f;
                }
                return;
            }
            cut = place_of(place_key(highest), first);
        } else if (by_k) {
            // 2. a bound on the k-th largest
            u64 bound = CL_LOWEST;
            if (k <= groups) {
                bound = max(bound, (u64)key_of<BF16>(nth_group(sh, groups, k - 1)) << CL_INDEX_BITS);
            } else if (least < s.top) {
                // that of the pieces', by a histogram between the lanes' smallest
                // maximum and the row's
                const float to_bin = (float)(CL_BINS - 1) / __fsub_rn(s.top, least);
                if (to_bin < INFINITY) {
                    clear_bins(row);
                    const uint4* keys = reinterpret_cast<const uint4*>(row.keys());
                    const uint32_t lo16 = key32(least) >> 16;
                    for (int g = tid; g * 8 < row.n_vecs(); g += CL_THREADS) {
                        const uint4 k8 = keys[g];
                        const uint32_t w[4] = {k8.x, k8.y, k8.z, k8.w};
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint32_t key = (w[i / 2] >> (16 * (i % 2))) & 0xFFFFu;
                            if (key < lo16 || g * 8 + i >= row.n_vecs()) continue;
                            const float y = __fmul_rn(__fsub_rn(s.top, from_key32(key << 16 | (BF16 && !(key >> 15) ? 0xFFFFu : 0u))), to_bin);
                            atomicAdd(&sh.count[max(0, min((int)y, CL_BINS - 1))], 1u);
                        }
                    }
                    find_bin(row, (float)k, 0.0f, 0);
                    if (sh.found_bin < CL_BINS - 1) {
                        const float z = __fsub_rn(s.top, (float)(sh.found_bin + 1) / to_bin * 1.0001f);
                        bound = max(bound, (u64)key_of<BF16>(z - fabsf(z) * 1e-6f) << CL_INDEX_BITS);
                    }
                }
            }
            // (what min-p drops counts too: it is among the k)
            uint32_t n = gather(row, bound, highest);
            bool listed = n <= CL_LIST;
            if (!listed) {
                const u64 cut_k = find_cut<BF16, false>(row, bound, highest, (uint32_t)k, 0.0f);
                if (k <= CL_LIST) {
                    n = gather(row, cut_k, highest);
                    listed = true;
                } else {
                    if (by_p) {
                        // (the sum in floats gives the unit alone)
                        refine_unit(row, sum_above(row, cut_k));
                        row.sync();
                        cut = max(cut, find_cut<BF16, true>(row, cut_k, highest, 0, top_p));
                    }
                    cut = max(cut, cut_k);
                }
            }
            if (listed) {
                // The cuts, in the list.
                if (rank == 0) {
                    const int all = min((int)n, CL_LIST);
                    sort_list(sh, all, bound, highest);
                    const int of_k = min(all, k);
                    u64 last = of_k > 0 ? sh.list[of_k - 1] : 0;
                    if (by_p) {
                        u64 m = 0, total;
                        for (int i = tid; i < of_k; i += CL_THREADS) m += weight(key_value<BF16>(place_key(sh.list[i])), s, row.sh->exp);
                        const u64 incl = block_scan(m, sh.warp_mass, lane, warp, total), goal = goal_of(top_p, total);
                        if (of_k <= CL_THREADS) {  // an entry per thread: what it added up is there
                            if (tid == 0) sh.found_place = 0;
                            __syncthreads();
                            if (tid < of_k && incl >= goal && (tid == 0 || incl - m < goal)) sh.found_place = sh.list[tid];
                            __syncthreads();
                            last = max(last, sh.found_place);
                        } else {
                            last = max(last, reach_in_list(row, of_k, false, 0, goal, goal));
                        }
                    }
                    last = max(last, cut);
                    if constexpr (DRAW) {
                        // how many of the sorted places are kept
                        int kept = 0;
                        for (int i = tid; i < of_k; i += CL_THREADS) kept += sh.list[i] >= last;
                        uint32_t total;
                        block_scan((uint32_t)kept, sh.warp_count, lane, warp, total);
                        draw_list(P, row, at_row, u, (int)total);
                    } else {
                        __syncthreads();
                        if (tid == 0) row.each_cta([&](CutShared* o) { o->found_place = last; });
                    }
                }
                if constexpr (DRAW) return;
                row.sync();
                cut = sh.found_place;
            }
        } else if (by_p) {
            float about;  // the sum of all weights, nearly
            uint32_t listed_n;
            u64 cut_p = cut_near_top(row, top_p, groups, highest, about, listed_n);
            if (cut_p) {
                cut = max(cut, cut_p);
                if constexpr (DRAW) {
                    if (rank == 0) {
                        uint32_t kept = 0, total;
                        for (int i = tid; i < (int)listed_n; i += CL_THREADS) kept += sh.list[i] >= cut;
                        block_scan(kept, sh.warp_count, lane, warp, total);
                        draw_list(P, row, at_row, u, (int)total);
                    }
                    return;
                }
            } else {
                cut_p = cut_by_mass(row, top_p, T, highest, about);
                summed = cut_p >= cut;
                cut = max(cut, cut_p);
            }
        }
        if constexpr (DRAW) {
            if (!summed) {
                row.sync();
                sum_above(row, cut);
            }
            if (draw_parts(P, row, at_row, u, cut, false)) return;
            sum_alone(row, cut);
            draw_parts(P, row, at_row, u, cut, true);
            return;
        }
    }
    if constexpr (!DRAW) {
        // 5. the row's output
        const bool valid = row_ok && settings_ok;
        constexpr uint32_t NONE = BF16 ? 0xFF80FF80u : 0xFF800000u;
        uint32_t kept = 0;
        const auto put = [&](int v, const uint4& x) {
            const int i0 = row.index(v);
            if (same && !row.partial(v)) {
                __stcs(reinterpret_cast<uint4*>(out + (int64_t)i0 * R::ES), x);  // (not read again: 2304 rows 243 us without, 229 so)
                return;
            }
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < R::E; ++e) {
                if (i0 + e < 0 || i0 + e >= P.V) continue;
                if constexpr (BF16) reinterpret_cast<uint16_t*>(out)[i0 + e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
                else reinterpret_cast<uint32_t*>(out)[i0 + e] = w[e];
            }
        };
        if (!valid || through) {
            for (int v = row.v0() + lane; v < row.v1(); v += 32)
                if (!through || row.partial(v)) put(v, row.load(v));
            if (valid && rank == 0 && tid == 0) kept = P.V;
        } else {
            const uint32_t lo16 = R::lo16_of(cut);
            for (int v = row.v0() + lane; v < row.v1(); v += 32)
                if (row.keys()[v] < lo16) put(v, make_uint4(NONE, NONE, NONE, NONE));
            each_hit(row, cut, [&](int v, const uint4& x, bool on) {
                if (!on) return;
                const int i0 = row.index(v);
                uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < R::E; ++e) {
                    if (place_of(key_of<BF16>(piece_elem<BF16>(x, e)), i0 + e) >= cut) {
                        ++kept;
                    } else {
                        if constexpr (BF16) w[e / 2] = e % 2 ? (w[e / 2] & 0xFFFFu) | 0xFF800000u : (w[e / 2] & 0xFFFF0000u) | 0xFF80u;
                        else w[e] = 0xFF800000u;
                    }
                }
                put(v, make_uint4(w[0], w[1], w[2], w[3]));
            });
        }
        if (P.n_kept && valid) {
            kept = __reduce_add_sync(0xFFFFFFFFu, kept);
            row.sync();
            if (lane == 0) row.of(&sh, 0)->part_mass[rank * CL_WARPS + warp] = kept;
            row.sync();
            if (rank == 0 && warp == 0) {
                u64 n = 0;
                for (int w = lane; w < warps; w += 32) n += sh.part_mass[w];
                n = warp_sum(n);
                if (lane == 0) P.n_kept[at_row] = (int32_t)n;
            }
        } else {
            row.sync();  // no CTA ends while another may look into its memory
        }
    }
}

// ---------------------------------------------------------------------------
// Launch.
// ---------------------------------------------------------------------------
constexpr int CL_ONE = 226 * 1024;  // shared memory of a CTA at most

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
    // Few rows are spread over several CTAs each, down to 4 pieces per thread: as
    // many as fill two per SM. Where a row may need its weights summed, a lone CTA's
    // row would keep all others waiting, so up to 4 CTAs per row while that makes no
    // more than 8 per SM (192 rows of 128256 fp32 with mixed settings: 214 us with
    // one CTA, 145 with two, 125 with four; the largest of 256 rows of 151936 bf16
    // alone: 16 us with one, 31 with four).
    const bool sums = !(!p.temperatures && p.temperature == 0.0f) && !(!p.top_ks && p.top_k > 0 && p.top_k <= CL_LIST);
    int cs = 1;
    while (cs < CL_MAX_CS && rows * cs <= (cs < 4 ? (int64_t)sms * (sums ? 4 : 1) : sms / 2) && vecs / cs > 4 * CL_THREADS) cs *= 2;
    p.slice_vecs = (vecs + cs - 1) / cs;
    const int smem = (int)sizeof(CutShared) + (p.slice_vecs + 15) / 8 * 16;
    if (smem > CL_ONE || rows * cs > INT32_MAX) return cudaErrorInvalidValue;
    p.longest_first = (p.temperatures || p.top_ks || p.top_ps) && p.B <= CL_ORDERED && rows * cs > 2 * sms;
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
