// The pages of a paged key/value cache, handed out on the GPU: every sequence
// holds as many as its context and new tokens need, what it has too many goes
// back on the stack of free pages, and the new tokens' slots follow.
//
// With need_b = ceil((ctx_b + new_b) / page_size): the pages of b's table from
// need_b on go on the stack, by sequence and place; then the missing ones are
// taken from its top in the same order, sequence b's i-th from below those of
// the sequences before it. Both places are prefix sums over the sequences
// (a scan), so the result is one that a loop over them would give.
//
// A step's call moves a few kilobytes and is all latency: lengths, scan, pushes,
// pops and rows depend on one another. One cluster of CTAs does it: each scans
// all sequences for itself (a few coalesced loads, no exchange), pushes its
// share, and after one cluster barrier, when the stack is whole, pops and writes
// its share of the tables and rows. Old lengths are kept in shared memory, so
// that the ones in place can be replaced meanwhile.
#include <cooperative_groups.h>

#include <atomic>

#include "paged_device.cuh"

namespace cg = cooperative_groups;

namespace sv {

constexpr int KP_THREADS = 512;
constexpr int KP_WARPS = KP_THREADS / 32;
constexpr int KP_CTAS = 8;

struct KpSequence {
    int lo, held;  // first row; pages held before, -1: left out
    int push, pop; // pages given back and wanted by the sequences before
    int ctx;
};

__device__ __forceinline__ int2 warp_scan2(int2 v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, v.x, o), y = __shfl_up_sync(0xFFFFFFFFu, v.y, o);
        if (lane >= o) v.x += x, v.y += y;
    }
    return v;
}

__global__ void __launch_bounds__(KP_THREADS, 1) kv_pages_kernel(const __grid_constant__ KvPagesParams P) {
    cluster_arrive_started();
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), CS = (int)cluster.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    extern __shared__ __align__(16) KpSequence seq[];  // [B + 1]
    __shared__ int2 warp_sums[KP_WARPS];
    __shared__ int taken;
    if (tid == 0) taken = 0;
    grid_dependency_wait();
    launch_dependents();

    // lengths and both prefix sums; every CTA for itself
    const int n_free = *P.n_free;
    int2 run = make_int2(0, 0);
    bool torn = n_free < 0 || n_free > P.n_pages, bad = false;
    for (int base = 0; base < P.B; base += KP_THREADS) {
        const int b = base + tid;
        int lo = 0, held = -1, ctx = 0;
        int2 mine = make_int2(0, 0);
        if (b < P.B) {
            lo = P.cu[b];
            const int hi = P.cu[b + 1], has = P.held[b];
            ctx = P.ctx[b];
            const bool rows_ok = lo >= 0 && lo <= hi && hi <= P.T;
            torn |= !rows_ok;
            const bool ok = rows_ok && ctx >= 0 && has >= 0 && has <= P.max_pages &&
                            (long long)ctx + (hi - lo) <= (long long)P.max_pages * P.page_size;
            if (ok) {
                held = has;
                const int need = (int)(((long long)ctx + (hi - lo) + P.page_size - 1) / P.page_size);
                mine = make_int2(max(has - need, 0), max(need - has, 0));
            } else {
                bad = true;
            }
        }
        const int2 incl = warp_scan2(mine, lane);
        __syncthreads();
        if (lane == 31) warp_sums[warp] = incl;
        __syncthreads();
        int2 before = run;
        for (int w = 0; w < KP_WARPS; ++w) {
            const int2 t = warp_sums[w];
            if (w < warp) before.x += t.x, before.y += t.y;
            run.x += t.x, run.y += t.y;
        }
        if (b < P.B) seq[b] = KpSequence{lo, held, before.x + incl.x - mine.x, before.y + incl.y - mine.y, ctx};
    }
    if (tid == 0) seq[P.B] = KpSequence{P.cu[P.B], -1, run.x, run.y, 0};
    // (more pages than there are: the sequences hold some twice)
    torn |= (long long)n_free + run.x > P.n_pages;
    torn = __syncthreads_or(torn);
    bad = __syncthreads_or(bad);
    const int top = torn ? 0 : n_free + run.x;
    if ((bad || torn) && rank == 0 && tid == 0) raise_flag(P.status, SV_FLAG_BAD_LENGTH);

    // The pages that move are numbered by sequence and place, and go round the
    // cluster's threads; f(b, i): the i-th of sequence b's. (With a warp per sequence
    // a few sequences that want hundreds of pages kept one warp busy: 30 us.)
    const auto each_page = [&](int KpSequence::*first, int count, auto&& f) {
        for (int x = rank * KP_THREADS + tid; x < count; x += CS * KP_THREADS) {
            int b = 0, end = P.B;  // first[b] <= x < first[end]
            while (end - b > 1) {
                const int mid = (b + end) >> 1;
                if (seq[mid].*first <= x) b = mid;
                else end = mid;
            }
            f(b, x - seq[b].*first);
        }
    };
    if (!torn) {
        each_page(&KpSequence::push, run.x, [&](int b, int i) {
            const int give = seq[b + 1].push - seq[b].push;
            int32_t* entry = P.table + (int64_t)b * P.table_stride + seq[b].held - give + i;
            const int page = *entry;
            if (page < 0 || page >= P.n_pages) raise_flag(P.status, SV_FLAG_BAD_PAGE);
            P.free_pages[n_free + seq[b].push + i] = page;
            *entry = -1;
        });
    }
    cluster_wait_started();
    cluster.sync();
    // the stack is whole, and every CTA has read the lengths

    // Page `i` from the stack's top.
    const auto popped = [&](int i) {
        const int page = P.free_pages[top - 1 - i];
        if (page < 0 || page >= P.n_pages) raise_flag(P.status, SV_FLAG_BAD_PAGE);
        return page;
    };
    if (!torn) {
        each_page(&KpSequence::pop, min(run.y, top), [&](int b, int i) {
            if (seq[b + 1].pop > top) return;  // not enough for all of its own: it gets none
            P.table[(int64_t)b * P.table_stride + seq[b].held + i] = popped(seq[b].pop + i);
        });
        int most = 0;
        bool none = false;
        for (int b = tid; b < P.B; b += KP_THREADS) {
            const KpSequence s = seq[b], after = seq[b + 1];
            const int give = after.push - s.push, want = after.pop - s.pop;
            const bool granted = want > 0 && after.pop <= top;
            none |= want > 0 && !granted;
            if (granted) most = max(most, after.pop);
            if (b % CS == rank && (give > 0 || granted)) P.held[b] = s.held - give + want;
        }
        if (rank == 0) {
            if (none) raise_flag(P.status, SV_FLAG_NO_PAGES);
            most = __reduce_max_sync(0xFFFFFFFFu, most);
            if (lane == 0 && most > 0) atomicMax(&taken, most);
            __syncthreads();
            if (tid == 0) *P.n_free = top - taken;
        }
    }
    if (P.slots || P.positions) {
        // A warp has a run of rows; a lane searches its first row's sequence and
        // steps on from there. Four rows at a time, so that their pages' loads fly
        // together (65,521 rows: 10.7 us one by one, 9.0 so).
        constexpr int U = 4;
        const int warps = CS * KP_WARPS;
        const long long per = ((P.T + (long long)warps - 1) / warps + 31) / 32 * 32;
        const int t0 = (int)min((rank * KP_WARPS + warp) * per, (long long)P.T), t1 = (int)min(t0 + per, (long long)P.T);
        const int first = seq[0].lo, past = seq[P.B].lo;
        int b = -1;
        for (long long tt = t0 + lane; tt < t1; tt += 32 * U) {
            int pos[U], page[U], in_page[U];
#pragma unroll
            for (int q = 0; q < U; ++q) {
                pos[q] = page[q] = -1;
                in_page[q] = 0;
                const long long tq = tt + 32 * q;
                if (tq >= t1 || torn || tq < first || tq >= past) continue;
                const int t = (int)tq;
                if (b < 0) {
                    int hi = P.B;  // seq[b].lo <= t < seq[hi].lo
                    b = 0;
                    while (hi - b > 1) {
                        const int mid = (b + hi) >> 1;
                        if (seq[mid].lo <= t) b = mid;
                        else hi = mid;
                    }
                }
                while (seq[b + 1].lo <= t) ++b;
                const KpSequence s = seq[b];
                if (s.held < 0) continue;
                pos[q] = s.ctx + (t - s.lo);
                const int j = (int)((uint32_t)pos[q] / (uint32_t)P.page_size);
                in_page[q] = pos[q] - j * P.page_size;
                if (j < s.held) page[q] = P.table[(int64_t)b * P.table_stride + j];
                else if (seq[b + 1].pop <= top) page[q] = P.free_pages[top - 1 - (s.pop + j - s.held)];
                else in_page[q] = -1;  // no page for it
            }
#pragma unroll
            for (int q = 0; q < U; ++q) {
                const long long t = tt + 32 * q;
                if (t >= t1) continue;
                const bool there = page[q] >= 0 && page[q] < P.n_pages;
                if (!there && pos[q] >= 0 && in_page[q] >= 0) raise_flag(P.status, SV_FLAG_BAD_PAGE);
                if (P.slots) P.slots[t] = there ? (int64_t)page[q] * P.page_size + in_page[q] : -1;
                if (P.positions) P.positions[t] = pos[q];
            }
        }
    }
}

cudaError_t launch_kv_pages(const KvPagesParams& p, cudaStream_t stream) {
    const int smem = (p.B + 1) * (int)sizeof(KpSequence);
    static std::atomic<int> attr_done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_done[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kv_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (KP_MAX_SEQUENCES + 1) * (int)sizeof(KpSequence));
        if (e != cudaSuccess) return e;
        attr_done[dev].store(1, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(KP_CTAS, 1, 1);
    cfg.blockDim = dim3(KP_THREADS, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = KP_CTAS;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kv_pages_kernel, p);
}

}  // namespace sv
