// Device helpers shared by the paged cache's kernels.
#pragma once

#include "paged.h"
#include "sv_device.cuh"

namespace sv {

__device__ __forceinline__ void raise_flag(uint32_t* status, uint32_t bits) {
    if (status) atomicOr(status, bits);
}

// A kernel that waits for all work before it lets the next one start only after
// that wait: a verify call with SV_ARG_OVERLAP_PREVIOUS reads its inputs before
// its own wait, and the work before this kernel may have written them.

// Lengths, tables, parents and results come from the kernels before, which may
// still run when this one starts: they are read after the grid's wait, and by
// plain loads, since a read-only load may use a line that was cached before.
// (A step's commit writes the lengths that the next step's append, started
// beside it, reads.)

// One sequence's chunk: n new tokens at packed rows q0.., ctx tokens before
// them in the cache. rows_ok: the packed rows themselves lie inside [0, T).
// ok also asks that the tokens fit the page table and, in a tree, that there
// is a parent for each.
struct Chunk {
    int q0, n, ctx;
    bool rows_ok, ok;
};

__device__ __forceinline__ Chunk load_chunk(const ChunkParams& p, int b) {
    Chunk s;
    const int lo = p.cu[b], hi = p.cu[b + 1];
    s.ctx = p.ctx[b];
    s.q0 = lo;
    s.rows_ok = lo >= 0 && lo <= hi && hi <= p.T;
    s.n = s.rows_ok ? hi - lo : 0;
    s.ok = s.rows_ok && s.ctx >= 0 && (long long)s.ctx + s.n <= (long long)p.max_pages * p.page_size &&
           (!p.parents || s.n <= p.N);
    return s;
}

// The page that holds slot `slot` of sequence b, or -1 (and its flag) where
// the table has none.
__device__ __forceinline__ int page_of(const ChunkParams& p, int b, int slot) {
    const int page = p.table[(int64_t)b * p.table_stride + slot / p.page_size];
    if (page >= 0 && page < p.n_pages) return page;
    raise_flag(p.status, SV_FLAG_BAD_PAGE);
    return -1;
}

// Warp-wide: lane i gets the set of nodes at or above node i in a tree of n
// <= 32 nodes (bit j: node j), by repeatedly joining a node's set with that
// of the highest node it has reached (5 doublings cover 32 nodes). Node 0 is
// the root; a node whose chain of parents has one outside [0, node) gets the
// empty set, and its lane raises the flag.
__device__ __forceinline__ uint32_t tree_sets(const ChunkParams& p, int b, int n, int lane) {
    int up = lane > 0 && lane < n ? p.parents[(int64_t)b * p.N + lane] : 0;
    bool good = lane == 0 || lane >= n || (up >= 0 && up < lane);
    if (!good) {
        raise_flag(p.status, SV_FLAG_BAD_TREE);
        up = 0;
    }
    uint32_t set = 1u << lane;
#pragma unroll
    for (int r = 0; r < 5; ++r) {
        set |= __shfl_sync(0xFFFFFFFFu, set, up);
        good = (__shfl_sync(0xFFFFFFFFu, (int)good, up) != 0) && good;
        up = __shfl_sync(0xFFFFFFFFu, up, up);
    }
    return good && lane < n ? set : 0u;
}

}  // namespace sv
