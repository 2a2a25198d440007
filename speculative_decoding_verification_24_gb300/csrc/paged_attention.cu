// Attention of each sequence's new tokens over its paged cache:
//   o[t, h] = sum_j softmax_j(scale q[t, h] . k[j, h / G]) v[j, h / G]
// over the slots j that token t sees (its context and itself; in a chain the
// chunk's tokens before it, in a tree its ancestors).
//
// One kernel for one token, a few drafts, a tree and a prompt's chunk. The G
// query heads of a kv head are packed with the tokens into rows (row = token
// * G + head), so keys and values are read once for all of them. A tile is
// 128 rows x 128 keys:
//   S = Q K^T        tcgen05.mma, both operands in shared memory, S in TMEM;
//   P = 2^(c S - m)  one thread per row: its 128 scores in registers, the
//                    running maximum m and sum l of a one-pass softmax (Milakov
//                    and Gimelshein, 2018), P rounded to the cache's type, as
//                    the product takes it, and written over S in TMEM;
//   O += P V         tcgen05.mma, P from TMEM, V from shared memory, O in TMEM.
// m is only raised (and O and l rescaled) when a score passes it by more than
// 2^8, as later work on attention has it: l and O share whatever m is used, so
// the result does not depend on it, and most tiles touch no O at all. In fp16 m lies 7 below the maximum: P is
// then at most 2^15 (65504 is the largest), and a weight is off by half a step
// of its own or 2^-32 of the row's largest (half the step of the subnormals,
// 2^-25, over 2^7). At the maximum itself that would be 2^-25, and 131,000 keys
// of 2^-25.2 beside one of 1 lost all of their 0.3 %, 7 half steps of the output.
//
// Two softmax warpgroups keep the tensor cores and the softmax busy at once:
// while one computes P, the other's products run. A chunk of more than 128
// rows gives each its own 128 rows and both use every key tile ("pair"); with
// at most 128 rows both hold the same rows, take alternate key tiles and join
// their (m, l, O) at the end ("split"), which for few rows halves the chain of
// dependent steps per byte.
//
// Work is counted in key tiles (and some units per item) over all (sequence,
// head, row tile) items in that order, and every CTA takes an equal, contiguous
// share of the total, cutting items where its share ends: one long context
// spreads over the whole GPU, and so does a ragged batch, without the host
// knowing the lengths. A cut item's pieces are written as (m, l, unscaled O) in
// fp32 and joined in order by whichever CTA finishes last, so the result does
// not depend on timing.
//
// What bounds it, with 32 query and 8 kv heads of 128 in bf16 (copy rate 6789
// GB/s, cuBLAS 1909 TFLOP/s):
//   many rows per key: a stream's chain. A tile's products take 1024 cycles of
//     the tensor cores per stream, its softmax about 1650 from scores to P, and
//     the next scores wait for O += P V, since P lies over S; two streams
//     overlap them, at about 2900 cycles for both streams' tiles. 4096 tokens
//     over 12288: 547-606 us replayed from a graph, 1.59-1.76 PFLOP/s, 83-92 %;
//     called one after another, at the power limit, 611-617 us, 82 %. With D =
//     64 the products halve and the chain stays: 434 us, 58 %.
//   few rows: HBM. 256 single tokens over up to 8192 keys each: 629-648 us,
//     6.7-6.9 TB/s, 99-101 % of the copy rate.
//   little work: latency. One token over 500 keys: 11 us, of which 2.3 find the
//     share, 2 bring the first scores, 3.4 are two tiles per stream, and 2.2
//     the join of the streams and the output.
//
// Warps: 0-3 and 4-7 softmax and output, 8 keys and 10 values (TMA, one box per
// page or 128 tokens), 9 the products, 11 queries (TMA).
// Every mbarrier wait is bounded (about a second; that for a buffer of queries
// by the share's length as well); one that gives up sets SV_FLAG_TIMEOUT, the
// others stop waiting, no further work is issued, what was issued is waited
// for, TMEM is freed and the rows concerned are NaN.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "paged_device.cuh"

namespace sv {

constexpr int PA_THREADS = 384;
constexpr int PA_SOFTMAX_THREADS = 256;
constexpr long long PA_WAIT_CYCLES = 1ll << 31;  // a wait gives up after about a second
constexpr long long PA_UNIT_CYCLES = 1ll << 13;  // more than a tile takes (3000); for waits that last as long as an item
constexpr float PA_RAISE = 8.0f;                 // log2 of how far the maximum may pass m (with PA_F16_BELOW)
constexpr float PA_F16_BELOW = 7.0f;             // how far m lies below the maximum in fp16, log2
constexpr int PA_TMEM_COLS = 512;                // S0, S1 (128 columns each), O0, O1 (D each)
constexpr int PA_SLAB_BYTES = PA_TILE * 128;     // 128 rows of 64 elements: one 128-byte-swizzled operand block

template <int D>
struct PaShape {
    static constexpr int SLABS = D / 64;
    static constexpr int TILE_BYTES = SLABS * PA_SLAB_BYTES;  // 128 rows of Q, K or V
    static constexpr int STAGES = 160 * 1024 / TILE_BYTES;    // K and V tiles in flight: 160 KB
    static constexpr int TILES_BYTES = (2 + STAGES) * TILE_BYTES;
};

// ---------------------------------------------------------------------------
// tcgen05 wrappers.
// ---------------------------------------------------------------------------
// Shared-memory matrix descriptor, 128-byte swizzle: start address, leading
// and stride byte offsets (all >> 4), descriptor version 1, layout code 2.
__device__ __forceinline__ uint64_t pa_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
           (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Instruction descriptor of kind::f16: fp32 accumulator, A and B both f16 or
// both bf16, 128 x n; b_mn: B is stored with n contiguous.
__host__ __device__ constexpr uint32_t pa_idesc(bool f16, int n, bool b_mn) {
    return (1u << 4) | (f16 ? 0u : (1u << 7) | (1u << 10)) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(PA_TILE >> 4) << 24);
}

// The products and commits are predicated, not branched to: `issue` is set in
// one lane of a converged warp.
// S = Q K^T: A and B from shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate, uint32_t issue) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(issue)
        : "memory");
}

// O += P V: A from TMEM.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate, uint32_t issue) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(issue)
        : "memory");
}

__device__ __forceinline__ void mma_commit(uint64_t* bar, uint32_t issue) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "setp.ne.b32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        ::"r"(smem_u32(bar)), "r"(issue)
        : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one;
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A warp's 32 lanes x n columns, one row per lane. The wait is part of the
// statement, so that no use of the registers can be scheduled before it.
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// Two such blocks at once.
__device__ __forceinline__ void tmem_ld2(uint32_t ta, uint32_t tb, uint32_t (&a)[32], uint32_t (&b)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%65];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]),
          "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]),
          "=r"(a[16]), "=r"(a[17]), "=r"(a[18]), "=r"(a[19]), "=r"(a[20]), "=r"(a[21]), "=r"(a[22]), "=r"(a[23]),
          "=r"(a[24]), "=r"(a[25]), "=r"(a[26]), "=r"(a[27]), "=r"(a[28]), "=r"(a[29]), "=r"(a[30]), "=r"(a[31]),
          "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]), "=r"(b[7]),
          "=r"(b[8]), "=r"(b[9]), "=r"(b[10]), "=r"(b[11]), "=r"(b[12]), "=r"(b[13]), "=r"(b[14]), "=r"(b[15]),
          "=r"(b[16]), "=r"(b[17]), "=r"(b[18]), "=r"(b[19]), "=r"(b[20]), "=r"(b[21]), "=r"(b[22]), "=r"(b[23]),
          "=r"(b[24]), "=r"(b[25]), "=r"(b[26]), "=r"(b[27]), "=r"(b[28]), "=r"(b[29]), "=r"(b[30]), "=r"(b[31])
        : "r"(ta), "r"(tb)
        : "memory");
}

__device__ __forceinline__ void tmem_ld2(uint32_t ta, uint32_t tb, uint32_t (&a)[64], uint32_t (&b)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%128];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
        "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, "
        "%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, "
        "%112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%129];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]),
          "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]),
          "=r"(a[16]), "=r"(a[17]), "=r"(a[18]), "=r"(a[19]), "=r"(a[20]), "=r"(a[21]), "=r"(a[22]), "=r"(a[23]),
          "=r"(a[24]), "=r"(a[25]), "=r"(a[26]), "=r"(a[27]), "=r"(a[28]), "=r"(a[29]), "=r"(a[30]), "=r"(a[31]),
          "=r"(a[32]), "=r"(a[33]), "=r"(a[34]), "=r"(a[35]), "=r"(a[36]), "=r"(a[37]), "=r"(a[38]), "=r"(a[39]),
          "=r"(a[40]), "=r"(a[41]), "=r"(a[42]), "=r"(a[43]), "=r"(a[44]), "=r"(a[45]), "=r"(a[46]), "=r"(a[47]),
          "=r"(a[48]), "=r"(a[49]), "=r"(a[50]), "=r"(a[51]), "=r"(a[52]), "=r"(a[53]), "=r"(a[54]), "=r"(a[55]),
          "=r"(a[56]), "=r"(a[57]), "=r"(a[58]), "=r"(a[59]), "=r"(a[60]), "=r"(a[61]), "=r"(a[62]), "=r"(a[63]),
          "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]), "=r"(b[7]),
          "=r"(b[8]), "=r"(b[9]), "=r"(b[10]), "=r"(b[11]), "=r"(b[12]), "=r"(b[13]), "=r"(b[14]), "=r"(b[15]),
          "=r"(b[16]), "=r"(b[17]), "=r"(b[18]), "=r"(b[19]), "=r"(b[20]), "=r"(b[21]), "=r"(b[22]), "=r"(b[23]),
          "=r"(b[24]), "=r"(b[25]), "=r"(b[26]), "=r"(b[27]), "=r"(b[28]), "=r"(b[29]), "=r"(b[30]), "=r"(b[31]),
          "=r"(b[32]), "=r"(b[33]), "=r"(b[34]), "=r"(b[35]), "=r"(b[36]), "=r"(b[37]), "=r"(b[38]), "=r"(b[39]),
          "=r"(b[40]), "=r"(b[41]), "=r"(b[42]), "=r"(b[43]), "=r"(b[44]), "=r"(b[45]), "=r"(b[46]), "=r"(b[47]),
          "=r"(b[48]), "=r"(b[49]), "=r"(b[50]), "=r"(b[51]), "=r"(b[52]), "=r"(b[53]), "=r"(b[54]), "=r"(b[55]),
          "=r"(b[56]), "=r"(b[57]), "=r"(b[58]), "=r"(b[59]), "=r"(b[60]), "=r"(b[61]), "=r"(b[62]), "=r"(b[63])
        : "r"(ta), "r"(tb)
        : "memory");
}

__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[128]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x128.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63, "
        "%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
        "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, "
        "%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, "
        "%112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%128];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]),
          "=r"(r[64]), "=r"(r[65]), "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]),
          "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]), "=r"(r[79]),
          "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]), "=r"(r[84]), "=r"(r[85]), "=r"(r[86]), "=r"(r[87]),
          "=r"(r[88]), "=r"(r[89]), "=r"(r[90]), "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95]),
          "=r"(r[96]), "=r"(r[97]), "=r"(r[98]), "=r"(r[99]), "=r"(r[100]), "=r"(r[101]), "=r"(r[102]), "=r"(r[103]),
          "=r"(r[104]), "=r"(r[105]), "=r"(r[106]), "=r"(r[107]), "=r"(r[108]), "=r"(r[109]), "=r"(r[110]), "=r"(r[111]),
          "=r"(r[112]), "=r"(r[113]), "=r"(r[114]), "=r"(r[115]), "=r"(r[116]), "=r"(r[117]), "=r"(r[118]), "=r"(r[119]),
          "=r"(r[120]), "=r"(r[121]), "=r"(r[122]), "=r"(r[123]), "=r"(r[124]), "=r"(r[125]), "=r"(r[126]), "=r"(r[127])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {"
        "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// A split item's keys and values are read once: marked to be evicted first,
// they do not push the kernel's own code out of L2. A pair's are read again by
// the CTAs of the chunk's other rows.
__device__ __forceinline__ uint64_t l2_evict_normal_policy() {
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int token, int head, int page,
                                            uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(token), "r"(head), "r"(page), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int head, int token, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(head), "r"(token), "r"(smem_u32(bar))
        : "memory");
}

// Waits for a phase; gives up after `cycles`, or at once when any wait of the
// CTA has given up and `err` is passed.
__device__ __forceinline__ bool pa_wait_until(uint64_t* bar, uint32_t parity, const int* err, long long cycles = PA_WAIT_CYCLES) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long start = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (err && *(volatile const int*)err) return false;
        if (clock64() - start > cycles) return mbar_try_wait(bar, parity);
    }
    return true;
}
__device__ __forceinline__ void pa_wait(uint64_t* bar, uint32_t parity, int* err, long long cycles = PA_WAIT_CYCLES) {
    if (!pa_wait_until(bar, parity, err, cycles)) atomicExch(err, 1);
}
__device__ __forceinline__ bool pa_failed(const int* err) { return *(volatile const int*)err != 0; }

// Named barrier 1: the 256 softmax threads (barrier 0 is __syncthreads).
__device__ __forceinline__ void softmax_barrier() {
    asm volatile("bar.sync 1, %0;" ::"n"(PA_SOFTMAX_THREADS) : "memory");
}

// ---------------------------------------------------------------------------
// Work: items in the order (sequence, kv head, row tile), laid end to end on
// one axis of W units. A unit is a key tile; an item begins with PA_ITEM_COST
// units for what it takes besides its tiles (first scores, output, and joining
// both streams: about 5000 cycles, a tile takes 1400 to 3000).
// ---------------------------------------------------------------------------
// sum over i < n of floor((a i + b) / 128). With a = 2^k (TT a power of two)
// the terms are floor((i + b / a) / q), q = 128 / a: runs of q equal ones.
// Otherwise the points below a line are counted by Euclid's algorithm on (a, m),
// the axes changing places at each step, the usual way for such sums (Graham,
// Knuth and Patashnik, Concrete Mathematics, section 3.5, treats them).
__device__ __noinline__ uint32_t floor_sum(uint32_t n, uint32_t a, uint32_t b) {
    const auto pairs_below = [](uint32_t x) { return (uint32_t)((uint64_t)x * (x - 1) / 2); };
    uint32_t m = PA_TILE, ans = n * (b / m) + pairs_below(n) * (a / m);
    a %= m;
    b %= m;
    if (a == 0 || n == 0) return ans;
    if ((a & (a - 1)) == 0) {
        const int k = 31 - __clz(a), q_shift = 7 - k;
        const auto below = [&](uint32_t x) {  // sum over i < x of floor(i / q)
            const uint32_t t = x >> q_shift;
            return (pairs_below(t) << q_shift) + t * (x - (t << q_shift));
        };
        return ans + below(n + (b >> k)) - below(b >> k);
    }
    while (true) {
        const uint64_t y = (uint64_t)a * n + b;
        if (y < m) return ans;
        n = (uint32_t)(y / m);
        b = (uint32_t)(y - (uint64_t)n * m);
        const uint32_t t = m;
        m = a;
        a = t;
        ans += n * (b / m) + pairs_below(n) * (a / m);
        a %= m;
        b %= m;
    }
}

__device__ __forceinline__ int tiles_of(int end) { return (int)(((long long)end + PA_TILE - 1) / PA_TILE); }

// Row tiles pair up; row-tile pair p covers tokens [2 TT p, 2 TT (p + 1)).
__device__ __forceinline__ int pairs_of(int n, int TT) { return n <= TT ? 1 : (n + 2 * TT - 1) / (2 * TT); }

// Units of one kv head's first p pairs (p < pairs: none of them the last).
__device__ __forceinline__ int units_before(int ctx, int TT, int p) {
    return p == 0 ? 0 : (int)floor_sum(p, 2 * TT, (uint32_t)ctx + 2 * TT + PA_TILE - 1) + p * PA_ITEM_COST;
}
__device__ __forceinline__ int units_per_head(int n, int ctx, int TT) {
    return n == 0 ? 0 : units_before(ctx, TT, pairs_of(n, TT) - 1) + tiles_of(ctx + n) + PA_ITEM_COST;
}

// The next sequence after b that has work; b becomes its number.
__device__ __forceinline__ Chunk next_chunk(const ChunkParams& ch, int& b) {
    Chunk s;
    int at = b;
    do {
        s = load_chunk(ch, ++at);
    } while (at + 1 < ch.B && (!s.ok || s.n == 0));
    b = at;
    return s;
}

// A walk over the items of a CTA's share, computed alike by every role. Places
// on the axis are int32: the host refuses batches whose bound on the
// total is larger.
struct Cursor {
    int begin, end;         // this CTA's share
    int u0;                 // where the current item begins
    int b, h, p;            // sequence, kv head, row-tile pair
    Chunk s;
    int tok0, ntok, tiles;  // the item's tokens within the chunk, its key tiles

    __device__ __forceinline__ void set_item(const PagedAttnParams& P) {
        tok0 = 2 * P.TT * p;
        ntok = min(s.n - tok0, 2 * P.TT);
        tiles = tiles_of(s.ctx + tok0 + ntok);
    }
    __device__ __forceinline__ bool valid() const { return u0 < end; }
    __device__ __forceinline__ void next(const PagedAttnParams& P) {
        u0 += PA_ITEM_COST + tiles;
        if (u0 >= end) return;
        if (tok0 + ntok == s.n) {
            p = 0;
            if (++h == P.ch.Hkv) {
                h = 0;
                // u0 < end <= W, so a later sequence has work
                s = next_chunk(P.ch, b);
            }
        } else {
            ++p;
        }
        set_item(P);
    }
    // the part of the item in this share
    __device__ __forceinline__ int t0() const { return max(begin - u0 - PA_ITEM_COST, 0); }
    __device__ __forceinline__ int t1() const { return min(end - u0 - PA_ITEM_COST, tiles); }
    __device__ __forceinline__ bool pair(const PagedAttnParams& P) const { return ntok > P.TT; }
};

// CTA c's share begins at u_c: W = active * size + extra, the first `extra`
// shares one unit longer. A boundary moves to an item's edge when it falls
// within PA_SNAP tiles of one: a piece of a few tiles costs more in joining
// than the uneven share does.
constexpr int PA_SNAP = 3;
struct Shares {
    int W, active, size, extra;

    __device__ __forceinline__ int begin(int c) const { return c * size + min(c, extra); }
    // the first boundary at or past x > 0
    __device__ __forceinline__ int first_at(int x) const {
        // unsigned: x + size may pass 2^31
        const uint32_t n = (uint32_t)size, longer = (uint32_t)extra * (n + 1), u = (uint32_t)x;
        return (int)(u <= longer ? (u + n) / (n + 1) : (uint32_t)extra + (u - longer + n - 1) / n);
    }
};
// A CTA gets at least this many units: below that, joining costs more than
// another CTA saves.
constexpr int PA_MIN_SHARE = 4;

struct PaShared {
    int scan[PA_THREADS / 32];
    Cursor at[2];
    Shares shares;
    uint64_t full[10], empty[10], s_full[2], p_half[2], p_full[2], o_full[2], q_full[2], q_empty[2], mma_done, never;
    float2 ml[2][PA_TILE];
    int loads[2][10];       // by producer and stage: phases of `full` up to its latest load
    int q_loads[2];         // the same of q_full
    uint32_t tmem;
    int last;               // this CTA finished an item last (1), and add_not_finite is due (2)
    int not_finite;         // a value that was cleared was not finite; stays set
    int err;
};
template <int D>
constexpr int PA_SMEM = PaShape<D>::TILES_BYTES + (int)sizeof(PaShared);
static_assert(PA_SMEM<64> <= 227 * 1024 && PA_SMEM<128> <= 227 * 1024, "shared memory of one CTA");

// Inclusive sums over the CTA's threads.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += t;
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    const int mine = lane < PA_THREADS / 32 ? warp_sums[lane] : 0;
    total = __reduce_add_sync(0xFFFFFFFFu, mine);
    return v + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? mine : 0);
}

// bad: a sequence that is left out; torn: its rows are not where rows can be.
__device__ __forceinline__ int sequence_units(const PagedAttnParams& P, int b, Chunk& s, bool& bad, bool& torn) {
    if (b >= P.ch.B) return 0;
    s = load_chunk(P.ch, b);
    bad |= !s.ok;
    torn |= !s.rows_ok;
    return s.ok ? units_per_head(s.n, s.ctx, P.TT) * P.ch.Hkv : 0;
}

// The item that holds place `raw`, in sequence b, whose items begin at `first`;
// c.begin: raw, or the item's edge if that is near.
__device__ __forceinline__ void place_boundary(const PagedAttnParams& P, const Shares& shares, int raw, int b, const Chunk& s, int first,
                                               int tiles, Cursor& out) {
    Cursor c;
    c.b = b;
    c.s = s;
    const int pairs = pairs_of(s.n, P.TT);
    const int per_head = (int)((uint32_t)tiles / (uint32_t)P.ch.Hkv), r = raw - first;
    c.h = (int)((uint32_t)r / (uint32_t)per_head);
    const int in_head = r - c.h * per_head;
    c.p = 0;
    int before = 0;
    if (pairs > 1) {
        // units_before(p) is close to p (ctx + TT + TT p) / 128 + p PA_ITEM_COST:
        // start from its root and step to the pair that holds in_head
        const float A = (float)P.TT, half = 0.5f * ((float)c.s.ctx + A + PA_TILE * PA_ITEM_COST);
        c.p = min(pairs - 1, max(0, (int)((sqrtf(half * half + A * (float)in_head * PA_TILE) - half) / A)));
        before = units_before(c.s.ctx, P.TT, c.p);
        while (before > in_head) before = units_before(c.s.ctx, P.TT, --c.p);
        while (c.p + 1 < pairs) {
            const int next = units_before(c.s.ctx, P.TT, c.p + 1);
            if (next > in_head) break;
            before = next;
            ++c.p;
        }
    }
    c.u0 = first + c.h * per_head + before;
    c.set_item(P);
    c.begin = raw;
    c.end = shares.W;
    const int item_end = c.u0 + PA_ITEM_COST + c.tiles;
    if (raw - c.u0 <= PA_ITEM_COST + PA_SNAP) {
        c.begin = c.u0;
    } else if (item_end - raw <= PA_SNAP) {
        c.begin = item_end;
        c.next(P);
    }
    out = c;
}

// Every thread: finds this CTA's share, and whether any sequence of the batch
// is left out (bad). Returns false when there is no work here.
__device__ __forceinline__ bool find_share(const PagedAttnParams& P, PaShared& sh, bool& bad) {
    const ChunkParams& ch = P.ch;
    const int tid = threadIdx.x;
    const bool one_turn = ch.B <= PA_THREADS;
    Chunk s = {};
    bool torn = false;
    int mine = sequence_units(P, tid, s, bad, torn), W;
    int incl = block_scan(mine, sh.scan, W);
    if (!one_turn) {
        for (int base = PA_THREADS; base < ch.B; base += PA_THREADS) {
            int total;
            __syncthreads();
            block_scan(sequence_units(P, base + tid, s, bad, torn), sh.scan, total);
            W += total;
        }
    }
    // Where cu_new descends, sequences may overlap, and their work may be more
    // than the host's bound on it: nothing is done.
    if (__syncthreads_or(torn)) {
        if (blockIdx.x == 0 && tid == 0) raise_flag(ch.status, SV_FLAG_BAD_LENGTH);
        bad = false;
        return false;
    }
    Shares shares = {};
    shares.W = W;
    shares.active = min((W + PA_MIN_SHARE - 1) / PA_MIN_SHARE, (int)gridDim.x);
    const bool here = (int)blockIdx.x < shares.active;
    int raw[2] = {0, 0};
    if (here) {
        shares.size = (int)((uint32_t)W / (uint32_t)shares.active);
        shares.extra = W - shares.size * shares.active;
        raw[0] = shares.begin(blockIdx.x);
        raw[1] = shares.begin(blockIdx.x + 1);
    }
    int run = 0;
    for (int base = 0; base < ch.B; base += PA_THREADS) {
        int total = 0;
        if (!one_turn) {
            bool again = false;
            __syncthreads();
            mine = sequence_units(P, base + tid, s, again, again);
            incl = block_scan(mine, sh.scan, total);
        }
        const int excl = run + incl - mine;
#pragma unroll 1
        for (int k = 0; k < 2; ++k)
            if (here && raw[k] >= excl && raw[k] < excl + mine) place_boundary(P, shares, raw[k], base + tid, s, excl, mine, sh.at[k]);
        run += total;
    }
    if (tid == 0) {
        if (here && raw[1] == W) sh.at[1].begin = W;
        sh.shares = shares;
    }
    bad = __syncthreads_or(bad);
    if (bad && blockIdx.x == 0 && tid == 0) raise_flag(ch.status, SV_FLAG_BAD_LENGTH);
    if (!here) return false;
    return sh.at[0].begin < sh.at[1].begin;
}

// This CTA's share, as each role starts on it. Every role reads it for itself:
// kept in registers across the branch, it cost the softmax threads spills.
__device__ __forceinline__ Cursor share_of(const PaShared& sh) {
    Cursor c = sh.at[0];
    c.end = sh.at[1].begin;
    return c;
}

// The pieces an item is cut into: the first boundary inside it (the item
// begins in the CTA before) and how many pieces there are.
__device__ __forceinline__ void pieces_of(const Shares& w, const Cursor& c, int& first_cta, int& pieces) {
    // boundaries more than PA_SNAP tiles from both its edges cut it
    const int first = c.u0 + PA_ITEM_COST;
    const int c_lo = w.first_at(first + PA_SNAP + 1), c_end = w.first_at(first + c.tiles - PA_SNAP);
    first_cta = c_lo - 1;
    pieces = c_end - c_lo + 1;
}

// Which ring entries (K and V tiles, in the order the products use them) tile
// i of a piece of m tiles has. Pair: K0 V0 K1 V1 ...; split: K0 K1 V0 K2 V1
// ... V(m-1).
__device__ __forceinline__ int ring_k(bool pair, int i) { return pair ? 2 * i : (i == 0 ? 0 : 2 * i - 1); }
__device__ __forceinline__ int ring_v(bool pair, int i, int m) { return pair ? 2 * i + 1 : (i == m - 1 ? 2 * m - 1 : 2 * i + 2); }

// Query buffers: a pair's stream w uses buffer w; split items use one each, in
// turn, so that the next item's queries load while this one runs.
// A query buffer is free after two arrivals: one from each stream of a split
// item, both from the one stream that uses it in a pair. A stream arrives when
// its last scores have been formed; one that has no tiles here arrives only
// after a barrier with the other, when the products have long taken the
// buffer: an earlier arrival could let it be filled twice before they look.
__device__ __forceinline__ void release_q(uint64_t* bar, bool pair) {
    mbar_arrive(bar);
    if (pair) mbar_arrive(bar);
}

__device__ __forceinline__ float max3(float a, float b, float c) {  // drops NaN, as fmaxf does
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Bit 15 (31) is set where the low (high) half of a pair is not finite: an
// exponent of all ones and one more carries into the sign's place.
template <bool F16>
__device__ __forceinline__ uint32_t not_finite_pair(uint32_t w) {
    constexpr uint32_t EXP = F16 ? 0x7C007C00u : 0x7F807F80u, ONE = F16 ? 0x04000400u : 0x00800080u;
    return ((w & EXP) + ONE) & 0x80008000u;
}

// A tile of values, by `threads` threads of a stream: rows from r0 on lie past
// the last key and hold whatever the page does, and weight 0 times infinity is
// not 0, so they become 0; rows from r1 on are not seen by every row of the
// item, and what is not finite there becomes 0 (see add_not_finite).
template <int D, bool F16>
__device__ __forceinline__ void clean_values(uint4* tile, int r1, int r0, int* not_finite, int thread, int threads) {
    constexpr int SLABS = D / 64, SLAB = PA_SLAB_BYTES / 16;
#pragma unroll 1
    for (int x = r1 * 8 + thread; x < r0 * 8; x += threads) {
        uint4 v[SLABS];
        bool bad = false;
#pragma unroll
        for (int j = 0; j < SLABS; ++j) v[j] = tile[j * SLAB + x];
#pragma unroll
        for (int j = 0; j < SLABS; ++j)
            bad |= (not_finite_pair<F16>(v[j].x) | not_finite_pair<F16>(v[j].y) | not_finite_pair<F16>(v[j].z) | not_finite_pair<F16>(v[j].w)) != 0;
        if (!bad) continue;
        *(volatile int*)not_finite = 1;
#pragma unroll 1
        for (int k = 0; k < SLABS * 4; ++k) {
            uint32_t* u = reinterpret_cast<uint32_t*>(tile + (k / 4) * SLAB + x) + k % 4;
            const uint32_t n = not_finite_pair<F16>(*u);
            *u &= ((n & 0x8000u) ? 0u : 0xFFFFu) | ((n >> 31) ? 0u : 0xFFFF0000u);
        }
    }
#pragma unroll 1
    for (int x = r0 * 8 + thread; x < PA_TILE * 8; x += threads)
#pragma unroll
        for (int j = 0; j < SLABS; ++j) tile[j * SLAB + x] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
}

// From which token of the chunk on a key may be one that a row of the item that
// begins with token tok0 does not see.
// (The tiles that hold such keys, and the last one, are cleaned by the warps
// that have no rows, if there are any, while the others go on: one token over
// 500 keys 11.05 us, 11.35 when all clean first. Where all have rows their scan
// costs 3 % of a prompt of 4096 tokens, which has many short items, and nothing
// measurable of the same over 12288.)
__device__ __forceinline__ int mixed_from(const ChunkParams& ch, int tok0) { return ch.parents ? 1 : tok0 + 1; }

__device__ __forceinline__ uint32_t add_release_acquire(uint32_t* p, uint32_t x) {
    uint32_t before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(before) : "l"(p), "r"(x) : "memory");
    return before;
}

template <bool F16>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
    uint32_t r;
    if constexpr (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool F16>
__device__ __forceinline__ float to_float(uint16_t x) {
    return F16 ? __half2float(__ushort_as_half(x)) : __uint_as_float((uint32_t)x << 16);
}

// N values of each lane's output row, rounded once. A lane's row is a line of
// its own, and a store costs the memory pipe about 2.5 cycles per line (2600
// cycles for a tile's half of the columns), so with many rows (`dense`) groups
// of N / 8 lanes first exchange 16-byte pieces, each lane's row for one piece
// of each row of the group, and a store then writes whole rows. A few rows are
// stored as they lie: the exchange took longer (256 contexts of at most 400
// tokens, 4 rows: 112 us with it, 94 without; 64 trees of 128 rows: 72 and 74).
template <bool F16, int N>
__device__ __forceinline__ void store_rows(char* row, bool valid, bool dense, const float (&x)[N], int lane) {
    constexpr int NP = N / 8;
    uint32_t w[NP][4];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i / 4][i % 4] = pack_pair<F16>(x[2 * i], x[2 * i + 1]);
    if (!dense) {
        if (valid) {
#pragma unroll
            for (int c = 0; c < NP; ++c) reinterpret_cast<uint4*>(row)[c] = make_uint4(w[c][0], w[c][1], w[c][2], w[c][3]);
        }
        return;
    }
#pragma unroll
    for (int s = 1; s < NP; s <<= 1) {
        const bool high = (lane & s) != 0;
#pragma unroll
        for (int c = 0; c < NP; ++c) {
            if (c & s) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, high ? w[c][q] : w[c | s][q], s);
                w[c][q] = high ? got : w[c][q];
                w[c | s][q] = high ? w[c | s][q] : got;
            }
        }
    }
    const unsigned long long mine = valid ? reinterpret_cast<unsigned long long>(row) : 0ull;
    const int piece = lane % NP;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        char* to = reinterpret_cast<char*>(__shfl_sync(0xFFFFFFFFu, mine, lane - piece + i));
        if (to) *reinterpret_cast<uint4*>(to + piece * 16) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
    }
}

__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Where row (i, g) of a row tile, token i and head g of its group, lives in
// the batch. Rows past TT * G are nobody's.
struct RowPlace {
    int token, head;  // packed row of q and out, query head
    bool valid;
};
__device__ __forceinline__ RowPlace place_row(const PagedAttnParams& P, const Cursor& c, int tile, int i, int g) {
    RowPlace x;
    const int in_chunk = c.tok0 + tile * P.TT + i;
    x.valid = i < P.TT && in_chunk < c.tok0 + c.ntok;
    x.token = c.s.q0 + in_chunk;
    x.head = c.h * P.G + g;
    return x;
}

// One piece's O is kept as [D / 4][rows] groups of 4 columns, so that lanes
// that hold rows write and read neighbouring 16 bytes.
__device__ __forceinline__ size_t part_at(const PagedAttnParams& P, int D, int slot, int row, int group) {
    return ((size_t)slot * (D / 4) + group) * P.rows_cap + row;
}

// Joins an item's pieces in their order, by the CTA that finished last. A
// thread takes 8 columns of a row over all pieces; with few rows several
// lanes share them, each a contiguous run of the pieces, joined at the end.
// One online pass: the loads of 4 pieces of 3 such units are in flight together.
// 19 pieces of 36 rows of 128 columns: 8 us, 22 bytes a cycle.
template <int D, bool F16>
__device__ __forceinline__ void join_pieces(const PagedAttnParams& P, const Cursor& c, int first_cta, int pieces) {
    const bool pair = c.pair(P);
    const int rows0 = (pair ? P.TT : c.ntok) * P.G, rows = c.ntok * P.G, units = rows * (D / 8);
    int share = 0;  // log2 of the lanes per unit
    while (share < 5 && (units << share) < PA_SOFTMAX_THREADS && (2 << share) <= pieces) ++share;
    const int per_lane = (pieces + (1 << share) - 1) >> share;
    const int lane_of = threadIdx.x & ((1 << share) - 1);
    const int f0 = lane_of * per_lane, f1 = min(f0 + per_lane, pieces);
    constexpr int U = 3, F = 4;  // units and pieces whose loads are in flight together
    const int stride = PA_SOFTMAX_THREADS >> share;
    for (int base = 0; base < units; base += U * stride) {
        int group[U], row[U];
        bool on[U];
        const float4* o_of[U];
        const float2* ml_of[U];
        float M[U], L[U];
        f32x2 acc[U][4];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int u = base + j * stride + ((int)threadIdx.x >> share);
            on[j] = u < units;
            group[j] = on[j] ? u / rows : 0;
            const int r = on[j] ? u - group[j] * rows : 0;
            row[j] = r < rows0 ? r : PA_TILE + r - rows0;
            o_of[j] = reinterpret_cast<const float4*>(P.part_o) + part_at(P, D, 0, row[j], 2 * group[j]);
            ml_of[j] = P.part_ml + row[j];
            M[j] = -INFINITY, L[j] = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[j][k] = 0ull;
        }
#pragma unroll 1
        for (int fb = f0; fb < f1; fb += F) {
            float2 ml[U][F];
            float4 a[U][F], b[U][F];
#pragma unroll
            for (int j = 0; j < U; ++j)
#pragma unroll
                for (int k = 0; k < F; ++k) {
                    // past the last piece, or the last unit, a load repeats one
                    // and its weight is 0: no branch parts the loads
                    const int f = min(fb + k, f1 - 1), slot = f == 0 ? 2 * first_cta + 1 : 2 * (first_cta + f);
                    const float4* src = o_of[j] + (size_t)(uint32_t)slot * ((D / 4) * P.rows_cap);
                    ml[j][k] = __ldcg(ml_of[j] + (uint32_t)(slot * P.rows_cap));
                    a[j][k] = __ldcg(src);
                    b[j][k] = __ldcg(src + P.rows_cap);
                    if (fb + k >= f1) ml[j][k].y = 0.0f;
                }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                // one weight per piece and one for what was joined before; a
                // piece that saw nothing of the row has weight 0 and zeros for
                // O, and NaN stays NaN
                float m = M[j];
#pragma unroll
                for (int k = 0; k < F; ++k) m = fmaxf(m, ml[j][k].x);
                const float old = L[j] == 0.0f ? 0.0f : ex2(M[j] - m);
                M[j] = m;
                L[j] *= old;
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[j][q] = mul2(acc[j][q], pack2(old, old));
#pragma unroll
                for (int k = 0; k < F; ++k) {
                    const float w = ml[j][k].y == 0.0f ? 0.0f : ex2(ml[j][k].x - m);
                    const f32x2 ww = pack2(w, w);
                    L[j] = fmaf(w, ml[j][k].y, L[j]);
                    acc[j][0] = fma2(pack2(a[j][k].x, a[j][k].y), ww, acc[j][0]);
                    acc[j][1] = fma2(pack2(a[j][k].z, a[j][k].w), ww, acc[j][1]);
                    acc[j][2] = fma2(pack2(b[j][k].x, b[j][k].y), ww, acc[j][2]);
                    acc[j][3] = fma2(pack2(b[j][k].z, b[j][k].w), ww, acc[j][3]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            for (int o = 1; o < (1 << share); o <<= 1) {
                const float m2 = __shfl_xor_sync(0xFFFFFFFFu, M[j], o), l2 = __shfl_xor_sync(0xFFFFFFFFu, L[j], o);
                const float m = fmaxf(M[j], m2);
                const float w1 = L[j] == 0.0f ? 0.0f : ex2(M[j] - m), w2 = l2 == 0.0f ? 0.0f : ex2(m2 - m);
                M[j] = m;
                L[j] = L[j] * w1 + l2 * w2;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    acc[j][k] = fma2(__shfl_xor_sync(0xFFFFFFFFu, acc[j][k], o), pack2(w2, w2), mul2(acc[j][k], pack2(w1, w1)));
            }
            if (!on[j] || lane_of != 0) continue;
            const int r = row[j] % PA_TILE, i = r / P.G;
            const RowPlace at = place_row(P, c, row[j] / PA_TILE, i, r - i * P.G);
            const float inv = L[j] == 0.0f ? 0.0f : 1.0f / L[j];
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float lo, hi;
                unpack2(acc[j][k], lo, hi);
                w[k] = pack_pair<F16>(lo * inv, hi * inv);
            }
            *reinterpret_cast<uint4*>(P.out + at.token * P.o_ts + at.head * P.o_hs + group[j] * 16) = make_uint4(w[0], w[1], w[2], w[3]);
            if (P.lse && group[j] == 0) P.lse[(size_t)at.token * P.Hq + at.head] = lse_of(M[j], L[j]);
        }
    }
}

// ---------------------------------------------------------------------------
// Roles.
// ---------------------------------------------------------------------------
// Warps 8 and 10: keys and values. A tile is 128 / box boxes of `box` tokens
// (the largest power of two that divides the page, at most 128) per 64
// columns; a lane issues one. A warp issues its boxes one lane after another,
// so keys and values have a warp each: 256 contexts in pages of 16 (32 boxes of
// 2 KB for a tile's keys and values) took 936 us with one warp for both, at 68
// % of the copy rate, and 693 with two. A box past the piece's last key is not
// loaded. A page the table does not have reads as zeros (a page coordinate past
// the last one).
template <int D>
__device__ __forceinline__ void load_kv(const PagedAttnParams& P, PaShared& sh, uint32_t ring, const CUtensorMap* map,
                                        bool is_v, int lane) {
    using S = PaShape<D>;
    const ChunkParams& ch = P.ch;
    const int box_shift = P.box_shift;
    const int my_box = lane / S::SLABS, my_slab = lane % S::SLABS;
    const bool has_box = my_box < (PA_TILE >> box_shift);
    const uint32_t my_dst = ring + my_slab * PA_SLAB_BYTES + (my_box << (box_shift + 7));
    const uint64_t once = l2_evict_first_policy(), again = l2_evict_normal_policy();
    int ring0 = 0;
    bool stop = false;
    for (Cursor c = share_of(sh); c.valid() && !stop; c.next(P)) {
        const bool pair = c.pair(P);
        const int t0 = c.t0(), m = c.t1() - t0;
        const int key_end = c.s.ctx + c.tok0 + c.ntok;
        const int32_t* table = ch.table + (int64_t)c.b * ch.table_stride;
        // page of this lane's box of tile t, and its first entry there
        auto page_at = [&](int t) -> int2 {
            const int key = t * PA_TILE + (my_box << box_shift);
            if (!has_box || key >= key_end) return make_int2(-1, 0);
            const int page_no = key / ch.page_size;
            int page = table[page_no];
            if (page < 0 || page >= ch.n_pages) {
                raise_flag(ch.status, SV_FLAG_BAD_PAGE);
                page = ch.n_pages;
            }
            return make_int2(page, key - page_no * ch.page_size);
        };
        int2 page = page_at(t0);
        for (int i = 0; i < m && !stop; ++i) {
            const int2 here = page;
            if (i + 1 < m) page = page_at(t0 + i + 1);  // looked up a tile ahead
            const int e = ring0 + (is_v ? ring_v(pair, i, m) : ring_k(pair, i)), s = e % S::STAGES, n = e / S::STAGES;
            if (n > 0) pa_wait(&sh.empty[s], (n - 1) & 1, &sh.err);
            stop = __any_sync(0xFFFFFFFFu, pa_failed(&sh.err));
            if (stop) continue;
            const int keys = min(key_end - (t0 + i) * PA_TILE, PA_TILE);
            const int boxes = (keys + (1 << box_shift) - 1) >> box_shift;
            if (lane == 0) {
                sh.loads[is_v][s] = n + 1;
                mbar_arrive_expect_tx(&sh.full[s], (uint32_t)(boxes * S::SLABS) << (box_shift + 7));
            }
            __syncwarp();
            if (my_box < boxes)
                tma_load_4d(my_dst + s * S::TILE_BYTES, map, my_slab * 64, here.y, c.h, here.x, &sh.full[s], pair ? again : once);
        }
        ring0 += 2 * m;
    }
}

// Warp 11: the rows of Q, by boxes of q_box tokens x G heads x 64 columns,
// which lie in shared memory as the rows of a tile do. q_box divides TT, so
// no box passes the tile; rows past the item's are other tokens' or zeros,
// and nothing is read from theirs. (A warp that copied the rows by 16 bytes
// took 11 us for a pair's 64 KB, exposed at every item.)
template <int D>
__device__ __forceinline__ void load_q(const PagedAttnParams& P, PaShared& sh, uint32_t q_smem, const CUtensorMap* map,
                                       int lane) {
    using S = PaShape<D>;
    const uint32_t box_bytes = (uint32_t)(P.q_box * P.G) * 128u;
    int fills[2] = {0, 0}, turn = 0;
    // a buffer is free when the item's last scores have been formed: the wait
    // lasts as long as the item, which is part of the share
    const long long patience = PA_WAIT_CYCLES + (sh.at[1].begin - sh.at[0].begin) * PA_UNIT_CYCLES;
    for (Cursor c = share_of(sh); c.valid(); c.next(P)) {
        const bool pair = c.pair(P);
        const int split_buf = turn;
        if (!pair) turn ^= 1;
        for (int w = 0; w < (pair ? 2 : 1); ++w) {
            const int buf = pair ? w : split_buf;
            const int n = fills[buf]++;
            if (n > 0) pa_wait(&sh.q_empty[buf], (n - 1) & 1, &sh.err, patience);
            if (__any_sync(0xFFFFFFFFu, pa_failed(&sh.err))) return;
            const int tok = c.tok0 + w * P.TT, boxes = (min(P.TT, c.tok0 + c.ntok - tok) + P.q_box - 1) / P.q_box;
            if (lane == 0) {
                sh.q_loads[buf] = n + 1;
                mbar_arrive_expect_tx(&sh.q_full[buf], (uint32_t)(boxes * S::SLABS) * box_bytes);
            }
            __syncwarp();
            const uint32_t dst = q_smem + buf * S::TILE_BYTES;
            for (int x = lane; x < boxes * S::SLABS; x += 32) {
                const int box = x / S::SLABS, slab = x % S::SLABS;
                tma_load_3d(dst + slab * PA_SLAB_BYTES + box * box_bytes, map, slab * 64, c.h * P.G, c.s.q0 + tok + box * P.q_box,
                            &sh.q_full[buf]);
            }
        }
    }
}

// Warp 9: the products. Both warpgroups' streams alternate, and the scores of
// a stream's next tile are issued right after its O += P V, so that they run
// while the other warpgroup computes its P. O += P V begins with the first
// half of P. The instructions take their operands from uniform registers, so
// the whole warp walks the items, one elected lane's predicate issues, and
// what descriptors and branches come from passes through a warp reduction,
// whose result is known to be uniform: with operands from a lane's registers
// the 16 instructions of a tile took 1950 cycles to issue, twice what they
// take to run.
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xFFFFFFFFu, x); }

template <int D, bool F16>
__device__ __forceinline__ void issue_products(const PagedAttnParams& P, PaShared& sh, uint32_t q_smem, uint32_t ring,
                                               uint32_t tmem_any, uint32_t issue) {
    using S = PaShape<D>;
    constexpr uint32_t ID_S = pa_idesc(F16, PA_TILE, false), ID_O = pa_idesc(F16, D, true);
    constexpr int KS = PA_TILE / 16;
    const uint32_t tmem = (uint32_t)uniform((int)tmem_any);
    const uint64_t q_desc = pa_desc(q_smem, 16, 1024), k_desc = pa_desc(ring, 16, 1024), v_desc = pa_desc(ring, PA_SLAB_BYTES, 1024);
    int ring0 = 0, p_phase = 0, q_phase[2] = {0, 0}, turn = 0;
    for (Cursor c = share_of(sh); __any_sync(0xFFFFFFFFu, c.valid()); c.next(P)) {
        const bool pair = __any_sync(0xFFFFFFFFu, c.pair(P));
        const int m = uniform(c.t1() - c.t0());
        // the first tile past each stream's own
        const int last0 = pair ? max(0, min(uniform(tiles_of(c.s.ctx + c.tok0 + P.TT) - c.t0()), m)) : m;
        const int step = pair ? 1 : 2;
        if (pair || turn == 0) {
            pa_wait(&sh.q_full[0], q_phase[0], &sh.err);
            q_phase[0] ^= 1;
        }
        if (pair || turn == 1) {
            pa_wait(&sh.q_full[1], q_phase[1], &sh.err);
            q_phase[1] ^= 1;
        }
        const int buf0 = pair ? 0 : turn, buf1 = pair ? 1 : turn;
        if (!pair) turn ^= 1;
        auto wait_full = [&](int e) { pa_wait(&sh.full[e % S::STAGES], (e / S::STAGES) & 1, &sh.err); };
        // Stream w's step i: O += P V of its tile i, then the scores of its
        // next one; the first steps have only the latter. A wait takes about
        // 100 cycles even for what is there: each is made once, and between
        // products that keep the tensor cores busy meanwhile.
        for (int i = -step; i < m; ++i) {
            const int w0 = pair ? 0 : i & 1, w1 = pair ? 1 : i & 1;
#pragma unroll 1
            for (int w = w0; w <= w1; ++w) {
                const int last = w == 0 ? last0 : m, next = i + step;
                const bool values = i >= 0 && i < last, keys = next < last;
                // the last use of a tile's keys or values by any stream, and the first
                const bool alone = !pair || w == 1;
                const int ev = ring0 + ring_v(pair, i, m), sv = ev % S::STAGES;
                const int ek = ring0 + ring_k(pair, next), sk = ek % S::STAGES;
                const uint64_t b = v_desc + (uint32_t)(sv * (S::TILE_BYTES >> 4));
                const uint32_t o = tmem + 2 * PA_TILE + w * D, p = tmem + w * PA_TILE;
                const int phase = (p_phase >> w) & 1;
                if (values) {
                    p_phase ^= 1 << w;
                    if (!pair || w == 0 || i >= last0) wait_full(ev);
                    pa_wait(&sh.p_half[w], phase, &sh.err);
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < KS / 2; ++k)
                        mma_ts(o, p + k * 8, b + (uint32_t)(k * 2048 >> 4), ID_O, k != 0 ? 1 : i >= step, issue);
                }
                if (keys && (!pair || w == 0 || next >= last0)) wait_full(ek);
                if (values) {
                    pa_wait(&sh.p_full[w], phase, &sh.err);
                    tc_fence_after();
#pragma unroll
                    for (int k = KS / 2; k < KS; ++k) mma_ts(o, p + k * 8, b + (uint32_t)(k * 2048 >> 4), ID_O, 1, issue);
                    if (alone) mma_commit(&sh.empty[sv], issue);
                    if (!keys) mma_commit(&sh.o_full[w], issue);
                }
                if (keys) {
                    tc_fence_after();
                    const uint64_t qa = q_desc + (uint32_t)((w == 0 ? buf0 : buf1) * (S::TILE_BYTES >> 4));
                    const uint64_t kb = k_desc + (uint32_t)(sk * (S::TILE_BYTES >> 4));
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = ((k / 4) * PA_SLAB_BYTES + (k % 4) * 32) >> 4;
                        mma_ss(p, qa + off, kb + off, ID_S, k != 0, issue);
                    }
                    mma_commit(&sh.s_full[w], issue);
                    if (alone) mma_commit(&sh.empty[sk], issue);
                }
            }
            // after a wait that gave up: what was issued read whatever was there
            if (__any_sync(0xFFFFFFFFu, pa_failed(&sh.err))) return;
        }
        ring0 += 2 * m;
    }
}

// A value of the chunk that is not finite is no business of the rows that do
// not see it, but in the product their weight 0 makes NaN of it. So it is
// cleared in the tile, where rows exist that do not see it, and added here to
// the rows that do: as their weight is positive, out + value is what the sum
// with it gives. A rare path, which a CTA takes for all its items from the
// first such value on: everything is found again from the item, and nothing of
// the usual path is kept for it. A node of a broken tree sees nothing, but
// the product had its weight 0 meet the whole context and the root: its row
// becomes 0. A warp's lanes take their rows; of a split item warpgroup w takes
// half of the columns, as it wrote them.
template <int D, bool F16>
__device__ __noinline__ void add_not_finite(const PagedAttnParams& P, int b, int h, int q0, int n, int ctx, int tok0, int ntok, int w) {
    const ChunkParams& ch = P.ch;
    const int tid = threadIdx.x & 127, lane = threadIdx.x & 31;
    const bool pair = ntok > P.TT;
    __syncwarp();  // store_rows may have had other lanes write this lane's row
    const int i = tid / P.G, g = tid - i * P.G, node = tok0 + (pair ? w * P.TT : 0) + i;
    const bool valid = i < P.TT && node < tok0 + ntok;
    uint32_t set = 0;
    if (ch.parents) set = __shfl_sync(0xFFFFFFFFu, tree_sets(ch, b, n, lane), valid ? node : 0);
    if (!valid) return;
    const int key_end = ctx + tok0 + ntok;
    const bool broken = ch.parents && set == 0;
    char* out = P.out + (int64_t)(q0 + node) * P.o_ts + (h * P.G + g) * P.o_hs;
    for (int col = pair ? 0 : w * (D / 2); col < (pair ? D : (w + 1) * (D / 2)); col += 8) {
        if (broken) {
            *reinterpret_cast<uint4*>(out + col * 2) = make_uint4(0, 0, 0, 0);
            continue;
        }
        float sum[8] = {};
        uint32_t hit = 0;
        for (int j = ctx + mixed_from(ch, tok0); j < key_end; ++j) {
            if (ch.parents ? !(set >> (j - ctx) & 1u) : j > ctx + node) continue;
            const int page = ch.table[(int64_t)b * ch.table_stride + j / ch.page_size];
            if (page < 0 || page >= ch.n_pages) continue;
            const uint4 v = *reinterpret_cast<const uint4*>(P.vc + page * P.vc_ps + (j % ch.page_size) * P.vc_ts + h * P.vc_hs + col * 2);
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (!(not_finite_pair<F16>(u[k / 2]) >> (k % 2 ? 31 : 15) & 1u)) continue;
                sum[k] += to_float<F16>((uint16_t)(u[k / 2] >> (k % 2 ? 16 : 0)));
                hit |= 1u << k;
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (!(hit >> k & 1u)) continue;
            uint16_t* o = reinterpret_cast<uint16_t*>(out) + col + k;
            *o = (uint16_t)pack_pair<F16>(to_float<F16>(*o) + sum[k], 0.0f);
        }
    }
}

// Half of a row's columns, to the output or, of a cut item, to this CTA's piece.
template <int D, bool F16>
__device__ __forceinline__ void put_columns(const PagedAttnParams& P, const RowPlace& at, bool whole, int slot, int row, int col,
                                            const float (&x)[D / 2], bool dense, int lane) {
    if (whole) {
        store_rows<F16, D / 2>(P.out + at.token * P.o_ts + at.head * P.o_hs + col * 2, at.valid, dense, x, lane);
    } else if (at.valid) {
        float4* part = reinterpret_cast<float4*>(P.part_o) + part_at(P, D, slot, row, col / 4);
#pragma unroll
        for (int k = 0; k < D / 8; ++k)
            __stcg(part + k * P.rows_cap, make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]));
    }
}

// Joins an item of few pieces by the CTA that finished last, whose own piece is
// still in TMEM: a thread keeps to its row, takes 32 columns at a time and adds
// the pieces in their order, its own from TMEM (the values it stored, formed
// again) and the others' from memory. Two pieces of 128 rows: 1.6 us, where
// join_pieces takes 6.5. cols: [col, col_end) of this thread's row; a, b and
// sa, sb: the addresses and weights of its own O.
constexpr int PA_FEW_PIECES = 3;
template <int D, bool F16>
__device__ __forceinline__ void join_few(const PagedAttnParams& P, const RowPlace& at, int first_cta, int pieces, int row, float m,
                                         float l, int col, int col_end, uint32_t a_at, uint32_t b_at, float sa, float sb, bool both,
                                         bool none, bool dense, int lane) {
    const int own = (int)blockIdx.x - first_cta;
    const auto slot_of = [&](int f) { return f == 0 ? 2 * first_cta + 1 : 2 * (first_cta + f); };
    float2 ml[PA_FEW_PIECES];
    float M = -INFINITY, L = 0.0f;
#pragma unroll
    for (int f = 0; f < PA_FEW_PIECES; ++f) {
        ml[f] = make_float2(m, l);
        if (f < pieces && f != own) ml[f] = __ldcg(P.part_ml + (size_t)slot_of(f) * P.rows_cap + row);
        if (f < pieces) M = fmaxf(M, ml[f].x);
    }
#pragma unroll
    for (int f = 0; f < PA_FEW_PIECES; ++f) {
        ml[f].x = f >= pieces || ml[f].y == 0.0f ? 0.0f : ex2(ml[f].x - M);
        if (f < pieces) L = fmaf(ml[f].x, ml[f].y, L);
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll 1
    for (; col < col_end; col += 32) {
        float acc[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) acc[k] = 0.0f;
#pragma unroll
        for (int f = 0; f < PA_FEW_PIECES; ++f) {
            if (f >= pieces) break;
            const float w = ml[f].x;
            if (f == own) {
                uint32_t x[32], y[32];
                tmem_ld2(a_at + col, b_at + col, x, y);
#pragma unroll
                for (int k = 0; k < 32; ++k) {
                    float v = none ? 0.0f : __uint_as_float(x[k]) * sa;
                    v = both ? fmaf(__uint_as_float(y[k]), sb, v) : v;
                    acc[k] = fmaf(w, v, acc[k]);
                }
            } else {
                const float4* src = reinterpret_cast<const float4*>(P.part_o) + part_at(P, D, slot_of(f), row, col / 4);
                float4 v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = __ldcg(src + k * P.rows_cap);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    acc[4 * k] = fmaf(w, v[k].x, acc[4 * k]);
                    acc[4 * k + 1] = fmaf(w, v[k].y, acc[4 * k + 1]);
                    acc[4 * k + 2] = fmaf(w, v[k].z, acc[4 * k + 2]);
                    acc[4 * k + 3] = fmaf(w, v[k].w, acc[4 * k + 3]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) acc[k] *= inv;
        store_rows<F16, 32>(P.out + at.token * P.o_ts + at.head * P.o_hs + col * 2, at.valid, dense, acc, lane);
    }
    if (P.lse && at.valid) P.lse[(size_t)at.token * P.Hq + at.head] = lse_of(M, L);
}

// Warps 0-3 (w = 0) and 4-7 (w = 1): softmax and output.
template <int D, bool F16>
__device__ __forceinline__ void softmax_rows(const PagedAttnParams& P, PaShared& sh, int w,
                                             char* q_smem, char* ring, uint32_t tmem_base) {
    using S = PaShape<D>;
    const int tid = threadIdx.x & 127, lane = threadIdx.x & 31, warp = tid >> 5;
    const uint32_t lanes = (uint32_t)(32 * warp) << 16;
    const uint32_t tmem_s = tmem_base + lanes + w * PA_TILE, tmem_o = tmem_base + lanes + 2 * PA_TILE + w * D;
    const int row_token = tid / P.G, row_head = tid - row_token * P.G;
    int s_count = 0, o_count = 0, ring0 = 0, turn = 0;
    const f32x2 cc = pack2(P.c, P.c);
    for (Cursor c = share_of(sh); c.valid(); c.next(P)) {
        const bool pair = c.pair(P);
        const int t0 = c.t0(), t1 = c.t1(), m_tiles = t1 - t0;
        const int key_end = c.s.ctx + c.tok0 + c.ntok;
        const RowPlace at = place_row(P, c, pair ? w : 0, row_token, row_head);
        const int tok_first = c.tok0 + (pair ? w * P.TT : 0);
        const int tile_rows = min(P.TT, c.tok0 + c.ntok - tok_first) * P.G;
        const bool warp_on = 32 * warp < tile_rows;
        // keys [0, seen) are visible, and in a tree the chunk's nodes in `set`
        int seen = at.valid ? at.token - c.s.q0 + c.s.ctx + 1 : 0;
        int seen_by_all = c.s.ctx + tok_first + 1;
        uint32_t set = 0;
        if (P.ch.parents) {
            const uint32_t sets = tree_sets(P.ch, c.b, c.s.n, lane);
            set = __shfl_sync(0xFFFFFFFFu, sets, at.valid ? at.token - c.s.q0 : 0);
            if (!at.valid) set = 0;
            // a node with a bad chain of parents sees nothing
            seen = set ? c.s.ctx : 0;
            // (-1: add_not_finite is due, also where there is no context)
            seen_by_all = __all_sync(0xFFFFFFFFu, !at.valid || set) ? c.s.ctx : -1;
        }
        const int buf = pair ? w : turn;
        if (!pair) turn ^= 1;
        // this stream's tiles: first, first + step, ... below last
        const int step = pair ? 1 : 2;
        const int last0 = !pair ? m_tiles : max(0, min(m_tiles, tiles_of(c.s.ctx + c.tok0 + P.TT) - t0));
        const int last = w == 0 ? last0 : m_tiles;
        float m = -INFINITY;
        f32x2 l2 = pack2(0.0f, 0.0f);
        int done = 0;
        // From this tile on there are values that no row, or not every row, sees;
        // the stream whose product reads a tile first cleans it: the warps that
        // have no rows, while the others go on, or all of them.
        const int clean_from = max(pair && w == 1 ? last0 : 0, (c.s.ctx + mixed_from(P.ch, c.tok0)) / PA_TILE - t0);
        const int cleaner = tile_rows > PA_TILE - 32 ? 0 : (tile_rows + 31) / 32;  // the first warp that does
        for (int i = pair ? 0 : w; i < last; i += step, ++done) {
            pa_wait(&sh.s_full[w], s_count & 1, &sh.err);
            ++s_count;
            tc_fence_after();
            const int key0 = (t0 + i) * PA_TILE;
            // this stream's last scores have been formed: it needs Q no more
            if (i + step >= last && tid == 0) release_q(&sh.q_empty[buf], pair);
            if (i >= clean_from && warp >= cleaner) {
                const int e = ring0 + ring_v(pair, i, m_tiles), s = e % S::STAGES;
                pa_wait(&sh.full[s], (e / S::STAGES) & 1, &sh.err);
                clean_values<D, F16>(reinterpret_cast<uint4*>(ring + s * S::TILE_BYTES),
                                     max(c.s.ctx + mixed_from(P.ch, c.tok0) - key0, 0), min(key_end - key0, PA_TILE), &sh.not_finite,
                                     tid - 32 * cleaner, 128 - 32 * cleaner);
                __syncwarp();
            }
            if (warp_on) {
                uint32_t r[PA_TILE];
                tmem_ld(tmem_s, r);
                if (key0 + PA_TILE > seen_by_all) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int n = seen - key0 - 32 * q;
                        uint32_t on = n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
                        if (set) {  // node j is key ctx + j, bit ctx + j - key0 - 32 q
                            const int at0 = c.s.ctx - key0 - 32 * q;
                            if (at0 >= 0 && at0 < 32) on |= set << at0;
                            else if (at0 < 0 && at0 > -32) on |= set >> -at0;
                        }
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!((on >> k) & 1u)) r[32 * q + k] = 0xFF800000u;  // -inf, whatever stood there
                    }
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < PA_TILE; k += 8) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) mx[j] = max3(mx[j], __uint_as_float(r[k + 2 * j]), __uint_as_float(r[k + 2 * j + 1]));
                }
                const float most = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                const float top = F16 ? fmaf(most, P.c, -PA_F16_BELOW) : most * P.c;
                if (done == 0) {
                    m = top;
                } else {
                    const bool raise = at.valid && top > m + PA_RAISE;
                    if (__any_sync(0xFFFFFFFFu, raise)) {
                        // O of the tiles before is complete: these scores were issued after it
                        const float f = raise ? ex2(m - top) : 1.0f;
                        if (raise) m = top;
                        l2 = mul2(l2, pack2(f, f));
#pragma unroll 1
                        for (int col = 0; col < D; col += 16) {
                            uint32_t o[16];
                            tmem_ld(tmem_o + col, o);
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            tmem_st(tmem_o + col, o);
                        }
                    }
                }
                const float mu = m == -INFINITY ? 0.0f : -m;
                const f32x2 mm = pack2(mu, mu);
                // a tile's weights are added up before l takes them: one by one a
                // long context's small weights would be rounded away
                f32x2 sum = pack2(0.0f, 0.0f);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t pk[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const int at2 = 32 * q + 2 * k;
                        const f32x2 e = ex2x2(fma2(pack2(__uint_as_float(r[at2]), __uint_as_float(r[at2 + 1])), cc, mm));
                        sum = at2 == 0 ? e : add2(sum, e);
                        float a, b;
                        unpack2(e, a, b);
                        pk[k] = pack_pair<F16>(a, b);
                    }
                    tmem_st(tmem_s + 16 * q, pk);
                    if (q == 1) {  // the product may begin with the first 64 keys
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.p_half[w]);
                    }
                }
                l2 = add2(l2, sum);
                tmem_wait_st();
            } else if (lane == 0) {
                mbar_arrive(&sh.p_half[w]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.p_full[w]);
            
        }
        ring0 += 2 * m_tiles;
        float l;
        {
            float a, b;
            unpack2(l2, a, b);
            l = a + b;
        }
        if (pa_failed(&sh.err)) l = __int_as_float(0x7fc00000);

        // What this warpgroup writes: a pair's stream its own rows' columns, of a
        // split item's one half of the columns of both streams' O (a warp's
        // TMEM lanes are the same rows in either).
        if (done > 0) {
            pa_wait(&sh.o_full[w], o_count & 1, &sh.err);
            ++o_count;
            tc_fence_after();
        }
        float mt = m, lt = l, f[2];
        f[0] = f[1] = l == 0.0f ? 0.0f : 1.0f;
        if (!pair) {
            sh.ml[w][tid] = make_float2(m, l);
            tc_fence_before();
            softmax_barrier();  // both streams' O is complete
            tc_fence_after();
            if (done == 0 && tid == 0) release_q(&sh.q_empty[buf], false);
            const float2 other = sh.ml[w ^ 1][tid];
            mt = fmaxf(m, other.x);
            const float mine = l == 0.0f ? 0.0f : ex2(m - mt), theirs = other.y == 0.0f ? 0.0f : ex2(other.x - mt);
            f[0] = w == 0 ? mine : theirs;
            f[1] = w == 0 ? theirs : mine;
            // in the same order in both warpgroups: a joined item's weights are
            // those that either has formed, whichever CTA ends last
            lt = fmaf(w == 0 ? other.y : l, f[1], __fmul_rn(w == 0 ? l : other.y, f[0]));
        }

        const bool whole = t0 == 0 && t1 == c.tiles;
        const int slot = 2 * (int)blockIdx.x + (t0 == 0 ? 1 : 0);
        const int cap_row = (pair ? w * PA_TILE : 0) + tid;
        const float scale = !whole ? 1.0f : lt == 0.0f ? 0.0f : 1.0f / lt;
        if (warp_on) {
            constexpr int C = D / 2;
            const uint32_t o_base = tmem_base + lanes + 2 * PA_TILE;
            const float sa = f[0] * scale, sb = f[1] * scale;
            const bool both = !pair && m_tiles > 1;
            const int done0 = pair ? done : 1;
#pragma unroll 1
            for (int half = pair ? 0 : w; half <= (pair ? 1 : w); ++half) {
                uint32_t a[C], b[C];
                tmem_ld2((pair ? tmem_o : o_base) + half * C, o_base + D + half * C, a, b);
                float x[C];
#pragma unroll
                for (int k = 0; k < C; ++k) {
                    const float y = done0 == 0 ? 0.0f : __uint_as_float(a[k]) * sa;
                    x[k] = both ? fmaf(__uint_as_float(b[k]), sb, y) : y;
                }
                put_columns<D, F16>(P, at, whole, slot, cap_row, half * C, x, tile_rows > 32, lane);
            }
        }
        if (at.valid && (pair || w == 0)) {
            if (!whole) __stcg(P.part_ml + (size_t)slot * P.rows_cap + cap_row, make_float2(mt, lt));
            else if (P.lse) P.lse[(size_t)at.token * P.Hq + at.head] = lse_of(mt, lt);
        }
        // O has been read (by both warpgroups, if both read it): the next
        // item's products may overwrite it
        tc_fence_before();
        if (!pair) softmax_barrier();
        // whether the rows written here miss what add_not_finite adds
        bool written = whole, rest = whole && *(volatile int*)&sh.not_finite;
        if (!whole) {
            int first_cta, pieces;
            pieces_of(sh.shares, c, first_cta, pieces);
            softmax_barrier();  // both warpgroups' rows are written
            if (pair && done == 0 && tid == 0) release_q(&sh.q_empty[buf], true);
            if (threadIdx.x == 0) {
                // the barrier has brought every thread's rows to this one; its
                // release passes them on, its acquire brings the others'
                // (one piece more, and above them how many found values to add)
                const uint32_t found = *(volatile int*)&sh.not_finite ? 1u << 16 : 0u;
                const uint32_t before = add_release_acquire(P.counters + first_cta, 1u + found);
                sh.last = (before & 0xFFFFu) != (uint32_t)(pieces - 1) ? 0 : (before + found) >> 16 ? 3 : 1;
                if (sh.last) P.counters[first_cta] = 0;
            }
            softmax_barrier();
            const int joins = sh.last;
            if (joins) {
                if (pieces > PA_FEW_PIECES) {
                    join_pieces<D, F16>(P, c, first_cta, pieces);
                } else if (warp_on) {
                    const uint32_t o_base = tmem_base + lanes + 2 * PA_TILE;
                    join_few<D, F16>(P, at, first_cta, pieces, cap_row, mt, lt, pair ? 0 : w * (D / 2), pair ? D : (w + 1) * (D / 2),
                                     pair ? tmem_o : o_base, o_base + D, f[0] * scale, f[1] * scale, !pair && m_tiles > 1,
                                     pair && done == 0, tile_rows > 32, lane);
                }
            }
            softmax_barrier();  // sh.last is read before the next item writes it, and the rows are written
            written = joins != 0;
            rest = (joins & 2) != 0;
        }
        // (seen_by_all < ctx: a node of a broken tree, which is no warp's usual row)
        if (__any_sync(0xFFFFFFFFu, rest || (written && seen_by_all < c.s.ctx)))
            add_not_finite<D, F16>(P, c.b, c.h, c.s.q0, c.s.n, c.s.ctx, c.tok0, c.ntok, w);
    }
}

// Rows of sequences that cannot be attended (flagged): zeros, lse -inf.
__device__ __forceinline__ void clear_bad_rows(const PagedAttnParams& P, int D) {
    for (int b = blockIdx.x; b < P.ch.B; b += gridDim.x) {
        const Chunk s = load_chunk(P.ch, b);
        if (s.ok || !s.rows_ok) continue;
        const int pieces = D / 8;
        for (long long x = threadIdx.x; x < (long long)s.n * P.Hq * pieces; x += PA_THREADS) {
            const long long row = x / pieces;
            const int64_t t = s.q0 + row / P.Hq, h = row % P.Hq;
            *reinterpret_cast<uint4*>(P.out + t * P.o_ts + h * P.o_hs + (x % pieces) * 16) = make_uint4(0, 0, 0, 0);
            if (P.lse && x % pieces == 0) P.lse[t * P.Hq + h] = -INFINITY;
        }
    }
}

template <int D, bool F16>
__global__ void __launch_bounds__(PA_THREADS, 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedAttnParams P) {
    using S = PaShape<D>;
    // 1024-byte alignment for the 128-byte swizzle atoms; nothing is static, so
    // that this begins at the CTA's first byte
    extern __shared__ __align__(1024) char smem[];
    char* q_smem = smem;
    char* ring = smem + 2 * S::TILE_BYTES;
    PaShared& sh = *reinterpret_cast<PaShared*>(smem + S::TILES_BYTES);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::STAGES; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(&sh.s_full[w], 1);
            mbar_init(&sh.p_half[w], 4);   // a warp each
            mbar_init(&sh.p_full[w], 4);
            mbar_init(&sh.o_full[w], 1);
            mbar_init(&sh.q_full[w], 1);
            mbar_init(&sh.q_empty[w], 2);  // release_q
        }
        mbar_init(&sh.mma_done, 1);
        mbar_init(&sh.never, 1);
        for (int s = 0; s < 10; ++s) sh.loads[0][s] = sh.loads[1][s] = 0;
        sh.q_loads[0] = sh.q_loads[1] = 0;
        sh.err = sh.not_finite = 0;
        fence_barrier_init();
    }
    if (warp == 8 && lane < 3)
        asm volatile("prefetch.tensormap [%0];"
                     ::"l"(reinterpret_cast<uint64_t>(lane == 0 ? &tm_k : lane == 1 ? &tm_v : &tm_q))
                     : "memory");
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&sh.tmem)), "r"(PA_TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    grid_dependency_wait();
    launch_dependents();

    bool bad = false;
    const bool work = find_share(P, sh, bad);
    if (bad) clear_bad_rows(P, D);
    if (work) {
        if (P.test_wait_timeout && threadIdx.x == 0) {
            // the failure path, tested: a barrier that nothing completes
            if (!mbar_wait(&sh.never, 0, 64)) atomicExch(&sh.err, 1);
        }
        // The CTA's registers, 384 x 168 at launch, move to the softmax threads:
        // 256 x 216 + 128 x 72 is the same sum.
        if (warp < 8) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 216;" ::: "memory");
            softmax_rows<D, F16>(P, sh, warp >> 2, q_smem, ring, tmem);
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 72;" ::: "memory");
            if (warp == 8 || warp == 10) {
                load_kv<D>(P, sh, smem_u32(ring), warp == 10 ? &tm_v : &tm_k, warp == 10, lane);
            } else if (warp == 9) {
                const uint32_t issue = elect_one();
                issue_products<D, F16>(P, sh, smem_u32(q_smem), smem_u32(ring), tmem, issue);
                // every product issued has completed before TMEM is released
                mma_commit(&sh.mma_done, issue);
                (void)pa_wait_until(&sh.mma_done, 0, nullptr);
            } else {
                load_q<D>(P, sh, smem_u32(q_smem), &tm_q, lane);
            }
        }
    }
    __syncthreads();
    // Every load issued has landed before the CTA ends: the products have used
    // them all, unless a wait gave up.
    if (work && sh.err && threadIdx.x < S::STAGES) {
        const int n = max(sh.loads[0][threadIdx.x], sh.loads[1][threadIdx.x]);
        if (n > 0) (void)pa_wait_until(&sh.full[threadIdx.x], (n - 1) & 1, nullptr);
        const int q = threadIdx.x < 2 ? sh.q_loads[threadIdx.x] : 0;
        if (q > 0) (void)pa_wait_until(&sh.q_full[threadIdx.x], (q - 1) & 1, nullptr);
    }
    if (warp == 9) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(PA_TMEM_COLS) : "memory");
    }
    __syncthreads();
    if (threadIdx.x == 0 && sh.err) raise_flag(P.ch.status, SV_FLAG_TIMEOUT);
}

template <int D, bool F16>
static cudaError_t launch(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const PagedAttnParams& p,
                          int grid, cudaStream_t stream) {
    auto kernel = paged_attention_kernel<D, F16>;
    static std::atomic<int> attr_done[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!attr_done[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PA_SMEM<D>);
        if (e != cudaSuccess) return e;
        attr_done[dev].store(1, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(PA_THREADS, 1, 1);
    cfg.dynamicSmemBytes = PA_SMEM<D>;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, tm_q, tm_k, tm_v, p);
}

cudaError_t launch_paged_attention(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                   const PagedAttnParams& p, int D, int f16, int sms, cudaStream_t stream) {
    const int grid = sms < PA_MAX_CTAS ? sms : PA_MAX_CTAS;
    if (D == 128)
        return f16 ? launch<128, true>(tm_q, tm_k, tm_v, p, grid, stream) : launch<128, false>(tm_q, tm_k, tm_v, p, grid, stream);
    return f16 ? launch<64, true>(tm_q, tm_k, tm_v, p, grid, stream) : launch<64, false>(tm_q, tm_k, tm_v, p, grid, stream);
}

}  // namespace sv
