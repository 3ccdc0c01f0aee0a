// Loading the paged cache's key and value tiles by TMA, shared by the
// attention kernels.
#pragma once
#include "q4_attn_sched.cuh"
#include "q4_tc.cuh"

namespace q4 {

constexpr int kKtLog2 = 7, kKt = 1 << kKtLog2;   // tokens of a key tile

// One lane of a converged warp.  The compiler knows a region behind it to be
// one thread's, so the operands of tcgen05.mma and of TMA copies go to uniform
// registers directly.  Behind a test of the lane number, or issued by many
// lanes at once, each took 90 to 110 cycles to issue: more than the 64 that an
// MMA runs, and 3500 for a tile of 16-token pages.
__device__ __forceinline__ bool elect_one() {
    uint32_t p = 0;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
        "[%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}
// tc::mbar_wait (the same bound, about two seconds) with its polling loop kept
// a loop: unrolled 64 times at each of a dozen places it made two thirds of
// these kernels' code, more than the instruction caches hold.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = tc::globaltimer();
#pragma unroll 1
    for (uint32_t i = 1;; ++i) {
        if (tc::mbar_try_wait(bar, parity)) return true;
        if (i % 64 == 0 && tc::globaltimer() - t0 > 2000000000ull) return false;
    }
}
// A bounded wait by a whole warp; once one has run out, no more waiting: the
// roles go through their loops, on whatever is there, and the CTA ends.
__device__ __forceinline__ bool wait_all(bool alive, uint32_t bar, uint32_t parity) {
    if (alive) alive = wait_bounded(bar, parity);
    return __all_sync(0xffffffffu, alive);
}

// Counts a piece in the workspace, by one thread behind a barrier: what the CTA wrote before is there for whoever
// counts later.
__device__ __forceinline__ int count_piece(int *ticket) {
    int before;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(ticket) : "memory");
    return before;
}
// Pieces counted so far; what they hold may be read.
__device__ __forceinline__ int pieces_counted(const int *ticket) {
    int n;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(n) : "l"(ticket) : "memory");
    return n;
}

// The pages of one key tile, as a loader warp holds them: lane i has page i.
struct TilePages {
    int page;                // this lane's
    unsigned wanted;         // pages with a visible key, one bit each
    int row;                 // first token within the page
};
struct PageWalk {
    const int32_t *table;
    int page_log2, box_log2, pages;      // tokens of a page and of a box (at most a tile's), pages of the cache

    __device__ PageWalk(const SchedParams &p, const Item &it, int cache_pages)
        : table(p.b.table + it.b * p.b.table_stride),
          page_log2(p.page_log2),
          box_log2(min(p.page_log2, kKtLog2)),
          pages(cache_pages) {}
    // Tile j (counted from it.first); a page index outside the cache becomes page 0 and sets `bad`.
    __device__ __forceinline__ TilePages tile(const Item &it, int j, int &bad) const {
        const int lane = threadIdx.x & 31, key_t = (it.first + j) << kKtLog2, key = key_t + (lane << box_log2);
        const bool mine = lane < (kKt >> box_log2) && key < it.hi && key + (1 << box_log2) > it.lo;
        TilePages t;
        t.page = mine ? table[key >> page_log2] : 0;
        if (t.page < 0 || t.page >= pages) {
            bad = kAttnBadPage;
            t.page = 0;
        }
        t.wanted = __ballot_sync(0xffffffffu, mine);
        t.row = key_t & ((1 << page_log2) - 1) & ~((1 << box_log2) - 1);
        return t;
    }
    // Copies a tile's pages of keys or values to dst [D / 64][128 tokens][64], swizzled; by a whole warp.
    template <int D>
    __device__ __forceinline__ void copy(const TilePages &t, uint32_t dst, const CUtensorMap *map, uint32_t bar,
                                         int head) const {
        if (elect_one()) tc::mbar_arrive_expect_tx(bar, __popc(t.wanted) * (D * 2) << box_log2);
        __syncwarp();
#pragma unroll 1
        for (int i0 = 0; i0 < (kKt >> box_log2); i0 += 4) {      // a tile has 1 to 16 pages
            int page[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) page[i] = __shfl_sync(0xffffffffu, t.page, i0 + i);
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (t.wanted >> (i0 + i) & 1)
#pragma unroll
                        for (int h = 0; h < D / 64; ++h)
                            tma_load_4d(dst + h * (kKt * 128) + ((i0 + i) << box_log2) * 128, map, bar, 64 * h, t.row, head,
                                        page[i]);
            }
            __syncwarp();
        }
    }
};

}  // namespace q4
