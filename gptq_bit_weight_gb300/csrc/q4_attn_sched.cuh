// How the attention kernels share out their work.
//
// A request's rows (new token x query head of the group, head fastest) are
// cut into row tiles of `step` rows, its context into key tiles of 2^kt_log2
// tokens.  An item is one (request, key/value head, row tile); its units are
// the key tiles its rows can see (one, without work, if they see nothing).
// All units of a call, item after item, are dealt to the CTAs in equal
// contiguous runs, so a CTA holds the end of one item, some whole ones and
// the beginning of another; pieces of a cut item meet in the workspace.
// Every CTA works the shares out for itself from the lengths in device
// memory: no host copy of them, no planning launch.
#pragma once
#include "q4_serve.h"

namespace q4 {

// x / d for 0 <= x < 2^31 with m = 2^32 / d rounded down: the high product is
// the quotient or one less.  (The compiler's division is some 25 instructions,
// and the walk over the items is in every role.)
struct FastDiv {
    uint32_t d, m;
    __host__ __device__ explicit FastDiv(int d_) : d(d_), m(d_ > 1 ? static_cast<uint32_t>((1ull << 32) / d_) : 0xffffffffu) {}
    __device__ __forceinline__ int operator()(int x) const {
        const uint32_t q = __umulhi(static_cast<uint32_t>(x), m);
        return static_cast<int>(q + (static_cast<uint32_t>(x) - q * d >= d));
    }
};

struct SchedParams {
    AttnBatch b;
    int hkv, page_log2, window;
    int kt_log2;      // log2 of the tokens of a key tile
    FastDiv group;    // query heads of a key/value head
    int step_log2;    // log2 of the rows of a row tile, or -1:
    FastDiv tokens;   // tokens of a row tile, where tiles hold whole tokens
};

struct Item {
    int b, head, tile, tiles;
    int q0, ql, kv;
    int t0, t1;      // first and last token of the row tile
    int lo, hi;      // keys [lo, hi) that some row of the tile sees; hi <= 0: none
    int first, n;    // key tiles
    int u;           // the item's first unit
};

__device__ __forceinline__ int row_tiles(const SchedParams &p, int ql) {
    if (p.step_log2 < 0) return p.tokens(ql + static_cast<int>(p.tokens.d) - 1);
    return (ql * static_cast<int>(p.group.d) + (1 << p.step_log2) - 1) >> p.step_log2;
}

// The tokens, keys and key tiles of row tile `it.tile`.
__device__ __forceinline__ void fill_tile(const SchedParams &p, Item &it) {
    if (p.step_log2 < 0) {
        it.t0 = it.tile * static_cast<int>(p.tokens.d);
        it.t1 = min(it.t0 + static_cast<int>(p.tokens.d), it.ql) - 1;
    } else {
        const int r0 = it.tile << p.step_log2, r1 = min(r0 + (1 << p.step_log2), it.ql * static_cast<int>(p.group.d));
        it.t0 = p.group(r0);
        it.t1 = p.group(r1 - 1);
    }
    const int own = it.kv - it.ql;                   // index of new token 0
    it.hi = min(own + it.t1 + 1, it.kv);
    it.lo = p.window > 0 ? max(0, own + it.t0 - p.window + 1) : 0;
    it.first = it.lo >> p.kt_log2;
    const int kt = 1 << p.kt_log2;
    it.n = it.hi > 0 ? ((it.hi + kt - 1) >> p.kt_log2) - it.first : 1;
}

// Units of row tiles i0, i0 + stride, .. of a request with ql tokens and a context of kv.
__device__ __forceinline__ long long tile_units(const SchedParams &p, int ql, int kv, int i0, int stride) {
    Item it;
    it.ql = ql;
    it.kv = kv;
    const int tiles = row_tiles(p, ql);
    long long sum = 0;
#pragma unroll 1
    for (it.tile = i0; it.tile < tiles; it.tile += stride) {
        fill_tile(p, it);
        sum += it.n;
    }
    return sum;
}

__device__ __forceinline__ void load_item_request(const SchedParams &p, Item &it) {
    const Request r = load_request(p.b, it.b, p.page_log2);
    it.q0 = r.q0;
    it.ql = r.ql;
    it.kv = r.kv;
    it.tiles = row_tiles(p, r.ql);
}

// Step to the next item; false after the last.
__device__ __forceinline__ bool next_item(const SchedParams &p, Item &it) {
    it.u += it.n;
    if (++it.tile == it.tiles) {
        it.tile = 0;
        if (++it.head == p.hkv) {
            it.head = 0;
#pragma unroll 1
            do {
                if (++it.b >= p.b.batch) return false;
                load_item_request(p, it);
            } while (it.tiles == 0);
        }
    }
    fill_tile(p, it);
    return true;
}

struct Share {
    int begin, end;          // units of this CTA
    uint32_t per;            // units of every CTA but the last with any
};

// Shared memory of sched_share.
struct SchedSmem {
    long long warp_sum[32];
    int b, head, tile, q0, ql, kv;
    int rem, u;
};

// Units of a lane's request (or of none: ql 0), by a whole warp.
__device__ __forceinline__ long long request_units(const SchedParams &p, const Request &r) {
    // a request of many row tiles is summed by all lanes
    const bool many = row_tiles(p, r.ql) > 4;
    long long units = many ? 0 : tile_units(p, r.ql, r.kv, 0, 1);
    const int lane = threadIdx.x & 31;
    for (unsigned left = __ballot_sync(0xffffffffu, many); left; left &= left - 1) {
        const int who = __ffs(left) - 1;
        long long s = tile_units(p, __shfl_sync(0xffffffffu, r.ql, who), __shfl_sync(0xffffffffu, r.kv, who), lane, 32);
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == who) units = s;
    }
    return units;
}
__device__ __forceinline__ long long prefix_sum(long long v) {       // inclusive, within a warp
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    return v;
}
__device__ __forceinline__ Share share_of(long long total, int cta, int ctas, int *status) {
    if (total >= 1ll << 31) {                        // units are counted in 32 bits: the call is not done
        if (cta == 0 && threadIdx.x == 0) atomicOr(status, kAttnTooLong);
        total = 0;
    }
    Share s;
    s.per = max((static_cast<uint32_t>(total) + ctas - 1) / ctas, 1u);
    s.begin = static_cast<int>(min(static_cast<long long>(cta) * s.per, total));
    s.end = static_cast<int>(min(s.begin + static_cast<long long>(s.per), total));
    return s;
}
// The row tile of it's request and head that holds unit `rem` of theirs, by a
// whole warp; `at` is that unit's number.  Sets it.tile and it.u.
__device__ __forceinline__ void find_tile(const SchedParams &p, Item &it, int rem, int at) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int base = 0;; base += 32) {
        it.tile = base + lane;
        it.n = 0;
        if (it.tile < it.tiles) fill_tile(p, it);
        int pre = it.n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, pre, o);
            if (lane >= o) pre += v;
        }
        const unsigned past = __ballot_sync(0xffffffffu, pre > rem);
        if (past) {
            const int who = __ffs(past) - 1;
            it.tile = base + who;
            it.u = at - (rem - __shfl_sync(0xffffffffu, pre - it.n, who));
            return;
        }
        if (base + 32 >= it.tiles) {                 // cannot be: the sums said otherwise
            it.tile = it.tiles - 1;
            it.u = at;
            return;
        }
        rem -= __shfl_sync(0xffffffffu, pre, 31);
    }
}

// This CTA's share and, if it has one, its first item.  Called by all NT
// threads of the CTA, which it synchronizes; `sm` must not be in use before or
// within the call.  A call of up to 32 requests is short, and this is at its
// head: every warp works its share out for itself.
template <int NT>
__device__ Share sched_share(const SchedParams &p, SchedSmem &sm, int cta, int ctas, int *status, Item &it) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (p.b.batch <= 32) {
        Request r{0, 0, 0, false};
        if (lane < p.b.batch) r = load_request(p.b, lane, p.page_log2);
        if (r.bad && cta == 0 && warp == 0) atomicOr(status, kAttnBadBatch);
        const long long units = request_units(p, r), mine = units * p.hkv, upto = prefix_sum(mine);
        const Share s = share_of(__shfl_sync(0xffffffffu, upto, 31), cta, ctas, status);
        if (s.begin < s.end) {
            const int who = __ffs(__ballot_sync(0xffffffffu, s.begin < upto)) - 1;
            const uint32_t each = static_cast<uint32_t>(__shfl_sync(0xffffffffu, units, who));
            const uint32_t rem = static_cast<uint32_t>(s.begin - __shfl_sync(0xffffffffu, upto - mine, who));
            it.b = who;
            it.head = static_cast<int>(rem / each);
            it.q0 = __shfl_sync(0xffffffffu, r.q0, who);
            it.ql = __shfl_sync(0xffffffffu, r.ql, who);
            it.kv = __shfl_sync(0xffffffffu, r.kv, who);
            it.tiles = row_tiles(p, it.ql);
            find_tile(p, it, static_cast<int>(rem - it.head * each), s.begin);
            fill_tile(p, it);
        }
        __syncthreads();
        return s;
    }
    const int chunk = (p.b.batch + NT - 1) / NT;     // requests of a thread, in order
    long long mine = 0, last = 0;
    Request r{0, 0, 0, false};
#pragma unroll 1
    for (int i = 0; i < chunk; ++i) {
        const int b = tid * chunk + i;
        r = Request{0, 0, 0, false};
        if (b < p.b.batch) {
            r = load_request(p.b, b, p.page_log2);
            if (r.bad && cta == 0) atomicOr(status, kAttnBadBatch);
        }
        last = request_units(p, r);
        mine += last * p.hkv;
    }
    const long long upto = prefix_sum(mine);
    if (lane == 31) sm.warp_sum[warp] = upto;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll 1
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += sm.warp_sum[w];
        total += sm.warp_sum[w];
    }
    const Share s = share_of(total, cta, ctas, status);
    before += upto - mine;
    if (s.begin < s.end && before <= s.begin && s.begin < before + mine) {
        // this thread's requests hold the first unit: find which
        uint32_t rem = static_cast<uint32_t>(s.begin - before);
        uint32_t units = static_cast<uint32_t>(last);
        int b = tid * chunk;
#pragma unroll 1
        for (;; ++b) {
            if (chunk > 1) {
                r = load_request(p.b, b, p.page_log2);
                units = static_cast<uint32_t>(tile_units(p, r.ql, r.kv, 0, 1));
            }
            if (rem < units * p.hkv) break;
            rem -= units * p.hkv;
        }
        const int head = static_cast<int>(rem / units);
        sm.b = b;
        sm.head = head;
        sm.rem = static_cast<int>(rem - head * units);
        sm.q0 = r.q0;
        sm.ql = r.ql;
        sm.kv = r.kv;
    }
    __syncthreads();
    if (s.begin >= s.end) return s;
    it.b = sm.b;
    it.head = sm.head;
    it.q0 = sm.q0;
    it.ql = sm.ql;
    it.kv = sm.kv;
    it.tiles = row_tiles(p, it.ql);
    if (warp == 0) {
        find_tile(p, it, sm.rem, s.begin);
        if (lane == 0) {
            sm.tile = it.tile;
            sm.u = it.u;
        }
    }
    __syncthreads();
    it.tile = sm.tile;
    it.u = sm.u;
    fill_tile(p, it);
    return s;
}

}  // namespace q4
