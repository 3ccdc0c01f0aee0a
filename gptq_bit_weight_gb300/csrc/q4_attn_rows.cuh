// Where the tokens of a step lie in the paged cache, shared by the kernels
// that write and read them token by token.
#pragma once
#include "q4_serve.h"

namespace q4 {

constexpr int kMaxTokens = 8;        // of one CTA: one warp looks each of them up

struct Token {
    int64_t page;     // in the cache; -1: no request's token, or out of range
    int slot, pos;    // within the page; rotary position
};

// Token t of the step, by a whole warp; the result is lane 0's.  max_pos > 0:
// its position (positions[t], or its index where that is NULL) has to be below.
__device__ __forceinline__ Token find_token(const AttnBatch &b, const AttnShape &s, int pages, int t,
                                            const int32_t *positions, int max_pos, int *status) {
    const int lane = threadIdx.x & 31;
    int before = 0;                                      // requests that end at or before t
    for (int i = lane; i < b.batch; i += 32) before += b.cu_q[i + 1] <= t;
    const int req = __reduce_add_sync(0xffffffffu, before);
    Token k{-1, 0, 0};
    if (lane == 0 && req < b.batch && b.cu_q[req] <= t) {
        const Request r = load_request(b, req, s.page_log2);
        const int idx = r.kv - r.ql + (t - r.q0);
        int bad = 0;
        // A length that had to be cut says nothing of where the token belongs: its index in the cut context
        // is another token's, and a table's padding may be another request's page.
        if (r.bad || idx < 0 || idx >= r.kv) {
            bad = kAttnBadBatch;
        } else {
            const int page = b.table[req * b.table_stride + (idx >> s.page_log2)];
            k.slot = idx & (s.page - 1);
            k.pos = positions ? positions[t] : idx;
            if (page < 0 || page >= pages) bad |= kAttnBadPage;
            else if (max_pos > 0 && (k.pos < 0 || k.pos >= max_pos)) bad |= kAttnBadPosition;
            else k.page = page;
        }
        if (bad) atomicOr(status, bad);
    }
    return k;
}

}  // namespace q4
