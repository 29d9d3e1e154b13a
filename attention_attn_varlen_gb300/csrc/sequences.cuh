// sequences.cuh -- what the kernels with a cache of states share: a packed
// sequence's rows and its slot of the state cache, checked.
#pragma once

#include "common.cuh"

namespace attn {

// Tokens [t0, t0 + n) of sequence b; n = 0 for bad offsets.
template <uint32_t SRC, class P>
__device__ __forceinline__ void sequence_rows(const P &p, int b, int64_t &t0, int &n, bool report) {
    const int64_t a = __ldg(p.cu + b), e = __ldg(p.cu + b + 1);
    bool ok = a >= 0 && e >= a && e <= p.total_tokens;
    t0 = ok ? a : 0;
    n = ok ? (int)(e - a) : 0;
    if (ok && n > p.max_seqlen) {
        ok = false;
        n = p.max_seqlen;
    }
    if (!ok && report) record_error(p.err, ERR_INDEX | SRC);
}

// State of sequence b, head h of `heads`: its address (null: none kept, or, STEP, the
// step refused the sequence) and whether the sequence starts from it.
template <uint32_t SRC, bool STEP, class P>
__device__ __forceinline__ float *sequence_state(const P &p, int heads, int b, int h, bool &from, bool report) {
    from = false;
    if (!p.state) return nullptr;
    const int64_t slot = __ldg(p.slots + b);
    if (!STEP && slot < 0) return nullptr;
    const int past = p.context_lens ? __ldg(p.context_lens + b) : 0;
    // one branch behind the three loads: they are in flight together
    const bool refused = STEP && p.cache_seqlens && __ldg(p.cache_seqlens + b) <= past;
    if (STEP && (slot < 0 || refused)) return nullptr;
    if (slot >= p.num_slots) {
        if (report) record_error(p.err, ERR_INDEX | SRC);
        return nullptr;
    }
    from = p.context_lens ? past > 0 : !p.start_zero;
    return p.state + (slot * heads + h) * (int64_t)p.D * p.D;
}

}  // namespace attn
