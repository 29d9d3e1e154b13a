// beam.cu -- beam search: the choice among beams and vocabulary, the request rows of the
// chosen beams, and the copies of states and cached rows that follow them.
#include "common.cuh"
#include "kernels.h"

namespace attn {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.4028234663852886e38f;   // the lowest fp32 value, where a running maximum starts

// ---------------------------------------------------------------------------
// Selection.  A candidate is (beam b, token t) with the score
//   scores[b] + logits[b][t] - log(sum_j e^{logits[b][j]}),
// the order: higher score; equal ones by beam; within a beam higher logit, equal ones
// by token.  Exponentials, their sums and the sums' mantissas' logarithms are in fp32 (a few 2^-22 of a row's
// normaliser), which sets how close candidates of different beams can be told apart; the scores are put together and
// compared in 64 bits, so that nothing is lost to a beam's score or to a large maximum besides, and the order within a
// beam is the logits' own.
//
// One pass over the logits: 64 groups of 8 beams, 131,072 bf16 logits each (134 MB), take 43 us (41 in a graph), 35 of
// them the scan (HBM alone: 20), which its instructions bound: 91 for eight logits of 32 lanes (34 without the
// candidates), the conversions, exponentials and
// comparisons (issue slots 60 % busy beside the merges' waits).  All but one logit in 1,000 masked, by -1e9, -1e10 or the
// type's lowest value alike: 51 us.  One group of 4 beams, 32,000 logits: 10.5 us in a graph, the
// two launches' latency.  A CTA takes a slice of a row, a warp a
// share of the slice in vectors of eight neighbours a lane; the warp keeps a sum of
// exponentials below a reference that moves when a logit lies far above it, and its
// k best logits as a sorted list, one a lane.  A key is the logit's bits in an order that compares as unsigned above
// the token's complement: distinct, and a larger one comes first.  What exceeds
// the list's last key goes to a buffer in shared memory, which is merged into the list 32 at a time.
// A second small launch joins the slices and the beams of a group.
// Every row is cut and summed in the same way: equal rows give equal sums.
// ---------------------------------------------------------------------------
constexpr int kScanWarps = 4;
template <typename T> constexpr int kScanAhead = 8 / sizeof(T);   // vectors of a warp in a step (64 bytes a lane)
constexpr float kFarAbove = 40.f;                    // a logit this far above the sum's reference moves it
// Largest reference for which 2^(x log2(e) - rn(ref log2(e))) is summed and what the rounding left, at most half a step
// of ref log2(e), is made good afterwards: 64 up to 2^31 (1.49e9), so that 2^-64 .. 2^64 times a sum stay finite and
// normal; from there on one factor may be 0 and the other infinite.  Masks of -1e9 are still below it.
constexpr float kFarOff = 1e9f;

__device__ __forceinline__ uint64_t key_of(float x, uint32_t token) {
    const uint32_t b = __float_as_uint(x + 0.f);     // -0 is 0
    return (uint64_t)(b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u)) << 32 | ~token;
}
__device__ __forceinline__ float key_logit(uint64_t key) {
    const uint32_t o = (uint32_t)(key >> 32);
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint32_t key_token(uint64_t key) { return ~(uint32_t)key; }
// no key: below every key of a logit above -inf
__device__ __forceinline__ uint64_t key_floor() { return key_of(-INFINITY, 0u) | 0xFFFFFFFFull; }

__device__ __forceinline__ uint64_t shfl64(uint64_t x, int from) { return __shfl_sync(0xffffffffu, x, from); }
__device__ __forceinline__ uint64_t shfl_up64(uint64_t x, int by) { return __shfl_up_sync(0xffffffffu, x, by); }

// one compare-exchange of a descending network over the lanes
__device__ __forceinline__ uint64_t exchange(uint64_t x, int lane, int stride, bool descending) {
    const uint64_t y = __shfl_xor_sync(0xffffffffu, x, stride);
    const bool keep_max = ((lane & stride) == 0) == descending;
    return (x > y) == keep_max ? x : y;
}

// 32 keys, one a lane -> descending
__device__ __forceinline__ uint64_t sort32(uint64_t x, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size *= 2) {
#pragma unroll
        for (int stride = size / 2; stride > 0; stride /= 2) x = exchange(x, lane, stride, (lane & size) == 0);
    }
    return x;
}

// the 32 largest of two descending lists, descending
__device__ __forceinline__ uint64_t merge32(uint64_t a, uint64_t b, int lane) {
    const uint64_t r = shfl64(b, 31 - lane);
    uint64_t x = a > r ? a : r;
#pragma unroll
    for (int stride = 16; stride > 0; stride /= 2) x = exchange(x, lane, stride, true);
    return x;
}

// Eight neighbouring logits of a row, as loaded: elements i .. i + 7, -inf behind the end.  MODE 0: the rows lie
// on 16-byte boundaries and come by way of shared memory, but for the row's end; 1: they need not, and 16 bytes come
// out of the two aligned pieces that hold them
template <typename T, int MODE> struct Eight {
    static constexpr int kWords = sizeof(T) * 2;     // 32-bit words
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const T *row, int i, int end) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + i), lo = at & ~(uintptr_t)15;
        constexpr int kPieces = kWords / 4 + 1;
        if (MODE == 1 && lo >= reinterpret_cast<uintptr_t>(row) &&
            lo + kPieces * 16 <= reinterpret_cast<uintptr_t>(row + end)) {
            // all of what is read is the row's own
            uint32_t x[kPieces * 4 + 1];
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
                const uint4 y = __ldg(reinterpret_cast<const uint4 *>(lo) + k);
                x[4 * k] = y.x, x[4 * k + 1] = y.y, x[4 * k + 2] = y.z, x[4 * k + 3] = y.w;
            }
            x[kPieces * 4] = 0;
            const uint32_t off = (uint32_t)(at - lo);
#pragma unroll
            for (int k = 0; k < kWords + 2; ++k) x[k] = off & 8 ? x[k + 2] : x[k];
#pragma unroll
            for (int k = 0; k < kWords + 1; ++k) x[k] = off & 4 ? x[k + 1] : x[k];
#pragma unroll
            for (int k = 0; k < kWords; ++k) w[k] = sizeof(T) == 2 ? __funnelshift_r(x[k], x[k + 1], (off & 2) * 8) : x[k];
            return;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint32_t b = sizeof(T) == 2 ? 0xFF80u : 0xFF800000u;
            if (i + j < end)
                b = sizeof(T) == 2 ? reinterpret_cast<const uint16_t *>(row)[i + j] : reinterpret_cast<const uint32_t *>(row)[i + j];
            if (sizeof(T) == 2) w[j / 2] = j & 1 ? w[j / 2] | b << 16 : b;
            else w[j] = b;
        }
    }
    // what copy() put into shared memory
    __device__ __forceinline__ void take(const uint4 *from) {
#pragma unroll
        for (int k = 0; k < kWords; k += 4) {
            const uint4 x = from[k / 4 * kScanWarps * 32];
            w[k] = x.x, w[k + 1] = x.y, w[k + 2] = x.z, w[k + 3] = x.w;
        }
    }
    static __device__ __forceinline__ void copy(uint4 *to, const T *from) {
#pragma unroll
        for (int k = 0; k < kWords / 4; ++k)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to + k * kScanWarps * 32)),
                         "l"(reinterpret_cast<const uint4 *>(from) + k)
                         : "memory");
    }
    __device__ __forceinline__ float get(int j) const {
        if (sizeof(T) == 2) return __uint_as_float(j & 1 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
        return __uint_as_float(w[j]);
    }
    __device__ __forceinline__ float top() const {
        if (sizeof(T) == 2) {
            // pairs as they are
            uint32_t m;
            asm("{.reg .b32 a, b;\n\tmax.bf16x2 a, %1, %2;\n\tmax.bf16x2 b, %3, %4;\n\tmax.bf16x2 %0, a, b;}"
                : "=r"(m)
                : "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]));
            return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
        }
        return max3f(max3f(get(0), get(1), get(2)), max3f(get(3), get(4), get(5)), fmaxf(get(6), get(7)));
    }
};

template <typename T, int MODE>
__global__ void __launch_bounds__(kScanWarps * 32, 8) beam_scan_kernel(const BeamParams p) {
    __shared__ uint64_t buf[kScanWarps][32];
    __shared__ float2 part[kScanWarps];
    // MODE 0: the next step's vectors arrive while a step's are gone through; a lane reads what it copied itself
    constexpr int kAhead = kScanAhead<T>, kStep = kAhead * kScanWarps * 256;
    __shared__ uint4 ring[MODE == 0 ? 2 * 4 * kScanWarps * 32 : 1];
    asm volatile("griddepcontrol.launch_dependents;");
    auto pick = [](const Eight<T, MODE> (&x)[kAhead], int v) {           // x[v], registers by choice
        Eight<T, MODE> y = x[0];
#pragma unroll
        for (int u = 1; u < kAhead; ++u) {
#pragma unroll
            for (int k = 0; k < y.kWords; ++k) y.w[k] = v == u ? x[u].w[k] : y.w[k];
        }
        return y;
    };
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x / p.slices, slice = blockIdx.x - row * p.slices;
    const T *x0 = reinterpret_cast<const T *>(p.logits) + (int64_t)row * p.row_stride;
    const int begin = slice * p.slice_len, end = min(p.V, begin + p.slice_len);
    uint64_t *mine = buf[warp];
    uint64_t list = key_floor(), last = list;            // last: the k-th key so far, or a bound below it
    float bound = -INFINITY;                             // its logit
    float ref = kLowest, sum = 0.f;                      // sum of e^(x - ref); (finite: -inf - -inf would be NaN)
    // the warps' sorted lists into buf[0]
    auto best_of_warps = [&](uint64_t own) {
        mine[lane] = own;
        __syncthreads();
#pragma unroll 1
        for (int half = kScanWarps / 2; half > 0; half /= 2) {
            if (warp < half) {
                own = merge32(own, buf[warp + half][lane], lane);
                mine[lane] = own;
            }
            __syncthreads();
        }
    };
    // (steps that end before the slice does need no look at each vector)
    auto slot = [&](int v, int it) { return ring + ((it & 1) * 4 + v * 4 / kAhead) * kScanWarps * 32 + threadIdx.x; };
    auto fetch = [&](int base, int it) {
        if (MODE != 0) return;
        const T *from = x0 + base + warp * 256 + lane * 8;
        if (base + kStep <= end) {
#pragma unroll
            for (int v = 0; v < kAhead; ++v) Eight<T, MODE>::copy(slot(v, it), from + v * kScanWarps * 256);
        } else {
#pragma unroll
            for (int v = 0; v < kAhead; ++v)
                if (base + (v * kScanWarps + warp) * 256 + lane * 8 + 8 <= end)
                    Eight<T, MODE>::copy(slot(v, it), from + v * kScanWarps * 256);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(begin, 0);
#pragma unroll 1
    for (int base = begin, it = 0; base < end; base += kStep, ++it) {
        fetch(base + kStep, it + 1);
        if (it > 1 && (it & (it - 1)) == 0) {
            // the CTA's k-th key so far is a bound for every warp, the tighter the further the scan has come
            best_of_warps(list);
            const uint64_t t = buf[0][p.k - 1];
            if (t > last) last = t, bound = key_logit(t);
            __syncthreads();
        }
        const int at = base + warp * 256 + lane * 8;
        Eight<T, MODE> x[kAhead];
        if (MODE == 0) asm volatile("cp.async.wait_group 1;" ::: "memory");
        if (MODE == 0 && base + kStep <= end) {
#pragma unroll
            for (int v = 0; v < kAhead; ++v) x[v].take(slot(v, it));
        } else {
#pragma unroll
            for (int v = 0; v < kAhead; ++v) {
                const int i = at + v * kScanWarps * 256;
                if (MODE == 0 && i + 8 <= end) x[v].take(slot(v, it));
                else x[v].load(x0, i, end);
            }
        }
        float high[kAhead], top = -INFINITY;
#pragma unroll
        for (int v = 0; v < kAhead; ++v) {
            high[v] = x[v].top();
            top = fmaxf(top, high[v]);
        }
        if (__any_sync(0xffffffffu, top > ref + kFarAbove)) {
            float m = top;
#pragma unroll
            for (int w = 16; w > 0; w /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
            m = fmaxf(m, ref);
            sum *= ex2((ref - m) * kLog2e);
            ref = m;
        }
        float s0 = 0.f, s1 = 0.f;
        if (fabsf(ref) <= kFarOff) {
            // 2^(x log2(e) - ref log2(e)), and what the second product's rounding leaves, once for all
            const float r = -__fmul_rn(ref, kLog2e);
#pragma unroll
            for (int v = 0; v < kAhead; ++v) {
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    float a, b;
                    fma2(a, b, x[v].get(j), x[v].get(j + 1), kLog2e, kLog2e, r, r);
                    add2(s0, s1, ex2(a), ex2(b));
                }
            }
            sum = fmaf(s0 + s1, ex2(-fmaf(ref, kLog2e, r)), sum);
        } else {
            // the difference itself is exact where it counts: as near to ref as 40, both are beyond 2^29
#pragma unroll 1
            for (int v = 0; v < kAhead; ++v) {
                const Eight<T, MODE> y = pick(x, v);
#pragma unroll
                for (int j = 0; j < 8; ++j) s0 += ex2((y.get(j) - ref) * kLog2e);
            }
            sum += s0;
        }
        if (base == begin) {
            // k lanes have a logit at or above the k-th largest of the lanes' maxima, here of all of the CTA's lanes: of
            // what comes after one in 500 exceeds it (k = 16)
            best_of_warps(sort32(key_of(top, 0u), lane));
            const uint64_t t = buf[0][p.k - 1];
            const uint64_t least = (t & 0xFFFFFFFF00000000ull) - 1;
            if (least > last) last = least, bound = key_logit(t);
            __syncthreads();
        }
        if (!__any_sync(0xffffffffu, top >= bound)) continue;
        // (rolled: four copies of this would not fit the instruction cache beside the rest)
#pragma unroll 1
        for (int v = 0; v < kAhead; ++v) {
            float hv = high[0];
#pragma unroll
            for (int u = 1; u < kAhead; ++u) hv = v == u ? high[u] : hv;
            if (!__any_sync(0xffffffffu, hv >= bound)) continue;
            const Eight<T, MODE> y = pick(x, v);
            const uint32_t token = (uint32_t)(at + v * kScanWarps * 256);
            uint32_t hit = __ballot_sync(0xffffffffu, key_of(hv, token) > last);
#pragma unroll 1
            for (; hit; hit &= hit - 1) {
                // this lane's eight, one to each of the first eight lanes
                const int src = __ffs(hit) - 1;
                Eight<T, MODE> z;
#pragma unroll
                for (int k = 0; k < y.kWords; ++k) z.w[k] = __shfl_sync(0xffffffffu, y.w[k], src);
                float xj = -INFINITY;
#pragma unroll
                for (int j = 0; j < 8; ++j) xj = lane == j ? z.get(j) : xj;
                const uint64_t key = key_of(xj, __shfl_sync(0xffffffffu, token, src) + lane);
                const bool in = lane < 8 && xj >= bound && key > last;           // (a NaN is not)
#pragma unroll 1
                for (uint32_t who = __ballot_sync(0xffffffffu, in); who; who &= who - 1) {
                    const uint64_t one = shfl64(key, __ffs(who) - 1), above = shfl_up64(list, 1);
                    const int place = __popc(__ballot_sync(0xffffffffu, list > one));
                    list = lane < place ? list : lane == place ? one : above;
                }
                const uint64_t kth = shfl64(list, p.k - 1);
                if (kth > last) last = kth, bound = key_logit(kth);
            }
        }
    }
    // the warps' lists and sums
#pragma unroll
    for (int w = 16; w > 0; w /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    if (lane == 0) part[warp] = make_float2(ref, sum);
    best_of_warps(list);
    if (warp == 0) {
        float2 all = part[0];
        for (int w = 1; w < kScanWarps; ++w) {
            const float2 b = part[w];
            const float m = fmaxf(all.x, b.x);
            all = make_float2(m, all.y * ex2((all.x - m) * kLog2e) + b.y * ex2((b.x - m) * kLog2e));
        }
        if (lane < p.k) p.keys[(int64_t)blockIdx.x * p.k + lane] = mine[lane];
        if (lane == 0) p.sums[blockIdx.x] = all;
    }
}

// A candidate in the order of the result: its score's bits in an order that compares as unsigned, then
// ~(beam, place in the beam's list).
struct Ranked {
    uint64_t score;
    uint32_t id;
};
__device__ __forceinline__ bool before(const Ranked &a, const Ranked &b) {
    return a.score > b.score || (a.score == b.score && a.id > b.id);
}
__device__ __forceinline__ uint64_t ordered(double x) {
    const uint64_t b = (uint64_t)__double_as_longlong(x + 0.0);
    return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double unordered(uint64_t o) {
    return __longlong_as_double((long long)(o >> 63 ? o ^ 0x8000000000000000ull : ~o));
}
__device__ __forceinline__ Ranked merge_ranked(Ranked a, Ranked b, int lane) {
    const Ranked r = {shfl64(b.score, 31 - lane), __shfl_sync(0xffffffffu, b.id, 31 - lane)};
    Ranked x = before(a, r) ? a : r;
#pragma unroll
    for (int stride = 16; stride > 0; stride /= 2) {
        const Ranked y = {__shfl_xor_sync(0xffffffffu, x.score, stride), __shfl_xor_sync(0xffffffffu, x.id, stride)};
        x = before(x, y) == ((lane & stride) == 0) ? x : y;
    }
    return x;
}

// A CTA per group, `per` warps (a power of two) for each beam: they share its slices.
__global__ void __launch_bounds__(1024) beam_join_kernel(const BeamParams p, int per) {
    __shared__ uint64_t slots[32][32];
    __shared__ Ranked lists[kBeamMax][32];
    __shared__ uint32_t token_of[kBeamMax][32];
    __shared__ double norm[kBeamMax];                 // log of the row's sum; NaN: the row has no candidates
    __shared__ float2 total[kBeamMax];
    __shared__ float score_of[kBeamMax];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = warp / per, part = warp - b * per, g = blockIdx.x;
    const int row = g * p.W + b;
    const float score_so_far = __ldg(p.scores + row);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    uint64_t list = key_floor();
    const uint64_t *keys = p.keys + (int64_t)row * p.slices * p.k;
    constexpr int kAhead = 4;                         // slices in flight
    for (int s0 = part; s0 < p.slices; s0 += kAhead * per) {
        uint64_t k[kAhead];
#pragma unroll
        for (int x = 0; x < kAhead; ++x)
            k[x] = s0 + x * per < p.slices && lane < p.k ? keys[(s0 + x * per) * p.k + lane] : key_floor();
#pragma unroll
        for (int x = 0; x < kAhead; ++x)
            if (s0 + x * per < p.slices) list = merge32(list, k[x], lane);
    }
    float top = kLowest, sum = 0.f;
    if (part == 0) {
        for (int s = lane; s < p.slices; s += 32) {
            const float2 x = p.sums[(int64_t)row * p.slices + s];
            const float m = fmaxf(top, x.x);
            sum = sum * ex2((top - m) * kLog2e) + x.y * ex2((x.x - m) * kLog2e);
            top = m;
        }
#pragma unroll
        for (int w = 16; w > 0; w /= 2) {
            const float t = __shfl_xor_sync(0xffffffffu, top, w), s = __shfl_xor_sync(0xffffffffu, sum, w);
            const float m = fmaxf(top, t);
            sum = sum * ex2((top - m) * kLog2e) + s * ex2((t - m) * kLog2e);
            top = m;
        }
    }
    for (int half = per / 2; half > 0; half /= 2) {
        if (part >= half && part < 2 * half) slots[warp][lane] = list;
        __syncthreads();
        if (part < half) list = merge32(list, slots[warp + half][lane], lane);
    }
    if (part == 0 && lane == 0) {
        total[b] = make_float2(top, sum);
        score_of[b] = score_so_far;
    }
    __syncthreads();
    if (warp == 0 && lane < p.W) {
        const float2 x = total[lane];
        const float score = score_of[lane];
        const bool some = x.y > 0.f && x.y < INFINITY;
        // a row of -inf alone and a score of -inf are masks, NaN and +inf mistakes
        if ((!some && !(x.y == 0.f)) || !(score < INFINITY)) record_error(p.err, ERR_RANGE | SRC_BEAM);
        // (the logarithm of the part in [0.7, 1.4) in fp32, off by 2^-25 and less; 64-bit units are few)
        int e;
        float m = frexpf(x.y, &e);
        if (m < 0.70710678f) m *= 2.f, --e;
        norm[lane] = some && score > -INFINITY && score < INFINITY
                         ? (double)x.x + ((double)e * 0.69314718055994530942 + (double)logf(m))
                         : __longlong_as_double(0x7FF8000000000000ll);
    }
    __syncthreads();
    const double score = (double)score_so_far + ((double)key_logit(list) - norm[b]);
    const bool real = list > key_floor() && norm[b] == norm[b];
    Ranked r = {real ? ordered(score) : 0ull, ~(uint32_t)(b * 32 + lane)};
    if (part == 0) {
        lists[b][lane] = r;
        token_of[b][lane] = key_token(list);
    }
    __syncthreads();
    for (int n = p.W; n > 1; n = (n + 1) / 2) {
        const int half = (n + 1) / 2;
        if (part == 0 && b + half < n) {
            r = merge_ranked(r, lists[b + half][lane], lane);
            lists[b][lane] = r;
        }
        __syncthreads();
    }
    if (warp == 0 && lane < p.k) {
        const uint32_t id = ~r.id;
        const bool some = r.score != 0;
        p.tokens[(int64_t)g * p.k + lane] = some ? (int32_t)token_of[id >> 5][id & 31] : -1;
        p.parents[(int64_t)g * p.k + lane] = some ? (int32_t)(id >> 5) : -1;
        p.out_scores[(int64_t)g * p.k + lane] = some ? (float)unordered(r.score) : -INFINITY;
    }
}

// ---------------------------------------------------------------------------
// A warp per group, a lane per beam: the lowest beam that goes on from a parent takes the
// parent's request row; the others take, in order, the rows of beams that nobody goes on
// from (as many: W beams, one row each), and name the parent's row as their source.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(128) beam_rows_kernel(const int32_t *parents, const int32_t *rows, int32_t *rows_out,
                                                        int32_t *source, int groups, int W, uint32_t *err) {
    const int g = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (g >= groups) return;
    const int64_t at = (int64_t)g * W + lane;
    int parent = -1, row = 0;
    if (lane < W) {
        parent = parents[at];
        row = rows[at];
        if (parent >= W) {
            record_error(err, ERR_INDEX | SRC_BEAM);
            parent = -1;
        }
    }
    const bool has = parent >= 0;
    const uint32_t same = __match_any_sync(0xffffffffu, has ? parent : -1);
    const bool first = has && (__ffs(same) - 1) == lane;
    const uint32_t alive = __reduce_or_sync(0xffffffffu, has ? 1u << parent : 0u);
    const uint32_t in = W == 32 ? 0xffffffffu : (1u << W) - 1u;
    const uint32_t others = __ballot_sync(0xffffffffu, lane < W && !first);
    // the n-th row that nobody goes on from, for the n-th of the others
    uint32_t spare = ~alive & in;
    for (int n = __popc(others & ((1u << lane) - 1u)); n > 0; --n) spare &= spare - 1u;
    const int from = first ? parent : spare ? __ffs(spare) - 1 : 0;
    const int mine = __shfl_sync(0xffffffffu, row, from);
    const int theirs = __shfl_sync(0xffffffffu, row, has ? parent : 0);
    if (lane < W) {
        rows_out[at] = mine;
        source[at] = first || !has ? -1 : theirs;
    }
}

// ---------------------------------------------------------------------------
// Copies.  No pair's source is another's destination, so pairs are independent: one
// pass, 2 bytes moved per byte copied (HBM): 64 states of 2 MB in 51 us, 5.2 TB/s.
// ---------------------------------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kCopyAhead = 8;

__global__ void __launch_bounds__(kCopyThreads) copy_states_kernel(uint4 *cache, const int32_t *src, const int32_t *dst,
                                                                   int64_t num_slots, int64_t slot_vecs, int parts,
                                                                   uint32_t *err) {
    const int i = blockIdx.x / parts, part = blockIdx.x - i * parts;
    const int64_t from = __ldg(src + i), to = __ldg(dst + i);
    if (from < 0 || from == to) return;
    if (from >= num_slots || to < 0 || to >= num_slots) {
        if (part == 0 && threadIdx.x == 0) record_error(err, ERR_INDEX | SRC_BEAM);
        return;
    }
    const uint4 *a = cache + from * slot_vecs;
    uint4 *b = cache + to * slot_vecs;
    const int64_t step = (int64_t)parts * kCopyThreads * kCopyAhead;
    for (int64_t x = (int64_t)part * kCopyThreads * kCopyAhead + threadIdx.x; x < slot_vecs; x += step) {
        uint4 v[kCopyAhead];
#pragma unroll
        for (int k = 0; k < kCopyAhead; ++k)
            if (x + k * kCopyThreads < slot_vecs) v[k] = __ldcs(a + x + k * kCopyThreads);
#pragma unroll
        for (int k = 0; k < kCopyAhead; ++k)
            if (x + k * kCopyThreads < slot_vecs) __stcs(b + x + k * kCopyThreads, v[k]);
    }
}

// Tokens [first, length) of request row src to request row dst, through both rows' pages.
// V: what a thread moves at a time.
template <typename V>
__global__ void __launch_bounds__(kCopyThreads) copy_kvcache_kernel(const CopyRowsParams p, int parts) {
    const int i = blockIdx.x / parts, part = blockIdx.x - i * parts;
    const int from = __ldg(p.src + i), to = __ldg(p.dst + i);
    if (from < 0 || from == to) return;
    const bool report = part == 0 && threadIdx.x == 0;
    bool ok = from < p.num_rows && to >= 0 && to < p.num_rows;
    int length = 0, first = 0;
    if (ok) {
        length = __ldg(p.seq_lens + from);
        ok = length >= 0 && length <= (int64_t)p.max_blocks << p.bs_log2 && length == __ldg(p.seq_lens + to);
        if (p.first) first = max(0, __ldg(p.first + from));
    }
    if (!ok) {
        if (report) record_error(p.err, ERR_INDEX | SRC_BEAM);
        return;
    }
    const int row_vecs = (int)(p.row_bytes / (int)sizeof(V));
    const int32_t *src_pages = p.page_table + (int64_t)from * p.max_blocks;
    const int32_t *dst_pages = p.page_table + (int64_t)to * p.max_blocks;
    const int64_t total = (int64_t)(length - first) * row_vecs;
    const int bs = 1 << p.bs_log2;
    bool bad = false;
    for (int64_t x = (int64_t)part * kCopyThreads + threadIdx.x; x < total; x += (int64_t)parts * kCopyThreads) {
        const int tok = (int)(x / row_vecs), v = (int)(x - (int64_t)tok * row_vecs), pos = first + tok;
        const int a = __ldg(src_pages + (pos >> p.bs_log2)), b = __ldg(dst_pages + (pos >> p.bs_log2));
        if (a < 0 || b < 0 || a >= p.num_blocks || b >= p.num_blocks) {
            bad = true;
            continue;
        }
        const int64_t sa = (((int64_t)a << p.bs_log2) + (pos & (bs - 1))) * row_vecs + v;
        const int64_t sb = (((int64_t)b << p.bs_log2) + (pos & (bs - 1))) * row_vecs + v;
        V w[3];
#pragma unroll
        for (int c = 0; c < 3; ++c)
            if (p.cache[c]) w[c] = reinterpret_cast<const V *>(p.cache[c])[sa];
#pragma unroll
        for (int c = 0; c < 3; ++c)
            if (p.cache[c]) reinterpret_cast<V *>(p.cache[c])[sb] = w[c];
    }
    if (bad) record_error(p.err, ERR_INDEX | SRC_BEAM);
}

}  // namespace

cudaError_t launch_beam_select(const BeamParams &p, cudaStream_t stream) {
    auto *scan = p.bf16 ? p.wide ? beam_scan_kernel<__nv_bfloat16, 0> : beam_scan_kernel<__nv_bfloat16, 1>
                        : p.wide ? beam_scan_kernel<float, 0> : beam_scan_kernel<float, 1>;
    main_kernel_event_before(stream);
    scan<<<(unsigned)(p.groups * p.W * p.slices), kScanWarps * 32, 0, stream>>>(p);
    main_kernel_event_after(stream);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.groups);
    int per = 1;
    while (per * 2 * p.W <= 32 && per * 2 <= p.slices) per *= 2;
    cfg.blockDim = dim3((unsigned)(p.W * per) * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, beam_join_kernel, p, per);
}

cudaError_t launch_beam_rows(const int32_t *parents, const int32_t *rows, int32_t *rows_out, int32_t *source,
                             int groups, int W, uint32_t *err, cudaStream_t stream) {
    beam_rows_kernel<<<(unsigned)((groups + 3) / 4), 128, 0, stream>>>(parents, rows, rows_out, source, groups, W, err);
    return cudaGetLastError();
}

// CTAs of a pair: 32 a multiprocessor with the pairs there are, a few times what one holds, at most one for
// every `per` units of its work
static int parts_of(int64_t work, int64_t per, int n, int num_sms) {
    int64_t parts = (work + per - 1) / per;
    const int64_t most = ((int64_t)num_sms * 8 * 4 + n - 1) / n;
    if (parts > most) parts = most;
    return (int)(parts < 1 ? 1 : parts);
}

cudaError_t launch_copy_states(void *cache, const int32_t *src, const int32_t *dst, int n, int64_t num_slots,
                               int64_t slot_bytes, int num_sms, uint32_t *err, cudaStream_t stream) {
    const int64_t vecs = slot_bytes / 16;
    const int parts = parts_of(vecs, kCopyThreads * kCopyAhead, n, num_sms);
    main_kernel_event_before(stream);
    copy_states_kernel<<<(unsigned)(n * parts), kCopyThreads, 0, stream>>>(reinterpret_cast<uint4 *>(cache), src, dst,
                                                                          num_slots, vecs, parts, err);
    main_kernel_event_after(stream);
    return cudaGetLastError();
}

cudaError_t launch_copy_kvcache(const CopyRowsParams &p, int num_sms, cudaStream_t stream) {
    const int64_t work = ((int64_t)p.max_blocks << p.bs_log2) * (p.row_bytes / 16 + 1);
    const int parts = parts_of(work, kCopyThreads, p.n, num_sms);
    const uintptr_t all = (uintptr_t)p.cache[0] | (uintptr_t)p.cache[1] | (uintptr_t)p.cache[2] | (uintptr_t)p.row_bytes;
    auto *kernel = (all & 15) == 0 ? copy_kvcache_kernel<uint4> : copy_kvcache_kernel<uint16_t>;
    main_kernel_event_before(stream);
    kernel<<<(unsigned)(p.n * parts), kCopyThreads, 0, stream>>>(p, parts);
    main_kernel_event_after(stream);
    return cudaGetLastError();
}

}  // namespace attn
