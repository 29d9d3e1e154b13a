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
// by token.  The logarithm of the sum and the scores are in 64 bits: which of two
// candidates comes first may hang on the last digits.
//
// One pass over the logits (HBM bounds it).  A CTA takes a slice of a row, a warp a
// share of the slice in vectors of eight neighbours a lane; every lane keeps a running
// maximum and the sum of exponentials, the warp the k best logits as a sorted list,
// one a lane.  A key is the logit's bits in an order that compares as unsigned above
// the token's complement: distinct, and a larger one comes first.  What exceeds
// the list's last key goes to a buffer in shared memory, which is merged into the list 32 at a time.
// A second small launch joins the slices and the beams of a group.
// Every row is cut and summed in the same way: equal rows give equal sums.
// ---------------------------------------------------------------------------
constexpr int kScanWarps = 8;
constexpr int kScanAhead = 4;                        // vectors of a warp in flight
constexpr int kScanBuf = 32 + 256;                   // keys waiting: less than 32, and one vector's

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

// eight neighbouring logits of a row from element i on; -inf behind the end
template <typename T, bool WIDE>
__device__ __forceinline__ void load8(const T *row, int i, int end, float (&x)[8]) {
    if (WIDE && i + 8 <= end) {
        if constexpr (sizeof(T) == 2) {
            const uint4 w = ldg_stream16(row + i);
            const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[2 * j] = __uint_as_float(r[j] << 16);
                x[2 * j + 1] = __uint_as_float(r[j] & 0xFFFF0000u);
            }
        } else {
            const uint4 w = ldg_stream16(row + i), y = ldg_stream16(row + i + 4);
            const uint32_t r[8] = {w.x, w.y, w.z, w.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(r[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = -INFINITY;
            if (i + j < end) x[j] = (float)row[i + j];
        }
    }
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(kScanWarps * 32) beam_scan_kernel(const BeamParams p) {
    __shared__ uint64_t buf[kScanWarps][kScanBuf];
    __shared__ float2 part[kScanWarps];
    asm volatile("griddepcontrol.launch_dependents;");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x / p.slices, slice = blockIdx.x - row * p.slices;
    const T *x0 = reinterpret_cast<const T *>(p.logits) + (int64_t)row * p.row_stride;
    const int begin = slice * p.slice_len, end = min(p.V, begin + p.slice_len);
    uint64_t *mine = buf[warp];
    uint64_t list = key_floor(), last = list;            // last: the k-th key so far
    int waiting = 0;
    float top = kLowest, sum = 0.f;                      // (finite: -inf - -inf would be NaN)
    const int per = (p.slice_len / (kScanWarps * 256) + kScanAhead - 1) / kScanAhead;
    auto flush = [&](int n) {                            // the first n <= 32 waiting keys into the list
        __syncwarp();
        const uint64_t k = lane < n ? mine[lane] : key_floor();
        list = merge32(list, sort32(k, lane), lane);
        const uint64_t kth = shfl64(list, p.k - 1);
        last = kth > last ? kth : last;
        __syncwarp();
    };
#pragma unroll 1
    for (int it = 0; it < per; ++it) {
        float x[kScanAhead][8];
        const int at = begin + (it * kScanAhead * kScanWarps + warp) * 256 + lane * 8;
#pragma unroll
        for (int v = 0; v < kScanAhead; ++v) load8<T, WIDE>(x0, at + v * kScanWarps * 256, end, x[v]);
        float high[kScanAhead];
#pragma unroll
        for (int v = 0; v < kScanAhead; ++v)
            high[v] = max3f(max3f(x[v][0], x[v][1], x[v][2]), max3f(x[v][3], x[v][4], x[v][5]), fmaxf(x[v][6], x[v][7]));
        const float lane_top = fmaxf(fmaxf(high[0], high[1]), fmaxf(high[2], high[3]));
        const float new_top = fmaxf(top, lane_top);
        sum *= ex2((top - new_top) * kLog2e);
        top = new_top;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int v = 0; v < kScanAhead; ++v) {
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                float a = x[v][j], b = x[v][j + 1];
                add2(a, b, -top, -top);
                fma2(a, b, a, b, kLog2e, kLog2e, 0.f, 0.f);
                add2(s0, s1, ex2(a), ex2(b));
            }
        }
        sum += s0 + s1;
        if (it == 0) {
            // k lanes have a logit at or above the k-th largest of the lanes' maxima
            const uint64_t t = shfl64(sort32(key_of(lane_top, 0u), lane), p.k - 1);
            const uint64_t bound = (t & 0xFFFFFFFF00000000ull) - 1;
            last = bound > last ? bound : last;
        }
#pragma unroll 1
        for (int v = 0; v < kScanAhead; ++v) {
            const float hv = v == 0 ? high[0] : v == 1 ? high[1] : v == 2 ? high[2] : high[3];
            if (!__any_sync(0xffffffffu, key_of(hv, 0u) > last)) continue;
            const uint32_t token = (uint32_t)(at + v * kScanWarps * 256);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float xj = v == 0 ? x[0][j] : v == 1 ? x[1][j] : v == 2 ? x[2][j] : x[3][j];
                const uint64_t key = key_of(xj, token + j);
                const bool in = key > last && xj == xj;
                const uint32_t who = __ballot_sync(0xffffffffu, in);
                if (in) mine[waiting + __popc(who & ((1u << lane) - 1u))] = key;
                waiting += __popc(who);
            }
            if (waiting < 32) continue;
            int done = 0;
            for (; waiting - done >= 32; done += 32) {
                flush(32);
                if (waiting - done > 32) {               // the rest moves up, 32 at a time, front to back
                    for (int m = 32; m < waiting - done; m += 32) {
                        const uint64_t k = m + lane < waiting - done ? mine[m + lane] : 0;
                        __syncwarp();
                        mine[m - 32 + lane] = k;
                        __syncwarp();
                    }
                }
            }
            waiting -= done;
        }
    }
    if (waiting > 0) flush(waiting);
    // the warps' lists and sums
#pragma unroll
    for (int w = 16; w > 0; w /= 2) {
        const float t = __shfl_xor_sync(0xffffffffu, top, w), s = __shfl_xor_sync(0xffffffffu, sum, w);
        const float m = fmaxf(top, t);
        sum = sum * ex2((top - m) * kLog2e) + s * ex2((t - m) * kLog2e);
        top = m;
    }
    __syncthreads();
    mine[lane] = list;
    if (lane == 0) part[warp] = make_float2(top, sum);
    __syncthreads();
#pragma unroll 1
    for (int half = kScanWarps / 2; half > 0; half /= 2) {
        if (warp < half) {
            list = merge32(list, buf[warp + half][lane], lane);
            mine[lane] = list;
            if (lane == 0) {
                const float2 a = part[warp], b = part[warp + half];
                const float m = fmaxf(a.x, b.x);
                part[warp] = make_float2(m, a.y * ex2((a.x - m) * kLog2e) + b.y * ex2((b.x - m) * kLog2e));
            }
        }
        __syncthreads();
    }
    if (warp == 0) {
        if (lane < p.k) p.keys[(int64_t)blockIdx.x * p.k + lane] = list;
        if (lane == 0) p.sums[blockIdx.x] = part[0];
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

// A CTA per group, a warp per beam.
__global__ void __launch_bounds__(1024) beam_join_kernel(const BeamParams p) {
    __shared__ Ranked lists[kBeamMax][32];
    __shared__ uint32_t token_of[kBeamMax][32];
    __shared__ double norm[kBeamMax];                 // log of the row's sum; NaN: the row has no candidates
    __shared__ float2 total[kBeamMax];
    const int lane = threadIdx.x & 31, b = threadIdx.x >> 5, g = blockIdx.x;
    const int row = g * p.W + b;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    uint64_t list = key_floor();
    const uint64_t *keys = p.keys + (int64_t)row * p.slices * p.k;
    for (int s = 0; s < p.slices; ++s) {
        const uint64_t k = lane < p.k ? keys[s * p.k + lane] : key_floor();
        list = s == 0 ? k : merge32(list, k, lane);
    }
    float top = kLowest, sum = 0.f;
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
    if (lane == 0) total[b] = make_float2(top, sum);
    __syncthreads();
    if (b == 0 && lane < p.W) {
        // the logarithms of all beams in one warp: 64-bit units are few
        const float2 x = total[lane];
        const float score = __ldg(p.scores + (int64_t)g * p.W + lane);
        const bool some = x.y > 0.f && x.y < INFINITY;
        // a row of -inf alone and a score of -inf are masks, NaN and +inf mistakes
        if ((!some && !(x.y == 0.f)) || !(score < INFINITY)) record_error(p.err, ERR_RANGE | SRC_BEAM);
        norm[lane] = some && score > -INFINITY && score < INFINITY ? (double)x.x + log((double)x.y)
                                                                   : __longlong_as_double(0x7FF8000000000000ll);
    }
    __syncthreads();
    const double score = (double)__ldg(p.scores + row) + ((double)key_logit(list) - norm[b]);
    const bool real = list > key_floor() && norm[b] == norm[b];
    Ranked r = {real ? ordered(score) : 0ull, ~(uint32_t)(b * 32 + lane)};
    lists[b][lane] = r;
    token_of[b][lane] = key_token(list);
    __syncthreads();
    for (int n = p.W; n > 1; n = (n + 1) / 2) {
        const int half = (n + 1) / 2;
        if (b + half < n) {
            r = merge_ranked(r, lists[b + half][lane], lane);
            lists[b][lane] = r;
        }
        __syncthreads();
    }
    if (b == 0 && lane < p.k) {
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
// pass, 2 bytes moved per byte copied (HBM).
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
// VEC: bytes of an access.
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
    auto *scan = p.bf16 ? p.wide ? beam_scan_kernel<__nv_bfloat16, true> : beam_scan_kernel<__nv_bfloat16, false>
                        : p.wide ? beam_scan_kernel<float, true> : beam_scan_kernel<float, false>;
    main_kernel_event_before(stream);
    scan<<<(unsigned)(p.groups * p.W * p.slices), kScanWarps * 32, 0, stream>>>(p);
    main_kernel_event_after(stream);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.groups);
    cfg.blockDim = dim3((unsigned)p.W * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, beam_join_kernel, p);
}

cudaError_t launch_beam_rows(const int32_t *parents, const int32_t *rows, int32_t *rows_out, int32_t *source,
                             int groups, int W, uint32_t *err, cudaStream_t stream) {
    beam_rows_kernel<<<(unsigned)((groups + 3) / 4), 128, 0, stream>>>(parents, rows, rows_out, source, groups, W, err);
    return cudaGetLastError();
}

// CTAs of a pair: enough to fill the GPU (eight a multiprocessor) with the pairs there are, at most one for
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
