// step_tables.cu -- page tables on the GPU: growing them by a step's new tokens
// (block table, slot mapping, positions, cu_seqlens of the step) and taking
// tokens back.
//
// With len_b the tokens request b has cached and n_b its new ones,
//   need_b = ceil((len_b + n_b) / bs) - ceil(len_b / bs)
// pages come off the top of the free list in request order, so request b's
// pages start at the exclusive prefix sum of need.  Everything else (slots,
// positions) is index arithmetic per token.
//
// Two launches: one CTA runs the prefix sums and settles who is served
// (tables_plan_kernel; it alone reads and writes seq_lens and num_free, so no
// other CTA can see them half-updated), then a grid writes the table rows and
// the tokens.  Nothing depends on the order of atomics.
#include "common.cuh"
#include "kernels.h"

namespace attn {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kTokensPerThread = 4;
constexpr int kTokensPerCta = kFillThreads * kTokensPerThread;
constexpr int kRowSeg = 512;               // table columns one warp writes per work item
constexpr int64_t kI32Max = 0x7fffffffll;

__device__ __forceinline__ int64_t warp_incl_scan(int64_t v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Inclusive prefix sum over the CTA (kPlanThreads threads); *total gets the sum.
// Every thread calls it; `part` holds 33 values and is free again on return.
__device__ __forceinline__ int64_t cta_incl_scan(int64_t v, int64_t *part, int64_t *total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    v = warp_incl_scan(v);
    if (lane == 31) part[w] = v;
    __syncthreads();
    if (w == 0) {
        const int64_t s = warp_incl_scan(part[lane]);
        __syncwarp();
        part[lane] = s;
    }
    __syncthreads();
    if (w > 0) v += part[w - 1];
    *total = part[kPlanThreads / 32 - 1];
    __syncthreads();
    return v;
}

__device__ __forceinline__ int clamp_i32(int64_t v, bool &bad) {
    if (v > kI32Max) {
        bad = true;
        return (int)kI32Max;
    }
    return (int)v;
}

// Claim of a request row by batch entry b: below every valid length, and the
// smaller the earlier the entry, so atomicMin leaves the first entry that names
// a row as its owner (a later one is a caller error and is not served).
__device__ __forceinline__ int claim_code(int b) { return -(kTablesMaxBatch + 1 - b); }

// Length of the request named by entry b; -1 if the entry is not usable.
__device__ __forceinline__ int row_length(const TablesParams &p, int b, int &row) {
    row = p.rows ? __ldg(p.rows + b) : b;
    if (row < 0 || row >= p.num_rows) return -1;
    const int len = __ldcg(p.seq_lens + row);
    return (len < 0 || (int64_t)len > ((int64_t)p.max_blocks << p.bs_log2)) ? -1 : len;
}

__device__ __forceinline__ int pages_of(int64_t len, int bs_log2) {
    return (int)((len + (1ll << bs_log2) - 1) >> bs_log2);
}

// GROW: context_lens, cache_seqlens, cu_q, cu_k, page_top (workspace: index in
// the free list just above the request's first new page), seq_lens, num_free.
// !GROW (trim): spans (workspace: first page taken back, pages before, place
// from the new top of the free list), seq_lens, num_free.
template <bool GROW>
__global__ void __launch_bounds__(kPlanThreads) tables_plan_kernel(const TablesParams p) {
    __shared__ int64_t part[33];
    __shared__ int moved_s;
    const int tid = threadIdx.x;
    asm volatile("griddepcontrol.launch_dependents;");
    bool bad = false, full = false;
    if (tid == 0) moved_s = 0;
    // lengths before the step (kept where the last pass finds them again), then the claims
    for (int b = tid; b < p.batch; b += kPlanThreads) {
        int row;
        const int len = row_length(p, b, row);
        p.before[b] = len;
        bad |= len < 0;
    }
    __syncthreads();
    for (int b = tid; b < p.batch; b += kPlanThreads) {
        if (p.before[b] >= 0) atomicMin(p.seq_lens + (p.rows ? __ldg(p.rows + b) : b), claim_code(b));
    }
    __syncthreads();

    const int nf_raw = __ldcg(p.num_free);
    const int nf = min(max(nf_raw, 0), p.num_pages);
    bad |= nf != nf_raw;
    int64_t base_n = 0, base_need = 0, base_k = 0;
    int moved = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kPlanThreads) {
        const int b = b0 + tid;
        const bool here = b < p.batch;
        int len = here ? p.before[b] : -1;
        const int row = here ? (p.rows ? __ldg(p.rows + b) : b) : -1;
        bool mine = false;
        if (len >= 0) {
            mine = __ldcg(p.seq_lens + row) == claim_code(b);
            bad |= !mine;
        }
        int64_t tot;
        if (GROW) {
            int64_t n = here ? __ldg(p.lens + b) : 0;
            if (n < 0) {
                bad = true;
                n = 0;
            }
            if (n > p.max_tokens) n = p.max_tokens + 1;   // cannot fit; keeps the sums small
            const int64_t cum_n = base_n + cta_incl_scan(n, part, &tot);
            base_n += tot;
            const int old_pages = pages_of(len < 0 ? 0 : len, p.bs_log2);
            const int want = pages_of((len < 0 ? 0 : len) + n, p.bs_log2);
            bool ok = mine;
            if (here && cum_n > p.max_tokens) bad = true, ok = false;
            if (ok && want > p.max_blocks) full = true, ok = false;
            const int need = ok ? want - old_pages : 0;
            const int64_t cum = base_need + cta_incl_scan(need, part, &tot);
            base_need += tot;
            if (need > 0) {
                if (cum > nf) full = true, ok = false;
                else moved = max(moved, (int)cum);
            }
            if (len < 0) len = 0;
            const int after = ok ? (int)(len + n) : len;
            const int64_t cum_k = base_k + cta_incl_scan(here ? after : 0, part, &tot);
            base_k += tot;
            if (here) {
                p.context_lens[b] = len;
                p.cache_seqlens[b] = after;
                p.cu_q[b + 1] = (int)min(cum_n, p.max_tokens);
                p.cu_k[b + 1] = clamp_i32(cum_k, bad);
                // a request that is not served has page_top -1: its tokens get slot -1
                p.page_top[b] = !ok ? -1 : need > 0 ? nf - (int)(cum - need) : 0;
                if (mine) p.seq_lens[row] = after;
            }
        } else {
            int keep = here ? __ldg(p.lens + b) : 0;
            if (keep < 0) {
                bad = true;
                keep = 0;
            }
            const int after = mine ? min(keep, len) : 0;
            const int old_pages = mine ? pages_of(len, p.bs_log2) : 0;
            const int kept = mine ? pages_of(after, p.bs_log2) : 0;
            const int freed = old_pages - kept;
            const int64_t cum = base_need + cta_incl_scan(freed, part, &tot);
            base_need += tot;
            bool ok = mine;
            if (freed > 0) {
                if (cum > p.num_pages - nf) bad = true, ok = false;   // more pages than the pool has
                else moved = max(moved, (int)cum);
            }
            if (here) {
                p.span[b] = make_int4(ok ? kept : 0, ok ? old_pages : 0, ok ? (int)(cum - freed) : 0, row);
                if (mine) p.seq_lens[row] = ok ? after : len;
            }
        }
    }
    if (moved) atomicMax(&moved_s, moved);
    const unsigned any_bad = __ballot_sync(0xffffffffu, bad), any_full = __ballot_sync(0xffffffffu, full);
    if ((tid & 31) == 0) {
        if (any_bad) record_error(p.err, ERR_INDEX | SRC_TABLES);
        if (any_full) record_error(p.err, ERR_CAPACITY | SRC_TABLES);
    }
    __syncthreads();
    if (tid == 0) {
        *p.num_free = GROW ? nf - moved_s : nf + moved_s;
        if (GROW) p.cu_q[0] = p.cu_k[0] = 0;
    }
}

// Page j of request b in this step (row: its row of page_table): below `before`
// from the table, from there on off the free list.  -1 (recorded) if the stored
// page is not one of the pool's.
__device__ __forceinline__ int page_of(const TablesParams &p, int row, int before, int top, int j, bool &bad) {
    int page;
    if (j < before) {
        page = __ldg(p.page_table + (int64_t)row * p.max_blocks + j);
    } else {
        page = __ldg(p.free_pages + (top - 1 - (j - before)));
    }
    if (page < 0 || page >= p.num_pages) {
        bad = true;
        page = -1;
    }
    return page;
}

// The first `row_ctas` CTAs write block_table (a warp per request and kRowSeg
// columns) and the new entries of page_table; the others write slot_mapping and
// positions, 4 consecutive tokens per thread.  page_table is read below a
// request's old page count and written from there on.
__global__ void __launch_bounds__(kFillThreads) tables_fill_kernel(const TablesParams p, int row_ctas) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    bool bad = false;
    if ((int)blockIdx.x < row_ctas) {
        const int segs = (p.max_blocks + kRowSeg - 1) / kRowSeg;
        const int64_t items = (int64_t)p.batch * segs;
        const int64_t step = (int64_t)row_ctas * (kFillThreads / 32);
        for (int64_t it = (int64_t)blockIdx.x * (kFillThreads / 32) + warp; it < items; it += step) {
            const int b = (int)(it / segs), j0 = (int)(it - (int64_t)b * segs) * kRowSeg;
            const int before = pages_of(p.context_lens[b], p.bs_log2);
            const int after = pages_of(p.cache_seqlens[b], p.bs_log2);
            const int top = p.page_top[b];
            const int row = p.rows ? __ldg(p.rows + b) : b;
            const int j1 = min(j0 + kRowSeg, p.max_blocks);
            for (int j = j0 + lane; j < j1; j += 32) {
                int page = -1;
                if (j < after) {
                    page = page_of(p, row, before, top, j, bad);
                    if (j >= before) p.page_table[(int64_t)row * p.max_blocks + j] = page;
                }
                p.block_table[(int64_t)b * p.max_blocks + j] = page;
            }
        }
    } else {
        const int64_t t0 = ((int64_t)blockIdx.x - row_ctas) * kTokensPerCta + threadIdx.x * kTokensPerThread;
        const int64_t total = p.cu_q[p.batch];
        // first request whose tokens end behind t0 (empty requests end where they start)
        int lo = 0, hi = p.batch;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (p.cu_q[mid + 1] > t0) hi = mid;
            else lo = mid + 1;
        }
        int b = lo, start = 0, end = -1, len = 0, before = 0, top = -1, row = 0;
        const int64_t mask = (1ll << p.bs_log2) - 1;
#pragma unroll
        for (int u = 0; u < kTokensPerThread; ++u) {
            const int64_t t = t0 + u;
            if (t >= p.max_tokens) break;
            int64_t slot = -1;
            int pos = 0;
            if (t < total) {
                if (t >= end) {
                    if (end >= 0) ++b;
                    while (p.cu_q[b + 1] <= t) ++b;
                    start = p.cu_q[b];
                    end = p.cu_q[b + 1];
                    len = p.context_lens[b];
                    before = pages_of(len, p.bs_log2);
                    top = p.page_top[b];
                    row = p.rows ? __ldg(p.rows + b) : b;
                }
                pos = (int)(len + (t - start));
                if (top >= 0) {
                    const int page = page_of(p, row, before, top, pos >> p.bs_log2, bad);
                    if (page >= 0) slot = ((int64_t)page << p.bs_log2) + (pos & mask);
                }
            }
            p.slot_mapping[t] = slot;
            p.positions[t] = pos;
        }
    }
    const unsigned any = __ballot_sync(0xffffffffu, bad);
    if (any && lane == 0) record_error(p.err, ERR_INDEX | SRC_TABLES);
}

// Pages kept..before of every request go back: the request order and page order
// that a grow of the same spans took them in, reversed, so growing and trimming
// by the same amounts restores the list.
__global__ void __launch_bounds__(kFillThreads) tables_release_kernel(const TablesParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int top = *p.num_free;
    bool bad = false;
    const int64_t step = (int64_t)gridDim.x * (kFillThreads / 32);
    for (int64_t b = (int64_t)blockIdx.x * (kFillThreads / 32) + warp; b < p.batch; b += step) {
        const int4 s = p.span[b];
        for (int j = s.x + lane; j < s.y; j += 32) {
            int32_t *at = p.page_table + (int64_t)s.w * p.max_blocks + j;
            const int page = *at;
            bad |= page < 0 || page >= p.num_pages;
            p.free_pages[top - 1 - (s.z + (j - s.x))] = page;
            *at = -1;
        }
    }
    const unsigned any = __ballot_sync(0xffffffffu, bad);
    if (any && lane == 0) record_error(p.err, ERR_INDEX | SRC_TABLES);
}

// Launch `k` as the programmatic dependent of the launch before it.
template <typename... A>
cudaError_t launch_dependent(void (*k)(A...), unsigned grid, unsigned block, cudaStream_t stream, A... a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a...);
}

}  // namespace

cudaError_t launch_step_tables(const TablesParams &p, int num_sms, cudaStream_t stream) {
    tables_plan_kernel<true><<<1, kPlanThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t items = (int64_t)p.batch * ((p.max_blocks + kRowSeg - 1) / kRowSeg);
    int64_t row_ctas = (items + kFillThreads / 32 - 1) / (kFillThreads / 32);
    if (row_ctas > 4 * num_sms) row_ctas = 4 * num_sms;
    const int64_t tok_ctas = (p.max_tokens + kTokensPerCta - 1) / kTokensPerCta;
    return launch_dependent(tables_fill_kernel, (unsigned)(row_ctas + tok_ctas), kFillThreads, stream, p,
                            (int)row_ctas);
}

cudaError_t launch_trim_pages(const TablesParams &p, int num_sms, cudaStream_t stream) {
    tables_plan_kernel<false><<<1, kPlanThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    int64_t grid = (p.batch + kFillThreads / 32 - 1) / (kFillThreads / 32);
    if (grid > 4 * num_sms) grid = 4 * num_sms;
    return launch_dependent(tables_release_kernel, (unsigned)grid, kFillThreads, stream, p);
}

}  // namespace attn
