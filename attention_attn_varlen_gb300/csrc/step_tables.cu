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
// One CTA runs the prefix sums and settles who is served (it alone reads and
// writes seq_lens and num_free, so no other CTA can see them half-updated); a
// second launch writes the table rows and the tokens, or the same CTA where that
// is little.  Nothing depends on the order of atomics.
//
// Small steps are bound by latency: the sums keep their entries in registers and
// scan up to 4,096 of them in one round.  Large ones are bound by writing 12 bytes
// per token and 4 per table entry: a CTA brings the offsets that its tokens span
// into shared memory, and a thread writes four neighbouring tokens or entries with
// 16-byte stores.  4,096 prompts with 4.2 M tokens: plan 17 us (one SM gathers all rows, lengths and
// claims, and waits for them most of the time), fill 20 (84 instructions a token, issue slots 56 %
// busy, stores that mostly stay in L2), trim 12 + 5.
#include "common.cuh"
#include "kernels.h"

namespace attn {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kTokens = 4;                 // neighbouring tokens per thread ...
constexpr int kGroups = 2;                 // ... twice per round
constexpr int kRowSeg = 512;               // table columns one warp writes per work item
// table entries and tokens that the planning CTA writes itself, a few per thread (64 requests of 64
// pages, one token each, grown and trimmed back: 21 us a pass, 13.2 in a graph; with second launches 25
// and 14.3)
constexpr int64_t kInlineWork = 16384;
constexpr int kSharedRows = kGroups * kPlanThreads * kTokens;   // request rows whose claims fit shared memory
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
// One barrier: every warp adds up the 32 warps' sums by itself.  `part` (32 values)
// must not be the one of the call before.
__device__ __forceinline__ int64_t cta_incl_scan(int64_t v, int64_t *part, int64_t *total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    v = warp_incl_scan(v);
    if (lane == 31) part[w] = v;
    __syncthreads();
    const int64_t s = warp_incl_scan(part[lane]);
    *total = __shfl_sync(0xffffffffu, s, 31);
    const int64_t below = __shfl_sync(0xffffffffu, s, (w + 31) & 31);
    return w > 0 ? v + below : v;
}

// The first request whose tokens end behind token t (empty requests end where they
// start; batch if none), by one warp: 31 of 32 candidates fall away with each load.
__device__ __forceinline__ int request_of(const int32_t *cu, int batch, int64_t t) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = batch;                    // the answer is in [lo, hi]
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32, probe = min(lo + (lane + 1) * step - 1, hi - 1);
        const unsigned behind = __ballot_sync(0xffffffffu, cu[probe + 1] > t);
        if (behind == 0) return hi;
        const int f = __ffs(behind) - 1;
        hi = min(lo + (f + 1) * step - 1, hi - 1);
        lo += f * step;
        if (step == 1) break;
    }
    return hi;
}

__device__ __forceinline__ int clamp_i32(int64_t v, bool &bad) {
    if (v > kI32Max) {
        bad = true;
        return (int)kI32Max;
    }
    return (int)v;
}

// Claim of a request row by batch entry b, in seq_lens itself where the rows are
// too many for shared memory: below every valid length, and the smaller the
// earlier the entry, so atomicMin leaves the first entry that names a row as its
// owner (a later one is a caller error and is not served).
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

// Page j of request b in this step (row: its row of page_table): below `before`
// from the table, from there on off the free list.  -1 (recorded) if the stored
// page is not one of the pool's.
__device__ __forceinline__ int page_of(const TablesParams &p, int64_t row, int before, int top, int j, bool &bad) {
    const int page = j < before ? p.page_table[row * p.max_blocks + j] : __ldg(p.free_pages + (top - 1 - (j - before)));
    if (page >= 0 && page < p.num_pages) return page;
    bad = true;
    return -1;
}

// block_table (a warp per request and kRowSeg columns) and the new entries of
// page_table, by warp `w` of `warps`.  page_table is read below a request's old
// page count and written from there on.
__device__ __forceinline__ void fill_rows(const TablesParams &p, int64_t w, int64_t warps, bool &bad) {
    const int lane = threadIdx.x & 31;
    const int segs = (p.max_blocks + kRowSeg - 1) / kRowSeg;
    const int64_t items = (int64_t)p.batch * segs;
    for (int64_t it = w; it < items; it += warps) {
        const int b = (int)(it / segs), j0 = (int)(it - (int64_t)b * segs) * kRowSeg;
        const int4 r = p.info[b];
        const int before = pages_of(r.x, p.bs_log2), after = pages_of(r.y, p.bs_log2), top = r.z;
        const int64_t row = r.w;
        const int j1 = min(j0 + kRowSeg, p.max_blocks);
        int32_t *out = p.block_table + (int64_t)b * p.max_blocks;
        if (p.vec_rows) {
#pragma unroll 4
            for (int j = j0 + 4 * lane; j < j1; j += 128) {
                int4 v = make_int4(-1, -1, -1, -1);
                if (j + 4 <= before) {          // all old pages
                    v = *reinterpret_cast<const int4 *>(p.page_table + row * p.max_blocks + j);
                    const int lim = p.num_pages;
                    if ((unsigned)v.x >= (unsigned)lim) bad = true, v.x = -1;
                    if ((unsigned)v.y >= (unsigned)lim) bad = true, v.y = -1;
                    if ((unsigned)v.z >= (unsigned)lim) bad = true, v.z = -1;
                    if ((unsigned)v.w >= (unsigned)lim) bad = true, v.w = -1;
                } else if (j < after) {
                    int *e = reinterpret_cast<int *>(&v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (j + i >= after) break;
                        e[i] = page_of(p, row, before, top, j + i, bad);
                        if (j + i >= before) p.page_table[row * p.max_blocks + j + i] = e[i];
                    }
                }
                *reinterpret_cast<int4 *>(out + j) = v;
            }
        } else {
            for (int j = j0 + lane; j < j1; j += 32) {
                int page = -1;
                if (j < after) {
                    page = page_of(p, row, before, top, j, bad);
                    if (j >= before) p.page_table[row * p.max_blocks + j] = page;
                }
                out[j] = page;
            }
        }
    }
}

// slot_mapping and positions of the tokens that CTA `cta` of `ctas` (THREADS
// threads) takes, kGroups x THREADS x kTokens at a time.  cu_s: shared memory for as
// many offsets and one more.
template <int THREADS>
__device__ __forceinline__ void fill_tokens(const TablesParams &p, int64_t cta, int64_t ctas, int *cu_s, bool &bad) {
    constexpr int SPAN = kGroups * THREADS * kTokens;
    __shared__ int range[2];
    const int mask = (int)((1ll << p.bs_log2) - 1);
    const int64_t total = p.cu_q[p.batch];
    for (int64_t base = cta * SPAN; base < p.max_tokens; base += ctas * SPAN) {
        // the requests of the span's first and last token
        if (threadIdx.x < 64) {
            const int w = threadIdx.x >> 5;
            const int at = request_of(p.cu_q, p.batch, w == 0 ? base : min(base + SPAN, total) - 1);
            if ((threadIdx.x & 31) == 0) range[w] = at;
        }
        __syncthreads();
        const int b0 = range[0], nb = range[1] - b0 + 1;      // of a span with tokens
        const bool shared = nb <= SPAN;
        if (base < total && shared)
            for (int i = threadIdx.x; i <= nb; i += THREADS) cu_s[i] = p.cu_q[b0 + i];
        __syncthreads();
        const int *cu = shared ? cu_s : p.cu_q + b0;
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
            const int64_t t0 = base + (int64_t)(k * THREADS + threadIdx.x) * kTokens;
            int64_t slot[kTokens];
            int pos[kTokens];
            int b = 0, start = 0, end = -1, before = 0;
            int4 r = make_int4(0, 0, -1, 0);
            if (t0 < total) {
                int lo = 0, hi = nb - 1;                      // requests may be empty inside the span
                while (lo < hi) {
                    const int mid = (lo + hi) >> 1;
                    if (cu[mid + 1] > t0) hi = mid;
                    else lo = mid + 1;
                }
                b = lo;
            }
            int at = -1, page = -1;                           // the page looked up last
#pragma unroll
            for (int u = 0; u < kTokens; ++u) {
                const int64_t t = t0 + u;
                slot[u] = -1;
                pos[u] = 0;
                if (t >= total) continue;
                if (t >= end) {
                    while (cu[b + 1] <= t) ++b;
                    start = cu[b];
                    end = cu[b + 1];
                    r = p.info[b0 + b];
                    before = pages_of(r.x, p.bs_log2);
                    at = -1;
                }
                pos[u] = (int)(r.x + (t - start));
                if (r.z < 0) continue;
                const int j = pos[u] >> p.bs_log2;
                if (j != at) page = page_of(p, r.w, before, r.z, at = j, bad);
                if (page >= 0) slot[u] = ((int64_t)page << p.bs_log2) + (pos[u] & mask);
            }
            if (p.vec_tokens && t0 + kTokens <= p.max_tokens) {
                longlong2 *s = reinterpret_cast<longlong2 *>(p.slot_mapping + t0);
                s[0] = make_longlong2(slot[0], slot[1]);
                s[1] = make_longlong2(slot[2], slot[3]);
                *reinterpret_cast<int4 *>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            } else {
#pragma unroll
                for (int u = 0; u < kTokens; ++u) {
                    if (t0 + u >= p.max_tokens) break;
                    p.slot_mapping[t0 + u] = slot[u];
                    p.positions[t0 + u] = pos[u];
                }
            }
        }
        __syncthreads();                                      // cu_s and range are written again
    }
}

// Pages kept..before of every request go back: the request order and page order
// that a grow of the same spans took them in, reversed, so growing and trimming
// by the same amounts restores the list.  `lost`: one of them is not one of the
// pool's; drop_lost takes it out.
__device__ __forceinline__ void release_rows(const TablesParams &p, int64_t w, int64_t warps, bool &lost) {
    const int lane = threadIdx.x & 31;
    const int top = *p.num_free;
    for (int64_t b = w; b < p.batch; b += warps) {
        const int4 s = p.span[b];
        for (int j = s.x + lane; j < s.y; j += 32) {
            int32_t *at = p.page_table + (int64_t)s.w * p.max_blocks + j;
            const int page = *at;
            lost |= page < 0 || page >= p.num_pages;
            p.free_pages[top - 1 - (s.z + (j - s.x))] = page;
            *at = -1;
        }
    }
}

// The pages just given back without those outside the pool, in the same order (one
// warp, after every release is visible to it).
__device__ void drop_lost(const TablesParams &p) {
    const int lane = threadIdx.x & 31, top = __ldcg(p.num_free);
    int moved = 0;
    for (int b = lane; b < p.batch; b += 32) {
        const int4 s = p.span[b];
        if (s.y > s.x) moved = max(moved, s.z + s.y - s.x);
    }
    int out = top - __reduce_max_sync(0xffffffffu, moved);
    for (int base = out; base < top; base += 32) {
        const int page = base + lane < top ? __ldcg(p.free_pages + base + lane) : -1;
        const bool good = page >= 0 && page < p.num_pages;
        const unsigned mask = __ballot_sync(0xffffffffu, good);   // everyone has read: out <= base
        if (good) p.free_pages[out + __popc(mask & ((1u << lane) - 1))] = page;
        out += __popc(mask);
    }
    if (lane == 0) *p.num_free = out;
}

__device__ __forceinline__ void report(const TablesParams &p, bool bad, bool full) {
    const unsigned any_bad = __ballot_sync(0xffffffffu, bad), any_full = __ballot_sync(0xffffffffu, full);
    if ((threadIdx.x & 31) == 0) {
        if (any_bad) record_error(p.err, ERR_INDEX | SRC_TABLES);
        if (any_full) record_error(p.err, ERR_CAPACITY | SRC_TABLES);
    }
}

// GROW: context_lens, cache_seqlens, cu_q, cu_k, seq_lens, num_free, info
// (workspace: length before and after, index in the free list just above the
// request's first new page or -1 if it is not served, row).
// !GROW (trim): span (workspace: kept pages, pages before, place from the new
// top of the free list, row), seq_lens, num_free.
// ITEMS consecutive entries per thread and round; `fill`: then writes the tables
// (or the released pages) as well.
template <bool GROW, int ITEMS>
__global__ void __launch_bounds__(kPlanThreads, 1) tables_plan_kernel(const TablesParams p, bool fill) {
    __shared__ int64_t part[3][32];
    __shared__ int moved_s;
    __shared__ int cu_s[kGroups * kPlanThreads * kTokens + 1];
    int *claim = cu_s;                         // entry that owns each row (free again for the fill)
    const bool in_smem = p.num_rows <= kSharedRows;
    const int tid = threadIdx.x;
    constexpr int ROUND = kPlanThreads * ITEMS;
    asm volatile("griddepcontrol.launch_dependents;");
    bool bad = false, full = false;
    if (tid == 0) moved_s = 0;
    if (in_smem)
        for (int i = tid; i < p.num_rows; i += kPlanThreads) claim[i] = p.batch;
    int row[ITEMS], len[ITEMS];
    // lengths before the step, then the claims (a round's entries stay in registers; where there
    // are several rounds the workspace keeps them)
    const bool one = p.batch <= ROUND;
    for (int b0 = 0; b0 < p.batch; b0 += ROUND) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int b = b0 + tid * ITEMS + i;
            row[i] = 0;
            len[i] = -1;
            if (b >= p.batch) continue;
            len[i] = row_length(p, b, row[i]);
            if (!one) p.before[b] = len[i];
            bad |= len[i] < 0;
        }
    }
    __syncthreads();
    for (int b0 = 0; b0 < p.batch; b0 += ROUND) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int b = b0 + tid * ITEMS + i;
            if (b >= p.batch) continue;
            if (!one) {
                row[i] = p.rows ? __ldg(p.rows + b) : b;
                len[i] = p.before[b];
            }
            if (len[i] < 0) continue;
            if (in_smem) atomicMin(&claim[row[i]], b);
            else atomicMin(p.seq_lens + row[i], claim_code(b));
        }
    }
    const int nf_raw = __ldcg(p.num_free);
    const int nf = min(max(nf_raw, 0), p.num_pages);
    bad |= nf != nf_raw;
    __syncthreads();

    int64_t base_n = 0, base_need = 0, base_k = 0, tot;
    int moved = 0, round = 0;
    for (int b0 = 0; b0 < p.batch; b0 += ROUND) {
        const int first = b0 + tid * ITEMS;
        bool mine[ITEMS], ok[ITEMS];
        int amount[ITEMS], need[ITEMS];        // amount: new tokens, or tokens to keep
        int64_t sum = 0;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int b = first + i;
            const bool here = b < p.batch;
            if (!one) {
                row[i] = here && p.rows ? __ldg(p.rows + b) : b;
                len[i] = here ? p.before[b] : -1;
            }
            amount[i] = here ? __ldg(p.lens + b) : 0;
            if (amount[i] < 0) bad = true, amount[i] = 0;
            mine[i] = len[i] >= 0 && (in_smem ? claim[row[i]] == b : __ldcg(p.seq_lens + row[i]) == claim_code(b));
            bad |= len[i] >= 0 && !mine[i];
            ok[i] = mine[i];
            sum += amount[i];
        }
        if (GROW) {
            int64_t cum_n = base_n + cta_incl_scan(sum, part[0], &tot) - sum;
            base_n += tot;
            sum = 0;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const int b = first + i;
                cum_n += amount[i];
                if (b < p.batch) {
                    if (cum_n > p.max_tokens) bad = true, ok[i] = false;
                    p.cu_q[b + 1] = (int)min(cum_n, p.max_tokens);
                }
                const int64_t now = len[i] < 0 ? 0 : len[i];
                const int64_t want = (now + amount[i] + (1ll << p.bs_log2) - 1) >> p.bs_log2;
                if (ok[i] && want > p.max_blocks) full = true, ok[i] = false;
                need[i] = ok[i] ? (int)want - pages_of(now, p.bs_log2) : 0;
                sum += need[i];
            }
            int64_t cum = base_need + cta_incl_scan(sum, part[1], &tot) - sum;
            base_need += tot;
            sum = 0;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const int b = first + i;
                cum += need[i];
                if (need[i] > 0) {
                    if (cum > nf) full = true, ok[i] = false;
                    else moved = (int)cum;
                }
                if (len[i] < 0) len[i] = 0;
                const int after = ok[i] ? len[i] + amount[i] : len[i];
                if (b < p.batch) {
                    p.context_lens[b] = len[i];
                    p.cache_seqlens[b] = after;
                    p.info[b] = make_int4(len[i], after, !ok[i] ? -1 : need[i] > 0 ? nf - (int)(cum - need[i]) : 0, row[i]);
                    if (mine[i]) p.seq_lens[row[i]] = after;
                    sum += after;
                }
                len[i] = after;
            }
            int64_t cum_k = base_k + cta_incl_scan(sum, part[2], &tot) - sum;
            base_k += tot;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                if (first + i >= p.batch) break;
                cum_k += len[i];
                p.cu_k[first + i + 1] = clamp_i32(cum_k, bad);
            }
        } else {
            int after[ITEMS], kept[ITEMS];
            sum = 0;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                after[i] = mine[i] ? min(amount[i], len[i]) : 0;
                kept[i] = pages_of(after[i], p.bs_log2);
                need[i] = mine[i] ? pages_of(len[i], p.bs_log2) - kept[i] : 0;
                sum += need[i];
            }
            int64_t cum = base_need + cta_incl_scan(sum, part[round++ & 1], &tot) - sum;
            base_need += tot;
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const int b = first + i;
                cum += need[i];
                if (need[i] > 0) {
                    if (cum > p.num_pages - nf) bad = true, ok[i] = false;   // more pages than the pool has
                    else moved = (int)cum;
                }
                if (b >= p.batch) break;
                p.span[b] = ok[i] ? make_int4(kept[i], kept[i] + need[i], (int)(cum - need[i]), row[i])
                                  : make_int4(0, 0, 0, 0);
                if (mine[i]) p.seq_lens[row[i]] = ok[i] ? after[i] : len[i];
            }
        }
    }
    if (moved) atomicMax(&moved_s, moved);
    __syncthreads();
    if (tid == 0) {
        *p.num_free = GROW ? nf - moved_s : nf + moved_s;
        if (!GROW) p.before[0] = 0;            // from here on the release's count
        if (GROW) p.cu_q[0] = p.cu_k[0] = 0;
    }
    if (fill) {
        __syncthreads();
        if (GROW) {
            fill_rows(p, tid >> 5, kPlanThreads / 32, bad);
            fill_tokens<kPlanThreads>(p, 0, 1, cu_s, bad);
        } else {
            bool lost = false;
            release_rows(p, tid >> 5, kPlanThreads / 32, lost);
            bad |= lost;
            if (__syncthreads_or(lost) && tid < 32) drop_lost(p);
        }
    }
    report(p, bad, full);
}

// The first `row_ctas` CTAs write the table rows, the others the tokens.
__global__ void __launch_bounds__(kFillThreads) tables_fill_kernel(const TablesParams p, int row_ctas) {
    __shared__ int cu_s[kGroups * kFillThreads * kTokens + 1];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    bool bad = false;
    if ((int)blockIdx.x < row_ctas)
        fill_rows(p, (int64_t)blockIdx.x * (kFillThreads / 32) + (threadIdx.x >> 5),
                  (int64_t)row_ctas * (kFillThreads / 32), bad);
    else
        fill_tokens<kFillThreads>(p, blockIdx.x - row_ctas, gridDim.x - row_ctas, cu_s, bad);
    report(p, bad, false);
}

__global__ void __launch_bounds__(kFillThreads) tables_release_kernel(const TablesParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    bool lost = false;
    release_rows(p, (int64_t)blockIdx.x * (kFillThreads / 32) + (threadIdx.x >> 5),
                 (int64_t)gridDim.x * (kFillThreads / 32), lost);
    report(p, lost, false);
    // the last CTA to get here takes out what any of them lost (before[0]: CTAs done, those that lost pages
    // above the 16th bit).  4,096 requests: 5.4 us with it, 4.6 without
    const int any = __syncthreads_or(lost);
    if (threadIdx.x >= 32) return;
    bool last = false;
    if (threadIdx.x == 0) {
        __threadfence();
        const int mine = any ? 0x10001 : 1, all = atomicAdd(p.before, mine) + mine;
        last = (all & 0xFFFF) == (int)gridDim.x && all > 0xFFFF;
    }
    if (__any_sync(0xffffffffu, last)) {
        __threadfence();
        drop_lost(p);
    }
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

template <bool GROW>
cudaError_t plan(const TablesParams &p, bool fill, cudaStream_t stream) {
    if (p.batch <= kPlanThreads) tables_plan_kernel<GROW, 1><<<1, kPlanThreads, 0, stream>>>(p, fill);
    else tables_plan_kernel<GROW, 4><<<1, kPlanThreads, 0, stream>>>(p, fill);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_step_tables(const TablesParams &p, int num_sms, cudaStream_t stream) {
    const bool fill = (int64_t)p.batch * p.max_blocks + p.max_tokens <= kInlineWork;
    cudaError_t e = plan<true>(p, fill, stream);
    if (e != cudaSuccess || fill) return e;
    const int64_t items = (int64_t)p.batch * ((p.max_blocks + kRowSeg - 1) / kRowSeg);
    int64_t row_ctas = (items + kFillThreads / 32 - 1) / (kFillThreads / 32);
    if (row_ctas > 4 * num_sms) row_ctas = 4 * num_sms;
    const int64_t span = (int64_t)kGroups * kFillThreads * kTokens;
    int64_t tok_ctas = (p.max_tokens + span - 1) / span;
    if (tok_ctas > 32 * num_sms) tok_ctas = 32 * num_sms;
    return launch_dependent(tables_fill_kernel, (unsigned)(row_ctas + tok_ctas), kFillThreads, stream, p,
                            (int)row_ctas);
}

cudaError_t launch_trim_pages(const TablesParams &p, int num_sms, cudaStream_t stream) {
    // how many pages come back is not known here: by the rows' width, as if half of each did
    const bool fill = (int64_t)p.batch * p.max_blocks <= kInlineWork;
    cudaError_t e = plan<false>(p, fill, stream);
    if (e != cudaSuccess || fill) return e;
    int64_t grid = (p.batch + kFillThreads / 32 - 1) / (kFillThreads / 32);
    if (grid > 4 * num_sms) grid = 4 * num_sms;                 // far below 2^15, what the release's count holds
    return launch_dependent(tables_release_kernel, (unsigned)grid, kFillThreads, stream, p);
}

}  // namespace attn
