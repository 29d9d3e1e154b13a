// linear_attn.cu -- linear attention with a decay for each head:
//   S_t = e^g S_{t-1} + v_t k_t^T          (S [Dv, Dk], fp32)
//   o_t = scale * S_t q_t
// over packed sequences (a prompt) or one token per sequence (decode), with a
// cache of states.
#include <mutex>

#include "chunks.cuh"
#include "kernels.h"
#include "sequences.cuh"

namespace attn {
namespace {

__device__ __forceinline__ void linear_rows(const LinearParams &p, int b, int64_t &t0, int &n, bool report) {
    sequence_rows<SRC_LINEAR>(p, b, t0, n, report);
}

template <bool STEP>
__device__ __forceinline__ float *linear_state(const LinearParams &p, int b, int h, bool &from, bool report) {
    return sequence_state<SRC_LINEAR, STEP>(p, p.Hkv, b, h, from, report);
}

// log_decay of head h, at most 0: a positive or NaN value counts as 0 and is reported.
__device__ __forceinline__ float linear_log_decay(const LinearParams &p, int h, bool report) {
    const float g = __ldg(p.log_decay + h);
    if (report && !(g <= 0.f)) record_error(p.err, ERR_RANGE | SRC_LINEAR);
    return fminf(g, 0.f);
}

// ---------------------------------------------------------------------------
// One token per sequence: every state is read and written once, 8 D^2 bytes per
// sequence and KV head, which bounds it (HBM; 4 operations per 8 bytes).  A lane
// holds four neighbouring columns of a row, a warp 32 lanes / (D / 4) rows at a
// time, kDecodeRows loads ahead of anything that uses them (4 KB a warp); the
// row sums of a warp's rows are reduced together (9 shuffles for 8 rows).  256
// sequences, 32 heads of 128: 151 us in the kernel, 7.1 TB/s; a CTA per state, each row
// reduced by itself: 275 us.  One sequence: 5 us, a launch and three dependent loads.
// PACKED (packed sequences of at most one token): sequence b's row is cu[b], and a
// sequence without a token leaves its state as it was; its own instance, since the loads and tests
// cost 0.2 us of one sequence, 0.5 of 64 with 8 states each (10.2 -> 10.7 us).
// ---------------------------------------------------------------------------
constexpr int kDecodeRows = 8;        // loads in flight per lane
constexpr int kDecodeWarps = 4;

template <int D, bool PACKED>
__global__ void __launch_bounds__(kDecodeWarps * 32) linear_decode_kernel(const LinearParams p) {
    constexpr int LPR = D / 4;                          // lanes per row
    constexpr int RPL = 32 / LPR;                       // rows per load
    constexpr int ROWS = kDecodeRows * RPL;             // rows per warp
    constexpr int CTAS = D / (ROWS * kDecodeWarps);     // CTAs per state
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int unit = blockIdx.x / CTAS, b = unit / p.Hkv, h = unit - b * p.Hkv;
    const int row0 = ((blockIdx.x - unit * CTAS) * kDecodeWarps + warp) * ROWS + (lane / LPR) * kDecodeRows;
    const int col = (lane & (LPR - 1)) * 4;
    const bool report = h == 0 && threadIdx.x == 0;
    int64_t t = b;
    int n = 1;
    if (PACKED) linear_rows(p, b, t, n, report);
    bool from;
    float *state = linear_state<PACKED>(p, b, h, from, report && n > 0);
    if (PACKED && n == 0) return;
    float4 S[kDecodeRows];                              // rows row0 .. row0 + 7, columns col .. col + 3
#pragma unroll
    for (int i = 0; i < kDecodeRows; ++i) {
        S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (from) S[i] = __ldcs(reinterpret_cast<const float4 *>(state + (row0 + i) * D + col));
    }
    const uint2 kr = *reinterpret_cast<const uint2 *>(p.k + t * p.k_stride + h * D + col);
    const uint4 vr = *reinterpret_cast<const uint4 *>(p.v + t * p.v_stride + h * D + row0);
    const float a = expf(linear_log_decay(p, h, b == 0 && threadIdx.x == 0));
    const float k0 = __uint_as_float(kr.x << 16), k1 = __uint_as_float(kr.x & 0xFFFF0000u);
    const float k2 = __uint_as_float(kr.y << 16), k3 = __uint_as_float(kr.y & 0xFFFF0000u);
    const uint32_t vw[4] = {vr.x, vr.y, vr.z, vr.w};
#pragma unroll
    for (int i = 0; i < kDecodeRows; ++i) {
        const float v = __uint_as_float(i & 1 ? vw[i / 2] & 0xFFFF0000u : vw[i / 2] << 16);
        S[i].x = fmaf(v, k0, a * S[i].x);
        S[i].y = fmaf(v, k1, a * S[i].y);
        S[i].z = fmaf(v, k2, a * S[i].z);
        S[i].w = fmaf(v, k3, a * S[i].w);
        if (state) __stcs(reinterpret_cast<float4 *>(state + (row0 + i) * D + col), S[i]);
    }
    for (int g = 0; g < p.G; ++g) {
        const int hq = h * p.G + g;
        const uint2 qr = *reinterpret_cast<const uint2 *>(p.q + t * p.q_stride + (int64_t)hq * D + col);
        const float q0 = __uint_as_float(qr.x << 16), q1 = __uint_as_float(qr.x & 0xFFFF0000u);
        const float q2 = __uint_as_float(qr.y << 16), q3 = __uint_as_float(qr.y & 0xFFFF0000u);
        float o[kDecodeRows];
#pragma unroll
        for (int i = 0; i < kDecodeRows; ++i)
            o[i] = fmaf(S[i].x, q0, fmaf(S[i].y, q1, fmaf(S[i].z, q2, S[i].w * q3)));
        // each step halves the rows a lane carries: the last bits of the lane number pick the row
        int w = LPR / 2;
#pragma unroll
        for (int n = kDecodeRows / 2; n > 0; n /= 2, w /= 2) {
            const bool up = lane & w;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float give = up ? o[i] : o[i + n], keep = up ? o[i + n] : o[i];
                o[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
            }
        }
#pragma unroll
        for (; w > 0; w /= 2) o[0] += __shfl_xor_sync(0xffffffffu, o[0], w);
        // row bits: 4, 2, 1 from lane bits LPR / 2, LPR / 4, LPR / 8
        const int row = (lane & (LPR - 1)) / (LPR / 8);
        if ((lane & (LPR / 8 - 1)) == 0)
            p.out[t * p.out_stride + (int64_t)hq * D + row0 + row] = __float2bfloat16_rn(o[0] * p.scale);
    }
}

cudaError_t launch_decode_kernel(const LinearParams &p, cudaStream_t stream) {
    const int64_t states = (int64_t)p.batch * p.Hkv;
    auto *kernel = p.D == 128 ? p.cu ? linear_decode_kernel<128, true> : linear_decode_kernel<128, false>
                              : p.cu ? linear_decode_kernel<64, true> : linear_decode_kernel<64, false>;
    main_kernel_event_before(stream);
    kernel<<<(unsigned)(p.D == 128 ? states * 4 : states), kDecodeWarps * 32, 0, stream>>>(p);
    main_kernel_event_after(stream);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Prompts, in chunks of 64 tokens on the tensor cores.
//
// With n tokens in a chunk, i and j counting them from 0 and S_0 the state before:
//   o_i = scale * sum_{j <= i} e^{(i-j) g} (q_i . k_j) v_j + scale * e^{(i+1) g} S_0 q_i
//   S_n = e^{n g} S_0 + sum_j e^{(n-1-j) g} v_j k_j^T
// Every exponent is <= 0: nothing overflows whatever the decay.
//
// As matrices with the value dimension in the 128 TMEM lanes (a product with M = 64
// takes as long as one with M = 128, and S and w V are then A operands read from TMEM):
//   QK     [i, j]   = Q K^T                 shared x shared
//   QS     [dv, i]  = S_0 Q^T               TMEM (S_0 as two bf16 parts) x shared
//   PV     [dv, i]  = V^T P^T               shared (V as loaded, exact) x shared (P as two bf16 parts)
//   KV     [dv, dk] = (w_j V)^T K           TMEM (two bf16 parts) and shared (the third) x shared
// with P = scale * e^{(i-j) g} QK (masked) and w_j = e^{(n-1-j) g}.
//
// Precision.  q, k and v are bf16 and exact.  P and S_0 only reach the bf16 output:
// two parts leave 2^-16 of each term, against the output's own 2^-8.  The state is
// fp32 and returned: w_j v_j in three parts is the fp32 product (2^-24); one
// or two parts would leave 1.7e-3 or 2.8e-6 of it.  S itself stays in fp32 registers;
// e^{64 g} multiplies it as hi + lo, so its rounding does not add up over chunks.
//
// Bound by what the chunks of a sequence wait for, KV -> S -> QS -> output rows, and by the shared
// memory that all roles and the tensor core's operands share: the tensor core is
// busy half of the time.  Per chunk of head_dim 128: KV 12 steps of 16 tokens (N = 128, 66 clocks
// each), QS 16 (N = 64, 33), PV and QK 8 each (both operands shared, 50): 2,100 clocks of the 3,500
// that a chunk takes; HBM's 64 KB would take 2,700 of them.
// So everything else is off the warps that issue, in roles that run side by side, each a
// chunk or less apart.
//
// Roles (32 warps, one CTA per SM):
//   0..7    V preparation: w V, three parts, transposed into TMEM and shared memory
//   8..23   state: fp32 registers; adds KV, then (the eight that see tokens' lanes) P of the next chunk, writes
//           S_0's two parts
//   24..27  output rows
//   28, 29  issue the loads; write the units' tables
//   30, 31  issue the MMAs: KV, QS, PV; QK (a chunk ahead)
// What counted, each measured on 16 prompts of a step (32 heads of 128): roles side by side
// instead of in turn 634 -> 387 us; PV's A straight from the loaded V, waits off the
// issuing threads 387 -> 324; operands warp-uniform and one code site per role's step, 64 -> 38 KB
// of code (the instruction cache is shared by all roles) 324 -> 294; fewer barriers 294 -> 280;
// P by the state's warps in the time between KV and QS, its factors loaded
// without branches 280 -> 266; waits that rarely read the timer 266 -> 261; output tiles as
// one bulk store each 261 -> 249; mixed-precision remainders 249 -> 243.  One CTA per SM that goes over
// its units, the next one's tables and copies under way while one ends: 96 short sequences
// 70 -> 47.5 us.
// ---------------------------------------------------------------------------

constexpr int LC = 64;                       // tokens of a chunk
constexpr int kChunkThreads = 1024;
constexpr int kChunkPanel = LC * 128;        // 64 rows x 128 bytes
constexpr uint32_t TC_S = 0;                 // TMEM columns: QK
constexpr uint32_t TC_INTRA = 64;            // PV
constexpr uint32_t TC_INTER = 128;           // QS
constexpr uint32_t TC_KV = 192;              // KV
constexpr uint32_t TC_STATE = 320;           // S_0: hi, lo (D / 2 of 64 columns each)
constexpr uint32_t TC_W = 448;               // (w V)^T: hi, mid (32 columns each)
constexpr int kDecayRow = kLinearDecayRow;   // floats of a head's decay table: e^{m g} for m = 0..64, the part
                                             // below fp32 of each, then e^{seg_len g} in two parts
constexpr int kBuckets = 256;

// A unit as its roles read it, behind its tables.
struct UnitInfo {
    int count;                        // tokens; 0: there is no such unit
    int t0, h, hk, row, slot, from, last;
    float a_full, a_full_lo, a_last, a_last_lo;   // e^{n g} over a full chunk and over the last one, two parts each
};

template <int D>
struct ChunkSmem {
    static constexpr int kPanels = D / 64;
    static constexpr int kQkPanel = 2 * kChunkPanel;             // 64 Q rows, then 64 K rows
    static constexpr int kVOff = kPanels * kQkPanel;
    static constexpr int kStageBytes = kVOff + kPanels * kChunkPanel;
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kPOff = kStages * kStageBytes;        // two chunks' P: hi, lo
    static constexpr int kLoOff = kPOff + 4 * kChunkPanel;       // the third part of w V, laid out like V
    static constexpr int kOutOff = kLoOff + kPanels * kChunkPanel;      // per output warp [64 tokens][32 dv] bf16
    static constexpr int kTabOff = kOutOff + 4 * LC * 64;
    // two units' tables: scale e^{m g}, zeros for m = -64..-1, then m = 0..63; m = 1..64; w of a full chunk, of
    // the last chunk.  Then the first non-finite token per dv, four chunks
    static constexpr int kTabFloats = 5 * LC + 16;               // ... and the unit itself (UnitInfo)
    static constexpr int kTabBytes = 2 * kTabFloats * 4 + 4 * 128 * 4;
    static constexpr int kBarOff = kTabOff + kTabBytes;
    static constexpr int kNumBars = 2 * kStages + 15;
    static constexpr int kBytes = kBarOff + kNumBars * 8 + 16 + 1024 /* alignment slack */;
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

// Registers of the calling warpgroup.  The kernel is launched with 64 a thread; the eight
// warpgroups' shares add up to that: V 2, state 4, output rows 1 (which keep theirs), the others 1.
constexpr int kVRegs = 56, kStateRegs = 72, kOutRegs = 64, kRestRegs = 48;
static_assert(2 * kVRegs + 4 * kStateRegs + kOutRegs + kRestRegs == 8 * 64, "register shares");

// a load that stays a load of its own: the compiler would put one under a condition behind a branch
__device__ __forceinline__ float lds_f32(const float *p) {
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(smem_u32(p)));
    return x;
}

// 8 keys of token i's row of P -> 16-byte chunk `ch` of both parts
__device__ __forceinline__ void put_p(uint8_t *ph, int i, int ch, float (&x)[8]) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        hi[k] = take_bf16(x[2 * k], x[2 * k + 1]);
        lo[k] = pack_bf16x2(x[2 * k], x[2 * k + 1]);
    }
    const uint32_t at = sw128_off(i, ch);
    *reinterpret_cast<uint4 *>(ph + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4 *>(ph + kChunkPanel + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

// A unit's entry in the work list, as the plan writes it.
struct alignas(16) ChunkUnit {
    int t0, n;          // first token, tokens
    int row;            // its start in the workspace's states (-1: none)
    int last;           // holds the sequence's last token
    int slot, from;     // state slot (-1: none), whether the sequence starts from it
    int head;           // first segment: the sequence's segments, else 0
    int more;           // has a successor
};
static_assert(sizeof(ChunkUnit) == kLinearUnitBytes, "workspace layout");

// The work list: a unit is a sequence, or a segment of seg_len tokens of a longer
// one; units with the most chunks come first.  CTA 0 writes the list, the others
// the heads' decay tables.
__global__ void __launch_bounds__(1024) linear_plan_kernel(const LinearParams p) {
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x;
    if (blockIdx.x > 0) {
        const int h = (blockIdx.x - 1) * 8 + (tid >> 7), m = tid & 127;
        if (h >= p.Hkv || m > LC + 1) return;
        const float x = linear_log_decay(p, h, m == 0) * (float)(m <= LC ? m : p.seg_len);
        // near 1, where a state is multiplied many times before it fades, as two parts that are
        // right to 2^-23 of x; elsewhere the fp32 value. Not 0 * -inf.
        float hi = 1.f, lo = 0.f;
        if (m > 0 && x < -0.3f) {
            hi = expf(x);
        } else if (m > 0) {
            const float y = expm1f(x);
            hi = 1.f + y;
            lo = y - (hi - 1.f);
        }
        float *row = p.decay + (int64_t)h * kDecayRow;
        if (m <= LC) {
            row[m] = hi;
            row[LC + 1 + m] = lo;
        } else {
            row[2 * LC + 2] = hi;
            row[2 * LC + 3] = lo;
        }
        return;
    }
    __shared__ int count[kBuckets], rows_s;
    for (int i = tid; i < kBuckets; i += 1024) count[i] = 0;
    if (tid == 0) rows_s = 0;
    __syncthreads();
    const int most = max(1, min(p.seg_len, p.max_seqlen));
    auto bucket = [&](int tokens) { return kBuckets - 1 - (int)((int64_t)tokens * (kBuckets - 1) / most); };
    for (int pass = 0; pass < 2; ++pass) {
        for (int b = tid; b < p.batch; b += 1024) {
            int64_t t0;
            int n;
            linear_rows(p, b, t0, n, pass == 0);
            if (n == 0) continue;
            const int segs = (n + p.seg_len - 1) / p.seg_len, tail = n - (segs - 1) * p.seg_len;
            if (pass == 0) {
                if (segs > 1) atomicAdd(&count[bucket(p.seg_len)], segs - 1);
                atomicAdd(&count[bucket(tail)], 1);
            } else {
                bool from;
                const float *state = linear_state<true>(p, b, 0, from, true);
                const int slot = state ? __ldg(p.slots + b) : -1;
                // a state of its own for every segment's start; heads that share a state
                // read a copy, since one of them writes the new one
                const bool rows = segs > 1 || (from && p.G > 1);
                int row = rows ? atomicAdd(&rows_s, segs) : -1;
                // offsets that overlap can ask for more than the workspace was sized for
                bool fits = row + segs <= p.state_rows;
                if (!fits) row = -1;
                for (int i = 0; i < segs; ++i) {
                    const int at = atomicAdd(&count[bucket(i < segs - 1 ? p.seg_len : tail)], 1);
                    const bool end = i == segs - 1;
                    if (at < p.max_units)
                        reinterpret_cast<ChunkUnit *>(p.units)[at] =
                            ChunkUnit{(int)t0 + i * p.seg_len, end ? tail : p.seg_len, row < 0 ? -1 : row + i, end,
                                      slot, from, i == 0 ? segs : 0, !end};
                    else fits = false;
                }
                if (!fits) record_error(p.err, ERR_INDEX | SRC_LINEAR);
            }
        }
        __syncthreads();
        if (pass == 0 && tid < 32) {
            // counts -> first places
            int base = 0;
            for (int i = 0; i < kBuckets; i += 32) {
                const int c = count[i + tid];
                int inc = c;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, inc, o);
                    if (tid >= o) inc += v;
                }
                count[i + tid] = base + inc - c;
                base += __shfl_sync(0xffffffffu, inc, 31);
            }
            if (tid == 0) *p.unit_count = min(base, p.max_units);
        }
        __syncthreads();
    }
}

// The states at the starts of a sequence's segments, in place of the segments'
// own sums that the state-only pass left there:
//   start_0 = the cached state or 0,  start_{s+1} = e^{seg_len g} start_s + own_s
__global__ void __launch_bounds__(256) linear_scan_kernel(const LinearParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if ((int)blockIdx.x >= *p.unit_count) return;
    const ChunkUnit e = reinterpret_cast<const ChunkUnit *>(p.units)[blockIdx.x];
    if (e.head == 0 || e.row < 0) return;
    const int h = blockIdx.y, D2 = p.D * p.D;
    const float *state = p.state + ((int64_t)e.slot * p.Hkv + h) * D2;   // read only if e.from
    const float *t = p.decay + (int64_t)h * kDecayRow + 2 * LC + 2;
    const float hi = t[0], lo = t[1];
    const int x = (blockIdx.z * 256 + threadIdx.x) * 4;
    if (x >= D2) return;
    float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
    if (e.from) run = *reinterpret_cast<const float4 *>(state + x);
    float *at = p.states + ((int64_t)e.row * p.Hkv + h) * D2 + x;
    const int64_t step = (int64_t)p.Hkv * D2;
    constexpr int kAhead = 8;   // loads in flight per thread: the sums are read before starts replace them
    for (int s0 = 0; s0 < e.head; s0 += kAhead) {
        float4 own[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (s0 + k + 1 < e.head) own[k] = *reinterpret_cast<const float4 *>(at + (s0 + k) * step);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (s0 + k >= e.head) break;
            *reinterpret_cast<float4 *>(at + (s0 + k) * step) = run;
            run.x = fmaf(hi, run.x, fmaf(lo, run.x, own[k].x));
            run.y = fmaf(hi, run.y, fmaf(lo, run.y, own[k].y));
            run.z = fmaf(hi, run.z, fmaf(lo, run.z, own[k].z));
            run.w = fmaf(hi, run.w, fmaf(lo, run.w, own[k].w));
        }
    }
}

// LOCAL: the state-only pass over the segments that have a successor: their own
// sums (from a zero state) go to the workspace.
template <int D, bool LOCAL>
__global__ void __launch_bounds__(kChunkThreads, 1)
    linear_chunk_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap omap,
                        const LinearParams p) {
    using S = ChunkSmem<D>;
    constexpr int ST = S::kStages, PAN = S::kPanels;
    extern __shared__ __align__(1024) uint8_t lsmem_raw[];
    // values from lane 0 are warp-uniform to the compiler, and so is what is computed from them
    auto uni = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    const int warp = uni(threadIdx.x >> 5), lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int heads = LOCAL ? p.Hkv : p.Hq;
    // The CTA's units: places blockIdx.x, 2 gridDim.x - 1 - blockIdx.x, 2 gridDim.x + blockIdx.x, ... of the
    // list (longest first), back and forth so that the CTAs' sums come out alike.  Warp 29 writes each
    // unit's tables, a unit ahead; the roles go by them.  Chunks are counted on from unit to unit (g), as
    // are the barriers' phases.
    const ChunkUnit *units = reinterpret_cast<const ChunkUnit *>(p.units);
    const int units_n = uni(*p.unit_count), total = units_n * heads, G = gridDim.x;
    auto place = [&](int k) { return k * G + ((k & 1) ? G - 1 - (int)blockIdx.x : (int)blockIdx.x); };
    if (place(0) >= total) return;
    auto chunks_of = [](int n) { return (n + LC - 1) / LC; };

    const uint32_t smb = (smem_u32(lsmem_raw) + 1023u) & ~1023u;          // shared-memory address, for descriptors
    uint8_t *sm = lsmem_raw + (smb - smem_u32(lsmem_raw));
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + S::kBarOff);
    uint64_t *full = bars, *empty = bars + ST;
    uint64_t *kv_go = bars + 2 * ST;         // [2], by chunk: (w V)^T is in place (and V's tail and non-finite entries
    //   are zeroed), the KV before has been read
    uint64_t *w_free = kv_go + 2;            // [2], by chunk: KV has read (w V)^T
    uint64_t *kv_ready = kv_go + 4;          // KV done
    uint64_t *qs_go = kv_go + 5;             // S_0 is in TMEM, P in shared memory, the chunk before has been read
    uint64_t *qs_done = kv_go + 6;           // QS has read S_0
    uint64_t *s_ready = kv_go + 7;           // QK done
    uint64_t *p_ready = kv_go + 8;           // P in shared memory, QK's columns free
    uint64_t *o_ready = kv_go + 9;           // QS and PV done
    uint64_t *drain = kv_go + 10;            // every MMA done
    uint64_t *tab_full = kv_go + 11;         // [2]: a unit's tables are written
    uint64_t *tab_free = kv_go + 13;         // [2]: ... and read for the last time
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + S::kNumBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float *tables = reinterpret_cast<float *>(sm + S::kTabOff);
    int *bad_at = reinterpret_cast<int *>(tables + 2 * S::kTabFloats);   // [4][128]
    // of unit number m: scale e^{j g} (zeros in front), scale e^{(j + 1) g}, w of a full and of the last chunk
    auto tab_of = [&](int m) { return tables + (m & 1) * S::kTabFloats + LC; };
    auto info_of = [&](int m) { return reinterpret_cast<UnitInfo *>(tables + (m & 1) * S::kTabFloats + 5 * LC); };

    // the loader sets the barriers up; its copies begin when everyone is past the set-up
    if (warp == 28 && lane == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1 + 8);     // the MMAs, the V warps
        }
        mbar_init(&kv_go[0], 8 + 16);        // V, state
        mbar_init(&kv_go[1], 8 + 16);
        mbar_init(&w_free[0], 1);
        mbar_init(&w_free[1], 1);
        mbar_init(kv_ready, 1);
        mbar_init(qs_go, 16 + 4);            // state, output
        mbar_init(qs_done, 1);
        mbar_init(s_ready, 1);
        mbar_init(p_ready, 8);               // the state warps of the lanes with tokens
        mbar_init(o_ready, 1);
        mbar_init(drain, 2);                 // each MMA thread
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tab_full[i], 1);
            mbar_init(&tab_free[i], LOCAL ? 8 + 16 + 1 : 30);   // every warp that reads them
        }
        abort_flag[0] = abort_flag[1] = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (!LOCAL && warp == 29) {
        // tokens 0..31 see no key behind 31: those halves of their rows of P stay zero
#pragma unroll 1
        for (int k = 0; k < 16; ++k)
            *reinterpret_cast<uint4 *>(sm + S::kPOff + (k >> 2) * kChunkPanel + sw128_off(lane, 4 + (k & 3))) =
                make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    if (threadIdx.x >= 64 && threadIdx.x < 64 + 2 * LC)
        tables[(threadIdx.x - 64) / LC * S::kTabFloats + (threadIdx.x & (LC - 1))] = 0.f;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uni((int)*tmem_slot);
    // Where a chunk's w V goes: the state-only pass has room for two chunks of it (32,768 tokens, 16 heads:
    // that pass 69 -> 60 us)
    constexpr int kWBufs = LOCAL ? 2 : 1;
    auto w_at = [](int gc) { return LOCAL && (gc & 1) ? TC_STATE : TC_W; };
    auto lo_at = [](int gc) { return LOCAL && (gc & 1) ? S::kPOff : S::kLoOff; };
    // waits for what the hardware finishes by itself run to the limit: their flag is their own
    volatile int &never = *(abort_flag + 1);
    // a warp's wait: every lane gets the same answer
    auto wait = [&](uint64_t *bar, int phase) {
        return __all_sync(0xffffffffu, chunk_wait(bar, (uint32_t)phase & 1u, abort_flag)) != 0;
    };

    if (warp < 8) {
        // ============================================================ V preparation: a warp per 16 value dimensions
        // In 8x8 fragments: ldmatrix transposes 8 tokens x 8 dv, a thread then holds two neighbouring tokens of
        // one dv, which is a 32-bit column of the A operand.
        fewer_regs<kVRegs>();
        const int grp = warp & 3, hl = warp >> 2;
        const uint32_t lane_base = tmem + ((uint32_t)(grp * 32 + hl * 16) << 16);
        const int q2 = (lane & 3) * 2;           // its tokens: 8 g + q2, + 1
        // head_dim 64: lane groups 2 and 3 repeat 0 and 1 (lanes 64..127 reach no output)
        const int d8 = ((grp * 32) & (D - 1)) / 8 + 2 * hl + ((lane >> 3) & 1);
        const uint32_t frag = S::kVOff + (d8 >> 3) * kChunkPanel + sw128_off((lane >> 4) * 8 + (lane & 7), d8 & 7);
        int g = 0;                               // chunks before unit m
        bool ok = true;
#pragma unroll 1
        for (int m = 0;; ++m) {
            if (!(ok = wait(&tab_full[m & 1], m >> 1))) break;
            const UnitInfo *u = info_of(m);
            const int count = uni(u->count), chunks = chunks_of(count);
            if (count == 0) break;
#pragma unroll 1
            for (int c = 0; c < chunks && ok; ++c) {
                const int gc = g + c, s = gc % ST, n = min(LC, count - c * LC);
                const float *w = tab_of(m) + (c + 1 < chunks ? 2 : 3) * LC + q2;
                uint8_t *stage = sm + s * S::kStageBytes;
                if (!(ok = wait(&full[s], gc / ST))) break;
                if (n < LC) {
                    // rows behind the sequence's end are zeroed (a weight of 0 would not cancel a NaN there)
                    const int per = (LC - n) * 8;
                    for (int x = threadIdx.x; x < per * 2 * PAN; x += 256) {
                        const int tile = x / per, r = x - tile * per, pan = tile >> 1;
                        uint8_t *at = tile & 1 ? stage + S::kVOff + pan * kChunkPanel
                                               : stage + pan * S::kQkPanel + kChunkPanel;
                        *reinterpret_cast<uint4 *>(at + n * 128 + r * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                // in two steps of 32 tokens; raw[2 g + x]: dv 8 x + lane / 4, tokens 32 step + 8 g + q2, + 1
                float zero0 = 0.f, zero1 = 0.f;             // NaN once a non-finite v went by
#pragma unroll 1
                for (int step = 0; step < 2; ++step) {
                    uint32_t raw[8], hi[8], mid[8], lo[8];
                    const uint32_t at = smem_u32(stage) + frag + step * 4096;
                    ldsm_x4_t(at, raw[0], raw[1], raw[2], raw[3]);
                    ldsm_x4_t(at + 2048, raw[4], raw[5], raw[6], raw[7]);
                    if (n < LC) {                           // (another warp may still be zeroing these rows)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int j = step * 32 + (i >> 1) * 8 + q2;
                            raw[i] &= (j < n ? 0xFFFFu : 0u) | (j + 1 < n ? 0xFFFF0000u : 0u);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 wj = *reinterpret_cast<const float2 *>(w + step * 32 + (i >> 1) * 8);
                        const float v0 = __uint_as_float(raw[i] << 16), v1 = __uint_as_float(raw[i] & 0xFFFF0000u);
                        float x0, x1;
                        if (!LOCAL) fma2(zero0, zero1, v0, v1, 0.f, 0.f, zero0, zero1);
                        fma2(x0, x1, v0, v1, wj.x, wj.y, 0.f, 0.f);
                        hi[i] = take_bf16(x0, x1);
                        mid[i] = take_bf16(x0, x1);
                        lo[i] = pack_bf16x2(x0, x1);
                    }
                    if (step == 0 && gc >= kWBufs) {
                        ok = wait(&w_free[(gc - kWBufs) & 1], (gc - kWBufs) >> 1);
                        tc_fence_after();
                    }
                    if (!ok) break;
                    tmem_st_16x128b_x4(lane_base + w_at(gc) + step * 16, hi);
                    tmem_st_16x128b_x4(lane_base + w_at(gc) + 32 + step * 16, mid);
                    if (grp * 32 < D) {
                        const uint32_t to = smem_u32(sm + lo_at(gc)) + (frag - S::kVOff) + step * 4096;
                        stsm_x4_t(to, lo[0], lo[1], lo[2], lo[3]);
                        stsm_x4_t(to + 2048, lo[4], lo[5], lo[6], lo[7]);
                    }
                }
                if (!ok) break;
                fence_proxy_async_smem();
                if (!LOCAL) {
                    const bool any_bad = __any_sync(0xffffffffu, !(zero0 + zero1 == 0.f));
                    if (any_bad) {
                        // a non-finite v: in PV it would reach the chunk's earlier tokens (0 * NaN), so it is
                        // zeroed there and the output warps write NaN from its token on
#pragma unroll 1
                        for (int r = 0; r < 2; ++r) {       // two rows of the fragment: dv 8 r + lane / 4
                            const int row = grp * 32 + hl * 16 + 8 * r + (lane >> 2);
                            int first = LC;
                            if (row < D)
                                for (int j = q2; j < n; j += (j & 1) ? 7 : 1) {
                                uint16_t *v = reinterpret_cast<uint16_t *>(
                                    stage + S::kVOff + (row >> 6) * kChunkPanel + sw128_off(j, (row & 63) >> 3) +
                                    (row & 7) * 2);
                                if ((*v & 0x7F80u) == 0x7F80u) {
                                    *v = 0;
                                    first = min(first, j);
                                }
                            }
                            first = min(first, __shfl_xor_sync(0xffffffffu, first, 1));
                            first = min(first, __shfl_xor_sync(0xffffffffu, first, 2));
                            if ((lane & 3) == 0 && row < D) bad_at[(gc & 3) * 128 + row] = first;
                        }
                        fence_proxy_async_smem();
                    } else if (lane < 16) {
                        bad_at[(gc & 3) * 128 + grp * 32 + hl * 16 + lane] = LC;
                    }
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&kv_go[gc & 1]);
                    mbar_arrive(&empty[s]);
                }
            }
            if (!ok) break;
            if (lane == 0) mbar_arrive(&tab_free[m & 1]);
            g += chunks;
        }
    } else if (warp < 24) {
        // ============================================================ state: thread = value dimension, a quarter of dk
        more_regs<kStateRegs>();
        const int grp = warp & 3, part = (warp - 8) >> 2, dv = grp * 32 + lane;
        const bool real = grp * 32 < D;      // warp-uniform
        const uint32_t lane_base = tmem + ((uint32_t)(grp * 32) << 16);
        constexpr int N = D / 4;             // columns per thread
        float St[N];
        auto publish = [&]() {               // S_0's two parts to TMEM
#pragma unroll
            for (int i = 0; i < N; i += 16) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    float x0 = St[i + 2 * k], x1 = St[i + 2 * k + 1];
                    hi[k] = take_bf16(x0, x1);
                    lo[k] = pack_bf16x2(x0, x1);
                }
                tmem_st8(lane_base + TC_STATE + (part * N + i) / 2, hi);
                tmem_st8(lane_base + TC_STATE + 64 + (part * N + i) / 2, lo);
            }
            tc_wait_st();
            tc_fence_before();
        };
        int g = 0;                               // chunks before unit m
        bool ok = true;
#pragma unroll 1
        for (int m = 0;; ++m) {
            if (!(ok = wait(&tab_full[m & 1], m >> 1))) break;
            const UnitInfo *u = info_of(m);
            const int count = uni(u->count), chunks = chunks_of(count);
            if (count == 0) break;
            float *state = u->slot < 0 ? nullptr : p.state + ((int64_t)u->slot * p.Hkv + u->hk) * D * D;
            float *own = u->row < 0 ? nullptr : p.states + ((int64_t)u->row * p.Hkv + u->hk) * D * D;
            const float *src = LOCAL ? nullptr : own ? own : u->from ? state : nullptr;
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (src && real) x = *reinterpret_cast<const float4 *>(src + dv * D + part * N + i);
                St[i] = x.x, St[i + 1] = x.y, St[i + 2] = x.z, St[i + 3] = x.w;
            }
#pragma unroll 1
            for (int c = -1; c < chunks; ++c) {
                const int gc = g + c;
                if (c >= 0) {
                    const bool mid = c + 1 < chunks;
                    const float a = mid ? u->a_full : u->a_last, a_lo = mid ? u->a_full_lo : u->a_last_lo;
                    if (!(ok = wait(kv_ready, gc))) break;
                    tc_fence_after();
                    if (real) {
#pragma unroll
                        for (int i = 0; i < N; i += 16) {
                            uint32_t kv[16];
                            tmem_ld16(lane_base + TC_KV + part * N + i, kv);
                            tc_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; k += 2) {
                                float x0, x1;
                                fma2(x0, x1, a_lo, a_lo, St[i + k], St[i + k + 1], __uint_as_float(kv[k]),
                                     __uint_as_float(kv[k + 1]));
                                fma2(St[i + k], St[i + k + 1], a, a, St[i + k], St[i + k + 1], x0, x1);
                            }
                        }
                        tc_fence_before();
                    }
                }
                __syncwarp();
                const bool first_or_read = c >= 0 || m == 0;
                if (lane == 0 && first_or_read) mbar_arrive(&kv_go[(gc + 1) & 1]);   // before the first: nothing to read
                if (!LOCAL && grp < 2 && first_or_read) {
                    // P of the next chunk: lane = token (lanes 64..127 hold none), 8 keys at a time, in turn among
                    // the warps of a lane group; tokens 0..31 see no key behind 31
                    const int of = c + 1 < chunks ? m : m + 1;        // its unit
                    if (!(ok = wait(&tab_full[of & 1], of >> 1))) break;
                    if (uni(info_of(of)->count) > 0) {
                        if (!(ok = wait(s_ready, gc + 1))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int k = part; k < 4 + 4 * grp; k += 4) {
                            const int d = dv - k * 8;
                            const float *e = tab_of(of) + d;
                            float f[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) f[j] = lds_f32(e - j);
                            uint32_t s[8];
                            float x[8];
                            tmem_ld8(lane_base + TC_S + k * 8, s);
                            tc_wait_ld();
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                // masked by choice, not by the table's zeros, which would keep a NaN
                                x[j] = j <= d ? __uint_as_float(s[j]) : 0.f;
#pragma unroll
                            for (int j = 0; j < 8; j += 2)
                                fma2(x[j], x[j + 1], x[j], x[j + 1], f[j], f[j + 1], 0.f, 0.f);
                            put_p(sm + S::kPOff + ((gc + 1) & 1) * 2 * kChunkPanel, dv, k, x);
                        }
                        fence_proxy_async_smem();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(p_ready);
                    }
                }
                if (!LOCAL && c + 1 < chunks) {
                    if (gc >= 0 && !(ok = wait(qs_done, gc))) break;
                    tc_fence_after();
                    if (real) publish();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(qs_go);
                }
            }
            if (!ok) break;
            float *dst = LOCAL ? own : u->last ? state : nullptr;
            __syncwarp();
            if (lane == 0) mbar_arrive(&tab_free[m & 1]);
            if (real && dst) {
#pragma unroll
                for (int i = 0; i < N; i += 4)
                    *reinterpret_cast<float4 *>(dst + dv * D + part * N + i) =
                        make_float4(St[i], St[i + 1], St[i + 2], St[i + 3]);
            }
            g += chunks;
        }
    } else if (warp < 28) {
        // ============================================================ output rows: a warp per 32 value dimensions
        // In 8x8 fragments (thread: two neighbouring tokens of one dv), transposed by stmatrix into the warp's
        // own [64 tokens][32 dv] tile, 16-byte chunks swizzled by token pair.
        if (!LOCAL) {
            const int grp = warp & 3, q2 = (lane & 3) * 2;
            const bool real = grp * 32 < D;
            const uint32_t lane_base = tmem + ((uint32_t)(grp * 32) << 16);
            uint8_t *stg = sm + S::kOutOff + grp * LC * 64;
            // stmatrix row address: token (lane / 16) * 8 + lane % 8 of its group, dv chunk lane / 8 % 2
            const int row0 = (lane >> 4) * 8 + (lane & 7), ch0 = (lane >> 3) & 1, sw = (row0 >> 1) & 3;
            const uint32_t stg_at = smem_u32(stg) + row0 * 64;
            if (lane == 0) mbar_arrive(qs_go);           // nothing to be read yet
            int g = 0;                               // chunks before unit m
            bool ok = true;
#pragma unroll 1
            for (int m = 0;; ++m) {
                if (!(ok = wait(&tab_full[m & 1], m >> 1))) break;
                const UnitInfo *u = info_of(m);
                const int count = uni(u->count), chunks = chunks_of(count);
                if (count == 0) break;
                const int t0 = u->t0, h = u->h;
#pragma unroll 1
                for (int c = 0; c < chunks; ++c) {
                    const int gc = g + c, n = min(LC, count - c * LC);
                    if (!(ok = wait(o_ready, gc))) break;
                    tc_fence_after();
                    if (!real) {
                        if (lane == 0) mbar_arrive(qs_go);
                        continue;
                    }
                    if (lane == 0) bulk_wait_read();             // the tile's last store
                    __syncwarp();
                    const int *bad_row = bad_at + (gc & 3) * 128 + grp * 32;
                    const bool any_bad = __any_sync(0xffffffffu, bad_row[lane] < LC);
#pragma unroll 1
                    for (int part = 0; part < 4; ++part) {      // 16 dv, 32 tokens
                        const int hl = part >> 1, g0 = (part & 1) * 4;
                        const uint32_t at = lane_base + ((uint32_t)hl << 20) + g0 * 8;
                        uint32_t x[16], y[16], r[8];
                        tmem_ld_16x256b_x4(at + TC_INTRA, x);
                        tmem_ld_16x256b_x4(at + TC_INTER, y);
                        const float *e = tab_of(m) + LC + g0 * 8 + q2;
                        tc_wait_ld();
                        if (part == 3) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(qs_go);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {           // tokens 8 (g0 + i / 2) + q2, + 1; dv + 8 (i % 2)
                            const float2 f = *reinterpret_cast<const float2 *>(e + (i / 2) * 8);
                            float o0, o1;
                            fma2(o0, o1, f.x, f.y, __uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1]),
                                 __uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
                            r[i] = pack_bf16x2(o0, o1);
                        }
                        const uint32_t to = stg_at + (uint32_t)(g0 * 512) + (((hl * 2 + ch0) ^ sw) << 4);
                        stsm_x4_t(to, r[0], r[1], r[2], r[3]);
                        stsm_x4_t(to + 1024, r[4], r[5], r[6], r[7]);
                    }
                    __syncwarp();
                    if (any_bad) {
                        // NaN from a dv's first non-finite token on
                        const int first = bad_row[lane];
                        for (int t = first; t < LC; ++t)
                            *reinterpret_cast<uint16_t *>(stg + t * 64 + (((lane >> 3) ^ ((t >> 1) & 3)) << 4) +
                                                          (lane & 7) * 2) =
                                0x7FC0;
                    }
                    __syncwarp();
                    if (n == LC) {
                        // one store of the tile; its swizzle is the copy engine's for rows of 64 bytes
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            tma_store_3d(&omap, stg, grp * 32, h, t0 + c * LC);
                            bulk_commit();
                        }
                    } else {
                        // rows behind the sequence stay as they are
                        __nv_bfloat16 *out = p.out + (t0 + (int64_t)c * LC) * p.out_stride + (int64_t)h * D + grp * 32;
#pragma unroll 1
                        for (int t = lane >> 2; t < n; t += 8)
                            *reinterpret_cast<uint4 *>(out + t * p.out_stride + (lane & 3) * 8) =
                                *reinterpret_cast<const uint4 *>(stg + t * 64 + (((lane & 3) ^ ((t >> 1) & 3)) << 4));
                        __syncwarp();
                    }
                }
                if (!ok) break;
                if (lane == 0) mbar_arrive(&tab_free[m & 1]);
                g += chunks;
            }
            if (lane == 0) bulk_wait_all();
            __syncwarp();
        }
    } else {
        fewer_regs<kRestRegs>();
        if (warp < 30) {
            // ============================================================ loads (warp 28), the units' tables (warp 29)
            const int half = warp - 28;
            // Both walk the CTA's places: `at` and `h` are the next one's unit and head, without a division
            const int up = 2 * (G - 1 - (int)blockIdx.x) + 1, down = 2 * (int)blockIdx.x + 1;   // to the next place
            // x / y of x < 2^18: off by less than 2^-20 of itself, and half a step away from the next integer
            auto quotient = [](int x, float inv) { return (int)(((float)x + 0.5f) * inv); };
            const float inv_heads = __fdividef(1.f, (float)heads), inv_g = __fdividef(1.f, (float)p.G);
            const int up_q = uni(quotient(up, inv_heads)), up_r = up - up_q * heads;
            const int down_q = uni(quotient(down, inv_heads)), down_r = down - down_q * heads;
            int k = 0, at = uni(quotient(blockIdx.x, inv_heads)), h = blockIdx.x - at * heads;
            auto step = [&]() {
                at += k & 1 ? down_q : up_q;
                h += k & 1 ? down_r : up_r;
                if (h >= heads) h -= heads, ++at;
                ++k;
            };
            int loaded = 0, left = 0, row = 0, load_h = 0;   // the loader: chunks so far, the unit it is in
            // the next chunk's copies, once its stage is free (lane 0 of warp 28); false: no more
            auto load = [&]() {
                while (left == 0) {
                    if (at >= units_n) return false;
                    const ChunkUnit *u = units + at;
                    if (!LOCAL || u->more) {
                        load_h = h;
                        row = u->t0;
                        left = chunks_of(u->n);
                    }
                    step();
                }
                const int s = loaded % ST, hk = LOCAL ? load_h : quotient(load_h, inv_g);
                if (loaded >= ST && !chunk_wait(&empty[s], (uint32_t)(loaded / ST - 1) & 1u, abort_flag)) return false;
                uint8_t *stage = sm + s * S::kStageBytes;
                mbar_arrive_expect_tx(&full[s], (LOCAL ? 2 : 3) * PAN * kChunkPanel);
#pragma unroll 1
                for (int x = 0; x < PAN; ++x) {
                    if (!LOCAL) tma_load_3d(stage + x * S::kQkPanel, &qmap, &full[s], x * 64, load_h, row);
                    tma_load_3d(stage + x * S::kQkPanel + kChunkPanel, &kmap, &full[s], x * 64, hk, row);
                    tma_load_3d(stage + S::kVOff + x * kChunkPanel, &vmap, &full[s], x * 64, hk, row);
                }
                ++loaded;
                --left;
                row += LC;
                return true;
            };
            // warp 29 writes the units' tables, a unit ahead; behind the last one an empty unit
            int written = 0;
            auto write_tables = [&]() {
                const int m = written++;
                if (m >= 2 && !wait(&tab_free[m & 1], (m >> 1) - 1)) return false;
                while (LOCAL && at < units_n && !units[at].more) step();
                const bool some = at < units_n;
                float *t = tab_of(m);
                UnitInfo *info = info_of(m);
                if (some) {
                    const int hk = LOCAL ? h : uni(quotient(h, inv_g));
                    const ChunkUnit u = units[at];
                    const int n_last = u.n - (chunks_of(u.n) - 1) * LC;
                    const float *decay = p.decay + (int64_t)hk * kDecayRow;
#pragma unroll
                    for (int j = lane; j < LC; j += 32) {
                        t[j] = p.scale * decay[j];
                        t[LC + j] = p.scale * decay[j + 1];
                        t[2 * LC + j] = decay[LC - 1 - j];
                        t[3 * LC + j] = j < n_last ? decay[n_last - 1 - j] : 0.f;
                    }
                    if (lane == 0)
                        *info = UnitInfo{u.n, u.t0, h, hk, u.row, u.slot, u.from, u.last && (LOCAL || h == hk * p.G),
                                         decay[LC], decay[2 * LC + 1], decay[n_last], decay[LC + 1 + n_last]};
                    step();
                } else if (lane == 0) {
                    info->count = 0;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&tab_full[m & 1]);
                return some;
            };
            if (half == 0 && lane == 0) {
                while (load()) {
                }
            }
            if (half == 1) {
                while (write_tables()) {
                }
            }
            // copies still in flight (after a wait that gave up) land before the CTA ends
            if (half == 0 && lane == 0)
                for (int d = max(0, loaded - ST); d < loaded; ++d)
                    chunk_wait(&full[d % ST], (uint32_t)(d / ST) & 1u, &never);
            __syncwarp();
        } else if (warp == 30) {
            // ============================================================ MMA: KV, QS, PV
            // In this order: while the output warps read PV's chunk, the tensor core has the next KV.
            // kv_go comes from threads that saw the chunk's copies land; qs_go from warps that wrote their part of
            // P before.
            int g = 0;                               // chunks before unit m
            bool ok = true;
#pragma unroll 1
            for (int m = 0;; ++m) {
                if (!(ok = wait(&tab_full[m & 1], m >> 1))) break;
                const int count = uni(info_of(m)->count), chunks = chunks_of(count);
                if (count == 0) break;
#pragma unroll 1
                for (int c = 0; c < chunks; ++c) {
                    const int gc = g + c, s = gc % ST;
                    const uint32_t qk = smb + s * S::kStageBytes;
                    if (!(ok = wait(&kv_go[gc & 1], gc >> 1))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        constexpr uint32_t id = idesc_bf16_f32(128, D, 1);
                        const uint64_t kd = sw128_desc(qk + kChunkPanel, S::kQkPanel, 1024);
                        const uint64_t ld = sw128_desc(smb + lo_at(gc), PAN == 2 ? kChunkPanel : 0, 1024);
#pragma unroll 1
                        for (int part = 0; part < 2; ++part) {
#pragma unroll
                            for (int k = 0; k < LC / 16; ++k)
                                tc_mma_ts(tmem + TC_KV, tmem + w_at(gc) + part * 32 + k * 8,
                                          kd + k * (16 * 128 >> 4), id, part + k > 0);
                        }
#pragma unroll
                        for (int k = 0; k < LC / 16; ++k)
                            tc_mma_ss(tmem + TC_KV, ld + k * (16 * 128 >> 4), kd + k * (16 * 128 >> 4), id | kAMnMajor,
                                      1);
                        tc_commit(kv_ready);
                        tc_commit(&w_free[gc & 1]);
                        if (LOCAL) tc_commit(&empty[s]);
                    }
                    __syncwarp();
                    if (LOCAL) continue;
                    if (!(ok = wait(qs_go, gc))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        constexpr uint32_t id = idesc_bf16_f32(128, LC, 0);
                        const uint64_t qd = sw128_desc(qk, 16, 1024);
#pragma unroll 1
                        for (int part = 0; part < 2; ++part) {
#pragma unroll
                            for (int k = 0; k < D / 16; ++k)
                                tc_mma_ts(tmem + TC_INTER, tmem + TC_STATE + part * 64 + k * 8,
                                          qd + (k / 4) * (S::kQkPanel >> 4) + (k % 4) * 2, id, part + k > 0);
                        }
                        tc_commit(qs_done);
                        // A = V^T straight from the loaded tile (dv along its 128-byte rows); head_dim 64: lanes
                        // 64..127 repeat the one panel
                        const uint64_t pd = sw128_desc(smb + S::kPOff + (gc & 1) * 2 * kChunkPanel, 16, 1024);
                        const uint64_t vd = sw128_desc(qk + S::kVOff, PAN == 2 ? kChunkPanel : 0, 1024);
#pragma unroll 1
                        for (int part = 0; part < 2; ++part) {
#pragma unroll
                            for (int k = 0; k < LC / 16; ++k)
                                tc_mma_ss(tmem + TC_INTRA, vd + k * (16 * 128 >> 4),
                                          pd + part * (kChunkPanel >> 4) + k * 2, id | kAMnMajor, part + k > 0);
                        }
                        tc_commit(o_ready);
                        tc_commit(&empty[s]);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (lane == 0) mbar_arrive(&tab_free[m & 1]);
                g += chunks;
            }
            // nothing of this CTA's is left in the tensor core when TMEM goes back
            if (elect_one()) tc_commit(drain);
            __syncwarp();
            chunk_wait(drain, 0u, &never);
            __syncwarp();
        } else {
            // ============================================================ MMA: QK, a chunk ahead
            if (!LOCAL) {
                int g = -1;                              // chunks before unit m; unit -1: the first chunk's
                bool ok = true;
#pragma unroll 1
                for (int m = -1;; ++m) {
                    int chunks = 1;
                    if (m >= 0) {
                        if (!(ok = wait(&tab_full[m & 1], m >> 1))) break;
                        chunks = uni(chunks_of(info_of(m)->count));
                        if (chunks == 0) break;
                    }
#pragma unroll 1
                    for (int c = 0; c < chunks; ++c) {
                        const int next = g + c + 1;
                        if (next > 0 && !(ok = wait(p_ready, next - 1))) break;
                        if (c + 1 == chunks && m >= 0) {
                            // the next chunk belongs to the next unit, if there is one
                            if (!(ok = wait(&tab_full[(m + 1) & 1], (m + 1) >> 1))) break;
                            if (uni(info_of(m + 1)->count) == 0) break;
                        }
                        if (!(ok = wait(&full[next % ST], next / ST))) break;
                        tc_fence_after();
                        if (elect_one()) {
                            // A = Q's 64 rows and the 64 behind them, whose products nobody reads
                            const uint64_t qd = sw128_desc(smb + (next % ST) * S::kStageBytes, 16, 1024);
                            constexpr uint32_t id = idesc_bf16_f32(128, LC, 0);
#pragma unroll
                            for (int k = 0; k < D / 16; ++k) {
                                const uint64_t d = qd + (k / 4) * (S::kQkPanel >> 4) + (k % 4) * 2;
                                tc_mma_ss(tmem + TC_S, d, d + (kChunkPanel >> 4), id, k > 0);
                            }
                            tc_commit(s_ready);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    if (m >= 0 && lane == 0) mbar_arrive(&tab_free[m & 1]);
                    g += chunks;
                }
            }
            if (elect_one()) tc_commit(drain);
            __syncwarp();
            chunk_wait(drain, 0u, &never);
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
    if (threadIdx.x == 0 && (abort_flag[0] | abort_flag[1])) record_error(p.err, ERR_TIMEOUT | SRC_LINEAR);
}

template <int D>
cudaError_t launch_chunks(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap,
                          const CUtensorMap &omap, const LinearParams &p, cudaStream_t stream) {
    using S = ChunkSmem<D>;
    static std::once_flag once[kMaxDev];
    static cudaError_t attr_err[kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [&] {
        attr_err[dev] = cudaFuncSetAttribute(linear_chunk_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             S::kBytes);
        if (attr_err[dev] == cudaSuccess)
            attr_err[dev] = cudaFuncSetAttribute(linear_chunk_kernel<D, true>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
    });
    if (attr_err[dev] != cudaSuccess) return attr_err[dev];
    linear_plan_kernel<<<1 + (p.Hkv + 7) / 8, 1024, 0, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // a CTA per SM at most: each goes over several units
    auto ctas = [&](int heads) { return (unsigned)min((int64_t)p.max_units * heads, (int64_t)p.num_sms); };
    const bool split = p.seg_len < p.max_seqlen;
    if (split) {
        e = launch_after(linear_chunk_kernel<D, true>, dim3(ctas(p.Hkv)), kChunkThreads, S::kBytes, stream, qmap, kmap,
                         vmap, omap, p);
        if (e != cudaSuccess) return e;
    }
    if (p.state_rows > 0) {
        e = launch_after(linear_scan_kernel, dim3(p.max_units, p.Hkv, D * D / 1024), 256, 0, stream, p);
        if (e != cudaSuccess) return e;
    }
    main_kernel_event_before(stream);
    e = launch_after(linear_chunk_kernel<D, false>, dim3(ctas(p.Hq)), kChunkThreads, S::kBytes, stream, qmap, kmap,
                     vmap, omap, p);
    main_kernel_event_after(stream);
    return e;
}

}  // namespace

cudaError_t launch_linear_varlen(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap,
                                 const CUtensorMap &omap, const LinearParams &p, cudaStream_t stream) {
    return p.D == 128 ? launch_chunks<128>(qmap, kmap, vmap, omap, p, stream)
                      : launch_chunks<64>(qmap, kmap, vmap, omap, p, stream);
}

cudaError_t launch_linear_decode(const LinearParams &p, cudaStream_t stream) { return launch_decode_kernel(p, stream); }

}  // namespace attn
