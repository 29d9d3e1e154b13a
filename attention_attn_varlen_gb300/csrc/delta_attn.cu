// delta_attn.cu -- linear attention by the gated delta rule:
//   u_t = beta_t (v_t - e^{g_t} S_{t-1} k_t)
//   S_t = e^{g_t} S_{t-1} + u_t k_t^T       (S [Dv, Dk], fp32)
//   o_t = scale * S_t q_t
// over packed sequences (prompts, a few tokens each) or one token per sequence
// (decode), with a cache of states.
#include <mutex>

#include "chunks.cuh"
#include "kernels.h"
#include "sequences.cuh"

namespace attn {
namespace {

// e^{log_decay} of token t and head h: a positive or NaN log_decay counts as 0 and is reported.
__device__ __forceinline__ float delta_decay(const DeltaParams &p, int64_t t, int h, bool report) {
    const float g = __ldg(p.log_decay + t * p.decay_stride + h);
    if (report && !(g <= 0.f)) record_error(p.err, ERR_RANGE | SRC_DELTA);
    return expf(fminf(g, 0.f));
}

// sums over the LPR lanes of a row, in every lane
template <int LPR> __device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int w = LPR / 2; w > 0; w /= 2) x += __shfl_xor_sync(0xffffffffu, x, w);
    return x;
}

// ---------------------------------------------------------------------------
// The recurrent form.  A lane holds four neighbouring columns of eight rows of S in
// registers, a warp 32 lanes / (D / 4) times eight rows; S is read and written
// once, whatever the number of tokens, 8 D^2 bytes per sequence and value head,
// which bounds one token per sequence (HBM).
// With S k and S q of the state before the token,
//   S_t q = e^g S q + u (k . q),
// so one reduction per token serves u and the output.  The sums of the eight rows are
// reduced together (9 shuffles), S k is then handed back to all lanes (7).
// ---------------------------------------------------------------------------
constexpr int kRecRows = 8;
constexpr int kRecWarps = 4;

template <int D, bool PACKED>
__global__ void __launch_bounds__(kRecWarps * 32) delta_recurrent_kernel(const DeltaParams p) {
    constexpr int LPR = D / 4;                          // lanes per row
    constexpr int RPL = 32 / LPR;                       // rows per load
    constexpr int ROWS = kRecRows * RPL;                // rows per warp
    constexpr int CTAS = D / (ROWS * kRecWarps);        // CTAs per state
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int unit = blockIdx.x / CTAS, b = unit / p.Hv, h = unit - b * p.Hv, hk = h / p.G;
    const int row0 = ((blockIdx.x - unit * CTAS) * kRecWarps + warp) * ROWS + (lane / LPR) * kRecRows;
    const int col = (lane & (LPR - 1)) * 4;
    const bool first_thread = blockIdx.x - unit * CTAS == 0 && threadIdx.x == 0;
    int64_t t = b;
    int n = 1;
    if (PACKED) sequence_rows<SRC_DELTA>(p, b, t, n, h == 0 && first_thread);
    bool from;
    float *state = sequence_state<SRC_DELTA, PACKED>(p, p.Hv, b, h, from, h == 0 && first_thread && n > 0);
    if (PACKED && n == 0) return;
    float4 S[kRecRows];                                 // rows row0 .. row0 + 7, columns col .. col + 3
#pragma unroll
    for (int i = 0; i < kRecRows; ++i) {
        S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (from) S[i] = __ldcs(reinterpret_cast<const float4 *>(state + (row0 + i) * D + col));
    }
#pragma unroll 1
    for (; n > 0; --n, ++t) {
        const uint2 kr = *reinterpret_cast<const uint2 *>(p.k + t * p.k_stride + (int64_t)hk * D + col);
        const uint2 qr = *reinterpret_cast<const uint2 *>(p.q + t * p.q_stride + (int64_t)hk * D + col);
        const uint4 vr = *reinterpret_cast<const uint4 *>(p.v + t * p.v_stride + (int64_t)h * D + row0);
        const float beta = __ldg(p.beta + t * p.beta_stride + h);
        const float a = delta_decay(p, t, h, first_thread);
        const float k0 = __uint_as_float(kr.x << 16), k1 = __uint_as_float(kr.x & 0xFFFF0000u);
        const float k2 = __uint_as_float(kr.y << 16), k3 = __uint_as_float(kr.y & 0xFFFF0000u);
        const float q0 = __uint_as_float(qr.x << 16), q1 = __uint_as_float(qr.x & 0xFFFF0000u);
        const float q2 = __uint_as_float(qr.y << 16), q3 = __uint_as_float(qr.y & 0xFFFF0000u);
        float rk = 1.f, rq = 1.f;
        if (p.norm) {
            rk = 1.f / sqrtf(row_sum<LPR>(fmaf(k0, k0, fmaf(k1, k1, fmaf(k2, k2, k3 * k3)))) + p.eps);
            rq = 1.f / sqrtf(row_sum<LPR>(fmaf(q0, q0, fmaf(q1, q1, fmaf(q2, q2, q3 * q3)))) + p.eps);
        }
        const float kq = row_sum<LPR>(fmaf(k0, q0, fmaf(k1, q1, fmaf(k2, q2, k3 * q3))));
        float sk[kRecRows], sq[kRecRows];
#pragma unroll
        for (int i = 0; i < kRecRows; ++i) {
            sk[i] = fmaf(S[i].x, k0, fmaf(S[i].y, k1, fmaf(S[i].z, k2, S[i].w * k3)));
            sq[i] = fmaf(S[i].x, q0, fmaf(S[i].y, q1, fmaf(S[i].z, q2, S[i].w * q3)));
        }
        // each step halves the rows a lane carries: the lane's bits LPR / 2, LPR / 4, LPR / 8 pick the row
        int w = LPR / 2;
#pragma unroll
        for (int m = kRecRows / 2; m > 0; m /= 2, w /= 2) {
            const bool up = lane & w;
#pragma unroll
            for (int i = 0; i < m; ++i) {
                sk[i] = (up ? sk[i + m] : sk[i]) + __shfl_xor_sync(0xffffffffu, up ? sk[i] : sk[i + m], w);
                sq[i] = (up ? sq[i + m] : sq[i]) + __shfl_xor_sync(0xffffffffu, up ? sq[i] : sq[i + m], w);
            }
        }
#pragma unroll
        for (; w > 0; w /= 2) {
            sk[0] += __shfl_xor_sync(0xffffffffu, sk[0], w);
            sq[0] += __shfl_xor_sync(0xffffffffu, sq[0], w);
        }
        w = LPR / 8;
#pragma unroll
        for (int m = 1; m < kRecRows; m *= 2, w *= 2) {
            const bool up = lane & w;
#pragma unroll
            for (int i = 0; i < m; ++i) {
                const float other = __shfl_xor_sync(0xffffffffu, sk[i], w);
                sk[i + m] = up ? sk[i] : other;
                sk[i] = up ? other : sk[i];
            }
        }
        const uint32_t vw[4] = {vr.x, vr.y, vr.z, vr.w};
        const float ark = a * rk;
        float u[kRecRows];
#pragma unroll
        for (int i = 0; i < kRecRows; ++i) {
            const float v = __uint_as_float(i & 1 ? vw[i / 2] & 0xFFFF0000u : vw[i / 2] << 16);
            u[i] = beta * (v - ark * sk[i]);
            const float uk = u[i] * rk;
            S[i].x = fmaf(uk, k0, a * S[i].x);
            S[i].y = fmaf(uk, k1, a * S[i].y);
            S[i].z = fmaf(uk, k2, a * S[i].z);
            S[i].w = fmaf(uk, k3, a * S[i].w);
        }
        // the row whose sum the lane holds
        const int row = (lane & (LPR - 1)) / (LPR / 8);
        float own = u[0];
#pragma unroll
        for (int i = 1; i < kRecRows; ++i) own = row == i ? u[i] : own;
        if ((lane & (LPR / 8 - 1)) == 0)
            p.out[t * p.out_stride + (int64_t)h * D + row0 + row] =
                __float2bfloat16_rn(p.scale * rq * fmaf(own * rk, kq, a * sq[0]));
    }
    if (state) {
#pragma unroll
        for (int i = 0; i < kRecRows; ++i) __stcs(reinterpret_cast<float4 *>(state + (row0 + i) * D + col), S[i]);
    }
}

// ---------------------------------------------------------------------------
// Prompts, in chunks of 64 tokens on the tensor cores.
//
// With G_i = g_1 + .. + g_i in a chunk, S_0 the state before it and r_i = 1 / |k_i| where keys
// are normalised on the way (else 1), the tokens' writes u~_i = r_i u_i solve
//   u~_i + sum_{j < i} A_ij u~_j = b_i v_i - c_i S_0 k_i,     A_ij = beta_i r_i^2 e^{G_i - G_j} k_i . k_j,
//   b_i = beta_i r_i,  c_i = beta_i r_i^2 e^{G_i}.
// With T = (I + A)^-1, lower triangular with ones on its diagonal, and R the right sides,
//   U~ = T R,   o_i = f_i S_0 q_i + sum_{j <= i} P_ij u~_j,   S_n = e^{G_n} S_0 + sum_j e^{G_n - G_j} u~_j k_j^T
// with f_i = scale e^{G_i} / |q_i| and P_ij = scale e^{G_i - G_j} q_i . k_j / |q_i|.  Every exponent is <= 0:
// nothing overflows whatever the decay.
//
// As matrices with the value dimension in the 128 TMEM lanes, so that S_0, R and U~ are A
// operands read from TMEM:
//   KQ [i, j]   = (Q; K) K^T     shared x shared
//   SK [dv, j]  = S_0 K^T        TMEM (three bf16 parts) x shared
//   SQ [dv, i]  = S_0 Q^T        TMEM (two parts) x shared
//   U  [dv, i]  = R^T T^T        TMEM (three parts) x shared (three parts): the five products above 2^-16
//   KV [dv, dk] = (w_j U~)^T K   TMEM (three parts) x shared,  w_j = e^{G_n - G_j}
//   PU [dv, i]  = U~^T P^T       TMEM (two parts) x shared (two parts)
//
// Precision.  q, k and v are bf16 and exact.  The state, R, T and w U~ are fp32 values in three bf16 parts,
// 2^-24 of each; S itself stays in fp32 registers.  What only reaches the bf16 output (S_0 and U~
// there, P) is taken as two parts, 2^-16 of a term against the output's own 2^-8.  T is solved for
// in fp32, its 32 x 32 diagonal blocks row by row, the block below them as -T22 A21 T11.  Sums of decays are in
// 64 bits and differences of them kept as two fp32 parts.
//
// What bounds it is a chunk's chain S -> SK -> R -> U -> w U~ -> KV -> S; SQ, KQ and PU run in its gaps.
//
// Roles (28 warps, one CTA per SM that goes over (sequence, value head) units):
//   0..15   the chain: thread = value dimension and a quarter of dk or of the tokens; S in registers
//   16..19  T and P of the next chunk: lanes are the rows of (Q; K)
//   20..23  output rows
//   24, 25  issue the loads; write the chunks' tables
//   26      issues the MMAs
// ---------------------------------------------------------------------------
constexpr int DC = 64;                       // tokens of a chunk
constexpr int kDeltaThreads = 28 * 32;
constexpr int kDeltaPanel = DC * 128;        // 64 rows x 128 bytes
// TMEM columns.  In turn in the same place: SK, U and then KV; S_0's third part, R and then w U~; S_0's first
// part and then U~'s two; S_0's second part and then KQ of the next chunk
constexpr uint32_t TM_KV = 0, TM_SK = 0, TM_U = 64;
constexpr uint32_t TM_S1 = 128, TM_UO = 128, TM_S2 = 192, TM_KQ = 192;
constexpr uint32_t TM_S3 = 256, TM_R = 256;  // (R: three parts of 32 columns)
constexpr uint32_t TM_SQ = 352, TM_PU = 416;
constexpr int kBlockStride = 36;             // floats of a row of a 32 x 32 block in shared memory
constexpr int kBlockFloats = 32 * kBlockStride;
constexpr int kDeltaBuckets = 256;

// A chunk as its roles read it, behind its tables.
struct DeltaChunk {
    int n;                            // tokens; 0: there is no such chunk
    int t0, h, first, last;           // first row; head; whether the unit starts or ends with it
    int slot, from;                   // state slot (-1: none), whether the unit starts from it
    float a, a_lo;                    // e^{G_n} in two parts
    int pad[7];
};

template <int D>
struct DeltaSmem {
    static constexpr int kPanels = D / 64;
    static constexpr int kQkPanel = 2 * kDeltaPanel;             // 64 Q rows, then 64 K rows
    static constexpr int kQkBytes = kPanels * kQkPanel, kVBytes = kPanels * kDeltaPanel;
    static constexpr int kQkStages = 3, kVStages = 2;
    static constexpr int kVOff = kQkStages * kQkBytes;
    static constexpr int kTOff = kVOff + kVStages * kVBytes;     // T: three parts
    static constexpr int kPOff = kTOff + 3 * kDeltaPanel;        // two chunks' P: two parts
    static constexpr int kOutOff = kPOff + 4 * kDeltaPanel;      // per output warp [64 tokens][32 dv] bf16
    static constexpr int kBlockOff = kOutOff + 4 * DC * 64;      // A11, then T11; A22, then T22; A21; A21 T11
    static constexpr int kTabOff = kBlockOff + 4 * kBlockFloats * 4;
    // two chunks' tables: G (two parts), beta, e^G, w, b, -c, f, and the chunk itself
    static constexpr int kTabFloats = 8 * DC + 16;
    static constexpr int kBadOff = kTabOff + 2 * kTabFloats * 4; // first non-finite token per dv, two chunks
    static constexpr int kBarOff = kBadOff + 2 * 128 * 4;
    static constexpr int kNumBars = 30;
    static constexpr int kBytes = kBarOff + kNumBars * 8 + 16 + 1024 /* alignment slack */;
    static_assert(kBytes <= 227 * 1024 && sizeof(DeltaChunk) == 64, "shared memory");
};

// Registers of the calling warpgroup.  The kernel is launched with 72 a thread; the seven warpgroups'
// shares add up to that: chain 4, T and P, output rows, the others.
constexpr int kChainRegs = 80, kSolveRegs = 88, kRowRegs = 56, kOtherRegs = 40;
static_assert(4 * kChainRegs + kSolveRegs + kRowRegs + kOtherRegs <= 7 * 72, "register shares");

// A unit's entry in the work list, as the plan writes it.
struct alignas(16) DeltaUnit {
    int t0, n;          // first token, tokens
    int slot, from;     // state slot (-1: none), whether the sequence starts from it
};
static_assert(sizeof(DeltaUnit) == kDeltaUnitBytes, "workspace layout");

// The work list: a unit is a sequence; the longest come first.
__global__ void __launch_bounds__(1024) delta_plan_kernel(const DeltaParams p) {
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x;
    __shared__ int count[kDeltaBuckets];
    for (int i = tid; i < kDeltaBuckets; i += 1024) count[i] = 0;
    __syncthreads();
    auto bucket = [&](int tokens) {
        return kDeltaBuckets - 1 - (int)((int64_t)tokens * (kDeltaBuckets - 1) / p.max_seqlen);
    };
    for (int pass = 0; pass < 2; ++pass) {
        for (int b = tid; b < p.batch; b += 1024) {
            int64_t t0;
            int n;
            sequence_rows<SRC_DELTA>(p, b, t0, n, pass == 0);
            if (n == 0) continue;
            const int at = atomicAdd(&count[bucket(n)], 1);
            if (pass == 1) {
                bool from;
                const float *state = sequence_state<SRC_DELTA, true>(p, p.Hv, b, 0, from, true);
                reinterpret_cast<DeltaUnit *>(p.units)[at] =
                    DeltaUnit{(int)t0, n, state ? __ldg(p.slots + b) : -1, from};
            }
        }
        __syncthreads();
        if (pass == 0 && tid < 32) {
            // counts -> first places
            int base = 0;
            for (int i = 0; i < kDeltaBuckets; i += 32) {
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
            if (tid == 0) *p.unit_count = base;
        }
        __syncthreads();
    }
}

// the chunks of a CTA's units, in order; places blockIdx.x, 2 gridDim.x - 1 - blockIdx.x, 2 gridDim.x + blockIdx.x,
// ... of the list (longest first), back and forth so that the CTAs' sums come out alike
struct DeltaWalk {
    int k = 0, h = 0, c = 0, chunks = 0;
    DeltaUnit u;
    // the next chunk; false: no more
    __device__ __forceinline__ bool step(const DeltaUnit *units, int units_n, int heads) {
        if (++c < chunks) return true;
        const int G = gridDim.x, place = k * G + ((k & 1) ? G - 1 - (int)blockIdx.x : (int)blockIdx.x);
        const int at = place / heads;
        if (at >= units_n) return false;
        h = place - at * heads;
        u = units[at];
        chunks = (u.n + DC - 1) / DC;
        c = 0;
        ++k;
        return true;
    }
};

// 1 / sqrt(x): the hardware's estimate and one step of Newton's method
__device__ __forceinline__ float inv_sqrt(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return x > 0.f ? y * fmaf(-0.5f * x * y, y, 1.5f) : y;
}

// x0, x1 as three bf16 parts
__device__ __forceinline__ void split3(float x0, float x1, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    hi = take_bf16(x0, x1);
    mid = take_bf16(x0, x1);
    lo = pack_bf16x2(x0, x1);
}

// non-finite entries of x become 0; returns the first one's place, 16 if there is none
__device__ __forceinline__ int drop_non_finite(float (&x)[16]) {
    int first = 16;
#pragma unroll
    for (int j = 15; j >= 0; --j) {
        const bool bad = !(fabsf(x[j]) < INFINITY);
        first = bad ? j : first;
        x[j] = bad ? 0.f : x[j];
    }
    return first;
}

template <int D>
__global__ void __launch_bounds__(kDeltaThreads, 1)
    delta_chunk_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap omap,
                       const DeltaParams p) {
    using S = DeltaSmem<D>;
    constexpr int PAN = S::kPanels, QS = S::kQkStages, VS = S::kVStages;
    extern __shared__ __align__(1024) uint8_t dsmem_raw[];
    // values from lane 0 are warp-uniform to the compiler, and so is what is computed from them
    auto uni = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    const int warp = uni(threadIdx.x >> 5), lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const DeltaUnit *units = reinterpret_cast<const DeltaUnit *>(p.units);
    const int units_n = uni(*p.unit_count);
    if ((int)blockIdx.x >= units_n * p.Hv) return;

    const uint32_t smb = (smem_u32(dsmem_raw) + 1023u) & ~1023u;          // shared-memory address, for descriptors
    uint8_t *sm = dsmem_raw + (smb - smem_u32(dsmem_raw));
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + S::kBarOff);
    uint64_t *qk_full = bars, *qk_empty = bars + 3;
    uint64_t *v_full = bars + 6, *v_empty = bars + 8;
    uint64_t *tab_full = bars + 10, *tab_free = bars + 12;   // [2], by chunk: its tables are written, read for the last time
    uint64_t *norms = bars + 14;             // [2]: b, c and f are written too
    uint64_t *o_done = bars + 16;            // [2]: SQ and PU done
    uint64_t *kq_done = bars + 18;           // KQ done
    uint64_t *kq_read = bars + 19;           // ... and read
    uint64_t *t_ready = bars + 20;           // T and P in shared memory
    uint64_t *s_ready = bars + 21;           // S_0 in TMEM, the KV before read
    uint64_t *sk_done = bars + 22;
    uint64_t *r_ready = bars + 23;           // R in TMEM
    uint64_t *u_done = bars + 24;
    uint64_t *w_ready = bars + 25;           // U~ and w U~ in TMEM
    uint64_t *kv_done = bars + 26;
    uint64_t *o_read = bars + 27;            // SQ and PU read
    uint64_t *solve = bars + 28;             // among the solving warps
    uint64_t *drain = bars + 29;             // every MMA done
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + S::kNumBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float *tables = reinterpret_cast<float *>(sm + S::kTabOff);
    int *bad_at = reinterpret_cast<int *>(sm + S::kBadOff);
    auto tab_of = [&](int gc) { return tables + (gc & 1) * S::kTabFloats; };
    auto info_of = [&](int gc) { return reinterpret_cast<DeltaChunk *>(tab_of(gc) + 8 * DC); };
    enum { T_GHI = 0, T_GLO = DC, T_BETA = 2 * DC, T_GAM = 3 * DC, T_W = 4 * DC, T_B = 5 * DC, T_C = 6 * DC, T_F = 7 * DC };

    if (warp == 24 && lane == 0) {
        for (int i = 0; i < QS; ++i) {
            mbar_init(&qk_full[i], 1);
            mbar_init(&qk_empty[i], 1 + 4);  // the MMAs, the solving warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 16);
            mbar_init(&tab_full[i], 1);
            mbar_init(&tab_free[i], 16 + 4 + 4 + 1);
            mbar_init(&norms[i], 4);
            mbar_init(&o_done[i], 1);
        }
        mbar_init(kq_done, 1);
        mbar_init(kq_read, 4);
        mbar_init(t_ready, 4);
        mbar_init(s_ready, 16);
        mbar_init(sk_done, 1);
        mbar_init(r_ready, 16);
        mbar_init(u_done, 1);
        mbar_init(w_ready, 16);
        mbar_init(kv_done, 1);
        mbar_init(o_read, 4);
        mbar_init(solve, 4);
        mbar_init(drain, 1);
        abort_flag[0] = abort_flag[1] = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (warp >= 16 && warp < 20) {
        // what lies above the diagonal blocks of T and P stays zero: rows 0..31, tokens 32..63 of every part
#pragma unroll 1
        for (int x = warp - 16; x < 7; x += 4) {
#pragma unroll
            for (int ch = 4; ch < 8; ++ch)
                *reinterpret_cast<uint4 *>(sm + S::kTOff + x * kDeltaPanel + sw128_off(lane, ch)) =
                    make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uni((int)*tmem_slot);
    // waits for what the hardware finishes by itself run to the limit: their flag is their own
    volatile int &never = *(abort_flag + 1);
    // a warp's wait: every lane gets the same answer
    auto wait = [&](uint64_t *bar, int phase) {
        return __all_sync(0xffffffffu, chunk_wait(bar, (uint32_t)phase & 1u, abort_flag)) != 0;
    };
    auto arrive = [&](uint64_t *bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };

    if (warp < 16) {
        // ============================================================ the chain
        more_regs<kChainRegs>();
        const int grp = warp & 3, part = warp >> 2, dv = grp * 32 + lane;
        const bool real = grp * 32 < D;      // warp-uniform; head_dim 64: lanes 64..127 reach no output
        const uint32_t lane_base = tmem + ((uint32_t)(grp * 32) << 16);
        constexpr int N = D / 4;             // columns of S per thread
        // its value dimension in a V tile, its tokens part * 16 ..
        const uint32_t v_at = smb + S::kVOff + ((dv & (D - 1)) >> 6) * kDeltaPanel + part * 16 * 128 + (dv & 7) * 2;
        const uint32_t v_ch = ((dv & 63) >> 3) << 4;
        float St[N];
#pragma unroll 1
        for (int gc = 0;; ++gc) {
            if (!wait(&tab_full[gc & 1], gc >> 1)) break;
            const DeltaChunk *info = info_of(gc);
            const float *tab = tab_of(gc);
            const int n = uni(info->n);
            if (n == 0) break;
            int *bad_row = bad_at + (gc & 1) * 128 + dv;
            if (info->first) {
                const float *src = info->from && info->slot >= 0
                                       ? p.state + ((int64_t)info->slot * p.Hv + info->h) * D * D + dv * D + part * N
                                       : nullptr;
#pragma unroll
                for (int i = 0; i < N; i += 4) {
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (src && real) x = *reinterpret_cast<const float4 *>(src + i);
                    St[i] = x.x, St[i + 1] = x.y, St[i + 2] = x.z, St[i + 3] = x.w;
                }
            }
            // ---- S_0's parts to TMEM; the first one where PU of the chunk before reads U~
            if (part == 0) *bad_row = DC;
            if (!wait(kq_read, gc)) break;
            {
                uint32_t s1[N / 2];
                if (real) {
#pragma unroll
                    for (int i = 0; i < N; i += 16) {
                        uint32_t s2[8], s3[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            split3(St[i + 2 * k], St[i + 2 * k + 1], s1[i / 2 + k], s2[k], s3[k]);
                        tmem_st8(lane_base + TM_S2 + (part * N + i) / 2, s2);
                        tmem_st8(lane_base + TM_S3 + (part * N + i) / 2, s3);
                    }
                }
                if (gc > 0 && !wait(&o_done[(gc - 1) & 1], (gc - 1) >> 1)) break;
                tc_fence_after();
                if (real) {
#pragma unroll
                    for (int i = 0; i < N / 2; i += 8) {
                        uint32_t s[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) s[k] = s1[i + k];
                        tmem_st8(lane_base + TM_S1 + part * N / 2 + i, s);
                    }
                    tc_wait_st();
                }
            }
            tc_fence_before();
            arrive(s_ready);
            // ---- R = b v - c S_0 k
            if (!wait(&norms[gc & 1], gc >> 1)) break;
            if (!wait(&v_full[gc % VS], gc / VS)) break;
            float x[16];
            {
                float v[16];
                const uint32_t at = v_at + (gc % VS) * S::kVBytes;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    uint16_t r;
                    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(at + j * 128 + (v_ch ^ ((j & 7) << 4))));
                    v[j] = __uint_as_float((uint32_t)r << 16);
                }
                const float4 *b4 = reinterpret_cast<const float4 *>(tab + T_B + part * 16);
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 b = b4[j / 4];
                    fma2(x[j], x[j + 1], b.x, b.y, v[j], v[j + 1], 0.f, 0.f);
                    fma2(x[j + 2], x[j + 3], b.z, b.w, v[j + 2], v[j + 3], 0.f, 0.f);
                }
            }
            arrive(&v_empty[gc % VS]);
            if (!wait(sk_done, gc)) break;
            tc_fence_after();
            if (real) {
                uint32_t sk[16];
                tmem_ld16(lane_base + TM_SK + part * 16, sk);
                const float4 *c4 = reinterpret_cast<const float4 *>(tab + T_C + part * 16);
                tc_wait_ld();
                float z0 = 0.f, z1 = 0.f;    // NaN once something non-finite went by
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 c = c4[j / 4];
                    fma2(x[j], x[j + 1], c.x, c.y, __uint_as_float(sk[j]), __uint_as_float(sk[j + 1]), x[j], x[j + 1]);
                    fma2(x[j + 2], x[j + 3], c.z, c.w, __uint_as_float(sk[j + 2]), __uint_as_float(sk[j + 3]), x[j + 2],
                         x[j + 3]);
                }
                if (n < DC) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) x[j] = part * 16 + j < n ? x[j] : 0.f;
                }
#pragma unroll
                for (int j = 0; j < 16; j += 2) fma2(z0, z1, x[j], x[j + 1], 0.f, 0.f, z0, z1);
                if (__any_sync(0xffffffffu, !(z0 + z1 == 0.f))) {
                    // T's zeros would not keep it from earlier tokens
                    const int first = drop_non_finite(x);
                    if (first < 16) atomicMin(bad_row, part * 16 + first);
                }
                uint32_t r1[8], r2[8], r3[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) split3(x[2 * k], x[2 * k + 1], r1[k], r2[k], r3[k]);
                tmem_st8(lane_base + TM_R + part * 8, r1);
                tmem_st8(lane_base + TM_R + 32 + part * 8, r2);
                tmem_st8(lane_base + TM_R + 64 + part * 8, r3);
                tc_wait_st();
            }
            tc_fence_before();
            arrive(r_ready);
            // ---- U~ and w U~
            if (!wait(u_done, gc)) break;
            tc_fence_after();
            if (real) {
                uint32_t u[16];
                tmem_ld16(lane_base + TM_U + part * 16, u);
                const float4 *w4 = reinterpret_cast<const float4 *>(tab + T_W + part * 16);
                tc_wait_ld();
                float z0 = 0.f, z1 = 0.f;
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = __uint_as_float(u[j]);
#pragma unroll
                for (int j = 0; j < 16; j += 2) fma2(z0, z1, x[j], x[j + 1], 0.f, 0.f, z0, z1);
                if (__any_sync(0xffffffffu, !(z0 + z1 == 0.f))) {
                    const int first = drop_non_finite(x);
                    if (first < 16) atomicMin(bad_row, part * 16 + first);
                }
                uint32_t r1[8], r2[8], r3[8];
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                    const float4 w = w4[k / 2];
                    float y0, y1;
                    fma2(y0, y1, x[2 * k], x[2 * k + 1], w.x, w.y, 0.f, 0.f);
                    split3(y0, y1, r1[k], r2[k], r3[k]);
                    fma2(y0, y1, x[2 * k + 2], x[2 * k + 3], w.z, w.w, 0.f, 0.f);
                    split3(y0, y1, r1[k + 1], r2[k + 1], r3[k + 1]);
                }
                tmem_st8(lane_base + TM_R + part * 8, r1);
                tmem_st8(lane_base + TM_R + 32 + part * 8, r2);
                tmem_st8(lane_base + TM_R + 64 + part * 8, r3);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    r1[k] = take_bf16(x[2 * k], x[2 * k + 1]);
                    r2[k] = pack_bf16x2(x[2 * k], x[2 * k + 1]);
                }
                tmem_st8(lane_base + TM_UO + part * 8, r1);
                tmem_st8(lane_base + TM_UO + 32 + part * 8, r2);
                tc_wait_st();
            }
            tc_fence_before();
            arrive(w_ready);
            // ---- S = e^{G_n} S + KV
            const float a = info->a, a_lo = info->a_lo;
            const bool last = info->last;
            float *dst = last && info->slot >= 0 ? p.state + ((int64_t)info->slot * p.Hv + info->h) * D * D + dv * D + part * N
                                                 : nullptr;
            if (!wait(kv_done, gc)) break;
            tc_fence_after();
            if (real) {
#pragma unroll
                for (int i = 0; i < N; i += 16) {
                    uint32_t kv[16];
                    tmem_ld16(lane_base + TM_KV + part * N + i, kv);
                    tc_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        float x0, x1;
                        fma2(x0, x1, a_lo, a_lo, St[i + k], St[i + k + 1], __uint_as_float(kv[k]),
                             __uint_as_float(kv[k + 1]));
                        fma2(St[i + k], St[i + k + 1], a, a, St[i + k], St[i + k + 1], x0, x1);
                    }
                }
                if (__any_sync(0xffffffffu, *bad_row < DC)) {
                    const bool bad = *bad_row < DC;
#pragma unroll
                    for (int i = 0; i < N; ++i) St[i] = bad ? __uint_as_float(0x7FC00000u) : St[i];
                }
            }
            tc_fence_before();
            arrive(&tab_free[gc & 1]);
            if (real && dst) {
#pragma unroll
                for (int i = 0; i < N; i += 4)
                    *reinterpret_cast<float4 *>(dst + i) = make_float4(St[i], St[i + 1], St[i + 2], St[i + 3]);
            }
        }
    } else if (warp < 20) {
        // ============================================================ T and P: lane = row of (Q; K)
        more_regs<kSolveRegs>();
        const int qd = warp & 3, row = qd * 32 + lane, i = row & 63;
        const bool keys = qd >= 2;
        const uint32_t lane_base = tmem + ((uint32_t)(qd * 32) << 16);
        float *blocks = reinterpret_cast<float *>(sm + S::kBlockOff);
        float *blk11 = blocks, *blk22 = blocks + kBlockFloats, *blk21 = blocks + 2 * kBlockFloats,
              *blkx = blocks + 3 * kBlockFloats;
        int turn = 0;                        // phases of `solve`
        auto together = [&]() {
            arrive(solve);
            return wait(solve, turn++);
        };
        // column `lane` of a 32 x 32 block of T: rows r, r + step of it, as three parts
        auto put_t = [&](int r, int step, int col, float x0, float x1) {
            uint32_t h[3];
            split3(x0, x1, h[0], h[1], h[2]);
            uint8_t *t = sm + S::kTOff + (col & 7) * 2;
            const uint32_t a0 = sw128_off(r, col >> 3), a1 = sw128_off(r + step, col >> 3);
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                *reinterpret_cast<uint16_t *>(t + x * kDeltaPanel + a0) = (uint16_t)h[x];
                *reinterpret_cast<uint16_t *>(t + x * kDeltaPanel + a1) = (uint16_t)(h[x] >> 16);
            }
        };
#pragma unroll 1
        for (int gc = 0;; ++gc) {
            if (!wait(&tab_full[gc & 1], gc >> 1)) break;
            const DeltaChunk *info = info_of(gc);
            float *tab = tab_of(gc);
            const int n = uni(info->n);
            if (n == 0) break;
            const int s = gc % QS;
            if (!wait(&qk_full[s], gc / QS)) break;
            uint8_t *tile = sm + s * S::kQkBytes + row * 128;
            if (keys && i >= n) {
                // rows behind the sequence's end are zeroed (a weight of 0 would not cancel a NaN there)
#pragma unroll 1
                for (int x = 0; x < PAN * 8; ++x)
                    *reinterpret_cast<uint4 *>(tile + (x >> 3) * S::kQkPanel + (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            if (n < DC) fence_proxy_async_smem();
            float r = 1.f;
            if (p.norm) {
                float s0 = 0.f, s1 = 0.f;
#pragma unroll 2
                for (int x = 0; x < PAN * 8; ++x) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(tile + (x >> 3) * S::kQkPanel +
                                                                     (((x & 7) ^ (row & 7)) << 4));
                    const uint32_t y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float e0 = __uint_as_float(y[k] << 16), e1 = __uint_as_float(y[k] & 0xFFFF0000u);
                        fma2(s0, s1, e0, e1, e0, e1, s0, s1);
                    }
                }
                r = inv_sqrt(s0 + s1 + p.eps);
            }
            float factor;                    // of the row of A or P
            if (keys) {
                const float beta = tab[T_BETA + i];
                tab[T_B + i] = beta * r;
                factor = beta * r * r;
                tab[T_C + i] = -factor * tab[T_GAM + i];
            } else {
                factor = p.scale * r;
                tab[T_F + i] = factor * tab[T_GAM + i];
            }
            arrive(&norms[gc & 1]);
            arrive(&qk_empty[s]);
            const float ghi = tab[T_GHI + i], glo = tab[T_GLO + i];
            if (!wait(kq_done, gc)) break;
            if (!keys && gc >= 2 && !wait(&o_done[gc & 1], (gc >> 1) - 1)) break;       // P's buffer
            tc_fence_after();
            // tokens 0..31 see no key behind 31
            uint8_t *ph = sm + S::kPOff + (gc & 1) * 2 * kDeltaPanel;
#pragma unroll 1
            for (int j0 = 0; j0 < 32 + 32 * (qd & 1); j0 += 8) {
                uint32_t kq[8];
                tmem_ld8(lane_base + TM_KQ + j0, kq);
                float x[8], g1[8], g2[8];
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    const float4 a = *reinterpret_cast<const float4 *>(tab + T_GHI + j0 + j);
                    const float4 b = *reinterpret_cast<const float4 *>(tab + T_GLO + j0 + j);
                    g1[j] = a.x, g1[j + 1] = a.y, g1[j + 2] = a.z, g1[j + 3] = a.w;
                    g2[j] = b.x, g2[j + 1] = b.y, g2[j + 2] = b.z, g2[j + 3] = b.w;
                }
                const int see = keys ? (i < n ? i : 0) : i + 1;      // columns that count
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = ex2((ghi - g1[j]) + (glo - g2[j])) * factor;
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    // masked by choice, not by a factor, which would keep a NaN
                    x[j] = j0 + j < see ? x[j] * __uint_as_float(kq[j]) : 0.f;
                if (keys) {
                    float *to = (qd == 2 ? blk11 : j0 < 32 ? blk21 : blk22) + lane * kBlockStride + (j0 & 31);
                    *reinterpret_cast<float4 *>(to) = make_float4(x[0], x[1], x[2], x[3]);
                    *reinterpret_cast<float4 *>(to + 4) = make_float4(x[4], x[5], x[6], x[7]);
                } else {
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        hi[k] = take_bf16(x[2 * k], x[2 * k + 1]);
                        lo[k] = pack_bf16x2(x[2 * k], x[2 * k + 1]);
                    }
                    const uint32_t at = sw128_off(i, j0 >> 3);
                    *reinterpret_cast<uint4 *>(ph + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(ph + kDeltaPanel + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            tc_fence_before();
            arrive(kq_read);
            if (!together()) break;
            if (gc > 0 && !wait(u_done, gc - 1)) break;              // T's place
            // T11 and T22, a warp each, a lane per column: x_r = [r = lane] - sum_{m < r} A_rm x_m
            if (qd == 0 || qd == 2) {
                float *blk = qd == 2 ? blk11 : blk22;
                const int t0 = qd == 2 ? 0 : 32;
                float x[32];
                x[0] = lane == 0 ? 1.f : 0.f;
#pragma unroll
                for (int q = 1; q < 32; ++q) {
                    float acc[4] = {lane == q ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int m = 0; m < q; m += 4) {
                        const float4 a = *reinterpret_cast<const float4 *>(blk + q * kBlockStride + m);
                        acc[0] = fmaf(-a.x, x[m], acc[0]);
                        if (m + 1 < q) acc[1] = fmaf(-a.y, x[m + 1], acc[1]);
                        if (m + 2 < q) acc[2] = fmaf(-a.z, x[m + 2], acc[2]);
                        if (m + 3 < q) acc[3] = fmaf(-a.w, x[m + 3], acc[3]);
                    }
                    x[q] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
                }
                __syncwarp();
#pragma unroll
                for (int q = 0; q < 32; ++q) {
                    x[q] = lane <= q ? x[q] : 0.f;
                    blk[q * kBlockStride + lane] = x[q];
                }
#pragma unroll
                for (int q = 0; q < 32; q += 2) put_t(t0 + q, 1, t0 + lane, x[q], x[q + 1]);
            }
            if (!together()) break;
            // A21 T11: eight rows a warp, a lane per column
            {
                float t[32];
#pragma unroll
                for (int m = 0; m < 32; ++m) t[m] = blk11[m * kBlockStride + lane];
#pragma unroll 2
                for (int q = qd * 8; q < qd * 8 + 8; ++q) {
                    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int m = 0; m < 32; m += 4) {
                        const float4 a = *reinterpret_cast<const float4 *>(blk21 + q * kBlockStride + m);
                        acc[0] = fmaf(a.x, t[m], acc[0]);
                        acc[1] = fmaf(a.y, t[m + 1], acc[1]);
                        acc[2] = fmaf(a.z, t[m + 2], acc[2]);
                        acc[3] = fmaf(a.w, t[m + 3], acc[3]);
                    }
                    blkx[q * kBlockStride + lane] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
                }
            }
            if (!together()) break;
            // T21 = -T22 (A21 T11): rows qd, qd + 4, ... a warp, as far as T22's triangle goes
            {
                float t[32], y[8];
#pragma unroll
                for (int m = 0; m < 32; ++m) t[m] = blkx[m * kBlockStride + lane];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int m = 0; m <= 4 * k; m += 4) {
                        const float4 a = *reinterpret_cast<const float4 *>(blk22 + (qd + 4 * k) * kBlockStride + m);
                        const bool end = m == 4 * k;     // the triangle ends with column qd of these four
                        acc[0] = fmaf(-a.x, t[m], acc[0]);
                        acc[1] = fmaf(-a.y, end && qd < 1 ? 0.f : t[m + 1], acc[1]);
                        acc[2] = fmaf(-a.z, end && qd < 2 ? 0.f : t[m + 2], acc[2]);
                        acc[3] = fmaf(-a.w, end && qd < 3 ? 0.f : t[m + 3], acc[3]);
                    }
                    y[k] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
                }
#pragma unroll
                for (int k = 0; k < 8; k += 2) put_t(32 + qd + 4 * k, 4, lane, y[k], y[k + 1]);
            }
            fence_proxy_async_smem();
            arrive(t_ready);
            arrive(&tab_free[gc & 1]);
        }
    } else if (warp < 24) {
        // ============================================================ output rows: a warp per 32 value dimensions
        // In 8x8 fragments (thread: two neighbouring tokens of one dv), transposed by stmatrix into the warp's
        // own [64 tokens][32 dv] tile, 16-byte chunks swizzled by token pair.
        fewer_regs<kRowRegs>();
        const int grp = warp & 3, q2 = (lane & 3) * 2;
        const bool real = grp * 32 < D;
        const uint32_t lane_base = tmem + ((uint32_t)(grp * 32) << 16);
        uint8_t *stg = sm + S::kOutOff + grp * DC * 64;
        // stmatrix row address: token (lane / 16) * 8 + lane % 8 of its group, dv chunk lane / 8 % 2
        const int row0 = (lane >> 4) * 8 + (lane & 7), ch0 = (lane >> 3) & 1, sw = (row0 >> 1) & 3;
        const uint32_t stg_at = smem_u32(stg) + row0 * 64;
#pragma unroll 1
        for (int gc = 0;; ++gc) {
            if (!wait(&tab_full[gc & 1], gc >> 1)) break;
            const DeltaChunk *info = info_of(gc);
            const int n = uni(info->n);
            if (n == 0) break;
            const int t0 = info->t0, h = info->h;
            if (!wait(&o_done[gc & 1], gc >> 1)) break;
            tc_fence_after();
            if (!real) {
                arrive(o_read);
                arrive(&tab_free[gc & 1]);
                continue;
            }
            if (lane == 0) bulk_wait_read();             // the tile's last store
            __syncwarp();
            const int first_bad = bad_at[(gc & 1) * 128 + grp * 32 + lane];
            const bool any_bad = __any_sync(0xffffffffu, first_bad < DC);
#pragma unroll 1
            for (int part = 0; part < 4; ++part) {      // 16 dv, 32 tokens
                const int hl = part >> 1, g0 = (part & 1) * 4;
                const uint32_t at = lane_base + ((uint32_t)hl << 20) + g0 * 8;
                uint32_t x[16], y[16], r[8];
                tmem_ld_16x256b_x4(at + TM_PU, x);
                tmem_ld_16x256b_x4(at + TM_SQ, y);
                const float *e = tab_of(gc) + T_F + g0 * 8 + q2;
                tc_wait_ld();
                if (part == 3) {
                    tc_fence_before();
                    arrive(o_read);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {           // tokens 8 (g0 + k / 2) + q2, + 1; dv + 8 (k % 2)
                    const float2 f = *reinterpret_cast<const float2 *>(e + (k / 2) * 8);
                    float o0, o1;
                    fma2(o0, o1, f.x, f.y, __uint_as_float(y[2 * k]), __uint_as_float(y[2 * k + 1]),
                         __uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]));
                    r[k] = pack_bf16x2(o0, o1);
                }
                const uint32_t to = stg_at + (uint32_t)(g0 * 512) + (((hl * 2 + ch0) ^ sw) << 4);
                stsm_x4_t(to, r[0], r[1], r[2], r[3]);
                stsm_x4_t(to + 1024, r[4], r[5], r[6], r[7]);
            }
            arrive(&tab_free[gc & 1]);
            if (any_bad) {
                // NaN from a dv's first non-finite token on
                for (int t = first_bad; t < DC; ++t)
                    *reinterpret_cast<uint16_t *>(stg + t * 64 + (((lane >> 3) ^ ((t >> 1) & 3)) << 4) + (lane & 7) * 2) =
                        0x7FC0;
            }
            __syncwarp();
            if (n == DC) {
                // one store of the tile; its swizzle is the copy engine's for rows of 64 bytes
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_3d(&omap, stg, grp * 32, h, t0);
                    bulk_commit();
                }
            } else {
                // rows behind the sequence stay as they are
                __nv_bfloat16 *out = p.out + (int64_t)t0 * p.out_stride + (int64_t)h * D + grp * 32;
#pragma unroll 1
                for (int t = lane >> 2; t < n; t += 8)
                    *reinterpret_cast<uint4 *>(out + t * p.out_stride + (lane & 3) * 8) =
                        *reinterpret_cast<const uint4 *>(stg + t * 64 + (((lane & 3) ^ ((t >> 1) & 3)) << 4));
                __syncwarp();
            }
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    } else {
        fewer_regs<kOtherRegs>();
        if (warp == 24) {
            // ============================================================ loads
            if (lane == 0) {
                DeltaWalk walk;
                int gc = 0;
                while (walk.step(units, units_n, p.Hv)) {
                    const int s = gc % QS, vs = gc % VS, rw = walk.u.t0 + walk.c * DC, hk = walk.h / p.G;
                    if (gc >= QS && !chunk_wait(&qk_empty[s], (uint32_t)(gc / QS - 1) & 1u, abort_flag)) break;
                    uint8_t *qk = sm + s * S::kQkBytes, *v = sm + S::kVOff + vs * S::kVBytes;
                    mbar_arrive_expect_tx(&qk_full[s], S::kQkBytes);
#pragma unroll 1
                    for (int x = 0; x < PAN; ++x) {
                        tma_load_3d(qk + x * S::kQkPanel + kDeltaPanel, &kmap, &qk_full[s], x * 64, hk, rw);
                        tma_load_3d(qk + x * S::kQkPanel, &qmap, &qk_full[s], x * 64, hk, rw);
                    }
                    // (the barriers below count a chunk's Q and K, then its V)
                    if (gc >= VS && !chunk_wait(&v_empty[vs], (uint32_t)(gc / VS - 1) & 1u, abort_flag)) {
                        chunk_wait(&qk_full[s], (uint32_t)(gc / QS) & 1u, &never);
                        break;
                    }
                    mbar_arrive_expect_tx(&v_full[vs], S::kVBytes);
#pragma unroll 1
                    for (int x = 0; x < PAN; ++x)
                        tma_load_3d(v + x * kDeltaPanel, &vmap, &v_full[vs], x * 64, walk.h, rw);
                    ++gc;
                }
                // copies still in flight (after a wait that gave up) land before the CTA ends
                for (int d = max(0, gc - QS); d < gc; ++d) chunk_wait(&qk_full[d % QS], (uint32_t)(d / QS) & 1u, &never);
                for (int d = max(0, gc - VS); d < gc; ++d) chunk_wait(&v_full[d % VS], (uint32_t)(d / VS) & 1u, &never);
            }
            __syncwarp();
        } else if (warp == 25) {
            // ============================================================ the chunks' tables: two tokens a lane
            DeltaWalk walk;
            const double kLog2e = 1.4426950408889634074;
#pragma unroll 1
            for (int gc = 0;; ++gc) {
                const bool some = walk.step(units, units_n, p.Hv);
                const int n = some ? min(DC, walk.u.n - walk.c * DC) : 0;
                const int64_t t0 = some ? walk.u.t0 + (int64_t)walk.c * DC : 0;
                float g[2] = {0.f, 0.f}, beta[2] = {0.f, 0.f};
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int64_t t = t0 + 2 * lane + x;
                    if (2 * lane + x < n) {
                        g[x] = __ldg(p.log_decay + t * p.decay_stride + walk.h);
                        beta[x] = __ldg(p.beta + t * p.beta_stride + walk.h);
                    }
                }
                if (!(g[0] <= 0.f && g[1] <= 0.f)) record_error(p.err, ERR_RANGE | SRC_DELTA);
                // (e^-256 is 0 in fp32, and so is what is below; -inf - -inf would be NaN)
                const double x0 = (double)fmaxf(fminf(g[0], 0.f), -256.f) * kLog2e;
                const double x1 = (double)fmaxf(fminf(g[1], 0.f), -256.f) * kLog2e;
                double inc = x0 + x1;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const double y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += y;
                }
                const double before = __shfl_up_sync(0xffffffffu, inc, 1);
                const double G0 = (lane ? before : 0.0) + x0, G1 = G0 + x1;
                const double all = __shfl_sync(0xffffffffu, G1, 31);
                if (gc >= 2 && !wait(&tab_free[gc & 1], (gc >> 1) - 1)) break;
                float *tab = tab_of(gc);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int i = 2 * lane + x;
                    const double G = x ? G1 : G0;
                    const float hi = (float)G;
                    tab[T_GHI + i] = hi;
                    tab[T_GLO + i] = (float)(G - (double)hi);
                    tab[T_BETA + i] = beta[x];
                    tab[T_GAM + i] = exp2f(hi);
                    tab[T_W + i] = i < n ? exp2f((float)(all - G)) : 0.f;
                }
                if (lane == 0) {
                    DeltaChunk *info = info_of(gc);
                    // near 1, where a state is multiplied many times before it fades, as two parts
                    const float y = (float)(all * 0.69314718055994530942);
                    float a = exp2f((float)all), a_lo = 0.f;
                    if (y > -0.3f) {
                        const float e = expm1f(y);
                        a = 1.f + e;
                        a_lo = e - (a - 1.f);
                    }
                    info->n = n;
                    info->t0 = (int)t0;
                    info->h = walk.h;
                    info->first = walk.c == 0;
                    info->last = some && walk.c + 1 == walk.chunks;
                    info->slot = some ? walk.u.slot : -1;
                    info->from = some ? walk.u.from : 0;
                    info->a = a;
                    info->a_lo = a_lo;
                }
                arrive(&tab_full[gc & 1]);
                if (!some) break;
            }
        } else if (warp == 26) {
            // ============================================================ MMAs
            auto kq = [&](int gc) {
                if (elect_one()) {
                    const uint64_t qd = sw128_desc(smb + (gc % QS) * S::kQkBytes, 16, 1024);
                    constexpr uint32_t id = idesc_bf16_f32(128, DC, 0);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint64_t d = qd + (k / 4) * (S::kQkPanel >> 4) + (k % 4) * 2;
                        tc_mma_ss(tmem + TM_KQ, d, d + (kDeltaPanel >> 4), id, k > 0);
                    }
                    tc_commit(kq_done);
                }
                __syncwarp();
            };
            // the chunk's tables, and its Q and K, are there; 0: no such chunk, -1: a wait gave up
            auto ready = [&](int gc) {
                if (!wait(&tab_full[gc & 1], gc >> 1)) return -1;
                if (uni(info_of(gc)->n) == 0) return 0;
                return wait(&qk_full[gc % QS], gc / QS) ? 1 : -1;
            };
            // a product whose B is lower triangular: 16 tokens j reach rows from theirs on
            auto triangle = [&](uint32_t d, uint32_t a, uint64_t b, bool add) {
#pragma unroll
                for (int k = 0; k < DC / 16; ++k)
                    tc_mma_ts(tmem + d + 16 * k, tmem + a + k * 8, b + k * 2 + (16 * k * 128 >> 4),
                              idesc_bf16_f32(128, DC - 16 * k, 0), add || k > 0);
            };
            int some = ready(0);
            if (some > 0) {
                tc_fence_after();
                kq(0);
            }
#pragma unroll 1
            for (int gc = 0; some > 0; ++gc) {
                const int s = gc % QS;
                const uint32_t qk = smb + s * S::kQkBytes;
                constexpr uint32_t id = idesc_bf16_f32(128, DC, 0);
                some = -1;
                if (!wait(s_ready, gc)) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t kd = sw128_desc(qk + kDeltaPanel, 16, 1024);
#pragma unroll
                    for (int part = 0; part < 3; ++part) {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            tc_mma_ts(tmem + TM_SK, tmem + (part == 0 ? TM_S1 : part == 1 ? TM_S2 : TM_S3) + k * 8,
                                      kd + (k / 4) * (S::kQkPanel >> 4) + (k % 4) * 2, id, part + k > 0);
                    }
                    tc_commit(sk_done);
                }
                __syncwarp();
                if (gc > 0 && !wait(o_read, gc - 1)) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t qd = sw128_desc(qk, 16, 1024);
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            tc_mma_ts(tmem + TM_SQ, tmem + (part == 0 ? TM_S1 : TM_S2) + k * 8,
                                      qd + (k / 4) * (S::kQkPanel >> 4) + (k % 4) * 2, id, part + k > 0);
                    }
                }
                __syncwarp();
                if (!wait(t_ready, gc)) break;
                if (!wait(r_ready, gc)) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t td = sw128_desc(smb + S::kTOff, 16, 1024);
                    triangle(TM_U, TM_R, td, false);
                    triangle(TM_U, TM_R + 32, td, true);
                    triangle(TM_U, TM_R, td + (kDeltaPanel >> 4), true);
                    triangle(TM_U, TM_R + 64, td, true);
                    triangle(TM_U, TM_R + 32, td + (kDeltaPanel >> 4), true);
                    triangle(TM_U, TM_R, td + (2 * kDeltaPanel >> 4), true);
                    tc_commit(u_done);
                }
                __syncwarp();
                // KQ a chunk ahead, in the time in which w U~ is made
                const int more = ready(gc + 1);
                if (more < 0) break;
                if (more > 0) {
                    if (!wait(kq_read, gc)) break;
                    tc_fence_after();
                    kq(gc + 1);
                }
                if (!wait(w_ready, gc)) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t kd = sw128_desc(qk + kDeltaPanel, S::kQkPanel, 1024);
                    constexpr uint32_t idk = idesc_bf16_f32(128, D, 1);
#pragma unroll
                    for (int part = 0; part < 3; ++part) {
#pragma unroll
                        for (int k = 0; k < DC / 16; ++k)
                            tc_mma_ts(tmem + TM_KV, tmem + TM_R + part * 32 + k * 8, kd + k * (16 * 128 >> 4), idk,
                                      part + k > 0);
                    }
                    tc_commit(kv_done);
                    tc_commit(&qk_empty[s]);
                    const uint64_t pd = sw128_desc(smb + S::kPOff + (gc & 1) * 2 * kDeltaPanel, 16, 1024);
                    triangle(TM_PU, TM_UO, pd, false);
                    triangle(TM_PU, TM_UO + 32, pd, true);
                    triangle(TM_PU, TM_UO, pd + (kDeltaPanel >> 4), true);
                    tc_commit(&o_done[gc & 1]);
                }
                arrive(&tab_free[gc & 1]);
                some = more;
            }
            // nothing of this CTA's is left in the tensor core when TMEM goes back
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
    if (threadIdx.x == 0 && (abort_flag[0] | abort_flag[1])) record_error(p.err, ERR_TIMEOUT | SRC_DELTA);
}

template <int D>
cudaError_t launch_delta_chunks(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap,
                                const CUtensorMap &omap, const DeltaParams &p, cudaStream_t stream) {
    using S = DeltaSmem<D>;
    static std::once_flag once[kMaxDev];
    static cudaError_t attr_err[kMaxDev];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDev) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [&] {
        attr_err[dev] =
            cudaFuncSetAttribute(delta_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
    });
    if (attr_err[dev] != cudaSuccess) return attr_err[dev];
    delta_plan_kernel<<<1, 1024, 0, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // a CTA per SM at most: each goes over several units
    const unsigned ctas = (unsigned)min((int64_t)p.batch * p.Hv, (int64_t)p.num_sms);
    main_kernel_event_before(stream);
    e = launch_after(delta_chunk_kernel<D>, dim3(ctas), kDeltaThreads, S::kBytes, stream, qmap, kmap, vmap, omap, p);
    main_kernel_event_after(stream);
    return e;
}

}  // namespace

cudaError_t launch_delta_recurrent(const DeltaParams &p, cudaStream_t stream) {
    const int64_t states = (int64_t)p.batch * p.Hv;
    auto *kernel = p.D == 128 ? p.cu ? delta_recurrent_kernel<128, true> : delta_recurrent_kernel<128, false>
                              : p.cu ? delta_recurrent_kernel<64, true> : delta_recurrent_kernel<64, false>;
    main_kernel_event_before(stream);
    kernel<<<(unsigned)(p.D == 128 ? states * 4 : states), kRecWarps * 32, 0, stream>>>(p);
    main_kernel_event_after(stream);
    return cudaGetLastError();
}

cudaError_t launch_delta_varlen(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap,
                                const CUtensorMap &omap, const DeltaParams &p, cudaStream_t stream) {
    return p.D == 128 ? launch_delta_chunks<128>(qmap, kmap, vmap, omap, p, stream)
                      : launch_delta_chunks<64>(qmap, kmap, vmap, omap, p, stream);
}

}  // namespace attn
