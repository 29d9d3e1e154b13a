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

// e^{log_decay}: a positive or NaN log_decay counts as 0 and is reported.
__device__ __forceinline__ float delta_decay(const DeltaParams &p, float g, bool report) {
    if (report && !(g <= 0.f)) record_error(p.err, ERR_RANGE | SRC_DELTA);
    return expf(fminf(g, 0.f));
}

// 1 / sqrt(x): the hardware's estimate and one step of Newton's method
__device__ __forceinline__ float inv_sqrt(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return x > 0.f ? y * fmaf(-0.5f * x * y, y, 1.5f) : y;
}

// sums over the LPR lanes of a row, in every lane
template <int LPR> __device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int w = LPR / 2; w > 0; w /= 2) x += __shfl_xor_sync(0xffffffffu, x, w);
    return x;
}

// ---------------------------------------------------------------------------
// The recurrent form.  S stays in registers and is read and written once, whatever the
// number of tokens, 8 D^2 bytes per sequence and value head, which bounds it (HBM).
// With S k and S q of the state before the token,
//   S_t q = e^g S q + u (k . q),
// so one reduction per token serves u and the output.
//
// One token: a lane holds four neighbouring columns of eight rows, a warp 32 lanes / (D / 4) times eight
// rows.  The sums of the eight rows are reduced together (9 shuffles), S k is
// then handed back to all lanes (7).  PACKED: packed sequences of at most one token; a sequence
// without one leaves its state as it was.  256 sequences, 32 heads of 128: 159 us, 6.8 TB/s.
// ---------------------------------------------------------------------------
constexpr int kRecRows = 8;
constexpr int kRecWarps = 4;

template <int D, bool PACKED>
__global__ void __launch_bounds__(kRecWarps * 32, 5) delta_one_kernel(const DeltaParams p) {
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
    const uint2 kr = *reinterpret_cast<const uint2 *>(p.k + t * p.k_stride + (int64_t)hk * D + col);
    const uint2 qr = *reinterpret_cast<const uint2 *>(p.q + t * p.q_stride + (int64_t)hk * D + col);
    const uint4 vr = *reinterpret_cast<const uint4 *>(p.v + t * p.v_stride + (int64_t)h * D + row0);
    const float beta = __ldg(p.beta + t * p.beta_stride + h);
    const float a = delta_decay(p, __ldg(p.log_decay + t * p.decay_stride + h), first_thread);
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
        if (state) __stcs(reinterpret_cast<float4 *>(state + (row0 + i) * D + col), S[i]);
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

// x0, x1 as three bf16 parts
__device__ __forceinline__ void split3(float x0, float x1, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    float r0, r1;
    hi = take_bf16(r0, r1, x0, x1);
    mid = take_bf16(r0, r1);
    lo = pack_bf16x2(r0, r1);
}

// four 8 x 8 matrices of 16-bit elements, their rows' addresses by lane
__device__ __forceinline__ void four_8x8(uint32_t (&r)[4], const void *at) { ldsm_x4(smem_u32(at), r[0], r[1], r[2], r[3]); }
// D = A(16x8, row) * B(8x8, col) + D
__device__ __forceinline__ void mma_bf16_16808(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(b0));
}

// Two to kDeltaShort tokens, n, without a product that waits for the one before: with k and q normalised (and q scaled),
// E_i the decay from the start to token i and R_ij the one from j to i,
//   u_i = beta_i (v_i - E_i S_0 k_i - sum_{j < i} R_ij k_i.k_j u_j),
//   o_i = E_i S_0 q_i + sum_{j <= i} R_ij q_i.k_j u_j,   S = E_n S_0 + sum_j R_nj u_j k_j^T,
// the decays as products of the tokens' own, so that small ones cost nothing.  The products go through mma.sync, with k
// and q as they come (bf16, exact; norms and decays are factors of the sums) and S_0 and u as three bf16 parts, 2^-24 of
// them, S_0 as two for the output.  A warp has 16 rows, S in the fragments' order with the columns of 16 permuted so that
// a lane's four are neighbours; a lane per row then solves for u.  NT: room for tokens, 8 or 16.  HBM bounds 64 sequences
// of 5 tokens, 32 heads of 128: 54 us (72 token after token, 60 by fp32 products; 41 for the states alone).  96 of 16
// tokens, 122 us (224 by fp32 products, 257 as a chunk; 65 for what is read and written): shared memory 68 % busy, DRAM
// 41 %, four warps a scheduler that wait for both.
template <int D, int NT>
__global__ void __launch_bounds__(kRecWarps * 32, 4) delta_few_kernel(const DeltaParams p) {
    constexpr int ROWS = 16, OWN = ROWS * kRecWarps, CTAS = D / OWN;    // rows of a warp, of a CTA; CTAs per state
    constexpr int KS = D / 16, LPT = D / 8;                             // steps of 16 columns; lanes per token
    __shared__ __align__(16) uint16_t k_s[NT][D + 8], q_s[NT][D + 8];   // columns permuted
    __shared__ float v_s[NT][OWN], sk_s[kRecWarps][NT][ROWS], sq_s[kRecWarps][NT][ROWS], u_s[kRecWarps][NT][ROWS];
    __shared__ float kk_s[NT][NT], qk_s[NT][NT];                        // R k.k, R q.k
    __shared__ float a_s[NT], beta_s[NT], rk_s[NT], rq_s[NT], ek_s[NT], eq_s[NT], w_s[NT], en_s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & (LPT - 1);
    const int g = lane >> 2, t = lane & 3;                              // of a fragment: row or token, pair of columns
    const int unit = blockIdx.x / CTAS, b = unit / p.Hv, h = unit - b * p.Hv, hk = h / p.G;
    const int cta_row = (blockIdx.x - unit * CTAS) * OWN, row0 = cta_row + warp * ROWS;
    const bool first_cta = cta_row == 0, report = h == 0 && first_cta && threadIdx.x == 0;
    int64_t t0;
    int n;
    sequence_rows<SRC_DELTA>(p, b, t0, n, report);
    bool from;
    float *state = sequence_state<SRC_DELTA, true>(p, p.Hv, b, h, from, report && n > 0);
    if (n == 0) return;
    // loads in the order of their use: LPT lanes per token with eight columns each, eight threads per token's values; S
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    uint4 kr, qr, vr = none;
    float decay, beta;
    auto load = [&](int i) {
        kr = qr = none;
        decay = beta = 0.f;
        if (i < n) {
            const int64_t at = t0 + i;
            kr = *(reinterpret_cast<const uint4 *>(p.k + at * p.k_stride + (int64_t)hk * D) + l);
            qr = *(reinterpret_cast<const uint4 *>(p.q + at * p.q_stride + (int64_t)hk * D) + l);
            beta = __ldg(p.beta + at * p.beta_stride + h);
            decay = __ldg(p.log_decay + at * p.decay_stride + h);
        }
    };
    load(warp * (32 / LPT) + lane / LPT);
    static_assert(OWN == 64 && NT * 8 <= kRecWarps * 32, "values");
    const int vi = threadIdx.x >> 3, vc = threadIdx.x & 7;
    if (vi < n) vr = *(reinterpret_cast<const uint4 *>(p.v + (t0 + vi) * p.v_stride + (int64_t)h * D + cta_row) + vc);
    float4 S[KS][2];                                    // rows g, g + 8; columns 16 s + 4 t ..
#pragma unroll
    for (int s = 0; s < KS; ++s) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            S[s][r] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (from) S[s][r] = __ldcs(reinterpret_cast<const float4 *>(state + (row0 + g + 8 * r) * D + 16 * s) + t);
        }
    }
    for (int i0 = warp * (32 / LPT); i0 < NT; i0 += kRecWarps * 32 / LPT) {
        const int i = i0 + lane / LPT;
        if (i0 >= kRecWarps * 32 / LPT) load(i);
        float rk = 1.f, rq = p.scale;
        if (p.norm) {
            const uint32_t kw[4] = {kr.x, kr.y, kr.z, kr.w}, qw[4] = {qr.x, qr.y, qr.z, qr.w};
            float ks = 0.f, qs = 0.f;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float k0 = __uint_as_float(kw[x] << 16), k1 = __uint_as_float(kw[x] & 0xFFFF0000u);
                const float q0 = __uint_as_float(qw[x] << 16), q1 = __uint_as_float(qw[x] & 0xFFFF0000u);
                ks = fmaf(k0, k0, fmaf(k1, k1, ks)), qs = fmaf(q0, q0, fmaf(q1, q1, qs));
            }
            rk = inv_sqrt(row_sum<LPT>(ks) + p.eps);
            rq = p.scale * inv_sqrt(row_sum<LPT>(qs) + p.eps);
        }
        // columns 4 t, 4 t + 1 of 16 at 2 t, 2 t + 1; 4 t + 2, 4 t + 3 at 8 + 2 t, 8 + 2 t + 1
        const int at = (l >> 1) * 16 + (l & 1) * 4;
        *reinterpret_cast<uint2 *>(&k_s[i][at]) = make_uint2(kr.x, kr.z);
        *reinterpret_cast<uint2 *>(&k_s[i][at + 8]) = make_uint2(kr.y, kr.w);
        *reinterpret_cast<uint2 *>(&q_s[i][at]) = make_uint2(qr.x, qr.z);
        *reinterpret_cast<uint2 *>(&q_s[i][at + 8]) = make_uint2(qr.y, qr.w);
        if (l == 0) a_s[i] = delta_decay(p, decay, first_cta), beta_s[i] = beta, rk_s[i] = rk, rq_s[i] = rq;
    }
    if (vi < n) {
        float4 *to = reinterpret_cast<float4 *>(v_s[vi]) + 2 * vc;
        to[0] = make_float4(__uint_as_float(vr.x << 16), __uint_as_float(vr.x & 0xFFFF0000u), __uint_as_float(vr.y << 16),
                            __uint_as_float(vr.y & 0xFFFF0000u));
        to[1] = make_float4(__uint_as_float(vr.z << 16), __uint_as_float(vr.z & 0xFFFF0000u), __uint_as_float(vr.w << 16),
                            __uint_as_float(vr.w & 0xFFFF0000u));
    }
    __syncthreads();
    // k_i.k_j (even warps), q_i.k_j (odd ones), eight j a warp
    if ((warp >> 1) * 8 < NT) {
        const bool of_q = warp & 1;
        const int j0 = (warp >> 1) * 8 + 2 * t, lr = lane & 7, lc = (lane >> 3) * 8;
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; s += 2) {
            uint32_t lo[4], hi[4] = {0u, 0u, 0u, 0u}, kj[4];
            four_8x8(lo, of_q ? &q_s[lr][s * 16 + lc] : &k_s[lr][s * 16 + lc]);
            if (NT == 16) four_8x8(hi, of_q ? &q_s[NT - 8 + lr][s * 16 + lc] : &k_s[NT - 8 + lr][s * 16 + lc]);
            four_8x8(kj, &k_s[(warp >> 1) * 8 + lr][s * 16 + lc]);
            mma_bf16_16816(c, lo[0], hi[0], lo[1], hi[1], kj[0], kj[1]);
            mma_bf16_16816(c, lo[2], hi[2], lo[3], hi[3], kj[2], kj[3]);
        }
        const float rj0 = rk_s[j0], rj1 = rk_s[j0 + 1];
#pragma unroll
        for (int r = 0; r < NT / 8; ++r) {
            const int i = g + 8 * r;
            if (i < n && j0 <= i) {
                const float ri = of_q ? rq_s[i] : rk_s[i];
                float *to = of_q ? qk_s[i] : kk_s[i];
                float x = 1.f;                          // R of j0 + 1, then of j0
                for (int m = i; m > j0 + 1; --m) x *= a_s[m];
                if (j0 < i) {
                    to[j0 + 1] = c[2 * r + 1] * x * ri * rj1;
                    x *= a_s[j0 + 1];
                }
                to[j0] = c[2 * r] * x * ri * rj0;
            }
        }
    }
    if (const int i = (int)threadIdx.x - (kRecWarps * 32 - NT); i >= 0 && i < n) {
        float e = 1.f, w = 1.f;
        for (int m = 0; m <= i; ++m) e *= a_s[m];
        for (int m = i + 1; m < n; ++m) w *= a_s[m];
        ek_s[i] = e * rk_s[i], eq_s[i] = e * rq_s[i], w_s[i] = w * rk_s[i];
        if (i == n - 1) en_s = e;
    }
    // S_0 k and S_0 q
    {
        float ck[NT / 8][4] = {}, cq[NT / 8][4] = {};
#pragma unroll
        for (int s = 0; s < KS; s += 2) {
            uint32_t kb[NT / 8][4], qb[NT / 8][4];
#pragma unroll
            for (int x = 0; x < NT / 8; ++x) {
                four_8x8(kb[x], &k_s[8 * x + (lane & 7)][s * 16 + (lane >> 3) * 8]);
                four_8x8(qb[x], &q_s[8 * x + (lane & 7)][s * 16 + (lane >> 3) * 8]);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                uint32_t a[3][4];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    split3(S[s + y][r].x, S[s + y][r].y, a[0][r], a[1][r], a[2][r]);
                    split3(S[s + y][r].z, S[s + y][r].w, a[0][2 + r], a[1][2 + r], a[2][2 + r]);
                }
#pragma unroll
                for (int part = 2; part >= 0; --part) {
#pragma unroll
                    for (int x = 0; x < NT / 8; ++x) {
                        mma_bf16_16816(ck[x], a[part][0], a[part][1], a[part][2], a[part][3], kb[x][2 * y], kb[x][2 * y + 1]);
                        if (part < 2)
                            mma_bf16_16816(cq[x], a[part][0], a[part][1], a[part][2], a[part][3], qb[x][2 * y],
                                           qb[x][2 * y + 1]);
                    }
                }
            }
        }
#pragma unroll
        for (int x = 0; x < NT / 8; ++x) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                sk_s[warp][8 * x + 2 * t + (y & 1)][g + 8 * (y >> 1)] = ck[x][y];
                sq_s[warp][8 * x + 2 * t + (y & 1)][g + 8 * (y >> 1)] = cq[x][y];
            }
        }
    }
    __syncthreads();
    // a lane per row
    if (lane < ROWS) {
        __nv_bfloat16 *out = p.out + t0 * p.out_stride + (int64_t)h * D + row0 + lane;
        float u[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            float last = 0.f;
            if (i < n) {
                float x = fmaf(-ek_s[i], sk_s[warp][i][lane], v_s[i][warp * ROWS + lane]), o = eq_s[i] * sq_s[warp][i][lane];
#pragma unroll
                for (int j = 0; j < i; ++j) {
                    x = fmaf(-kk_s[i][j], u[j], x);
                    o = fmaf(qk_s[i][j], u[j], o);
                }
                u[i] = beta_s[i] * x;
                o = fmaf(qk_s[i][i], u[i], o);
                out[i * p.out_stride] = __float2bfloat16_rn(o);
                last = w_s[i] * u[i];
            }
            u_s[warp][i][lane] = last;
        }
    }
    if (!state) return;
    __syncwarp();
    const float e = en_s;
    uint32_t u[3][NT / 4];                              // rows g, g + 8; tokens 2 t, 2 t + 1, then those behind 8
#pragma unroll
    for (int x = 0; x < NT / 4; ++x) {
        const int i = 2 * t + 8 * (x >> 1), r = g + 8 * (x & 1);
        split3(u_s[warp][i][r], u_s[warp][i + 1][r], u[0][x], u[1][x], u[2][x]);
    }
#pragma unroll
    for (int s = 0; s < KS; s += NT == 8 ? 2 : 1) {
        uint32_t kb[4];                                 // columns of 8: four of 8 tokens, two of 16
        if (NT == 8) ldsm_x4_t(smem_u32(&k_s[lane & 7][s * 16 + (lane >> 3) * 8]), kb[0], kb[1], kb[2], kb[3]);
        else ldsm_x4_t(smem_u32(&k_s[(lane & 15) & (NT - 1)][s * 16 + (lane >> 4) * 8]), kb[0], kb[1], kb[2], kb[3]);
#pragma unroll
        for (int x = 0; x < (NT == 8 ? 4 : 2); ++x) {
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int part = 2; part >= 0; --part) {
                if (NT == 8) mma_bf16_16808(c, u[part][0], u[part][1], kb[x]);
                else mma_bf16_16816(c, u[part][0], u[part][1], u[part][NT / 4 - 2], u[part][NT / 4 - 1], kb[(2 * x) & 3],
                                    kb[(2 * x + 1) & 3]);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float4 &y = S[s + x / 2][r];
                if (x & 1) fma2(y.z, y.w, e, e, y.z, y.w, c[2 * r], c[2 * r + 1]);
                else fma2(y.x, y.y, e, e, y.x, y.y, c[2 * r], c[2 * r + 1]);
            }
        }
    }
#pragma unroll
    for (int s = 0; s < KS; ++s) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
            __stcs(reinterpret_cast<float4 *>(state + (row0 + g + 8 * r) * D + 16 * s) + t, S[s][r]);
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
//   U  [dv, i]  = R^T T^T        TMEM (three parts) x shared (three parts): the six products above 2^-24
//   KV [dv, dk] = (w_j U~)^T K   TMEM (three parts) x shared,  w_j = e^{G_n - G_j}
//   PU [dv, i]  = U~^T P^T       TMEM (two parts) x shared (two parts)
//
// Precision.  q, k and v are bf16 and exact.  The state, R, T and w U~ are fp32 values in three bf16 parts,
// 2^-24 of each; S itself stays in fp32 registers.  What only reaches the bf16 output (S_0 and U~
// there, P) is taken as two parts, 2^-16 of a term against the output's own 2^-8.  T is solved for
// in fp32: its 16 x 16 diagonal blocks column by column, then the blocks below pairs of them, of
// 16 and of 32, as -T22 A21 T11 (by mma.sync, which waits behind the chain's products, slower).  Sums of decays are in 64
// bits and differences of them kept as two fp32 parts.
//
// What bounds it: a chunk takes 9,000 to 9,500 clocks, as does the next chunk's T beside the chain S -> SK -> R -> U ->
// w U~ -> KV -> S (2,900 in its products, the rest in the warps that split operands into parts); the schedulers they share
// are busy 59 % of the time and saturated where both run, the tensor core 33 %.  SQ, KQ and PU run in the chain's
// gaps.  34,053 tokens in 16 prompts, 32 heads of 128: 573 us (token after token 10,600); 32,768 tokens of one, 16
// heads: 787 us in segments, 2,240 in one piece (35,000); 96 prompts of 1 to 150 tokens, 16 heads of 64: 93 us.
//
// Roles (32 warps, one CTA per SM that goes over (sequence, value head) units):
//   0..15   the chain: thread = value dimension and a quarter of dk or of the tokens; S in registers
//   16..23  T and P of the next chunk
//   24..27  norms of the next chunk, output rows of the one before
//   28, 29  issue the loads; write the chunks' tables
//   30, 31  issues the MMAs; waits for the chain (a warp of it that polled would take its time and issue slots)
// The roles share the SM's instruction cache, and their code is larger than it: one code site per kind of step, loops
// where a step repeats, and waits of a few instructions.
// ---------------------------------------------------------------------------
constexpr int DC = 64;                       // tokens of a chunk
constexpr int kDeltaThreads = 32 * 32;
constexpr int kChainSync = 17 * 32;          // the chain's warps and the one that waits for them
constexpr int kDeltaPanel = DC * 128;        // 64 rows x 128 bytes
// TMEM columns.  In turn in the same place: SK, U and then KV; S_0's third part, R and then w U~; S_0's first
// part and then U~'s two; S_0's second part and then KQ of the next chunk
constexpr uint32_t TM_KV = 0, TM_SK = 0, TM_U = 64;
constexpr uint32_t TM_S1 = 128, TM_UO = 128, TM_KQ = 192;    // (S_0: three parts of 64 columns)
constexpr uint32_t TM_R = 256;               // (three parts of 32 columns)
constexpr uint32_t TM_SQ = 352, TM_PU = 416;
constexpr int kAStride = 68;                 // floats of a row of A^T, and of T's and the products' rows
constexpr int kDeltaBuckets = 256;

// A chunk as its roles read it, behind its tables.
struct DeltaChunk {
    int n;                            // tokens; 0: there is no such chunk
    int t0, h, first;                 // first row; head; whether the unit starts with it
    float a, a_lo;                    // e^{G_n} in two parts
    int bad;                          // the first token whose row of A is not finite
    int ident;                        // the unit starts from the identity and has no values
    const float *src;                 // first chunk: the unit's state (null: zero, or the identity)
    float *dst;                       // last chunk: where the state goes (null: nowhere)
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
    static constexpr int kAOff = kOutOff + 4 * DC * 64;          // A^T, block by block replaced by T^T
    static constexpr int kTabOff = kAOff + DC * kAStride * 4;
    // three chunks' tables: G (two parts), beta, e^G, w, b, -c, f, P's row factors, and the chunk itself
    static constexpr int kTabs = 3, kTabFloats = 9 * DC + 16;
    static constexpr int kBadOff = kTabOff + kTabs * kTabFloats * 4;     // first non-finite token per dv, two chunks
    static constexpr int kBarOff = kBadOff + 2 * 128 * 4;
    static constexpr int kNumBars = 30;
    static constexpr int kBytes = kBarOff + kNumBars * 8 + 32 + 1024 /* alignment slack */;
    static_assert(kBytes <= 227 * 1024 && sizeof(DeltaChunk) <= 64, "shared memory");
    // scratch of the solve, where T goes in the end
    static_assert(DC * kAStride * 4 <= 3 * kDeltaPanel, "scratch");
};

// Registers of the calling warpgroup.  The kernel is launched with 64 a thread; the eight warpgroups'
// shares add up to that: chain 4, T and P 2 (which keep theirs), output rows, the others.
constexpr int kChainRegs = 72, kSolveRegs = 64, kRowRegs = 56, kOtherRegs = 40;
static_assert(4 * kChainRegs + 2 * kSolveRegs + kRowRegs + kOtherRegs == 8 * 64, "register shares");

// A unit's entry in the work list, as the plan writes it.
struct alignas(16) DeltaUnit {
    int t0, n;          // first token, tokens
    int slot, from;     // state slot (-1: none), whether the sequence starts from it
    int row;            // its place among the workspace's states (-1: none)
    int last, more;     // holds the sequence's last token; has a successor
    int head;           // first segment: the sequence's segments, else 0
};
static_assert(sizeof(DeltaUnit) == kDeltaUnitBytes, "workspace layout");

// The work list: a unit is a sequence, or a segment of seg_len tokens of a longer one; the longest come first.
__global__ void __launch_bounds__(1024) delta_plan_kernel(const DeltaParams p) {
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x;
    __shared__ int count[kDeltaBuckets], rows_s;
    for (int i = tid; i < kDeltaBuckets; i += 1024) count[i] = 0;
    if (tid == 0) rows_s = 0;
    __syncthreads();
    const int most = max(1, min(p.seg_len, p.max_seqlen));
    auto bucket = [&](int tokens) { return kDeltaBuckets - 1 - (int)((int64_t)tokens * (kDeltaBuckets - 1) / most); };
    for (int pass = 0; pass < 2; ++pass) {
        for (int b = tid; b < p.batch; b += 1024) {
            int64_t t0;
            int n;
            sequence_rows<SRC_DELTA>(p, b, t0, n, pass == 0);
            if (n == 0) continue;
            const int segs = (n + p.seg_len - 1) / p.seg_len, tail = n - (segs - 1) * p.seg_len;
            if (pass == 0) {
                if (segs > 1) atomicAdd(&count[bucket(p.seg_len)], segs - 1);
                atomicAdd(&count[bucket(tail)], 1);
                continue;
            }
            bool from;
            const float *state = sequence_state<SRC_DELTA, true>(p, p.Hv, b, 0, from, true);
            const int slot = state ? __ldg(p.slots + b) : -1;
            int row = segs > 1 ? atomicAdd(&rows_s, segs) : -1;
            // offsets that overlap can ask for more than the workspace was sized for
            bool fits = row + segs <= p.state_rows || segs == 1;
            if (!fits) row = -1;
            for (int i = 0; i < segs; ++i) {
                const bool end = i == segs - 1;
                const int at = atomicAdd(&count[bucket(end ? tail : p.seg_len)], 1);
                if (at < p.max_units && (row >= 0 || segs == 1))
                    reinterpret_cast<DeltaUnit *>(p.units)[at] =
                        DeltaUnit{(int)t0 + i * p.seg_len, end ? tail : p.seg_len, slot, from, row < 0 ? -1 : row + i, end,
                                  !end, i == 0 ? segs : 0};
                else {
                    fits = false;
                    // (left out: an entry without tokens)
                    if (at < p.max_units) reinterpret_cast<DeltaUnit *>(p.units)[at] = DeltaUnit{0, 0, -1, 0, -1, 0, 0, 0};
                }
            }
            if (!fits) record_error(p.err, ERR_INDEX | SRC_DELTA);
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
            if (tid == 0) *p.unit_count = min(base, p.max_units);
        }
        __syncthreads();
    }
}

// The states at the starts of a sequence's segments, in place of what the segments make of a zero state
// (`own`): with `turn` what they make of the identity,
//   start_0 = the cached state or 0,  start_{s+1} = start_s turn_s + own_s.
// A CTA has 16 rows of a head's state: rows do not meet.  Its threads have four rows of four columns each, and one half
// of them every other 16 terms of a sum; the turns come through a ring, ahead over the segments' ends.  The turns of 8 of 9
// segments, 16 heads of 128: 42 us (144 with the turns read where they are used).
constexpr int kJoinRows = 32, kJoinStages = 4;          // rows of a turn in a place of the ring; its places
template <int D>
__global__ void __launch_bounds__(2 * D) delta_join_kernel(const DeltaParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if ((int)blockIdx.x >= *p.unit_count) return;
    const DeltaUnit e = reinterpret_cast<const DeltaUnit *>(p.units)[blockIdx.x];
    if (e.head == 0 || e.row < 0) return;
    constexpr int COLS = D / 4, BLOCKS = D / kJoinRows;  // float4 columns; ring places of a turn
    extern __shared__ float4 ring[];                    // [place][row][column], then start and the other half's sums
    float4 *start = ring + kJoinStages * kJoinRows * COLS, *sums = start + 16 * COLS;      // [row][column]
    const int tid = threadIdx.x, half = tid / D, col = tid % COLS, r0 = tid % D / COLS * 4;
    const int64_t step = (int64_t)p.Hv * D * D / 4, at = (int64_t)(blockIdx.z * 16 + r0) * COLS + col;
    const int h = blockIdx.y;
    float4 *own = reinterpret_cast<float4 *>(p.states) + ((int64_t)e.row * p.Hv + h) * D * COLS + at;
    const float4 *turn = reinterpret_cast<const float4 *>(p.states) + ((int64_t)(p.state_rows + e.row) * p.Hv + h) * D * COLS;
    const int blocks = (e.head - 1) * BLOCKS;
    auto fetch = [&](int i) {
        if (i < blocks) {
            const float4 *src = turn + i / BLOCKS * step + i % BLOCKS * kJoinRows * COLS;
            const uint32_t to = smem_u32(ring + i % kJoinStages * kJoinRows * COLS);
#pragma unroll
            for (int x = 0; x < kJoinRows * COLS / (2 * D); ++x) {
                const int y = x * 2 * D + tid;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + y * 16), "l"(src + y) : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kJoinStages - 1; ++i) fetch(i);
    float4 run[4], next[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        run[r] = next[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (half) continue;
        if (e.from)
            run[r] = reinterpret_cast<const float4 *>(p.state)[((int64_t)e.slot * p.Hv + h) * D * COLS + at + r * COLS];
        next[r] = own[r * COLS];
    }
    for (int s = 0, i = 0;; ++s, own += step) {
        if (!half) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                own[r * COLS] = run[r];
                start[(r0 + r) * COLS + col] = run[r];
                run[r] = next[r];
                if (s + 2 < e.head) next[r] = own[step + r * COLS];
            }
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) run[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (s + 1 == e.head) break;
#pragma unroll 1
        for (int k0 = 0; k0 < D; k0 += kJoinRows, ++i) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kJoinStages - 2) : "memory");
            __syncthreads();                            // its copies are there; the place before is read
            fetch(i + kJoinStages - 1);
            const float4 *m = ring + (i % kJoinStages * kJoinRows + half * (kJoinRows / 2)) * COLS + col;
            const float4 *x = start + r0 * COLS + (k0 + half * (kJoinRows / 2)) / 4;
#pragma unroll
            for (int k = 0; k < kJoinRows / 2; k += 4) {
                const float4 m0 = m[k * COLS], m1 = m[(k + 1) * COLS], m2 = m[(k + 2) * COLS], m3 = m[(k + 3) * COLS];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float4 y = x[r * COLS + k / 4];
                    fma2(run[r].x, run[r].y, y.x, y.x, m0.x, m0.y, run[r].x, run[r].y);
                    fma2(run[r].z, run[r].w, y.x, y.x, m0.z, m0.w, run[r].z, run[r].w);
                    fma2(run[r].x, run[r].y, y.y, y.y, m1.x, m1.y, run[r].x, run[r].y);
                    fma2(run[r].z, run[r].w, y.y, y.y, m1.z, m1.w, run[r].z, run[r].w);
                    fma2(run[r].x, run[r].y, y.z, y.z, m2.x, m2.y, run[r].x, run[r].y);
                    fma2(run[r].z, run[r].w, y.z, y.z, m2.z, m2.w, run[r].z, run[r].w);
                    fma2(run[r].x, run[r].y, y.w, y.w, m3.x, m3.y, run[r].x, run[r].y);
                    fma2(run[r].z, run[r].w, y.w, y.w, m3.z, m3.w, run[r].z, run[r].w);
                }
            }
        }
        if (half) {
#pragma unroll
            for (int r = 0; r < 4; ++r) sums[(r0 + r) * COLS + col] = run[r];
        }
        __syncthreads();
        if (!half) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float4 y = sums[(r0 + r) * COLS + col];
                run[r].x += y.x, run[r].y += y.y, run[r].z += y.z, run[r].w += y.w;
            }
        }
    }
}
template <int D> constexpr int kJoinBytes = (kJoinStages * kJoinRows + 2 * 16) * D * 4;

// x as a value that the compiler takes for a new one: what is computed from it stays where it is used.  Addresses
// kept from chunk to chunk would leave a phase's own loads too few registers to be in flight together.
__device__ __forceinline__ int renew(int x) {
    asm volatile("" : "+r"(x));
    return x;
}

// The chunks of a CTA's units, in order: places blockIdx.x, 2 gridDim.x - 1 - blockIdx.x, 2 gridDim.x + blockIdx.x, ...
// of the list (longest first), back and forth so that the CTAs' sums come out alike; walked without a division.
struct DeltaWalk {
    int heads, units_n, up_q, up_r, down_q, down_r;      // to the next place: unit and head
    int at, hd, place;                                   // the next unit's
    int left, row, h;                                    // this chunk on: tokens of its unit, first row, head
    const DeltaUnit *unit;                               // its unit
    bool first;
    __device__ __forceinline__ DeltaWalk(int units_n, int heads) : heads(heads), units_n(units_n) {
        const int up = 2 * ((int)gridDim.x - 1 - (int)blockIdx.x) + 1, down = 2 * (int)blockIdx.x + 1;
        up_q = up / heads, up_r = up - up_q * heads, down_q = down / heads, down_r = down - down_q * heads;
        at = (int)blockIdx.x / heads, hd = (int)blockIdx.x - at * heads, place = left = 0;
    }
    // to the next chunk (local: of the units that have a successor alone); its tokens, 0: there is none
    __device__ __forceinline__ int step(const DeltaUnit *units, bool local) {
        if (left > DC) {
            left -= DC, row += DC, first = false;
            return min(left, DC);
        }
        left = 0;
        while (left == 0 && at < units_n) {
            unit = units + at;
            if (!local || unit->more) left = unit->n;
            row = unit->t0, h = hd, first = true;
            at += place & 1 ? down_q : up_q;
            hd += place & 1 ? down_r : up_r;
            if (hd >= heads) hd -= heads, ++at;
            ++place;
        }
        return min(left, DC);
    }
};

// non-finite entries among x[from + 4 g], x[from + 4 g + 1] become 0; returns the first one's 4 g or 4 g + 1, 16 if there
// is none
__device__ __forceinline__ int drop_non_finite(float (&x)[16], int from) {
    int first = 16;
#pragma unroll
    for (int g = 12; g >= 0; g -= 4) {
#pragma unroll
        for (int e = 1; e >= 0; --e) {
            const bool bad = !(fabsf(x[from + g + e]) < INFINITY);
            first = bad ? g + e : first;
            x[from + g + e] = bad ? 0.f : x[from + g + e];
        }
    }
    return first;
}

// LOCAL: the pass over the segments that have a successor, without outputs: what each makes of a zero state
// (heads 0 .. Hv - 1) and of the identity without values (heads Hv ..) goes to the workspace.
template <int D, bool LOCAL>
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
    const int units_n = uni(*p.unit_count), heads = LOCAL ? 2 * p.Hv : p.Hv;
    if ((int)blockIdx.x >= units_n * heads) return;

    const uint32_t smb = (smem_u32(dsmem_raw) + 1023u) & ~1023u;          // shared-memory address, for descriptors
    uint8_t *sm = dsmem_raw + (smb - smem_u32(dsmem_raw));
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + S::kBarOff);
    uint64_t *qk_full = bars, *qk_empty = bars + 3;
    uint64_t *v_full = bars + 6, *v_empty = bars + 8;
    uint64_t *tab_full = bars + 10, *tab_free = bars + 13;   // [3], by chunk: its tables are written, read for the last time
    uint64_t *norms = bars + 16;             // [2]: b, c and f are written too
    uint64_t *o_done = bars + 18;            // [2]: SQ and PU done
    uint64_t *kq_done = bars + 20;           // KQ done
    uint64_t *kq_read = bars + 21;           // ... and read
    uint64_t *t_ready = bars + 22;           // T and P in shared memory
    uint64_t *go = bars + 23;                // [2]: SK, then U done
    uint64_t *s_ready = bars + 25;           // S_0 in TMEM, the KV before read
    uint64_t *x_ready = bars + 26;           // R, then U~ and w U~ in TMEM
    uint64_t *kv_done = bars + 27;
    uint64_t *o_read = bars + 28;            // SQ and PU read
    uint64_t *drain = bars + 29;             // every MMA done
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + S::kNumBars);
    volatile int *stop = reinterpret_cast<volatile int *>(tmem_slot + 1);     // [4]: a role stops; 2's in turn by chunk
    volatile int *late = stop + 4;                                            // a wait gave up: the others do so too
    volatile int *never = stop + 5;      // ... but for those for what the hardware finishes by itself
    float *tables = reinterpret_cast<float *>(sm + S::kTabOff);
    int *bad_at = reinterpret_cast<int *>(sm + S::kBadOff);
    // chunk gc's tables lie at tab = gc % 3, in its turn gc / 3
    auto tab_of = [&](int tab) { return tables + tab * S::kTabFloats; };
    auto info_of = [&](int tab) { return reinterpret_cast<DeltaChunk *>(tab_of(tab) + 9 * DC); };
    enum { T_GHI = 0, T_GLO = DC, T_BETA = 2 * DC, T_GAM = 3 * DC, T_W = 4 * DC, T_B = 5 * DC, T_C = 6 * DC, T_F = 7 * DC,
           T_P = 8 * DC };

    if (warp == 28 && lane == 0) {
        for (int i = 0; i < QS; ++i) {
            mbar_init(&qk_full[i], 1);
            mbar_init(&qk_empty[i], 1 + 4);  // the MMAs, the norms
            mbar_init(&tab_full[i], 1);
            mbar_init(&tab_free[i], 16 + 8 + 4 + 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 16);
            mbar_init(&norms[i], 4);
            mbar_init(&o_done[i], 1);
            mbar_init(&go[i], 1);
        }
        mbar_init(kq_done, 1);
        mbar_init(kq_read, 8);
        mbar_init(t_ready, 8);
        mbar_init(s_ready, 16);
        mbar_init(x_ready, 16);
        mbar_init(kv_done, 1);
        mbar_init(o_read, 4);
        mbar_init(drain, 1);
        for (int i = 0; i < 6; ++i) stop[i] = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (warp >= 16 && warp < 20) {
        // P: tokens 0..31 see no key behind 31
#pragma unroll
        for (int ch = 4; ch < 8; ++ch)
            *reinterpret_cast<uint4 *>(sm + S::kPOff + (warp - 16) * kDeltaPanel + sw128_off(lane, ch)) =
                make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uni((int)*tmem_slot);
    // a warp's wait: every lane gets the same answer
    auto wait = [&](uint64_t *bar, int phase) {
        return __all_sync(0xffffffffu, chunk_wait_each(bar, (uint32_t)phase & 1u, late)) != 0;
    };
    auto arrive = [&](uint64_t *bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    // A role of several warps: one of them waits (the others' polling would take issue slots from those that
    // work) and the rest behind a barrier of the role.  A wait that gives up makes those at the role's next chunk
    // give up at once, and these stop the role, all of its warps together: its flag is written before that barrier alone,
    // and not again before every warp has read it.
    auto role_wait = [&](int flag, uint64_t *bar, int phase) {
        if (!wait(bar, phase)) stop[flag] = 1;
    };
    auto role_sync = [](int role, int threads) {
        asm volatile("bar.sync %0, %1;" ::"r"(role + 1), "r"(threads) : "memory");
    };
    auto next_tab = [](int &tab, int &turn) {
        if (++tab == S::kTabs) tab = 0, ++turn;
    };

    if (warp < 16) {
        // ============================================================ the chain
        more_regs<kChainRegs>();
        const bool real = (warp & 3) * 32 < D;       // warp-uniform; head_dim 64: lanes 64..127 reach no output
        constexpr int N = D / 4;             // columns of S per thread
        float St[N];
        int tab_i = 0, turn = 0;
#pragma unroll 1
        for (int gc = 0;; ++gc) {
            role_sync(0, kChainSync);
            tc_fence_after();
            if (uni(info_of(tab_i)->n) == 0 || stop[0]) break;
            {
                const int tid = renew(threadIdx.x), grp = (tid >> 5) & 3, part = tid >> 7, dv = tid & 127;
                const DeltaChunk *info = info_of(tab_i);
                if (info->first) {
                    const float *src = info->src;
                    const int one = LOCAL && info->ident ? dv - part * N : -1;       // the column of the identity's 1
#pragma unroll
                    for (int i = 0; i < N; i += 4) {
                        float4 x = make_float4(one == i, one == i + 1, one == i + 2, one == i + 3);
                        if (!LOCAL && src && real) x = *reinterpret_cast<const float4 *>(src + dv * D + part * N + i);
                        St[i] = x.x, St[i + 1] = x.y, St[i + 2] = x.z, St[i + 3] = x.w;
                    }
                }
                // ---- S_0's parts to TMEM
                if (part == 0) bad_at[(gc & 1) * 128 + dv] = DC;
                if (real) {
                    const uint32_t to = tmem + ((uint32_t)grp << 21) + TM_S1 + part * N / 2;
#pragma unroll
                    for (int i = 0; i < N; i += 16) {
                        uint32_t s1[8], s2[8], s3[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) split3(St[i + 2 * k], St[i + 2 * k + 1], s1[k], s2[k], s3[k]);
                        tmem_st8(to + i / 2, s1);
                        tmem_st8(to + 64 + i / 2, s2);
                        tmem_st8(to + 128 + i / 2, s3);
                    }
                    tc_wait_st();
                }
                tc_fence_before();
                arrive(s_ready);
            }
            // ---- R = b v - c S_0 k, then U~ and w U~
#pragma unroll 1
            for (int pass = 0; pass < 2; ++pass) {
                role_sync(0, kChainSync);
                tc_fence_after();
                if (real) {
                    // in 8x8 fragments: 16 value dimensions and 32 tokens a warp; pair 2 g + r of a thread: tokens
                    // 8 g + q2, + 1 of its dimension dv + 8 r
                    const int tid = renew(threadIdx.x), grp = (tid >> 5) & 3, low = (tid >> 7) & 1, th = (tid >> 8) * 32;
                    const int l = tid & 31, q2 = (l & 3) * 2, dv0 = grp * 32 + low * 16;
                    const uint32_t lane_base = tmem + ((uint32_t)grp << 21) + ((uint32_t)low << 20);
                    uint32_t u[16];
                    tmem_ld_16x256b_x4(lane_base + (pass ? TM_U : TM_SK) + th, u);
                    const float *tab = tab_of(tab_i) + th + q2;
                    float x[16];
                    if (pass) {
                        tc_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) x[j] = __uint_as_float(u[j]);
                    } else {
                        // V transposed on the way: a matrix is 8 tokens of 8 dimensions, chunks swizzled by token
                        const uint32_t at = smb + S::kVOff + (gc & 1) * S::kVBytes + ((dv0 & (D - 1)) >> 6) * kDeltaPanel +
                                            (th + (l >> 4) * 8 + (l & 7)) * 128 +
                                            (((((dv0 & 63) >> 3) + ((l >> 3) & 1)) ^ (l & 7)) << 4);
                        uint32_t v[8];
                        ldsm_x4_t(at, v[0], v[1], v[2], v[3]);
                        ldsm_x4_t(at + 16 * 128, v[4], v[5], v[6], v[7]);
                        if (LOCAL && info_of(tab_i)->ident) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) v[k] = 0u;
                        }
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const float2 b = *reinterpret_cast<const float2 *>(tab + T_B + 8 * g);
#pragma unroll
                            for (int k = 2 * g; k < 2 * g + 2; ++k)
                                fma2(x[2 * k], x[2 * k + 1], b.x, b.y, __uint_as_float(v[k] << 16),
                                     __uint_as_float(v[k] & 0xFFFF0000u), 0.f, 0.f);
                        }
                        tc_wait_ld();
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const float2 c = *reinterpret_cast<const float2 *>(tab + T_C + 8 * g);
#pragma unroll
                            for (int j = 4 * g; j < 4 * g + 4; j += 2)
                                fma2(x[j], x[j + 1], c.x, c.y, __uint_as_float(u[j]), __uint_as_float(u[j + 1]), x[j], x[j + 1]);
                        }
                    }
                    float z0 = 0.f, z1 = 0.f;        // NaN once something non-finite went by
#pragma unroll
                    for (int j = 0; j < 16; j += 2) fma2(z0, z1, x[j], x[j + 1], 0.f, 0.f, z0, z1);
                    if (__any_sync(0xffffffffu, !(z0 + z1 == 0.f))) {
                        // the triangles' zeros would not keep it from earlier tokens
                        int *bad = bad_at + (gc & 1) * 128 + dv0 + (l >> 2);
                        const int first[2] = {drop_non_finite(x, 0), drop_non_finite(x, 2)};
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            if (first[r] < 16) atomicMin(bad + 8 * r, th + (first[r] >> 2) * 8 + q2 + (first[r] & 1));
                    }
                    uint32_t r1[8], r2[8], r3[8];
                    if (pass) {
                        if (!LOCAL) {
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                float y0, y1;
                                r1[k] = take_bf16(y0, y1, x[2 * k], x[2 * k + 1]);
                                r2[k] = pack_bf16x2(y0, y1);
                            }
                            tmem_st_16x128b_x4(lane_base + TM_UO + th / 2, r1);
                            tmem_st_16x128b_x4(lane_base + TM_UO + 32 + th / 2, r2);
                        }
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const float2 w = *reinterpret_cast<const float2 *>(tab + T_W + 8 * g);
#pragma unroll
                            for (int j = 4 * g; j < 4 * g + 4; j += 2) fma2(x[j], x[j + 1], w.x, w.y, x[j], x[j + 1], 0.f, 0.f);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) split3(x[2 * k], x[2 * k + 1], r1[k], r2[k], r3[k]);
                    tmem_st_16x128b_x4(lane_base + TM_R + th / 2, r1);
                    tmem_st_16x128b_x4(lane_base + TM_R + 32 + th / 2, r2);
                    tmem_st_16x128b_x4(lane_base + TM_R + 64 + th / 2, r3);
                    tc_wait_st();
                }
                tc_fence_before();
                arrive(x_ready);
                if (pass == 0) arrive(&v_empty[gc & 1]);
            }
            // ---- S = e^{G_n} S + KV
            role_sync(0, kChainSync);
            tc_fence_after();
            if (real) {
                const int tid = renew(threadIdx.x), grp = (tid >> 5) & 3, part = tid >> 7, dv = tid & 127;
                const DeltaChunk *info = info_of(tab_i);
                const bool bad = min(bad_at[(gc & 1) * 128 + dv], info->bad) < DC;
                const float a = bad ? __uint_as_float(0x7FC00000u) : info->a, a_lo = info->a_lo;
#pragma unroll
                for (int i = 0; i < N; i += 16) {
                    uint32_t kv[16];
                    tmem_ld16(tmem + ((uint32_t)grp << 21) + TM_KV + part * N + i, kv);
                    tc_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        float x0, x1;
                        fma2(x0, x1, a_lo, a_lo, St[i + k], St[i + k + 1], __uint_as_float(kv[k]),
                             __uint_as_float(kv[k + 1]));
                        fma2(St[i + k], St[i + k + 1], a, a, St[i + k], St[i + k + 1], x0, x1);
                    }
                }
                if (float *dst = info->dst) {
#pragma unroll
                    for (int i = 0; i < N; i += 4)
                        *reinterpret_cast<float4 *>(dst + dv * D + part * N + i) = make_float4(St[i], St[i + 1], St[i + 2], St[i + 3]);
                }
            }
            tc_fence_before();
            arrive(&tab_free[tab_i]);
            next_tab(tab_i, turn);
        }
    } else if (warp < 24) {
        // ============================================================ T and P
        const int w8 = warp - 16, qd = warp & 3, half = w8 >> 2;
        const bool keys = qd >= 2;           // lane = row of (Q; K)
        float *At = reinterpret_cast<float *>(sm + S::kAOff);            // [j][i]
        float *Tm = reinterpret_cast<float *>(sm + S::kTOff);            // [i][j % 32], T11 and the diagonal blocks
        float *X = At + DC / 2 * kAStride;                                  // [i][j]: A21 T11
        int tab_i = 0, turn = 0;
#pragma unroll 1
        for (int gc = 0;; ++gc) {
            if (w8 == 7) {                   // (the first one done with a chunk)
                role_wait(1, &tab_full[tab_i], turn);
                if (info_of(tab_i)->n) role_wait(1, lane ? kq_done : &norms[gc & 1], lane ? gc : gc >> 1);
            }
            role_sync(1, 256);
            tc_fence_after();
            const int n = uni(info_of(tab_i)->n);
            if (n == 0 || stop[1]) break;
            // up to 32 tokens: the rows behind them are the identity's, in T too
            const bool low = n <= DC / 2;
            if ((LOCAL && !keys) || (low && (qd & 1))) {
                arrive(kq_read);             // no P, or no use of these rows of it
                if (keys) {
                    float *to = At + DC / 2 + renew(lane);
#pragma unroll 8
                    for (int j = half * 32; j < half * 32 + 32; ++j) to[j * kAStride] = j == DC / 2 + lane ? 1.f : 0.f;
                }
            } else {
                const int i = (qd & 1) * 32 + renew(lane);
                const float *tab = tab_of(tab_i);
                const float ghi = tab[T_GHI + i], glo = tab[T_GLO + i], factor = tab[(keys ? T_BETA : T_P) + i];
                const int see = keys ? (i < n ? i : 0) : i + 1;              // columns that count
                // KQ follows PU of the chunk before the last: P's place is free.
                // Tokens 0..31 see no key behind 31; two warps share a row's columns, eight at a time
                const int width = 16 + 16 * (qd & 1);
                const uint32_t from = tmem + ((uint32_t)(qd * 32) << 16) + TM_KQ;
                uint32_t next[8];
                tmem_ld8(from + half * width, next);
#pragma unroll 1
                for (int j0 = half * width; j0 < half * width + width; j0 += 8) {
                    float x[8], g[8];
#pragma unroll
                    for (int j = 0; j < 8; j += 4) {
                        const float4 a = *reinterpret_cast<const float4 *>(tab + T_GHI + j0 + j);
                        const float4 b = *reinterpret_cast<const float4 *>(tab + T_GLO + j0 + j);
                        fma2(x[j], x[j + 1], a.x, a.y, -1.f, -1.f, ghi, ghi);
                        fma2(x[j + 2], x[j + 3], a.z, a.w, -1.f, -1.f, ghi, ghi);
                        fma2(g[j], g[j + 1], b.x, b.y, -1.f, -1.f, glo, glo);
                        fma2(g[j + 2], g[j + 3], b.z, b.w, -1.f, -1.f, glo, glo);
                    }
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        add2(x[j], x[j + 1], g[j], g[j + 1]);
                        fma2(x[j], x[j + 1], ex2(x[j]), ex2(x[j + 1]), factor, factor, 0.f, 0.f);
                    }
                    tc_wait_ld();
#pragma unroll
                    for (int j = 0; j < 8; j += 2)
                        fma2(x[j], x[j + 1], x[j], x[j + 1], __uint_as_float(next[j]), __uint_as_float(next[j + 1]), 0.f, 0.f);
                    if (!__all_sync(0xffffffffu, j0 + 8 <= see)) {
                        // masked by choice, not by a factor, which would keep a NaN
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = j0 + j < see ? x[j] : 0.f;
                    }
                    float z = 0.f, z1 = 0.f;     // NaN once something non-finite went by
#pragma unroll
                    for (int j = 0; j < 8; j += 2) fma2(z, z1, x[j], x[j + 1], 0.f, 0.f, z, z1);
                    z += z1;
                    if (keys && !(z == 0.f)) {
                        // a zero of T would not keep it from earlier tokens: 0 here, and NaN from this token on later
                        atomicMin(&info_of(tab_i)->bad, i);
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = fabsf(x[j]) < INFINITY ? x[j] : 0.f;
                    }
                    tmem_ld8(from + ((j0 + 8) & 63), next);              // (behind the last ones: not used)
                    if (keys) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) At[(j0 + j) * kAStride + i] = x[j];
                    } else {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            hi[k] = take_bf16(x[2 * k], x[2 * k + 1]);
                            lo[k] = pack_bf16x2(x[2 * k], x[2 * k + 1]);
                        }
                        uint8_t *to = sm + S::kPOff + (gc & 1) * 2 * kDeltaPanel + sw128_off(i, j0 >> 3);
                        *reinterpret_cast<uint4 *>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4 *>(to + kDeltaPanel) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                }
                tc_wait_ld();
                tc_fence_before();
                arrive(kq_read);
            }
            // T11 by a warp of A's rows 0..31, T22 by the one that made its block of A.  T11 is there first, so that
            // A21 T11 is made beside T22.
            if (qd == 2) role_sync(3, 64);
            if (w8 == 2 || (w8 == 7 && !low)) {
                if (gc > 0) wait(&go[1], gc - 1);                    // U of the chunk before done: T's place
                const int jb = w8 == 2 ? 0 : 32;
                {
                    // its two 16 x 16 diagonal blocks, a lane per column: x_q = [q = column] - sum_{m < q} A_qm x_m
                    const int l = renew(lane), col = l & 15, at = jb + (l & 16);
                    float *blk = At + at * (kAStride + 1);
                    float x[16];
#pragma unroll
                    for (int q = 0; q < 16; ++q) x[q] = q == col ? 1.f : 0.f;
#pragma unroll
                    for (int m = 0; m < 15; ++m) {
#pragma unroll
                        for (int q = (m + 1) & ~3; q < 16; q += 4) {
                            const float4 a = *reinterpret_cast<const float4 *>(blk + m * kAStride + q);
                            if (q > m) x[q] = fmaf(-a.x, x[m], x[q]);
                            if (q + 1 > m) x[q + 1] = fmaf(-a.y, x[m], x[q + 1]);
                            if (q + 2 > m) x[q + 2] = fmaf(-a.z, x[m], x[q + 2]);
                            if (q + 3 > m) x[q + 3] = fmaf(-a.w, x[m], x[q + 3]);
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < 16; q += 4)
                        *reinterpret_cast<float4 *>(blk + col * kAStride + q) = make_float4(x[q], x[q + 1], x[q + 2], x[q + 3]);
                    float *to = Tm + at * kAStride + l;
#pragma unroll
                    for (int q = 0; q < 16; ++q) to[q * kAStride] = x[q];
                }
                // the block below them: A21 T11, in the place where T21 = -T22 (A21 T11) goes; four rows of two columns a lane
#pragma unroll 1
                for (int second = 0; second < 2; ++second) {
                    __syncwarp();
                    const int l = renew(lane), r0 = (l >> 3) * 4, c = (l & 7) * 2;
                    const float *left = At + (jb + 16 * second) * kAStride + jb + 16 + r0;
                    float *right = Tm + (jb + 16 * second) * kAStride + c;
                    float y[2][4] = {};
#pragma unroll 8
                    for (int m = 0; m < 16; ++m) {
                        const float4 a = *reinterpret_cast<const float4 *>(left + m * kAStride);
                        const float2 b = *reinterpret_cast<const float2 *>(right + m * kAStride);
                        fma2(y[0][0], y[0][1], a.x, a.y, b.x, b.x, y[0][0], y[0][1]);
                        fma2(y[0][2], y[0][3], a.z, a.w, b.x, b.x, y[0][2], y[0][3]);
                        fma2(y[1][0], y[1][1], a.x, a.y, b.y, b.y, y[1][0], y[1][1]);
                        fma2(y[1][2], y[1][3], a.z, a.w, b.y, b.y, y[1][2], y[1][3]);
                    }
                    __syncwarp();
                    const float sign = second ? -1.f : 1.f;
                    float *to = Tm + (jb + 16 + r0) * kAStride + c;
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        *reinterpret_cast<float2 *>(to + k * kAStride) = make_float2(sign * y[0][k], sign * y[1][k]);
                    if (second) {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            *reinterpret_cast<float4 *>(At + (jb + c + e) * kAStride + jb + 16 + r0) =
                                make_float4(-y[e][0], -y[e][1], -y[e][2], -y[e][3]);
                    }
                }
            }
            if (low) role_sync(1, 256);
            else if (w8 != 7) role_sync(4, 224);
            // the block below, of 32 x 32: X = A21 T11, then -T22 X.  A task has 8 rows and 16 columns; a lane adds up
            // every other term for four rows of two columns and comes to hold one of them.
#pragma unroll 1
            for (int second = low ? 2 : 0; second < 2; ++second) {
                // (first: of columns 0..15 by the warps of P; 16..31, half as long, by those of A)
                int task = second ? w8 : ((w8 & 1) + (w8 >> 2) * 2) * 2;
                if (!second && keys) task = w8 == 2 ? 1 : w8 == 3 ? 3 : w8 == 6 ? 5 : 8;
#pragma unroll 1
                for (; task < 8; task = !second && task == 5 ? 7 : 8) {
                    const int l = renew(lane), odd = l >> 4, c = (task & 1) * 16 + (l & 7) * 2;
                    const int r0 = (task >> 1) * 8 + ((l >> 3) & 1) * 4;
                    // T11's columns begin at the diagonal, T22's rows end there
                    const int m0 = second ? 0 : (task & 1) * 16, m1 = second && task < 4 ? 16 : 32;
                    const float *left = At + (32 * second + m0 + odd) * kAStride + 32 + r0;
                    const float *right = (second ? X : Tm) + (m0 + odd) * kAStride + c;
                    float y[2][4] = {};
#pragma unroll 1
                    for (int m = m0; m < m1; m += 16, left += 16 * kAStride, right += 16 * kAStride) {
#pragma unroll
                        for (int k = 0; k < 16; k += 2) {
                            const float4 a = *reinterpret_cast<const float4 *>(left + k * kAStride);
                            const float2 b = *reinterpret_cast<const float2 *>(right + k * kAStride);
                            fma2(y[0][0], y[0][1], a.x, a.y, b.x, b.x, y[0][0], y[0][1]);
                            fma2(y[0][2], y[0][3], a.z, a.w, b.x, b.x, y[0][2], y[0][3]);
                            fma2(y[1][0], y[1][1], a.x, a.y, b.y, b.y, y[1][0], y[1][1]);
                            fma2(y[1][2], y[1][3], a.z, a.w, b.y, b.y, y[1][2], y[1][3]);
                        }
                    }
                    float acc[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        acc[k] = (odd ? y[1][k] : y[0][k]) + __shfl_xor_sync(0xffffffffu, odd ? y[0][k] : y[1][k], 16);
                    if (second) {
                        *reinterpret_cast<float4 *>(At + (c + odd) * kAStride + 32 + r0) =
                            make_float4(-acc[0], -acc[1], -acc[2], -acc[3]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k) X[(r0 + k) * kAStride + c + odd] = acc[k];
                    }
                }
                role_sync(1, 256);
            }
            // T's three parts: T11, T22, T21, a lane per row, eight columns at a time
#pragma unroll 1
            for (int x = w8; x < 12; x += 8) {
                const int r = (x >= 4 ? 32 : 0) + renew(lane), j = (x >> 2 == 1 ? 32 : 0) + 8 * (x & 3);
                uint32_t h[3][4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    split3(At[(j + 2 * k) * kAStride + r], At[(j + 2 * k + 1) * kAStride + r], h[0][k], h[1][k], h[2][k]);
                uint8_t *t = sm + S::kTOff + sw128_off(r, j >> 3);
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    *reinterpret_cast<uint4 *>(t + k * kDeltaPanel) = make_uint4(h[k][0], h[k][1], h[k][2], h[k][3]);
            }
            fence_proxy_async_smem();
            arrive(t_ready);
            arrive(&tab_free[tab_i]);
            next_tab(tab_i, turn);
        }
    } else if (warp < 28) {
        // ============================================================ norms, output rows: a warp per 32 rows of (Q; K),
        // then per 32 value dimensions, in 8x8 fragments (thread: two neighbouring tokens of one dv), transposed by
        // stmatrix into the warp's own [64 tokens][32 dv] tile, 16-byte chunks swizzled by token pair.
        fewer_regs<kRowRegs>();
        const int grp = warp & 3, q2 = (lane & 3) * 2;
        const int row = grp * 32 + lane, i = row & 63;
        const bool real = grp * 32 < D, keys = grp >= 2;
        const uint32_t lane_base = tmem + ((uint32_t)(grp * 32) << 16);
        uint8_t *stg = sm + S::kOutOff + grp * DC * 64;
        // stmatrix row address: token (lane / 16) * 8 + lane % 8 of its group, dv chunk lane / 8 % 2
        const int row0 = (lane >> 4) * 8 + (lane & 7), ch0 = (lane >> 3) & 1, sw = (row0 >> 1) & 3;
        const uint32_t stg_at = smem_u32(stg) + row0 * 64;
        int tab_i = 0, turn = 0, last_tab = 0;
#pragma unroll 1
        for (int gc = 0;; ++gc) {
            if (grp == 0) {
                role_wait(2 + (gc & 1), &tab_full[tab_i], turn);
                const int n = info_of(tab_i)->n;
                if (n) role_wait(2 + (gc & 1), &qk_full[gc % QS], gc / QS);       // (LOCAL: K alone)
                if (n && n < DC) role_wait(2 + (gc & 1), &v_full[gc & 1], gc >> 1);
            }
            role_sync(2, 128);
            const int more = uni(info_of(tab_i)->n);
            if (stop[2 + (gc & 1)]) break;
            if (more > 0) {
                // ---- norms of this chunk
                const int s = gc % QS;
                float *tab = tab_of(tab_i);
                uint8_t *tile = sm + s * S::kQkBytes + row * 128;
                const bool behind = keys && i >= more;
                if (more < DC) {
                    // K's and V's rows behind the sequence's end are zeroed: a weight of 0 would not cancel a NaN there
                    uint8_t *v = sm + S::kVOff + (gc & 1) * S::kVBytes + i * 128;
#pragma unroll 1
                    for (int x = 0; x < PAN * 8; ++x) {
                        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
                        if (behind) {
                            *reinterpret_cast<uint4 *>(tile + (x >> 3) * S::kQkPanel + (x & 7) * 16) = none;
                            *reinterpret_cast<uint4 *>(v + (x >> 3) * kDeltaPanel + (x & 7) * 16) = none;
                        }
                    }
                    fence_proxy_async_smem();
                }
                float r = 1.f;
                if (p.norm && (!LOCAL || keys)) {
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
                if (behind) r = 0.f;
                // rows of K: b, -c, A's row factor (in beta's place); rows of Q: nothing, f, P's
                const float first = keys ? tab[T_BETA + i] * r : p.scale * r, second = keys ? first * r : first;
                tab[(keys ? T_B : T_P) + i] = first;
                tab[(keys ? T_BETA : T_P) + i] = second;
                tab[(keys ? T_C : T_F) + i] = (keys ? -second : second) * tab[T_GAM + i];
                arrive(&norms[gc & 1]);
                arrive(&qk_empty[s]);
                if (LOCAL) arrive(&tab_free[tab_i]);
            }
            if (!LOCAL && gc > 0) {
                // ---- outputs of the one before
                const int oc = gc - 1;
                const DeltaChunk *info = info_of(last_tab);
                const int n = uni(info->n), t0 = info->t0, h = info->h;
                if (grp == 0) wait(&o_done[oc & 1], oc >> 1);
                role_sync(2, 128);
                tc_fence_after();
                int first_bad = DC;
                if (real) {
                    if (lane == 0) bulk_wait_read();             // the tile's last store
                    __syncwarp();
                    first_bad = min(bad_at[(oc & 1) * 128 + grp * 32 + lane], info->bad);
#pragma unroll 1
                    for (int part = 0; part < 4; ++part) {      // 16 dv, 32 tokens
                        const int hl = part >> 1, g0 = (part & 1) * 4;
                        const uint32_t at = lane_base + ((uint32_t)hl << 20) + g0 * 8;
                        uint32_t x[16], y[16], r[8];
                        tmem_ld_16x256b_x4(at + TM_PU, x);
                        tmem_ld_16x256b_x4(at + TM_SQ, y);
                        const float *e = tab_of(last_tab) + T_F + g0 * 8 + q2;
                        tc_wait_ld();
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
                }
                tc_fence_before();
                arrive(o_read);
                arrive(&tab_free[last_tab]);
                // NaN from a dv's first non-finite token on
                for (int t = first_bad; t < DC; ++t)
                    *reinterpret_cast<uint16_t *>(stg + t * 64 + (((lane >> 3) ^ ((t >> 1) & 3)) << 4) + (lane & 7) * 2) =
                        0x7FC0;
                __syncwarp();
                if (real && n == DC) {
                    // one store of the tile; its swizzle is the copy engine's for rows of 64 bytes
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(&omap, stg, grp * 32, h, t0);
                        bulk_commit();
                    }
                } else if (real) {
                    // rows behind the sequence stay as they are
                    __nv_bfloat16 *out = p.out + (int64_t)t0 * p.out_stride + (int64_t)h * D + grp * 32;
#pragma unroll 1
                    for (int t = lane >> 2; t < n; t += 8)
                        *reinterpret_cast<uint4 *>(out + t * p.out_stride + (lane & 3) * 8) =
                            *reinterpret_cast<const uint4 *>(stg + t * 64 + (((lane & 3) ^ ((t >> 1) & 3)) << 4));
                    __syncwarp();
                }
            }
            if (more == 0) break;
            last_tab = tab_i;
            next_tab(tab_i, turn);
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    } else {
        fewer_regs<kOtherRegs>();
        if (warp == 28) {
            // ============================================================ loads
            DeltaWalk walk(units_n, heads);
            // x / y of x < 2^18: off by less than 2^-20 of itself, and half a step away from the next integer
            const float inv_g = __fdividef(1.f, (float)p.G);
            int gc = 0, qk_gone = 0;
#pragma unroll 1
            while (walk.step(units, LOCAL)) {
                const int s = gc % QS, hv = LOCAL && walk.h >= p.Hv ? walk.h - p.Hv : walk.h;
                const int hk = (int)(((float)hv + 0.5f) * inv_g);
                if (gc >= QS && !wait(&qk_empty[s], gc / QS - 1)) break;
                if (elect_one()) {
                    uint8_t *to = sm + s * S::kQkBytes;
                    mbar_arrive_expect_tx(&qk_full[s], LOCAL ? S::kQkBytes / 2 : S::kQkBytes);
#pragma unroll 1
                    for (int x = 0; x < PAN; ++x, to += S::kQkPanel) {
                        tma_load_3d(to + kDeltaPanel, &kmap, &qk_full[s], x * 64, hk, walk.row);
                        if (!LOCAL) tma_load_3d(to, &qmap, &qk_full[s], x * 64, hk, walk.row);
                    }
                }
                __syncwarp();
                ++qk_gone;
                if (gc >= VS && !wait(&v_empty[gc & 1], (gc >> 1) - 1)) break;
                if (elect_one()) {
                    uint8_t *to = sm + S::kVOff + (gc & 1) * S::kVBytes;
                    mbar_arrive_expect_tx(&v_full[gc & 1], S::kVBytes);
#pragma unroll 1
                    for (int x = 0; x < PAN; ++x)
                        tma_load_3d(to + x * kDeltaPanel, &vmap, &v_full[gc & 1], x * 64, hv, walk.row);
                }
                __syncwarp();
                ++gc;
            }
            // copies still in flight (after a wait that gave up) land before the CTA ends
#pragma unroll 1
            for (int d = max(0, qk_gone - QS); d < qk_gone; ++d)
                chunk_wait_each(&qk_full[d % QS], (uint32_t)(d / QS) & 1u, never);
#pragma unroll 1
            for (int d = max(0, gc - VS); d < gc; ++d) chunk_wait_each(&v_full[d & 1], (uint32_t)(d >> 1) & 1u, never);
            __syncwarp();
        } else if (warp == 29) {
            // ============================================================ the chunks' tables, two tokens a lane
            DeltaWalk walk(units_n, heads);
            const double kLog2e = 1.4426950408889634074;
            int tab_i = 0, turn = -1;                                    // (turn of the tables' last readers)
#pragma unroll 1
            while (true) {
                const int n = walk.step(units, LOCAL);
                const bool ident = LOCAL && walk.h >= p.Hv;
                const int h = ident ? walk.h - p.Hv : walk.h;
                float g[2] = {0.f, 0.f}, beta[2] = {0.f, 0.f};
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int64_t t = walk.row + 2 * lane + x;
                    if (2 * lane + x < n) {
                        g[x] = __ldg(p.log_decay + t * p.decay_stride + h);
                        beta[x] = __ldg(p.beta + t * p.beta_stride + h);
                    }
                }
                if (!(g[0] <= 0.f && g[1] <= 0.f)) record_error(p.err, ERR_RANGE | SRC_DELTA);
                // (e^-256 is 0 in fp32, and so is what is below; -inf - -inf would be NaN)
                const double x0 = (double)fmaxf(fminf(g[0], 0.f), -256.f) * kLog2e;
                const double x1 = (double)fmaxf(fminf(g[1], 0.f), -256.f) * kLog2e;
                double inc = x0 + x1;
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) {
                    const double y = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += y;
                }
                const double all = __shfl_sync(0xffffffffu, inc, 31);
                if (turn >= 0 && !wait(&tab_free[tab_i], turn)) break;
                float *tab = tab_of(tab_i);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int i = 2 * lane + x;
                    const double Gi = x ? inc : inc - x1;
                    const float hi = (float)Gi;
                    tab[T_GHI + i] = hi;
                    tab[T_GLO + i] = (float)(Gi - (double)hi);
                    tab[T_BETA + i] = beta[x];
                    tab[T_GAM + i] = ex2(hi);
                    tab[T_W + i] = i < n ? ex2((float)(all - Gi)) : 0.f;
                }
                // e^{G_n} near 1, where a state is multiplied many times before it fades, as two parts: e^y - 1 by its
                // series up to y^9, 2^-33 of it for y >= -0.3
                const float y = (float)(all * 0.69314718055994530942);
                float a = ex2((float)all), a_lo = 0.f;
                if (y > -0.3f) {
                    float e = 1.f / 362880.f;
                    e = fmaf(e, y, 1.f / 40320.f), e = fmaf(e, y, 1.f / 5040.f), e = fmaf(e, y, 1.f / 720.f);
                    e = fmaf(e, y, 1.f / 120.f), e = fmaf(e, y, 1.f / 24.f), e = fmaf(e, y, 1.f / 6.f);
                    e = fmaf(e, y, 0.5f), e = fmaf(e, y, 1.f) * y;
                    a = 1.f + e;
                    a_lo = e - (a - 1.f);
                }
                if (lane == 0) {
                    const float *src = nullptr;
                    float *dst = nullptr;
                    if (n && (walk.first || walk.left <= DC)) {
                        const DeltaUnit u = *walk.unit;
                        float *cached = u.slot < 0 ? nullptr : p.state + ((int64_t)u.slot * p.Hv + h) * D * D;
                        float *kept = u.row < 0 ? nullptr
                                                : p.states + ((int64_t)(u.row + (ident ? p.state_rows : 0)) * p.Hv + h) * D * D;
                        src = kept ? kept : u.from ? cached : nullptr;
                        if (walk.left <= DC) dst = LOCAL ? kept : u.last ? cached : nullptr;
                    }
                    *info_of(tab_i) = DeltaChunk{n, walk.row, walk.h, walk.first, a, a_lo, DC, ident, src, dst};
                }
                arrive(&tab_full[tab_i]);
                next_tab(tab_i, turn);
                if (n == 0) break;
            }
        } else if (warp == 30) {
            // ============================================================ MMAs
            // four steps of 16 of K with A in TMEM
            auto four = [&](uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t d_step, uint32_t b_step,
                            uint32_t id_step, bool add) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc_mma_ts(tmem + d + k * d_step, tmem + a + k * 8, b + k * b_step, id - k * id_step, add || k > 0);
            };
            // S_0 times K or Q: parts of S_0 and panels of the tile
            auto times = [&](uint32_t d, uint32_t tile, int parts) {
                const uint64_t b = sw128_desc(tile, 16, 1024);
#pragma unroll 1
                for (int x = 0; x < parts * PAN; ++x) {
                    const int part = PAN == 2 ? x >> 1 : x, pan = PAN == 2 ? x & 1 : 0;
                    four(d, TM_S1 + part * 64 + pan * 32, b + pan * (S::kQkPanel >> 4), idesc_bf16_f32(128, DC, 0), 0, 2, 0,
                         x > 0);
                }
            };
            // a product whose B is lower triangular (16 tokens j reach rows from theirs on), of parts of A and B in turn,
            // a digit each
            auto triangle = [&](uint32_t d, uint32_t a, uint32_t tile, int products, uint32_t of_a, uint32_t of_b) {
                const uint64_t b = sw128_desc(tile, 16, 1024);
#pragma unroll 1
                for (int x = 0; x < products; ++x)
                    four(d, a + (of_a >> 4 * x & 3) * 32, b + (of_b >> 4 * x & 3) * (kDeltaPanel >> 4),
                         idesc_bf16_f32(128, DC, 0), 16, 2 + (16 * 128 >> 4), (16u >> 3) << 17, x > 0);
            };
            // KQ of chunk gc, if there is one
            auto kq = [&](int gc, int tab_i, int turn) {
                if (!wait(&tab_full[tab_i], turn)) return -1;
                if (uni(info_of(tab_i)->n) == 0) return 0;
                if (!wait(&qk_full[gc % QS], gc / QS)) return -1;
                if (gc > 0 && !wait(kq_read, gc - 1)) return -1;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t qd = sw128_desc(smb + (gc % QS) * S::kQkBytes, 16, 1024);
#pragma unroll 1
                    for (int x = 0; x < PAN; ++x) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint64_t d = qd + x * (S::kQkPanel >> 4) + k * 2;
                            tc_mma_ss(tmem + TM_KQ, d, d + (kDeltaPanel >> 4), idesc_bf16_f32(128, DC, 0), x + k > 0);
                        }
                    }
                    tc_commit(kq_done);
                }
                __syncwarp();
                return 1;
            };
            int tab_i = 0, turn = 0;
            // in the order of the chain; KQ a chunk ahead, in the time in which R is made
#pragma unroll 1
            for (int gc = -1;; ++gc) {
                const uint32_t qk = smb + (gc % QS) * S::kQkBytes;
                int old_tab = tab_i;
                if (gc >= 0) {
                    next_tab(tab_i, turn);
                    if (!wait(s_ready, gc)) break;
                    tc_fence_after();
                    if (elect_one()) {
                        times(TM_SK, qk + kDeltaPanel, 3);
                        tc_commit(&go[0]);
                    }
                    __syncwarp();
                    if (!LOCAL) {
                        if (gc > 0 && !wait(o_read, gc - 1)) break;
                        tc_fence_after();
                        if (elect_one()) times(TM_SQ, qk, 2);
                        __syncwarp();
                    }
                }
                const int more = kq(gc + 1, tab_i, turn);
                if (more < 0 || (gc < 0 && more == 0)) break;
                if (gc < 0) continue;
                if (!wait(t_ready, gc) || !wait(x_ready, 2 * gc)) break;
                tc_fence_after();
                if (elect_one()) {
                    // parts of R and of T: (1, 1), (2, 1), (1, 2), (3, 1), (2, 2), (1, 3)
                    triangle(TM_U, TM_R, smb + S::kTOff, 6, 0x012010, 0x210100);
                    tc_commit(&go[1]);
                }
                __syncwarp();
                if (!wait(x_ready, 2 * gc + 1)) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t kd = sw128_desc(qk + kDeltaPanel, S::kQkPanel, 1024);
#pragma unroll 1
                    for (int x = 0; x < 3; ++x)
                        four(TM_KV, TM_R + x * 32, kd, idesc_bf16_f32(128, D, 1), 0, 16 * 128 >> 4, 0, x > 0);
                    tc_commit(kv_done);
                    tc_commit(&qk_empty[gc % QS]);
                    if (!LOCAL) {
                        // parts of U~ and of P: (1, 1), (2, 1), (1, 2)
                        triangle(TM_PU, TM_UO, smb + S::kPOff + (gc & 1) * 2 * kDeltaPanel, 3, 0x010, 0x100);
                        tc_commit(&o_done[gc & 1]);
                    }
                }
                arrive(&tab_free[old_tab]);
                if (more == 0) break;
            }
            // nothing of this CTA's is left in the tensor core when TMEM goes back
            if (elect_one()) tc_commit(drain);
            __syncwarp();
            chunk_wait_each(drain, 0u, never);
            __syncwarp();
        } else {
            // ============================================================ the chain's waits
            int tab_i = 0, turn = 0;
#pragma unroll 1
            for (int gc = 0;; ++gc) {
                role_wait(0, &tab_full[tab_i], turn);
                const bool more = info_of(tab_i)->n;
                if (more) {
                    // four barriers at once, one a lane
                    const bool done = !LOCAL && gc > 0 && lane == 2;
                    uint64_t *bar = done ? &o_done[(gc - 1) & 1] : lane == 1 ? &norms[gc & 1] : &v_full[gc & 1];
                    role_wait(0, lane == 3 ? kq_read : bar, lane == 3 ? gc : done ? (gc - 1) >> 1 : gc >> 1);
                }
                role_sync(0, kChainSync);
                if (!more || stop[0]) break;
#pragma unroll 1
                for (int x = 0; x < 3; ++x) {
                    wait(x == 2 ? kv_done : &go[x], gc);
                    role_sync(0, kChainSync);
                }
                next_tab(tab_i, turn);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
    if (threadIdx.x == 0 && (*late | *never)) record_error(p.err, ERR_TIMEOUT | SRC_DELTA);
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
        attr_err[dev] = cudaFuncSetAttribute(delta_chunk_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             S::kBytes);
        if (attr_err[dev] == cudaSuccess)
            attr_err[dev] = cudaFuncSetAttribute(delta_chunk_kernel<D, true>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
        if (attr_err[dev] == cudaSuccess)
            attr_err[dev] = cudaFuncSetAttribute(delta_join_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 kJoinBytes<D>);
    });
    if (attr_err[dev] != cudaSuccess) return attr_err[dev];
    delta_plan_kernel<<<1, 1024, 0, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // a CTA per SM at most: each goes over several units
    auto ctas = [&](int heads) { return (unsigned)min((int64_t)p.max_units * heads, (int64_t)p.num_sms); };
    if (p.seg_len < p.max_seqlen) {
        e = launch_after(delta_chunk_kernel<D, true>, dim3(ctas(2 * p.Hv)), kDeltaThreads, S::kBytes, stream, qmap, kmap,
                         vmap, omap, p);
        if (e == cudaSuccess)
            e = launch_after(delta_join_kernel<D>, dim3(p.max_units, p.Hv, D / 16), 2 * D, kJoinBytes<D>, stream, p);
        if (e != cudaSuccess) return e;
    }
    main_kernel_event_before(stream);
    e = launch_after(delta_chunk_kernel<D, false>, dim3(ctas(p.Hv)), kDeltaThreads, S::kBytes, stream, qmap, kmap, vmap,
                     omap, p);
    main_kernel_event_after(stream);
    return e;
}

}  // namespace

cudaError_t launch_delta_recurrent(const DeltaParams &p, cudaStream_t stream) {
    const int64_t states = (int64_t)p.batch * p.Hv;
    auto *kernel = p.max_seqlen > 8   ? p.D == 128 ? delta_few_kernel<128, 16> : delta_few_kernel<64, 16>
                   : p.max_seqlen > 1 ? p.D == 128 ? delta_few_kernel<128, 8> : delta_few_kernel<64, 8>
                   : p.D == 128     ? p.cu ? delta_one_kernel<128, true> : delta_one_kernel<128, false>
                                    : p.cu ? delta_one_kernel<64, true> : delta_one_kernel<64, false>;
    main_kernel_event_before(stream);
    kernel<<<(unsigned)(p.D == 64 ? states : p.max_seqlen > 1 ? states * 2 : states * 4), kRecWarps * 32, 0, stream>>>(p);
    main_kernel_event_after(stream);
    return cudaGetLastError();
}

cudaError_t launch_delta_varlen(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap,
                                const CUtensorMap &omap, const DeltaParams &p, cudaStream_t stream) {
    return p.D == 128 ? launch_delta_chunks<128>(qmap, kmap, vmap, omap, p, stream)
                      : launch_delta_chunks<64>(qmap, kmap, vmap, omap, p, stream);
}

}  // namespace attn
