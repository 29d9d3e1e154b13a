// delta_attn.cu -- linear attention by the gated delta rule:
//   u_t = beta_t (v_t - e^{g_t} S_{t-1} k_t)
//   S_t = e^{g_t} S_{t-1} + u_t k_t^T       (S [Dv, Dk], fp32)
//   o_t = scale * S_t q_t
// over packed sequences (prompts, a few tokens each) or one token per sequence
// (decode), with a cache of states.
#include "common.cuh"
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

}  // namespace attn
