// linear_attn.cu -- linear attention with a decay for each head:
//   S_t = e^g S_{t-1} + v_t k_t^T          (S [Dv, Dk], fp32)
//   o_t = scale * S_t q_t
// over packed sequences (a prompt) or one token per sequence (decode), with a
// cache of states.
#include "common.cuh"
#include "kernels.h"

namespace attn {
namespace {

constexpr int kLinStage = 16;   // tokens staged in shared memory at a time

// Tokens [t0, t0 + n) of sequence b; n = 0 for bad offsets (recorded once by the
// CTA of head 0).
__device__ __forceinline__ bool linear_rows(const LinearParams &p, int b, int64_t &t0, int &n, bool report) {
    if (!p.cu) {
        t0 = b;
        n = 1;
        return true;
    }
    const int64_t a = __ldg(p.cu + b), e = __ldg(p.cu + b + 1);
    bool ok = a >= 0 && e >= a && e <= p.total_tokens;
    t0 = ok ? a : 0;
    n = ok ? (int)(e - a) : 0;
    if (ok && n > p.max_seqlen) {
        ok = false;
        n = p.max_seqlen;
    }
    if (!ok && report) record_error(p.err, ERR_INDEX | SRC_LINEAR);
    return ok;
}

// State of sequence b, KV head h: its address (null: none kept) and whether the
// sequence starts from it.
__device__ __forceinline__ float *linear_state(const LinearParams &p, int b, int h, bool &from, bool report) {
    from = false;
    if (!p.state) return nullptr;
    const int64_t slot = __ldg(p.slots + b);
    if (slot < 0) return nullptr;
    if (slot >= p.num_slots) {
        if (report) record_error(p.err, ERR_INDEX | SRC_LINEAR);
        return nullptr;
    }
    from = p.context_lens ? __ldg(p.context_lens + b) > 0 : !p.start_zero;
    return p.state + (slot * p.Hkv + h) * (int64_t)p.D * p.D;
}

// log_decay of head h, at most 0: a positive or NaN value counts as 0 and is reported.
__device__ __forceinline__ float linear_log_decay(const LinearParams &p, int h, bool report) {
    const float g = __ldg(p.log_decay + h);
    if (report && !(g <= 0.f)) record_error(p.err, ERR_RANGE | SRC_LINEAR);
    return fminf(g, 0.f);
}

// One CTA per (sequence, KV head), token after token; the state in registers.
// Thread (dv, half) holds the float4s 2 m + half of row dv.
template <int D>
__global__ void __launch_bounds__(2 * D) linear_tokens_kernel(const LinearParams p) {
    __shared__ float ks[kLinStage][D], vs[kLinStage][D], qs[kLinStage][D];
    const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
    const int dv = tid >> 1, half = tid & 1;
    int64_t t0;
    int n;
    linear_rows(p, b, t0, n, h == 0 && tid == 0);
    if (n == 0) return;   // the state stays as it was
    bool from;
    float *state = linear_state(p, b, h, from, h == 0 && tid == 0);
    float S[D / 2];
#pragma unroll
    for (int m = 0; m < D / 8; ++m) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (from) x = *reinterpret_cast<const float4 *>(state + dv * D + 4 * (2 * m + half));
        S[4 * m] = x.x, S[4 * m + 1] = x.y, S[4 * m + 2] = x.z, S[4 * m + 3] = x.w;
    }
    const float a = expf(linear_log_decay(p, h, tid == 0));
    for (int c = 0; c < n; c += kLinStage) {
        const int m = min(kLinStage, n - c);
        __syncthreads();
        for (int x = tid; x < m * D; x += 2 * D) {
            const int64_t t = t0 + c + x / D;
            const int d = x % D;
            ks[x / D][d] = __bfloat162float(p.k[t * p.k_stride + h * D + d]);
            vs[x / D][d] = __bfloat162float(p.v[t * p.v_stride + h * D + d]);
        }
        for (int g = 0; g < p.G; ++g) {
            // every query head of the group runs over the same tokens; the state advances with the last
            __syncthreads();
            const int hq = h * p.G + g;
            for (int x = tid; x < m * D; x += 2 * D)
                qs[x / D][x % D] = __bfloat162float(p.q[(t0 + c + x / D) * p.q_stride + hq * D + x % D]);
            __syncthreads();
            float R[D / 2];
#pragma unroll
            for (int i = 0; i < D / 2; ++i) R[i] = S[i];
            for (int t = 0; t < m; ++t) {
                const float v = vs[t][dv];
                float o = 0.f;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const float4 k4 = *reinterpret_cast<const float4 *>(&ks[t][4 * (2 * i + half)]);
                    const float4 q4 = *reinterpret_cast<const float4 *>(&qs[t][4 * (2 * i + half)]);
                    R[4 * i] = fmaf(v, k4.x, a * R[4 * i]);
                    R[4 * i + 1] = fmaf(v, k4.y, a * R[4 * i + 1]);
                    R[4 * i + 2] = fmaf(v, k4.z, a * R[4 * i + 2]);
                    R[4 * i + 3] = fmaf(v, k4.w, a * R[4 * i + 3]);
                    o = fmaf(R[4 * i], q4.x, o);
                    o = fmaf(R[4 * i + 1], q4.y, o);
                    o = fmaf(R[4 * i + 2], q4.z, o);
                    o = fmaf(R[4 * i + 3], q4.w, o);
                }
                o += __shfl_xor_sync(0xffffffffu, o, 1);
                if (half == 0) p.out[(t0 + c + t) * p.out_stride + hq * D + dv] = __float2bfloat16_rn(o * p.scale);
            }
            if (g == p.G - 1) {
#pragma unroll
                for (int i = 0; i < D / 2; ++i) S[i] = R[i];
            }
        }
    }
    if (state) {
#pragma unroll
        for (int m = 0; m < D / 8; ++m)
            *reinterpret_cast<float4 *>(state + dv * D + 4 * (2 * m + half)) =
                make_float4(S[4 * m], S[4 * m + 1], S[4 * m + 2], S[4 * m + 3]);
    }
}

cudaError_t launch_tokens(const LinearParams &p, cudaStream_t stream) {
    const dim3 grid(p.Hkv, p.batch);
    main_kernel_event_before(stream);
    if (p.D == 128) linear_tokens_kernel<128><<<grid, 256, 0, stream>>>(p);
    else linear_tokens_kernel<64><<<grid, 128, 0, stream>>>(p);
    main_kernel_event_after(stream);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_varlen(const LinearParams &p, int num_sms, cudaStream_t stream) {
    (void)num_sms;
    return launch_tokens(p, stream);
}

cudaError_t launch_linear_decode(const LinearParams &p, int num_sms, cudaStream_t stream) {
    (void)num_sms;
    return launch_tokens(p, stream);
}

}  // namespace attn
