// rope_store.cu -- rotary positions (one or several axes) applied to q and k,
// fused with the scatter of k and v into the paged caches.
//
// Pair i of a head turns by angle = pos[axis(i)][token] * inv_freq[i]:
//   (a, b) -> scale * (a cos - b sin, a sin + b cos)
// where (a, b) are elements (i, i + half) or, interleaved, (2i, 2i + 1) of the
// first 2 * half; the rest of the head passes through.
//
// Angles.  In fp32 the product loses the fraction of a turn that matters once
// pos * inv_freq is large (position 10^6: 0.06 rad).  Here inv_freq / 2 pi is a
// 64-bit binary fraction of a turn and the product with the integer position
// wraps modulo one turn by itself: an error of 2^-52 of inv_freq * pos remains.  Its
// top 32 bits are the angle as a signed fraction of half a turn, rounded to fp32 (2^-25
// of half a turn at most) and handed to sincospif.
//
// Bound by HBM: q, k, v are read once, q_out, k and v rows written once.  A CTA
// takes a tile of tokens; the tile's sines and cosines are computed once into
// shared memory (one per token and pair, shared by all heads) while the first loads
// are in flight.  A work item is 32 bytes of a row: 8 pairs (two 16-byte vectors),
// 16 pass-through elements or 16 elements of v.  8,503 tokens of 32/8 heads of 128 with
// V / 16: 38.7 us in the kernel, 5.8 TB/s of what is read and written; 32,768 tokens without it 127 us,
// 6.3 TB/s; 64 tokens 7 us, a launch, the sines and one load's latency.
#include "common.cuh"
#include "kernels.h"

namespace attn {
namespace {

// 96 threads, 2 items of 32 bytes in flight each, 12 CTAs per SM (56 registers): 16,384-token
// and larger calls are fastest with small CTAs, whose loads and stores overlap those of their
// neighbours (32,768 tokens 32/8 heads of 128: 256 threads x 3 items 146 us, 64 x 3 134, 96 x 2
// 128.5, 64 x 6 172)
constexpr int kRopeThreads = 96;
constexpr int kRopeUnroll = 2;
constexpr int kRopeMinBlocks = 12;

// VEC pairs of one item: two vectors of VEC bf16
template <int VEC> struct RopeVec;
template <> struct RopeVec<8> {
    typedef uint4 type;
    static __device__ __forceinline__ uint4 load(const void *p) { return ldg_stream16(p); }
    static __device__ __forceinline__ void get(const uint4 &v, float (&x)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint4 put(const float (&x)[8]) {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                          pack_bf16x2(x[6], x[7]));
    }
    static __device__ __forceinline__ uint4 div16(const uint4 &v) {
        return make_uint4(bf16x2_to_f16x2_div16(v.x), bf16x2_to_f16x2_div16(v.y), bf16x2_to_f16x2_div16(v.z),
                          bf16x2_to_f16x2_div16(v.w));
    }
    // |v| >= 2^20 (bf16 pattern 0x4980) or non-finite in any element
    static __device__ __forceinline__ bool big(const uint4 &v) {
        const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                    __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
        return (m & 0xFFFFu) >= 0x4980u || (m >> 16) >= 0x4980u;
    }
};
template <> struct RopeVec<1> {
    typedef uint16_t type;
    static __device__ __forceinline__ uint16_t load(const void *p) { return __ldg((const uint16_t *)p); }
    static __device__ __forceinline__ void get(const uint16_t &v, float (&x)[1]) {
        x[0] = __uint_as_float((uint32_t)v << 16);
    }
    static __device__ __forceinline__ uint16_t put(const float (&x)[1]) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(x[0]));
    }
    static __device__ __forceinline__ uint16_t div16(const uint16_t &v) {
        const float x = __uint_as_float((uint32_t)v << 16) * 0.0625f;
        return __half_as_ushort(__float2half_rn(fminf(fmaxf(x, -65504.f), 65504.f)));
    }
    static __device__ __forceinline__ bool big(const uint16_t &v) { return (v & 0x7FFFu) >= 0x4980u; }
};

// cosine and sine of the angle of pair i of token t
__device__ __forceinline__ float2 rope_turn(const RopeParams &p, int64_t t, int i) {
    const double f = (double)__ldg(p.inv_freq + i) * 0.15915494309189535;   // turns per position
    const uint64_t f64 = __double2ull_rn((f - floor(f)) * 18446744073709551616.0);
    const int64_t pos = __ldg(p.positions + (int64_t)p.axis[i] * p.axis_stride + t);
    const int32_t half_turns = (int32_t)(((uint64_t)pos * f64) >> 32);
    float s, c;
    sincospif((float)half_turns * 4.656612873077393e-10f, &s, &c);          // 2^-31
    return make_float2(c * p.scale, s * p.scale);
}

// An item of a token: its two vectors, and where they are in the row.
template <int VEC>
struct RopeItem {
    typedef typename RopeVec<VEC>::type V;
    V x0, x1;
    int pair;        // first pair of a rotated item, -1: copied
    int off0, off1;  // element offsets of the two vectors inside the head
    int head;        // 0 .. Hq + 2 Hkv - 1 over q, k, v
};

template <int VEC, bool INTER>
__device__ __forceinline__ void rope_load(const RopeParams &p, int64_t t, int it, int per_head, uint32_t head_magic,
                                          RopeItem<VEC> &r) {
    r.head = head_magic ? __umulhi(it, head_magic) : it / per_head;
    const int c = it - r.head * per_head;
    const bool is_v = r.head >= p.Hq + p.Hkv;
    const __nv_bfloat16 *row;
    if (r.head < p.Hq) row = p.q + t * p.q_stride + (int64_t)r.head * p.D;
    else if (!is_v) row = p.k + t * p.k_stride + (int64_t)(r.head - p.Hq) * p.D;
    else row = p.v + t * p.v_stride + (int64_t)(r.head - p.Hq - p.Hkv) * p.D;
    r.pair = !is_v && c * VEC < p.half ? c * VEC : -1;
    if (r.pair >= 0 && !INTER) {
        r.off0 = c * VEC;
        r.off1 = p.half + c * VEC;
    } else {
        r.off0 = 2 * c * VEC;
        r.off1 = r.off0 + VEC;
    }
    r.x0 = RopeVec<VEC>::load(row + r.off0);
    r.x1 = RopeVec<VEC>::load(row + r.off1);
}

template <int VEC, bool INTER>
__device__ __forceinline__ void rope_write(const RopeParams &p, int64_t t, int64_t slot, const float2 *turn,
                                           RopeItem<VEC> &r, bool &big) {
    typedef RopeVec<VEC> RV;
    typedef typename RV::type V;
    if (r.pair >= 0) {
        float a[VEC], b[VEC], u[VEC], w[VEC];
        RV::get(r.x0, a);
        RV::get(r.x1, b);
        if (INTER && VEC > 1) {
            // pairs are neighbours: vector 0 holds pairs 0..VEC/2-1, vector 1 the others
#pragma unroll
            for (int i = 0; i < VEC; i += 2) {
                const float2 e = turn[r.pair + i / 2], f = turn[r.pair + VEC / 2 + i / 2];
                u[i] = a[i] * e.x - a[i + 1 < VEC ? i + 1 : i] * e.y;
                w[i] = b[i] * f.x - b[i + 1 < VEC ? i + 1 : i] * f.y;
                if (i + 1 < VEC) {
                    u[i + 1] = a[i] * e.y + a[i + 1] * e.x;
                    w[i + 1] = b[i] * f.y + b[i + 1] * f.x;
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float2 e = turn[r.pair + i];
                u[i] = a[i] * e.x - b[i] * e.y;
                w[i] = a[i] * e.y + b[i] * e.x;
            }
        }
        r.x0 = RV::put(u);
        r.x1 = RV::put(w);
    }
    __nv_bfloat16 *dst = nullptr;
    if (r.head < p.Hq) {
        dst = p.q_out + t * p.q_out_stride + (int64_t)r.head * p.D;
    } else if (r.head < p.Hq + p.Hkv) {
        if (p.k_out) {
            __nv_bfloat16 *o = p.k_out + t * p.k_out_stride + (int64_t)(r.head - p.Hq) * p.D;
            *reinterpret_cast<V *>(o + r.off0) = r.x0;
            *reinterpret_cast<V *>(o + r.off1) = r.x1;
        }
        if (slot >= 0) dst = p.k_cache + (slot * p.Hkv + (r.head - p.Hq)) * p.D;
    } else if (slot >= 0) {
        const int64_t at = (slot * p.Hkv + (r.head - p.Hq - p.Hkv)) * p.D;
        dst = p.v_cache + at;
        if (p.v16_cache) {
            big = big || RV::big(r.x0) || RV::big(r.x1);
            *reinterpret_cast<V *>(p.v16_cache + at + r.off0) = RV::div16(r.x0);
            *reinterpret_cast<V *>(p.v16_cache + at + r.off1) = RV::div16(r.x1);
        }
    }
    if (dst) {
        *reinterpret_cast<V *>(dst + r.off0) = r.x0;
        *reinterpret_cast<V *>(dst + r.off1) = r.x1;
    }
}

// tile_tokens consecutive tokens per CTA; shared memory: their sines and cosines.
// A thread loads kRopeUnroll items (32 bytes each) before it uses the first; the
// first ones are in flight while the sines and cosines are computed.
template <int VEC, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, kRopeMinBlocks) rope_store_kernel(const RopeParams p, int tile_tokens, int per_tok,
                                                                  uint32_t tok_magic, int per_head,
                                                                  uint32_t head_magic) {
    extern __shared__ float2 turns[];   // [tile_tokens][half]
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * tile_tokens;
    const int nt = (int)min((int64_t)tile_tokens, p.num_tokens - t0);
    const int items = nt * per_tok;
    bool bad = false, big = false, ready = false;
    for (int x0 = tid; x0 < items || !ready; x0 += kRopeThreads * kRopeUnroll) {
        RopeItem<VEC> r[kRopeUnroll];
        int64_t slot[kRopeUnroll];
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            const int x = x0 + u * kRopeThreads;
            slot[u] = -1;
            if (x >= items) continue;
            const int t = tok_magic ? __umulhi(x, tok_magic) : x / per_tok;
            if (p.k_cache) slot[u] = __ldg(p.slot_mapping + t0 + t);
            rope_load<VEC, INTER>(p, t0 + t, x - t * per_tok, per_head, head_magic, r[u]);
        }
        if (!ready) {
            for (int x = tid; x < nt * p.half; x += kRopeThreads) {
                const int t = x / p.half;
                turns[x] = rope_turn(p, t0 + t, x - t * p.half);
            }
            __syncthreads();
            ready = true;
        }
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            const int x = x0 + u * kRopeThreads;
            if (x >= items) continue;
            const int t = tok_magic ? __umulhi(x, tok_magic) : x / per_tok;
            int64_t s = slot[u];
            if (s >= p.num_slots) {
                bad = true;
                s = -1;
            }
            rope_write<VEC, INTER>(p, t0 + t, s, turns + t * p.half, r[u], big);
        }
    }
    const unsigned any_bad = __ballot_sync(0xffffffffu, bad), any_big = __ballot_sync(0xffffffffu, big);
    if ((tid & 31) == 0) {
        if (any_bad) record_error(p.err, ERR_INDEX | SRC_ROPE);
        if (any_big) record_error(p.err, ERR_RANGE | SRC_ROPE);
    }
}

// ceil(2^32 / d): __umulhi(x, it) is x / d for every x < 2^32 / d (0 for d = 1: divide)
uint32_t magic_of(int d) { return d > 1 ? (uint32_t)(((1ull << 32) + d - 1) / d) : 0; }

template <int VEC, bool INTER>
cudaError_t launch(const RopeParams &p, int num_sms, cudaStream_t stream) {
    const int per_head = p.D / (2 * VEC), per_tok = (p.Hq + p.Hkv + (p.v ? p.Hkv : 0)) * per_head;
    // one round of loads per thread, but first of all a CTA for every SM
    int64_t tile = (int64_t)kRopeUnroll * kRopeThreads / per_tok;
    if (tile > p.num_tokens / (2 * num_sms)) tile = p.num_tokens / (2 * num_sms);
    if (tile < 1) tile = 1;
    const bool magic = tile * (int64_t)per_tok * per_tok < (1ll << 32);
    const int64_t grid = (p.num_tokens + tile - 1) / tile;
    main_kernel_event_before(stream);
    rope_store_kernel<VEC, INTER><<<(unsigned)grid, kRopeThreads, tile * p.half * sizeof(float2), stream>>>(
        p, (int)tile, per_tok, magic ? magic_of(per_tok) : 0, per_head, magic ? magic_of(per_head) : 0);
    main_kernel_event_after(stream);
    return cudaGetLastError();
}

}  // namespace

// vec: every row, head and rotated half starts on a 16-byte boundary
cudaError_t launch_rope_store(const RopeParams &p, bool vec, int num_sms, cudaStream_t stream) {
    if (p.num_tokens == 0) return cudaSuccess;
    if (p.interleaved) return vec ? launch<8, true>(p, num_sms, stream) : launch<1, true>(p, num_sms, stream);
    return vec ? launch<8, false>(p, num_sms, stream) : launch<1, false>(p, num_sms, stream);
}

}  // namespace attn
