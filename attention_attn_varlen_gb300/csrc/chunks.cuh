// chunks.cuh -- what the kernels share that run a sequence in chunks with its state
// on the tensor cores: TMEM accesses, splits into bf16 parts, bounded waits, register
// shares, dependent launches.
#pragma once

#include "common.cuh"

namespace attn {

constexpr uint32_t kAMnMajor = 1u << 15;     // instruction descriptor: A along M in its 128-byte rows

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// A tcgen05.ld or .st takes about 40 clocks of its warp whatever its width: wide shapes.
// 16 lanes x 16 columns of 32 bits in the 8x8 matrix fragment layout: thread t holds (lane
// t / 4, column t % 4) and (lane t / 4 + 8, same column) of each group of four columns
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// 16 lanes x 32 columns: thread t gets, of each group of eight columns, (lane t / 4, columns
// 2 (t % 4) and + 1) and the same of lane t / 4 + 8
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

template <int N> __device__ __forceinline__ void more_regs() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void fewer_regs() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// one lane of the warp, the same every time; the operands of what it issues stay warp-uniform
// values to the compiler, which one of `lane == 0` does not give: 30 against 50 clocks per
// tcgen05.mma issued
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// four transposed 8x8 b16 matrices to shared memory (row addresses from lanes 8 m .. 8 m + 7)
__device__ __forceinline__ void stsm_x4_t(uint32_t addr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r0), "r"(r1),
                 "r"(r2), "r"(r3)
                 : "memory");
}

// x0, x1 -> their bf16 part (packed); r0, r1 become what is left (exact): fused multiply-adds
// that read the bf16 halves as they are, -1 times them (4 % fewer instructions than with their widening, 248 -> 243 us)
__device__ __forceinline__ uint32_t take_bf16(float &r0, float &r1, float x0, float x1) {
    const uint32_t h = pack_bf16x2(x0, x1);
    // (the outputs last: they may have the inputs' registers)
    asm("{\n\t.reg .b16 l, u, m;\n\t.reg .f32 a, b;\n\tmov.b32 {l, u}, %2;\n\tmov.b16 m, 0xBF80;\n\t"    // -1
        "fma.rn.f32.bf16 a, l, m, %3;\n\tfma.rn.f32.bf16 b, u, m, %4;\n\tmov.f32 %0, a;\n\tmov.f32 %1, b;\n\t}"
        : "=f"(r0), "=f"(r1)
        : "r"(h), "f"(x0), "f"(x1));
    return h;
}
__device__ __forceinline__ uint32_t take_bf16(float &x0, float &x1) { return take_bf16(x0, x1, x0, x1); }

// mbar_wait in few instructions: the kernel's roles share the instruction cache, and with a call
// in it the warpgroups could not have register shares of their own.  Gives up after about a
// second, or once another role has; the kernel's end reports it.
__device__ __forceinline__ bool chunk_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    uint32_t t0 = 0, t;
#pragma unroll 1
    do {
        // the timer only once in a while: its read would hold up what is waited for (16 prompts 266 -> 259 us)
#pragma unroll 1
        for (int i = 0; i < 16; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
        if (t0 == 0) t0 = t;
    } while (t - t0 < (uint32_t)kWaitLimitNs && !*abort);
    *abort = 1;
    return false;
}

// The same in fewer instructions, with the timer read at each try, which suits kernels in which a warp of its own
// does the waiting (the delta rule's prompts: 574 us, 589 with the one above; linear attention's 141, 139 with it).
// Gives up after 2^30 ns.
__device__ __forceinline__ bool chunk_wait_each(uint64_t *bar, uint32_t parity, volatile int *abort) {
    uint32_t t0, t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t0));
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
        asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
        if (((t - t0) >> 30) | *abort) {
            *abort = 1;
            return false;
        }
    }
    return true;
}

// kernel<<<grid, block, smem>>> as the programmatic dependent of the launch before it
template <typename... K, typename... A>
cudaError_t launch_after(void (*k)(K...), dim3 grid, unsigned block, size_t smem, cudaStream_t stream, const A &...a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a...);
}

}  // namespace attn
