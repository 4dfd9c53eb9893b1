// softmax_layer.cuh -- what the kernels of the softmax-attention layers' operators share (pages.cu,
// qkrope.cu, attn_decode.cu): a division by a fixed number, packed arithmetic, programmatic launches.
#pragma once
#include "dr_common.cuh"

namespace dr {

// n / d for 0 <= n < 2^31, d >= 1, by a product: with 2^(s-1) < d <= 2^s and m = ceil(2^(31+s) / d)
// (32 bits), m d exceeds 2^(31+s) by less than d <= 2^s, so n m / 2^(31+s) exceeds n / d by less than
// 1 / d and has the same whole part.
struct FastDiv {
    uint32_t m;
    int s, d;
    FastDiv() = default;
    explicit FastDiv(int by) : s(0), d(by) {
        while (s < 31 && (1u << s) < (uint32_t)by) ++s;
        m = (uint32_t)(((1ull << (31 + s)) + (uint64_t)by - 1) / (uint64_t)by);
    }
    __device__ __forceinline__ int div(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> (31 + s)); }
};

// Elements of a paged cache from a page, a token, a head to the next (a head's channels are dense).
struct CacheStrides {
    long long page, token, head;
    __host__ __device__ bool operator==(const CacheStrides &o) const {
        return page == o.page && token == o.token && head == o.head;
    }
};

namespace f32x2 {
// Two fp32 numbers in a 64-bit register pair: Blackwell's packed arithmetic takes one issue slot
// for both.
typedef unsigned long long f2;
__device__ __forceinline__ f2 mk(float lo, float hi) {
    f2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void un(f2 x, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x)); }
__device__ __forceinline__ f2 mul(f2 a, f2 b) {
    f2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 fma(f2 a, f2 b, f2 c) {
    f2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f2 sub(f2 a, f2 b) {
    f2 d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float sum2(f2 x) {
    float a, b;
    un(x, a, b);
    return a + b;
}
}  // namespace f32x2

// Programmatic launch of a kernel that begins with after_previous(): it is set up while the kernel
// before it on the stream still runs (from when every block of that one has called let_next() or
// ended) and waits in after_previous() for that one's end.
template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}
// Nothing of global memory is touched before after_previous().  let_next() stands where a block's
// work ends, unless the next kernel is known to be small: blocks that are placed while others of
// this kernel still hold their SMs fall unevenly (a call of 256 blocks, replayed in a graph: 18.0 us
// with the trigger at its start, 14.5 with it at the end; behind another library's kernel on a stream such a
// call takes 18 us wherever the trigger stands).
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;"); }

}  // namespace dr
