// dr_common.cuh -- shared device helpers and argument structs of libdeltarule.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dr {

enum : int { VAR_DELTANET = 0, VAR_GATED = 1, VAR_KDA = 2 };

// Device error word: set by kernels whose bounded waits expire; read and cleared
// by delta_rule_sync_status().  Bit values below.  The library is one translation
// unit (delta_rule_lib.cu), so this is the only definition.
enum : int { DEVERR_TIMEOUT = 1 };
__device__ int g_dev_error = 0;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

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

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

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

// Problem geometry shared by all kernels.  N = number of chunks = ceil(T / C).
struct Geo {
    int B, T, H, dk, dv, C, N, variant;
    // element offset of token row (b, t, h) in a [B,T,H,*] tensor, before the *d
    __host__ __device__ __forceinline__ size_t row(int b, int t, int h) const {
        return ((size_t)b * T + t) * H + h;
    }
    // index of chunk n of (b, h) in chunk-major workspaces [B,H,N,...]
    __host__ __device__ __forceinline__ size_t chunk(int b, int h, int n) const {
        return ((size_t)b * H + h) * N + n;
    }
};

// Forward / backward tensor arguments (device pointers; see include/delta_rule.h).
struct Tensors {
    const void *q, *k, *v, *alpha, *beta;
    const float *S0;
    void *out, *u;
    float *S_T;
    const void *dout, *du;
    const float *dS_T;
    void *dq, *dk, *dv, *dalpha, *dbeta;
    float *dS0;
    // the fused forward (delta_rule_fwd_fused): q, k, alpha, beta hold the raw projections and
    // logits; the post-operation's gate logits and weight, and its output y
    const void *gate_o;
    const float *w_norm;
    void *y;
};

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
// this kernel still hold their SMs fall unevenly (a call whose 256 blocks began so took 18.0 us
// instead of 14.5).
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;"); }

// Optional launch timing: records ev[i] on the stream just before kernel launch i
// and ev[n_launches] after the last one (the *_timed entry points).  Inactive
// when ev is null.
struct Rec {
    cudaEvent_t *ev = nullptr;
    int n = 0, i = 0;
    bool bad = false;  // an event could not be recorded (invalid handle)
    void mark(cudaStream_t s) {
        if (ev && i < n && cudaEventRecord(ev[i++], s) != cudaSuccess) {
            cudaGetLastError();  // consume it: it is not a launch failure
            bad = true;
        }
    }
};

}  // namespace dr
