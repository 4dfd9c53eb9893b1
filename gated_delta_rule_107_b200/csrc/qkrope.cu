// qkrope.cu -- the queries and keys of a softmax-attention layer: RMS norm of each head with a
// weight, and the rotation of channel pairs by the token's position, in one pass over memory.
//
// Per (token, head) row x of d channels, eps = 1e-6:
//   n = x r,  r = 1 / sqrt(mean(x^2) + eps),  y = n w
//   the first rot channels in pairs (a, b) -> (a cos - b sin, b cos + a sin), the pair's angle
//   position * inv_freq[i]; pair i is (i, i + rot/2), or (2i, 2i + 1) when interleaved
// Backward, for g = the gradient rotated back:
//   dw = sum over rows of g n,   dx = r (g w - n mean(g w n))
//
// A token's angles are the same for all its heads, so a group of d / (2 VEC) lanes takes one token
// and walks its heads: each lane owns two 16-byte vectors of every row, chosen so that the two
// halves of each channel pair meet in one lane, and computes its own angles once per token.  The
// angle is reduced to a fraction of a turn in 64 bits (position * inv_freq / 2 pi, minus the
// nearest whole number), because in 32 bits a position of 10^6 leaves an error of 0.06 rad; the
// fraction is then exact enough in 32 bits.
#include <type_traits>

#include "qkrope.cuh"
#include "prepost.cuh"

namespace dr {
namespace qkr {

constexpr float EPS = 1e-6f;
constexpr int THREADS = 256;
constexpr int PF_FWD = 5, PF_BWD = 5;  // slots of the rows ahead
constexpr int FWD_CTAS = 148 * 64, BWD_CTAS = 1184;  // at most; the backward's are also its partial sums
constexpr double INV_2PI = 0.15915494309189533577;

using pp::Vec;

// The lanes of a token and the two vectors a lane owns of each row (indexes of 16-byte vectors).
template <typename E, int D> struct Lay {
    static constexpr int VEC = 16 / (int)sizeof(E), LPT = D / (2 * VEC), TPW = 32 / LPT;
    int ia, ib;
    bool turned;  // the two vectors take part in the rotation
    __device__ __forceinline__ Lay(int j, int rot) {
        const int half = rot / (2 * VEC);
        turned = j < half;
        ia = turned ? j : 2 * j;
        ib = turned ? j + half : 2 * j + 1;
    }
};

template <int LPT> __device__ __forceinline__ float sum_group(float x) {
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// cosines and sines of a lane's VEC angles at a position; turns: the lane's first in the table of
// all of them, in turns per position
template <int VEC, bool INTER>
__device__ __forceinline__ void angles(int pos, const double *turns, int apart, bool turned, float *cs, float *sn) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        cs[i] = 1.f;
        sn[i] = 0.f;
        if (turned) {
            const double t = (double)pos * turns[INTER && i >= VEC / 2 ? apart + i : i];
            sincospif(2.f * (float)(t - rint(t)), &sn[i], &cs[i]);
        }
    }
}

__device__ __forceinline__ void cp16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The rows ahead of a lane: each lane copies the very vectors that it will use into a ring of its
// own in shared memory (PF slots of NV vectors, a vector of the warp's 32 lanes side by side), so
// that a warp has PF - 1 rows' loads in flight without holding them in registers, and no lane
// waits for another.  A slot is filled again one row after its values were used.
template <int NV, int PF> struct Ring {
    uint4 *base;
    int put = 0, got = 0;
    static constexpr int WARP_BYTES = PF * NV * 32 * 16;
    __device__ __forceinline__ Ring(char *smem) {
        base = reinterpret_cast<uint4 *>(smem + (threadIdx.x >> 5) * WARP_BYTES) + (threadIdx.x & 31);
    }
    __device__ __forceinline__ uint4 *slot(int s, int v) { return base + (s * NV + v) * 32; }
    __device__ __forceinline__ void pushed() {
        cp_commit();
        put = put + 1 == PF ? 0 : put + 1;
    }
    __device__ __forceinline__ void popped() { got = got + 1 == PF ? 0 : got + 1; }
};

// rotates the pairs of (a, b) by the angles, or back (DIR = -1)
template <int VEC, bool INTER, int DIR>
__device__ __forceinline__ void rotate(float *a, float *b, const float *cs, const float *sn) {
    if (INTER) {
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const float c0 = cs[i], s0 = DIR * sn[i], c1 = cs[VEC / 2 + i], s1 = DIR * sn[VEC / 2 + i];
            const float a0 = a[2 * i], a1 = a[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
            a[2 * i] = a0 * c0 - a1 * s0;
            a[2 * i + 1] = a1 * c0 + a0 * s0;
            b[2 * i] = b0 * c1 - b1 * s1;
            b[2 * i + 1] = b1 * c1 + b0 * s1;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float c = cs[i], s = DIR * sn[i], x = a[i], y = b[i];
            a[i] = x * c - y * s;
            b[i] = y * c + x * s;
        }
    }
}

template <typename E, int D>
__device__ __forceinline__ void load_w(const float *w, const Lay<E, D> &l, float *wa, float *wb) {
    constexpr int VEC = Lay<E, D>::VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        wa[i] = w ? w[l.ia * VEC + i] : 1.f;
        wb[i] = w ? w[l.ib * VEC + i] : 1.f;
    }
}

// inv_freq in turns per position, for the whole CTA
template <int D> __device__ __forceinline__ void fill_turns(double *turns, const QkRope &p) {
    for (int i = threadIdx.x; i < p.rot / 2; i += THREADS) turns[i] = p.inv_freq[i] * INV_2PI;
    __syncthreads();
}
// the lane's first angle in that table, and (interleaved) where its second vector's begin
template <typename E, int D, bool INTER> __device__ __forceinline__ int first_turn(const Lay<E, D> &l, int j, int *apart) {
    constexpr int VEC = Lay<E, D>::VEC;
    *apart = (l.ib - l.ia) * (VEC / 2) - VEC / 2;
    return INTER ? l.ia * (VEC / 2) : j * VEC;
}

// The heads are cut into chunks of hpg (blockIdx.y), so that a call of few tokens still has many
// warps: a chunk [h0, h1) of the Hq + Hk (cache: + Hk values) heads.
template <typename E, int D, bool INTER, bool CACHE>
__global__ void __launch_bounds__(THREADS, 3) k_qkrope(const QkRope p, int hpg) {
    using L = Lay<E, D>;
    constexpr int VEC = L::VEC, LPT = L::LPT, TPW = L::TPW;
    extern __shared__ __align__(16) char ring_smem[];
    __shared__ double turns[D / 2];
    const int lane = threadIdx.x & 31, j = lane % LPT;
    const L l(j, p.rot);
    const int heads = p.Hq + p.Hk * (CACHE ? 2 : 1);
    const int h0 = blockIdx.y * hpg, h1 = min(heads, h0 + hpg);
    const size_t step = (size_t)gridDim.x * (THREADS / 32) * TPW;
    size_t n0 = ((size_t)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5)) * TPW;

    Ring<2, PF_FWD> ring(ring_smem);
    auto token = [&](size_t at) { return min(at + lane / LPT, p.N - 1); };  // behind the last: computed, not stored
    size_t ln = n0;  // the row whose load is next
    int lh = h0;
    auto push = [&]() {
        if (ln < p.N) {
            const size_t n = token(ln);
            const E *src;
            if (lh < p.Hq) src = (const E *)p.q + n * p.qs + lh * D;
            else if (!CACHE || lh < p.Hq + p.Hk) src = (const E *)p.k + n * p.ks + (lh - p.Hq) * D;
            else src = (const E *)p.v + n * p.vs + (lh - p.Hq - p.Hk) * D;
            cp16(ring.slot(ring.put, 0), src + l.ia * VEC);
            cp16(ring.slot(ring.put, 1), src + l.ib * VEC);
            if (++lh == h1) {
                lh = h0;
                ln += step;
            }
        }
        ring.pushed();
    };
#pragma unroll
    for (int i = 0; i < PF_FWD - 1; ++i) push();
    fill_turns<D>(turns, p);
    int apart;
    const double *mine = turns + first_turn<E, D, INTER>(l, j, &apart);
    for (; n0 < p.N; n0 += step) {
        const bool act = n0 + lane / LPT < p.N;
        const size_t n = token(n0);
        float cs[VEC], sn[VEC];
        angles<VEC, INTER>(p.pos ? p.pos[n] : (int)(n % p.T), mine, apart, l.turned, cs, sn);
        E *qdst = (E *)p.qo + n * ((size_t)p.Hq * D), *kdst = nullptr, *vdst = nullptr;
        if (CACHE) {
            const long long slot = p.slots[n];
            if (slot >= 0 && slot < p.n_slots) {
                const long long pg = slot / p.page, in = slot - pg * p.page;
                kdst = (E *)p.kc + pg * p.kps + in * ((long long)p.Hk * D);
                vdst = (E *)p.vc + pg * p.vps + in * ((long long)p.Hk * D);
            }
        } else {
            kdst = (E *)p.ko + n * ((size_t)p.Hk * D);
        }
        // heads [from, to) of one tensor, to dst, dense in the head
        auto run = [&](E *dst, const float *w, int from, int to) {
            if (from >= to) return;
            float wa[VEC], wb[VEC];
            load_w<E, D>(w, l, wa, wb);
            for (int h = from; h < to; ++h) {
                float a[VEC], b[VEC], ss = 0.f;
                cp_wait<PF_FWD - 2>();
                Vec<E, VEC>::ld(reinterpret_cast<const E *>(ring.slot(ring.got, 0)), a);
                Vec<E, VEC>::ld(reinterpret_cast<const E *>(ring.slot(ring.got, 1)), b);
                push();
                ring.popped();
#pragma unroll
                for (int i = 0; i < VEC; ++i) ss += a[i] * a[i] + b[i] * b[i];
                const float r = rsqrtf(sum_group<LPT>(ss) * (1.f / D) + EPS);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    a[i] *= r * wa[i];
                    b[i] *= r * wb[i];
                }
                rotate<VEC, INTER, 1>(a, b, cs, sn);
                if (act && dst) {
                    Vec<E, VEC>::st(dst + h * D + l.ia * VEC, a);
                    Vec<E, VEC>::st(dst + h * D + l.ib * VEC, b);
                }
            }
        };
        run(qdst, p.wq, min(h0, p.Hq), min(h1, p.Hq));
        run(kdst, p.wk, max(h0 - p.Hq, 0), min(h1 - p.Hq, p.Hk));
        if (CACHE) {
            for (int h = max(h0 - p.Hq - p.Hk, 0); h < h1 - p.Hq - p.Hk; ++h) {
                cp_wait<PF_FWD - 2>();
                const uint4 a = *ring.slot(ring.got, 0), b = *ring.slot(ring.got, 1);
                push();
                ring.popped();
                if (act && vdst) {
                    *reinterpret_cast<uint4 *>(vdst + h * D + l.ia * VEC) = a;
                    *reinterpret_cast<uint4 *>(vdst + h * D + l.ib * VEC) = b;
                }
            }
        }
    }
}

// part (or null): [CTA][2][D], the CTA's sums of the weights' gradients (query, key)
template <typename E, int D, bool INTER>
__global__ void __launch_bounds__(THREADS, 2) k_qkrope_bwd(const QkRope p, int hpg) {
    using L = Lay<E, D>;
    constexpr int VEC = L::VEC, LPT = L::LPT, TPW = L::TPW, WARPS = THREADS / 32;
    extern __shared__ __align__(16) char ring_smem[];
    __shared__ float red[WARPS][2][D];
    __shared__ double turns[D / 2];
    __shared__ __align__(16) float wsh[2][D];  // the weights (in registers they would be spilled)
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = lane % LPT;
    const L l(j, p.rot);
    const int h0 = blockIdx.y * hpg, h1 = min(p.Hq + p.Hk, h0 + hpg);
    const size_t step = (size_t)gridDim.x * WARPS * TPW;
    size_t n0 = ((size_t)blockIdx.x * WARPS + warp) * TPW;

    Ring<4, PF_BWD> ring(ring_smem);
    auto token = [&](size_t at) { return min(at + lane / LPT, p.N - 1); };
    size_t ln = n0;
    int lh = h0;
    auto push = [&]() {
        if (ln < p.N) {
            const size_t n = token(ln);
            const bool isq = lh < p.Hq;
            const E *x = isq ? (const E *)p.q + n * p.qs + lh * D : (const E *)p.k + n * p.ks + (lh - p.Hq) * D;
            const E *g = isq ? (const E *)p.gq + (n * p.Hq + lh) * D : (const E *)p.gk + (n * p.Hk + lh - p.Hq) * D;
            cp16(ring.slot(ring.put, 0), x + l.ia * VEC);
            cp16(ring.slot(ring.put, 1), x + l.ib * VEC);
            cp16(ring.slot(ring.put, 2), g + l.ia * VEC);
            cp16(ring.slot(ring.put, 3), g + l.ib * VEC);
            if (++lh == h1) {
                lh = h0;
                ln += step;
            }
        }
        ring.pushed();
    };
#pragma unroll
    for (int i = 0; i < PF_BWD - 1; ++i) push();
    for (int i = threadIdx.x; i < 2 * D; i += THREADS) {
        const float *w = i < D ? p.wq : p.wk;
        wsh[i / D][i % D] = w ? w[i % D] : 1.f;
    }
    fill_turns<D>(turns, p);
    int apart;
    const double *mine = turns + first_turn<E, D, INTER>(l, j, &apart);
    float dwq[2 * VEC] = {}, dwk[2 * VEC] = {};
    for (; n0 < p.N; n0 += step) {
        const bool act = n0 + lane / LPT < p.N;
        const size_t n = token(n0);
        float cs[VEC], sn[VEC];
        angles<VEC, INTER>(p.pos ? p.pos[n] : (int)(n % p.T), mine, apart, l.turned, cs, sn);
        auto run = [&](E *dst, const float *w, float *dw, int from, int to) {
            for (int h = from; h < to; ++h) {
                float a[VEC], b[VEC], ga[VEC], gb[VEC], ss = 0.f, sg = 0.f;
                cp_wait<PF_BWD - 2>();
                Vec<E, VEC>::ld(reinterpret_cast<const E *>(ring.slot(ring.got, 0)), a);
                Vec<E, VEC>::ld(reinterpret_cast<const E *>(ring.slot(ring.got, 1)), b);
                Vec<E, VEC>::ld(reinterpret_cast<const E *>(ring.slot(ring.got, 2)), ga);
                Vec<E, VEC>::ld(reinterpret_cast<const E *>(ring.slot(ring.got, 3)), gb);
                push();
                ring.popped();
                rotate<VEC, INTER, -1>(ga, gb, cs, sn);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    ss += a[i] * a[i] + b[i] * b[i];
                    sg += a[i] * (ga[i] * w[l.ia * VEC + i]) + b[i] * (gb[i] * w[l.ib * VEC + i]);
                }
                const float r = rsqrtf(sum_group<LPT>(ss) * (1.f / D) + EPS);
                const float c = sum_group<LPT>(sg) * (1.f / D) * r * r;  // mean(g w n) / r, n = x r
                if (act) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        dw[i] += ga[i] * (a[i] * r);
                        dw[VEC + i] += gb[i] * (b[i] * r);
                        a[i] = r * (ga[i] * w[l.ia * VEC + i] - a[i] * c);
                        b[i] = r * (gb[i] * w[l.ib * VEC + i] - b[i] * c);
                    }
                    Vec<E, VEC>::st(dst + h * D + l.ia * VEC, a);
                    Vec<E, VEC>::st(dst + h * D + l.ib * VEC, b);
                }
            }
        };
        run((E *)p.dq + n * p.dqs, wsh[0], dwq, min(h0, p.Hq), min(h1, p.Hq));
        run((E *)p.dk + n * p.dks, wsh[1], dwk, max(h0 - p.Hq, 0), min(h1 - p.Hq, p.Hk));
    }
    if (!p.part) return;
    // over the warp's tokens, then over the warps in order
#pragma unroll
    for (int i = 0; i < 2 * VEC; ++i) {
#pragma unroll
        for (int o = LPT; o < 32; o <<= 1) {
            dwq[i] += __shfl_xor_sync(0xffffffffu, dwq[i], o);
            dwk[i] += __shfl_xor_sync(0xffffffffu, dwk[i], o);
        }
        if (lane < LPT) {
            const int at = (i < VEC ? l.ia * VEC + i : l.ib * VEC + i - VEC);
            red[warp][0][at] = dwq[i];
            red[warp][1][at] = dwk[i];
        }
    }
    __syncthreads();
    const size_t cta = (size_t)blockIdx.y * gridDim.x + blockIdx.x;
    for (int x = threadIdx.x; x < 2 * D; x += THREADS) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) s += (&red[w][0][0])[x];
        p.part[cta * 2 * D + x] = s;
    }
}

// dwq, dwk = the partials' sums in order: 32 columns a CTA, 32 partials at a time
template <int D> __global__ void __launch_bounds__(1024) k_qkrope_dw(const float *part, int n, float *dwq, float *dwk) {
    __shared__ float red[32][33];
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5, col = blockIdx.x * 32 + cx;
    float s = 0.f;
    for (int r = ry; r < n; r += 32) s += part[(size_t)r * 2 * D + col];
    red[ry][cx] = s;
    __syncthreads();
    s = warp_sum(red[cx][ry]);  // warp ry: column ry of the CTA's 32
    const int at = blockIdx.x * 32 + ry;
    if (cx == 0) {
        if (at < D) {
            if (dwq) dwq[at] = s;
        } else if (dwk) {
            dwk[at - D] = s;
        }
    }
}

// Grid: tokens over x, head chunks over y.  The heads are only cut when whole tokens would leave
// the GPU short of warps (16 an SM).
struct Grid {
    dim3 grid;
    int hpg;
};
static Grid plan(size_t N, int heads, int tpw, size_t max_ctas) {
    const size_t warps = (N + tpw - 1) / tpw, want = 148 * 16;
    const int chunks = (int)min((size_t)heads, max((size_t)1, want / max((size_t)1, warps)));
    const int hpg = (heads + chunks - 1) / chunks, ny = (heads + hpg - 1) / hpg;
    const size_t nx = min((warps + THREADS / 32 - 1) / (THREADS / 32), max((size_t)1, max_ctas / ny));
    return {dim3((unsigned)nx, (unsigned)ny), hpg};
}

template <typename E, int D, bool INTER> static cudaError_t fwd(const QkRope &p, cudaStream_t s) {
    const bool cache = p.slots != nullptr;
    const Grid g = plan(p.N, p.Hq + p.Hk * (cache ? 2 : 1), Lay<E, D>::TPW, FWD_CTAS);
    auto go = [&](auto kern) -> cudaError_t {
        constexpr int smem = Ring<2, PF_FWD>::WARP_BYTES * (THREADS / 32);
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        kern<<<g.grid, THREADS, smem, s>>>(p, g.hpg);
        return cudaGetLastError();
    };
    return cache ? go(k_qkrope<E, D, INTER, true>) : go(k_qkrope<E, D, INTER, false>);
}

template <typename E, int D, bool INTER> static cudaError_t bwd(const QkRope &p, cudaStream_t s) {
    const Grid g = plan(p.N, p.Hq + p.Hk, Lay<E, D>::TPW, BWD_CTAS);
    constexpr int smem = Ring<4, PF_BWD>::WARP_BYTES * (THREADS / 32);
    const cudaError_t e = cudaFuncSetAttribute(k_qkrope_bwd<E, D, INTER>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    QkRope a = p;
    if (!p.dwq && !p.dwk) a.part = nullptr;
    k_qkrope_bwd<E, D, INTER><<<g.grid, THREADS, smem, s>>>(a, g.hpg);
    if (a.part) k_qkrope_dw<D><<<2 * D / 32, 1024, 0, s>>>(a.part, (int)(g.grid.x * g.grid.y), p.dwq, p.dwk);
    return cudaGetLastError();
}

template <typename F> static cudaError_t by_type(const QkRope &p, bool bf16, F f) {
    return bf16 ? f((__nv_bfloat16 *)nullptr) : f((float *)nullptr);
}

}  // namespace qkr

// one partial of both weights' gradients per CTA
size_t qkrope_ws_bytes(int d) { return (size_t)qkr::BWD_CTAS * 2 * d * sizeof(float); }

cudaError_t qkrope_run(const QkRope &p, bool bf16, cudaStream_t s) {
    return qkr::by_type(p, bf16, [&](auto *e) -> cudaError_t {
        using E = std::remove_pointer_t<decltype(e)>;
        if (p.d == 128) return p.interleaved ? qkr::fwd<E, 128, true>(p, s) : qkr::fwd<E, 128, false>(p, s);
        return p.interleaved ? qkr::fwd<E, 64, true>(p, s) : qkr::fwd<E, 64, false>(p, s);
    });
}

cudaError_t qkrope_bwd_run(const QkRope &p, bool bf16, cudaStream_t s) {
    return qkr::by_type(p, bf16, [&](auto *e) -> cudaError_t {
        using E = std::remove_pointer_t<decltype(e)>;
        if (p.d == 128) return p.interleaved ? qkr::bwd<E, 128, true>(p, s) : qkr::bwd<E, 128, false>(p, s);
        return p.interleaved ? qkr::bwd<E, 64, true>(p, s) : qkr::bwd<E, 64, false>(p, s);
    });
}

}  // namespace dr
