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
// channels of each pair meet in one lane, and computes its own angles once per token.  The
// angle is reduced to a fraction of a turn in 64 bits (position * inv_freq / 2 pi, minus the
// nearest whole number), because in 32 bits a position of 10^6 leaves an error of 0.06 rad; the
// fraction is then exact enough in 32 bits.
//
// What bounds it is moving each element twice (forward) or three times (backward).  At 8 x 4096
// tokens of 10 heads of 128 channels in bf16: forward 30.6 us for 168 MB (5.5 TB/s, 85 % of a plain
// copy's rate), backward 46.0 us for 252 MB (85 %), in calls replayed in a graph; 31.6 and 47.8 (82 %)
// behind other kernels on a stream.  8192 tokens of 16 + 2 + 2 heads into the cache, 84 MB: 14.5 us (89 %)
// in a graph, 18.2 (71 %) on a stream, most likely because its 256 blocks, a wave that is not full, fall
// unevenly on the SMs there.  To get there the loads run ahead through shared memory (with loads into
// registers the forward took 50.8 us, its warps waiting), the arithmetic is packed (without, 70 % of
// all issue slots were taken), and neighbouring lanes always hold neighbouring vectors (with the
// channels behind rot two vectors a lane side by side, 32768 tokens with half of the channels
// rotated took 118 us backward instead of 86).
#include <cfloat>
#include <type_traits>

#include "qkrope.cuh"
#include "prepost.cuh"

namespace dr {
namespace qkr {

constexpr float EPS = 1e-6f;
constexpr int THREADS = 256;
constexpr int PF_FWD = 5, PF_BWD = 3;  // slots of the rows ahead (backward with 2: 52.0 us at 8 x 4096, 3: 46.1, 4: 48.2)
constexpr long long WARPS_WANTED = 16 * 148;
constexpr int BWD_CTAS = 2 * 148;         // one wave; they are also the number of its partial sums
constexpr double INV_2PI = 0.15915494309189533577;

using namespace dr::f32x2;

// The lanes of a token and what a lane holds of each row: two 16-byte vectors (indexes ia, ib),
// chosen so that the two channels of each pair meet in the lane, as VEC first and VEC second
// channels of pairs, two to a register pair: channels i of the vectors a and b (pairs (i, i + rot/2)),
// or the even and the odd channels of both (interleaved).  Channels behind rot are held alike and
// not turned.
template <typename E, int D, bool INTER> struct Lay {
    static constexpr int VEC = 16 / (int)sizeof(E), N2 = VEC / 2, LPT = D / (2 * VEC), TPW = 32 / LPT;
    int j, ia, ib;
    bool turned;  // the lane's pairs take part in the rotation
    __device__ __forceinline__ Lay(int j_, int rot) : j(j_) {
        const int half = rot / (2 * VEC);
        turned = j < half;
        ia = turned ? j : j + half;  // neighbouring lanes hold neighbouring vectors
        ib = turned ? j + half : j + LPT;
    }
    // the channel of the i-th first (0) or second (1) number
    __device__ __forceinline__ int channel(int second, int i) const {
        if (INTER) return (i < VEC / 2 ? ia : ib) * VEC + 2 * (i % (VEC / 2)) + second;
        return (second ? ib : ia) * VEC + i;
    }
    // the pair (its index into inv_freq) of the i-th numbers
    __device__ __forceinline__ int pair(int i) const {
        return INTER ? (i < VEC / 2 ? ia : ib) * (VEC / 2) + i % (VEC / 2) : j * VEC + i;
    }
};

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// a row's two vectors to numbers and back
template <bool INTER> __device__ __forceinline__ void open(const uint4 &a, const uint4 &b, f2 *A, f2 *B, __nv_bfloat16 *) {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (INTER) {
            const uint32_t p = i < 2 ? u[2 * i] : v[2 * i - 4], q = i < 2 ? u[2 * i + 1] : v[2 * i - 3];
            A[i] = mk(lo_f(p), lo_f(q));
            B[i] = mk(hi_f(p), hi_f(q));
        } else {
            A[i] = mk(lo_f(u[i]), hi_f(u[i]));
            B[i] = mk(lo_f(v[i]), hi_f(v[i]));
        }
    }
}
template <bool INTER> __device__ __forceinline__ void open(const uint4 &a, const uint4 &b, f2 *A, f2 *B, float *) {
    const float u[4] = {__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w)};
    const float v[4] = {__uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w)};
    if (INTER) {
        A[0] = mk(u[0], u[2]); B[0] = mk(u[1], u[3]);
        A[1] = mk(v[0], v[2]); B[1] = mk(v[1], v[3]);
    } else {
        A[0] = mk(u[0], u[1]); A[1] = mk(u[2], u[3]);
        B[0] = mk(v[0], v[1]); B[1] = mk(v[2], v[3]);
    }
}
__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&x);
}
template <bool INTER> __device__ __forceinline__ void close(const f2 *A, const f2 *B, uint4 &a, uint4 &b, __nv_bfloat16 *) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x, y, z, t;
        un(A[i], x, y);
        un(B[i], z, t);
        w[INTER ? 2 * i : i] = INTER ? bf2(x, z) : bf2(x, y);
        w[INTER ? 2 * i + 1 : 4 + i] = INTER ? bf2(y, t) : bf2(z, t);
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
    b = make_uint4(w[4], w[5], w[6], w[7]);
}
template <bool INTER> __device__ __forceinline__ void close(const f2 *A, const f2 *B, uint4 &a, uint4 &b, float *) {
    float x[4], y[4];  // firsts, seconds
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        un(A[i], x[2 * i], x[2 * i + 1]);
        un(B[i], y[2 * i], y[2 * i + 1]);
    }
    auto put = [](float p, float q, float r, float s) {
        return make_uint4(__float_as_uint(p), __float_as_uint(q), __float_as_uint(r), __float_as_uint(s));
    };
    a = INTER ? put(x[0], y[0], x[1], y[1]) : put(x[0], x[1], x[2], x[3]);
    b = INTER ? put(x[2], y[2], x[3], y[3]) : put(y[0], y[1], y[2], y[3]);
}

template <int LPT> __device__ __forceinline__ float sum_group(float x) {
#pragma unroll
    for (int o = LPT / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// What all tokens share, in shared memory: inv_freq in turns per position (0 for channels that are
// not turned) and both weights, in the order in which the lanes hold them.
template <typename E, int D, bool INTER> struct Shared {
    using L = Lay<E, D, INTER>;
    static constexpr int VEC = L::VEC, LPT = L::LPT;
    double turns[VEC][LPT];
    float4 w[2][VEC / 2][LPT];  // firsts, then seconds

    __device__ __forceinline__ void fill(const QkRope &p) {
        for (int x = threadIdx.x; x < 2 * D; x += THREADS) {
            const int which = x / D, at = x % D, j = at / (2 * VEC), i = at % (2 * VEC);
            const L l(j, p.rot);
            const int ch = l.channel(i >= VEC, i % VEC);
            const float *src = which ? p.wk : p.wq;
            reinterpret_cast<float *>(&w[which][i / 4][j])[i % 4] = src ? src[ch] : 1.f;
            if (which == 0 && i < VEC) turns[i][j] = l.turned ? p.inv_freq[l.pair(i)] * INV_2PI : 0.0;
        }
        __syncthreads();
    }
    __device__ __forceinline__ void weights(int which, int j, f2 *A, f2 *B) const {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const float4 u = w[which][i][j], v = w[which][VEC / 4 + i][j];
            A[2 * i] = mk(u.x, u.y); A[2 * i + 1] = mk(u.z, u.w);
            B[2 * i] = mk(v.x, v.y); B[2 * i + 1] = mk(v.z, v.w);
        }
    }
    // Cosines and sines of a lane's angles.  fp32 results, the weights' gradients of every type among
    // them, take sincospif (2 ulp; backward 45.7 -> 46.0 us at 8 x 4096).  Where all results are bf16
    // (FAST) the fast sine and cosine serve, off by less than 2^-20 here: a 4096th of the rounding of the
    // pair's larger channel, and a few instructions instead of some forty (8 x 4096 tokens 30.6 us instead
    // of 31.1, 8192 into the cache 14.5 instead of 15.1; a series of eleven terms in packed arithmetic 31.1
    // and 15.8).
    template <bool FAST> __device__ __forceinline__ void angles(int pos, int j, f2 *cs, f2 *sn) const {
        const double p = (double)pos;
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
            float c[2], s[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const double t = p * turns[i + k][j];
                const float f = (float)(t - rint(t));
                if (FAST) {
                    s[k] = __sinf(6.28318530717958647692f * f);
                    c[k] = __cosf(6.28318530717958647692f * f);
                } else {
                    sincospif(2.f * f, &s[k], &c[k]);
                }
            }
            cs[i / 2] = mk(c[0], c[1]);
            sn[i / 2] = mk(s[0], s[1]);
        }
    }
};

// (A, B) -> (A cos - B sin, B cos + A sin), or BACK
template <int N2, bool BACK> __device__ __forceinline__ void rotate(f2 *A, f2 *B, const f2 *cs, const f2 *sn) {
#pragma unroll
    for (int i = 0; i < N2; ++i) {
        const f2 x = A[i], y = B[i];
        if (BACK) {
            A[i] = fma(x, cs[i], mul(y, sn[i]));
            B[i] = sub(mul(y, cs[i]), mul(x, sn[i]));
        } else {
            A[i] = sub(mul(x, cs[i]), mul(y, sn[i]));
            B[i] = fma(y, cs[i], mul(x, sn[i]));
        }
    }
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

// The rows ahead of a lane: each lane copies the very vectors that it will use into a ring of its
// own in shared memory (PF slots of NV vectors, a vector of the warp's 32 lanes side by side), so
// that a warp has PF - 1 rows' loads in flight without holding them in registers, and no lane
// waits for another.  A slot is filled again one row after its values were used.
template <int NV, int PF> struct Ring {
    static constexpr int VECTOR = 32 * 16, SLOT = NV * VECTOR, WARP_BYTES = PF * SLOT;
    uint32_t base, put, got;
    __device__ __forceinline__ explicit Ring(char *smem) {
        base = (uint32_t)__cvta_generic_to_shared(smem) + (threadIdx.x >> 5) * WARP_BYTES + (threadIdx.x & 31) * 16;
        put = got = base;
    }
    __device__ __forceinline__ void pushed() {
        cp_commit();
        put = put == base + (PF - 1) * SLOT ? base : put + SLOT;
    }
    __device__ __forceinline__ void popped() { got = got == base + (PF - 1) * SLOT ? base : got + SLOT; }
    static __device__ __forceinline__ void wait() { cp_wait<PF - 2>(); }
};

// The heads are cut into chunks of hpg (blockIdx.y), so that a call of few tokens still has many
// warps: a chunk [h0, h1) of the Hq + Hk (cache: + Hk values) heads.
template <typename E, int D, bool INTER, bool CACHE>
__global__ void __launch_bounds__(THREADS, 3) k_qkrope(const QkRope p, int hpg) {
    using L = Lay<E, D, INTER>;
    constexpr int VEC = L::VEC, N2 = L::N2, LPT = L::LPT, TPW = L::TPW;
    extern __shared__ __align__(16) char ring_smem[];
    __shared__ Shared<E, D, INTER> sh;
    const int lane = threadIdx.x & 31, j = lane % LPT;
    const L l(j, p.rot);
    const int heads = p.Hq + p.Hk * (CACHE ? 2 : 1);
    const int h0 = blockIdx.y * hpg, h1 = min(heads, h0 + hpg);
    const unsigned N = (unsigned)p.N, step = gridDim.x * (THREADS / 32) * TPW;  // N < 2^31: no sum wraps
    unsigned n0 = (blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5)) * TPW;

    after_previous();
    Ring<2, PF_FWD> ring(ring_smem);
    auto token = [&](unsigned at) { return (size_t)min(at + lane / LPT, N - 1); };  // behind the last: computed, not stored
    unsigned ln = n0;               // the token whose row is copied next,
    int lh = h0, left = 0;        // the head behind it, how many of the tensor's rows are left,
    const E *src = nullptr;       // the row
    auto push = [&]() {
        if (ln < N) {
            if (left == 0) {  // the next tensor of the token
                const size_t n = token(ln);
                if (lh < p.Hq) {
                    src = (const E *)p.q + n * p.qs + lh * D;
                    left = min(h1, p.Hq) - lh;
                } else if (!CACHE || lh < p.Hq + p.Hk) {
                    src = (const E *)p.k + n * p.ks + (lh - p.Hq) * D;
                    left = min(h1, p.Hq + p.Hk) - lh;
                } else {
                    src = (const E *)p.v + n * p.vs + (lh - p.Hq - p.Hk) * D;
                    left = h1 - lh;
                }
                lh += left;
            }
            cp16(ring.put, src + l.ia * VEC);
            cp16(ring.put + ring.VECTOR, src + l.ib * VEC);
            src += D;
            if (--left == 0 && lh == h1) {
                lh = h0;
                ln += step;
            }
        }
        ring.pushed();
    };
#pragma unroll
    for (int i = 0; i < PF_FWD - 1; ++i) push();
    sh.fill(p);
    for (; n0 < N; n0 += step) {
        const bool act = n0 + lane / LPT < N;
        const size_t n = token(n0);
        f2 cs[N2], sn[N2];
        sh.template angles<sizeof(E) == 2>(p.pos ? p.pos[n] : (int)((unsigned)n % (unsigned)p.T), j, cs, sn);
        // heads [from, to) of one tensor, to dst, `apart` from head to head
        auto run = [&](E *dst, long long apart, int which, int from, int to) {
            if (from >= to) return;
            f2 wA[N2], wB[N2];
            sh.weights(which, j, wA, wB);
            const bool store = act && dst;
            dst += from * apart;
#pragma unroll 1
            for (int h = from; h < to; ++h, dst += apart) {
                f2 A[N2], B[N2], ss = 0;
                ring.wait();
                const uint32_t at = ring.got;
                open<INTER>(lds16(at), lds16(at + ring.VECTOR), A, B, (E *)nullptr);
                push();
                ring.popped();
#pragma unroll
                for (int i = 0; i < N2; ++i) {
                    ss = fma(A[i], A[i], ss);
                    ss = fma(B[i], B[i], ss);
                    A[i] = mul(A[i], wA[i]);
                    B[i] = mul(B[i], wB[i]);
                }
                rotate<N2, false>(A, B, cs, sn);
                const float mean = sum_group<LPT>(sum2(ss)) * (1.f / D), r = rsqrtf(mean + EPS);
                if (!(mean <= FLT_MAX) && !l.turned) {
                    // A turn by nothing makes NaN of the channel beside an infinite one: the row's values as
                    // they were (its slot is filled again by the next push).  Behind the sum, so that the
                    // turn still runs beside it (8192 tokens of 20 heads: 14.0 -> 14.4 us; with the branch
                    // around the turn 15.4).
                    open<INTER>(lds16(at), lds16(at + ring.VECTOR), A, B, (E *)nullptr);
#pragma unroll
                    for (int i = 0; i < N2; ++i) {
                        A[i] = mul(A[i], wA[i]);
                        B[i] = mul(B[i], wB[i]);
                    }
                }
                const f2 rr = mk(r, r);
#pragma unroll
                for (int i = 0; i < N2; ++i) {
                    A[i] = mul(A[i], rr);
                    B[i] = mul(B[i], rr);
                }
                uint4 a, b;
                close<INTER>(A, B, a, b, (E *)nullptr);
                if (store) {
                    *reinterpret_cast<uint4 *>(dst + l.ia * VEC) = a;
                    *reinterpret_cast<uint4 *>(dst + l.ib * VEC) = b;
                }
            }
        };
        run((E *)p.qo + n * ((size_t)p.Hq * D), D, 0, min(h0, p.Hq), min(h1, p.Hq));
        E *kdst = CACHE ? nullptr : (E *)p.ko + n * ((size_t)p.Hk * D), *vdst = nullptr;
        if (CACHE) {
            const long long slot = p.slots[n];
            if (slot >= 0 && slot < p.n_slots) {
                const long long pg = slot / p.page, in = slot - pg * p.page;
                kdst = (E *)p.kc + pg * p.kcs.page + in * p.kcs.token;
                vdst = (E *)p.vc + pg * p.vcs.page + in * p.vcs.token;
            }
        }
        run(kdst, CACHE ? p.kcs.head : D, 1, max(h0 - p.Hq, 0), min(h1 - p.Hq, p.Hk));
        if (CACHE) {
            for (int h = max(h0 - p.Hq - p.Hk, 0); h < h1 - p.Hq - p.Hk; ++h) {
                ring.wait();
                const uint4 a = lds16(ring.got), b = lds16(ring.got + ring.VECTOR);
                push();
                ring.popped();
                if (act && vdst) {
                    *reinterpret_cast<uint4 *>(vdst + h * p.vcs.head + l.ia * VEC) = a;
                    *reinterpret_cast<uint4 *>(vdst + h * p.vcs.head + l.ib * VEC) = b;
                }
            }
        }
    }
    let_next();
}

// The rows of TPW tokens side by side are a warp's item: TPW tokens x one head.  The items, head by head and then on to the next tokens, are one list cut
// into runs of `per`, one a warp, which may begin and end inside the heads of its tokens.
template <int TPW> struct Items {
    unsigned tok;    // the first of the current tokens
    int head, heads, todo;
    __device__ __forceinline__ Items(const QkRope &p, int h, long long per) : heads(h) {
        const long long all = (long long)((p.N + TPW - 1) / TPW) * h;
        const long long first = ((long long)blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5)) * per;
        todo = (int)max(0ll, min(per, all - first));
        tok = (unsigned)(first / h) * TPW;
        head = (int)(first % h);
    }
};

__device__ const uint4 no_row[32] = {};  // a row of zeros of the largest type and size

// part (or null): [CTA][2][D], the CTA's sums of the weights' gradients (query, key)
template <typename E, int D, bool INTER>
__global__ void __launch_bounds__(THREADS, 2) k_qkrope_bwd(const QkRope p, long long per) {
    using L = Lay<E, D, INTER>;
    constexpr int VEC = L::VEC, N2 = L::N2, LPT = L::LPT, TPW = L::TPW, WARPS = THREADS / 32;
    extern __shared__ __align__(16) char ring_smem[];
    __shared__ Shared<E, D, INTER> sh;
    __shared__ float red[WARPS][2][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = lane % LPT;
    const L l(j, p.rot);
    Items<TPW> now(p, p.Hq + p.Hk, per);

    if (p.part) let_next();  // k_qkrope_dw: few blocks, wanted at once
    after_previous();
    Ring<4, PF_BWD> ring(ring_smem);
    const unsigned N = (unsigned)p.N;
    auto token = [&](unsigned at) { return (size_t)min(at + lane / LPT, N - 1); };
    Items<TPW> next = now;
    int left = 0, apart = D;
    const E *src = nullptr, *grad = nullptr;
    auto push = [&]() {
        if (next.todo > 0) {
            if (left == 0) {
                const size_t n = token(next.tok);
                const int h = next.head;
                if (h < p.Hq) {
                    src = (const E *)p.q + n * p.qs + h * D;
                    grad = (const E *)p.gq + (n * p.Hq + h) * D;
                    left = p.Hq - h;
                } else {
                    src = (const E *)p.k + n * p.ks + (h - p.Hq) * D;
                    grad = (const E *)p.gk + (n * p.Hk + h - p.Hq) * D;
                    left = next.heads - h;
                }
                if (next.tok + lane / LPT >= N) {  // behind the last token: rows of zeros, which add nothing to dw
                    src = grad = reinterpret_cast<const E *>(no_row);
                    apart = 0;
                }
                next.head += left;
                if (next.head == next.heads) {
                    next.head = 0;
                    next.tok += TPW;
                }
            }
            cp16(ring.put, src + l.ia * VEC);
            cp16(ring.put + ring.VECTOR, src + l.ib * VEC);
            cp16(ring.put + 2 * ring.VECTOR, grad + l.ia * VEC);
            cp16(ring.put + 3 * ring.VECTOR, grad + l.ib * VEC);
            src += apart;
            grad += apart;
            --left;
            --next.todo;
        }
        ring.pushed();
    };
#pragma unroll
    for (int i = 0; i < PF_BWD - 1; ++i) push();
    sh.fill(p);
    f2 dwq[2 * N2] = {}, dwk[2 * N2] = {};  // firsts, then seconds
    while (now.todo > 0) {
        const bool act = now.tok + lane / LPT < N;
        const size_t n = token(now.tok);
        const int h0 = now.head, h1 = min(now.heads, h0 + now.todo);
        f2 cs[N2], sn[N2];
        sh.template angles<false>(p.pos ? p.pos[n] : (int)((unsigned)n % (unsigned)p.T), j, cs, sn);
        auto run = [&](E *dst, int which, f2 *dw, int from, int to) {
            dst += from * D;
#pragma unroll 1
            for (int h = from; h < to; ++h, dst += D) {
                f2 A[N2], B[N2], gA[N2], gB[N2], ss = 0, sg = 0;
                ring.wait();
                open<INTER>(lds16(ring.got + 2 * ring.VECTOR), lds16(ring.got + 3 * ring.VECTOR), gA, gB, (E *)nullptr);
                open<INTER>(lds16(ring.got), lds16(ring.got + ring.VECTOR), A, B, (E *)nullptr);
                push();
                ring.popped();
                if (l.turned) rotate<N2, true>(gA, gB, cs, sn);  // a turn by nothing: see k_qkrope
#pragma unroll
                for (int i = 0; i < N2; ++i) {
                    ss = fma(A[i], A[i], ss);
                    ss = fma(B[i], B[i], ss);
                }
                const float r = rsqrtf(sum_group<LPT>(sum2(ss)) * (1.f / D) + EPS);
                const f2 rr = mk(r, r);
                f2 wA[N2], wB[N2];
                sh.weights(which, j, wA, wB);
#pragma unroll
                for (int i = 0; i < N2; ++i) {  // x to n = x r, dw += g n, g to g w
                    A[i] = mul(A[i], rr);
                    B[i] = mul(B[i], rr);
                    dw[i] = fma(gA[i], A[i], dw[i]);
                    dw[N2 + i] = fma(gB[i], B[i], dw[N2 + i]);
                    gA[i] = mul(gA[i], wA[i]);
                    gB[i] = mul(gB[i], wB[i]);
                    sg = fma(gA[i], A[i], sg);
                    sg = fma(gB[i], B[i], sg);
                }
                const float c = sum_group<LPT>(sum2(sg)) * (-1.f / D);  // - mean(g w n)
                const f2 cc = mk(c, c);
#pragma unroll
                for (int i = 0; i < N2; ++i) {
                    gA[i] = mul(fma(A[i], cc, gA[i]), rr);
                    gB[i] = mul(fma(B[i], cc, gB[i]), rr);
                }
                uint4 a, b;
                close<INTER>(gA, gB, a, b, (E *)nullptr);
                if (act) {
                    *reinterpret_cast<uint4 *>(dst + l.ia * VEC) = a;
                    *reinterpret_cast<uint4 *>(dst + l.ib * VEC) = b;
                }
            }
        };
        run((E *)p.dq + n * p.dqs, 0, dwq, min(h0, p.Hq), min(h1, p.Hq));
        run((E *)p.dk + n * p.dks, 1, dwk, max(h0 - p.Hq, 0), min(h1 - p.Hq, p.Hk));
        now.todo -= h1 - h0;
        now.head = 0;
        now.tok += TPW;
    }
    if (!p.part) return;
    // over the warp's tokens, then over the warps in order
#pragma unroll
    for (int i = 0; i < 2 * N2; ++i) {
        float x[4];
        un(dwq[i], x[0], x[1]);
        un(dwk[i], x[2], x[3]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int o = LPT; o < 32; o <<= 1) x[k] += __shfl_xor_sync(0xffffffffu, x[k], o);
            if (lane < LPT) red[warp][k >> 1][l.channel(i >= N2, 2 * (i % N2) + (k & 1))] = x[k];
        }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < 2 * D; x += THREADS) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) s += (&red[w][0][0])[x];
        p.part[(size_t)blockIdx.x * 2 * D + x] = s;
    }
}

// dwq, dwk = the partials' sums in order: 32 columns a CTA, 32 partials at a time
template <int D> __global__ void __launch_bounds__(1024) k_qkrope_dw(const float *part, int n, float *dwq, float *dwk) {
    __shared__ float red[32][33];
    after_previous();
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5, col = blockIdx.x * 32 + cx;
    float s = 0.f;
    for (int r = ry; r < n; r += 32 * 10) {  // all of a thread's partials at once: at most BWD_CTAS / 32
        float x[10];
#pragma unroll
        for (int k = 0; k < 10; ++k) x[k] = r + 32 * k < n ? part[(size_t)(r + 32 * k) * 2 * D + col] : 0.f;
#pragma unroll
        for (int k = 0; k < 10; ++k) s += x[k];
    }
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
    let_next();
}

template <typename E, int D, bool INTER> static cudaError_t fwd(const QkRope &p, cudaStream_t s) {
    // A warp's tokens with all their heads, and as many CTAs as that gives, which the hardware deals
    // out as others end (8 x 4096 tokens: 30.3 us; one wave of CTAs with equal runs of rows 33.0).
    // Where that leaves the GPU short of 16 warps an SM, the heads are cut.
    const bool cache = p.slots != nullptr;
    constexpr int TPW = Lay<E, D, INTER>::TPW, WARPS = THREADS / 32;
    const long long heads = p.Hq + p.Hk * (cache ? 2 : 1), groups = (long long)((p.N + TPW - 1) / TPW);
    const long long chunks = max(1ll, min(heads, WARPS_WANTED / groups));
    const int hpg = (int)((heads + chunks - 1) / chunks);
    const dim3 grid((unsigned)min((groups + WARPS - 1) / WARPS, 1ll << 20), (unsigned)((heads + hpg - 1) / hpg));
    auto go = [&](auto kern) -> cudaError_t {
        constexpr int smem = Ring<2, PF_FWD>::WARP_BYTES * (THREADS / 32);
        static_assert(smem + sizeof(Shared<E, D, INTER>) <= 48 * 1024, "fits without an opt-in");
        return launch_after(kern, grid, dim3(THREADS), smem, s, p, hpg);
    };
    return cache ? go(k_qkrope<E, D, INTER, true>) : go(k_qkrope<E, D, INTER, false>);
}

template <typename E, int D, bool INTER> static cudaError_t bwd(const QkRope &p, cudaStream_t s) {
    // one wave of CTAs with equal runs: each CTA's sums of the weights' gradients cost it a reduction
    // (8 x 4096 tokens: 45.5 us; a warp for every tokens' heads, 1024 CTAs, 53.5)
    constexpr int TPW = Lay<E, D, INTER>::TPW, WARPS = BWD_CTAS * (THREADS / 32);
    const long long items = (long long)((p.N + TPW - 1) / TPW) * (p.Hq + p.Hk), per = (items + WARPS - 1) / WARPS;
    const int ctas = (int)((items + per * (THREADS / 32) - 1) / (per * (THREADS / 32)));
    constexpr int smem = Ring<4, PF_BWD>::WARP_BYTES * (THREADS / 32);
    cudaError_t e = cudaFuncSetAttribute(k_qkrope_bwd<E, D, INTER>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    QkRope a = p;
    if (!p.dwq && !p.dwk) a.part = nullptr;
    e = launch_after(k_qkrope_bwd<E, D, INTER>, dim3(ctas), dim3(THREADS), smem, s, a, per);
    if (e != cudaSuccess || !a.part) return e;
    return launch_after(k_qkrope_dw<D>, dim3(2 * D / 32), dim3(1024), 0, s, (const float *)a.part, ctas, p.dwq, p.dwk);
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
