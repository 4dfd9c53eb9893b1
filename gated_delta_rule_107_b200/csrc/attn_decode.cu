// attn_decode.cu -- softmax attention of one new token per request over a paged key-value cache.
//
// For request r with n = lens[r] cached tokens (the new one among them) and query head h of the
// group that shares key head h / (Hq / Hk), over the tokens t in [max(0, n - window), n):
//   s_t = scale q . k_t,  o = sum_t e^{s_t} v_t / sum_t e^{s_t},  lse = log sum_t e^{s_t}
// formed in one pass over the cache with the running maximum m and sum l of each head (in base 2:
// s_t log2 e), fp32 throughout.
//
// What bounds it is reading the cache once: a key head's rows serve the G = Hq / Hk heads of its
// group, 2 G flops a byte in bf16, far below what the tensor cores need to be busy; so the design
// is about bytes in flight (128 KB an SM) and an even split.  In calls replayed in a graph three requests
// of 200001 tokens (1.23 GB) are read at 6.6 TB/s, the rate of a plain copy, 64 ragged ones of up to 16384
// (540 MB) at 5.9; behind other kernels on a stream at 6.4 and 5.7.  Small calls are the chain of launch,
// lengths, table, rows, join: 7.8 us for one request of 2000 tokens.
//   Work.  The piece is a tile of tokens of one (request, key head[, block of its query heads]): as
//     many as make 4 KB of keys and 4 KB of values (8, 16 or 32).  The tiles of all requests form one
//     list, cut into equal contiguous runs, one per CTA, however ragged the lengths: a run may hold
//     parts of several (request, head) segments.  A segment's start and join cost a CTA about as long
//     as COST tiles, so each counts that much more in the list (units; the tiles come behind them).  A
//     segment inside one CTA's run is finished there; one that crosses runs leaves fp32 partials
//     (m, l, o) in the workspace, at most two a CTA, which k_attn_join adds in the order of the runs
//     (no atomics: results do not change from run to run).
//   Loads.  Each warp takes every fourth tile of its CTA's run through a pipeline of its own in
//     shared memory, 16-byte asynchronous copies, rows swizzled by 16-byte chunk; the pipeline
//     runs on across segments, and warps meet only at a segment's end.  (With a contiguous run for
//     every warp, none of which waits for another, long contexts were 3 to 5 % slower, their warps
//     reading four places of the cache at once, and only batches of more than a thousand contexts of
//     a tile or two faster.)
//   bf16.  The tile's tokens, 16 at a time, are the rows of mma.m16n8k16, the group's query heads its
//     columns: S^T = K Q^T, then o^T = V^T P^T with P^T transposed in registers.  A group of up to
//     8 heads is one n8 column block, of 16 two (larger groups are taken 16 heads at a time, and
//     their rows read again for each block), so no row is spent on padding to 16 heads, and tcgen05's
//     smallest tile (64 or 128 rows through tensor memory) would be mostly padding.  P enters with
//     all of its 24 bits, as three bf16 numbers of 8 bits each that are multiplied one after another
//     (with two, 2^-17 of p, outputs that are small against the values were off by more than fp32 sums
//     are), and a tile's products are summed from zero and then added to o in fp32: the tensor cores
//     cut what they add to a sum, and cutting the running sum a thousand times lost 2^-16 of it.  The
//     additional products hide behind the loads as long as several are in flight (three requests of
//     200001 tokens: 187.3 us in a graph, 192 on a stream; with two products into the running sum 186.5
//     and 188; with a kernel of 168 registers, and so fewer in flight, 194 and 201), less so in wide
//     groups.  For 400 MB groups of up to 8 heads reach 87 % of the copy's rate (64 channels 77 %), of 16
//     73 % (65 %; with two products 78 and 69 %), of 32 38 % (34 %).
//   fp32.  CUDA cores, 1, 2, 4 or up to 8 heads at a time, packed arithmetic: a lane holds 4 channels
//     of the heads' queries and outputs.  For 400 MB groups of up to 4 are bound by the loads (86 to 92 %
//     of the copy's rate), of 8 by two warps a scheduler working through their tiles (61 to 69 %).
// Tokens that are masked (or whose table entry is no page) are neither read nor seen: their rows
// in shared memory are zero-filled, their scores -inf.  A request with none gives o = 0, lse = -inf.
#include <math_constants.h>

#include "attn_decode.cuh"
#include "prepost.cuh"

namespace dr {
namespace ad {

using namespace dr::f32x2;

constexpr int WARPS = 4, THREADS = WARPS * 32;
constexpr int MAX_CTAS = 296;     // two a SM
constexpr int MIN_UNITS = WARPS;  // a CTA's run is at least one tile a warp
constexpr int COST = 6;           // of a segment, in tiles (64 requests of up to 500 tokens, 8 key heads: 21.6 us; with 4 24.3, with 2 29.3)
constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.69314718055994530942f;

struct Args {
    AttnDecode a;
    int G, GB, RB;       // query heads of a group; heads of a block; blocks of a group
    float *part;         // [2 * MAX_CTAS][GB][D]: o, not divided by l
    float2 *ml;          // [2 * MAX_CTAS][GB]: m, l
    int4 *head;          // [MAX_CTAS]: the split segment that begins in a CTA: request, key head, block, last CTA
    float scale2;
    FastDiv by_page;
    double inv_ctas;     // 1 / CTAs
    bool whole;          // a tile never crosses a page (the page is a multiple of the tile)
    bool alike;          // both caches have the same strides: one offset serves both
};

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
// 16 bytes, or 16 zero bytes (nothing is read then)
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void ldsm4(uint32_t *r, uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t *r, uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t trans8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^x for a weight or for a factor of what was summed before, not below the smallest normal number: an
// infinite value that is seen makes its channel infinite, and a weight of zero would make 0 inf = NaN of
// it.  Sums of finite values notice 2^-126 no more than they notice zero.  NaN stays.
__device__ __forceinline__ float weight(float x) {
    float y;
    asm("max.NaN.f32 %0, %1, 0f00800000;" : "=f"(y) : "f"(ex2(x)));
    return y;
}
// what is subtracted from scores: -inf minus -inf (nothing seen yet) would be NaN
__device__ __forceinline__ float base_of(float m) { return m == -CUDART_INF_F ? 0.f : m; }
// the sum of the weights: 0 where no score was above -inf (every weight is 2^-126 then); a NaN stays
__device__ __forceinline__ float sum_of(float m, float l) { return m == -CUDART_INF_F && l == l ? 0.f : l; }

// log of the sum l (base 2 maximum m); nothing seen: -inf; a NaN stays
__device__ __forceinline__ float lse_of(float m, float l) { return l > 0.f ? (m + log2f(l)) * LN2 : (l == l ? -CUDART_INF_F : l); }

// The visible tokens of request r and its tiles.
struct Span {
    int first, n, tile0, tiles;
    template <int TILE> __device__ __forceinline__ void set(const AttnDecode &a, int r) {
        const long long room = (long long)a.width * a.page;
        n = max(a.lens[r], 0);
        first = a.window > 0 && n > a.window ? n - a.window : 0;  // counts back from the length, which may lie behind the table
        if (n > room) n = (int)room;
        tile0 = first / TILE;
        tiles = n > first ? (n - 1) / TILE - tile0 + 1 : 0;
    }
};

// A place in the list: request r, segment (key head, block of query heads) of it, tile; `unit` is the
// tile's place in the list from the beginning of the CTA's run.
struct Place {
    int r, seg, tile, unit;
    Span sp;
};
__device__ __forceinline__ long long units_of(const Span &sp) { return sp.tiles > 0 ? sp.tiles + COST : 0; }

// The CTA's run [u0, u0 + len) of the list's units, `per` units for every run but the last; the
// request r0 in which it begins, whose first unit is `base`.
struct Run {
    long long u0, base;
    int len, per, r0;
};

// total / CTAs, rounded up (a 64-bit division takes a third of a microsecond): the product is off by
// less than one
__device__ __forceinline__ int per_cta(long long total, double inv_ctas) {
    const long long n = gridDim.x;
    long long q = (long long)((double)total * inv_ctas);
    q -= q * n >= total && q > 0;
    while (q * n < total) ++q;
    return (int)q;
}
// in / units for a small quotient
__device__ __forceinline__ int small_quotient(long long in, long long units) {
    int q = (int)__fdividef((float)in, (float)units);
    while ((long long)(q + 1) * units <= in) ++q;
    while ((long long)q * units > in) --q;
    return q;
}

// All threads of the CTA; every CTA finds its run from the lengths alone.
template <int TILE> __device__ __forceinline__ Run find_run(const Args &x, int segs) {
    __shared__ long long wsum[WARPS], found[2];
    const AttnDecode &a = x.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int each = (a.R + THREADS - 1) / THREADS, b0 = min(a.R, tid * each), b1 = min(a.R, b0 + each);
    long long mine = 0;
    Span sp;
    for (int r = b0; r < b1; ++r) {
        sp.template set<TILE>(a, r);
        mine += units_of(sp) * segs;
    }
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    long long before = inc - mine, total = 0;
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += wsum[w];
        total += wsum[w];
    }
    Run run;
    run.per = max(MIN_UNITS, per_cta(total, x.inv_ctas));
    run.u0 = min(total, (long long)run.per * blockIdx.x);
    run.len = (int)min(total - run.u0, (long long)run.per);
    if (run.len > 0 && before <= run.u0 && run.u0 < before + mine) {
        int r = b0;
        for (; r < b1; ++r) {
            sp.template set<TILE>(a, r);
            const long long w = units_of(sp) * segs;
            if (run.u0 < before + w) break;
            before += w;
        }
        found[0] = r;
        found[1] = before;
    }
    __syncthreads();
    run.r0 = run.len > 0 ? (int)found[0] : 0;
    run.base = run.len > 0 ? found[1] : 0;
    return run;
}

constexpr int NOWHERE = 0x7fffffff;  // the unit of a place behind the list

// moves `by` tiles on
template <int TILE> __device__ __forceinline__ void advance(Place &pl, int by, int segs, const AttnDecode &a) {
    pl.tile += by;
    pl.unit += by;
    while (pl.tile >= pl.sp.tiles) {
        pl.tile -= pl.sp.tiles;
        pl.unit += COST;
        if (++pl.seg == segs) {
            pl.seg = 0;
            do {
                if (++pl.r >= a.R) {
                    pl.unit = NOWHERE;
                    return;
                }
                pl.sp.template set<TILE>(a, pl.r);
            } while (pl.sp.tiles == 0);
        }
    }
}

// One warp's pipeline of tiles.  A stage is the K rows, then the V rows, of a tile.
template <typename E, int D, int TILE_, int STAGES> struct Pipe {
    static constexpr int TILE = TILE_;
    static constexpr int ROW = D * (int)sizeof(E), CPR = ROW / 16, E16 = 16 / (int)sizeof(E);  // bytes, 16-byte chunks of a row
    static constexpr int HALF = TILE * ROW, STAGE = 2 * HALF;
    static constexpr int RPI = 32 / (CPR < 32 ? CPR : 32);          // rows a warp copies with one instruction
    static_assert(CPR <= 32, "a row is at most one instruction");

    // 16-byte chunk c of row r: the chunk index is exclusive-ored with the row's low bits, so that
    // eight rows at one chunk lie in eight different banks groups
    static __device__ __forceinline__ uint32_t at(int r, int c) { return r * ROW + ((c ^ (r & 7)) << 4); }

    // What a tile's copies need: the lane's token (lane % TILE) is row `in` of page pg (-1: not seen;
    // read ahead of the copies, since the table is a read of its own), key head h.
    struct Want {
        int pg, in, h;
    };
    static __device__ __forceinline__ Want want(const Args &x, const Place &pl) {
        const AttnDecode &a = x.a;
        const int t = (pl.sp.tile0 + pl.tile) * TILE + (threadIdx.x & (TILE - 1));
        Want w = {-1, 0, pl.seg / x.RB};
        if (t >= pl.sp.first && t < pl.sp.n) {
            const int col = x.by_page.div(t);
            const int *at = a.table + (size_t)pl.r * a.width + col;
            w.in = t - col * a.page;
            w.pg = *at;
            // the entries that this CTA reads some tiles on
            if ((threadIdx.x & (TILE - 1)) == 0 && col + AHEAD < a.width) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + AHEAD));
        }
        return w;
    }
    static constexpr int AHEAD = 128;
    static constexpr uint32_t ALL = 0xffffffffu >> (32 - TILE);  // every token of a tile

    // copies the tile into the stage; returns the bits of its live tokens
    static __device__ __forceinline__ uint32_t load(uint32_t stage, const Args &x, const Want &w) {
        const AttnDecode &a = x.a;
        const int lane = threadIdx.x & 31;
        const bool seen = w.pg >= 0 && w.pg < a.n_pages;
        const uint32_t live = __ballot_sync(0xffffffffu, seen) & ALL;
        const int c = lane % CPR, row0 = lane / CPR, e16 = E16;
        auto offset = [&](const CacheStrides &st) { return (size_t)w.pg * st.page + (size_t)w.in * st.token + (size_t)w.h * st.head; };
        const size_t ko = seen ? offset(a.ks) : 0;
        if (x.whole && live == ALL) {  // rows of one page: evenly spaced from the first one's
            const size_t kt = a.ks.token, vt = a.vs.token, vo = x.alike ? ko : offset(a.vs);
            const E *k = (const E *)a.kc + __shfl_sync(0xffffffffu, ko, 0) + row0 * kt + c * e16;
            const E *v = (const E *)a.vc + __shfl_sync(0xffffffffu, vo, 0) + row0 * vt + c * e16;
#pragma unroll
            for (int i = 0; i < TILE; i += RPI) {
                cp16(stage + at(i + row0, c), k + i * kt, true);
                cp16(stage + HALF + at(i + row0, c), v + i * vt, true);
            }
            return live;
        }
        const size_t vo = seen && !x.alike ? offset(a.vs) : 0;
#pragma unroll
        for (int i = 0; i < TILE; i += RPI) {
            const int row = i + row0;
            const size_t k = __shfl_sync(0xffffffffu, ko, row), v = x.alike ? k : __shfl_sync(0xffffffffu, vo, row);
            const bool ok = live >> row & 1;
            cp16(stage + at(row, c), (const E *)a.kc + k + c * e16, ok);
            cp16(stage + HALF + at(row, c), (const E *)a.vc + v + c * e16, ok);
        }
        return live;
    }
};

// ------------------------------------------------------------------ one warp's arithmetic
// Each keeps, for the heads of a block, m (base 2), l and o, and offers
//   fetch(q row of the block's first head, heads): reads the queries; begin(): they are the ones from now
//   tile(stage, live)
//   finish(m, l, o): l summed over lanes, all three to shared memory, o as [head][slot_of(head, channel)];
//     l = 0 and o = 0 where no score was above -inf, whatever the values hold

// where a head's channel lies in a row of o in shared memory: blocks of 8 channels exchanged so that
// the matrix fragments (8 channels of four pairs of heads at once) fall into different banks
__device__ __forceinline__ int slot_of(int head, int ch) { return ch ^ ((head >> 1 & 3) << 3); }

template <int D, int NT> struct Mma {  // bf16: blocks of 8 NT heads
    typedef __nv_bfloat16 E;
    static constexpr int GB = 8 * NT, STAGES = 3, CTAS = MAX_CTAS, SUB = 128 / D;  // 16 SUB tokens a tile
    static constexpr int NPART = 3;  // bf16 numbers that make up a weight: 8 bits each of its 24
    static constexpr int KB = 4;     // blocks of 16 channels whose products are in flight at once
    static_assert(D / 16 % KB == 0, "whole blocks");
    typedef Pipe<E, D, 16 * SUB, STAGES> P;
    uint32_t q[D / 16][NT][2], qn[D / 16][NT][2];
    f2 o[D / 16][NT][2];  // heads 2 t and 2 t + 1 of channel g, of channel g + 8
    float m[NT][2], l[NT][2];

    __device__ __forceinline__ void fetch(const E *src, int heads) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const bool in = j * 8 + g < heads;
                const E *s = src + (in ? j * 8 + g : 0) * D + k * 16 + 2 * t;
                qn[k][j][0] = in ? *reinterpret_cast<const uint32_t *>(s) : 0u;
                qn[k][j][1] = in ? *reinterpret_cast<const uint32_t *>(s + 8) : 0u;
            }
    }
    __device__ __forceinline__ void begin() {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            m[j][0] = m[j][1] = -CUDART_INF_F;
            l[j][0] = l[j][1] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                q[k][j][0] = qn[k][j][0];
                q[k][j][1] = qn[k][j][1];
                o[k][j][0] = o[k][j][1] = 0;
            }
        }
    }
    __device__ __forceinline__ void tile(uint32_t stage, uint32_t live, float scale2, void *) {
        const int lane = threadIdx.x & 31, g = lane >> 2;
        // scores of token g (0, 1) and g + 8 (2, 3) of 16, heads 2 t and 2 t + 1 of each block of 8; two
        // accumulators, so that half as many products wait on one another
        float s[SUB][NT][4];
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
            float s1[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[u][j][i] = s1[j][i] = 0.f;
#pragma unroll
            for (int k = 0; k < D / 16; k += 2) {
                uint32_t a[4], b[4];
                ldsm4(a, stage + P::at(u * 16 + (lane & 15), k * 2 + (lane >> 4)));
                ldsm4(b, stage + P::at(u * 16 + (lane & 15), k * 2 + 2 + (lane >> 4)));
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    mma(s[u][j], a, q[k][j][0], q[k][j][1]);
                    mma(s1[j], b, q[k + 1][j][0], q[k + 1][j][1]);
                }
            }
            const bool lo = live >> (u * 16 + g) & 1, hi = live >> (u * 16 + g + 8) & 1;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    s[u][j][i] = lo ? (s[u][j][i] + s1[j][i]) * scale2 : -CUDART_INF_F;
                    s[u][j][i + 2] = hi ? (s[u][j][i + 2] + s1[j][i + 2]) * scale2 : -CUDART_INF_F;
                }
        }
        float mx[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mx[j][i] = fmaxf(s[0][j][i], s[0][j][i + 2]);
#pragma unroll
                for (int u = 1; u < SUB; ++u) mx[j][i] = fmaxf(mx[j][i], fmaxf(s[u][j][i], s[u][j][i + 2]));
            }
#pragma unroll
        for (int d = 4; d < 32; d <<= 1)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                mx[j][0] = fmaxf(mx[j][0], __shfl_xor_sync(0xffffffffu, mx[j][0], d));
                mx[j][1] = fmaxf(mx[j][1], __shfl_xor_sync(0xffffffffu, mx[j][1], d));
            }
        f2 f[NT];
        float from[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            float fj[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float mn = fmaxf(m[j][i], mx[j][i]);
                from[j][i] = base_of(mn);
                fj[i] = weight(m[j][i] - from[j][i]);
                m[j][i] = mn;
                l[j][i] *= fj[i];
            }
            f[j] = mk(fj[0], fj[1]);
        }
        const int row = (lane & 7) + ((lane >> 4) << 3), c0 = lane >> 3 & 1;
        uint32_t part[SUB][NPART][NT][2];
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    p[i] = weight(s[u][j][i] - from[j][i & 1]);
                    l[j][i & 1] += p[i];
                }
                // Each part but the last is the largest bf16 number below what is left, so that no part of
                // a weight is zero or negative and an infinite value never meets one; the parts of weights
                // below 2^-102 may have to be lifted to the smallest bf16 number, 2^-133.
#pragma unroll
                for (int x = 0; x < NPART; ++x) {
                    int w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int b = __float_as_int(p[i]);
                        w[i] = x == 0 ? b - 1 : (x < NPART - 1 ? __viaddmax_s32(b, -1, 0x10000) : max(b, 0x10000));
                        p[i] -= __int_as_float(w[i] & 0xFFFF0000);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) part[u][x][j][i] = trans8(__byte_perm(w[2 * i], w[2 * i + 1], 0x7632));
                }
            }
        // A product's sum is cut, not rounded, where it is added to what was there, so the tile's sum
        // starts from zero, its small parts first, and is added to o in fp32.
        const uint32_t v = stage + P::HALF;
#pragma unroll
        for (int k0 = 0; k0 < D / 16; k0 += KB) {
            uint32_t a[KB][SUB][4];
            float c[KB][NT][4] = {};
#pragma unroll
            for (int k = 0; k < KB; ++k)
#pragma unroll
                for (int u = 0; u < SUB; ++u) ldsm4t(a[k][u], v + P::at(u * 16 + row, 2 * (k0 + k) + c0));
#pragma unroll
            for (int x = NPART - 1; x >= 0; --x)
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int k = 0; k < KB; ++k)
#pragma unroll
                        for (int j = 0; j < NT; ++j) mma(c[k][j], a[k][u], part[u][x][j][0], part[u][x][j][1]);
#pragma unroll
            for (int k = 0; k < KB; ++k)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    o[k0 + k][j][0] = fma(o[k0 + k][j][0], f[j], mk(c[k][j][0], c[k][j][1]));
                    o[k0 + k][j][1] = fma(o[k0 + k][j][1], f[j], mk(c[k][j][2], c[k][j][3]));
                }
        }
    }
    __device__ __forceinline__ void finish(float *sm, float *sl, float *so) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[j][i] += __shfl_xor_sync(0xffffffffu, l[j][i], d);
                const int head = j * 8 + 2 * t + i;
                const float sum = sum_of(m[j][i], l[j][i]);
                if (g == 0) {
                    sm[head] = m[j][i];
                    sl[head] = sum;
                }
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float x[2];
                        un(o[k][j][c], x[0], x[1]);
                        so[head * D + slot_of(head, k * 16 + 8 * c + g)] = sum == 0.f ? 0.f : x[i];
                    }
            }
    }
    static constexpr int EXTRA = 0;  // bytes of shared memory of the warp's own
};

// The N values of 2 MASK neighbouring lanes added up, each lane keeping max(1, N / (2 MASK)) of the sums
// in v[0], v[1], ...: its highest bit names the half, the next one the half of that, and so on; once a
// single sum is left, the lanes of the remaining bits all keep it.
template <int N, int MASK> __device__ __forceinline__ void scatter_sums(float *v) {
    if constexpr (MASK > 0) {
        constexpr int HALF = N > 1 ? N / 2 : 1;
#pragma unroll
        for (int i = 0; i < HALF; ++i) {
            if constexpr (N > 1) {
                const bool up = threadIdx.x & MASK;
                const float send = up ? v[i] : v[i + HALF], keep = up ? v[i + HALF] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, MASK);
            } else {
                v[i] += __shfl_xor_sync(0xffffffffu, v[i], MASK);
            }
        }
        scatter_sums<HALF, MASK / 2>(v);
    }
}

// fp32: blocks of H heads, at most 8.  A lane holds 4 channels of the block's queries in registers and
// forms its part of the scores of 8 rows (its half-warp's rows where a row has 16 chunks); the parts
// are added so that each lane ends with the scores of one token and C heads.  (With the queries in
// shared memory, every lane of a token reading all of them, blocks of 8 heads were bound by shared
// memory: 113 us instead of 89 for 32 requests of 1525 tokens, 64 / 8 heads of 128 channels.)
template <int D, int H> struct Simt {
    typedef float E;
    static constexpr int GB = H, STAGES = 3, CTAS = MAX_CTAS, TILE = 1024 / D;
    typedef Pipe<E, D, TILE, STAGES> P;
    static constexpr int LR = D / 4, TP = 32 / LR;         // lanes of a row, rows side by side
    static constexpr int LT = LR / 8;                      // lanes of a token, once the scores are added
    static constexpr int HG = H < LT ? H : LT, C = H / HG;  // groups of heads, heads of a lane
    f2 o[GB][2], q[GB][2], qn[GB][2];
    float m[C], l[C];
    // the tile's p and the heads' factors, each twice (one packed operand); the next warp's stages behind
    // it stay aligned
    static constexpr int EXTRA = ((TILE + 1) * GB * 8 + 127) / 128 * 128;
    f2 *ps;

    // the lane's token of a tile, its first head, and whether it is the first of lanes with the same
    static __device__ __forceinline__ int token() { return (threadIdx.x % LR / LT) * TP + (threadIdx.x & 31) / LR; }
    static __device__ __forceinline__ int head() { return threadIdx.x % LT / (LT / HG) * C; }
    static __device__ __forceinline__ bool first() { return threadIdx.x % LT % (LT / HG) == 0; }

    __device__ __forceinline__ void fetch(const E *src, int heads) {
        const int c = threadIdx.x % LR;
#pragma unroll
        for (int h = 0; h < GB; ++h) {
            const float4 x = h < heads ? *reinterpret_cast<const float4 *>(src + h * D + 4 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
            qn[h][0] = mk(x.x, x.y);
            qn[h][1] = mk(x.z, x.w);
        }
    }
    __device__ __forceinline__ void begin() {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            m[c] = -CUDART_INF_F;
            l[c] = 0.f;
        }
#pragma unroll
        for (int h = 0; h < GB; ++h) {
            q[h][0] = qn[h][0];
            q[h][1] = qn[h][1];
#pragma unroll
            for (int c = 0; c < 2; ++c) o[h][c] = 0;
        }
    }
    __device__ __forceinline__ void tile(uint32_t, uint32_t live, float scale2, const char *base) {
        const int lane = threadIdx.x & 31;
        float s[8 * GB];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 k = *reinterpret_cast<const float4 *>(base + P::at(i * TP + lane / LR, lane % LR));
            const f2 k0 = mk(k.x, k.y), k1 = mk(k.z, k.w);
#pragma unroll
            for (int h = 0; h < GB; ++h) s[i * GB + h] = sum2(fma(k1, q[h][1], mul(k0, q[h][0])));
        }
        scatter_sums<8 * GB, LR / 2>(s);
        const int t = token(), h0 = head();
        const bool ok = live >> t & 1;
        float mx[C];
#pragma unroll
        for (int c = 0; c < C; ++c) mx[c] = s[c] = ok ? s[c] * scale2 : -CUDART_INF_F;
#pragma unroll
        for (int d = LT; d < 32; d <<= 1)
#pragma unroll
            for (int c = 0; c < C; ++c) mx[c] = fmaxf(mx[c], __shfl_xor_sync(0xffffffffu, mx[c], d));
        bool up = false;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const float mn = fmaxf(m[c], mx[c]);
            const float f = weight(m[c] - base_of(mn)), p = weight(s[c] - base_of(mn));
            up = up || m[c] != mn;
            m[c] = mn;
            l[c] = l[c] * f + p;
            if (first()) {
                ps[t * GB + h0 + c] = mk(p, p);
                if (t == 0) ps[TILE * GB + h0 + c] = mk(f, f);
            }
        }
        up = __any_sync(0xffffffffu, up);
        __syncwarp();
        if (up) {
#pragma unroll
            for (int h = 0; h < GB; ++h)
#pragma unroll
                for (int c = 0; c < 2; ++c) o[h][c] = mul(o[h][c], ps[TILE * GB + h]);
        }
        const char *v = base + P::HALF;
#pragma unroll 4
        for (int i = 0; i < 8; ++i) {
            const int u = i * TP + lane / LR;
            const float4 y = *reinterpret_cast<const float4 *>(v + P::at(u, lane % LR));
            const f2 x0 = mk(y.x, y.y), x1 = mk(y.z, y.w);
            if constexpr (GB == 1) {
                o[0][0] = fma(ps[u], x0, o[0][0]);
                o[0][1] = fma(ps[u], x1, o[0][1]);
            } else {
#pragma unroll
                for (int h = 0; h < GB; h += 2) {
                    const ulonglong2 p = *reinterpret_cast<const ulonglong2 *>(ps + u * GB + h);
                    o[h][0] = fma(p.x, x0, o[h][0]);
                    o[h][1] = fma(p.x, x1, o[h][1]);
                    o[h + 1][0] = fma(p.y, x0, o[h + 1][0]);
                    o[h + 1][1] = fma(p.y, x1, o[h + 1][1]);
                }
            }
        }
        __syncwarp();  // ps is free for the next tile
    }
    __device__ __forceinline__ void finish(float *sm, float *sl, float *so) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int d = LT; d < 32; d <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], d);
            l[c] = sum_of(m[c], l[c]);
            if (first() && token() == 0) {
                sm[head() + c] = m[c];
                sl[head() + c] = l[c];
            }
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < GB; ++h) {
            float x[4];
            un(o[h][0], x[0], x[1]);
            un(o[h][1], x[2], x[3]);
#pragma unroll
            for (int d = LR; d < 32; d <<= 1)  // the rows side by side
#pragma unroll
                for (int c = 0; c < 4; ++c) x[c] += __shfl_xor_sync(0xffffffffu, x[c], d);
            if (lane < LR)
                *reinterpret_cast<float4 *>(so + h * D + slot_of(h, 4 * lane)) =
                    sl[h] == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(x[0], x[1], x[2], x[3]);
        }
    }
};

template <class C, int D> constexpr int warp_bytes() { return C::STAGES * C::P::STAGE + C::EXTRA; }
template <class C, int D> constexpr int smem_bytes() { return WARPS * warp_bytes<C, D>(); }

template <class C, int D> __global__ void __launch_bounds__(THREADS, MAX_CTAS / 148) k_attn(const Args x) {
    typedef typename C::E E;
    typedef typename C::P P;
    constexpr int GB = C::GB, STAGES = C::STAGES, TILE = P::TILE;
    extern __shared__ __align__(128) char smem[];
    __shared__ float sm_m[WARPS][GB], sm_l[WARPS][GB];
    __shared__ int sm_at[WARPS];
    static_assert(GB * D * 4 <= P::STAGE, "a warp's o fits a stage");
    static_assert(warp_bytes<C, D>() % 128 == 0, "every warp's stages are aligned");
    const AttnDecode &a = x.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int segs = a.Hk * x.RB;
    let_next();  // k_attn_join: small blocks, wanted at once
    after_previous();
    const Run run = find_run<TILE>(x, segs);
    for (int r = blockIdx.x; r < a.R; r += gridDim.x) {  // requests that see nothing
        Span sp = {};
        sp.template set<TILE>(a, r);
        if (sp.tiles > 0) continue;
        for (int i = tid; i < a.Hq * D; i += THREADS) ((E *)a.out)[(size_t)r * a.Hq * D + i] = from_f<E>(0.f);
        if (a.lse)
            for (int i = tid; i < a.Hq; i += THREADS) a.lse[(size_t)r * a.Hq + i] = -CUDART_INF_F;
    }
    // the place of the run's first tile
    Place here;
    here.unit = NOWHERE;
    if (run.len > 0) {
        here.r = run.r0;
        here.sp.template set<TILE>(a, here.r);
        const long long in = run.u0 - run.base;  // not negative, inside request r0
        here.seg = small_quotient(in, units_of(here.sp));
        const int off = (int)(in - here.seg * units_of(here.sp)) - COST;
        here.tile = max(off, 0);
        here.unit = max(-off, 0);
    }
    if (here.unit >= run.len) {  // no tile in the run
        if (tid == 0) x.head[blockIdx.x] = make_int4(-1, 0, 0, 0);
        return;
    }

    char *mine = smem + warp * warp_bytes<C, D>();
    const uint32_t stages = smem_u32(mine);
    // the warp's loads run STAGES - 1 tiles ahead of its arithmetic, the table's entries one more;
    // warp w takes the run's tiles w, w + WARPS, ...
    __shared__ uint32_t lives[WARPS][STAGES];
    Place next = here;
    typename P::Want ahead[STAGES] = {};
    bool there[STAGES];
#pragma unroll
    for (int i = 0; i < STAGES; ++i) {
        if (next.unit < run.len) advance<TILE>(next, i == 0 ? warp : WARPS, segs, a);
        there[i] = next.unit < run.len;
        if (there[i]) ahead[i] = P::want(x, next);
    }
    int put = 0, got = 0;
    auto issue = [&](const typename P::Want &w, bool is) {
        if (is) {
            const uint32_t bits = P::load(stages + put * P::STAGE, x, w);
            if (lane == 0) lives[warp][put] = bits;
        }
        cp_commit();
        put = put + 1 == STAGES ? 0 : put + 1;
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) issue(ahead[i], there[i]);
    typename P::Want coming = ahead[STAGES - 1];
    bool comes = there[STAGES - 1];

    C c;
    if constexpr (C::EXTRA > 0) c.ps = reinterpret_cast<f2 *>(mine + STAGES * P::STAGE);
    int done = 0, mytile = warp;  // the run's tiles before the current segment; the warp's next one
    auto fetch = [&](const Place &pl) {
        const int h = pl.seg / x.RB, rb = pl.seg - h * x.RB;
        c.fetch((const E *)a.q + ((size_t)pl.r * a.Hq + h * x.G + rb * GB) * D, min(GB, x.G - rb * GB));
    };
    fetch(here);
    for (int part = 0; here.unit < run.len; ++part) {
        const int h = here.seg / x.RB, rb = here.seg - h * x.RB, head0 = h * x.G + rb * GB;
        const int heads = min(GB, x.G - rb * GB);
        const int rest = here.sp.tiles - here.tile, now = min(rest, run.len - here.unit), upto = done + now;
        const bool whole = here.tile == 0 && now == rest;
        c.begin();
        for (; mytile < upto; mytile += WARPS) {
            cp_wait<STAGES - 2>();
            __syncwarp();
            const uint32_t bits = lives[warp][got];
            issue(coming, comes);
            if (comes) advance<TILE>(next, WARPS, segs, a);
            comes = next.unit < run.len;
            if (comes) coming = P::want(x, next);
            c.tile(stages + got * P::STAGE, bits, x.scale2, mine + got * P::STAGE);
            got = got + 1 == STAGES ? 0 : got + 1;
            __syncwarp();
        }
        // the queries of the segment behind this one, while the warps join
        Place then = here;
        advance<TILE>(then, rest, segs, a);
        if (then.unit < run.len) fetch(then);
        // each warp's o goes to the stage that it will fill next, and which holds nothing now
        c.finish(sm_m[warp], sm_l[warp], reinterpret_cast<float *>(mine + put * P::STAGE));
        if (lane == 0) sm_at[warp] = warp * warp_bytes<C, D>() + put * P::STAGE;
        __syncthreads();  // all warps are done with the segment
        const size_t slot = 2 * blockIdx.x + (part > 0);
        for (int i = tid; i < heads * (D / 8); i += THREADS) {
            const int hd = i / (D / 8), ch = (i - hd * (D / 8)) * 8;
            float mx = sm_m[0][hd], s = 0.f, o[8] = {};
#pragma unroll
            for (int w = 1; w < WARPS; ++w) mx = fmaxf(mx, sm_m[w][hd]);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                const float l = sm_l[w][hd], f = l == 0.f ? 0.f : weight(sm_m[w][hd] - mx);  // l = 0: m may be -inf
                s += l * f;
                const float4 *p = reinterpret_cast<const float4 *>(smem + sm_at[w]) + (hd * D + slot_of(hd, ch)) / 4;
                const float4 u = p[0], v = p[1];
                o[0] += u.x * f; o[1] += u.y * f; o[2] += u.z * f; o[3] += u.w * f;
                o[4] += v.x * f; o[5] += v.y * f; o[6] += v.z * f; o[7] += v.w * f;
            }
            if (whole) {
                const float inv = s > 0.f ? 1.f / s : (s == s ? 0.f : s);
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] *= inv;
                E *dst = (E *)a.out + ((size_t)here.r * a.Hq + head0 + hd) * D + ch;
#pragma unroll
                for (int k = 0; k < 8; k += P::E16) pp::Vec<E, P::E16>::st(dst + k, o + k);
                if (a.lse && ch == 0) a.lse[(size_t)here.r * a.Hq + head0 + hd] = lse_of(mx, s);
            } else {
                float4 *dst = reinterpret_cast<float4 *>(x.part + (slot * GB + hd) * D + ch);
                dst[0] = make_float4(o[0], o[1], o[2], o[3]);
                dst[1] = make_float4(o[4], o[5], o[6], o[7]);
                if (ch == 0) x.ml[slot * GB + hd] = make_float2(mx, s);
            }
        }
        if (tid == 0 && then.unit >= run.len) {  // the run's last segment
            int last = -1;
            if (here.tile == 0 && !whole) last = (int)((run.u0 + here.unit + rest - 1) / run.per);  // its last tile's run
            x.head[blockIdx.x] = last < 0 ? make_int4(-1, 0, 0, 0) : make_int4(here.r, h, rb | (part > 0) << 16, last);
        }
        __syncthreads();  // the stages and the statistics are read
        done = upto;
        here = then;
    }
}

// The split segment that begins in run blockIdx.x: its head blockIdx.y, or (gridDim.y = 1) all of its
// heads, their parts added in order, four parts' reads at a time.  A block's warps share a head's
// parts; where a block has all heads and the parts are few, each warp takes heads of its own.
template <typename E, int D> __global__ void __launch_bounds__(256) k_attn_join(const Args x) {
    constexpr int NC = D / 32, JW = 8, FEW = 8;
    __shared__ float red[JW][D], wm[JW], wl[JW];
    after_previous();
    const int4 hd = x.head[blockIdx.x];
    if (hd.x < 0) return;
    const int rb = hd.z & 0xffff, slot0 = hd.z >> 16, GB = x.GB, heads = min(GB, x.G - rb * GB);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = hd.w - (int)blockIdx.x + 1;
    const size_t row0 = (size_t)hd.x * x.a.Hq + hd.y * x.G + rb * GB;
    const bool apart = n <= FEW && gridDim.y == 1 && GB > 1;
    const int step = apart ? 1 : JW;
    for (int in = apart ? warp : (int)blockIdx.y; in < heads; in += apart ? JW : (int)gridDim.y) {
        float o[NC] = {}, m = -CUDART_INF_F, l = 0.f;
        for (int i = apart ? 0 : warp; i < n; i += 4 * step) {
            float2 ml[4];
            float y[4][NC], mb = m;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int k = i + u * step < n ? i + u * step : 0;  // behind the last part: the first one's, dropped
                // a CTA's second slot only for a segment that begins behind another
                const size_t at = (size_t)(2 * (blockIdx.x + k) + (k == 0 ? slot0 : 0)) * GB + in;
                ml[u] = x.ml[at];
#pragma unroll
                for (int c = 0; c < NC; ++c) y[u][c] = x.part[at * D + c * 32 + lane];
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i + u * step < n) mb = fmaxf(mb, ml[u].x);
            const float g = m == mb ? 1.f : weight(m - mb);  // equal: both may be -inf
            m = mb;
            l *= g;
#pragma unroll
            for (int c = 0; c < NC; ++c) o[c] *= g;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (i + u * step >= n) break;
                const float f = ml[u].y == 0.f ? 0.f : weight(ml[u].x - m);  // l = 0: the part's m may be -inf
                l += ml[u].y * f;
#pragma unroll
                for (int c = 0; c < NC; ++c) o[c] += f * y[u][c];
            }
        }
        const size_t row = row0 + in;
        if (apart) {
#pragma unroll
            for (int c = 0; c < NC; ++c) ((E *)x.a.out)[row * D + c * 32 + lane] = from_f<E>(l > 0.f ? o[c] / l : (l == l ? 0.f : l));
        } else {
            __syncthreads();  // the head before is read
#pragma unroll
            for (int c = 0; c < NC; ++c) red[warp][c * 32 + lane] = o[c];
            if (lane == 0) {
                wm[warp] = m;
                wl[warp] = l;
            }
            __syncthreads();
            float g[JW];
#pragma unroll
            for (int w = 0; w < JW; ++w) m = fmaxf(m, wm[w]);
            l = 0.f;
#pragma unroll
            for (int w = 0; w < JW; ++w) {
                g[w] = wl[w] == 0.f ? 0.f : weight(wm[w] - m);
                l += wl[w] * g[w];
            }
            for (int c = threadIdx.x; c < D; c += JW * 32) {
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < JW; ++w) s += red[w][c] * g[w];
                ((E *)x.a.out)[row * D + c] = from_f<E>(l > 0.f ? s / l : (l == l ? 0.f : l));
            }
        }
        if (x.a.lse && lane == 0 && (apart || warp == 0)) x.a.lse[row] = lse_of(m, l);
    }
    let_next();
}

template <class C, int D> static cudaError_t launch(Args x, cudaStream_t s) {
    const AttnDecode &a = x.a;
    x.GB = C::GB;
    x.RB = (x.G + C::GB - 1) / C::GB;
    x.head = (int4 *)a.ws;
    x.ml = (float2 *)(x.head + MAX_CTAS);
    x.part = (float *)(x.ml + 2 * MAX_CTAS * C::GB);  // 16-byte aligned
    x.whole = a.page % C::P::TILE == 0;
    const int smem = smem_bytes<C, D>();
    cudaError_t e = cudaFuncSetAttribute(k_attn<C, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // no more CTAs than the tables have room for runs
    const double tiles = (double)a.R * a.Hk * x.RB * ((double)a.width * a.page / C::P::TILE + 1 + COST);
    const int ctas = tiles / MIN_UNITS < C::CTAS - 1 ? (int)(tiles / MIN_UNITS) + 1 : C::CTAS;
    x.inv_ctas = 1.0 / ctas;
    e = launch_after(k_attn<C, D>, dim3(ctas), dim3(THREADS), smem, s, x);
    if (e != cudaSuccess) return e;
    // With few segments each may have many parts, and every head gets a block of its own; with more
    // than an eighth of the CTAs there are a handful of parts on average, and one block takes a
    // segment's heads, a warp each (200 requests of up to 2000 tokens: 41.4 us, with a block for every
    // head of every run, most of them with nothing to do, 43.7; one request of 2000 tokens the other
    // way round).
    const bool many = (double)a.R * a.Hk * x.RB * 8 > MAX_CTAS;
    return launch_after(k_attn_join<typename C::E, D>, dim3(ctas, many ? 1 : C::GB), dim3(256), 0, s, x);
}

static int heads_per_block(int G, bool bf16) {
    if (bf16) return G <= 8 ? 8 : 16;
    return G <= 2 ? G : (G <= 4 ? 4 : 8);
}

template <int D> static cudaError_t simt(const Args &x, int GB, cudaStream_t s) {
    return GB == 1 ? launch<Simt<D, 1>, D>(x, s)
                   : (GB == 2 ? launch<Simt<D, 2>, D>(x, s) : (GB == 4 ? launch<Simt<D, 4>, D>(x, s) : launch<Simt<D, 8>, D>(x, s)));
}

}  // namespace ad

size_t attn_decode_ws_bytes(int Hq, int Hk, int d, bool bf16) {
    const int GB = ad::heads_per_block(Hq / Hk, bf16);
    return ad::MAX_CTAS * sizeof(int4) + (size_t)2 * ad::MAX_CTAS * GB * (d + 2) * sizeof(float);
}

cudaError_t attn_decode_run(const AttnDecode &p, bool bf16, cudaStream_t s) {
    ad::Args x = {};
    x.a = p;
    if (p.n_pages == 0) x.a.width = 0;  // no page: nothing is seen, no address is formed
    x.G = p.Hq / p.Hk;
    x.scale2 = p.scale * ad::LOG2E;
    x.by_page = FastDiv(p.page);
    x.alike = p.ks == p.vs;
    const int GB = ad::heads_per_block(x.G, bf16);
    if (!bf16) return p.d == 128 ? ad::simt<128>(x, GB, s) : ad::simt<64>(x, GB, s);
    if (p.d == 128)
        return GB == 8 ? ad::launch<ad::Mma<128, 1>, 128>(x, s) : ad::launch<ad::Mma<128, 2>, 128>(x, s);
    return GB == 8 ? ad::launch<ad::Mma<64, 1>, 64>(x, s) : ad::launch<ad::Mma<64, 2>, 64>(x, s);
}

}  // namespace dr
