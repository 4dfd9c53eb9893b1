// pages.cu -- pages of a key-value cache given to the requests of a batch, and each new token's
// place in the cache, from the requests' lengths alone.
//
// Request r holds cached[r] tokens in have = ceil(cached / page) pages and gets fresh[r] more, so
// need = ceil((cached + fresh) / page) pages.  With c, t the exclusive prefix sums over the
// requests of fresh and of need - have:
//   page j of request r, have <= j < need, is the (t[r] + j - have)th page from the top of the
//     stack of free pages (-1 behind its end)
//   token n, c[r] <= n < c[r + 1], has position p = cached[r] + n - c[r] and slot
//     page(p / page) * page + p % page (-1 where that page is -1)
//
// One launch, and what a CTA writes depends on no other CTA: every CTA forms both prefix sums over
// all requests for itself in shared memory (96 KB at the most requests; 509 requests take about a
// microsecond), finds the request of a token or a page by bisection, and takes the page number of
// a token from the table where the request had the page before and from the stack where it is
// new.  So no CTA reads a table entry that another writes.  What bounds it is the launch and that
// chain of dependent reads (lengths, prefix sums, bisection, page number), not the bytes, 12 a token:
// 66 tokens take 3.1 us, 1.04 million 7.9 (1.6 TB/s).
#include <limits.h>

#include "pages.cuh"

namespace dr {
namespace pgs {

constexpr int MAX_THREADS = 1024, MAX_CTAS = 148;

__device__ __forceinline__ int add_sat(int a, int b) {  // both >= 0; associative
    const unsigned s = (unsigned)a + (unsigned)b;
    return s > (unsigned)INT_MAX ? INT_MAX : (int)s;
}
// pages of n tokens, at most the table's width
__device__ __forceinline__ int pages_of(int n, const Pages &p) {
    const int q = p.by_page.div(n);
    return min(q + (n != q * p.page), p.width);
}
// the last i in [lo, hi) with sum[i] <= x, where sum[lo] <= x
__device__ __forceinline__ int find(const int *sum, int lo, int hi, int x) {
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sum[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

// UNROLL: tokens of a lane; a warp takes 32 UNROLL neighbouring tokens at a time
template <int UNROLL> __global__ void __launch_bounds__(MAX_THREADS) k_pages(const Pages p) {
    extern __shared__ int sh[];
    int *c = sh, *t = c + p.R + 1, *had = t + p.R + 1;  // prefix sums [R + 1]: new tokens, new pages; cached tokens [R]
    __shared__ int wsum[2][MAX_THREADS / 32];
    const int threads = blockDim.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    after_previous();
    // each thread sums a run of requests, then the runs are scanned over the CTA
    const int per = (p.R + threads - 1) / threads, r0 = min(p.R, tid * per), r1 = min(p.R, r0 + per);
    int sc = 0, st = 0;
    for (int r = r0; r < r1; ++r) {
        const int a = max(p.cached[r], 0), f = max(p.fresh[r], 0);
        had[r] = a;
        c[r] = f;
        t[r] = pages_of(add_sat(a, f), p) - pages_of(a, p);
        sc = add_sat(sc, c[r]);
        st = add_sat(st, t[r]);
    }
    int ic = sc, it = st;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int xc = __shfl_up_sync(0xffffffffu, ic, o), xt = __shfl_up_sync(0xffffffffu, it, o);
        if (lane >= o) {
            ic = add_sat(ic, xc);
            it = add_sat(it, xt);
        }
    }
    if (lane == 31) {
        wsum[0][warp] = ic;
        wsum[1][warp] = it;
    }
    // exclusive inside the warp: the inclusive sum of the lane before
    int ec = __shfl_up_sync(0xffffffffu, ic, 1), et = __shfl_up_sync(0xffffffffu, it, 1);
    if (lane == 0) ec = et = 0;
    __syncthreads();
    // the sums of the warps before, by shuffles (saturated sums may be added in any order)
    int bc = lane < warp ? wsum[0][lane] : 0, bt = lane < warp ? wsum[1][lane] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        bc = add_sat(bc, __shfl_xor_sync(0xffffffffu, bc, o));
        bt = add_sat(bt, __shfl_xor_sync(0xffffffffu, bt, o));
    }
    ec = add_sat(ec, bc);
    et = add_sat(et, bt);
    for (int r = r0; r < r1; ++r) {
        const int xc = c[r], xt = t[r];
        c[r] = ec;
        t[r] = et;
        ec = add_sat(ec, xc);
        et = add_sat(et, xt);
    }
    if ((r0 < p.R && r1 == p.R) || (p.R == 0 && tid == 0)) {
        c[p.R] = ec;
        t[p.R] = et;
    }
    __syncthreads();

    const int total = c[p.R], taken = t[p.R], free = min(max(*p.n_free, 0), p.F);
    // unsigned: an index below 2^31 plus a stride does not wrap
    const unsigned gtid = blockIdx.x * threads + tid, gsize = gridDim.x * threads;
    auto page_of = [&](int nth) { return nth < free ? p.free_pages[free - 1 - nth] : -1; };
    for (unsigned r = gtid; r <= (unsigned)p.R; r += gsize) {
        p.cu_new[r] = c[r];
        if (r < (unsigned)p.R) p.lens[r] = add_sat(had[r], max(p.fresh[r], 0));
    }
    if (gtid == 0) *p.n_left = free - taken;
    // from the last thread down: where there are more warps than tokens' worth, those take the pages
    for (unsigned u = gsize - 1 - gtid; u < (unsigned)taken; u += gsize) {
        const int i = (int)u, r = find(t, 0, p.R, i);
        const int j = pages_of(had[r], p) + i - t[r];
        p.table[(size_t)r * p.width + j] = page_of(i);
    }
    for (unsigned w = (gtid >> 5) * (32 * UNROLL); w < (unsigned)p.N; w += gsize * UNROLL) {
        int r[UNROLL], pos[UNROLL], pg[UNROLL];
        if (w < (unsigned)total) {  // the requests of the warp's first and last token, then the lanes' between them
            const int last = (int)min(w + (32 * UNROLL - 1), (unsigned)total - 1);
            const int r0 = find(c, 0, p.R, (int)w), r1 = c[r0 + 1] > last ? r0 + 1 : find(c, r0, p.R, last) + 1;
#pragma unroll
            for (int k = 0; k < UNROLL; ++k) r[k] = find(c, r0, r1, min((int)w + lane + 32 * k, last));
        }
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
            const unsigned n = w + lane + 32 * k;
            pos[k] = 0;
            pg[k] = -1;
            if (n < (unsigned)total && n < (unsigned)p.N) {
                const int a = had[r[k]];
                pos[k] = add_sat(a, (int)n - c[r[k]]);
                const int j = p.by_page.div(pos[k]), have = pages_of(a, p);
                if (j < p.width) pg[k] = j < have ? p.table[(size_t)r[k] * p.width + j] : page_of(t[r[k]] + j - have);
            }
        }
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
            const unsigned n = w + lane + 32 * k;
            if (n >= (unsigned)p.N) break;
            p.positions[n] = pos[k];
            p.slots[n] = pg[k] < 0 ? -1ll : (long long)pg[k] * p.page + (pos[k] - p.by_page.div(pos[k]) * p.page);
        }
    }
    let_next();
}

}  // namespace pgs

cudaError_t pages_run(const Pages &args, cudaStream_t s) {
    Pages p = args;
    p.by_page = FastDiv(p.page);
    auto bytes = [](int R) { return (3 * (size_t)R + 2) * sizeof(int); };
    const size_t smem = bytes(p.R);
    // One token a lane in CTAs of 256 threads while one wave of them holds all tokens (66 tokens of 64
    // requests: 3.1 us, four a lane 5.1), else eight a lane, whose reads overlap and whose search is
    // shared, in CTAs of 1024, so that the prefix sums are formed once an SM (10^6 tokens of 509
    // requests: 7.9 us, four a lane 9.4, one a lane 15.3).  The requests' own outputs need a thread each as well.
    const long long most = p.N > p.R ? p.N : p.R;
    auto go = [&](auto kern, int threads, int unroll) -> cudaError_t {
        // Without this a launch has 48 KB, the kernel's static part among them.  The most that any call
        // needs, whatever this one does: another thread's launch may come between.
        if (smem > 32 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       (int)bytes(PAGES_MAX_REQUESTS));
            if (e != cudaSuccess) return e;
        }
        long long ctas = (most + threads * unroll - 1) / (threads * unroll);
        ctas = ctas < 1 ? 1 : (ctas > pgs::MAX_CTAS ? pgs::MAX_CTAS : ctas);
        return launch_after(kern, dim3((unsigned)ctas), dim3(threads), smem, s, p);
    };
    return most <= 256 * pgs::MAX_CTAS ? go(pgs::k_pages<1>, 256, 1) : go(pgs::k_pages<8>, pgs::MAX_THREADS, 8);
}

}  // namespace dr
