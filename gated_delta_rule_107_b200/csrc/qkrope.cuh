// qkrope.cuh -- norm of query and key heads with the rotation by position (qkrope.cu).
#pragma once
#include "softmax_layer.cuh"

namespace dr {

// Arguments of one call (device pointers; N = B * T tokens, d channels a head).
//   forward   q, k -> qo, ko (dense [N][H][d])
//   cache     q, k, v -> qo (dense) and the token's slot of kc, vc
//   backward  q, k, gq, gk (gradients of qo, ko, dense) -> dq, dk (rows dqs, dks apart), dwq, dwk
// Strides are in elements: from a token to the next (q, k, v, dq, dk; a token's heads are dense); of
// kc, vc see CacheStrides.
struct QkRope {
    const void *q, *k, *v;
    long long qs, ks, vs;
    const float *wq, *wk;
    const double *inv_freq;
    const int *pos;
    size_t N;
    int T, Hq, Hk, d, rot;
    bool interleaved;
    void *qo, *ko;
    // cache
    const long long *slots;
    void *kc, *vc;
    CacheStrides kcs, vcs;
    long long n_slots;
    int page;
    // backward
    const void *gq, *gk;
    void *dq, *dk;
    long long dqs, dks;
    float *dwq, *dwk, *part;
};

size_t qkrope_ws_bytes(int d);
cudaError_t qkrope_run(const QkRope &p, bool bf16, cudaStream_t s);       // forward; cache when p.slots
cudaError_t qkrope_bwd_run(const QkRope &p, bool bf16, cudaStream_t s);

}  // namespace dr
