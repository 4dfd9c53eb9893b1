// attn_decode.cuh -- attention of one new token over a paged key-value cache (attn_decode.cu).
#pragma once
#include "softmax_layer.cuh"

namespace dr {

// Arguments of one call (device pointers).  q, out [R, Hq, d] and lse [R, Hq] dense; kc, vc pages of
// `page` tokens with the strides ks, vs; table [R, width]; lens [R].
struct AttnDecode {
    const void *q, *kc, *vc;
    const int *table, *lens;
    void *out;
    float *lse;
    CacheStrides ks, vs;
    int R, Hq, Hk, d, page, n_pages, width, window;
    float scale;
    void *ws;
};
size_t attn_decode_ws_bytes(int Hq, int Hk, int d, bool bf16);
cudaError_t attn_decode_run(const AttnDecode &p, bool bf16, cudaStream_t s);

}  // namespace dr
