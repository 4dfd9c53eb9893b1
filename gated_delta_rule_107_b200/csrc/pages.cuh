// pages.cuh -- pages of a key-value cache given to requests (pages.cu).
#pragma once
#include "softmax_layer.cuh"

namespace dr {

constexpr int PAGES_MAX_REQUESTS = 8192;

// Arguments of one call (device pointers; R requests, `width` table entries each, N tokens).
struct Pages {
    const int *cached, *fresh, *free_pages, *n_free;
    int *table;
    int *lens, *cu_new, *positions, *n_left;
    long long *slots;
    int R, F, width, page, N;
    FastDiv by_page;  // set by pages_run
};
cudaError_t pages_run(const Pages &p, cudaStream_t s);

}  // namespace dr
