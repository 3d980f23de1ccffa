// delta.h -- the gated delta rule's arguments and sizes, shared by its
// translation units.
#ifndef SRNL_LAYERS_DELTA_H
#define SRNL_LAYERS_DELTA_H

#include "common.h"

namespace srnl_i {

// One call: the public parameters with strides filled in, and its buffers.
struct DeltaArgs {
    const void *q, *k, *v;
    const float *g, *beta, *state;
    const int *lengths;
    int B, T, Hk, H, Dk, Dv;
    long long qs, ks, vs;        // elements between tokens
    bool bf;
    float scale, eps;
    void *out;
    float *state_out;
};

// The tokens of item b that count.
__device__ __forceinline__ int delta_tokens(const DeltaArgs &a, int b)
{
    if (!a.lengths)
        return a.T;
    const int n = a.lengths[b];
    return n < 0 ? 0 : n > a.T ? a.T : n;
}

srnl_status launch_delta_step(const DeltaArgs &a, hipStream_t st);

}  // namespace srnl_i

#endif
