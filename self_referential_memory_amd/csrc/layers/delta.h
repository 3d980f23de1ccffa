// delta.h -- the gated delta rule's arguments and sizes, shared by its
// translation units.
//
// In chunks of 64 tokens, with G the sums of g inside a chunk, S0 and S1 the
// states before and after it, hats for normalised rows and b = diag(beta):
//   M_ij = e^(G_i - G_j) k^_i.k^_j (j < i),  P_ij = scale e^(G_i - G_j) q^_i.k^_j (j <= i)
//   X = (I + M b)^-1,  E = X (V - e^G K^ S0),  U = b E
//   O = scale e^G Q^ S0 + P U,  S1 = e^(G_63) S0 + (e^(G_63 - G) K^)^T U
// and backward, D1 and D0 the gradients of S1 and S0:
//   dU = e^(G_63 - G) K^ D1 + P^T dO,  dV = X^T b dU
//   D0 = e^(G_63) D1 + (scale e^G Q^)^T dO - (e^G K^)^T dV
// (tokens as rows). The error E = V - S^T K before beta, and not U, is what is kept: beta may be 0.
// Every exponent is a difference of later and earlier sums, at most 0 for g <= 0.
//
// Kernels: per chunk X and P (delta_prep.hip); the states from chunk to chunk
// with the outputs, and their gradients back (delta_chain.hip); the gradients of
// q, k, g and beta per chunk (delta_grads.hip); single tokens (delta_step.hip).
#ifndef SRNL_LAYERS_DELTA_H
#define SRNL_LAYERS_DELTA_H

#include "common.h"

namespace srnl_i {

constexpr int DELTA_CHUNK = 64;
constexpr int DELTA_SQUARE = 64 * 64 * 6;      // bytes of X or P of one chunk, at most
// a chunk's row factors: what the chain takes at once (e^G / |k|, e^(G_63 - G) beta
// / |k|, beta, scale e^G / |q|), and e^G, e^(G_63 - G), 1/|k|, 1/|q|, G in two floats
enum { VEC_READK = 0, VEC_WRITE = 64, VEC_BETA = 128, VEC_READQ = 192, VEC_GAM = 256, VEC_END = 320, VEC_RK = 384,
       VEC_RQ = 448, VEC_GHI = 512, VEC_GLO = 576, VEC_FLOATS = 640 };

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
    int N;                       // chunks of an item
    // per (item, head, chunk), in this order
    char *X, *P;                 // [64][64] split values, as operands
    float *vec;                  // [VEC_FLOATS]
    float *E;                    // record: [64][Dv]
    float *S0;                   // record: [Dk][Dv]
    // backward
    const void *dout;
    const float *dstate_out;
    void *dq, *dk, *dv;
    float *dg, *dbeta, *dstate;
    float *dV;                   // [64][Dv]
    float *D1;                   // [Dk][Dv]
    float *dq_part, *dk_part;    // [B][T][H][Dk], where heads share q and k
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
srnl_status launch_delta_prep(const DeltaArgs &a, bool transposed, hipStream_t st);
srnl_status launch_delta_chain(const DeltaArgs &a, bool backward, hipStream_t st);
srnl_status launch_delta_grads(const DeltaArgs &a, hipStream_t st);

// f<BF16, width of k padded to 32, 64 or 128>
#define SRNL_DELTA_DISPATCH(a, CALL)                                                             \
    do {                                                                                         \
        if ((a).bf) {                                                                            \
            if ((a).Dk <= 32) { CALL(true, 32); } else if ((a).Dk <= 64) { CALL(true, 64); }     \
            else { CALL(true, 128); }                                                            \
        } else {                                                                                 \
            if ((a).Dk <= 32) { CALL(false, 32); } else if ((a).Dk <= 64) { CALL(false, 64); }   \
            else { CALL(false, 128); }                                                           \
        }                                                                                        \
    } while (0)

}  // namespace srnl_i

#endif
