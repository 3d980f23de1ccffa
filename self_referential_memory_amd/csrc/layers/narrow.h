// narrow.h -- both gradients of a linear layer whose weights fit in LDS beside
// a slice of rows (kernels in narrow.inc).
#ifndef SRNL_LAYERS_NARROW_H
#define SRNL_LAYERS_NARROW_H

#include "linear.h"

namespace srnl_i {

constexpr int kThreads = 512;                 // eight waves
constexpr int kLdsWords = 81920;              // all 160 KB: one block a CU
constexpr int kMaxPieces = 4;                 // 8-element pieces of dz, or of x, per thread and slice (6 of both)

struct NarrowArgs {
    Operand dz, w, x;
    long long M;
    int K, N;
    Epilogue dx;
    float *dw, *db;        // [blocks][N][K], [blocks][N]; db may be NULL
};

constexpr int narrow_parts(Source s) { return s == BF16 ? 1 : 3; }
constexpr int narrow_width(int n) { return n <= 64 ? 64 : n <= 128 ? 128 : 256; }

// Rows per slice for widths rounded up: the most that LDS, the pieces a thread
// holds in flight and two dx tiles a wave allow; 0 where not even 32 fit.
constexpr int narrow_rows(int kp, int np, Source sz, Source sw, Source sx)
{
    if (kp * np > 16384)
        return 0;
    for (int bm = 128; bm >= 32; bm /= 2) {
        const int words = narrow_parts(sz) * bm * np + narrow_parts(sx) * bm * kp + narrow_parts(sw) * np * kp;
        const int most = 8 * kThreads * kMaxPieces;
        if (words <= kLdsWords && bm * np <= most && bm * kp <= most && bm * (np + kp) <= most * 3 / 2 &&
            (bm / 32) * (kp / 32) <= 16 &&
            bm * np >= 8 * kThreads && bm * kp >= 8 * kThreads)
            return bm;
    }
    return 0;
}

// Partial weight (and bias) gradients that narrow_launch leaves for the caller
// to join, one a block; 0 where it does not take the layer. Every block should
// have a few slices.
inline int narrow_bwd_parts(long long M, int K, int N, Source sz, Source sw, Source sx)
{
    if (K % 8 || N % 8 || K > 256 || N > 256)
        return 0;
    const int bm = narrow_rows(narrow_width(K), narrow_width(N), sz, sw, sx);
    return bm && M >= 512LL * bm ? 256 : 0;
}

template <Source SZ>
__attribute__((visibility("hidden"))) srnl_status narrow_launch(const NarrowArgs &g, int blocks, Source sw, Source sx,
                                                                hipStream_t st);
template <> srnl_status narrow_launch<BF16>(const NarrowArgs &, int, Source, Source, hipStream_t);
template <> srnl_status narrow_launch<FP32>(const NarrowArgs &, int, Source, Source, hipStream_t);
template <> srnl_status narrow_launch<SLOPE_BF16>(const NarrowArgs &, int, Source, Source, hipStream_t);
template <> srnl_status narrow_launch<SLOPE_FP32>(const NarrowArgs &, int, Source, Source, hipStream_t);

}  // namespace srnl_i

#endif
