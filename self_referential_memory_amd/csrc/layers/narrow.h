// narrow.h -- both gradients of a linear layer whose weights fit in LDS beside
// a slice of rows (kernels in narrow.inc).
#ifndef SRNL_LAYERS_NARROW_H
#define SRNL_LAYERS_NARROW_H

#include "linear.h"

namespace srnl_i {

struct NarrowArgs {
    Operand dz, w, x;
    long long M;
    int K, N;
    Epilogue dx;
    float *dw, *db;        // [blocks][N][K], [blocks][N]; db may be NULL
};

template <Source SZ>
__attribute__((visibility("hidden"))) srnl_status narrow_launch(const NarrowArgs &g, int blocks, Source sw, Source sx,
                                                                hipStream_t st);
template <> srnl_status narrow_launch<BF16>(const NarrowArgs &, int, Source, Source, hipStream_t);
template <> srnl_status narrow_launch<FP32>(const NarrowArgs &, int, Source, Source, hipStream_t);
template <> srnl_status narrow_launch<SLOPE_BF16>(const NarrowArgs &, int, Source, Source, hipStream_t);
template <> srnl_status narrow_launch<SLOPE_FP32>(const NarrowArgs &, int, Source, Source, hipStream_t);

}  // namespace srnl_i

#endif
