// narrow_slope_fp32.hip -- the narrow linear backward kernels for dz as dy act'(z), dy in fp32.
#define NARROW_SZ SLOPE_FP32
#include "narrow.inc"
