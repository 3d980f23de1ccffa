// narrow_slope_bf16.hip -- the narrow linear backward kernels for dz as dy act'(z), dy in bf16.
#define NARROW_SZ SLOPE_BF16
#include "narrow.inc"
