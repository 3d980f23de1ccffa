// narrow_fp32.hip -- the narrow linear backward kernels for dz as fp32.
#define NARROW_SZ FP32
#include "narrow.inc"
