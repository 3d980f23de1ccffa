// narrow_bf16.hip -- the narrow linear backward kernels for dz as bf16.
#define NARROW_SZ BF16
#include "narrow.inc"
