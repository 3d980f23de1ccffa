// error.h -- the error record behind srnl_last_error(), shared by the
// library's translation units.
#ifndef SRNL_LAYERS_ERROR_H
#define SRNL_LAYERS_ERROR_H

#include "srnl.h"

// Sets srnl_last_error()'s text on the calling thread and returns s (operator_unit.hip).
__attribute__((visibility("hidden"))) srnl_status srnl_set_error(srnl_status s, const char *msg) noexcept;

#endif
