// operator_unit.hip -- the operator's translation unit (srnl.hip, complete in
// itself) with its error record opened to the layers' units.
#include "../srnl.hip"

#include "error.h"

srnl_status srnl_set_error(srnl_status s, const char *msg) noexcept
{
    try {
        g_last_error = msg;
    } catch (...) {      // no memory for the text: the status still stands
    }
    return s;
}
