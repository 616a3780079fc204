// Status and error text of the C ABI, shared by its source files.
#pragma once

#include "q4gemv.h"

namespace q4 {

// Sets the calling thread's text for q4_last_error() and returns `code`.
q4_status set_status(q4_status code, const char* text);

}  // namespace q4
