// The calling thread's error message, shared by the parts of the C ABI layer
// (la_api.cpp, la_muon_api.cpp). Not installed.
#pragma once

#include "layeradam.h"

namespace la {

// Records the message of a failed call and returns its status.
la_status fail(la_status code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

// Clears the message and returns LA_OK.
la_status ok();

// Launch facts and environment overrides read once (la_api.cpp).
int max_grid();

}  // namespace la
