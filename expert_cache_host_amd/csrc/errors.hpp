// The thread's error message behind moe_last_error (kept in api.cpp).
#pragma once
#include <string>

#include "../../include/moe_cache.h"

namespace moe {

// Clears the calling thread's message (the start of every C entry).
void clear_error();
// Sets it and returns `st`; never throws.
moe_status set_error(moe_status st, const char *msg);

}  // namespace moe
