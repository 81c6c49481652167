// Error reporting shared by the files of the C-ABI host layer.
#pragma once

#include "../../include/flashbev.h"

namespace fbev {

// Records the calling thread's last-error text and returns `s`.
fbev_status fail(fbev_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

}  // namespace fbev
