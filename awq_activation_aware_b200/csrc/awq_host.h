// What the library's two translation units tell each other (not part of its ABI).
#pragma once

#include <cstdint>

namespace awq_host {

// The limit set by awq_set_wait_timeout_ms.
uint32_t wait_timeout_ms();

// Reads and clears the error word of the cache operators' kernels (0: none raised); false if CUDA fails.
bool take_kv_errors(unsigned *flags);

}  // namespace awq_host
