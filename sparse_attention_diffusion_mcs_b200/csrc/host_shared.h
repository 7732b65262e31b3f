// host_shared.h -- what the library's translation units share on the host.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mcs {

// this device's status word (null when no device is current)
unsigned *device_status_word();
// the bound on any single wait inside a kernel, in nanoseconds
uint64_t wait_limit_ns();
// 2D tensor map over `rows` rows of `row_bytes` bytes (64 or 128), boxes of
// box_rows whole rows, swizzled by the row's width; rows behind the end read as 0
bool map_byte_rows(CUtensorMap *m, const void *base, int row_bytes, size_t rows, unsigned box_rows);

}  // namespace mcs
