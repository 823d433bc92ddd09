// pgd_host.h -- host-side state shared by the C ABI's translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pgd.h"

namespace pgd {

// SM count and device flag word of the current device.
pgd_status device_info(int *sms, uint32_t **flags);

// Limit of the kernels' pipeline waits in ns (pgd_debug_set_wait_limit_ns).
uint64_t wait_limit_ns();

// cuTensorMapEncodeTiled for a bf16 or byte tensor of `rank` dimensions, with
// the 128-byte swizzle; strides in bytes for dimensions 1 .. rank - 1.
pgd_status encode_tiled_map(CUtensorMap *m, const void *base, int elem_bytes, int rank,
                            const uint64_t *dims, const uint64_t *strides, const uint32_t *box);

}  // namespace pgd
