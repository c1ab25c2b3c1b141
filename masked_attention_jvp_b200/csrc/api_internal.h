// Shared by the C-ABI front ends: error text, device check, wait limit and the
// TMA descriptor encoder (defined in api.cpp).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "causaljvp.h"

namespace caj {

// Records the error's text for caj_last_cuda_error; returns CAJ_ERR_CUDA.
caj_status cuda_fail(cudaError_t e);
// CAJ_OK on an sm_100 device (cached per device).
caj_status check_device();
uint64_t wait_timeout_ns();
int32_t fault_mode();
// 2-D bf16 map over rows of `cols` elements, `ld` elements apart (a multiple of
// 8), box = 64 columns x box_rows, 128-byte swizzle, zero fill outside.
bool encode_map_2d_ld(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, int64_t ld, int box_rows);
// Output tiles of 32 rows of 64 bytes (32 bf16 or 16 fp32 columns), 64-byte swizzle, over
// contiguous rows.
bool encode_out_2d(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, bool f32);

inline bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace caj
