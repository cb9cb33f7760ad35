// fa_internal.h -- checks shared by the library's translation units (not part
// of the C ABI; hidden symbols).
#pragma once

#include <cuda.h>

#include "fa.h"

namespace fa_detail {

// Every argument check of fa_fwd_ex that needs no device, except the
// caller-owned workspace clause (which fa_fwd_static_workspace replaces).
fa_status validate_args(const fa_fwd_params *p);

// FA_OK when the current device is an sm_100 device the library supports
// (cached per device ordinal); FA_ERR_UNSUPPORTED or FA_ERR_CUDA otherwise.
fa_status probe_current_device();

// The same, with the device's ordinal and its number of SMs.
fa_status current_device(int *dev, int *num_sms);

// The tensor map of a cache's codes: [tiles][lines][line_bytes] with boxes of one tile's
// lines by 128 bytes, 128-byte swizzle.
fa_status encode_cache_map(CUtensorMap *map, const void *codes, long long tiles, int lines, int line_bytes);

// Device ordinals are below this (current_device refuses others).
constexpr int kMaxDevices = 64;

inline bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// The rule of fa_rotary_init's result (rotary->ready and its dim within d).
fa_status validate_rotary(const fa_rotary *r, int d);

}  // namespace fa_detail
