// Host-side pieces that the entry points share (defined in api.cu): the per-device state and its
// architecture check, and TMA tensor maps.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "svdq.h"

namespace svdq {

struct DeviceState {
  svdq_status arch = SVDQ_OK;
  int index = 0;  // CUDA device number
  int num_sms = 0;
  uint32_t *err = nullptr;  // the device's error word
};

// Checks the current device once; SVDQ_OK and its state, or why it cannot be used.
svdq_status device_check(DeviceState **out);

// 2-d tensor map: `outer` rows of `inner` elements, row_bytes apart.
bool make_map(CUtensorMap *m, CUtensorMapDataType dt, const void *base, uint64_t inner, uint64_t outer,
              uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swz);

// 3-d tensor map of a contiguous array; boxes of one outer index.
bool make_map_3d(CUtensorMap *m, CUtensorMapDataType dt, const void *base, uint64_t inner, uint64_t middle, uint64_t outer,
                 uint64_t elem_bytes, uint32_t box_inner, uint32_t box_middle, CUtensorMapSwizzle swz);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace svdq
