// host.h -- the host-side helpers that the library's C entry points share
// (defined in api.cu).  None of them synchronises, allocates or copies.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "../../include/rd.h"
#include "wait_bound.h"

namespace rd {

constexpr int64_t kMaxDim = 0x7FFFFFFF;
// widest output of a grouped product: the last tile (at most 256 columns or, of dw, rows) ends within 32 bits
constexpr int64_t kMaxWidth = kMaxDim - 255;

// bound of every wait inside the kernels (rd_set_tuning, or the default)
WaitBound wait_limit();

// SM count of the current device, and whether it is an sm_103 part
rd_status current_device(int* sms);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
  if (a == nullptr || b == nullptr || na == 0 || nb == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

// tensor map of 2-byte elements; dims/strides innermost first
rd_status encode(CUtensorMap* map, const void* base, int rank, const uint64_t* dims,
                 const uint64_t* strides_bytes, const uint32_t* box,
                 CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);

// checks shared by the grouped calls
rd_status check_groups(int64_t m, int64_t k, int64_t n, const int32_t* group_sizes,
                       int32_t g_total, int32_t group_offset, int32_t g_local,
                       const int32_t* limit, const int32_t* status);

int grid_for(int sms, int64_t tiles_upper_bound);
int pair_grid(int sms, int64_t pair_tiles_upper_bound);
// whether a grouped product runs on CTA pairs, and the m-tiles per band of its tile order
constexpr int32_t kBandRows = 6144;  // default rows of a band (bf16 rows: 48 MB at k = 4096)
bool use_pair(int sms, int64_t m, int32_t g_total);
bool variant_forced();  // by rd_set_tuning
int32_t band_tiles(bool pair, int32_t default_rows = kBandRows);

}  // namespace rd
