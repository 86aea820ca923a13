// Tensor maps of the operators (host): cuTensorMapEncodeTiled through the runtime.
#pragma once
#include <cuda.h>

#include "ops_host.h"

namespace tre {

// A tensor of `rank` dimensions (fastest first) of `dims` entries, `strides` bytes apart from
// the second dimension on, boxes of `box` entries; entries outside the tensor read as zero.
tre_status encode_map(const char* op, CUtensorMapDataType type, int rank, const void* base,
                      const uint64_t* dims, const uint64_t* strides, const uint32_t* box,
                      CUtensorMapSwizzle swizzle, CUtensorMap* out);

}  // namespace tre
