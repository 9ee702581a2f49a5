// What the host files of the C ABI share (api.cu has the bodies).
#pragma once

#include <cuda.h>

#include "llsa.h"

namespace llsa {

// LLSA_OK, or why the descriptor is refused.
int check_desc(const llsa_desc* d);

// cuTensorMapEncodeTiled, fetched from the driver once (no link-time libcuda);
// NULL where there is no driver.
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled();

}  // namespace llsa
