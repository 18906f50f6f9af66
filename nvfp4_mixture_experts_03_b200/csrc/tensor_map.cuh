// The driver's tensor-map encoder, as both hosts of TMA kernels get it.
#pragma once
#include <cuda.h>

namespace nvmoe {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();   // cuTensorMapEncodeTiled, or null

}  // namespace nvmoe
