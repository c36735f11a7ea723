// Tensor maps for TMA: the driver's encoder.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

namespace kda {

// cuTensorMapEncodeTiled from the driver, looked up once through the runtime (chunk_tc.cu); NULL if absent.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

}  // namespace kda
