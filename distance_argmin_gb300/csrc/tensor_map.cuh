// The driver's tensor-map encoder, looked up once.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

namespace km {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

}  // namespace km
