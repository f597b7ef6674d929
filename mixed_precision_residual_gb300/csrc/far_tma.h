// The driver's tensor-map encoder, looked up once (far_gemm.cu).
#pragma once

#include <cudaTypedefs.h>

namespace far {

int get_encoder(PFN_cuTensorMapEncodeTiled_v12000* fn);

}  // namespace far
