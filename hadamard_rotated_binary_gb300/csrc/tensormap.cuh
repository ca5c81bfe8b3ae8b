// The driver's TMA descriptor encoder, looked up once (bitlin_api.cu).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

PFN_cuTensorMapEncodeTiled_v12000 bitlin_tensormap_encode_fn();
