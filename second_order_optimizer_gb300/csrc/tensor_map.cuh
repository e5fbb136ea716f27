// The driver's tensor-map encoder, looked up once (null when the driver lacks it).
#pragma once
#include <cudaTypedefs.h>

namespace kfac {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();
}  // namespace kfac
