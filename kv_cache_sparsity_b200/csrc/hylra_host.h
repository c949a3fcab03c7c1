// hylra_host.h - host-side state that the library's CUDA translation units share.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

namespace hylra {

// Limit of the kernels' bounded waits for launches made now, in SM clocks
// (hylra_set_wait_limit).
long long host_wait_limit();

// The driver's tensor map encoder; nullptr when the driver has none.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

}  // namespace hylra
