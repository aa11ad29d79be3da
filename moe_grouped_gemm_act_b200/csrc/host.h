// host.h -- what the host sides of the MXFP4 and routing translation units share.
#pragma once

#include <cuda_runtime.h>

#include "dg.h"

namespace dg {

// A CUDA call's outcome as a status.  A failure is taken out of the runtime's
// last-error slot: the next entry point that asks for it would report it as its own.
inline int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return DG_OK;
  (void)cudaGetLastError();
  return DG_ERR_CUDA;
}

}  // namespace dg
