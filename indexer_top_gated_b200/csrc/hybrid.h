// hybrid.h - what dsa.cu and hybrid.cu share.
#pragma once

#include <cuda_runtime.h>

#include "dsa.h"

namespace dsa {

// Per-device setup of the current device (once per context), and its SM count.
dsa_status hybrid_device(int* num_sms);
// Adds to the calling thread's launch count.
void count_launches(int n);
// Shared-memory limits of the kernels in hybrid.cu; part of the per-device setup.
cudaError_t hybrid_allow_smem();

}  // namespace dsa
