// hybrid.h - what dsa.cu and hybrid.cu share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "dsa.h"

namespace dsa {

// Per-device setup of the current device (once per context): its SM count and the address of
// its status word.
struct HybridDevice {
  int num_sms;
  int* status;
};
dsa_status hybrid_device(HybridDevice* out);
// TMA map of bf16 rows: `width` elements each, `stride` elements apart; boxes of box_cols x
// box_rows, swizzled over the 64 or 128 bytes of a box row.
dsa_status make_row_map(CUtensorMap* map, const void* base, int64_t rows, int64_t width,
                        int64_t stride, int box_cols, int box_rows);
// Adds to the calling thread's launch count.
void count_launches(int n);
// Shared-memory limits of the kernels in hybrid.cu; part of the per-device setup.
cudaError_t hybrid_allow_smem();

}  // namespace dsa
