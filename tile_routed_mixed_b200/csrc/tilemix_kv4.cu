// Kernels of the paged 4-bit K/V cache (sm_100a): the page plan, rows in and
// out, and attention.  One translation unit: they share a device status word.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "tilemix.h"
#include "tilemix_internal.h"
#include "tilemix_kv4.h"
#include "tilemix_mma.cuh"
#include "tilemix_ptx.cuh"

namespace tilemix {

// Latched device status of the paged cache's calls (kStatusBadPages); read and
// cleared by tilemix_get_error() beside the attention kernels' word.
__device__ unsigned int g_kv4_status;

int kv4_read_and_clear_status(unsigned int* status) {
  unsigned int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_kv4_status, sizeof(v));
  if (e != cudaSuccess) return static_cast<int>(e);
  const unsigned int zero = 0;
  if (v != 0) e = cudaMemcpyToSymbol(g_kv4_status, &zero, sizeof(zero));
  *status = v;
  return static_cast<int>(e);
}

}  // namespace tilemix

#include "tilemix_kv4_plan.cuh"
#include "tilemix_kv4_rows.cuh"
#include "tilemix_kv4_attn.cuh"
