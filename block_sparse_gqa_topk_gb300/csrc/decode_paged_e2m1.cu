// decode_paged_e2m1.cu -- the kernels of decode_paged.cuh over 4-bit caches.
#include "decode_paged.cuh"

namespace msa {

cudaError_t launch_decode_e2m1(const PagedDecode& p, int d, int d_idx, cudaStream_t stream) {
  return d == 128 ? launch_kind<128, MSA_CACHE_E2M1>(p, d_idx, stream)
                  : launch_kind<64, MSA_CACHE_E2M1>(p, d_idx, stream);
}

}  // namespace msa
