// Decode kernels of head dimension 128.
#include "decode.cuh"

namespace sa {

cudaError_t run_decode_d128(const DecodeArgs& p, cudaStream_t st, size_t* bytes,
                             bool* no_work) {
  return run_decode<128>(p, st, bytes, no_work);
}

}  // namespace sa
