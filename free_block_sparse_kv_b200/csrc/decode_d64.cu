// Decode kernels of head dimension 64.
#include "decode.cuh"

namespace sa {

cudaError_t run_decode_d64(const DecodeArgs& p, cudaStream_t st, size_t* bytes,
                            bool* no_work) {
  return run_decode<64>(p, st, bytes, no_work);
}

}  // namespace sa
