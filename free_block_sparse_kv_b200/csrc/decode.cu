// Choice of the decode kernels by head dimension (a file of instances each, to compile side
// by side).
#include "launch.h"

namespace sa {

cudaError_t run_decode_d64(const DecodeArgs& p, cudaStream_t st, size_t* bytes, bool* no_work);
cudaError_t run_decode_d128(const DecodeArgs& p, cudaStream_t st, size_t* bytes, bool* no_work);

cudaError_t decode_work_bytes(const DecodeArgs& p, size_t* bytes) {
  return p.c.d == 64 ? run_decode_d64(p, nullptr, bytes, nullptr)
                     : run_decode_d128(p, nullptr, bytes, nullptr);
}

cudaError_t launch_decode(const DecodeArgs& p, cudaStream_t st, bool* no_work) {
  return p.c.d == 64 ? run_decode_d64(p, st, nullptr, no_work)
                     : run_decode_d128(p, st, nullptr, no_work);
}

}  // namespace sa
