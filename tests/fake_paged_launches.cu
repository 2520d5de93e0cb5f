// The launches of the rotary and paged-cache operators as host code, beside fake_cuda_runtime.cpp.
#include <cstring>

#include "spa_paged.cuh"

namespace spa {
static char last[512];
int set_last_error(int code, const char* msg) {
  std::strncpy(last, msg, sizeof last - 1);
  return code;
}
cudaError_t launch_rope(const void*, void*, Strides3, Strides3, const int64_t*, const int64_t*, int, int, int, int, int, int,
                        const RopeTabAny&, cudaStream_t) {
  return cudaSuccess;
}
// An append that finds a position out of range.
cudaError_t launch_page_append(const PagePool& pool, AppendArgs, int, int, const RopeTab128&, int, cudaStream_t) {
  *pool.err |= kErrStartPos;
  return cudaSuccess;
}
cudaError_t launch_page_read(const PagePool&, const ReadArgs&, int, int, cudaStream_t) { return cudaSuccess; }
int page_attend_setup(int) { return 1; }
cudaError_t launch_page_attend(const PagedAttendArgs&, int, int, const RopeTab128&, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_clear_bits(unsigned* word, unsigned bits, cudaStream_t) {
  *word &= ~bits;
  return cudaSuccess;
}
}  // namespace spa

extern "C" const char* fake_last_error() { return spa::last; }
