// api.h -- what the translation units that hold C entry points share (defined
// in api.cu): the thread's error string and launch count, the SM count, and
// span checks of plain [.., d] tensors.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/attn.h"

namespace attn {

int num_sms();  // of the current device
void api_begin();  // clears this thread's error string and launch count
attn_status_t api_fail(attn_status_t s, const char* fmt, ...);
// cudaSuccess: adds n to the launch count; otherwise ATTN_ERR_CUDA
attn_status_t api_launched(cudaError_t e, int n, const char* what);

// Where a strided tensor lies: `rows` rows of `width` bytes, `pitch` bytes
// apart, from `lo` on.  Two tensors that are slices of one buffer (queries and
// keys of one projection) have interleaved rows: same pitch, other columns.
struct Region {
  uintptr_t lo = 0;
  int64_t rows = 0, pitch = 0, width = 0;
  uintptr_t hi() const { return rows > 0 ? lo + (uintptr_t)((rows - 1) * pitch + width) : lo; }
};

inline bool regions_overlap(const Region& a, const Region& b) {
  if (a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  if (a.lo >= b.hi() || b.lo >= a.hi()) return false;
  if (a.pitch != b.pitch || a.width > a.pitch || b.width > b.pitch) return true;
  // same pitch: compare the columns, modulo the pitch
  const int64_t d = (int64_t)((a.lo <= b.lo ? b.lo - a.lo : a.lo - b.lo) % (uintptr_t)a.pitch);
  const int64_t w0 = a.lo <= b.lo ? a.width : b.width, w1 = a.lo <= b.lo ? b.width : a.width;
  return d < w0 || d + w1 > a.pitch;
}

}  // namespace attn
