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

// Where a strided tensor lies: `bytes` bytes from `lo` on and, closer, one or more
// ways to see it as rows of `width` bytes, `pitch` bytes apart (cut between any two
// of its axes whose outer strides allow that).  Each way covers all of the tensor,
// so two tensors that are slices of one buffer along any axis (queries and keys of
// one projection) are apart if some pitch shows them in different columns.
struct Region {
  struct Rows {
    int64_t pitch, width;
  };
  uintptr_t lo = 0;
  int64_t bytes = 0;
  Rows rows[3];
  int ways = 0;
};

inline bool regions_overlap(const Region& a, const Region& b) {
  if (a.bytes <= 0 || b.bytes <= 0) return false;
  if (a.lo >= b.lo + (uintptr_t)b.bytes || b.lo >= a.lo + (uintptr_t)a.bytes) return false;
  const Region &x = a.lo <= b.lo ? a : b, &y = a.lo <= b.lo ? b : a;
  for (int i = 0; i < x.ways; ++i)
    for (int j = 0; j < y.ways; ++j) {
      const Region::Rows r = x.rows[i], q = y.rows[j];
      if (r.pitch != q.pitch) continue;
      const int64_t at = (int64_t)((y.lo - x.lo) % (uintptr_t)r.pitch);  // y's first column
      if (at >= r.width && at + q.width <= r.pitch) return false;
    }
  return true;
}

}  // namespace attn
