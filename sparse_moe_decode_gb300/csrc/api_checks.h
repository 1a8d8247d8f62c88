// api_checks.h -- argument checks that the C entry points share (internal).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_gb300.h"

namespace moe {

constexpr int64_t kMaxStride = int64_t(1) << 31;  // elements: offsets stay far inside 63 bits

inline bool aligned(const void *p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline bool ptr_ok(const void *p, uintptr_t a = 16) { return p != nullptr && aligned(p, a); }
inline bool opt_ok(const void *p, uintptr_t a = 16) { return p == nullptr || aligned(p, a); }

// Rows of `w` elements of `size` bytes, `ld` elements apart.
struct Span {
  const void *p;
  int64_t rows, w, ld;
  int size;
};

inline bool overlap(const Span &a, const Span &b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t ea = pa + static_cast<uintptr_t>((a.rows - 1) * a.ld + a.w) * a.size;
  const uintptr_t eb = pb + static_cast<uintptr_t>((b.rows - 1) * b.ld + b.w) * b.size;
  if (pa >= eb || pb >= ea) return false;
  // columns of one buffer: equal strides keep them apart in every row
  const uintptr_t ld = static_cast<uintptr_t>(a.ld) * a.size;
  if (ld == 0 || ld != static_cast<uintptr_t>(b.ld) * b.size) return true;
  const uintptr_t d = (pb >= pa) ? (pb - pa) % ld : (ld - (pa - pb) % ld) % ld;
  return d < static_cast<uintptr_t>(a.w) * a.size ||
         ld - d < static_cast<uintptr_t>(b.w) * b.size;
}

inline bool stride_ok(int64_t ld, int64_t least, int64_t multiple) {
  return ld >= least && ld <= kMaxStride && ld % multiple == 0;
}

inline moe_status check_ws(const void *ws, size_t ws_bytes, size_t need) {
  if (!ptr_ok(ws, 256)) return MOE_ERR_INVALID_ARG;
  return ws_bytes < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

inline moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace moe
