// delta_seq.cuh -- where a sequence's tokens and state lie (device side).
#pragma once

#include "common.cuh"
#include "mixer.h"

namespace moe {

struct DeltaSeqRange {
  int start, len, slot;
  bool ok;
};

// Sequence b's rows and slot; not ok (nothing of it may be touched) when its
// slot is negative, or when its bounds or slot are out of range, which also
// sets MOE_DEV_BAD_INDEX.
__device__ __forceinline__ DeltaSeqRange delta_seq_range(const DeltaSeqs &s, int b) {
  DeltaSeqRange r;
  r.slot = s.slots ? s.slots[b] : b;
  if (s.cu_seqlens) {
    const int lo = s.cu_seqlens[b], hi = s.cu_seqlens[b + 1];
    r.ok = lo >= 0 && lo <= hi && hi <= s.N;
    r.start = lo;
    r.len = r.ok ? hi - lo : 0;
  } else {
    r.ok = true;
    r.start = b * s.T;
    r.len = s.T;
  }
  if (!r.ok || r.slot >= s.n_slots) {
    r.ok = false;
    set_status(s.status, MOE_DEV_BAD_INDEX);
  }
  if (r.slot < 0) r.ok = false;
  return r;
}

// The decay's logarithm as the kernels take it: exp(-128) is 0 in fp32, so
// nothing changes below that, and sums of clamped values stay finite.  NaN
// passes.
__device__ __forceinline__ float delta_log_decay(float g) { return g < -128.0f ? -128.0f : g; }

}  // namespace moe
