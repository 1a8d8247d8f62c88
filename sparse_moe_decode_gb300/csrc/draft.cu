// draft.cu -- which tokens of a draft stand, and the one more after them.
//
// A cluster of 8 blocks takes a sequence.  Each finds the first token that is
// not accepted (u q < p as exact products in 64 bits); then the blocks share
// out the row of V weights max(p - q, 0): their sums by segments of 1024, the
// total over the cluster, and the block whose segments hold r * total looks
// for the place in that one segment again.  Bound by memory for many
// sequences (one row of p and q each, read once), by the chain of loads for
// few.  Sums of the weights are pairs of fp32 (48 bits, exact differences),
// added up in 64 bits: the place that r falls into does not depend on the
// order, but for ties within 2^-48 of the total.
#include <cooperative_groups.h>

#include "attn.h"
#include "common.cuh"
#include "early.cuh"

namespace moe {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCluster = 8;
constexpr int kSegment = 1024;
// of one block's share
constexpr int kMaxSegments = (1 << 24) / kSegment / kCluster;

struct DraftShared {
  double seg[kMaxSegments];
  double warp_sum[kWarps];
  double total;  // of the block
  int stop, token, bad;
  int positive;  // last place with a positive weight in a segment
};

// x - y = hi + lo, exactly (Moller, Knuth).
__device__ __forceinline__ void exact_diff(float x, float y, float &hi, float &lo) {
  hi = x - y;
  const float t = hi - x;
  lo = (x - (hi - t)) - (y + t);
}

struct DraftRow {
  const float *p, *q;  // q nullable
  int one;             // the place whose q is 1 where q is null; -1: none
  bool aligned;        // both rows start on 16 bytes

  __device__ __forceinline__ float less(int j) const {
    return q ? q[j] : j == one ? 1.0f : 0.0f;
  }
  __device__ __forceinline__ double weight(int j) const {
    const double w = static_cast<double>(p[j]) - static_cast<double>(less(j));
    return w > 0.0 ? w : 0.0;
  }
};

__device__ __forceinline__ bool usable(float x) { return x >= 0.0f && x < INFINITY; }

// Sum of the weights at j0 .. j0 + kSegment - 1 (those below V), one warp.
__device__ __forceinline__ double segment_sum(const DraftRow &row, int64_t j0, int V, int lane,
                                              bool &bad) {
  float hi = 0.0f, lo = 0.0f;
  const auto add = [&](float p, float q) {
    bad |= !usable(p) | !usable(q);
    float d, e;
    exact_diff(p, q, d, e);
    if (!(d > 0.0f)) d = e = 0.0f;  // (a difference that rounds to 0 is 0)
    const float s = hi + d, t = s - hi;
    lo += ((hi - (s - t)) + (d - t)) + e;
    hi = s;
  };
  if (row.aligned && j0 + kSegment <= V) {
    float4 p[kSegment / 128], q[kSegment / 128];
#pragma unroll
    for (int i = 0; i < kSegment / 128; ++i) {
      const int64_t j = j0 + i * 128 + lane * 4;
      p[i] = __ldg(reinterpret_cast<const float4 *>(row.p + j));
      if (row.q) q[i] = __ldg(reinterpret_cast<const float4 *>(row.q + j));
      else
        q[i] = make_float4(row.less(j), row.less(j + 1), row.less(j + 2), row.less(j + 3));
    }
#pragma unroll
    for (int i = 0; i < kSegment / 128; ++i) {
      add(p[i].x, q[i].x), add(p[i].y, q[i].y), add(p[i].z, q[i].z), add(p[i].w, q[i].w);
    }
  } else {
#pragma unroll 8
    for (int i = 0; i < kSegment / 32; ++i) {
      const int64_t j = j0 + i * 32 + lane;
      if (j < V) add(row.p[j], row.less(static_cast<int>(j)));
    }
  }
  double s = static_cast<double>(hi) + static_cast<double>(lo);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  return s;
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
verify_draft_kernel(const DraftArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  DraftShared *sh = reinterpret_cast<DraftShared *>(smem);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int b = blockIdx.x / kCluster;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  early_begin();
  const int32_t *drafted = a.draft_tokens + static_cast<int64_t>(b) * a.T;
  const float *u = a.uniform + static_cast<int64_t>(b) * (a.T + 1);
  if (warp == 0) {
    int stop = a.T, token = -1;
    for (int i0 = 0; i0 < a.T; i0 += 32) {
      const int i = i0 + lane;
      int d = -1;
      bool stands = true;
      if (i < a.T) {
        d = drafted[i];
        stands = false;
        if (d >= 0 && d < a.V) {
          const float p = a.target[b * a.target_seq_ld + i * a.target_ld + d];
          const float q = a.draft ? a.draft[b * a.draft_seq_ld + i * a.draft_ld + d] : 1.0f;
          stands = static_cast<double>(u[i]) * static_cast<double>(q) < static_cast<double>(p);
        }
      }
      const unsigned fell = __ballot_sync(0xFFFFFFFFu, !stands);
      if (fell) {
        const int first = __ffs(fell) - 1;
        stop = i0 + first;
        token = __shfl_sync(0xFFFFFFFFu, d, first);
        break;
      }
    }
    if (lane == 0) sh->stop = stop, sh->token = token, sh->bad = 0;
  }
  __syncthreads();
  const int stop = sh->stop, token = sh->token;
  const bool outside = token >= a.V;  // not a token
  int32_t *out = a.tokens + static_cast<int64_t>(b) * (a.T + 1);
  if (outside) {  // (all blocks of the cluster)
    if (rank == 0) {
      for (int i = tid; i <= a.T; i += kThreads) out[i] = -1;
      if (tid == 0) {
        a.accepted[b] = 0;
        set_status(a.status, MOE_DEV_BAD_INDEX);
      }
    }
    return;
  }
  DraftRow row;
  row.p = a.target + b * a.target_seq_ld + stop * a.target_ld;
  row.q = nullptr, row.one = -1;
  if (token >= 0) {
    if (a.draft) row.q = a.draft + b * a.draft_seq_ld + stop * a.draft_ld;
    else row.one = token;
  }
  const int all = static_cast<int>((static_cast<int64_t>(a.V) + kSegment - 1) / kSegment);
  const int per = (all + kCluster - 1) / kCluster;
  const int seg0 = rank * per, segs = min(per, all - seg0);  // may be below 0
  double total = 0.0, before = 0.0;
  bool any_bad = false;
  int last_rank = 0;  // that has any weight
  for (int round = 0; round < 2; ++round) {
    row.aligned = (reinterpret_cast<uintptr_t>(row.p) | reinterpret_cast<uintptr_t>(row.q)) % 16 == 0;
    bool bad = false;
    for (int s = warp; s < segs; s += kWarps) {
      const double v =
          segment_sum(row, static_cast<int64_t>(seg0 + s) * kSegment, a.V, lane, bad);
      if (lane == 0) sh->seg[s] = v;
    }
    if (bad) sh->bad = 1;
    __syncthreads();
    if (warp == 0) {
      double sum = 0.0;
      for (int s = lane; s < segs; s += 32) sum += sh->seg[s];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      if (lane == 0) sh->total = sum;
    }
    cluster.sync();
    total = before = 0.0;
    for (int k = 0; k < kCluster; ++k) {
      const DraftShared *other = cluster.map_shared_rank(sh, k);
      if (k == rank) before = total;
      total += other->total;
      if (other->total > 0.0) last_rank = k;
      any_bad |= other->bad != 0;
    }
    cluster.sync();  // nobody's sums change or end before all have read them
    // p never exceeds q: p itself
    if (any_bad || total > 0.0 || (!row.q && row.one < 0)) break;
    row.q = nullptr, row.one = -1;
  }
  if (any_bad || !(total > 0.0)) {
    if (rank == 0) {
      for (int i = tid; i <= a.T; i += kThreads) out[i] = -1;
      if (tid == 0) {
        a.accepted[b] = 0;
        set_status(a.status, MOE_DEV_NONFINITE);
      }
    }
    return;
  }
  if (rank == 0) {
    for (int i = tid; i <= a.T; i += kThreads)
      if (i != stop) out[i] = i < stop ? drafted[i] : -1;
    if (tid == 0) a.accepted[b] = stop;
  }
  // The block whose weights hold the aim, or (the aim rounded up to the total)
  // the last one that has any.
  const double aim = static_cast<double>(u[a.T]) * total, mine = sh->total;
  if (aim < total ? aim < before || !(aim < before + mine) : rank != last_rank) return;
  // The segment: the first whose running sum passes the aim, else the last
  // with any weight (all threads do the same).
  double run = before, start = before;
  int found = -1;
  for (int s = 0; s < segs; ++s) {
    const double v = sh->seg[s];
    if (v > 0.0) {
      found = s, start = run;
      run += v;
      if (run > aim) break;
    }
  }
  if (found < 0) return;
  // Its weights in order: four to a thread.
  const int64_t j0 = static_cast<int64_t>(seg0 + found) * kSegment + tid * 4;
  double w[4], sum = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = j0 + i < a.V ? row.weight(static_cast<int>(j0 + i)) : 0.0;
    sum += w[i];
  }
  double incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double n = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) sh->warp_sum[warp] = incl;
  if (tid == 0) sh->stop = INT32_MAX, sh->positive = -1;
  __syncthreads();
  double c = start;
  for (int k = 0; k < warp; ++k) c += sh->warp_sum[k];
  c += incl - sum;
  int hit = INT32_MAX, last = -1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c += w[i];
    if (w[i] > 0.0) {
      last = static_cast<int>(j0) + i;
      if (c > aim && hit == INT32_MAX) hit = last;
    }
  }
  if (hit != INT32_MAX) atomicMin(&sh->stop, hit);
  if (last >= 0) atomicMax(&sh->positive, last);
  __syncthreads();
  // (sums in another order may end a rounding short of the aim)
  if (tid == 0) out[stop] = sh->stop != INT32_MAX ? sh->stop : sh->positive;
}

}  // namespace

cudaError_t launch_verify_draft(const DraftArgs &a, cudaStream_t s) {
  // (the segments' sums come first: no more of them than the rows have)
  return launch_early(verify_draft_kernel, dim3(a.B * kCluster), kThreads, sizeof(DraftShared), s,
                      a);
}

}  // namespace moe
