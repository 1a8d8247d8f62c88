// draft.cu -- which tokens of a draft stand, and the one more after them.
//
// A cluster of up to 8 blocks takes a sequence.  Each finds the first token that is
// not accepted (u q < p as exact products in 64 bits); then the blocks share
// out the row of V weights max(p - q, 0): their sums by segments of 512, the
// total over the cluster, and the block whose segments hold r * total looks
// for the place in that one segment again.  Bound by memory for many
// sequences (one row of p and q each, read once), by the chain of loads for
// few.
//
// Weights and sums are pairs of fp32 (differences exact, 48 bits kept): the
// place that r falls into does not depend on the order of the sums, but for
// borders within some 2^-45 of the total.  Adding in 64 bits took longer than
// the loads: a warp's addition occupies the SM for 16 cycles.
#include <cooperative_groups.h>

#include "attn.h"
#include "common.cuh"
#include "early.cuh"
#include "kernels.h"

namespace moe {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCluster = 8;  // at most
constexpr int kSegment = 512;
constexpr int kBlocks = 4;  // an SM

// hi + lo, |lo| at most half a step of hi.
struct Pair {
  float hi, lo;
};

// x - y = hi + lo, exactly (Moller, Knuth).
__device__ __forceinline__ Pair exact_diff(float x, float y) {
  Pair r;
  r.hi = x - y;
  const float t = r.hi - x;
  r.lo = (x - (r.hi - t)) - (y + t);
  return r;
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const float s = a.hi + b.hi, t = s - a.hi;
  const float e = ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo);
  Pair r;
  r.hi = s + e;
  r.lo = e - (r.hi - s);
  return r;
}
__device__ __forceinline__ Pair times(Pair a, float f) {
  const float p = a.hi * f, e = fmaf(a.hi, f, -p) + a.lo * f;
  Pair r;
  r.hi = p + e;
  r.lo = e - (r.hi - p);
  return r;
}
__device__ __forceinline__ bool above(Pair a, Pair b) {
  return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo);
}
__device__ __forceinline__ Pair shuffle_xor(Pair a, int o) {
  return Pair{__shfl_xor_sync(0xFFFFFFFFu, a.hi, o), __shfl_xor_sync(0xFFFFFFFFu, a.lo, o)};
}
// The sum over the lanes up to this one, and over all.
__device__ __forceinline__ Pair scan(Pair a, int lane, Pair &all) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair b{__shfl_up_sync(0xFFFFFFFFu, a.hi, o), __shfl_up_sync(0xFFFFFFFFu, a.lo, o)};
    if (lane >= o) a = add(b, a);
  }
  all = Pair{__shfl_sync(0xFFFFFFFFu, a.hi, 31), __shfl_sync(0xFFFFFFFFu, a.lo, 31)};
  return a;
}

struct DraftShared {
  Pair totals[kCluster];  // of all blocks of the cluster
  uint32_t worst[kCluster];
  uint32_t warp_worst[kWarps];
  Pair warp_sum[kWarps];
  Pair start;  // the sum before the segment of the aim
  int stop, token, found, hit, last;
  // the segments' sums follow
};

struct DraftRow {
  const float *p, *q;  // q nullable
  int one;             // the place whose q is 1 where q is null; -1: none

  __device__ __forceinline__ float less(int64_t j) const {
    return q ? q[j] : j == one ? 1.0f : 0.0f;
  }
};

__device__ __forceinline__ Pair weight(float p, float q) {
  Pair d = exact_diff(p, q);
  if (!(d.hi > 0.0f)) d.hi = d.lo = 0.0f;  // (a difference that rounds to 0 is 0)
  return d;
}

// A block's values of one segment, 16 a lane.
struct Segment {
  float4 p[kSegment / 128], q[kSegment / 128];

  __device__ __forceinline__ void load(const DraftRow &row, int64_t j0, int V, int lane,
                                       bool aligned) {
#pragma unroll
    for (int i = 0; i < kSegment / 128; ++i) {
      const int64_t j = j0 + i * 128 + lane * 4;
      if (aligned && j + 4 <= V) {
        p[i] = __ldg(reinterpret_cast<const float4 *>(row.p + j));
        q[i] = row.q ? __ldg(reinterpret_cast<const float4 *>(row.q + j))
                     : make_float4(row.less(j), row.less(j + 1), row.less(j + 2), row.less(j + 3));
      } else {
        float a[4], b[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          a[k] = j + k < V ? __ldg(row.p + j + k) : 0.0f;
          b[k] = j + k < V ? row.less(j + k) : 0.0f;
        }
        p[i] = make_float4(a[0], a[1], a[2], a[3]);
        q[i] = make_float4(b[0], b[1], b[2], b[3]);
      }
    }
  }
  // The lane's weights' sum; `worst`: the largest bits of a value, above all
  // finite positive ones' where one is negative, infinite or NaN.
  __device__ __forceinline__ Pair sum(uint32_t &worst) const {
    Pair s{0.0f, 0.0f};
    const auto one = [&](float x, float y) {
      // (-0 + 0 = 0)
      worst = max(worst, max(__float_as_uint(x + 0.0f), __float_as_uint(y + 0.0f)));
      const Pair d = weight(x, y);
      const float t = s.hi + d.hi, u = t - s.hi;
      s.lo += ((s.hi - (t - u)) + (d.hi - u)) + d.lo;
      s.hi = t;
    };
#pragma unroll
    for (int i = 0; i < kSegment / 128; ++i) {
      one(p[i].x, q[i].x), one(p[i].y, q[i].y), one(p[i].z, q[i].z), one(p[i].w, q[i].w);
    }
    return add(Pair{s.hi, 0.0f}, Pair{s.lo, 0.0f});
  }
};

__global__ void __launch_bounds__(kThreads, kBlocks)
verify_draft_kernel(const DraftArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  DraftShared *sh = reinterpret_cast<DraftShared *>(smem);
  Pair *seg = reinterpret_cast<Pair *>(sh + 1);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int cluster_size = static_cast<int>(cluster.num_blocks());
  const int b = blockIdx.x / cluster_size;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  early_begin();
  // (no block writes to another's shared memory before that one is there)
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  const auto all_here = [] { asm volatile("barrier.cluster.wait;" ::: "memory"); };
  const int32_t *drafted = a.draft_tokens + static_cast<int64_t>(b) * a.T;
  const float *u = a.uniform + static_cast<int64_t>(b) * (a.T + 1);
  const float r = fmaxf(u[a.T], 0.0f);  // (a NaN is 0; from 1 on the last weight is taken)
  if (warp == 0) {
    int stop = a.T, token = -1;
    for (int i0 = 0; i0 < a.T; i0 += 32) {
      const int i = i0 + lane;
      int d = -1;
      bool stands = true;
      if (i < a.T) {
        d = drafted[i];
        const float ui = u[i];
        stands = false;
        if (d >= 0 && d < a.V) {
          const float p = a.target[b * a.target_seq_ld + i * a.target_ld + d];
          const float q = a.draft ? a.draft[b * a.draft_seq_ld + i * a.draft_ld + d] : 1.0f;
          stands = static_cast<double>(ui) * static_cast<double>(q) < static_cast<double>(p);
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
    if (lane == 0) sh->stop = stop, sh->token = token, sh->found = -1;
  }
  __syncthreads();
  const int stop = sh->stop, token = sh->token;
  int32_t *out = a.tokens + static_cast<int64_t>(b) * (a.T + 1);
  const auto refuse = [&](uint32_t bits) {
    if (rank == 0) {
      for (int i = tid; i <= a.T; i += kThreads) out[i] = -1;
      if (tid == 0) {
        a.accepted[b] = 0;
        set_status(a.status, bits);
      }
    }
  };
  if (token >= a.V) {  // not a token (all blocks of the cluster)
    all_here();
    refuse(MOE_DEV_BAD_INDEX);
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
  const int per = (all + cluster_size - 1) / cluster_size;
  const int seg0 = rank * per, segs = max(0, min(per, all - seg0));
  Pair total, before, mine;
  uint32_t worst = 0;
  int last_rank = 0;  // that has any weight
  for (int round = 0; round < 2; ++round) {
    const bool aligned =
        (reinterpret_cast<uintptr_t>(row.p) | reinterpret_cast<uintptr_t>(row.q)) % 16 == 0;
    uint32_t bits = 0;
    Pair part{0.0f, 0.0f};  // of this warp's segments
    for (int s = warp; s < segs; s += kWarps) {
      Segment now;
      now.load(row, static_cast<int64_t>(seg0 + s) * kSegment, a.V, lane, aligned);
      Pair v = now.sum(bits);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v = add(v, shuffle_xor(v, o));
      if (lane == 0) seg[s] = v;
      part = add(part, v);
    }
    bits = __reduce_max_sync(0xFFFFFFFFu, bits);
    if (lane == 0) sh->warp_worst[warp] = bits, sh->warp_sum[warp] = part;
    __syncthreads();
    if (round == 0) all_here();
    if (tid < cluster_size) {  // every block hears of every other's
      Pair t = sh->warp_sum[0];
      uint32_t x = sh->warp_worst[0];
      for (int k = 1; k < kWarps; ++k) {
        t = add(t, sh->warp_sum[k]);
        x = max(x, sh->warp_worst[k]);
      }
      DraftShared *other = cluster.map_shared_rank(sh, tid);
      other->totals[rank] = t;
      other->worst[rank] = x;
    }
    cluster.sync();
    total = before = Pair{0.0f, 0.0f};
    for (int k = 0; k < cluster_size; ++k) {
      const Pair t = sh->totals[k];
      if (k == rank) before = total;
      total = add(total, t);
      worst = max(worst, sh->worst[k]);
      if (t.hi > 0.0f) last_rank = k;
    }
    mine = add(before, sh->totals[rank]);
    // p never exceeds q: p itself
    if (worst >= 0x7F800000u || total.hi > 0.0f || (!row.q && row.one < 0)) break;
    cluster.sync();  // all have read
    row.q = nullptr, row.one = -1;
  }
  // (a block may end: its last remote store was before the barrier)
  if (worst >= 0x7F800000u || !(total.hi > 0.0f && total.hi < INFINITY)) {
    refuse(MOE_DEV_NONFINITE);
    return;
  }
  if (rank == 0) {
    for (int i = tid; i <= a.T; i += kThreads)
      if (i != stop) out[i] = i < stop ? drafted[i] : -1;
    if (tid == 0) a.accepted[b] = stop;
  }
  // The block whose weights hold the aim, or (the aim rounded up to the total)
  // the last one that has any.
  const Pair aim = times(total, r);
  if (above(total, aim) ? above(before, aim) || !above(mine, aim) : rank != last_rank) return;
  // The segment: the first whose running sum is above the aim, else the last
  // with any weight.
  if (warp == 0) {
    Pair run = before, start = before;
    int found = -1;
    for (int s0 = 0; s0 < segs; s0 += 32) {
      const Pair v = s0 + lane < segs ? seg[s0 + lane] : Pair{0.0f, 0.0f};
      Pair sum;
      const Pair to = add(run, scan(v, lane, sum));
      const unsigned some = __ballot_sync(0xFFFFFFFFu, v.hi > 0.0f);
      const unsigned over = __ballot_sync(0xFFFFFFFFu, v.hi > 0.0f && above(to, aim));
      if (some) {
        const int l = over ? __ffs(over) - 1 : 31 - __clz(some);
        found = s0 + l;
        // the sum before it: up to the lane before
        const Pair prev{__shfl_sync(0xFFFFFFFFu, to.hi, max(l - 1, 0)),
                        __shfl_sync(0xFFFFFFFFu, to.lo, max(l - 1, 0))};
        start = l > 0 ? prev : run;
      }
      if (over) break;
      run = add(run, sum);
    }
    if (lane == 0) sh->found = found, sh->start = start, sh->hit = INT32_MAX, sh->last = -1;
  }
  __syncthreads();
  if (sh->found < 0) return;
  // Its weights in order: two to a thread.
  const int64_t j0 = static_cast<int64_t>(seg0 + sh->found) * kSegment + tid * 2;
  Pair w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = j0 + i < a.V ? weight(row.p[j0 + i], row.less(j0 + i)) : Pair{0.0f, 0.0f};
  Pair sum;
  const Pair both = add(w[0], w[1]);
  Pair c = scan(both, lane, sum);
  if (lane == 31) sh->warp_sum[warp] = c;
  c = Pair{__shfl_up_sync(0xFFFFFFFFu, c.hi, 1), __shfl_up_sync(0xFFFFFFFFu, c.lo, 1)};
  if (lane == 0) c = Pair{0.0f, 0.0f};
  __syncthreads();
  Pair base = sh->start;
  for (int k = 0; k < warp; ++k) base = add(base, sh->warp_sum[k]);
  c = add(base, c);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    c = add(c, w[i]);
    if (w[i].hi > 0.0f) {
      atomicMax(&sh->last, static_cast<int>(j0) + i);
      if (above(c, aim)) atomicMin(&sh->hit, static_cast<int>(j0) + i);
    }
  }
  __syncthreads();
  // (sums in another order may end a rounding short of the aim)
  if (tid == 0) out[stop] = sh->hit != INT32_MAX ? sh->hit : sh->last;
}

}  // namespace

cudaError_t launch_verify_draft(const DraftArgs &a, cudaStream_t s) {
  // As many blocks a sequence as all run at once (128 sequences in clusters of 4
  // take 36.6 us, of 8 in two rounds 38.1), as far as a block has room for its
  // segments' sums.
  const int64_t room = static_cast<int64_t>(tc_sm_count()) * kBlocks;
  const int all = (a.V - 1) / kSegment + 1;
  const auto smem_of = [&](int c) { return sizeof(DraftShared) + (all + c - 1) / c * sizeof(Pair); };
  int cluster = kCluster;
  while (cluster > 1 && a.B * static_cast<int64_t>(cluster) > room &&
         smem_of(cluster / 2) <= 48 * 1024)
    cluster /= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_of(cluster);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_draft_kernel, a);
}

}  // namespace moe
