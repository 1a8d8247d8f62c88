// attn_sched.cuh -- how the attention kernels share out a batch, from lengths
// that only the device knows.
//
// A tile is R consecutive rows of one sequence and key/value head, a row being
// a (token, head of the group) pair; its work is the KT-wide key tiles that
// any of its rows sees.  All tiles' key tiles, one after another (sequence,
// head, tile, key tile), are cut into equal shares, one for each block; a
// share's pieces are segments of one tile each.  A tile counts C key tiles more
// than it has, for what beginning and ending it costs.  A tile that lies in one share
// is finished there; otherwise its segments leave unnormalised sums (and the
// softmax's maximum and total) for attn_combine_kernel.  Every block finds its
// share by itself: a scan over the sequences, whose key tiles have a closed
// form.
#pragma once

#include "attn.h"
#include "common.cuh"

namespace moe {

struct AttnSeq {
  int start, n, len;  // rows start .. start + n - 1, len positions; n == 0: skipped
};

// One thread of the grid says so for each sequence that is out of range.
__device__ __forceinline__ AttnSeq attn_seq(const AttnBatch &a, int b, bool report) {
  AttnSeq s;
  int end;
  if (a.cu) {
    s.start = a.cu[b], end = a.cu[b + 1];
  } else {
    s.start = b * a.T, end = s.start + a.T;
  }
  s.len = a.lens[b];
  const bool bounds = s.start >= 0 && s.start <= end && end <= a.N;
  s.n = bounds ? end - s.start : 0;
  const bool bad = !bounds || (s.n > 0 && s.len > 0 &&
                               (s.len < s.n || s.len > (static_cast<int64_t>(a.cols) << a.page_shift)));
  if (bad && report) set_status(a.status, MOE_DEV_BAD_INDEX);
  if (bad || s.len <= 0) s.n = 0;
  return s;
}

// (Out of line: code that runs once costs its way through the instruction caches.)
static __device__ __noinline__ uint64_t div_wide(uint64_t x, uint64_t m) { return x / m; }

// x / m and x % m; divisions of 64 bits take several times as long.
__device__ __forceinline__ uint64_t div_mod(uint64_t x, uint32_t m, uint32_t &rest) {
  if ((x >> 32) == 0) {
    const uint32_t d = static_cast<uint32_t>(x) / m;
    rest = static_cast<uint32_t>(x) - d * m;
    return d;
  }
  const uint64_t d = div_wide(x, m);
  rest = static_cast<uint32_t>(x - d * m);
  return d;
}

// sum over i < n of floor((a i + b) / m), m > 0 (Euclid's steps).
static __device__ __noinline__ int64_t floor_sum(uint64_t n, uint32_t m, uint64_t a, uint64_t b) {
  uint64_t sum = 0;
  while (n > 0) {
    uint32_t ra, rb;
    const uint64_t da = div_mod(a, m, ra), db = div_mod(b, m, rb);
    sum += da * (n * (n - 1) / 2) + db * n;
    const uint64_t top = ra * n + rb;
    if (top < m) break;
    n = div_mod(top, m, rb);
    b = rb;
    a = m, m = ra;
  }
  return static_cast<int64_t>(sum);
}

// The tiles of one sequence and head.  A tile's keys end behind its last
// row's position and begin, under a window, with its first row's first key.
template <int R, int KT, int C>
struct AttnTiles {
  int ctx, len, group, window, count;
  int rows;  // at most 2^20 tokens of 64 heads

  __device__ __forceinline__ AttnTiles() {}
  __device__ __forceinline__ AttnTiles(const AttnSeq &s, int group_, int window_)
      : ctx(s.len - s.n), len(s.len), group(group_), window(window_) {
    rows = s.n * group;
    count = (rows + R - 1) / R;
  }
  // (ctx + row / group) / KT = (ctx * group + row) / (KT * group), both floors
  __device__ __forceinline__ int hi(int t) const {
    if (t + 1 >= count) return (len - 1) / KT + 1;
    uint32_t rest;
    return static_cast<int>(div_mod(static_cast<int64_t>(ctx) * group + (t + 1LL) * R - 1,
                                    KT * group, rest)) + 1;
  }
  __device__ __forceinline__ int lo(int t) const {
    if (!window) return 0;
    const int64_t x = (static_cast<int64_t>(ctx) - window + 1) * group + static_cast<int64_t>(t) * R;
    uint32_t rest;
    return x <= 0 ? 0 : static_cast<int>(div_mod(x, KT * group, rest));
  }
  // units (key tiles, and C a tile) of the tiles before t
  __device__ __forceinline__ int64_t before(int t) const {
    if (t == 0) return 0;
    if (count == 1) return hi(0) - lo(0) + C;
    const uint32_t m = KT * group;
    const int n = t < count ? t : count - 1;
    int64_t sum = floor_sum(n, m, R, static_cast<int64_t>(ctx) * group + R - 1) + n +
                  static_cast<int64_t>(C) * t;
    if (t == count) sum += hi(count - 1);
    if (window) {
      const int64_t x0 = (static_cast<int64_t>(ctx) - window + 1) * group;
      const int64_t i0 = x0 >= 0 ? 0 : (-x0 + R - 1) / R;
      if (t > i0) sum -= floor_sum(t - i0, m, R, x0 + i0 * R);
    }
    return sum;
  }
};

// What a block leaves for attn_combine_kernel about the tile that it began and
// did not finish.
struct AttnOpen {
  int32_t last;            // the block that finishes it; -1: there is none
  int32_t rows;            // of the tile
  int32_t start, row0;     // the sequence's first token row, the tile's first row
  int32_t head, pad[3];
};

// Token of a tile row and head within its group.
__device__ __forceinline__ int attn_token(const AttnBatch &a, int row) {
  return static_cast<int>((static_cast<uint64_t>(row) * a.group_inverse) >> 32);
}

// The first position whose page the tile with first row `row0` reads: pages that lie
// wholly before its first row's window may have been given back.  In their place come
// zeros: page number a.pages is behind the cache's last row, where a tiled copy fills.
__device__ __forceinline__ int attn_first_read(const AttnBatch &a, int ctx, int row0) {
  if (!a.window) return 0;
  const int first = ctx + attn_token(a, row0) - a.window + 1;
  return first <= 0 ? 0 : first >> a.page_shift << a.page_shift;
}

struct AttnShare {  // in shared memory
  int64_t at, per, total, offset;  // first unit, a share's, all, within the sequence
  int64_t scan[32];
  int64_t each;  // units of one head of the sequence
  AttnSeq s;
  int32_t seq;
};

// Sequences whose rows are in (least, most] take part.
struct AttnRange {
  int32_t least, most;
};

// Units of one head of sequence b, which is given back too.
template <int R, int KT, int C>
__device__ __forceinline__ int64_t attn_units(const AttnBatch &a, const AttnRange &r, int b,
                                              bool report, AttnSeq &s) {
  s = attn_seq(a, b, report);
  const int rows = s.n * a.group;
  if (s.n == 0 || rows <= r.least || rows > r.most) return 0;
  const AttnTiles<R, KT, C> t(s, a.group, a.window);
  return t.before(t.count);
}

// All threads of the block (a multiple of 32, at most 1024): this block's
// share.  seq = -1: nothing to do.
template <int R, int KT, int C>
__device__ __forceinline__ void attn_share(const AttnBatch &a, const AttnRange &r, int least_share,
                                           AttnShare *sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
  AttnSeq s;
  const auto find = [&](int64_t at, int64_t each, int64_t incl, int b) {
    const int64_t first = incl - each * a.kv_heads;
    if (at >= first && at < incl) sh->seq = b, sh->offset = at - first, sh->each = each, sh->s = s;
  };
  const auto share_of = [&](int64_t total) {
    uint32_t rest;
    const int64_t per = div_mod(total + gridDim.x - 1, gridDim.x, rest);
    return per < least_share ? static_cast<int64_t>(least_share) : per;
  };
  // an inclusive scan over the warp
  const auto warp_scan = [&](int64_t v) {
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t n = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += n;
    }
    return v;
  };
  if (tid == 0) sh->seq = -1;
  if (a.B <= 32) {  // one warp does it
    if (warp == 0) {
      __syncwarp();
      const int64_t each =
          lane < a.B ? attn_units<R, KT, C>(a, r, lane, blockIdx.x == 0, s) : 0;
      const int64_t incl = a.B == 1 ? each * a.kv_heads : warp_scan(each * a.kv_heads);
      const int64_t total = __shfl_sync(0xFFFFFFFFu, incl, a.B - 1);
      const int64_t per = share_of(total), at = per * blockIdx.x;
      if (lane == 0) sh->at = at, sh->per = per, sh->total = total;
      if (lane < a.B && at < total) find(at, each, incl, lane);
    }
    __syncthreads();
    return;
  }
  const bool one = a.B <= nt;
  int64_t mine = 0, sum = 0;
  for (int b = tid; b < a.B; b += nt) {
    mine = attn_units<R, KT, C>(a, r, b, blockIdx.x == 0, s);
    sum += mine;
  }
  // over the threads; the total through sh->scan
  const auto scan = [&](int64_t v, int64_t &total) {
    v = warp_scan(v);
    __syncthreads();
    if (lane == 31) sh->scan[warp] = v;
    __syncthreads();
    total = 0;
    for (int w = 0; w < nt / 32; ++w) {
      if (w == warp) v += total;
      total += sh->scan[w];
    }
    return v;
  };
  int64_t total, incl = scan(sum * a.kv_heads, total);
  const int64_t per = share_of(total), at = per * blockIdx.x;
  if (tid == 0) sh->at = at, sh->per = per, sh->total = total;
  __syncthreads();
  if (at >= total) return;
  if (one) {
    if (tid < a.B) find(at, mine, incl, tid);
  } else {
    int64_t base = 0;
    for (int b0 = 0; b0 < a.B && base <= at; b0 += nt) {
      const int b = b0 + tid;
      const int64_t each = b < a.B ? attn_units<R, KT, C>(a, r, b, false, s) : 0;
      int64_t round;
      incl = base + scan(each * a.kv_heads, round);
      if (b < a.B) find(at, each, incl, b);
      base += round;
    }
  }
  __syncthreads();
}

// A block's way through its share, segment by segment.  Every warp walks it
// by itself and sees the same.
template <int R, int KT, int C>
struct AttnWalk {
  int b, head, tile, at, left_in_tile;
  int64_t left, next_unit;  // units left of the share; of all, before the next segment
  AttnSeq s;
  AttnTiles<R, KT, C> t;

  // the current segment (of sequence b and head)
  int cur;            // its tile
  int k0, k1;         // key tiles
  bool begins, ends;  // the tile's first, last
  int64_t tile_end;   // of all units

  __device__ __forceinline__ void init(const AttnBatch &a, const AttnShare &sh) {
    b = sh.seq;
    left = 0;
    if (b < 0) return;
    left = sh.total - sh.at < sh.per ? sh.total - sh.at : sh.per;
    next_unit = sh.at;
    s = sh.s;
    t = AttnTiles<R, KT, C>(s, a.group, a.window);
    int64_t rem = sh.offset;
    head = 0;
    if (rem >= sh.each) {
      if ((sh.each | rem) >> 32) head = static_cast<int>(div_wide(rem, sh.each));
      else head = static_cast<int>(static_cast<uint32_t>(rem) / static_cast<uint32_t>(sh.each));
      rem -= sh.each * head;
    }
    // before(low) <= rem < before(high): the lanes try 32 places at a time
    int low = 0, high = t.count;
    int64_t first = 0;  // before(low)
    const int lane = threadIdx.x & 31;
    while (high - low > 1) {
      const int step = (high - low + 31) / 32, mid = low + step * lane;
      const int64_t there = mid < high ? t.before(mid) : 0;
      const unsigned fits = __ballot_sync(0xFFFFFFFFu, mid < high && there <= rem);
      const int last = 31 - __clz(fits);  // (lane 0's does)
      first = __shfl_sync(0xFFFFFFFFu, there, last);
      low += step * last;
      high = min(high, low + step);
    }
    tile = low;
    at = static_cast<int>(rem - first);
  }
  __device__ __forceinline__ bool next(const AttnBatch &a, const AttnRange &r) {
    if (left <= 0) return false;
    if (tile == t.count) {
      tile = 0;
      if (++head == a.kv_heads) {
        head = 0;
        do {
          if (++b >= a.B) {
            left = 0;
            return false;
          }
          s = attn_seq(a, b, false);
        } while (s.n == 0 || s.n * a.group <= r.least || s.n * a.group > r.most);
        t = AttnTiles<R, KT, C>(s, a.group, a.window);
      }
    }
    if (at < C) {  // the C units come first
      const int skip = C - at < left ? C - at : static_cast<int>(left);
      at += skip, left -= skip, next_unit += skip;
      if (left == 0) return false;
    }
    const int lo = t.lo(tile), whole = t.hi(tile) - lo, done = at - C;
    const int n = whole - done < left ? whole - done : static_cast<int>(left);
    k0 = lo + done, k1 = k0 + n;
    begins = done == 0, ends = done + n == whole;
    tile_end = next_unit + whole - done;
    cur = tile;
    left -= n, next_unit += n;
    if (ends) at = 0, ++tile;
    else at += n;
    return true;
  }
};

}  // namespace moe
