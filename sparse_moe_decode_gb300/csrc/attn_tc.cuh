// attn_tc.cuh -- attention of many rows (prompts, chunks, long drafts): both
// products on the 5th-generation tensor cores.
//
// A tile is R = 128 NQ rows (token, head of the group) of one sequence and
// key/value head: NQ = 2 query tiles of 128 rows where their sums fit tensor
// memory (head_dim <= 128), else one.  Key tiles are 128 keys.  Per key tile
// and query tile
//   S = q k^T       128 x 128, both operands in shared memory,
//   p = 2^(s - m)   by the 128 threads that hold a row of S each,
//   O += p v        p in tensor memory (over S, bf16 or fp16 pairs), v in
//                   shared memory, O in tensor memory (fp32),
// with the running maximum m.  O is brought to a new maximum only when a
// row's grows by more than 2^8 (its exponentials stay far inside fp32 and
// bf16), and the thread that holds the row does it.  While one query tile's
// softmax runs, the other's products do (NQ = 2: the tensor cores have 2048
// cycles of work a key tile and the exponentials half of that); with NQ = 1
// two key tiles' S alternate.
//
// K and V come through a ring of 16 KB units: K 128 keys by 64 columns
// (K-major operand), V as many keys as fill one by all columns (MN-major
// operand: a key's values lie along N).  8-bit codes come through a ring of
// their own and become fp16 code * scale (rounded once) under a power of two a
// key tile, for the values one that only grows within a segment; O follows it.
// Weights are then fp16 under 2^7.  Exact codes, with the scales on S's columns
// and on the weights as the streaming kernel has them, cost the softmax's
// threads more than the conversion: 1370 us for what takes 888 now.
//
// Warps: 4 NQ softmax; 4 (NQ = 2) or 8 that convert; one that fetches; NQ that
// issue products, a query tile each and by turns, so that while one waits for
// its weights the other's products run; one that plans the segments one ahead
// (every warp for itself: 61 us for a prompt of 2048, 52 now) and prepares the scales.
// Registers move from the others to the softmax.  Every wait is bounded (the lanes of a
// warp, converged, wait on one barrier and have one answer; a vote at each wait took 4
// to 11 % more); after one that gave up, all later ones do at once, copies and products
// in flight are waited for, and MOE_DEV_TIMEOUT is set.
//
// Measured, 4096 tokens over 16384, 16 heads on 4, pages of 64 (TFLOP/s of the
// products below the diagonal; 1910 measured for a plain bf16 product):
//   head_dim       64    128    256
//   bf16          895   1520   1355
//   int8          695   1045    780
//   e4m3          710   1085    855
// 64: the exponentials, one for each 4 * 64 operations.  128: tensor cores,
// less the turns' gaps.  256 (one query tile): each K and V is read by 128
// rows, 128 KB a key tile from the L2.  8-bit: the conversion, its
// reads and writes of shared memory beside the products' own.  Short prompts:
// some 8 us from launch to the first product, and the join.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "attn_args.cuh"
#include "delta_mma.cuh"
#include "early.cuh"
#include "sm100_ptx.cuh"

namespace moe {

constexpr int kTcTileCost = 2;  // beginning and ending a tile, in key tiles

template <int D, int KV>
struct TcShape {
  static constexpr bool kBytes = KV != MOE_KV_BF16;
  static constexpr int kNQ = D == 256 ? 1 : 2, kR = 128 * kNQ, kKT = 128;
  static constexpr int kChunks = D / 64;        // 128-byte columns: units of K a tile, and of V
  static constexpr int kVKeys = 128 / kChunks;  // keys of a unit of V
  static constexpr int kUnit = 16384, kRaw = kUnit / 2;
  static constexpr int kQ = kNQ * 128 * D * 2;
  static constexpr int kScaleSlots = 4;
  static constexpr int kScales = kBytes ? kScaleSlots * 256 * 4 : 0;
  static constexpr int kFixed = kQ + kScales + 2048 + kNQ * 512;  // + barriers, row factors
  static constexpr int kRoom = 232448 - kFixed;
  // (With two query tiles room for converted units pays more than for raw ones: 16
  // heads of 128, 4096 over 16384, 8 and 3 slots 461 us, 6 and 7 472; one tile: as long)
  static constexpr int kUnits = kBytes ? kRoom / (kUnit + kRaw) + (kNQ == 2 ? 2 : 0) : kRoom / kUnit;
  static constexpr int kRaws = kBytes ? (kRoom - kUnits * kUnit) / kRaw : 0;
  static constexpr int kSmem = kFixed + kUnits * kUnit + kRaws * kRaw;
  static constexpr int kSoftWarps = 4 * kNQ;
  // (with one query tile each key tile's conversion serves half as many products)
  static constexpr int kConvWarps = !kBytes ? 0 : kNQ == 1 ? 8 : 4;
  static constexpr int kFetchWarp = kSoftWarps + kConvWarps, kMmaWarp = kFetchWarp + 1;
  static constexpr int kPlanWarp = kMmaWarp + kNQ;
  static constexpr int kThreads = 128 * ((kPlanWarp + 4) / 4);  // whole groups of four warps
  static constexpr int kReaders = kSoftWarps + kConvWarps + 1 + kNQ;  // of the plan
  // Registers a thread at launch, and what the softmax's warps and the rest
  // have of them (0: no more than a thread can have anyway).
  static constexpr int kRegs = kThreads == 512 ? 128 : 168;
  static constexpr int kSoftRegs = kThreads == 256 ? 0 : kBytes ? 192 : 216;
  static constexpr int kRestRegs = kNQ == 1 ? 104 : kBytes ? 64 : 72;
  static_assert(kSoftRegs * kSoftWarps + kRestRegs * (kThreads / 32 - kSoftWarps) <=
                    kRegs * (kThreads / 32) || kSoftRegs == 0, "registers");
  static constexpr uint32_t kS = 0, kO = 256;  // columns of tensor memory
  // a key tile's K and the V before it are there together (NQ = 2)
  static_assert(kUnits <= 12 && kRaws <= 12 && kUnits >= (kNQ == 2 ? 2 * kChunks : 5), "ring");
};

// A segment of a tile, as the planning warp hands it to the others.
struct __align__(16) TcSegment {
  int32_t there;           // 0: there is no more
  int32_t b, start, len;   // the sequence, its first row, its positions
  int32_t head, row0, rows, ctx;  // the tile: its first row and rows; positions before the rows'
  int32_t k0, k1;          // key tiles
  int32_t q0[2], q1[2];    // those that query tile i has to do with: q0[i] .. q1[i] - 1
  int32_t begins, last;    // the tile's first segment; the block with its last one, -1: this
  // (selects: an index would put the segment into local memory)
  __device__ __forceinline__ int first(int i) const { return i ? q0[1] : q0[0]; }
  __device__ __forceinline__ int end(int i) const { return i ? q1[1] : q1[0]; }
  __device__ __forceinline__ bool has(int i, int kt) const { return kt >= first(i) && kt < end(i); }
};
static_assert(sizeof(TcSegment) == 64, "segment");

struct TcSmem {
  TcSegment plan[4];
  uint64_t plan_full[4], plan_empty[4];
  uint64_t full[12], empty[12], raw_full[12], raw_empty[12];
  uint64_t scale_raw[4], scale_full[4], scale_empty[4];
  float k_unit[4], v_unit[4];  // what 1 stands for in a key tile's fp16 keys, values
  uint64_t q_raw[2], q_full[2], q_empty[2], s_full[2], p_full[2], o_done[2], o_last[2], turn[2], done;
  AttnShare share;
  uint32_t tmem_holder;
  int abort;
};
static_assert(sizeof(TcSmem) <= 2048, "shared memory");

// Operand descriptors in two words (128-byte swizzle, groups of 8 rows 1024
// bytes apart): the upper is the same for all; the lower is the address / 16
// and, for V, how far on its next 64 columns are.  q and k lie along K; V has
// its N along a row (rows are keys).
constexpr uint32_t kDescUpper = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lower(uint32_t saddr, uint32_t next) {
  return ((saddr & 0x3FFFFu) >> 4) | ((next >> 4) << 16);
}
constexpr uint32_t kIdescTransB = 1u << 16;

// One lane of the warp, the same each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// Four products of K = 16 after one another (one thread).  Issued one by one,
// each with descriptors of its own, they took some 120 cycles each, twice what
// they take to run.
__device__ __forceinline__ void mma_ss4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                        bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t;\n\t.reg .b64 da, db;\n\t.reg .b32 x, y;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t"
      "add.u32 x, %1, 2;\n\tadd.u32 y, %2, 2;\n\t"
      "mov.b64 da, {x, %3};\n\tmov.b64 db, {y, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, t;\n\t"
      "add.u32 x, %1, 4;\n\tadd.u32 y, %2, 4;\n\t"
      "mov.b64 da, {x, %3};\n\tmov.b64 db, {y, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, t;\n\t"
      "add.u32 x, %1, 6;\n\tadd.u32 y, %2, 6;\n\t"
      "mov.b64 da, {x, %3};\n\tmov.b64 db, {y, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, t;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(kDescUpper), "r"(idesc), "r"(accumulate ? 1 : 0)
      : "memory");
}
// Two, A in tensor memory: b and b + 2048 bytes.
__device__ __forceinline__ void mma_ts2(uint32_t d, uint32_t a, uint32_t b, uint32_t b2,
                                        uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t;\n\t.reg .b64 db;\n\t.reg .b32 x;\n\t"
      "setp.ne.b32 p, %6, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
      "mov.b64 db, {%2, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %5, p;\n\t"
      "add.u32 x, %1, 8;\n\tmov.b64 db, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %5, t;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(b2), "r"(kDescUpper), "r"(idesc), "r"(accumulate ? 1 : 0)
      : "memory");
}

__device__ __forceinline__ __half2 bits_h2(uint32_t v) {
  return *reinterpret_cast<const __half2 *>(&v);
}

template <int N>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N > 0 ? N : 24));
}
template <int N>
__device__ __forceinline__ void leave_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

template <int D, int KV>
__global__ void __launch_bounds__((TcShape<D, KV>::kThreads), 1)
attn_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
               const __grid_constant__ CUtensorMap tm_q, const AttnBatch a, const AttnRange range, const AttnArgs p) {
  using S = TcShape<D, KV>;
  constexpr bool kBytes = S::kBytes;
  constexpr int NQ = S::kNQ, R = S::kR, kChunks = S::kChunks, kUnits = S::kUnits;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *q_area = smem;
  uint8_t *ring = q_area + S::kQ;
  uint8_t *raw = ring + kUnits * S::kUnit;
  float *scales = reinterpret_cast<float *>(raw + S::kRaws * S::kRaw);
  float *q_factor = scales + S::kScales / 4;
  TcSmem *sh = reinterpret_cast<TcSmem *>(q_factor + NQ * 128);
  volatile int *abort = &sh->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 12; ++i) {
      ptx::mbar_init(&sh->full[i], kBytes ? S::kConvWarps : 1);
      ptx::mbar_init(&sh->empty[i], NQ);
      ptx::mbar_init(&sh->raw_full[i], 1);
      ptx::mbar_init(&sh->raw_empty[i], S::kConvWarps + (kBytes ? 0 : 1));
    }
    for (int i = 0; i < 4; ++i) {
      ptx::mbar_init(&sh->plan_full[i], 1);
      ptx::mbar_init(&sh->plan_empty[i], S::kReaders);
      ptx::mbar_init(&sh->scale_raw[i], 1);
      ptx::mbar_init(&sh->scale_full[i], 1);
      ptx::mbar_init(&sh->scale_empty[i], S::kSoftWarps + S::kConvWarps);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sh->q_raw[i], 1);
      ptx::mbar_init(&sh->q_full[i], p.q_copy && !kBytes ? 1 : 4);
      ptx::mbar_init(&sh->q_empty[i], 1);
      ptx::mbar_init(&sh->turn[i], 1);
      ptx::mbar_init(&sh->s_full[i], 1);
      ptx::mbar_init(&sh->p_full[i], 4);
      ptx::mbar_init(&sh->o_done[i], 1);
      ptx::mbar_init(&sh->o_last[i], 1);
    }
    ptx::mbar_init(&sh->done, NQ);
    sh->abort = 0;
    ptx::fence_mbar_init();
    ptx::tma_prefetch_desc(&tm_k);
    ptx::tma_prefetch_desc(&tm_v);
  }
  early_begin();
  if (threadIdx.x == 0) p.parts.open[blockIdx.x].last = -1;
  attn_share<R, 128, kTcTileCost>(a, range, p.least_share, &sh->share);
  if (sh->share.seq < 0) return;
  if (warp == S::kMmaWarp) {
    ptx::tmem_alloc(&sh->tmem_holder, 512);
    ptx::tmem_relinquish();
    ptx::tc_fence_before();
  }
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sh->tmem_holder;
  uint32_t seg_n = 0;
  bool ok = true;
  const auto next_segment = [&]() {
    const uint32_t slot = seg_n % 4;
    TcSegment s;
    s.there = 0;
    ok = ok && ptx::mbar_wait(&sh->plan_full[slot], (seg_n / 4) & 1, abort, p.budget);
    if (ok) s = sh->plan[slot];
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&sh->plan_empty[slot]);
    ++seg_n;
    return s;
  };
  const int page = 1 << a.page_shift;
  const int k_box = page < 128 ? page : 128, v_box = page < S::kVKeys ? page : S::kVKeys;

  if (warp < S::kSoftWarps) {  // ------------------------------------ softmax
    if (S::kSoftRegs) take_registers<S::kSoftRegs>();
    const int qi = warp / 4, wq = warp % 4;
    const uint32_t lanes = static_cast<uint32_t>(wq) << 21;  // TMEM lane 32 wq
    const uint32_t o_at = tmem + lanes + S::kO + qi * D;
    const float sign = p.scale_log2 < 0.0f ? -1.0f : 1.0f;
    const float c_all = fabsf(p.scale_log2);
    // 8-bit: weights enter as fp16 of 2^7 times them, 11 bits down to 2^-21
    constexpr float kPower = kBytes ? 7.0f : 0.0f;
    uint32_t items = 0, tiles = 0, segs = 0, q_tiles = 0;
    for (TcSegment w = next_segment(); w.there; w = next_segment()) {
      const int rows = w.rows;
      const int r = qi * 128 + wq * 32 + lane;  // this thread's row of the tile
      const bool live = r < rows;
      const int my_row = w.row0 + (live ? r : rows - 1);
      const int token = attn_token(a, my_row), head = w.head * a.group + my_row - token * a.group;
      const int pos = w.ctx + token;
      const int warp_pos = __shfl_sync(0xFFFFFFFFu, pos, 0);  // the warp's first and last
      const int warp_last = __shfl_sync(0xFFFFFFFFu, pos, 31);
      const bool idle = qi * 128 + wq * 32 >= rows;  // none of the warp's rows is the tile's
      const bool mine = w.first(qi) < w.end(qi);
      float factor = c_all;
      if (kBytes && p.q_copy && mine) {
        // ---- this thread's row of q as it lies in its place, made fp16
        ok = ptx::mbar_wait(&sh->q_raw[qi], q_tiles++ & 1, abort, p.budget);
        if (!ok) break;
        if (!idle) {
          const int row = wq * 32 + lane;
          uint8_t *at = q_area + qi * kChunks * 16384 + row * 128;
          float top = 0.0f;
#pragma unroll 1
          for (int ch = 0; ch < kChunks; ++ch)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint4 x = *reinterpret_cast<const uint4 *>(at + ch * 16384 + ((i ^ (row & 7)) << 4));
              top = max3_abs(max3_abs(top, bf16_lo(x.x), bf16_hi(x.x)), bf16_lo(x.y), bf16_hi(x.y));
              top = max3_abs(max3_abs(top, bf16_lo(x.z), bf16_hi(x.z)), bf16_lo(x.w), bf16_hi(x.w));
            }
          float mult, inv;
          pow2_scale(top, mult, inv);
          factor *= inv;
          mult = c_all == 0.0f ? 0.0f : mult * sign;
          const auto half = [&](uint32_t v) {
            if (c_all == 0.0f) return 0u;  // all scores are 0
            return h2_bits(__floats2half2_rn(bf16_lo(v) * mult, bf16_hi(v) * mult));
          };
#pragma unroll 1
          for (int ch = 0; ch < kChunks; ++ch)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint4 *x = reinterpret_cast<uint4 *>(at + ch * 16384 + ((i ^ (row & 7)) << 4));
              *x = make_uint4(half(x->x), half(x->y), half(x->z), half(x->w));
            }
          ptx::fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh->q_full[qi]);
      } else if (!p.q_copy && mine) {  // ---- this warp's 32 rows of q
        const int64_t q_off = (w.start + token) * p.q_ld + head * D;
        constexpr int kLanes = D / 8, kRows = 32 / kLanes, kBatch = 4;
        const int l16 = lane % kLanes;
        uint8_t *q_dst = q_area + qi * kChunks * 16384 + (l16 >> 3) * 16384;
#pragma unroll 1
        for (int b0 = 0; b0 < 32; b0 += kBatch * kRows) {
          uint4 x[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int rr = b0 + i * kRows + lane / kLanes;
            const int64_t off = __shfl_sync(0xFFFFFFFFu, q_off, rr);
            const bool has = qi * 128 + wq * 32 + rr < rows;
            x[i] = has ? ld_nc(p.q + off + l16 * 8) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int rr = b0 + i * kRows + lane / kLanes;
            uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            if (c_all == 0.0f) v[0] = v[1] = v[2] = v[3] = 0u;  // all scores are 0
            if (kBytes) {
              float top = 0.0f;
#pragma unroll
              for (int j = 0; j < 4; ++j) top = max3_abs(top, bf16_lo(v[j]), bf16_hi(v[j]));
#pragma unroll
              for (int o = kLanes / 2; o > 0; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
              float mult, inv;
              pow2_scale(top, mult, inv);
              if (l16 == 0) q_factor[qi * 128 + wq * 32 + rr] = inv;
              mult *= sign;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                v[j] = h2_bits(__floats2half2_rn(bf16_lo(v[j]) * mult, bf16_hi(v[j]) * mult));
            } else if (sign < 0.0f) {
#pragma unroll
              for (int j = 0; j < 4; ++j) v[j] ^= 0x80008000u;
            }
            const int row = wq * 32 + rr;
            *reinterpret_cast<uint4 *>(q_dst + row * 128 + (((l16 & 7) ^ (row & 7)) << 4)) =
                make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh->q_full[qi]);
        if (kBytes) factor *= q_factor[qi * 128 + wq * 32 + lane];
      }
      if (c_all == 0.0f) factor = 1.0f;
      float m = -INFINITY, l = 0.0f;
      float unit = 1.0f;  // (8-bit) what 1 of O stands for
      bool begun = false;
      for (int kt = w.k0; kt < w.k1 && ok; ++kt) {
        const uint32_t slot = tiles % S::kScaleSlots;
        if (kBytes) {
          ok = ptx::mbar_wait(&sh->scale_full[slot], (tiles / S::kScaleSlots) & 1, abort, p.budget);
          if (!ok) break;
          ++tiles;
        }
        if (w.has(qi, kt)) {
          const int sb = NQ == 2 ? qi : static_cast<int>(items & 1);
          const uint32_t s_at = tmem + lanes + S::kS + sb * 128;
          // 8-bit: kept inside fp32, since -inf times 0 and 0 times inf are NaN.  (Zero rows of q
          // and tiles of zero keys give less than 2^-126: |S| < 2^38, all scores are 0.)  Found
          // before the wait, it costs nothing (behind it 1.5 % with heads of 128).
          const float f_tile =
              kBytes ? fminf(fmaxf(factor * sh->k_unit[slot], 0x1p-126f), 0x1.fffffep127f) : factor;
          ok = ptx::mbar_wait(&sh->s_full[sb], NQ == 2 ? items & 1 : (items >> 1) & 1, abort,
                              p.budget);
          if (!ok) break;
          if (idle) {
            if (lane == 0) {
              ptx::mbar_arrive(&sh->p_full[sb]);
              if (kBytes) ptx::mbar_arrive(&sh->scale_empty[slot]);
            }
            ++items;
            begun = true;
            continue;
          }
          ptx::tc_fence_after();
          float s[128];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            ptx::tmem_ld32(s_at + 32 * i, *reinterpret_cast<float(*)[32]>(s + 32 * i));
          ptx::tmem_wait_ld();
          float o_factor = 1.0f;
          if (kBytes) {  // (powers of two, growing)
            const float now = sh->v_unit[slot];
            if (begun) o_factor = unit * pow2_inverse(now);
            unit = now;
          }
          const int key0 = kt * 128, hi = pos - key0;  // (the row's own position)
          if (key0 + 127 > warp_pos || (a.window && key0 + a.window <= warp_last)) {
            // some row of the warp does not see all of the tile: bits for what it sees
            const int lo = a.window ? hi - a.window + 1 : 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int h = hi - 32 * j, l = lo - 32 * j;
              const uint32_t upto = h >= 31 ? 0xFFFFFFFFu : h < 0 ? 0u : (2u << h) - 1u;
              const uint32_t from = l <= 0 ? 0xFFFFFFFFu : l >= 32 ? 0u : 0xFFFFFFFFu << l;
              const uint32_t sees = upto & from;
#pragma unroll
              for (int i = 0; i < 32; ++i)
                s[32 * j + i] = sees & (1u << i) ? s[32 * j + i] : -INFINITY;
            }
          }
          const auto largest = [&]() {
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 128; i += 8)
#pragma unroll
              for (int j = 0; j < 4; ++j) top[j] = max3(top[j], s[i + 2 * j], s[i + 2 * j + 1]);
            return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * f_tile;
          };
          // p = 2^(s - m) (2^7 of that as fp16) into S's place.  m is the maximum of
          // the tiles before, which nearly always does: only where the tile's total
          // says that m is far too small is it found anew, and the tile done again.
          float total;
          const auto form = [&]() {
            const float b = kPower - (m == -INFINITY ? 0.0f : m);
            const float2 f2 = make_float2(f_tile, f_tile), b2 = make_float2(b, b);
            float2 sum[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] = make_float2(0.0f, 0.0f);
            uint32_t pk[16];
            // in steps, so that the exponentials of 16 keys are on their way together
#pragma unroll
            for (int h = 0; h < 8; ++h) {
              float2 x[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                x[i] = fma2(make_float2(s[16 * h + 2 * i], s[16 * h + 2 * i + 1]), f2, b2);
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i].x = attn_exp2(x[i].x), x[i].y = attn_exp2(x[i].y);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                sum[i & 3] = add2(x[i], sum[i & 3]);
                pk[8 * (h & 1) + i] = kBytes ? h2_bits(__float22half2_rn(x[i]))
                                             : pack_bf16(x[i].x, x[i].y);
              }
              if (h & 1) tmem_st16(s_at + 8 * (h - 1), pk);
            }
            const float2 both = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
            total = both.x + both.y;
            return total > 0x1p15f || m == -INFINITY;
          };
          const auto higher = [&]() {
            const float mt = largest();
            // (by a whole power of two, so that O's factor is exact)
            return m == -INFINITY ? mt : mt > m ? m + ceilf(mt - m) : m;
          };
          // (A comparison that NaN fails: a row whose maximum is NaN raises nothing, and the
          // searches below end however many rows of the warp see nothing.)
          const auto raise = [&](float up) {
            if (up > m) {
              const float f = attn_exp2(m - up);
              l *= f, o_factor *= f;
              m = up;
            }
          };
          // With 8-bit caches one place in the code finds the first maximum and later ones,
          // since the kernel does not fit the instruction caches (4096 over 16384, 16 heads
          // of 128, 485 us with two, 461 with one; with bf16 313 with two, 331 with one).
          // Where no row's has changed there is no more to do: rows that see nothing.
          if (kBytes) {
            bool far = !begun, again = far;
            for (bool first = true;; first = false) {
              if (again) {
                const float up = far ? higher() : m;
                if (!first && !__any_sync(0xFFFFFFFFu, up > m)) break;
                raise(up);
              }
              far = form();
              again = __any_sync(0xFFFFFFFFu, far);
              if (!again) break;
            }
          } else {
            if (!begun) m = largest();
            while (true) {
              const bool far = form();
              if (!__any_sync(0xFFFFFFFFu, far)) break;
              const float up = far ? higher() : m;
              if (!__any_sync(0xFFFFFFFFu, up > m)) break;
              raise(up);
            }
          }
          if (begun && __any_sync(0xFFFFFFFFu, o_factor != 1.0f)) {
            // O's products so far are complete.  (Those before the last are: the
            // scores just read were issued after them.)
            ok = ptx::mbar_wait(&sh->o_done[qi], (items - 1) & 1, abort, p.budget);
            if (!ok) break;
            ptx::tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < D; i += 16) {
              float o[16];
              uint32_t u[16];
              ptx::tmem_ld16(o_at + i, o);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j) u[j] = __float_as_uint(o[j] * o_factor);
              tmem_st16(o_at + i, u);
            }
          }
          l += total;
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sh->p_full[sb]);
          begun = true;
          ++items;
        }
        if (kBytes) {
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&sh->scale_empty[slot]);
        }
      }
      if (!ok) break;
      // ----------------------------------------------- the segment's end
      const bool whole = w.begins && w.last < 0;
      const int part = 2 * blockIdx.x + (w.begins ? 1 : 0);
      if (!whole && w.begins && threadIdx.x == 0) {
        AttnOpen d;
        d.last = w.last;
        d.rows = rows, d.start = w.start, d.row0 = w.row0, d.head = w.head;
        p.parts.open[blockIdx.x] = d;
      }
      // Beside scores of this size m's rounding is an exponent of its own: 2^(s f - m) of the
      // largest may leave fp16 or bf16.  (s f rounded by itself, as m is, took 3 to 9 %
      // more with bf16, and as long with 8-bit caches only where all rows do so.)
      if (live && fabsf(m) > 0x1p26f && m != -INFINITY) set_status(a.status, MOE_DEV_NONFINITE);
      const int64_t at = static_cast<int64_t>(part) * p.parts.rows + r;
      if (!whole && live) p.parts.ml[at] = make_float2(m - kPower, l);
      if (begun) {
        ok = ptx::mbar_wait(&sh->o_last[qi], segs++ & 1, abort, p.budget);
        if (!ok) break;
        ptx::tc_fence_after();
        const float inv_l = whole ? 1.0f / l : 1.0f, f = kBytes ? 1.0f : inv_l;
        moe_bf16 *dst = p.out + (w.start + token) * p.out_ld + head * D;
#pragma unroll 1
        for (int i = 0; i < D; i += 32) {
          float o[32];
          ptx::tmem_ld32(o_at + i, o);
          ptx::tmem_wait_ld();
          if (!live) continue;
          if (kBytes) {  // (the product of both factors may be below fp32's normal numbers)
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = o[j] * inv_l * unit;
          }
          if (whole) {
#pragma unroll
            for (int j = 0; j < 32; j += 8)
              *reinterpret_cast<uint4 *>(dst + i + j) =
                  make_uint4(pack_bf16(o[j] * f, o[j + 1] * f), pack_bf16(o[j + 2] * f, o[j + 3] * f),
                             pack_bf16(o[j + 4] * f, o[j + 5] * f),
                             pack_bf16(o[j + 6] * f, o[j + 7] * f));
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<float4 *>(p.parts.at(part, D, i + j, r)) =
                  make_float4(o[j] * f, o[j + 1] * f, o[j + 2] * f, o[j + 3] * f);
          }
        }
        ptx::tc_fence_before();
      }
    }
    ptx::tmem_wait_st();  // (after a wait that gave up some may be on their way)
    if (!ok && lane == 0) set_status(a.status, MOE_DEV_TIMEOUT);
  } else {
    if (S::kSoftRegs) leave_registers<S::kRestRegs>();
    if (warp == S::kFetchWarp) {  // ------------------------------------ fetch
      const uint64_t pol = ptx::policy_evict_last();
      uint32_t n = 0, tiles = 0, q_tiles[2] = {0, 0};
      // With 8 units a key tile (16 heads of 256, bf16) this warp would be what bounds
      // the kernel: there one lane issues a key tile's copies, some 25 cycles each, with
      // all their slots waited for together (pages of 64: 1130 -> 1350 TFLOP/s, of 16:
      // 820 -> 1265).  With 4 units, or where the conversion leaves slots one by one,
      // lanes with a copy each, some 65 cycles, take 1 to 10 % less than that.
      constexpr uint32_t kSlots = kBytes ? S::kRaws : kUnits, kGroup = !kBytes && NQ == 1 ? kChunks : 1;
      uint32_t slot = 0, phase = 1;
      const int k_shift = 31 - __clz(k_box), v_shift = 31 - __clz(v_box);
      constexpr int kSlotBytes = kBytes ? S::kRaw : S::kUnit;
      uint8_t *slots = kBytes ? raw : ring;
      uint64_t *full = kBytes ? sh->raw_full : sh->full, *empty = kBytes ? sh->raw_empty : sh->empty;
      for (TcSegment w = next_segment(); w.there && ok; w = next_segment()) {
        const int32_t *table = a.table + w.b * a.table_ld;
        const int len = w.len, first_read = attn_first_read(a, w.ctx, w.row0);
        // lane i: the page of position kt * 128 + i * page
        const auto pages_of = [&](int kt) {
          const int64_t pos = static_cast<int64_t>(kt) * 128 + static_cast<int64_t>(lane) * page;
          int id = 0;
          if (pos < first_read) {
            id = a.pages;
          } else if (kt < w.k1 && lane * k_box < 128 && pos < len) {
            id = table[pos >> a.page_shift];
            if (id < 0 || id >= a.pages) {
              set_status(a.status, MOE_DEV_BAD_INDEX);
              id = 0;
            }
          }
          return id;
        };
        // lane i: the cache's row of position i << shift of the tile whose pages `ids` are
        const auto rows_of = [&](int ids, int kt, int shift) {
          const int at = (lane << shift) & 127;
          const int id = __shfl_sync(0xFFFFFFFFu, ids, at >> a.page_shift);
          return static_cast<int>(
              ((static_cast<int64_t>(id) * a.kv_heads + w.head) << a.page_shift) +
              ((kt * 128 + at) & (page - 1)));
        };
        // Units of K or V from the tile's `first`, kGroup of them; box i of the tile
        // comes from row `rows` of lane i, and positions there are `there`.
        const auto units = [&](const CUtensorMap *tm, int rows, auto which, int first, int there) {
          constexpr bool is_v = which.value;
          uint32_t mine = slot + lane % kGroup, parity = phase;
          if (mine >= kSlots) mine -= kSlots, parity ^= 1;
          ok = ptx::mbar_wait(&empty[mine], parity, abort, p.budget);
          if (kGroup > 1) ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) return;
          // a unit's boxes; a unit of K has the tile's, one of V its share of them
          constexpr int kKeys = is_v ? S::kVKeys : 128, kRow = (is_v ? D : 64) * (kBytes ? 1 : 2);
          constexpr int kKeyBits = kKeys == 128 ? 7 : kKeys == 64 ? 6 : 5;
          const int shift = is_v ? v_shift : k_shift, per_shift = kKeyBits - shift;
          const int bytes = kRow << shift, b0 = is_v ? first << per_shift : 0;
          const int all = min((is_v ? kGroup : 1) << per_shift, ((there - 1) >> shift) + 1 - b0);
          if (lane < kGroup) {
            const int have = is_v ? min(max(all - (lane << per_shift), 0), 1 << per_shift) : all;
            ptx::mbar_expect_tx(&full[mine], have * bytes);
          }
          const auto box = [&](int i, int row) {
            const int at = (is_v ? i & ((1 << per_shift) - 1) : i) * bytes;
#pragma unroll
            for (int c = 0; c < (is_v ? 1 : kGroup); ++c) {
              uint32_t to = slot + (is_v ? i >> per_shift : c);
              if (to >= kSlots) to -= kSlots;
              ptx::tma_load_3d(slots + to * kSlotBytes + at, tm, 0, row, is_v ? 0 : first + c,
                               &full[to], pol);
            }
          };
          if (kGroup == 1) {
            const int row = __shfl_sync(0xFFFFFFFFu, rows, b0 + lane);
            if (lane < all) box(lane, row);
          } else {
#pragma unroll 1
            for (int i = 0; i < all; i += 2) {
              const int r0 = __shfl_sync(0xFFFFFFFFu, rows, b0 + i);
              const int r1 = __shfl_sync(0xFFFFFFFFu, rows, b0 + i + 1);
              if (elect_one()) {
                box(i, r0);
                if (i + 1 < all) box(i + 1, r1);
              }
            }
          }
          __syncwarp();
          n += kGroup, slot += kGroup;
          if (slot >= kSlots) slot -= kSlots, phase ^= 1;
        };
        const auto k_units = [&](int rows, int kt) {
          for (int c = 0; c < kChunks && ok; c += kGroup)
            units(&tm_k, rows, std::false_type(), c, len - kt * 128);
        };
        const auto v_units = [&](int ids, int kt) {
          const int rows = rows_of(ids, kt, v_shift);
          for (int u = 0; u < kChunks && ok; u += kGroup) units(&tm_v, rows, std::true_type(), u, len - kt * 128);
        };
        if (p.q_copy) {
          // (rows behind the sequence's last are of no use and do no harm)
          for (int i = 0; i < NQ && ok; ++i) {
            if (w.first(i) >= w.end(i)) continue;
            uint64_t *here = kBytes ? &sh->q_raw[i] : &sh->q_full[i];
            ok = ptx::mbar_wait(&sh->q_empty[i], (q_tiles[i] & 1) ^ 1, abort, p.budget);
            if (!ok) break;
            ++q_tiles[i];
            if (lane == 0) ptx::mbar_expect_tx(here, kChunks * 16384);
            __syncwarp();
            if (lane < kChunks)
              ptx::tma_load_3d(q_area + (i * kChunks + lane) * 16384, &tm_q, lane * 64,
                               w.head * a.group, w.start + attn_token(a, w.row0 + 128 * i), here, pol);
          }
        }
        int before = 0, ids = pages_of(w.k0);
        for (int kt = w.k0; kt <= w.k1 && ok; ++kt) {
          const int next = kt < w.k1 ? pages_of(kt + 1) : 0;
          if (NQ == 2 && kt > w.k0) v_units(before, kt - 1);
          if (kt < w.k1) {
            const int rows = rows_of(ids, kt, k_shift);
            if (kBytes && ok) {
              const uint32_t slot = tiles % S::kScaleSlots;
              ok = ptx::mbar_wait(&sh->scale_empty[slot], ((tiles / S::kScaleSlots) & 1) ^ 1, abort,
                                  p.budget);
              if (!ok) break;
              const int have = min(128 >> k_shift, ((len - kt * 128 - 1) >> k_shift) + 1);
              if (elect_one()) ptx::mbar_expect_tx(&sh->scale_raw[slot], 2 * have * k_box * 4);
              __syncwarp();
              if (lane < have) {
                const uint32_t dst = ptx::smem_u32(scales + slot * 256 + lane * k_box);
                // (scales before first_read are not looked at)
                const int from = kt * 128 + (lane << k_shift) < first_read ? 0 : rows;
                bulk_load(dst, p.k_scale + from, k_box * 4, &sh->scale_raw[slot]);
                bulk_load(dst + 512, p.v_scale + from, k_box * 4, &sh->scale_raw[slot]);
              }
              ++tiles;
            }
            if (ok) k_units(rows, kt);
          }
          if (NQ == 1 && kt > w.k0 && ok) v_units(before, kt - 1);
          before = ids, ids = next;
        }
      }
      // The block does not end before its copies have landed, whoever gives up waiting
      // for them, and when.
      if (lane == 0) {
        int never = 0;
#pragma unroll 1
        for (uint32_t k = 0; k < kSlots && k < n; ++k) {
          const uint32_t j = n - 1 - k;
          ptx::mbar_wait(&full[j % kSlots], (j / kSlots) & 1, &never, ptx::kDrainBudgetNs);
        }
        for (int i = 0; i < NQ; ++i)
          if (q_tiles[i] > 0)
            ptx::mbar_wait(kBytes ? &sh->q_raw[i] : &sh->q_full[i], (q_tiles[i] - 1) & 1, &never,
                           ptx::kDrainBudgetNs);
#pragma unroll 1
        for (uint32_t k = 0; k < S::kScaleSlots && k < tiles; ++k) {
          const uint32_t j = tiles - 1 - k;
          ptx::mbar_wait(&sh->scale_raw[j % S::kScaleSlots], (j / S::kScaleSlots) & 1, &never,
                         ptx::kDrainBudgetNs);
        }
        if (*abort) set_status(a.status, MOE_DEV_TIMEOUT);
      }
      __syncwarp();
    } else if (kBytes && warp >= S::kSoftWarps && warp < S::kFetchWarp) {  // -- convert
      constexpr uint32_t kConvWarps = S::kConvWarps > 0 ? S::kConvWarps : 1;
      constexpr uint32_t kRaws = S::kRaws > 0 ? S::kRaws : 1;
      constexpr int kChunkBits = kChunks == 4 ? 2 : kChunks - 1;
      uint32_t n = 0;
      // 128 rows of 64 codes, 16 of a row at a time, become rows of 64 fp16 code *
      // scale, rounded once: a key's scale is two fp16 terms (22 bits, since it moves
      // all of a score), a value's one (it moves a weight by as much as the weight's
      // own rounding; two terms there too: 942 us for 902).  Values whose key is `dead`
      // or later become 0.  (A warp for each unit, or two units at a time, took longer:
      // the ring is short.)
      const int t = threadIdx.x - 32 * S::kSoftWarps;
      const int v_shift = 31 - __clz(v_box);
      constexpr int kEach = 512 / (32 * kConvWarps);
      const auto unit = [&](const uint32_t *sc, bool is_v, int dead) {
        const uint32_t rs = n % kRaws, us = n % kUnits;
        ok = ok && ptx::mbar_wait(&sh->raw_full[rs], (n / kRaws) & 1, abort, p.budget);
        if (!ok) return;
        const uint4 *src = reinterpret_cast<const uint4 *>(raw + rs * S::kRaw) + t;
        uint8_t *dst = ring + us * S::kUnit;
        uint4 v[kEach];
        uint32_t scale[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const int row = i * (8 * kConvWarps) + t / 4;
          v[i] = src[i * (32 * kConvWarps)];
          int key = row;
          if (is_v) {
            key = (row >> (v_shift + kChunkBits) << v_shift) + (row & (v_box - 1));
            if (key >= dead) v[i] = make_uint4(0, 0, 0, 0);
          }
          scale[i] = sc[key];
        }
        ok = ptx::mbar_wait(&sh->empty[us], ((n / kUnits) & 1) ^ 1, abort, p.budget);
        if (!ok) return;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const int row = i * (8 * kConvWarps) + t / 4, c = 2 * (t & 3);
          const __half2 hi = bits_h2(__byte_perm(scale[i], 0, 0x1010));
          const __half2 lo = bits_h2(__byte_perm(scale[i], 0, 0x3232));
          uint32_t h[8];
          codes_to_f16x2<KV>(v[i].x, h[0], h[1]), codes_to_f16x2<KV>(v[i].y, h[2], h[3]);
          codes_to_f16x2<KV>(v[i].z, h[4], h[5]), codes_to_f16x2<KV>(v[i].w, h[6], h[7]);
          if (is_v) {
#pragma unroll
            for (int k = 0; k < 8; ++k) h[k] = h2_bits(__hmul2(bits_h2(h[k]), hi));
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              h[k] = h2_bits(__hfma2(bits_h2(h[k]), hi, __hmul2(bits_h2(h[k]), lo)));
          }
          *reinterpret_cast<uint4 *>(dst + row * 128 + ((c ^ (row & 7)) << 4)) =
              make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4 *>(dst + row * 128 + (((c + 1) ^ (row & 7)) << 4)) =
              make_uint4(h[4], h[5], h[6], h[7]);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(&sh->full[us]);
          ptx::mbar_arrive(&sh->raw_empty[rs]);
        }
        ++n;
      };
      uint32_t tiles = 0, v_tiles = 0;
      for (TcSegment w = next_segment(); w.there && ok; w = next_segment()) {
        const auto v_units = [&](int kt) {
          const uint32_t slot = v_tiles++ % S::kScaleSlots;
          const uint32_t *sc = reinterpret_cast<const uint32_t *>(scales + slot * 256 + 128);
          for (int u = 0; u < kChunks && ok; ++u)
            unit(sc + u * S::kVKeys, true, w.len - kt * 128 - u * S::kVKeys);
          __syncwarp();
          if (ok && lane == 0) ptx::mbar_arrive(&sh->scale_empty[slot]);
        };
        for (int kt = w.k0; kt <= w.k1 && ok; ++kt) {
          if (NQ == 2 && kt > w.k0) v_units(kt - 1);
          if (kt < w.k1 && ok) {
            const uint32_t slot = tiles % S::kScaleSlots;
            ok = ptx::mbar_wait(&sh->scale_full[slot], (tiles++ / S::kScaleSlots) & 1, abort, p.budget);
            const uint32_t *sc = reinterpret_cast<const uint32_t *>(scales + slot * 256);
            for (int c = 0; c < kChunks && ok; ++c) unit(sc, false, 0);
          }
          if (NQ == 1 && kt > w.k0 && ok) v_units(kt - 1);
        }
      }
    } else if (warp == S::kPlanWarp) {  // --------------------------------- plan
      AttnWalk<R, 128, kTcTileCost> w;
      w.init(a, sh->share);
      // The next segment; whether there is one.
      const auto plan = [&]() {
        const bool more = w.next(a, range);
        ok = ok && ptx::mbar_wait(&sh->plan_empty[seg_n % 4], ((seg_n / 4) & 1) ^ 1, abort, p.budget);
        if (ok && lane == 0) {
          TcSegment s;
          s.there = more;
          if (more) {
            s.b = w.b, s.start = w.s.start, s.len = w.s.len, s.head = w.head, s.ctx = w.t.ctx;
            s.row0 = w.cur * R, s.rows = min(w.t.rows - s.row0, R);
            s.k0 = w.k0, s.k1 = w.k1;
            s.begins = w.begins;
            s.last = w.ends ? -1 : static_cast<int>((w.tile_end - 1) / sh->share.per);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              s.q0[i] = s.q1[i] = 0;
              if (i < NQ && 128 * i < s.rows) {
                const int first = s.ctx + attn_token(a, s.row0 + 128 * i);
                const int last = s.ctx + attn_token(a, s.row0 + min(128 * i + 127, s.rows - 1));
                s.q0[i] = max(w.k0, a.window && first >= a.window ? (first - a.window + 1) / 128 : 0);
                s.q1[i] = max(s.q0[i], min(w.k1, last / 128 + 1));
              }
            }
          }
          sh->plan[seg_n % 4] = s;
          ptx::mbar_arrive(&sh->plan_full[seg_n % 4]);
        }
        __syncwarp();
        ++seg_n;
        return more && ok;
      };
      if (!kBytes) {
        while (plan()) {}
      } else {
        // ... and the scales of its key tiles, four keys a lane: under powers of two
        // that bring the largest (of the tile's keys, of the segment's values so far)
        // into [2^5, 2^6), as two fp16 terms.  A value's scale that is not finite
        // makes its key NaN and itself 0: the rows that see it are NaN, and 0 times it
        // is not NaN where it is hidden.
        const auto magnitude = [](float x) { return fabsf(x) < INFINITY ? fabsf(x) : 0.0f; };
        const auto largest = [&](const float (&x)[4]) {
          const float top = fmaxf(fmaxf(magnitude(x[0]), magnitude(x[1])),
                                  fmaxf(magnitude(x[2]), magnitude(x[3])));
          return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top)));
        };
        const auto power = [](float top) {
          const int e = static_cast<int>(__float_as_uint(top) >> 23);
          return __uint_as_float(static_cast<uint32_t>(min(259 - e, 253)) << 23);
        };
        const auto two_terms = [](float x) {
          const __half hi = __float2half_rn(x), lo = __float2half_rn(x - __half2float(hi));
          return static_cast<uint32_t>(__half_as_ushort(hi)) |
                 (static_cast<uint32_t>(__half_as_ushort(lo)) << 16);
        };
        uint32_t tiles = 0;
        bool more = plan();
        while (more) {
          const int k0 = w.k0, k1 = w.k1, len = w.s.len;
          const int first_read = attn_first_read(a, w.t.ctx, w.cur * R);
          more = plan();  // (one ahead)
          float v_top = 0.0f;
          for (int kt = k0; kt < k1 && ok; ++kt, ++tiles) {
            const uint32_t slot = tiles % S::kScaleSlots;
            ok = ptx::mbar_wait(&sh->scale_raw[slot], (tiles / S::kScaleSlots) & 1, abort, p.budget);
            if (!ok) break;
            float4 *ks = reinterpret_cast<float4 *>(scales + slot * 256) + lane, *vs = ks + 32;
            const float4 kx = *ks, vx = *vs;
            float k[4] = {kx.x, kx.y, kx.z, kx.w}, v[4] = {vx.x, vx.y, vx.z, vx.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (kt * 128 + 4 * lane + i >= len || kt * 128 + 4 * lane < first_read)
                k[i] = v[i] = 0.0f;  // (pages begin at multiples of 16)
              if (!(fabsf(v[i]) < INFINITY)) k[i] = v[i] - v[i], v[i] = 0.0f;
            }
            const float k_up = power(largest(k));
            v_top = fmaxf(v_top, largest(v));
            const float v_up = power(v_top);
            *reinterpret_cast<uint4 *>(ks) = make_uint4(two_terms(k[0] * k_up), two_terms(k[1] * k_up),
                                                        two_terms(k[2] * k_up), two_terms(k[3] * k_up));
            *reinterpret_cast<uint4 *>(vs) = make_uint4(two_terms(v[0] * v_up), two_terms(v[1] * v_up),
                                                        two_terms(v[2] * v_up), two_terms(v[3] * v_up));
            if (lane == 0)
              sh->k_unit[slot] = pow2_inverse(k_up), sh->v_unit[slot] = pow2_inverse(v_up);
            ptx::fence_proxy_async_smem();  // (before the slot's next copy)
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&sh->scale_full[slot]);
          }
        }
      }
    } else if (warp >= S::kMmaWarp && warp < S::kMmaWarp + NQ) {  // --- products
      // One warp a query tile: while one waits, the other's products run.
      const int qi = warp - S::kMmaWarp;
      const uint32_t type = kBytes ? ptx::idesc_f16_f32(128, 128) : ptx::idesc_bf16_f32(128, 128);
      const uint32_t type_v = (kBytes ? ptx::idesc_f16_f32(128, D) : ptx::idesc_bf16_f32(128, D)) |
                              kIdescTransB;
      const uint32_t q_at = ptx::smem_u32(q_area) + qi * kChunks * 16384;
      const uint32_t ring_at = ptx::smem_u32(ring);
      constexpr int kVSteps = S::kVKeys / 16;
      uint32_t v_step[kVSteps];  // where 16 keys' values begin in a unit, / 16
#pragma unroll
      for (int k = 0; k < kVSteps; ++k)
        v_step[k] = (16 * k / v_box * (v_box * D * 2) + 16 * k % v_box * 128) >> 4;
      uint32_t n = 0, segs = 0, items = 0, turns = 0;  // units, segments, key tiles so far
      for (TcSegment w = next_segment(); w.there && ok; w = next_segment()) {
        bool q_here = false, o_begun = false;
        const auto buffer = [&](uint32_t item) { return NQ == 2 ? qi : static_cast<int>(item & 1); };
        const auto parity = [&](uint32_t item) { return NQ == 2 ? item & 1 : (item >> 1) & 1; };
        const auto arrived = [&](uint32_t u) {
          ok = ok && ptx::mbar_wait(&sh->full[u % kUnits], (u / kUnits) & 1, abort, p.budget);
          return ok;
        };
        // Values behind the sequence's end: 0 (the slots hold what was there; with
        // two query tiles both warps do so).
        const auto clear_tail = [&](uint32_t n0, int left) {
          for (int u = 0; u < kChunks; ++u) {
            uint4 *at = reinterpret_cast<uint4 *>(ring + (n0 + u) % kUnits * S::kUnit);
            for (int i = lane; i < 1024; i += 32) {  // 16 bytes each
              const int row = i / 8;
              const int key = u * S::kVKeys + row / (v_box * kChunks) * v_box + row % v_box;
              if (key >= left) at[i] = make_uint4(0, 0, 0, 0);
            }
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
        };
        const auto here = [&](uint32_t n0) {
          for (int u = 0; u < kChunks; ++u)
            if (!arrived(n0 + u)) return;
        };
        // S from the units n0 .. of a key tile, which are here
        const auto qk = [&](uint32_t n0, bool ends) {
          const uint32_t s_at = tmem + S::kS + buffer(items) * 128;
          if (elect_one()) {
            for (int c = 0; c < kChunks; ++c)
              mma_ss4(s_at, desc_lower(q_at + c * 16384, 16),
                      desc_lower(ring_at + (n0 + c) % kUnits * S::kUnit, 16), type, c > 0);
            if (NQ == 2) ptx::mbar_arrive(&sh->turn[1 - qi]);
            ptx::mma_commit(&sh->s_full[buffer(items)]);
            for (int c = 0; c < kChunks; ++c) ptx::mma_commit(&sh->empty[(n0 + c) % kUnits]);
            if (ends) ptx::mma_commit(&sh->q_empty[qi]);
          }
          __syncwarp();
          ++items;
        };
        // The p of the key tile before the newest `ahead`.
        const auto weights = [&](int ahead) {
          const uint32_t item = items - 1 - ahead;
          ok = ok && ptx::mbar_wait(&sh->p_full[buffer(item)], parity(item), abort, p.budget);
        };
        // O += p v.  `ends`: the segment's last (a barrier of its own: o_done's
        // phases before may go by unseen)
        const auto pv = [&](uint32_t n0, int ahead, bool ends) {
          const uint32_t p_at = tmem + S::kS + buffer(items - 1 - ahead) * 128;
          if (elect_one()) {
            for (int u = 0; u < kChunks; ++u) {
              const uint32_t v_at =
                  desc_lower(ring_at + (n0 + u) % kUnits * S::kUnit, v_box * 128);
#pragma unroll
              for (int k = 0; k < kVSteps; k += 2)
                mma_ts2(tmem + S::kO + qi * D, p_at + u * (S::kVKeys / 2) + 8 * k,
                        v_at + v_step[k], v_at + v_step[k + 1], type_v, o_begun || u > 0 || k > 0);
            }
            ptx::mma_commit(&sh->o_done[qi]);
            if (ends) ptx::mma_commit(&sh->o_last[qi]);
            for (int u = 0; u < kChunks; ++u) ptx::mma_commit(&sh->empty[(n0 + u) % kUnits]);
          }
          __syncwarp();
          o_begun = true;
        };
        const auto pass = [&](uint32_t n0) {  // a key tile of no row of this query tile
          if (elect_one())
            for (int u = 0; u < kChunks; ++u) ptx::mma_commit(&sh->empty[(n0 + u) % kUnits]);
          __syncwarp();
        };
        for (int kt = w.k0; kt <= w.k1; ++kt) {
          const bool has_k = kt < w.k1, has_v = kt > w.k0;
          const bool do_k = has_k && w.has(qi, kt), do_v = has_v && w.has(qi, kt - 1);
          const int left = w.len - (kt - 1) * 128;
          // All that the products need is waited for before the first of them: the
          // tensor cores have room for few, and stand still during a wait.
          if (do_k && !q_here) {
            q_here = true;
            ok = ok && ptx::mbar_wait(&sh->q_full[qi], segs++ & 1, abort, p.budget);
          }
          if (NQ == 1) {
            if (has_k) {
              here(n);
              if (!ok) break;
              ptx::tc_fence_after();
              qk(n, kt + 1 == w.k1), n += kChunks;
            }
            if (has_v) {
              here(n);
              if (ok && !kBytes && left < 128) clear_tail(n, left);
              weights(has_k ? 1 : 0);
              if (!ok) break;
              ptx::tc_fence_after();
              pv(n, has_k ? 1 : 0, kt == w.k1), n += kChunks;
            }
            continue;
          }
          uint32_t nv = n;
          if (has_v) here(n), n += kChunks;
          if (has_k) here(n);
          if (ok && do_v && !kBytes && left < 128) clear_tail(nv, left);
          if (do_v) weights(0);
          // The query tiles take turns: each one's softmax then falls into the
          // other's products, not into the other's softmax.
          ok = ok && ptx::mbar_wait(&sh->turn[qi], (turns++ & 1) ^ (qi == 0 ? 1 : 0), abort, p.budget);
          if (!ok) break;
          ptx::tc_fence_after();
          if (do_v) pv(nv, 0, kt == w.end(qi));
          else if (has_v) pass(nv);
          if (do_k) {
            qk(n, kt + 1 == w.end(qi));
          } else {
            if (elect_one()) ptx::mbar_arrive(&sh->turn[1 - qi]);
            if (has_k) pass(n);
          }
          if (has_k) n += kChunks;
        }
      }
      // all products are complete before tensor memory is given back
      if (elect_one()) {
        int never = 0;
        ptx::mma_commit(&sh->done);
        ptx::mbar_wait(&sh->done, 0, &never, ptx::kDrainBudgetNs);
        if (*abort) set_status(a.status, MOE_DEV_TIMEOUT);
      }
      __syncwarp();
    }
  }
  __syncthreads();
  if (warp == S::kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

}  // namespace moe
