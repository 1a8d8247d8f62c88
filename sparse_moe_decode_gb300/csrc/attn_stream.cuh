// attn_stream.cuh -- attention of few rows (single tokens, short drafts) over
// long contexts: the cache streams through, bound by its bytes.
//
// out = softmax(scale q k^T) v for a tile of 16 rows, in one pass over the keys
// with the running maximum m and total l of the softmax.  A block has four
// warps that compute, and one that fetches.  Of the 64 keys of a key tile each
// warp takes 16 for the scores, and then a quarter of the columns for the
// values; the weights pass between them as operand fragments in shared memory,
// one barrier a tile.  No key is read twice, and a warp's sums are 16 rows of
// head_dim / 4 columns in registers, finished where they are (with the keys
// shared out for the values as well, four times the registers, and joining the
// warps' sums took 1.2 to 3.1 us a segment).  K and V tiles come through a ring
// of shared-memory slots (TMA, 128-byte swizzle, one box a page); products are
// mma.sync m16n8k16 with fp32 sums.
//
// m is that of the tiles before, which nearly always does; only where a weight
// comes out above 2^13 or so do the warps find the maximum anew.
//
// 8-bit codes are made fp16 in registers, exactly; q then takes a power of two
// a row (fp16 keeps all of bf16's digits within 2^-28 of the row's largest).
// A key's scale multiplies its column of q k^T; a value's scale multiplies its
// weight, and the products t = p s_v enter as fp16 under a power of two a row
// that follows the largest, so that they keep 11 digits whatever the scales are.
//
// Measured: 128 sequences of 1 .. 16384 positions, 32 heads on 8 of 128, bf16
// 640 us, 6.75 TB/s, the rate of a copy.  int8 halves the bytes and the time
// is then that of the conversions and products (32 sequences of up to 8192: 67
// us, 4.5 TB/s; issue slots 57 % used, ALU 46 %; e4m3 64.5 us).  One sequence of 4099: 11.3 us,
// launches, page table, one round trip and the join.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include "attn_args.cuh"
#include "delta_mma.cuh"
#include "early.cuh"
#include "sm100_ptx.cuh"

namespace moe {

constexpr int kStreamTileCost = 1;  // beginning and ending a tile, in key tiles

template <int D, int KV>
struct StreamShape {
  static constexpr int kR = kStreamRows, kKT = 64, kWarps = 4;
  static constexpr bool kBytes = KV != MOE_KV_BF16;  // 8-bit codes
  static constexpr int kRow = D * (kBytes ? 1 : 2);  // bytes of a cached row
  static constexpr int kTile = kKT * kRow, kSlot = kTile + (kBytes ? 256 : 0);
  static constexpr int kSteps = D / 16;
  static constexpr int kThreads = 160;
  static constexpr int kQ = kR * D * 2, kP = 2 * kWarps * 512;  // fragments of q, of the weights
  static constexpr int kFixed = kQ + kP + 2048;                 // + barriers, maxima, the share
  static constexpr int kBlocks = kTile > 16384 ? 2 : 3;         // an SM
  static constexpr int kFit = (233472 / kBlocks - 1024 - kFixed) / kSlot;
  static constexpr int kSlots = kFit > 12 ? 12 : kFit;
  static constexpr int kSmem = kFixed + kSlots * kSlot;
  static_assert(kSlots >= 3, "ring");
};

struct StreamSmem {  // behind the slots, their scales, q and the weights
  uint64_t full[12], empty[12];
  AttnShare share;
  float top[4][kStreamRows], most[4][kStreamRows], l[4][kStreamRows];
  int abort;
};
static_assert(sizeof(StreamSmem) <= 2048, "shared memory");

// Offset of 16 bytes c of row r16 + r within a tile, where r16 is a multiple
// of 16 and boxes of `box` rows lie one after another.
template <int ROW>
struct TileRows {
  uint32_t base, step;  // of the 16 rows; from one 128-byte column to the next
  __device__ __forceinline__ TileRows(int r16, int box) {
    if (ROW <= 128) {
      base = r16 * ROW, step = 0;
    } else {
      base = (r16 / box) * box * ROW + (r16 % box) * 128;
      step = box * 128;
    }
  }
  __device__ __forceinline__ uint32_t at(int r, int c) const {
    if (ROW == 64)
      return base + (r >> 1) * 128 + ((((r & 1) * 4 + c) ^ ((r >> 1) & 7)) << 4);
    return base + (c >> 3) * step + r * 128 + (((c & 7) ^ (r & 7)) << 4);
  }
};

template <int KV>
__device__ __forceinline__ void attn_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (KV == MOE_KV_BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    mma16(c, a, b0, b1);
}

// All compute warps meet; whether any thread says so.
__device__ __forceinline__ bool meet_any(bool mine) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(mine ? 1u : 0u)
      : "memory");
  return r != 0;
}

template <int D, int KV>
__global__ void __launch_bounds__(160, (StreamShape<D, KV>::kBlocks))
attn_stream_kernel(const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const AttnBatch a, const AttnRange range,
                   const AttnArgs p) {
  using S = StreamShape<D, KV>;
  constexpr int kSlots = S::kSlots, R = S::kR, kSteps = S::kSteps;
  constexpr bool kBytes = S::kBytes;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint4 *qf = reinterpret_cast<uint4 *>(smem + kSlots * S::kTile);
  uint4 *weights = qf + S::kQ / 16;  // [2][4 warps' keys][32 lanes]
  float *scales = reinterpret_cast<float *>(weights + S::kP / 16);
  StreamSmem *sh = reinterpret_cast<StreamSmem *>(scales + (kBytes ? kSlots * 64 : 0));
  volatile int *abort = &sh->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      ptx::mbar_init(&sh->full[i], 1);
      ptx::mbar_init(&sh->empty[i], 4);
    }
    sh->abort = 0;
    ptx::fence_mbar_init();
    ptx::tma_prefetch_desc(&tm_k);
    ptx::tma_prefetch_desc(&tm_v);
  }
  early_begin();
  if (threadIdx.x == 0) p.parts.open[blockIdx.x].last = -1;
  attn_share<R, 64, kStreamTileCost>(a, range, p.least_share, &sh->share);
  if (sh->share.seq < 0) return;
  AttnWalk<R, 64, kStreamTileCost> w;
  w.init(a, sh->share);
  const int page = 1 << a.page_shift;
  const int box = page < 64 ? page : 64;  // positions

  if (warp == 4) {  // ------------------------------------------------ fetch
    const uint64_t pol = ptx::policy_evict_first();
    uint32_t n = 0;  // slots filled
    bool stop = false;
    const int per_tile = 64 / box;
    while (!stop && w.next(a, range)) {
      const int32_t *table = a.table + w.b * a.table_ld;
      const int tiles = w.k1 - w.k0;
      const int boxes = (w.s.len + box - 1) / box;  // that the sequence has
      const int first_read = attn_first_read(a, w.t.ctx, w.cur * R);
      int page_of = 0;                              // lane i's box of the 32 fetched next
      for (int i = 0; i < tiles && !stop; ++i) {
        const int b0 = (w.k0 + i) * per_tile;
        if ((i * per_tile) % 32 == 0) {
          const int bx = b0 + lane;
          page_of = 0;
          if (bx * box < first_read) {
            page_of = a.pages;
          } else if (bx < boxes && bx < w.k1 * per_tile) {
            page_of = table[(static_cast<int64_t>(bx) * box) >> a.page_shift];
            if (page_of < 0 || page_of >= a.pages) {
              set_status(a.status, MOE_DEV_BAD_INDEX);
              page_of = 0;
            }
          }
        }
        const int have = min(per_tile, boxes - b0);
#pragma unroll
        for (int kv = 0; kv < 2 && !stop; ++kv, ++n) {
          const uint32_t slot = n % kSlots;
          const bool free = ptx::mbar_wait(&sh->empty[slot], ((n / kSlots) & 1) ^ 1, abort, p.budget);
          if (!__all_sync(0xFFFFFFFFu, free)) {  // (lanes issue and account for copies together)
            stop = true;
            break;
          }
          if (lane == 0)
            ptx::mbar_expect_tx(&sh->full[slot], have * box * (S::kRow + (kBytes ? 4 : 0)));
          __syncwarp();
          const int at = (i * per_tile) % 32;
          // lanes 0 .. have - 1 issue a box each
          const int id = __shfl_sync(0xFFFFFFFFu, page_of, (at + lane) & 31);
          if (lane < have) {
            const int64_t row =
                ((static_cast<int64_t>(id) * a.kv_heads + w.head) << a.page_shift) +
                (((b0 + lane) * box) & (page - 1));
            uint8_t *dst = smem + slot * S::kTile + lane * box * S::kRow;
            const CUtensorMap *tm = kv ? &tm_v : &tm_k;
            // (rows of 64 bytes lie two to a line)
            ptx::tma_load_3d(dst, tm, 0, static_cast<int>(S::kRow == 64 ? row >> 1 : row), 0,
                             &sh->full[slot], pol);
            if (kBytes)
              bulk_load(ptx::smem_u32(scales + slot * 64 + lane * box),
                        (kv ? p.v_scale : p.k_scale) + (id < a.pages ? row : 0), box * 4,
                        &sh->full[slot]);
          }
        }
      }
    }
    // The block does not end before its copies have landed, whoever gives up waiting for
    // them, and when.
    if (lane == 0) {
      int never = 0;
      for (uint32_t k = 0; k < kSlots && k < n; ++k) {
        const uint32_t j = n - 1 - k;
        ptx::mbar_wait(&sh->full[j % kSlots], (j / kSlots) & 1, &never, ptx::kDrainBudgetNs);
      }
      if (*abort) set_status(a.status, MOE_DEV_TIMEOUT);
    }
    return;
  }

  // ------------------------------------------------------------- compute
  constexpr int kCols = D / 4;                   // of this warp
  const int g = lane >> 2, c = lane & 3;
  uint32_t n = 0;
  const uint32_t smem_at = ptx::smem_u32(smem);
  // ldmatrix rows: lane l gives row l % 8 of block l / 8
  const int row_k = (lane & 7) + (kBytes ? ((lane >> 3) & 1) : (lane >> 4)) * 8;
  const int col_k = kBytes ? lane >> 4 : (lane >> 3) & 1;
  const int row_v = (lane & 7) + ((lane >> 3) & 1) * 8;

  while (w.next(a, range)) {
    const int row0 = w.cur * R;
    const int rows = min(w.t.rows - row0, R);
    const int ctx = w.t.ctx;
    // this thread's two rows
    int pos[2], out_row[2];
    float factor[2];
    {
      const moe_bf16 *src[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = row0 + min(g + 8 * i, rows - 1);
        const int token = attn_token(a, at), h = w.head * a.group + at - token * a.group;
        pos[i] = ctx + token;
        src[i] = p.q + (w.s.start + token) * p.q_ld + h * D;
        out_row[i] = h;
        factor[i] = p.scale_log2;
      }
      constexpr int kMine = kSteps / 4;
      uint4 f[kMine];
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        const int ks = j * 4 + warp;
        if (kBytes) {
          const uint2 x = *reinterpret_cast<const uint2 *>(src[0] + ks * 16 + 4 * c);
          const uint2 y = *reinterpret_cast<const uint2 *>(src[1] + ks * 16 + 4 * c);
          f[j] = make_uint4(x.x, y.x, x.y, y.y);
        } else {
          const auto ld = [&](int i, int o) {
            return *reinterpret_cast<const uint32_t *>(src[i] + ks * 16 + 2 * c + o);
          };
          f[j] = make_uint4(ld(0, 0), ld(1, 0), ld(0, 8), ld(1, 8));
        }
      }
      if (kBytes) {
        float top[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
          const uint32_t v[4] = {f[j].x, f[j].z, f[j].y, f[j].w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            top[i >> 1] = max3_abs(top[i >> 1], bf16_lo(v[i]), bf16_hi(v[i]));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 1));
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 2));
          if (c == 0) sh->top[warp][g + 8 * i] = top[i];
        }
        ptx::named_barrier(1, 128);
        float mult[2], inv;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          for (int k = 0; k < 4; ++k) top[i] = fmaxf(top[i], sh->top[k][g + 8 * i]);
          pow2_scale(top[i], mult[i], inv);
          factor[i] *= inv;
        }
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
          const auto half = [&](uint32_t v, float m) {
            return h2_bits(__floats2half2_rn(bf16_lo(v) * m, bf16_hi(v) * m));
          };
          f[j] = make_uint4(half(f[j].x, mult[0]), half(f[j].y, mult[1]), half(f[j].z, mult[0]),
                            half(f[j].w, mult[1]));
        }
      }
      // (the fragments of the segment before have been read: the warps have met
      // since)
#pragma unroll
      for (int j = 0; j < kMine; ++j) qf[(j * 4 + warp) * 32 + lane] = f[j];
      ptx::named_barrier(1, 128);
    }
    const int first_pos = ctx + attn_token(a, row0);
    const int last_pos = ctx + attn_token(a, row0 + rows - 1);

    float o[kCols / 8][4];
#pragma unroll
    for (int i = 0; i < kCols / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    float ref[2] = {0x1p-110f, 0x1p-110f};  // (8-bit) powers of two: o's sums times ref / 2^7

    bool ok = true;
    for (int kt = w.k0; kt < w.k1; ++kt, n += 2) {
      const int key0 = kt * 64 + warp * 16;
      const uint32_t k_slot = n % kSlots, v_slot = (n + 1) % kSlots;
      // (after a wait that gave up, every wait does so at once: the warps go on
      // meeting at their barriers to the end, but give no slot back, since copies into
      // it may be on their way)
      ok = ptx::mbar_wait(&sh->full[k_slot], (n / kSlots) & 1, abort, p.budget) && ok;
      float s[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = -INFINITY;
      if (key0 <= last_pos && (!a.window || key0 + 16 > first_pos - a.window + 1)) {
        const uint32_t tile = smem_at + k_slot * S::kTile;
        const TileRows<S::kRow> rows16(warp * 16, box);
        // two sums each, so that a product does not wait for the one before it
        float t[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
          t[i][0] = t[i][1] = t[i][2] = t[i][3] = 0.0f;
        }
#pragma unroll
        for (int ks = 0; ks < kSteps; ks += 2) {
          uint32_t b[8];
          if (kBytes) {
            uint32_t x[4];
            ldsm4(x, tile + rows16.at(row_k, ks + col_k));
#pragma unroll
            for (int i = 0; i < 4; ++i) codes_to_f16x2<KV>(x[i], b[2 * i], b[2 * i + 1]);
          } else {
            uint32_t x[4], y[4];
            ldsm4(x, tile + rows16.at(row_k, 2 * ks + col_k));
            ldsm4(y, tile + rows16.at(row_k, 2 * ks + 2 + col_k));
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = x[i], b[4 + i] = y[i];
          }
          const uint4 q0 = qf[ks * 32 + lane], q1 = qf[(ks + 1) * 32 + lane];
          const uint32_t a0[4] = {q0.x, q0.y, q0.z, q0.w}, a1[4] = {q1.x, q1.y, q1.z, q1.w};
          attn_mma<KV>(s[0], a0, b[0], b[1]);
          attn_mma<KV>(s[1], a0, b[2], b[3]);
          attn_mma<KV>(t[0], a1, b[4], b[5]);
          attn_mma<KV>(t[1], a1, b[6], b[7]);
        }
        const float *ksc = scales + k_slot * 64 + warp * 16 + 2 * c;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 f = kBytes ? *reinterpret_cast<const float2 *>(ksc + 8 * i)
                                  : make_float2(1.0f, 1.0f);
          s[i][0] = (s[i][0] + t[i][0]) * (factor[0] * f.x);
          s[i][1] = (s[i][1] + t[i][1]) * (factor[0] * f.y);
          s[i][2] = (s[i][2] + t[i][2]) * (factor[1] * f.x);
          s[i][3] = (s[i][3] + t[i][3]) * (factor[1] * f.y);
        }
        if (key0 + 16 > first_pos + 1 || (a.window && key0 <= last_pos - a.window)) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int key = key0 + 8 * i + 2 * c + (j & 1), ps = pos[j >> 1];
              if (key > ps || (a.window && key <= ps - a.window)) s[i][j] = -INFINITY;
            }
        }
      }
      __syncwarp();
      if (lane == 0 && ok) ptx::mbar_arrive(&sh->empty[k_slot]);
      float2 vs[2];
      if (kBytes) {
        ok = ptx::mbar_wait(&sh->full[v_slot], ((n + 1) / kSlots) & 1, abort, p.budget) && ok;
        const float *vsc = scales + v_slot * 64 + warp * 16 + 2 * c;
        vs[0] = *reinterpret_cast<const float2 *>(vsc);
        vs[1] = *reinterpret_cast<const float2 *>(vsc + 8);
      }

      float e[2][4], sum[2], most[2];  // the weights
      // under m and ref; `most`: the largest with their scales (8-bit)
      const auto form = [&]() {
        sum[0] = sum[1] = most[0] = most[1] = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            e[i][j] = attn_exp2(s[i][j] - (m[j >> 1] == -INFINITY ? 0.0f : m[j >> 1]));
            sum[j >> 1] += e[i][j];
            if (kBytes) {
              // a hidden key's weight is 0 whatever its scale
              e[i][j] = e[i][j] == 0.0f ? 0.0f : e[i][j] * ((j & 1) ? vs[i].y : vs[i].x);
              most[j >> 1] = fmaxf(most[j >> 1], e[i][j]);
            }
          }
      };
      const auto hand_over = [&]() {
        uint4 f;
        if (kBytes) {
          const float f0 = pow2_inverse(ref[0]) * 0x1p7f, f1 = pow2_inverse(ref[1]) * 0x1p7f;
          f.x = h2_bits(__floats2half2_rn(e[0][0] * f0, e[0][1] * f0));
          f.y = h2_bits(__floats2half2_rn(e[0][2] * f1, e[0][3] * f1));
          f.z = h2_bits(__floats2half2_rn(e[1][0] * f0, e[1][1] * f0));
          f.w = h2_bits(__floats2half2_rn(e[1][2] * f1, e[1][3] * f1));
        } else {
          f = make_uint4(pack_bf16(e[0][0], e[0][1]), pack_bf16(e[0][2], e[0][3]),
                         pack_bf16(e[1][0], e[1][1]), pack_bf16(e[1][2], e[1][3]));
        }
        weights[((kt & 1) * 4 + warp) * 32 + lane] = f;
      };
      // The largest of the four warps' (and the four lanes' of a row) values.
      const auto over_warps = [&](float (&x)[2], float (*shared)[kStreamRows]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          x[i] = fmaxf(x[i], __shfl_xor_sync(0xFFFFFFFFu, x[i], 1));
          x[i] = fmaxf(x[i], __shfl_xor_sync(0xFFFFFFFFu, x[i], 2));
          if (c == 0) shared[warp][g + 8 * i] = x[i];
        }
        ptx::named_barrier(1, 128);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          for (int k = 0; k < 4; ++k) x[i] = fmaxf(x[i], shared[k][g + 8 * i]);
      };
      bool again = true;
      if (kt > w.k0) {
        form();
        hand_over();
        bool far = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          far |= sum[i] > 0x1p15f;
          if (kBytes) far |= most[i] >= 256.0f * ref[i] && ref[i] < 0x1p126f;
          // (nothing seen so far)
          far |= m[i] == -INFINITY && fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]),
                                            fmaxf(s[1][2 * i], s[1][2 * i + 1])) > -INFINITY;
        }
        again = meet_any(far);
      }
      if (again) {  // (all warps)
        float top[2], alpha[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          top[i] = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
        over_warps(top, sh->top);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          alpha[i] = 1.0f;
          if (top[i] > m[i]) {
            // (by a whole power of two: o's factor is exact)
            const float up = m[i] == -INFINITY ? top[i] : m[i] + ceilf(top[i] - m[i]);
            alpha[i] = attn_exp2(m[i] - up);
            m[i] = up;
          }
          l[i] *= alpha[i];
        }
        form();
        if (kBytes) {
          float all[2] = {most[0], most[1]};
          over_warps(all, sh->most);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float now = ref[i] * alpha[i];
            ref[i] = all[i] >= 256.0f * now || kt == w.k0 ? pow2_floor(all[i]) : fmaxf(now, 0x1p-110f);
            alpha[i] = now * pow2_inverse(ref[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < kCols / 8; ++i) {
          o[i][0] *= alpha[0], o[i][1] *= alpha[0];
          o[i][2] *= alpha[1], o[i][3] *= alpha[1];
        }
        hand_over();
        ptx::named_barrier(1, 128);
      }
      l[0] += sum[0], l[1] += sum[1];
      if (!kBytes)
        ok = ptx::mbar_wait(&sh->full[v_slot], ((n + 1) / kSlots) & 1, abort, p.budget) && ok;
      // Behind the last position the slot holds what was there before: 0 in place
      // of values that may not be finite.
      const bool tail = KV != MOE_KV_INT8 && kt * 64 + 64 > w.s.len;
      const uint32_t tile = smem_at + v_slot * S::kTile;
      const auto keep_of = [&](int key) {  // of keys key + 2c, + 1
        const int over = w.s.len - (key + 2 * c);
        return over >= 2 ? 0xFFFFFFFFu : over == 1 ? 0x0000FFFFu : 0u;
      };
#pragma unroll
      for (int k = 0; k < 4; k += 2) {  // 32 keys
        uint32_t wf[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 x = weights[((kt & 1) * 4 + k + h) * 32 + lane];
          wf[h][0] = x.x, wf[h][1] = x.y, wf[h][2] = x.z, wf[h][3] = x.w;
        }
        if (kBytes) {
          const TileRows<S::kRow> rows16(16 * k + (lane >> 4) * 16, box);
#pragma unroll
          for (int j = 0; j < kCols / 16; ++j) {
            uint32_t b[4];  // keys 0-7, 8-15, 16-23, 24-31
            ldsm4_t(b, tile + rows16.at(row_v, warp * (kCols / 16) + j));
            if (tail) {
#pragma unroll
              for (int i = 0; i < 4; ++i) b[i] &= keep_of(kt * 64 + 16 * k + 8 * i);
            }
            uint32_t ev[4], od[4];  // of columns 2g, 2g + 1
#pragma unroll
            for (int i = 0; i < 4; ++i) codes_to_f16x2_apart<KV>(b[i], ev[i], od[i]);
            attn_mma<KV>(o[2 * j], wf[0], ev[0], ev[1]);
            attn_mma<KV>(o[2 * j + 1], wf[0], od[0], od[1]);
            attn_mma<KV>(o[2 * j], wf[1], ev[2], ev[3]);
            attn_mma<KV>(o[2 * j + 1], wf[1], od[2], od[3]);
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const TileRows<S::kRow> rows16(16 * (k + h), box);
#pragma unroll
            for (int j = 0; j < kCols / 16; ++j) {
              uint32_t b[4];
              ldsm4_t(b, tile + rows16.at(row_v, warp * (kCols / 8) + 2 * j + (lane >> 4)));
              if (tail) {
#pragma unroll
                for (int i = 0; i < 4; ++i) b[i] &= keep_of(kt * 64 + 16 * (k + h) + 8 * (i & 1));
              }
              attn_mma<KV>(o[2 * j], wf[h], b[0], b[1]);
              attn_mma<KV>(o[2 * j + 1], wf[h], b[2], b[3]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0 && ok) ptx::mbar_arrive(&sh->empty[v_slot]);
    }
    if (!ok && lane == 0) set_status(a.status, MOE_DEV_TIMEOUT);

    // ------------------------------------------------- the segment's end
    float total[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
      l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
      if (c == 0) sh->l[warp][g + 8 * i] = l[i];
    }
    ptx::named_barrier(1, 128);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i;
      total[i] = (sh->l[0][r] + sh->l[1][r]) + (sh->l[2][r] + sh->l[3][r]);
    }
    const bool whole = w.begins && w.ends;
    const int part = 2 * blockIdx.x + (w.begins ? 1 : 0);
    if (!whole && w.begins && threadIdx.x == 0) {
      AttnOpen d;
      d.last = static_cast<int>((w.tile_end - 1) / sh->share.per);
      d.rows = rows, d.start = w.s.start, d.row0 = row0, d.head = w.head;
      p.parts.open[blockIdx.x] = d;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = g + 8 * i;
      if (r >= rows) continue;
      if (!whole && warp == 0 && c == 0)
        p.parts.ml[static_cast<int64_t>(part) * R + r] = make_float2(m[i], total[i]);
      float f = whole ? 1.0f / total[i] : 1.0f;
      if (kBytes) f *= ref[i] * 0x1p-7f;
      moe_bf16 *dst = p.out + (w.s.start + pos[i] - ctx) * p.out_ld + out_row[i] * D;
#pragma unroll
      for (int j = 0; j < kCols / (kBytes ? 16 : 8); ++j) {
        if (kBytes) {
          const int d = warp * kCols + 16 * j + 4 * c;
          const float4 v = make_float4(o[2 * j][2 * i] * f, o[2 * j + 1][2 * i] * f,
                                       o[2 * j][2 * i + 1] * f, o[2 * j + 1][2 * i + 1] * f);
          if (whole)
            *reinterpret_cast<uint2 *>(dst + d) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
          else
            *reinterpret_cast<float4 *>(p.parts.at(part, D, d, r)) = v;
        } else {
          const int d = warp * kCols + 8 * j + 2 * c;
          const float x = o[j][2 * i] * f, y = o[j][2 * i + 1] * f;
          if (whole) *reinterpret_cast<uint32_t *>(dst + d) = pack_bf16(x, y);
          else
            *reinterpret_cast<float2 *>(p.parts.at(part, D, d, r) + (d & 2)) = make_float2(x, y);
        }
      }
    }
  }
}

}  // namespace moe
