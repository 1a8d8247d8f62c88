// attn_stream.cuh -- attention of few rows (single tokens, drafts) over long
// contexts: the cache streams through, bound by its bytes.
//
// out = softmax(scale q k^T) v for a tile of R = 16 WR rows, in one pass over
// the keys with the running maximum m and total l of the softmax.  A block has
// four warps that compute, and one that fetches: WR of them take 16 rows each,
// WK = 4 / WR share out the 64 keys of a key tile among themselves (so that
// with up to 16 rows no key is read twice from shared memory).  Each keeps its
// own m, l and sums; they are joined when the segment ends.  K and V tiles
// come through a ring of shared-memory slots (TMA, 128-byte swizzle, one box a
// page); products are mma.sync m16n8k16 with fp32 sums.
//
// 8-bit codes are made fp16 in registers, exactly; q then takes a power of two
// a row (fp16 keeps all of bf16's digits within 2^-28 of the row's largest).
// A key's scale multiplies its column of q k^T; a value's scale multiplies its
// weight, and the products t = p s_v enter as fp16 under a power of two a row
// that follows their running maximum, so that they keep 11 digits whatever the
// scales are.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include "attn_args.cuh"
#include "delta_mma.cuh"
#include "early.cuh"
#include "sm100_ptx.cuh"

namespace moe {

constexpr int kStreamTileCost = 1;  // beginning and ending a tile, in key tiles

template <int D, int KV, int WR>
struct StreamShape {
  static constexpr int kWK = 4 / WR, kR = 16 * WR, kKT = 64, kNK = kKT / kWK;
  static constexpr bool kBytes = KV != MOE_KV_BF16;  // 8-bit codes
  static constexpr int kRow = D * (kBytes ? 1 : 2);  // bytes of a cached row
  static constexpr int kTile = kKT * kRow;
  static constexpr int kSteps = D / 16;
  static constexpr int kThreads = 160;
  // the rows' fragments of q; reused when the warps' sums are joined
  static constexpr int kQ = kR * D * 2;
  static constexpr int kJoinCols = kQ >= 64 * 64 * 4 ? 64 : 32;  // at a time
  static constexpr int kJoin = kWK == 1 ? 0 : 64 * kJoinCols * 4;
  static constexpr int kQArea = kQ > kJoin ? kQ : kJoin;
  // two blocks an SM where that leaves three slots, else one
  static constexpr int kFixed = kQArea + 2048;  // + barriers, m and l, the share
  static constexpr int kHalf = (233472 / 2 - 1024 - kFixed) / (kTile + 256);
  static constexpr int kWhole = (232448 - kFixed) / (kTile + 256);
  static constexpr int kBlocks = kHalf >= 3 ? 2 : 1;
  static constexpr int kFit = kBlocks == 2 ? kHalf : kWhole;
  static constexpr int kSlots = kFit > 12 ? 12 : kFit;
  static constexpr int kSmem = kFixed + kSlots * (kTile + 256);
  static_assert(kSlots >= 3, "ring");
};

struct StreamSmem {  // behind the slots, their scales and the q area
  uint64_t full[12], empty[12];
  AttnShare share;
  float m[64], l[64], qmax[64];
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

template <int D, int KV, int WR>
__global__ void __launch_bounds__(160, (StreamShape<D, KV, WR>::kBlocks))
attn_stream_kernel(const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const AttnBatch a, const AttnRange range,
                   const AttnArgs p) {
  using S = StreamShape<D, KV, WR>;
  constexpr int kSlots = S::kSlots, kWK = S::kWK, R = S::kR, kNK = S::kNK, kSteps = S::kSteps;
  constexpr bool kBytes = S::kBytes;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *q_area = smem + kSlots * S::kTile;
  float *scales = reinterpret_cast<float *>(q_area + S::kQArea);
  StreamSmem *sh = reinterpret_cast<StreamSmem *>(scales + kSlots * 64);
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
      int page_of = 0;                              // lane i's box of the 32 fetched next
      for (int i = 0; i < tiles && !stop; ++i) {
        const int b0 = (w.k0 + i) * per_tile;
        if ((i * per_tile) % 32 == 0) {
          const int bx = b0 + lane;
          page_of = 0;
          if (bx < boxes && bx < w.k1 * per_tile) {
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
          if (!ptx::mbar_wait(&sh->empty[slot], ((n / kSlots) & 1) ^ 1, abort, p.budget)) {
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
                        (kv ? p.v_scale : p.k_scale) + row, box * 4, &sh->full[slot]);
          }
        }
      }
    }
    if (*abort) {  // let the copies in flight land before exiting
      if (lane == 0) {
        set_status(a.status, MOE_DEV_TIMEOUT);
        int never = 0;
        for (uint32_t k = 0; k < kSlots && k < n; ++k) {
          const uint32_t j = n - 1 - k;
          ptx::mbar_wait(&sh->full[j % kSlots], (j / kSlots) & 1, &never, ptx::kDrainBudgetNs);
        }
      }
      __syncwarp();
    }
    return;
  }

  // ------------------------------------------------------------- compute
  const int wr = warp / kWK, wk = warp % kWK;
  const int g = lane >> 2, c = lane & 3;
  uint4 *qf = reinterpret_cast<uint4 *>(q_area) + wr * kSteps * 32;
  float *join = reinterpret_cast<float *>(q_area);
  uint32_t n = 0;
  const uint32_t smem_at = ptx::smem_u32(smem);
  // ldmatrix rows: lane l gives row l % 8 of block l / 8
  const int row_k = (lane & 7) + (kBytes ? ((lane >> 3) & 1) : (lane >> 4)) * 8;
  const int col_k = kBytes ? lane >> 4 : (lane >> 3) & 1;
  const int row_v = (lane & 7) + ((lane >> 3) & 1) * 8, col_v = lane >> 4;

  while (w.next(a, range)) {
    const int row0 = w.cur * R;
    const int rows = min(w.t.rows - row0, R);
    const int ctx = w.t.ctx;
    // this thread's two rows
    int pos[2];
    float factor[2];
    bool live[2];
    {
      const moe_bf16 *src[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = wr * 16 + g + 8 * i;
        live[i] = r < rows;
        const int at = row0 + (live[i] ? r : rows - 1);
        const int token = at / a.group, h = at % a.group;
        pos[i] = ctx + token;
        src[i] = p.q + (w.s.start + token) * p.q_ld + (w.head * a.group + h) * D;
        factor[i] = p.scale_log2;
      }
      constexpr int kMine = (kSteps + kWK - 1) / kWK;
      uint4 f[kMine];
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        const int ks = j * kWK + wk;
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
      ptx::named_barrier(1, 128);  // the q area and the maxima are free
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
          if (c == 0) sh->qmax[wk * R + wr * 16 + g + 8 * i] = top[i];
        }
        if (kWK > 1) {
          ptx::named_barrier(1, 128);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            for (int k = 0; k < kWK; ++k)
              top[i] = fmaxf(top[i], sh->qmax[k * R + wr * 16 + g + 8 * i]);
        }
        float mult[2], inv;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
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
#pragma unroll
      for (int j = 0; j < kMine; ++j) qf[(j * kWK + wk) * 32 + lane] = f[j];
      ptx::named_barrier(1, 128);
    }
    const int first_pos = ctx + row0 / a.group;
    const int last_pos = ctx + (row0 + rows - 1) / a.group;

    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    float ref[2] = {0x1p-110f, 0x1p-110f};  // (8-bit) powers of two: o's sums times ref / 2^13

    bool ok = true;
    for (int kt = w.k0; kt < w.k1; ++kt, n += 2) {
      const int key0 = kt * 64 + wk * kNK;
      const bool active = key0 <= last_pos &&
                          (!a.window || key0 + kNK > first_pos - a.window + 1);
      float s[kNK / 8][4];
      {
        const uint32_t slot = n % kSlots;
        if (!(ok = ptx::mbar_wait(&sh->full[slot], (n / kSlots) & 1, abort, p.budget))) break;
        if (active) {
          const uint32_t tile = smem_at + slot * S::kTile;
#pragma unroll
          for (int i = 0; i < kNK / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
#pragma unroll
          for (int k16 = 0; k16 < kNK / 16; ++k16) {
            const TileRows<S::kRow> rows16(wk * kNK + k16 * 16, box);
#pragma unroll
            for (int ks = 0; ks < kSteps; ks += kBytes ? 2 : 1) {
              uint32_t b[4];
              if (kBytes) {
                ldsm4(b, tile + rows16.at(row_k, ks + col_k));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint4 qv = qf[(ks + h) * 32 + lane];
                  const uint32_t av[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    uint32_t lo, hi;
                    codes_to_f16x2<KV>(b[2 * h + i], lo, hi);
                    attn_mma<KV>(s[2 * k16 + i], av, lo, hi);
                  }
                }
              } else {
                ldsm4(b, tile + rows16.at(row_k, 2 * ks + col_k));
                const uint4 qv = qf[ks * 32 + lane];
                const uint32_t av[4] = {qv.x, qv.y, qv.z, qv.w};
                attn_mma<KV>(s[2 * k16], av, b[0], b[1]);
                attn_mma<KV>(s[2 * k16 + 1], av, b[2], b[3]);
              }
            }
          }
          if (kBytes) {
            const float *ksc = scales + slot * 64 + wk * kNK + 2 * c;
#pragma unroll
            for (int i = 0; i < kNK / 8; ++i) {
              const float2 f = *reinterpret_cast<const float2 *>(ksc + 8 * i);
              s[i][0] *= factor[0] * f.x, s[i][1] *= factor[0] * f.y;
              s[i][2] *= factor[1] * f.x, s[i][3] *= factor[1] * f.y;
            }
          } else {
#pragma unroll
            for (int i = 0; i < kNK / 8; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) s[i][j] *= factor[0];
          }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sh->empty[slot]);
      }
      const bool edge = key0 + kNK > first_pos + 1 ||
                        (a.window && key0 <= last_pos - a.window);
      const uint32_t slot = (n + 1) % kSlots;
      uint32_t pf[kNK / 16][4];
      if (active) {
        if (edge) {
#pragma unroll
          for (int i = 0; i < kNK / 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int key = key0 + 8 * i + 2 * c + (j & 1), ps = pos[j >> 1];
              if (key > ps || (a.window && key <= ps - a.window)) s[i][j] = -INFINITY;
            }
        }
        float top[2] = {-INFINITY, -INFINITY}, alpha[2], base[2];
#pragma unroll
        for (int i = 0; i < kNK / 8; ++i) {
          top[0] = fmaxf(top[0], fmaxf(s[i][0], s[i][1]));
          top[1] = fmaxf(top[1], fmaxf(s[i][2], s[i][3]));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 1));
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], 2));
          top[i] = fmaxf(top[i], m[i]);
          base[i] = top[i] == -INFINITY ? 0.0f : top[i];
          alpha[i] = attn_exp2(m[i] - base[i]);
          m[i] = top[i];
          l[i] *= alpha[i];
        }
#pragma unroll
        for (int i = 0; i < kNK / 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[i][j] = attn_exp2(s[i][j] - base[j >> 1]);
            l[j >> 1] += s[i][j];
          }
        if (!kBytes) {
#pragma unroll
          for (int i = 0; i < kNK / 16; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              pf[i][j] = bf16x2(s[2 * i + (j >> 1)][2 * (j & 1)], s[2 * i + (j >> 1)][2 * (j & 1) + 1]);
        }
        if (!(ok = ptx::mbar_wait(&sh->full[slot], ((n + 1) / kSlots) & 1, abort, p.budget))) break;
        if (kBytes) {
          const float *vsc = scales + slot * 64 + wk * kNK + 2 * c;
          float most[2] = {0.0f, 0.0f};
#pragma unroll
          for (int i = 0; i < kNK / 8; ++i) {
            const float2 f = *reinterpret_cast<const float2 *>(vsc + 8 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              // a hidden key's weight is 0 whatever its scale
              s[i][j] = s[i][j] == 0.0f ? 0.0f : s[i][j] * ((j & 1) ? f.y : f.x);
              most[j >> 1] = fmaxf(most[j >> 1], s[i][j]);
            }
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            most[i] = fmaxf(most[i], __shfl_xor_sync(0xFFFFFFFFu, most[i], 1));
            most[i] = fmaxf(most[i], __shfl_xor_sync(0xFFFFFFFFu, most[i], 2));
            const float up = pow2_floor(fmaxf(ref[i] * alpha[i], most[i]));
            const float inv = pow2_inverse(up);
            alpha[i] = alpha[i] * ref[i] * inv;  // (in this order: at most 2)
            ref[i] = up;
            base[i] = inv * 0x1p13f;
          }
#pragma unroll
          for (int i = 0; i < kNK / 16; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float f = base[j & 1];
              pf[i][j] = h2_bits(__floats2half2_rn(s[2 * i + (j >> 1)][2 * (j & 1)] * f,
                                                   s[2 * i + (j >> 1)][2 * (j & 1) + 1] * f));
            }
        }
        if (__any_sync(0xFFFFFFFFu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[i][0] *= alpha[0], o[i][1] *= alpha[0];
            o[i][2] *= alpha[1], o[i][3] *= alpha[1];
          }
        }
        // Behind the last position the slot holds what was there before: 0 in
        // place of values that may not be finite.
        const bool tail = KV != MOE_KV_INT8 && key0 + kNK > w.s.len;
        const uint32_t tile = smem_at + slot * S::kTile;
#pragma unroll
        for (int k16 = 0; k16 < kNK / 16; ++k16) {
          const TileRows<S::kRow> rows16(wk * kNK + k16 * 16, box);
          uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};  // of keys 2c, 2c + 1; 8 on
          if (tail) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int over = w.s.len - (key0 + k16 * 16 + 8 * h + 2 * c);  // keys there
              keep[h] = over >= 2 ? 0xFFFFFFFFu : over == 1 ? 0x0000FFFFu : 0u;
            }
          }
#pragma unroll
          for (int j = 0; j < D / (kBytes ? 32 : 16); ++j) {
            uint32_t b[4];
            ldsm4_t(b, tile + rows16.at(row_v, 2 * j + col_v));
            if (tail) b[0] &= keep[0], b[1] &= keep[1], b[2] &= keep[0], b[3] &= keep[1];
            if (kBytes) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                // b[2h]: keys 2c, 2c + 1 of columns 2g, 2g + 1
                uint32_t e0, o0, e1, o1;
                codes_to_f16x2_apart<KV>(b[2 * h], e0, o0);
                codes_to_f16x2_apart<KV>(b[2 * h + 1], e1, o1);
                attn_mma<KV>(o[4 * j + 2 * h], pf[k16], e0, e1);
                attn_mma<KV>(o[4 * j + 2 * h + 1], pf[k16], o0, o1);
              }
            } else {
              attn_mma<KV>(o[2 * j], pf[k16], b[0], b[1]);
              attn_mma<KV>(o[2 * j + 1], pf[k16], b[2], b[3]);
            }
          }
        }
      } else {
        if (!(ok = ptx::mbar_wait(&sh->full[slot], ((n + 1) / kSlots) & 1, abort, p.budget))) break;
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sh->empty[slot]);
    }
    // (a wait that gave up: every wait from here on does so at once, and the
    // block still meets at its barriers)
    if (!ok && lane == 0) set_status(a.status, MOE_DEV_TIMEOUT);

    // ------------------------------------------------- the segment's end
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
      l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
      if (kBytes) {
        const float f = ref[i] * 0x1p-13f;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[j][2 * i] *= f, o[j][2 * i + 1] *= f;
      }
    }
    const bool whole = w.begins && w.ends;
    const int part = 2 * blockIdx.x + (w.begins ? 1 : 0);
    if (!whole && w.begins && threadIdx.x == 0) {
      AttnOpen d;
      d.last = static_cast<int>((w.tile_end - 1) / sh->share.per);
      d.rows = rows, d.start = w.s.start, d.row0 = row0, d.head = w.head;
      p.parts.open[blockIdx.x] = d;
    }
    const auto out_at = [&](int r) {  // row r of the tile
      const int token = (row0 + r) / a.group, h = (row0 + r) % a.group;
      return p.out + (w.s.start + token) * p.out_ld + (w.head * a.group + h) * D;
    };
    const auto part_at = [&](int r, int d) { return p.parts.at(part, D, d, r); };
    float2 *part_ml = p.parts.ml + static_cast<int64_t>(part) * p.parts.rows;
    if (kWK == 1) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = wr * 16 + g + 8 * i;
        if (!live[i]) continue;
        const float f = whole ? 1.0f / l[i] : 1.0f;
        moe_bf16 *dst = out_at(r);
        if (!whole && c == 0) part_ml[r] = make_float2(m[i], l[i]);
#pragma unroll
        for (int j = 0; j < D / (kBytes ? 16 : 8); ++j) {
          if (kBytes) {
            const float4 v = make_float4(o[2 * j][2 * i] * f, o[2 * j + 1][2 * i] * f,
                                         o[2 * j][2 * i + 1] * f, o[2 * j + 1][2 * i + 1] * f);
            const int d = 16 * j + 4 * c;
            if (whole)
              *reinterpret_cast<uint2 *>(dst + d) = make_uint2(bf16x2(v.x, v.y), bf16x2(v.z, v.w));
            else
              *reinterpret_cast<float4 *>(part_at(r, d)) = v;
          } else {
            const int d = 8 * j + 2 * c;
            const float x = o[j][2 * i] * f, y = o[j][2 * i + 1] * f;
            if (whole) *reinterpret_cast<uint32_t *>(dst + d) = bf16x2(x, y);
            else *reinterpret_cast<float2 *>(part_at(r, d) + (d & 2)) = make_float2(x, y);
          }
        }
      }
    } else {
      constexpr int kCols = S::kJoinCols;
      if (c == 0)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sh->m[wk * R + wr * 16 + g + 8 * i] = m[i];
          sh->l[wk * R + wr * 16 + g + 8 * i] = l[i];
        }
      ptx::named_barrier(1, 128);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = wr * 16 + g + 8 * i;
        float top = -INFINITY;
        for (int k = 0; k < kWK; ++k) top = fmaxf(top, sh->m[k * R + r]);
        const float f = top == -INFINITY ? 0.0f : attn_exp2(m[i] - top);
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[j][2 * i] *= f, o[j][2 * i + 1] *= f;
      }
      // each thread joins 16 WR kCols / 128 columns of one row at a time
      constexpr int kEach = R * kCols / 128;
      const int r = threadIdx.x * kEach / kCols, d0 = threadIdx.x * kEach % kCols;
      float top = -INFINITY, total = 0.0f;
      for (int k = 0; k < kWK; ++k) top = fmaxf(top, sh->m[k * R + r]);
      for (int k = 0; k < kWK; ++k)
        total += sh->l[k * R + r] * (top == -INFINITY ? 0.0f : attn_exp2(sh->m[k * R + r] - top));
      if (!whole && d0 == 0 && r < rows) part_ml[r] = make_float2(top, total);
      const float f = whole ? 1.0f / total : 1.0f;
      moe_bf16 *dst = r < rows ? out_at(r) : nullptr;
#pragma unroll
      for (int d = 0; d < D; d += kCols) {
        float *mine = join + (wk * R + wr * 16) * kCols;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int j = 0; j < kCols / (kBytes ? 16 : 8); ++j) {
            const int at = (g + 8 * i) * kCols;
            if (kBytes) {
              const int jj = d / 16 + j;
              *reinterpret_cast<float4 *>(mine + at + 16 * j + 4 * c) =
                  make_float4(o[2 * jj][2 * i], o[2 * jj + 1][2 * i], o[2 * jj][2 * i + 1],
                              o[2 * jj + 1][2 * i + 1]);
            } else {
              const int jj = d / 8 + j;
              *reinterpret_cast<float2 *>(mine + at + 8 * j + 2 * c) =
                  make_float2(o[jj][2 * i], o[jj][2 * i + 1]);
            }
          }
        }
        ptx::named_barrier(1, 128);
        if (r < rows) {
#pragma unroll
          for (int e = 0; e < kEach; e += 4) {
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < kWK; ++k) {
              const float4 x =
                  *reinterpret_cast<const float4 *>(join + (k * R + r) * kCols + d0 + e);
              v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
            }
            if (whole)
              *reinterpret_cast<uint2 *>(dst + d + d0 + e) =
                  make_uint2(bf16x2(v.x * f, v.y * f), bf16x2(v.z * f, v.w * f));
            else
              *reinterpret_cast<float4 *>(part_at(r, d + d0 + e)) = v;
          }
        }
        if (d + kCols < D) ptx::named_barrier(1, 128);
      }
    }
  }
}

}  // namespace moe
