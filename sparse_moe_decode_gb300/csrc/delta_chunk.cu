// delta_chunk.cu -- the gated delta rule over prompts, 64 tokens at a time.
//
// Within a chunk that starts from state S (rows = value channels, columns =
// key channels), with G the running sum of g, gamma_i = e^{G_i} and
// Gamma_ij = e^{G_i - G_j}:
//   u_i = beta_i (v_i - gamma_i S k_i) - sum_{j<i} beta_i Gamma_ij (k_i.k_j) u_j
//   o_i = gamma_i S q_i + sum_{j<=i} Gamma_ij (q_i.k_j) u_j
//   S' = gamma_64 S + sum_j Gamma_64,j u_j k_j^T.
// The first line is a unit lower-triangular system: u = T x with T = (I + L)^-1.
//
// Two kernels.  delta_prep_kernel, one CTA per (chunk, value head), forms
// what does not depend on the state: T, the masked q.k products P, the
// decays, and k and q as fp16.  delta_chain_kernel walks a sequence's chunks
// with the state in registers: a warp owns 16 state rows (all of their
// columns), and the three products of its chain -- S k^T, T x, u k^T -- hand
// their results on as the next one's A operand without leaving the warp's
// registers (an accumulator fragment of mma.sync m16n8 is an A fragment of
// the next k16 step), so that no barrier lies on the chain.  A second warp
// per 16 rows forms the outputs from copies of the operands.  mma.sync
// rather than tcgen05: the chain is bound by its dependent steps, and a
// round trip of each through tensor memory costs more than the products.
//
// Precision.  k and q are bf16: scaled by a power of two per token they are
// exact in fp16 (elements within 2^29 of the token's largest).  S, x, u and T
// are fp32 and enter the products as two fp16 terms under a power-of-two
// scale per row, 22 bits; products accumulate in fp32 and the state is summed
// in fp32 registers.  The outputs, which are rounded to bf16 once, take P, S
// and u as single fp16 terms (2^-11, an eighth of the rounding to come).
#include <cuda_runtime.h>

#include <atomic>

#include "common.cuh"
#include "delta_mma.cuh"
#include "delta_seq.cuh"
#include "kernels.h"
#include "mixer.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kC = 64;  // tokens per chunk
constexpr int kTile = kC * kC * 2;  // bytes of a 64 x 64 fp16 tile
// Per (chunk, value head): T's two terms, P, then vectors of 64 fp32.
enum { kVecC, kVecBeta, kVecT, kVecD, kVecO, kVecP, kVecMisc, kVecs };
constexpr int kHeadBlob = 3 * kTile + kVecs * kC * 4;
constexpr int kHeader = 256;      // status word, flags
constexpr int kFlagWord = 16;     // header word: some bound of the call is bad
constexpr int kPrepThreads = 256;

template <int DK>
constexpr int kKeyBlob = 2 * kC * DK * 2;  // per (chunk, key head): k, then q, as fp16

// Tiles of fp16 in 16-byte pieces, rows of COLS values; a row's pieces are
// permuted within groups of eight by its number, so that eight rows' pieces of
// one column lie in different banks.
template <int COLS>
__device__ __forceinline__ uint32_t tile_at(int row, int piece) {
  return static_cast<uint32_t>(row * COLS * 2 + ((piece ^ (row & 7)) << 4));
}

// Sequence b's first chunk slot: chunks of different sequences never share
// one, whatever the lengths.
__device__ __forceinline__ int slot_base(const DeltaSeqs &s, int b) {
  return (s.cu_seqlens ? s.cu_seqlens[b] : b * s.T) / kC + b;
}

// ------------------------------------------------------------------- prep

constexpr int kTLd = kC + 4;  // row stride of T

// T's rows have room for four values beside them: the tokens' factors.
enum { kGLo = kC, kKappa, kRho };

template <int DK>
struct PrepSmem {
  alignas(128) uint8_t key[kKeyBlob<DK>];
  // L (fp32, permuted) until T's two terms replace it; P; the vectors, of
  // which kVecT holds the sums of g until T's scales replace them
  alignas(128) uint8_t head[kHeadBlob];
  float t[kC * kTLd];  // T; blocks of 16 above the diagonal are never touched
};

// Where L(i, j) lies: pieces of four columns permuted by the row, so that
// eight rows' pieces of one column lie in different banks.
__device__ __forceinline__ int l_at(int i, int j) { return i * kC + (j ^ ((i & 7) << 2)); }

// The power of two that brings a token's values below 2^15 (bounded by their
// 2-norm), and its inverse: their bf16 digits are exact in fp16 down to 2^-25
// of the norm and off by 2^-39 of it below that.
__device__ __forceinline__ void token_scale(float ss, float &mult, float &inv) {
  const int e = static_cast<int>((__float_as_uint(ss) >> 23) & 255u);
  const int m = 142 - ((e - 125) >> 1);  // 127 + 15 - ceil((e - 126) / 2)
  mult = __uint_as_float(static_cast<uint32_t>(m) << 23);
  inv = __uint_as_float(static_cast<uint32_t>(254 - m) << 23);
}

// A 16 x 8 tile (rows r0, columns c0) of A B over k in [k0, k1): fp32 values
// as two tf32 terms each, three products.
template <class FA, class FB>
__device__ __forceinline__ void product(float (&acc)[4], int r0, int c0, int k0, int k1, FA a_of,
                                        FB b_of, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = 0.0f;
  for (int k = k0; k < k1; k += 8) {
    uint32_t ah[4], al[4], bh[2], bl[2];
    split_tf32(a_of(r0 + g, k + t), ah[0], al[0]);
    split_tf32(a_of(r0 + g + 8, k + t), ah[1], al[1]);
    split_tf32(a_of(r0 + g, k + t + 4), ah[2], al[2]);
    split_tf32(a_of(r0 + g + 8, k + t + 4), ah[3], al[3]);
    split_tf32(b_of(k + t, c0 + g), bh[0], bl[0]);
    split_tf32(b_of(k + t + 4, c0 + g), bh[1], bl[1]);
    mma8(acc, ah, bl[0], bl[1]);
    mma8(acc, al, bh[0], bh[1]);
    mma8(acc, ah, bh[0], bh[1]);
  }
}

// One CTA per chunk and key head, for `heads` of the value heads that read
// it.  Warps 0..3 take k (k k^T, L, T's diagonal blocks), warps 4..7 take q
// (q k^T, P), 16 tokens each.
template <int DK>
__global__ void __launch_bounds__(kPrepThreads, 3)
delta_prep_kernel(moe_delta_dims d, moe_delta_inputs in, DeltaSeqs seq, int heads, uint8_t *ws,
                  uint8_t *ws_key, uint8_t *ws_head) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  PrepSmem<DK> &sm = *reinterpret_cast<PrepSmem<DK> *>(smem_raw);
  __shared__ float red[kPrepThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ratio = d.v_heads / d.qk_heads;
  const int slot = blockIdx.x, h0 = blockIdx.y * heads, hk = h0 / ratio;

  if (slot == 0 && h0 == 0) {
    // one CTA looks at every bound: a call with a bad one does nothing
    bool bad = false;
    if (seq.cu_seqlens)
      for (int b = tid; b < seq.B; b += kPrepThreads) {
        const int lo = seq.cu_seqlens[b], hi = seq.cu_seqlens[b + 1];
        bad |= lo < 0 || lo > hi || hi > seq.N;
      }
    bad = __syncthreads_or(bad);
    if (tid == 0) {
      reinterpret_cast<uint32_t *>(ws)[kFlagWord] = bad;
      if (bad) set_status(seq.status, MOE_DEV_BAD_INDEX);
    }
  }

  // whose chunk this is: the last sequence whose slots start at or before it
  int lo = 0, hi = seq.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (slot_base(seq, mid) <= slot) lo = mid;
    else hi = mid;
  }
  const DeltaSeqRange r = delta_seq_range(seq, lo);
  const int chunk = slot - slot_base(seq, lo);
  if (!r.ok || chunk < 0 || chunk >= (r.len + kC - 1) / kC) return;
  const int left = min(kC, r.len - chunk * kC);  // tokens of this chunk
  const int64_t row0 = static_cast<int64_t>(r.start) + chunk * kC;

  const int w = warp & 3;          // this warp's 16 tokens
  const bool is_q = warp >= 4;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t kt = ptx::smem_u32(sm.key);

  // k and q: scaled to fp16, and the tokens' factors.  Eight lanes a row.
  {
    constexpr int kPieces = DK / 64;  // 16-byte pieces of a lane
    const moe_bf16 *src = is_q ? in.q : in.k;
    const int64_t ld = is_q ? in.q_ld : in.k_ld;
    const int piece = lane & 7;
    uint4 raw[4][kPieces];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int i = 16 * w + 4 * p + (lane >> 3);
#pragma unroll
      for (int e = 0; e < kPieces; ++e)
        raw[p][e] = i < left ? *reinterpret_cast<const uint4 *>(src + (row0 + i) * ld + hk * DK +
                                                                (piece + 8 * e) * 8)
                             : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int i = 16 * w + 4 * p + (lane >> 3);
      float2 x[kPieces][4], sum = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int e = 0; e < kPieces; ++e) {
        const uint32_t u[4] = {raw[p][e].x, raw[p][e].y, raw[p][e].z, raw[p][e].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[e][j] = make_float2(bf16_lo(u[j]), bf16_hi(u[j]));
          sum = fma2(x[e][j], x[e][j], sum);
        }
      }
      float ss = sum.x + sum.y;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
      float mult, inv;
      token_scale(ss, mult, inv);
#pragma unroll
      for (int e = 0; e < kPieces; ++e) {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = h2_bits(__float22half2_rn(mul2(x[e][j], make_float2(mult, mult))));
        *reinterpret_cast<uint4 *>(sm.key + (is_q ? kKeyBlob<DK> / 2 : 0) +
                                   tile_at<DK>(i, piece + 8 * e)) =
            make_uint4(o[0], o[1], o[2], o[3]);
      }
      if (d.qk_norm) inv = inv / sqrtf(ss + d.qk_eps);
      if (is_q) inv *= d.scale;
      if (piece == 0) sm.t[i * kTLd + (is_q ? kRho : kKappa)] = i < left ? inv : 0.0f;
    }
  }
  __syncthreads();

  // rows of k k^T or q k^T: the tiles left of the diagonal block, and its two
  float off[6][4] = {}, dia[2][4] = {};
  {
    const uint32_t at = kt + (is_q ? kKeyBlob<DK> / 2 : 0);
    const int b_row = (lane & 7) + ((lane >> 4) << 3), b_piece = (lane >> 3) & 1;
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) {
      uint32_t a[4], b[4];
      ldsm4(a, at + tile_at<DK>(16 * w + (lane & 15), 2 * s + (lane >> 4)));
      ldsm4(b, kt + tile_at<DK>(16 * w + b_row, 2 * s + b_piece));
      mma16(dia[0], a, b[0], b[1]);
      mma16(dia[1], a, b[2], b[3]);
#pragma unroll
      for (int np = 0; np < 3; ++np)
        if (np < w) {
          ldsm4(b, kt + tile_at<DK>(16 * np + b_row, 2 * s + b_piece));
          mma16(off[2 * np], a, b[0], b[1]);
          mma16(off[2 * np + 1], a, b[2], b[3]);
        }
    }
  }

  float *vec = reinterpret_cast<float *>(sm.head + 3 * kTile);
  float *ghi = vec + kVecT * kC;
  float *L = reinterpret_cast<float *>(sm.head);
  float *T = sm.t;
  for (int hh = 0; hh < heads; ++hh) {
    const int h = h0 + hh;
    // Decays: sums of g in fp64, in units of log 2, kept as two fp32 terms, so
    // that differences of large sums keep their digits.
    if (warp == 4) {
      const int i = 2 * lane;
      double g0 = 0.0, g1 = 0.0;
      float be0 = 0.0f, be1 = 0.0f;
      if (i < left) {
        g0 = delta_log_decay(in.g[(row0 + i) * in.g_ld + h]);
        be0 = in.beta[(row0 + i) * in.beta_ld + h];
      }
      if (i + 1 < left) {
        g1 = delta_log_decay(in.g[(row0 + i + 1) * in.g_ld + h]);
        be1 = in.beta[(row0 + i + 1) * in.beta_ld + h];
      }
      double sum = g0 + g1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double up = __shfl_up_sync(kFull, sum, o);
        if (lane >= o) sum += up;
      }
      const double kLog2E = 1.4426950408889634;
      const double second = sum * kLog2E, first = (sum - g1) * kLog2E;
      const double total = __shfl_sync(kFull, second, 31);
      const float2 sh = make_float2(static_cast<float>(first), static_cast<float>(second));
      const float2 kap = make_float2(T[i * kTLd + kKappa], T[(i + 1) * kTLd + kKappa]);
      const float2 rho = make_float2(T[i * kTLd + kRho], T[(i + 1) * kTLd + kRho]);
      const float2 gamma = make_float2(exp2f(sh.x), exp2f(sh.y));
      *reinterpret_cast<float2 *>(ghi + i) = sh;
      T[i * kTLd + kGLo] = static_cast<float>(first - sh.x);
      T[(i + 1) * kTLd + kGLo] = static_cast<float>(second - sh.y);
      *reinterpret_cast<float2 *>(vec + kVecBeta * kC + i) = make_float2(be0, be1);
      *reinterpret_cast<float2 *>(vec + kVecC * kC + i) =
          make_float2(-be0 * gamma.x * kap.x, -be1 * gamma.y * kap.y);
      *reinterpret_cast<float2 *>(vec + kVecO * kC + i) =
          make_float2(rho.x * gamma.x, rho.y * gamma.y);
      // the update's factors, Gamma_64,j kappa_j, over a power of two above
      // the largest
      float2 dd = make_float2(exp2f(static_cast<float>(total - first)) * kap.x,
                              exp2f(static_cast<float>(total - second)) * kap.y);
      float dmax = fmaxf(dd.x, dd.y);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dmax = fmaxf(dmax, __shfl_xor_sync(kFull, dmax, o));
      float up, down;
      pow2_above(dmax, up, down);
      *reinterpret_cast<float2 *>(vec + kVecD * kC + i) = make_float2(dd.x * down, dd.y * down);
      if (lane == 0) {
        vec[kVecMisc * kC] = exp2f(static_cast<float>(total));  // gamma_64
        vec[kVecMisc * kC + 2] = up;
      }
    }
    __syncthreads();

    // L = beta_i kappa_i Gamma_ij kappa_j k_i.k_j below the diagonal, P =
    // rho_i Gamma_ij kappa_j q_i.k_j up to it.  Left of the diagonal block
    // Gamma_ij = e^{G_i - G_r} e^{G_r - G_j} about the block's first token r:
    // both factors are decays, and the product underflows only where Gamma does.
    {
      const int ref = 16 * w, i0 = ref + g, i1 = i0 + 8;
      const float rh = ghi[ref], rl = T[ref * kTLd + kGLo];
      const float h0r = ghi[i0], l0r = T[i0 * kTLd + kGLo], h1r = ghi[i1],
                  l1r = T[i1 * kTLd + kGLo];
      float f0, f1;
      if (is_q) {
        f0 = T[i0 * kTLd + kRho], f1 = T[i1 * kTLd + kRho];
      } else {
        f0 = vec[kVecBeta * kC + i0] * T[i0 * kTLd + kKappa];
        f1 = vec[kVecBeta * kC + i1] * T[i1 * kTLd + kKappa];
      }
      const float a0 = f0 * exp2f((h0r - rh) + (l0r - rl));
      const float a1 = f1 * exp2f((h1r - rh) + (l1r - rl));
      // P's row scale from norms: by their scales k and q stay below 2^15, so
      // |P_ij| <= rho_i max kappa 2^30, which goes to 2^11 or less (room for
      // decays that grow by up to 2^5).
      float s0 = 1.0f, s1 = 1.0f;
      if (is_q) {
        float kmax = fmaxf(T[lane * kTLd + kKappa], T[(lane + 32) * kTLd + kKappa]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) kmax = fmaxf(kmax, __shfl_xor_sync(kFull, kmax, o));
        float up0, up1;
        pow2_above(fabsf(f0) * kmax, up0, s0);
        pow2_above(fabsf(f1) * kmax, up1, s1);
        s0 *= 0x1p-19f, s1 *= 0x1p-19f;
        if (t == 0) vec[kVecP * kC + i0] = up0 * 0x1p19f, vec[kVecP * kC + i1] = up1 * 0x1p19f;
      }
      uint8_t *P = sm.head + 2 * kTile + 4 * t;
      // one tile: eight columns from `col` of this warp's rows
      const auto put_tile = [&](int col, float2 top, float2 low) {
        if (is_q) {
          *reinterpret_cast<__half2 *>(P + tile_at<kC>(i0, col / 8)) =
              __float22half2_rn(mul2(top, make_float2(s0, s0)));
          *reinterpret_cast<__half2 *>(P + tile_at<kC>(i1, col / 8)) =
              __float22half2_rn(mul2(low, make_float2(s1, s1)));
        } else {
          *reinterpret_cast<float2 *>(L + l_at(i0, col + 2 * t)) = top;
          *reinterpret_cast<float2 *>(L + l_at(i1, col + 2 * t)) = low;
        }
      };
#pragma unroll
      for (int n = 0; n < 6; ++n) {
        if (n < 2 * w) {
          const int j = 8 * n + 2 * t;
          const float2 gj = *reinterpret_cast<const float2 *>(ghi + j);
          const float *tj = T + j * kTLd;
          const float2 col =
              make_float2(tj[kKappa] * exp2f((rh - gj.x) + (rl - tj[kGLo])),
                          tj[kTLd + kKappa] * exp2f((rh - gj.y) + (rl - tj[kTLd + kGLo])));
          put_tile(8 * n, mul2(make_float2(off[n][0], off[n][1]), mul2(col, make_float2(a0, a0))),
                   mul2(make_float2(off[n][2], off[n][3]), mul2(col, make_float2(a1, a1))));
        }
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = (e >> 1) ? i1 : i0, j = ref + 8 * q + 2 * t + (e & 1);
          const float *tj = T + j * kTLd;
          const float diff = (((e >> 1) ? h1r : h0r) - ghi[j]) + (((e >> 1) ? l1r : l0r) - tj[kGLo]);
          const bool on = is_q ? j <= i : j < i;
          v[e] = on ? ((e >> 1) ? f1 : f0) * exp2f(diff) * tj[kKappa] * dia[q][e] : 0.0f;
        }
        put_tile(ref + 8 * q, make_float2(v[0], v[1]), make_float2(v[2], v[3]));
      }
      if (!is_q) {
        __syncwarp();
        // T's 16 x 16 diagonal block by substitution, a lane per column
        const int c = lane & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float v = i == c ? 1.0f : 0.0f;
#pragma unroll
          for (int j = 0; j < i; j += 4) {
            const float4 l = *reinterpret_cast<const float4 *>(L + l_at(ref + i, ref + j));
            v = fmaf(-l.x, x[j], v);
            if (j + 1 < i) v = fmaf(-l.y, x[j + 1], v);
            if (j + 2 < i) v = fmaf(-l.z, x[j + 2], v);
            if (j + 3 < i) v = fmaf(-l.w, x[j + 3], v);
          }
          x[i] = v;
        }
        if (lane < 16)
#pragma unroll
          for (int i = 0; i < 16; ++i) T[(ref + i) * kTLd + ref + c] = x[i];
      }
    }
    __syncthreads();

    // [A 0; B C]^-1 = [A^-1 0; -C^-1 B A^-1 C^-1] for blocks of 16, then 32.
    // B A^-1 waits in the block's own place.
    const auto l_of = [&](int i, int j) { return L[l_at(i, j)]; };
    const auto t_of = [&](int i, int j) { return T[i * kTLd + j]; };
    const auto put = [&](const float(&acc)[4], int r0, int c0, float sign) {
      float *p = T + (r0 + g) * kTLd + c0 + 2 * t;
      *reinterpret_cast<float2 *>(p) = make_float2(sign * acc[0], sign * acc[1]);
      *reinterpret_cast<float2 *>(p + 8 * kTLd) = make_float2(sign * acc[2], sign * acc[3]);
    };
    float acc[4];
    if (warp < 4) {
      // a warp's eight columns of B A^-1 are all that it reads of it
      const int o = 32 * (warp >> 1), c0 = o + 8 * (warp & 1);
      product(acc, o + 16, c0, c0, o + 16, l_of, t_of, lane);
      put(acc, o + 16, c0, 1.0f);
      __syncwarp();
      product(acc, o + 16, c0, o + 16, o + 32, t_of, t_of, lane);
      __syncwarp();
      put(acc, o + 16, c0, -1.0f);
    }
    __syncthreads();
    {
      const int r0 = 32 + 16 * (warp >> 2), c0 = 8 * (warp & 3);
      product(acc, r0, c0, c0, 32, l_of, t_of, lane);  // T(k, c) = 0 for k < c
      put(acc, r0, c0, 1.0f);
      __syncthreads();
      product(acc, r0, c0, 32, r0 + 16, t_of, t_of, lane);
      __syncthreads();
      put(acc, r0, c0, -1.0f);
    }
    __syncthreads();

    // T's rows as two fp16 terms in L's place, four threads a row, and a power
    // of two above every row's sum
    {
      const int i = tid >> 2, q = tid & 3;
      float2 v[2][4];
      float mx = 0.0f, sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int p = q + 4 * e;
        if (p / 2 <= i / 16) {
          const float4 a = *reinterpret_cast<const float4 *>(T + i * kTLd + 8 * p);
          const float4 b = *reinterpret_cast<const float4 *>(T + i * kTLd + 8 * p + 4);
          v[e][0] = make_float2(a.x, a.y), v[e][1] = make_float2(a.z, a.w);
          v[e][2] = make_float2(b.x, b.y), v[e][3] = make_float2(b.z, b.w);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            mx = max3_abs(mx, v[e][j].x, v[e][j].y);
            sum += fabsf(v[e][j].x) + fabsf(v[e][j].y);
          }
        }
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
        sum += __shfl_xor_sync(kFull, sum, o);
      }
      float most = sum;
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) most = fmaxf(most, __shfl_xor_sync(kFull, most, o));
      if (lane == 0) red[warp] = most;
      __syncthreads();
      most = red[0];
#pragma unroll
      for (int o = 1; o < kPrepThreads / 32; ++o) most = fmaxf(most, red[o]);
      float mult, inv, up, down;
      pow2_above(most, up, down);
      pow2_scale(mx, mult, inv);
      if (q == 0) vec[kVecT * kC + i] = inv * down;
      if (tid == 0) vec[kVecMisc * kC + 1] = up;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int p = q + 4 * e;
        if (p / 2 <= i / 16) {
          uint32_t hw[4], lw[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) split_h2(mul2(v[e][j], make_float2(mult, mult)), hw[j], lw[j]);
          const uint32_t at = tile_at<kC>(i, p);
          *reinterpret_cast<uint4 *>(sm.head + at) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
          *reinterpret_cast<uint4 *>(sm.head + kTile + at) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
        }
      }
    }
    ptx::fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      bulk_store(ws_head + (static_cast<size_t>(slot) * d.v_heads + h) * kHeadBlob,
                 ptx::smem_u32(sm.head), kHeadBlob);
      if (h % ratio == 0)
        bulk_store(ws_key + (static_cast<size_t>(slot) * d.qk_heads + hk) * kKeyBlob<DK>,
                   ptx::smem_u32(sm.key), kKeyBlob<DK>);
      bulk_store_wait();
    }
    if (hh + 1 < heads) __syncthreads();  // the copy has left the head's place
  }
}

// ------------------------------------------------------------------ chain

// Shared memory of one group of three warps (16 state rows): what the two
// chain warps exchange, what they hand to the output warp, the value rows and
// the output rows.
template <int DK>
struct GroupSmem {
  uint4 s_frag[DK / 16][32];    // S as A fragments, fp16
  uint4 u_frag[4][32];          // u likewise
  float4 x_part[2][8][32];      // each half's S k^T
  uint4 w_frag[4][2][32];       // the update's A fragments, two terms
  float2 s_inv[2][32], u_inv[32];
  alignas(16) uint8_t v[3][kC * 32];  // 16 value channels of the chunk's tokens
  alignas(16) uint8_t o[kC * 32];
};

template <int DK, int GROUPS>
struct ChainCfg {
  // one CTA per SM: the ring takes what the groups leave of its shared memory
  static constexpr int kStageBytes = kKeyBlob<DK> + kHeadBlob;
  static constexpr int kStages = GROUPS >= 4 && DK == 128 ? 2 : 3;
  // With stages to spare the output warp waits for a chunk's operands half a
  // chunk ahead and the group's barrier passes them on; otherwise the chain
  // warps wait for them where they need them.
  static constexpr bool kAhead = kStages >= 3;
  // A warp of its own for the ring where that leaves the others registers
  // enough (four warps share a quarter of the SM's); else the first output
  // warp brings the stages in.
  static constexpr bool kProducer = GROUPS < 4;
  static constexpr int kThreads = 32 * (3 * GROUPS + kProducer);
  static constexpr int kSmem =
      kStages * kStageBytes + GROUPS * static_cast<int>(sizeof(GroupSmem<DK>)) + 64;
};

// 16-byte pieces of the 32-byte token rows of v and o, permuted so that eight
// rows' pieces of one column lie in different banks.
__device__ __forceinline__ uint32_t row32_at(int row, int piece) {
  return static_cast<uint32_t>(row * 32 + ((piece ^ ((row >> 2) & 1)) << 4));
}

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(kFull, v, 1));
  return fmaxf(v, __shfl_xor_sync(kFull, v, 2));
}

// An accumulator tile of 16 rows x 8 columns: rows lane / 4 (top) and
// lane / 4 + 8 (low), columns 2 (lane % 4), + 1.
struct Acc {
  float2 top, low;
};

__device__ __forceinline__ void mma16(Acc &c, const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  float f[4] = {c.top.x, c.top.y, c.low.x, c.low.y};
  ::moe::mma16(f, a, b0, b1);
  c.top = make_float2(f[0], f[1]), c.low = make_float2(f[2], f[3]);
}

// A fragments (two terms) of the 16 columns of tiles p and q, scaled by rows.
__device__ __forceinline__ void split_frag(const Acc &p, const Acc &q, float2 m0, float2 m1,
                                           uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  split_h2(mul2(p.top, m0), hi[0], lo[0]);
  split_h2(mul2(p.low, m1), hi[1], lo[1]);
  split_h2(mul2(q.top, m0), hi[2], lo[2]);
  split_h2(mul2(q.low, m1), hi[3], lo[3]);
}

// Power-of-two scales of the two rows a lane holds, from N tiles.
template <int N>
__device__ __forceinline__ void row_scales(const Acc (&x)[N], float &m0, float &m1, float &i0,
                                           float &i1) {
  float a = 0.0f, b = 0.0f;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    a = max3_abs(a, x[n].top.x, x[n].top.y);
    b = max3_abs(b, x[n].low.x, x[n].low.y);
  }
  pow2_scale(quad_max(a), m0, i0);
  pow2_scale(quad_max(b), m1, i1);
}

template <int DK, int GROUPS>
__global__ void __launch_bounds__(ChainCfg<DK, GROUPS>::kThreads, 1)
delta_chain_kernel(moe_delta_dims d, moe_delta_inputs in, DeltaSeqs seq, const uint8_t *ws,
                   const uint8_t *ws_key, const uint8_t *ws_head, moe_bf16 *out, int64_t out_ld,
                   unsigned long long budget_ns) {
  using Cfg = ChainCfg<DK, GROUPS>;
  constexpr int kStages = Cfg::kStages;
  constexpr int kHalf = DK / 2;  // key channels of a chain warp
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t *ring = smem_raw;
  GroupSmem<DK> *groups = reinterpret_cast<GroupSmem<DK> *>(ring + kStages * Cfg::kStageBytes);
  uint64_t *full = reinterpret_cast<uint64_t *>(groups + GROUPS), *empty = full + kStages;
  int *abort_flag = reinterpret_cast<int *>(empty + kStages);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int tiles = d.v_dim / (16 * GROUPS);
  const int tile = blockIdx.x % tiles;
  const int h = (blockIdx.x / tiles) % d.v_heads;
  const int b = blockIdx.x / tiles / d.v_heads;
  if (reinterpret_cast<const uint32_t *>(ws)[kFlagWord]) return;
  const DeltaSeqRange r = delta_seq_range(seq, b);
  if (!r.ok) return;
  const int hk = h / (d.v_heads / d.qk_heads);
  const int chunks = (r.len + kC - 1) / kC;
  const int base = slot_base(seq, b);

  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 3 * GROUPS);
    }
    ptx::fence_mbar_init();
  }
  __syncthreads();

  const auto issue = [&](int c) {  // the operands of chunk c: keys and queries, the head's part
    const int s = c % kStages;
    const uint32_t dst = ptx::smem_u32(ring + s * Cfg::kStageBytes);
    const size_t at = static_cast<size_t>(base) + c;
    ptx::mbar_expect_tx(&full[s], Cfg::kStageBytes);
    bulk_load(dst, ws_key + (at * d.qk_heads + hk) * kKeyBlob<DK>, kKeyBlob<DK>, &full[s]);
    bulk_load(dst + kKeyBlob<DK>, ws_head + (at * d.v_heads + h) * kHeadBlob, kHeadBlob, &full[s]);
  };
  // Waits for the stage that chunk c - kStages has left; false if it gave up.
  const auto wait_empty = [&](int c) {
    return c < kStages || ptx::mbar_wait(&empty[c % kStages], (c / kStages - 1) & 1, abort_flag,
                                         budget_ns);
  };
  // Copies in flight land before the CTA's shared memory is given up.
  const auto drain = [&](int issued) {
    int ignore = 0;
    for (int c = max(0, issued - kStages); c < issued; ++c)
      ptx::mbar_wait(&full[c % kStages], (c / kStages) & 1, &ignore, ptx::kDrainBudgetNs);
    if (*reinterpret_cast<volatile int *>(abort_flag)) set_status(seq.status, MOE_DEV_TIMEOUT);
  };
  if (Cfg::kProducer && warp == 3 * GROUPS) {
    if (lane == 0) {
      int c = 0;
      for (; c < chunks && wait_empty(c); ++c) issue(c);
      drain(c);
    }
    return;
  }

  // Chain warps 2 g, 2 g + 1 (the halves of the key channels), output warp
  // 2 GROUPS + g.  The three warps of a group meet twice per chunk: bar_x
  // (both halves of S k^T and the copy of S are there), bar_w (u is there, and
  // the next chunk's values).  Every buffer of the group is written before one
  // of the two, read between it and the other, and so free again when its
  // writer comes back to it.
  const bool chain = warp < 2 * GROUPS;
  const int group = chain ? warp >> 1 : warp - 2 * GROUPS, half = warp & 1;
  GroupSmem<DK> &gs = groups[group];
  const int bar_x = 1 + 2 * group, bar_w = 2 + 2 * group;
  const int dv0 = (tile * GROUPS + group) * 16;
  const int g = lane >> 2, t = lane & 3;
  // a wait that gave up is not repeated: the loops below run to their end on
  // whatever the ring holds, so that all warps of a group pass every barrier
  bool dead = false;
  // B fragments of two n8 tiles from rows (plain) or columns (trans) of a tile
  const int b_row = (lane & 7) + ((lane >> 4) << 3), b_piece = (lane >> 3) & 1;
  const int bt_row = (lane & 7) + (((lane >> 3) & 1) << 3), bt_piece = lane >> 4;

  if (chain) {
    constexpr int kSteps = kHalf / 16;
    const int64_t at = ((static_cast<int64_t>(r.slot) * d.v_heads + h) * d.v_dim + dv0 + g) * DK +
                       half * kHalf + 2 * t;
    Acc S[kHalf / 8];
#pragma unroll
    for (int n = 0; n < kHalf / 8; ++n) {
      S[n].top = S[n].low = make_float2(0.0f, 0.0f);
      if (seq.state_in) {
        S[n].top = *reinterpret_cast<const float2 *>(seq.state_in + at + 8 * n);
        S[n].low = *reinterpret_cast<const float2 *>(seq.state_in + at + 8 * DK + 8 * n);
      }
    }
    const uint32_t v_at =
        ptx::smem_u32(gs.v[0]) + row32_at((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);
    // T's fragments that this half needs (below)
    const int np_of[2] = {half ? 1 : 0, half ? 2 : 3};
    if (chunks) bar_sync(bar_w, 96);
    float m0, m1, i0, i1;
    row_scales(S, m0, m1, i0, i1);
    for (int c = 0; c < chunks; ++c) {
      const int st = c % kStages;
      const uint32_t kt = ptx::smem_u32(ring + st * Cfg::kStageBytes);
      const uint32_t tt = kt + kKeyBlob<DK>;
      const float *vec =
          reinterpret_cast<const float *>(ring + st * Cfg::kStageBytes + kKeyBlob<DK> + 3 * kTile);
      if (!Cfg::kAhead && !dead)
        dead = !ptx::mbar_wait(&full[st], (c / kStages) & 1, abort_flag, budget_ns);
      gs.s_inv[half][lane] = make_float2(i0, i1);
      // this half's share of X^T = S k^T (16 value channels x 64 tokens)
      Acc X[8] = {}, Y[8];
      float2 cc[8];
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        uint32_t hi[4], lo[4], bb[4][4];
#pragma unroll
        for (int np = 0; np < 4; ++np)
          ldsm4(bb[np], kt + tile_at<DK>(16 * np + b_row, half * (kHalf / 8) + 2 * s + b_piece));
        split_frag(S[2 * s], S[2 * s + 1], make_float2(m0, m0), make_float2(m1, m1), hi, lo);
        gs.s_frag[half * kSteps + s][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          mma16(X[2 * np], hi, bb[np][0], bb[np][1]);
          mma16(X[2 * np + 1], hi, bb[np][2], bb[np][3]);
        }
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          mma16(X[2 * np], lo, bb[np][0], bb[np][1]);
          mma16(X[2 * np + 1], lo, bb[np][2], bb[np][3]);
        }
        if (s > 0) continue;
        // beta_i v_i, in the shadow of the products
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          uint32_t vv[4];
          ldsm4_t(vv, v_at + (c % 3) * kC * 32 + np * 16 * 32);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int n = 2 * np + q;
            const float2 be = *reinterpret_cast<const float2 *>(vec + kVecBeta * kC + 8 * n + 2 * t);
            cc[n] = *reinterpret_cast<const float2 *>(vec + kVecC * kC + 8 * n + 2 * t);
            Y[n].top = mul2(be, make_float2(bf16_lo(vv[2 * q]), bf16_hi(vv[2 * q])));
            Y[n].low = mul2(be, make_float2(bf16_lo(vv[2 * q + 1]), bf16_hi(vv[2 * q + 1])));
          }
        }
      }
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        X[n].top = mul2(X[n].top, make_float2(i0, i0));
        X[n].low = mul2(X[n].low, make_float2(i1, i1));
        gs.x_part[half][n][lane] = make_float4(X[n].top.x, X[n].top.y, X[n].low.x, X[n].low.y);
        Y[n].top = fma2(cc[n], X[n].top, Y[n].top);
        Y[n].low = fma2(cc[n], X[n].low, Y[n].low);
      }
      bar_sync(bar_x, 96);
      // x_i = beta_i v_i - c_i (S k_i), with the other half's share; vec holds -c_i
      {
        float4 y[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) y[n] = gs.x_part[half ^ 1][n][lane];
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          X[n].top = fma2(cc[n], make_float2(y[n].x, y[n].y), Y[n].top);
          X[n].low = fma2(cc[n], make_float2(y[n].z, y[n].w), Y[n].low);
        }
      }
      // u = T x.  Column tiles 2 np, 2 np + 1 of u^T take the tokens of k16
      // steps 0 .. np; the halves take np = 0 and 3, and np = 1 and 2: five
      // steps each.
      uint32_t th[4][2][4], tl[4][2][4];
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (s <= np_of[j]) {
            const uint32_t a = tt + tile_at<kC>(16 * np_of[j] + b_row, 2 * s + b_piece);
            ldsm4(th[s][j], a);
            ldsm4(tl[s][j], a + kTile);
          }
      const float gamma = vec[kVecMisc * kC], tau = vec[kVecMisc * kC + 1];
      const float back = tau * vec[kVecMisc * kC + 2];
      float2 ts[2][2], dd[2][2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int at_n = 8 * (2 * np_of[j] + q) + 2 * t;
          ts[j][q] = *reinterpret_cast<const float2 *>(vec + kVecT * kC + at_n);
          dd[j][q] = *reinterpret_cast<const float2 *>(vec + kVecD * kC + at_n);
        }
      row_scales(X, m0, m1, i0, i1);
      Acc U[2][2] = {}, V[2][2] = {}, W[2][2] = {};
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        uint32_t hi[4], lo[4];
        split_frag(X[2 * s], X[2 * s + 1], make_float2(m0, m0), make_float2(m1, m1), hi, lo);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (s <= np_of[j])
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              mma16(U[j][q], hi, th[s][j][2 * q], th[s][j][2 * q + 1]);
              mma16(V[j][q], hi, tl[s][j][2 * q], tl[s][j][2 * q + 1]);
              mma16(W[j][q], lo, th[s][j][2 * q], th[s][j][2 * q + 1]);
            }
      }
      // Rescaled by T's row scales and down by a bound of its row sums, u
      // stays below 2^15 (the scale of x), and so does w_j = Gamma_64,j
      // kappa_j u_j over the largest such factor.
      gs.u_inv[lane] = make_float2(i0 * tau, i1 * tau);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t f[4], hi[4], lo[4];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float2 one = make_float2(1.0f, 1.0f);
          const float2 top =
              mul2(fma2(U[j][q].top, one, fma2(V[j][q].top, one, W[j][q].top)), ts[j][q]);
          const float2 low =
              mul2(fma2(U[j][q].low, one, fma2(V[j][q].low, one, W[j][q].low)), ts[j][q]);
          f[2 * q] = h2_bits(__float22half2_rn(top));
          f[2 * q + 1] = h2_bits(__float22half2_rn(low));
          split_h2(mul2(top, dd[j][q]), hi[2 * q], lo[2 * q]);
          split_h2(mul2(low, dd[j][q]), hi[2 * q + 1], lo[2 * q + 1]);
        }
        gs.w_frag[np_of[j]][0][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        gs.w_frag[np_of[j]][1][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        gs.u_frag[np_of[j]][lane] = make_uint4(f[0], f[1], f[2], f[3]);
      }
      bar_sync(bar_w, 96);
      // S = gamma S + sum_j w_j k_j^T, 32 key channels at a time
      uint32_t wh[4][4], wl[4][4];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint4 a = gs.w_frag[s][0][lane], e = gs.w_frag[s][1][lane];
        wh[s][0] = a.x, wh[s][1] = a.y, wh[s][2] = a.z, wh[s][3] = a.w;
        wl[s][0] = e.x, wl[s][1] = e.y, wl[s][2] = e.z, wl[s][3] = e.w;
      }
      const float2 gamma2 = make_float2(gamma, gamma);
      const float2 b0 = make_float2(i0 * back, i0 * back), b1 = make_float2(i1 * back, i1 * back);
      float a0 = 0.0f, a1 = 0.0f;
#pragma unroll
      for (int np = 0; np < kSteps; np += 2) {
        Acc acc[4] = {};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          uint32_t bb[2][4];
#pragma unroll
          for (int j = 0; j < 2; ++j)
            ldsm4_t(bb[j], kt + tile_at<DK>(16 * s + bt_row,
                                            half * (kHalf / 8) + 2 * (np + j) + bt_piece));
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            mma16(acc[2 * j], wh[s], bb[j][0], bb[j][1]);
            mma16(acc[2 * j + 1], wh[s], bb[j][2], bb[j][3]);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            mma16(acc[2 * j], wl[s], bb[j][0], bb[j][1]);
            mma16(acc[2 * j + 1], wl[s], bb[j][2], bb[j][3]);
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          Acc &a = S[2 * np + q];
          a.top = fma2(acc[q].top, b0, mul2(gamma2, a.top));
          a.low = fma2(acc[q].low, b1, mul2(gamma2, a.low));
          a0 = max3_abs(a0, a.top.x, a.top.y);
          a1 = max3_abs(a1, a.low.x, a.low.y);
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&empty[st]);
      pow2_scale(quad_max(a0), m0, i0);
      pow2_scale(quad_max(a1), m1, i1);
    }
    if (seq.state_out) {
#pragma unroll
      for (int n = 0; n < kHalf / 8; ++n) {
        *reinterpret_cast<float2 *>(seq.state_out + at + 8 * n) = S[n].top;
        *reinterpret_cast<float2 *>(seq.state_out + at + 8 * DK + 8 * n) = S[n].low;
      }
    }
    return;
  }

  // Output warp: o_i = rho_i gamma_i (S q_i) + sum_j P_ij u_j.  It also brings
  // in the group's values.
  const bool producer = !Cfg::kProducer && group == 0 && lane == 0;
  int issued = 0;
  const uint32_t v_smem = ptx::smem_u32(gs.v[0]);
  const moe_bf16 *v_src = in.v + static_cast<int64_t>(r.start) * in.v_ld + h * d.v_dim + dv0;
  const auto fetch_v = [&](int c) {  // the group's channels of chunk c, zeros past the end
    if (c < chunks) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int i = p * 16 + (lane >> 1), piece = lane & 1, row = c * kC + i;
        const bool live = row < r.len;
        cp_async16(v_smem + (c % 3) * kC * 32 + row32_at(i, piece),
                   v_src + (live ? row * in.v_ld : 0) + piece * 8, live);
      }
    }
    cp_async_commit();
  };
  const auto wait_full = [&](int c) {
    if (!dead) dead = !ptx::mbar_wait(&full[c % kStages], (c / kStages) & 1, abort_flag, budget_ns);
  };
  if (chunks) {
    if (producer)
      for (; issued < min(chunks, kStages); ++issued) issue(issued);
    fetch_v(0);
    fetch_v(1);
    wait_full(0);
    cp_async_wait<1>();
    bar_sync(bar_w, 96);
  }
  const uint32_t o_at = ptx::smem_u32(gs.o) + row32_at((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);
  moe_bf16 *o_dst = out + static_cast<int64_t>(r.start) * out_ld + h * d.v_dim + dv0;
  for (int c = 0; c < chunks; ++c) {
    const int st = c % kStages;
    const uint32_t qt = ptx::smem_u32(ring + st * Cfg::kStageBytes) + kKeyBlob<DK> / 2;
    const uint32_t pt = qt + kKeyBlob<DK> / 2 + 2 * kTile;
    const float *vec =
        reinterpret_cast<const float *>(ring + st * Cfg::kStageBytes + kKeyBlob<DK> + 3 * kTile);
    if (producer && c > 0 && issued < chunks && !dead) {
      dead = !wait_empty(issued);
      if (!dead) issue(issued++);
    }
    if (!Cfg::kProducer) __syncwarp();
    fetch_v(c + 2);
    if (!Cfg::kAhead) wait_full(c);
    bar_sync(bar_x, 96);
    Acc O[8] = {};
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      // the halves of S have scales of their own
      Acc acc[8] = {};
#pragma unroll
      for (int s = 0; s < kHalf / 16; ++s) {
        const uint4 f = gs.s_frag[side * (kHalf / 16) + s][lane];
        const uint32_t a[4] = {f.x, f.y, f.z, f.w};
        uint32_t bb[4][4];
#pragma unroll
        for (int np = 0; np < 4; ++np)
          ldsm4(bb[np], qt + tile_at<DK>(16 * np + b_row, side * (kHalf / 8) + 2 * s + b_piece));
#pragma unroll
        for (int np = 0; np < 4; ++np) {
          mma16(acc[2 * np], a, bb[np][0], bb[np][1]);
          mma16(acc[2 * np + 1], a, bb[np][2], bb[np][3]);
        }
      }
      const float2 si = gs.s_inv[side][lane];
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        O[n].top = fma2(acc[n].top, make_float2(si.x, si.x), O[n].top);
        O[n].low = fma2(acc[n].low, make_float2(si.y, si.y), O[n].low);
      }
    }
    if (Cfg::kAhead && c + 1 < chunks) wait_full(c + 1);
    cp_async_wait<1>();
    __syncwarp();
    bar_sync(bar_w, 96);
    const float2 ui = gs.u_inv[lane];
    Acc I[8] = {};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const uint4 f = gs.u_frag[s][lane];
      const uint32_t a[4] = {f.x, f.y, f.z, f.w};
      uint32_t bb[4][4];
#pragma unroll
      for (int np = s; np < 4; ++np)
        ldsm4(bb[np], pt + tile_at<kC>(16 * np + b_row, 2 * s + b_piece));
#pragma unroll
      for (int np = s; np < 4; ++np) {
        mma16(I[2 * np], a, bb[np][0], bb[np][1]);
        mma16(I[2 * np + 1], a, bb[np][2], bb[np][3]);
      }
    }
#pragma unroll
    for (int np = 0; np < 4; ++np) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int n = 2 * np + q;
        const float2 oq = *reinterpret_cast<const float2 *>(vec + kVecO * kC + 8 * n + 2 * t);
        const float2 pi = *reinterpret_cast<const float2 *>(vec + kVecP * kC + 8 * n + 2 * t);
        const float2 top = fma2(mul2(I[n].top, make_float2(ui.x, ui.x)), pi, mul2(O[n].top, oq));
        const float2 low = fma2(mul2(I[n].low, make_float2(ui.y, ui.y)), pi, mul2(O[n].low, oq));
        w[2 * q] = pack_bf16(top.x, top.y);
        w[2 * q + 1] = pack_bf16(low.x, low.y);
      }
      // transposed back: token rows of 16 channels
      stsm4_t(o_at + np * 16 * 32, w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&empty[st]);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int i = p * 16 + (lane >> 1), piece = lane & 1, row = c * kC + i;
      if (row < r.len)
        *reinterpret_cast<uint4 *>(o_dst + row * out_ld + piece * 8) =
            *reinterpret_cast<const uint4 *>(gs.o + row32_at(i, piece));
    }
    __syncwarp();
  }
  cp_async_wait<0>();
  if (producer) drain(issued);
}

// Sets a kernel's shared-memory limit once per device.
template <class F>
cudaError_t allow_smem(F kernel, int bytes, std::atomic<uint64_t> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <int DK, int GROUPS>
cudaError_t launch_chain(const moe_delta_dims &d, const moe_delta_inputs &in, const DeltaSeqs &seq,
                         const uint8_t *ws, const uint8_t *ws_key, const uint8_t *ws_head,
                         moe_bf16 *out, int64_t out_ld, cudaStream_t s) {
  using Cfg = ChainCfg<DK, GROUPS>;
  static_assert(Cfg::kSmem <= 227 * 1024, "shared memory of one SM");
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(delta_chain_kernel<DK, GROUPS>, Cfg::kSmem, done);
  if (e != cudaSuccess) return e;
  const int64_t grid = static_cast<int64_t>(seq.B) * d.v_heads * (d.v_dim / (16 * GROUPS));
  delta_chain_kernel<DK, GROUPS><<<static_cast<unsigned>(grid), Cfg::kThreads, Cfg::kSmem, s>>>(
      d, in, seq, ws, ws_key, ws_head, out, out_ld, tc_wait_budget_ns());
  return cudaGetLastError();
}

// Chunks times key heads from which a CTA of the first kernel serves all the
// value heads of its key head.
constexpr size_t kPrepShare = 1000;

template <int DK>
cudaError_t launch(const moe_delta_dims &d, const moe_delta_inputs &in, const DeltaSeqs &seq,
                   uint8_t *ws, moe_bf16 *out, int64_t out_ld, cudaStream_t s) {
  const size_t slots = static_cast<size_t>(seq.N) / kC + seq.B;
  uint8_t *ws_key = ws + kHeader;
  uint8_t *ws_head = ws_key + slots * d.qk_heads * kKeyBlob<DK>;
  constexpr int kSmem = sizeof(PrepSmem<DK>);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(delta_prep_kernel<DK>, kSmem, done);
  if (e != cudaSuccess) return e;
  const int ratio = d.v_heads / d.qk_heads;
  const int heads = slots * d.qk_heads >= kPrepShare ? ratio : 1;
  const dim3 grid(static_cast<unsigned>(slots), d.v_heads / heads);
  delta_prep_kernel<DK><<<grid, kPrepThreads, kSmem, s>>>(d, in, seq, heads, ws, ws_key, ws_head);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int64_t groups = static_cast<int64_t>(seq.B) * d.v_heads * (d.v_dim / 16);
  if (groups <= 2 * 152)
    return launch_chain<DK, 2>(d, in, seq, ws, ws_key, ws_head, out, out_ld, s);
  return launch_chain<DK, 4>(d, in, seq, ws, ws_key, ws_head, out, out_ld, s);
}

}  // namespace

size_t delta_chunk_workspace(const moe_delta_dims &d, int N, int B) {
  const size_t slots = static_cast<size_t>(N) / kC + B;
  const size_t key = d.qk_dim == 128 ? kKeyBlob<128> : kKeyBlob<64>;
  return kHeader + slots * (d.qk_heads * key + static_cast<size_t>(d.v_heads) * kHeadBlob);
}

cudaError_t launch_delta_chunk(const moe_delta_dims &d, const moe_delta_inputs &in,
                               const DeltaSeqs &seq, void *ws, moe_bf16 *out, int64_t out_ld,
                               cudaStream_t s) {
  return d.qk_dim == 128 ? launch<128>(d, in, seq, static_cast<uint8_t *>(ws), out, out_ld, s)
                         : launch<64>(d, in, seq, static_cast<uint8_t *>(ws), out, out_ld, s);
}

}  // namespace moe
