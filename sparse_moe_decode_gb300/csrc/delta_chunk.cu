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
// Two kernels.  delta_prep_kernel, a CTA per chunk and key head, forms what
// does not depend on the state: T, the masked q.k products P, the decays, and k
// and q as fp16.  delta_chain_kernel walks a sequence's chunks with the state in
// registers, 16 of its rows to a group of four warps.  Two of them are the
// chain, each with half of the key channels: S k^T, T x and u k^T follow one
// another there, and the two exchange shares through shared memory.  The other
// two form the outputs from copies of the operands, a phase behind, and bring in
// the next chunks.  mma.sync: the chain is bound by the latency of its dependent
// steps, each of few products whose results the next one needs in registers.  A
// form with tcgen05, where each would pass through tensor memory, has not been
// built or measured; where there are several pieces of work for every SM it may
// be the better one.
//
// Precision.  k and q are bf16: scaled by a power of two per token they are
// exact in fp16 down to 2^-25 of the token's norm.  S, x, u and T are fp32 and
// enter the products as two fp16 terms under a power-of-two scale per row, 22
// bits; products accumulate in fp32 and the state is summed in fp32 registers.
// The scales are of the largest value where one warp holds a row (S) and of a
// bound from norms where two would have to agree (x, u).  The outputs, which
// are rounded to bf16 once, take P, S and u as single fp16 terms: off by up to
// 2^-10 of the sum of their terms' absolute values, a quarter of the rounding to
// come where the terms do not cancel.
//
// What bounds it (GB300, 32 value heads of 128 x 128 on 16 key heads).  A chunk
// of the chain takes 1.73 us on whatever SM it runs, so one prompt of 8192
// tokens takes 222 us there and 82 us in the preparation, of 31 us for the
// bytes.  A CTA's pieces of work (32 state rows of one sequence, or 16) follow one
// another, longest sequences first, with the next one's chunks, values and
// state on their way during the last one's chunks: 240 us for 13 sequences of
// 6007 tokens in all and 115 us for 32 of 64 (244 and 137 us with a CTA for each
// piece, when that was changed).  (Each in a fixed order of pieces was slower, 263 us for
// the 13.)  Measured and slower: four chain warps a group with a quarter of the
// channels each (393 against 338 us for 8192 tokens then), one output warp a
// group (369), and a ninth warp for the copies (446: 168 registers a thread).
#include <cuda_runtime.h>

#include <atomic>

#include "common.cuh"
#include "delta_mma.cuh"
#include "delta_seq.cuh"
#include "early.cuh"
#include "kernels.h"
#include "mixer.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kC = 64;  // tokens per chunk
// A lower triangle of 64 x 64 fp16: ten blocks of 16 x 16, (np, s) for rows 16
// np .., columns 16 s .., one after another.
constexpr int kBlock = 16 * 16 * 2;
constexpr int kTri = 10 * kBlock;
// Per (chunk, value head): what the chain warps read -- T's two terms and
// vectors of 64 fp32 --, then what the output warps read, P and two vectors.
enum { kVecC, kVecBeta, kVecT, kVecD, kVecMisc, kVecsA };
enum { kVecO, kVecP, kVecsB };
enum { kGamma, kTau, kDUp, kCMax };  // of kVecMisc
constexpr int kPartA = 2 * kTri + kVecsA * kC * 4;
constexpr int kPartB = kTri + kVecsB * kC * 4;
constexpr int kHeadBlob = kPartA + kPartB;
constexpr int kHeader = 256;      // status word, and these words
enum {
  kFlagWord = 16,  // some bound of the call is bad: it does nothing
  kCountWord,      // records of the list
  kGroupsWord,     // groups of 16 state rows that a CTA of the chain works on
  kNextWord,       // pieces of work that the chain's CTAs have asked for
};
constexpr int kPrepThreads = 256;
constexpr int kPrepCtas = 3;      // of the first kernel on an SM

// Products with k, q or P under their scales can be 2^17 times their true size:
// they leave the accumulators 2^16 smaller, and the factors of the tokens, which
// they meet next, are so much larger.  (The factors first instead: 8192 tokens 315
// against 312.5 us.)
constexpr float kUp = 0x1p16f, kDown = 0x1p-16f;

template <int DK>
constexpr int kKeyBlob = 2 * kC * DK * 2;  // per (chunk, key head): k, then q, as fp16

// Tiles of fp16 in 16-byte pieces, rows of COLS values; a row's pieces are
// permuted within groups of eight by its number, so that eight rows' pieces of
// one column lie in different banks.
template <int COLS>
__device__ __forceinline__ uint32_t tile_at(int row, int piece) {
  return static_cast<uint32_t>(row * COLS * 2 + ((piece ^ (row & 7)) << 4));
}

// 16-byte pieces of 32-byte rows (blocks of a triangle, rows of v and o),
// permuted so that eight rows' pieces of one column lie in different banks.
__device__ __forceinline__ uint32_t row32_at(int row, int piece) {
  return static_cast<uint32_t>(row * 32 + ((piece ^ ((row >> 2) & 1)) << 4));
}
__device__ __forceinline__ int block_of(int np, int s) { return np * (np + 1) / 2 + s; }
// Piece `piece` (of eight columns) of row i of a triangle.
__device__ __forceinline__ uint32_t tri_at(int i, int piece) {
  return static_cast<uint32_t>(block_of(i >> 4, piece >> 1) * kBlock) + row32_at(i & 15, piece & 1);
}

// Where the chunks of a call lie: `count` slots, a sequence's first one at its
// first row / tokens + each * its number.  Chunks of different sequences never
// share one, whatever the lengths: with (64, 1), and with (kDeltaShort + 1, 0),
// since only longer sequences have chunks and no more than a (kDeltaShort + 1)th
// of their tokens.  Whichever takes fewer.
struct ChunkSlots {
  int tokens, each;
  size_t count;
};
ChunkSlots chunk_slots(int N, int B) {
  const size_t by_seq = static_cast<size_t>(N) / kC + B;
  const size_t by_row = static_cast<size_t>(N) / (kDeltaShort + 1) + 1;
  return by_row < by_seq ? ChunkSlots{kDeltaShort + 1, 0, by_row} : ChunkSlots{kC, 1, by_seq};
}

__device__ __forceinline__ int slot_base(const DeltaSeqs &s, const ChunkSlots &at, int b) {
  return (s.cu_seqlens ? s.cu_seqlens[b] : b * s.T) / at.tokens + at.each * b;
}

__device__ __forceinline__ int first_slot(const DeltaSeqRange &r, const ChunkSlots &at, int b) {
  return r.start / at.tokens + at.each * b;
}

// ------------------------------------------------------------------- prep

constexpr int kTLd = kC + 4;     // row stride of T
constexpr int kPrepHeads = 4;    // value heads of one CTA at most

template <int DK>
struct PrepSmem {
  // k and q until their products are formed; then those (tiles of 16 x 8 in the
  // order of the accumulators, 2 w + 2 of warp w) and L (blocks of 16 x 16)
  union {
    alignas(128) uint8_t key[kKeyBlob<DK>];
    struct {
      float4 kk[20][32], qk[20][32];
      float l[10 * 256];
    };
  };
  alignas(128) uint8_t head[kHeadBlob];
  float t[kC * kTLd];  // T; blocks of 16 above the diagonal are never touched
  // the tokens' factors; per head the sums of g in units of log 2 (two terms)
  // and beta
  float kappa[kC], rho[kC], ghi[kPrepHeads][kC], glo[kPrepHeads][kC], beta[kPrepHeads][kC];
  // Gamma's factors about the first token r of each block of rows:
  // kappa_j e^{G_r - G_j} for the columns left of it, e^{G_i - G_r}
  float col[4][kC], row[kC];
};

// The power of two that brings a token's values below 2^15 (bounded by their
// 2-norm), and its inverse: their bf16 digits are exact in fp16 down to 2^-25
// of the norm and off by 2^-39 of it below that.
__device__ __forceinline__ void token_scale(float ss, float &mult, float &inv) {
  const int e = static_cast<int>((__float_as_uint(ss) >> 23) & 255u);
  const int m = 142 - ((e - 125) >> 1);  // 127 + 15 - ceil((e - 126) / 2)
  mult = __uint_as_float(static_cast<uint32_t>(m) << 23);
  inv = __uint_as_float(static_cast<uint32_t>(254 - m) << 23);
}

// Where L(i, j) lies: blocks of 16 x 16, their pieces of four columns permuted
// by the row, so that eight rows' pieces of one column lie in different banks.
__device__ __forceinline__ int l_at(int i, int j) {
  return block_of(i >> 4, j >> 4) * 256 + (i & 15) * 16 + ((j & 15) ^ (((i >> 1) & 3) << 2));
}

// A 16 x 8 tile of A B over `pairs` pairs of k8 steps; a is the shared address of
// this lane's row g and column t of A (rows `a_ld` bytes apart, its four pieces
// of a pair permuted by `a_x`, pairs `a_step` apart), b that of row t, column g
// of B (rows of T).  fp32 values as two tf32 terms each, three products.
__device__ __forceinline__ void product(float (&acc)[4], uint32_t a, uint32_t a_ld, uint32_t a_x,
                                        uint32_t a_step, uint32_t b, int pairs) {
  float part[3][4] = {};
#pragma unroll 1
  for (; pairs > 0; --pairs, a += a_step, b += 16 * kTLd * 4) {
    float x[2][4], y[2][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint32_t left = a + (((2 * s) ^ a_x) << 4), right = a + (((2 * s + 1) ^ a_x) << 4);
      x[s][0] = lds(left), x[s][1] = lds(left + 8 * a_ld);
      x[s][2] = lds(right), x[s][3] = lds(right + 8 * a_ld);
      y[s][0] = lds(b + 8 * s * kTLd * 4), y[s][1] = lds(b + (8 * s + 4) * kTLd * 4);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint32_t ah[4], al[4], bh[2], bl[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) split_tf32(x[s][i], ah[i], al[i]);
#pragma unroll
      for (int i = 0; i < 2; ++i) split_tf32(y[s][i], bh[i], bl[i]);
      mma8(part[0], ah, bl[0], bl[1]);
      mma8(part[1], al, bh[0], bh[1]);
      mma8(part[2], ah, bh[0], bh[1]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = part[2][i] + (part[0][i] + part[1][i]);
}

// (hi, lo) += (h, l), pairs whose sum is the value: no digit of the larger
// terms is lost (Knuth's two-sum).
__device__ __forceinline__ void add_exact(float &hi, float &lo, float h, float l) {
  const float s = __fadd_rn(hi, h), t = __fsub_rn(s, hi);
  const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(h, t));
  hi = s, lo = __fadd_rn(__fadd_rn(lo, l), e);
}

// The largest of 32 values >= 0 (their bits order like the values).
__device__ __forceinline__ float warp_max_pos(float v) {
  return __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(v)));
}

// What the second kernel has to do, by one CTA: a record {first row, tokens,
// state slot, first chunk slot} per sequence that is not short, of 256 at a time
// the longest first.  A call with a bad bound does nothing.
__device__ void list_sequences(const DeltaSeqs &seq, const ChunkSlots &at, int rows, int sms,
                               uint32_t *head, int4 *list, int *lens) {
  const int tid = threadIdx.x;
  int count = 0, longest = 0;
  long long chunks = 0;
  bool bad = false;
  for (int b0 = 0; b0 < seq.B; b0 += kPrepThreads) {
    const int b = b0 + tid;
    DeltaSeqRange r{};
    int len = 0;
    if (b < seq.B) {
      if (seq.cu_seqlens) {
        const int lo = seq.cu_seqlens[b], hi = seq.cu_seqlens[b + 1];
        bad |= lo < 0 || lo > hi || hi > seq.N;
      }
      r = delta_seq_range(seq, b);
      if (r.ok && r.len > kDeltaShort) len = r.len;
    }
    lens[tid] = len;
    const int here = __syncthreads_count(len > 0);
    if (len > 0) {
      int rank = 0;
      for (int i = 0; i < min(kPrepThreads, seq.B - b0); ++i)
        rank += lens[i] > len || (lens[i] == len && i < tid);
      list[count + rank] = make_int4(r.start, len, r.slot, first_slot(r, at, b));
      longest = max(longest, len), chunks += (len + kC - 1) / kC;
    }
    count += here;
    __syncthreads();
  }
  bad = __syncthreads_or(bad);
  // Groups to a CTA.  One alone takes 0.8 of the time for a chunk, but all work
  // twice as many CTAs: for the better where the longest sequence decides, that
  // is where its chunks are more than 1.6 times an SM's share of them all with
  // two groups (2048 tokens of 8 heads of 128 58.8 against 69.4 us).
  using Wide = unsigned long long;
  Wide *sum = reinterpret_cast<Wide *>(lens);
  if (tid == 0) sum[0] = sum[1] = 0;
  __syncthreads();
  if (chunks) atomicAdd(&sum[0], static_cast<Wide>(chunks));
  if (longest) atomicMax(&sum[1], static_cast<Wide>((longest + kC - 1) / kC));
  __syncthreads();
  if (tid == 0) {
    head[kFlagWord] = bad, head[kCountWord] = count, head[kNextWord] = 0;
    head[kGroupsWord] = 5 * sum[1] * sms > 8 * sum[0] * (rows / 32) ? 1 : 2;
    if (bad) set_status(seq.status, MOE_DEV_BAD_INDEX);
  }
}

// One CTA per chunk and key head, for `heads` of the value heads that read
// it.  Warps 0..3 take k (k k^T, L, T's diagonal blocks), warps 4..7 take q
// (q k^T, P), 16 tokens each.
//
// Bound by the instructions it issues (0.6 per cycle and scheduler, 82 us for
// the 4096 chunks and heads of 8192 tokens, where it moves 1.8 TB/s): the tensor
// pipe is active for 16 % of the time; the inverse, the decays of the triangles
// and the conversions are the rest.  80 registers leave three CTAs an SM, which wait for
// barriers in turn; two CTAs with 128 took the same time.  The products wait
// in shared memory, in the place of k and q: kept in registers they spilled
// (2048 tokens 97 against 93 us).
template <int DK>
__global__ void __launch_bounds__(kPrepThreads, kPrepCtas)
delta_prep_kernel(moe_delta_dims d, moe_delta_inputs in, DeltaSeqs seq, ChunkSlots slots, int heads,
                  int sms, uint8_t *ws, int4 *list, uint8_t *ws_key, uint8_t *ws_head) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  PrepSmem<DK> &sm = *reinterpret_cast<PrepSmem<DK> *>(smem_raw);
  __shared__ float red[kPrepThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ratio = d.v_heads / d.qk_heads;
  const int slot = static_cast<int>(blockIdx.x) - 1, h0 = blockIdx.y * heads, hk = h0 / ratio;

  early_begin();
  if (slot < 0) {  // the first CTAs have no chunk
    if (blockIdx.y == 0)
      list_sequences(seq, slots, d.v_heads * d.v_dim, sms, reinterpret_cast<uint32_t *>(ws), list,
                     reinterpret_cast<int *>(smem_raw));
    return;
  }

  // whose chunk this is: the last sequence whose slots start at or before it,
  // a 32nd of those left per round of loads
  int b = 0, hi = seq.B;
  while (hi - b > 1) {
    const int step = (hi - b + 31) >> 5, at = b + lane * step;
    const bool before = at < hi && slot_base(seq, slots, at) <= slot;
    b += step * (31 - __clz(__ballot_sync(kFull, before) | 1u));
    hi = min(hi, b + step);
  }
  const DeltaSeqRange r = delta_seq_range(seq, b);
  const int chunk = slot - first_slot(r, slots, b);
  if (!r.ok || r.len <= kDeltaShort || chunk < 0 || chunk >= (r.len + kC - 1) / kC) return;
  const int left = min(kC, r.len - chunk * kC);  // tokens of this chunk
  const int64_t row0 = static_cast<int64_t>(r.start) + chunk * kC;

  const int w = warp & 3;          // this warp's 16 tokens
  const bool is_q = warp >= 4;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t kt = ptx::smem_u32(sm.key);

  // k and q come in as they are, each piece to the place of its fp16 form; eight
  // lanes a row.  Meanwhile warp w sums head w's decays, in units of log 2 as
  // two fp32 terms each, so that differences of large sums keep their digits.
  {
    constexpr int kPieces = DK / 64;  // 16-byte pieces of a lane
    const int piece = lane & 7, row = 16 * w + (lane >> 3);
    const moe_bf16 *src = is_q ? in.q : in.k;
    const int64_t ld = is_q ? in.q_ld : in.k_ld;
    uint8_t *tile = sm.key + (is_q ? kKeyBlob<DK> / 2 : 0);
    // one CTA of a key head's writes them out, whole lines from registers
    const bool keeps_key = h0 % ratio == 0;
    uint8_t *key_out = ws_key + (static_cast<size_t>(slot) * d.qk_heads + hk) * kKeyBlob<DK> +
                       (is_q ? kKeyBlob<DK> / 2 : 0);
    src += row0 * ld + hk * DK + piece * 8;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int i = row + 4 * p;
#pragma unroll
      for (int e = 0; e < kPieces; ++e)
        cp_async16(kt + (is_q ? kKeyBlob<DK> / 2 : 0) + tile_at<DK>(i, piece + 8 * e),
                   src + (i < left ? i * ld : 0) + 64 * e, i < left);
    }
    cp_async_commit();
    if (warp < heads) {
      const int64_t i = row0 + 2 * lane;
      float g0 = 0.0f, g1 = 0.0f, be0 = 0.0f, be1 = 0.0f;
      if (2 * lane < left)
        g0 = in.g[i * in.g_ld + h0 + warp], be0 = in.beta[i * in.beta_ld + h0 + warp];
      if (2 * lane + 1 < left)
        g1 = in.g[(i + 1) * in.g_ld + h0 + warp], be1 = in.beta[(i + 1) * in.beta_ld + h0 + warp];
      g0 = delta_log_decay(g0), g1 = delta_log_decay(g1);
      float hi1 = g0, lo1 = 0.0f;
      add_exact(hi1, lo1, g1, 0.0f);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float h = __shfl_up_sync(kFull, hi1, o), l = __shfl_up_sync(kFull, lo1, o);
        if (lane >= o) add_exact(hi1, lo1, h, l);
      }
      float hi0 = hi1, lo0 = lo1;  // without this lane's second token
      add_exact(hi0, lo0, -g1, 0.0f);
      // times log2 e, as two terms too
      constexpr double kLog2E = 1.4426950408889634;
      constexpr float kHi = static_cast<float>(kLog2E);
      constexpr float kLo = static_cast<float>(kLog2E - static_cast<double>(kHi));
      const float p0 = hi0 * kHi, p1 = hi1 * kHi;
      *reinterpret_cast<float2 *>(&sm.ghi[warp][2 * lane]) = make_float2(p0, p1);
      *reinterpret_cast<float2 *>(&sm.glo[warp][2 * lane]) =
          make_float2(fmaf(hi0, kHi, -p0) + fmaf(hi0, kLo, lo0 * kHi),
                      fmaf(hi1, kHi, -p1) + fmaf(hi1, kLo, lo1 * kHi));
      *reinterpret_cast<float2 *>(&sm.beta[warp][2 * lane]) = make_float2(be0, be1);
    }
    cp_async_wait<0>();  // each lane converts what it brought in
#pragma unroll 2
    for (int p = 0; p < 4; ++p) {
      const int i = row + 4 * p;
      float2 x[kPieces][4], sum = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int e = 0; e < kPieces; ++e) {
        const uint4 raw = *reinterpret_cast<const uint4 *>(tile + tile_at<DK>(i, piece + 8 * e));
        const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
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
        const uint4 all = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4 *>(tile + tile_at<DK>(i, piece + 8 * e)) = all;
        if (keeps_key) *reinterpret_cast<uint4 *>(key_out + tile_at<DK>(i, piece + 8 * e)) = all;
      }
      if (d.qk_norm) inv *= rsqrtf(ss + d.qk_eps);
      if (is_q) inv *= d.scale;
      if (piece == 0) (is_q ? sm.rho : sm.kappa)[i] = i < left ? inv : 0.0f;
    }
  }
  __syncthreads();

  // Rows of k k^T or q k^T, up to the diagonal block; then, once nobody reads k
  // and q any more, into their place.
  float4(*prod)[32] = (is_q ? sm.qk : sm.kk) + w * (w + 1);
  {
    float acc[8][4] = {};
    // a row's pieces are permuted by its number mod 8, which is lane % 8 for
    // every row that a lane addresses
    constexpr uint32_t kRow = DK * 2;
    const uint32_t a_at = kt + (is_q ? kKeyBlob<DK> / 2 : 0) + (16 * w + (lane & 15)) * kRow;
    const uint32_t b_at = kt + ((lane & 7) + ((lane >> 4) << 3)) * kRow;
#pragma unroll 2
    for (int s = 0; s < DK / 16; ++s) {
      uint32_t a[4], b[4][4];
      const uint32_t bc = ((2 * s + ((lane >> 3) & 1)) ^ (lane & 7)) << 4;
      ldsm4(a, a_at + (((2 * s + (lane >> 4)) ^ (lane & 7)) << 4));
#pragma unroll
      for (int np = 0; np < 4; ++np)
        if (np <= w) ldsm4(b[np], b_at + np * 16 * kRow + bc);
#pragma unroll
      for (int np = 0; np < 4; ++np)
        if (np <= w) {
          mma16(acc[2 * np], a, b[np][0], b[np][1]);
          mma16(acc[2 * np + 1], a, b[np][2], b[np][3]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < 8; ++n)
      if (n < 2 * w + 2) prod[n][lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
  }

  float *vec = reinterpret_cast<float *>(sm.head + 2 * kTri);
  float *vec_b = reinterpret_cast<float *>(sm.head + kPartA + kTri);
  float *L = sm.l, *T = sm.t;
  const uint32_t l_base = ptx::smem_u32(L), t_at = ptx::smem_u32(T);
  for (int hh = 0; hh < heads; ++hh) {
    const int h = h0 + hh;
    const float *ghi = sm.ghi[hh], *glo = sm.glo[hh];
    // Left of the diagonal block Gamma_ij = e^{G_i - G_r} e^{G_r - G_j} about
    // the block's first token r: both factors are decays, and the product
    // underflows only where Gamma does.
    {
      const int j = tid & 63, rb = tid >> 6;
      if (j < 16 * rb)
        sm.col[rb][j] = sm.kappa[j] * exp2f((ghi[16 * rb] - ghi[j]) + (glo[16 * rb] - glo[j]));
      else if (j < 16 * rb + 16)
        sm.row[j] = exp2f((ghi[j] - ghi[16 * rb]) + (glo[j] - glo[16 * rb]));
    }
    if (warp == 4) {
      // the chain's and the outputs' factors of the tokens; the update's,
      // Gamma_64,j kappa_j, over a power of two above the largest
      const int i = 2 * lane;
      const float2 sh = *reinterpret_cast<const float2 *>(ghi + i);
      const float2 sl = *reinterpret_cast<const float2 *>(glo + i);
      const float2 be = *reinterpret_cast<const float2 *>(sm.beta[hh] + i);
      const float2 kap = *reinterpret_cast<const float2 *>(sm.kappa + i);
      const float2 rho = *reinterpret_cast<const float2 *>(sm.rho + i);
      const float th = ghi[kC - 1], tl = glo[kC - 1];
      const float2 gamma = make_float2(exp2f(sh.x), exp2f(sh.y));
      const float2 cc = make_float2(-be.x * gamma.x * kap.x, -be.y * gamma.y * kap.y);
      const float2 dd = make_float2(exp2f((th - sh.x) + (tl - sl.x)) * kap.x,
                                    exp2f((th - sh.y) + (tl - sl.y)) * kap.y);
      const float dmax = warp_max_pos(fmaxf(dd.x, dd.y));
      const float cmax = warp_max_pos(fmaxf(fabsf(cc.x), fabsf(cc.y)));
      float up, down;
      pow2_above(dmax, up, down);
      *reinterpret_cast<float2 *>(vec + kVecBeta * kC + i) = be;
      *reinterpret_cast<float2 *>(vec + kVecC * kC + i) = mul2(cc, make_float2(kUp, kUp));
      *reinterpret_cast<float2 *>(vec + kVecD * kC + i) = make_float2(dd.x * down, dd.y * down);
      *reinterpret_cast<float2 *>(vec_b + kVecO * kC + i) =
          make_float2(rho.x * gamma.x * kUp, rho.y * gamma.y * kUp);
      if (lane == 31) {
        vec[kVecMisc * kC + kGamma] = gamma.y;
        vec[kVecMisc * kC + kDUp] = up;
        vec[kVecMisc * kC + kCMax] = cmax;
      }
    }
    __syncthreads();

    // L = beta_i kappa_i Gamma_ij kappa_j k_i.k_j below the diagonal, P =
    // rho_i Gamma_ij kappa_j q_i.k_j up to it
    {
      const int ref = 16 * w, i0 = ref + g, i1 = i0 + 8;
      const float h0r = ghi[i0], l0r = glo[i0], h1r = ghi[i1], l1r = glo[i1];
      float f0, f1;
      if (is_q) {
        f0 = sm.rho[i0], f1 = sm.rho[i1];
      } else {
        f0 = sm.beta[hh][i0] * sm.kappa[i0];
        f1 = sm.beta[hh][i1] * sm.kappa[i1];
      }
      // P's row scale from norms: by their scales k and q stay below 2^15, so
      // |P_ij| <= rho_i max kappa 2^30, which goes to 2^11 or less (room for
      // decays that grow by up to 2^5).
      float s0 = 1.0f, s1 = 1.0f;
      if (is_q) {
        const float kmax = warp_max_pos(fmaxf(sm.kappa[lane], sm.kappa[lane + 32]));
        float up0, up1;
        pow2_above(fabsf(f0) * kmax, up0, s0);
        pow2_above(fabsf(f1) * kmax, up1, s1);
        s0 *= 0x1p-19f, s1 *= 0x1p-19f;
        if (t == 0) {
          vec_b[kVecP * kC + i0] = up0 * (0x1p19f * kUp);
          vec_b[kVecP * kC + i1] = up1 * (0x1p19f * kUp);
        }
      }
      f0 *= s0, f1 *= s1;
      const float a0 = f0 * sm.row[i0], a1 = f1 * sm.row[i1];
      uint8_t *P = sm.head + kPartA + 4 * t;
      // one tile: eight columns from `col` of this warp's rows
      const auto put_tile = [&](int col, float2 top, float2 low) {
        if (is_q) {
          *reinterpret_cast<__half2 *>(P + tri_at(i0, col / 8)) = __float22half2_rn(top);
          *reinterpret_cast<__half2 *>(P + tri_at(i1, col / 8)) = __float22half2_rn(low);
        } else {
          *reinterpret_cast<float2 *>(L + l_at(i0, col + 2 * t)) = top;
          *reinterpret_cast<float2 *>(L + l_at(i1, col + 2 * t)) = low;
        }
      };
#pragma unroll 1
      for (int n = 0; n < 2 * w; ++n) {
        const float4 y = prod[n][lane];
        const float2 col = *reinterpret_cast<const float2 *>(&sm.col[w][8 * n + 2 * t]);
        put_tile(8 * n, mul2(make_float2(y.x, y.y), mul2(col, make_float2(a0, a0))),
                 mul2(make_float2(y.z, y.w), mul2(col, make_float2(a1, a1))));
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int j = ref + 8 * q + 2 * t;
        const float2 gj = *reinterpret_cast<const float2 *>(ghi + j);
        const float2 lj = *reinterpret_cast<const float2 *>(glo + j);
        const float2 kj = *reinterpret_cast<const float2 *>(sm.kappa + j);
        const float4 y = prod[2 * w + q][lane];
        float v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = (e >> 1) ? i1 : i0, jj = j + (e & 1);
          const float diff = (((e >> 1) ? h1r : h0r) - ((e & 1) ? gj.y : gj.x)) +
                             (((e >> 1) ? l1r : l0r) - ((e & 1) ? lj.y : lj.x));
          const bool on = is_q ? jj <= i : jj < i;
          v[e] = on ? ((e >> 1) ? f1 : f0) * exp2f(diff) * ((e & 1) ? kj.y : kj.x) * v[e] : 0.0f;
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

    // [A 0; B C]^-1 = [A^-1 0; -C^-1 B A^-1 C^-1] for blocks of 16 (two pairs,
    // four warps), then of 32 (all warps; a warp has 16 x 8).  B A^-1 waits in
    // the block's own place.  T(k, c) = 0 for k < c, and its blocks above the
    // diagonal do not exist.
#pragma unroll 1
    for (int round = 0; round < 4; ++round) {
      const bool wide = round >= 2, second = round & 1;
      const bool on = wide || warp < 4;
      const int o = wide ? 0 : 32 * (warp >> 1);
      const int r0 = wide ? 32 + 16 * (warp >> 2) : o + 16;
      const int c0 = wide ? 8 * (warp & 3) : o + 8 * (warp & 1);
      int k0 = wide ? (second ? 32 : 16 * ((warp & 3) >> 1)) : (second ? o + 16 : o);
      const int pairs = !wide ? 1 : second ? 1 + (warp >> 2) : 2 - ((warp & 3) >> 1);
      float acc[4];
      if (on)
        product(acc, second ? t_at + ((r0 + g) * kTLd + k0 + t) * 4
                            : l_base + (block_of(r0 >> 4, k0 >> 4) * 256 + g * 16 + t) * 4,
                4 * (second ? kTLd : 16), second ? 0 : (g >> 1) & 3, 4 * (second ? 16 : 256),
                t_at + ((k0 + t) * kTLd + c0 + g) * 4, pairs);
      if (second) __syncthreads();
      if (on) {
        const float sign = second ? -1.0f : 1.0f;
        float *p = T + (r0 + g) * kTLd + c0 + 2 * t;
        *reinterpret_cast<float2 *>(p) = make_float2(sign * acc[0], sign * acc[1]);
        *reinterpret_cast<float2 *>(p + 8 * kTLd) = make_float2(sign * acc[2], sign * acc[3]);
      }
      __syncthreads();
    }

    // T's rows as two fp16 terms, four threads a row, and a power
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
      if (tid == 0) vec[kVecMisc * kC + kTau] = up;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int p = q + 4 * e;
        if (p / 2 <= i / 16) {
          uint32_t hw[4], lw[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            split_h2(mul2(v[e][j], make_float2(mult, mult)), hw[j], lw[j]);
          const uint32_t at = tri_at(i, p);
          *reinterpret_cast<uint4 *>(sm.head + at) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
          *reinterpret_cast<uint4 *>(sm.head + kTri + at) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
        }
      }
    }
    ptx::fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      bulk_store(ws_head + (static_cast<size_t>(slot) * d.v_heads + h) * kHeadBlob,
                 ptx::smem_u32(sm.head), kHeadBlob);
      bulk_store_wait(hh + 1 == heads);
    }
    if (hh + 1 < heads) __syncthreads();  // the copy has left the head's place
  }
}

// ------------------------------------------------------------------ chain

// How the chain runs: kHalves chain warps and two output warps per group of 16
// state rows, up to kGroups groups per CTA, one CTA per SM.
constexpr int kHalves = 2;
constexpr int kGroups = 2;

template <int DK>
struct Chain {
  static constexpr int kCols = DK / kHalves;  // key channels of a chain warp
  static constexpr int kSteps = kCols / 16;   // k16 steps of its share of S k^T
  // Ring stages: for the chain warps k, T and their vectors; for the output
  // warps q, P and theirs.
  static constexpr int kStageA = kKeyBlob<DK> / 2 + kPartA;
  static constexpr int kStageB = kKeyBlob<DK> / 2 + kPartB;
  static constexpr int kStages = 3;
  // Eight warps, two to a quarter of the SM, may have 255 registers each; a
  // ninth would cost every one of them a third.  So the four output warps
  // bring in the rings' stages, one of a chunk's four copies each (issuing a
  // bulk copy holds its thread for some 500 cycles).
  static constexpr int kQueue = 8;
  static constexpr int kThreads = 32 * (kHalves + 2) * kGroups;

  // What the warps of a group hand one another.
  struct Group {
    uint4 s_frag[DK / 16][32];           // S as A fragments, fp16
    uint4 u_frag[4][32];                 // u likewise
    float4 x_part[4][2][32];             // shares of S k^T for the block's owner
    float4 y[4][2][32];                  // beta v
    uint4 x_frag[4][2][32];              // x as A fragments, two terms
    uint4 w_frag[4][2][32];              // the update's, two terms
    float2 s_inv[kHalves][32], v_max[2][32], u_inv[32];
    alignas(16) uint8_t v[3][kC * 32];   // 16 value channels of the chunk's tokens
    alignas(16) uint8_t o[kC * 32];      // output rows on their way out
  };
  static constexpr int kSmem = kStages * (kStageA + kStageB) +
                               kGroups * static_cast<int>(sizeof(Group)) + 256;
};

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

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return fma2(a, both(1.0f), b); }

// A fragments (two terms) of the 16 columns of tiles p and q, scaled by rows.
__device__ __forceinline__ void split_frag(const Acc &p, const Acc &q, float m0, float m1,
                                           uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  split_h2(mul2(p.top, both(m0)), hi[0], lo[0]);
  split_h2(mul2(p.low, both(m1)), hi[1], lo[1]);
  split_h2(mul2(q.top, both(m0)), hi[2], lo[2]);
  split_h2(mul2(q.low, both(m1)), hi[3], lo[3]);
}

__device__ __forceinline__ void put4(uint4 *p, const uint32_t (&v)[4]) {
  *p = make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void get4(const uint4 *p, uint32_t (&v)[4]) {
  const uint4 w = *p;
  v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
}

template <int DK>
__global__ void __launch_bounds__(Chain<DK>::kThreads, 1)
delta_chain_kernel(moe_delta_dims d, moe_delta_inputs in, DeltaSeqs seq, uint8_t *ws,
                   const int4 *list, const uint8_t *ws_key, const uint8_t *ws_head, moe_bf16 *out,
                   int64_t out_ld, unsigned long long budget_ns) {
  using C = Chain<DK>;
  using Group = typename C::Group;
  constexpr int kKeyTile = kKeyBlob<DK> / 2, kStages = C::kStages;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t *ring_a = smem_raw, *ring_b = ring_a + kStages * C::kStageA;
  Group *groups = reinterpret_cast<Group *>(ring_b + kStages * C::kStageB);
  uint64_t *full = reinterpret_cast<uint64_t *>(groups + kGroups);
  int *abort_flag = reinterpret_cast<int *>(full + kStages), *fed_by = abort_flag + 1;
  volatile int *queue = fed_by + 4;  // [kQueue]

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < kStages; ++s) ptx::mbar_init(&full[s], 4);
    ptx::fence_mbar_init();
  }
  const int ratio = d.v_heads / d.qk_heads, grid = static_cast<int>(gridDim.x);
  // pieces per sequence with one group to a CTA
  const int most = d.v_heads * (d.v_dim / 16), bid = static_cast<int>(blockIdx.x);
  const int one = bid / most, two = min(2 * bid / most, seq.B - 1);
  early_begin();
  // The work: the state rows of a CTA, of one head of one sequence, are a piece,
  // index (sequence of the list, head, rows).  A CTA's pieces number 0, 1 and 2
  // are given; for those after it asks, through the first output warp, which of
  // them is next.  That warp publishes number k + 3 when it begins number k, so
  // that all know it after that chunk's bar_x.
  uint32_t *head = reinterpret_cast<uint32_t *>(ws);
  const uint32_t bad = head[kFlagWord];
  const int count = static_cast<int>(head[kCountWord]);
  const int groups_on = static_cast<int>(head[kGroupsWord]);
  const int4 first_one = list[one], first_two = list[two];  // (meaningless past the count)
  if (bad) return;
  const int4 first = groups_on == 1 ? first_one : first_two;
  const int rows = 16 * groups_on, per = groups_on == 1 ? most : most / 2, total = count * per;
  const int tiles = d.v_dim >> (3 + groups_on);  // a power of two
  struct Place {
    int b, h, row;
  };
  const auto place_of = [&](int index) {
    const int t = index >> (31 - __clz(tiles)), b = t / d.v_heads;
    return Place{b, t - b * d.v_heads, (index & (tiles - 1)) * rows};
  };
  const auto piece_at = [&](int k) {
    return k < 3 ? bid + k * grid : queue[k % C::kQueue];
  };
  __syncthreads();

  // Group g's chain warps are 2 g and 2 g + 1 (half of the key channels each), its
  // output warps 4 + 2 g and 5 + 2 g (half of the tokens each); those of a group
  // alone are 6 and 7, so that each warp has a scheduler, and the others leave.
  // The warps meet three times per chunk: all of the CTA
  // at bar_x (the shares of S k^T, the copy of S and beta v are there; nobody
  // reads the previous chunk's stage any more), a group's chain warps at bar_y (x
  // is there), a group at bar_w (u is there, and the next chunk's operands).
  // Every buffer of the group is written before one of them, read after it, and
  // free again when its writer comes back to it: x_part, y and v_max x|y, s_frag
  // x|w, x_frag y|w, w_frag and u_frag w|next x.
  const bool chain = warp < kHalves * kGroups;
  const int part = warp & 1;
  const int group = chain || groups_on == 1 ? (warp >> 1) % 3 : (warp >> 1) - 2;
  if (group >= groups_on) return;
  Group &gs = groups[group];
  const int bar_x = 0, bar_y = 1 + 2 * group, bar_w = bar_y + 1, bar_out = 1 + 2 * kGroups;
  constexpr int kGroup = 32 * (kHalves + 2);
  const int all = kGroup * groups_on;
  const int g = lane >> 2, t = lane & 3;
  // B fragments of two n8 tiles from rows (plain) or columns (trans) of a tile
  const int b_row = (lane & 7) + ((lane >> 4) << 3), b_piece = (lane >> 3) & 1;
  const int bt_row = (lane & 7) + (((lane >> 3) & 1) << 3), bt_piece = lane >> 4;

  if (chain) {
    // The 16-token blocks whose x and u this warp forms.  u's block np takes
    // np + 1 steps: blocks 0 and 3, and 1 and 2, make equal pairs.
    const int own[2] = {part, 3 - part};
    const auto owner = [](int np) { return min(np, 3 - np); };
    int st = 0, index = piece_at(0);
    int4 record = first;
    Place place = place_of(index);
    if (index < total) bar_sync(bar_w, kGroup);  // the first chunk's operands are there
    for (int k = 0; index < total; ++k) {
      const int chunks = (record.y + kC - 1) / kC;
      const int64_t state = static_cast<int64_t>(record.z) * d.v_heads + place.h;
      const int64_t at =
          (state * d.v_dim + place.row + group * 16 + g) * DK + part * C::kCols + 2 * t;
      index = piece_at(k + 1);
      if (index < total) {
        place = place_of(index);
        record = list[place.b];
      }
      Acc S[2 * C::kSteps];
#pragma unroll
      for (int n = 0; n < 2 * C::kSteps; ++n) {
        S[n].top = S[n].low = both(0.0f);
        if (seq.state_in) {
          S[n].top = *reinterpret_cast<const float2 *>(seq.state_in + at + 8 * n);
          S[n].low = *reinterpret_cast<const float2 *>(seq.state_in + at + 8 * DK + 8 * n);
        }
      }
      float m0, m1, i0, i1;
      {
        float a0 = 0.0f, a1 = 0.0f;
#pragma unroll
        for (int n = 0; n < 2 * C::kSteps; ++n) {
          a0 = max3_abs(a0, S[n].top.x, S[n].top.y);
          a1 = max3_abs(a1, S[n].low.x, S[n].low.y);
        }
        pow2_scale(quad_max(a0), m0, i0);
        pow2_scale(quad_max(a1), m1, i1);
      }
      for (int c = 0; c < chunks; ++c) {
        const uint32_t kt = ptx::smem_u32(ring_a + st * C::kStageA), tt = kt + kKeyTile;
        const float *vec =
            reinterpret_cast<const float *>(ring_a + st * C::kStageA + kKeyTile + 2 * kTri);
        gs.s_inv[part][lane] = make_float2(i0, i1);
        // this warp's share of X^T = S k^T (16 value channels x 64 tokens)
        Acc X[8] = {};
#pragma unroll
        for (int s = 0; s < C::kSteps; ++s) {
          uint32_t hi[4], lo[4], bb[4][4];
#pragma unroll
          for (int np = 0; np < 4; ++np)
            ldsm4(bb[np],
                  kt + tile_at<DK>(16 * np + b_row, part * (C::kCols / 8) + 2 * s + b_piece));
          split_frag(S[2 * s], S[2 * s + 1], m0, m1, hi, lo);
          put4(&gs.s_frag[part * C::kSteps + s][lane], hi);
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
        }
        const float x0 = i0 * kDown, x1 = i1 * kDown;
        Acc mine[2][2];
#pragma unroll
        for (int np = 0; np < 4; ++np)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            Acc &x = X[2 * np + q];
            x.top = mul2(x.top, both(x0)), x.low = mul2(x.low, both(x1));
            if (owner(np) != part)
              gs.x_part[np][q][lane] = make_float4(x.top.x, x.top.y, x.low.x, x.low.y);
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (np == own[j]) mine[j][q] = x;
          }
        // T's fragments of the own blocks, a step ahead of their use
        uint32_t th[2][2][4], tl[2][2][4];
        const auto load_t = [&](int s) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (s <= own[j]) {
              const uint32_t a = tt + block_of(own[j], s) * kBlock + row32_at(b_row, b_piece);
              ldsm4(th[s & 1][j], a);
              ldsm4(tl[s & 1][j], a + kTri);
            }
        };
        load_t(0);
        float2 cc[2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int q = 0; q < 2; ++q)
            cc[j][q] =
                *reinterpret_cast<const float2 *>(vec + kVecC * kC + 16 * own[j] + 8 * q + 2 * t);
        const float4 misc = *reinterpret_cast<const float4 *>(vec + kVecMisc * kC);
        bar_sync(bar_x, all);
        // x_i = beta_i v_i - c_i (S k_i); vec holds -c_i 2^16.  Its scale comes from
        // norms, so that the warps agree on it without another exchange:
        // |S k_i| <= |S| |k_i|, where k_i (scaled) stays below 2^15 and each
        // share of S below 2^15 i0 per element.
        const float2 si = add2(gs.s_inv[0][lane], gs.s_inv[1][lane]);
        const float2 va = gs.v_max[0][lane], vb = gs.v_max[1][lane];
        const float2 vm = make_float2(fmaxf(va.x, vb.x), fmaxf(va.y, vb.y));
        const float gamma = misc.x, tau = misc.y, back = misc.y * misc.z;
        const float reach = misc.w * (0x1p30f * (C::kCols == 32 ? 5.66f : 8.0f));  // sqrt
        // (A run that writes nothing has a bound of 0.)
        float n0, n1, j0, j1;
        pow2_scale(fmaf(reach, si.x, vm.x), n0, j0);
        pow2_scale(fmaf(reach, si.y, vm.y), n1, j1);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 y[2] = {gs.x_part[own[j]][0][lane], gs.x_part[own[j]][1][lane]};
          const float4 z[2] = {gs.y[own[j]][0][lane], gs.y[own[j]][1][lane]};
          Acc x[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            x[q].top = add2(mine[j][q].top, make_float2(y[q].x, y[q].y));
            x[q].low = add2(mine[j][q].low, make_float2(y[q].z, y[q].w));
            x[q].top = fma2(cc[j][q], x[q].top, make_float2(z[q].x, z[q].y));
            x[q].low = fma2(cc[j][q], x[q].low, make_float2(z[q].z, z[q].w));
          }
          uint32_t hi[4], lo[4];
          split_frag(x[0], x[1], n0, n1, hi, lo);
          put4(&gs.x_frag[own[j]][0][lane], hi);
          put4(&gs.x_frag[own[j]][1][lane], lo);
        }
        float2 ts[2][2], dd[2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int col = 16 * own[j] + 8 * q + 2 * t;
            ts[j][q] = *reinterpret_cast<const float2 *>(vec + kVecT * kC + col);
            dd[j][q] = *reinterpret_cast<const float2 *>(vec + kVecD * kC + col);
          }
        bar_sync(bar_y, 32 * kHalves);
        // u = T x
        Acc U[2][2] = {}, V[2][2] = {}, W[2][2] = {};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          if (s > own[1]) continue;  // the larger one
          uint32_t hi[4], lo[4];
          get4(&gs.x_frag[s][0][lane], hi);
          get4(&gs.x_frag[s][1][lane], lo);
          if (s < 3) load_t(s + 1);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (s <= own[j])
#pragma unroll
              for (int q = 0; q < 2; ++q) {
                mma16(U[j][q], hi, th[s & 1][j][2 * q], th[s & 1][j][2 * q + 1]);
                mma16(V[j][q], hi, tl[s & 1][j][2 * q], tl[s & 1][j][2 * q + 1]);
                mma16(W[j][q], lo, th[s & 1][j][2 * q], th[s & 1][j][2 * q + 1]);
              }
        }
        // Rescaled by T's row scales and down by a bound of its row sums, u
        // stays below 2^15 (the scale of x), and so does w_j = Gamma_64,j
        // kappa_j u_j over the largest such factor.
        if (part == 0) gs.u_inv[lane] = make_float2(j0 * tau, j1 * tau);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t f[4], hi[4], lo[4];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float2 top = mul2(add2(U[j][q].top, add2(V[j][q].top, W[j][q].top)), ts[j][q]);
            const float2 low = mul2(add2(U[j][q].low, add2(V[j][q].low, W[j][q].low)), ts[j][q]);
            f[2 * q] = h2_bits(__float22half2_rn(top));
            f[2 * q + 1] = h2_bits(__float22half2_rn(low));
            split_h2(mul2(top, dd[j][q]), hi[2 * q], lo[2 * q]);
            split_h2(mul2(low, dd[j][q]), hi[2 * q + 1], lo[2 * q + 1]);
          }
          put4(&gs.w_frag[own[j]][0][lane], hi);
          put4(&gs.w_frag[own[j]][1][lane], lo);
          put4(&gs.u_frag[own[j]][lane], f);
        }
        bar_sync(bar_w, kGroup);
        // S = gamma S + sum_j w_j k_j^T, up to 32 key channels at a time
        uint32_t wh[4][4], wl[4][4];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          get4(&gs.w_frag[s][0][lane], wh[s]);
          get4(&gs.w_frag[s][1][lane], wl[s]);
        }
        const float2 b0 = both(j0 * back), b1 = both(j1 * back);
        constexpr int kAt = 2;  // 16-channel blocks at a time
        float a0 = 0.0f, a1 = 0.0f;
#pragma unroll
        for (int np = 0; np < C::kSteps; np += kAt) {
          Acc acc[2 * kAt] = {};
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            uint32_t bb[kAt][4];
#pragma unroll
            for (int j = 0; j < kAt; ++j)
              ldsm4_t(bb[j], kt + tile_at<DK>(16 * s + bt_row,
                                              part * (C::kCols / 8) + 2 * (np + j) + bt_piece));
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
              mma16(acc[2 * j], wh[s], bb[j][0], bb[j][1]);
              mma16(acc[2 * j + 1], wh[s], bb[j][2], bb[j][3]);
            }
#pragma unroll
            for (int j = 0; j < kAt; ++j) {
              mma16(acc[2 * j], wl[s], bb[j][0], bb[j][1]);
              mma16(acc[2 * j + 1], wl[s], bb[j][2], bb[j][3]);
            }
          }
#pragma unroll
          for (int q = 0; q < 2 * kAt; ++q) {
            Acc &a = S[2 * np + q];
            a.top = fma2(acc[q].top, b0, mul2(both(gamma), a.top));
            a.low = fma2(acc[q].low, b1, mul2(both(gamma), a.low));
            a0 = max3_abs(a0, a.top.x, a.top.y);
            a1 = max3_abs(a1, a.low.x, a.low.y);
          }
        }
        if (++st == kStages) st = 0;
        pow2_scale(quad_max(a0), m0, i0);
        pow2_scale(quad_max(a1), m1, i1);
      }
      if (seq.state_out) {
#pragma unroll
        for (int n = 0; n < 2 * C::kSteps; ++n) {
          *reinterpret_cast<float2 *>(seq.state_out + at + 8 * n) = S[n].top;
          *reinterpret_cast<float2 *>(seq.state_out + at + 8 * DK + 8 * n) = S[n].low;
        }
      }
    }
    return;
  }

  // Output warps: o_i = rho_i gamma_i (S q_i) + sum_j P_ij u_j.  They also bring
  // in the group's values, as beta v in the chain's accumulator layout.  Each
  // has two of the four 16-token blocks, an equal share of P's triangle.
  const int side = part;
  const int own[2] = {side, 3 - side};
  const int my_row = lane >> 1;  // of a block, and the half row this lane copies
  const uint32_t v_smem = ptx::smem_u32(gs.v[0]), v_to = v_smem + row32_at(my_row, lane & 1);
  const uint32_t v_at = v_smem + row32_at(b_row, b_piece);
  // The only wait for a chunk's operands: bar_w passes it on.  One that gave
  // up is not repeated; the loops run to their end on whatever the ring holds,
  // so that all warps pass every barrier.
  bool dead = false;
  const auto wait_full = [&](int stage, uint32_t parity) {
    if (!dead)
      dead = __any_sync(kFull, !ptx::mbar_wait(&full[stage], parity, abort_flag, budget_ns));
  };
  // beta v of a chunk (the last copy but one) and its largest per row
  const auto values = [&](int slot, int stage) {
    cp_async_wait<1>();
    __syncwarp();
    const float *vec =
        reinterpret_cast<const float *>(ring_a + stage * C::kStageA + kKeyTile + 2 * kTri);
    float top = 0.0f, low = 0.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t vv[4];
      ldsm4_t(vv, v_at + slot * kC * 32 + own[j] * 16 * 32);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float2 be =
            *reinterpret_cast<const float2 *>(vec + kVecBeta * kC + 16 * own[j] + 8 * q + 2 * t);
        const float2 y0 = mul2(be, make_float2(bf16_lo(vv[2 * q]), bf16_hi(vv[2 * q])));
        const float2 y1 = mul2(be, make_float2(bf16_lo(vv[2 * q + 1]), bf16_hi(vv[2 * q + 1])));
        gs.y[own[j]][q][lane] = make_float4(y0.x, y0.y, y1.x, y1.y);
        top = max3_abs(top, y0.x, y0.y);
        low = max3_abs(low, y1.x, y1.y);
      }
    }
    gs.v_max[side][lane] = make_float2(quad_max(top), quad_max(low));
  };
  // Of every chunk's four copies -- k or T's part into ring a, q or P's into
  // ring b -- this warp's first lanes have one each.
  const int mine = 2 / groups_on;
  const bool copies = lane < mine;
  const int copy = (2 * group + side) * mine + (copies ? lane : 0);
  const bool into_b = copy & 2, of_head = copy & 1;
  const size_t from_step = of_head ? static_cast<size_t>(d.v_heads) * kHeadBlob
                                   : static_cast<size_t>(d.qk_heads) * kKeyBlob<DK>;
  const uint32_t copy_bytes = !of_head ? kKeyTile : into_b ? kPartB : kPartA;
  const uint32_t to_step = into_b ? C::kStageB : C::kStageA;
  const uint32_t to = ptx::smem_u32(into_b ? ring_b : ring_a) + (of_head ? kKeyTile : 0);
  int fed = 0;  // chunks under way
  // The next chunk to bring in, two before the one worked on: of piece number
  // `ahead`, `left` tokens from its first on.  The record of the piece after it
  // is under way; of those brought in but not yet begun (two at most), their
  // tokens and where their outputs go wait in line.
  int ahead = -1, left = 0, index = piece_at(0);
  int4 record = first;
  Place place = place_of(index);
  const uint8_t *from = nullptr;
  const moe_bf16 *v_src = nullptr, *v_now = nullptr;  // v_now, v_left: the chunk brought in last
  int v_left = 0;
  moe_bf16 *line_dst[2] = {};
  int line_len[2] = {};
  const auto bring_in = [&](int stage, bool alive) {
    const bool begins = left <= 0 && index < total;
    if (begins) {
      ++ahead;
      const int h = place.h, dv = place.row + group * 16;
      const bool second = line_len[0] > 0;
      moe_bf16 *dst = out + (static_cast<int64_t>(record.x) + my_row) * out_ld + h * d.v_dim + dv +
                      (lane & 1) * 8;
      (second ? line_dst[1] : line_dst[0]) = dst;
      (second ? line_len[1] : line_len[0]) = record.y;
      const size_t base = record.w;
      left = record.y;
      from = of_head ? ws_head + (base * d.v_heads + h) * kHeadBlob + (into_b ? kPartA : 0)
                     : ws_key + (base * d.qk_heads + h / ratio) * kKeyBlob<DK> +
                           (into_b ? kKeyTile : 0);
      v_src = in.v + (static_cast<int64_t>(record.x) + my_row) * in.v_ld + h * d.v_dim + dv +
              (lane & 1) * 8;
      // the group's state, a line of 128 bytes each, on its way into L2
      constexpr int kLines = DK / 32;
      const int line = 32 * side + lane;
      if (ahead > 0 && seq.state_in && line < 16 * kLines)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(
            seq.state_in + ((static_cast<int64_t>(record.z) * d.v_heads + h) * d.v_dim + dv +
                            line / kLines) * DK + line % kLines * 32));
    }
    v_now = v_src, v_left = left;
    if (left > 0) {
      if (alive) {
        if (copies) {
          mbar_expect(&full[stage], copy_bytes);
          bulk_load(to + stage * to_step, from, copy_bytes, &full[stage]);
        }
        ++fed;
      }
      v_src += kC * in.v_ld, from += from_step, left -= kC;
    }
    if (begins) {
      index = piece_at(ahead + 1);
      if (index < total) {
        place = place_of(index);
        record = list[place.b];
      }
    }
  };
  // the own blocks of its values, zeros past the end
  const auto fetch_v = [&](int slot) {
    if (v_left > 0) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const bool live = 16 * own[j] + my_row < v_left;
        cp_async16(v_to + slot * kC * 32 + own[j] * 16 * 32,
                   live ? v_now + 16 * own[j] * in.v_ld : in.v, live);
      }
    }
    cp_async_commit();
  };
  int st = 0;  // stage of the rings, and slot of the values
  static_assert(kStages == 3, "as many as slots of the values");
  uint32_t parity = 0;
  // the piece worked on: its number, its tokens from this chunk on
  int number = -1, now = 0;
  moe_bf16 *o_dst = nullptr;
  const bool asks = group == 0 && side == 0 && lane == 0;
  int asked = total;  // its answer: piece number + 3
  if (asks && total > 3 * grid) asked = 3 * grid + atomicAdd(&head[kNextWord], 1u);
  const auto begin_next = [&] {
    now = line_len[0], o_dst = line_dst[0];
    line_len[0] = line_len[1], line_dst[0] = line_dst[1], line_len[1] = 0;
    ++number;
    if (asks) {
      queue[(number + 3) % C::kQueue] = asked;
      if (asked < total) asked = 3 * grid + atomicAdd(&head[kNextWord], 1u);
    }
  };
  if (piece_at(0) < total) {
    bring_in(0, true);
    fetch_v(0);
    bring_in(1, true);
    begin_next();
    wait_full(0, 0);
    bar_sync(bar_w, kGroup);
  }
  const uint32_t o_at = ptx::smem_u32(gs.o) + row32_at(b_row, b_piece);
  const uint8_t *o_from = gs.o + row32_at(my_row, lane & 1);
  // The next chunk can be brought in any time after bar_x, when the stage of the
  // one before is free.  Issuing its copy takes 500 cycles; where S q^T has half
  // as many products the chain waits for them less before bar_w, else after it:
  // 8 prompts (8 heads of 64) 111 us before it and 120 after, 8192 tokens (32 heads
  // of 128) 320.7 before it and 312.5 after.
  constexpr bool kLate = DK == 128;
  const auto bring_next = [&] {
    const int given_up = *reinterpret_cast<volatile int *>(abort_flag);
    bring_in(st == 0 ? kStages - 1 : st - 1, !__any_sync(kFull, given_up));
  };
  for (int n = 0; now > 0; ++n) {
    const uint32_t qt = ptx::smem_u32(ring_b + st * C::kStageB), pt = qt + kKeyTile;
    const float *vec = reinterpret_cast<const float *>(ring_b + st * C::kStageB + kKeyTile + kTri);
    const int next = st + 1 == kStages ? 0 : st + 1;
    fetch_v(next);
    values(st, st);
    uint32_t bb[2][2][4];
    const auto load_q = [&](int s) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        ldsm4(bb[s & 1][j], qt + tile_at<DK>(16 * own[j] + b_row, 2 * s + b_piece));
    };
    load_q(0);
    bar_sync(bar_x, all);
    // The shares of S have scales of their own: brought to the largest.
    uint32_t a[DK / 16][4];
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) get4(&gs.s_frag[s][lane], a[s]);
    const float2 si[2] = {gs.s_inv[0][lane], gs.s_inv[1][lane]};
    const float2 most = make_float2(fmaxf(si[0].x, si[1].x), fmaxf(si[0].y, si[1].y));
    float down0, down1, unused;
    pow2_above(most.x * 0.5f, unused, down0);  // 1 / most, a power of two
    pow2_above(most.y * 0.5f, unused, down1);
    Acc O[2][2] = {};
#pragma unroll
    for (int s = 0; s < DK / 16; ++s) {
      const float2 f = si[s / C::kSteps];
      const __half2 f0 = __float2half2_rn(f.x * down0), f1 = __float2half2_rn(f.y * down1);
      if (s + 1 < DK / 16) load_q(s + 1);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        a[s][e] = h2_bits(__hmul2(*reinterpret_cast<const __half2 *>(&a[s][e]), (e & 1) ? f1 : f0));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mma16(O[j][0], a[s], bb[s & 1][j][0], bb[s & 1][j][1]);
        mma16(O[j][1], a[s], bb[s & 1][j][2], bb[s & 1][j][3]);
      }
    }
    // what the second product needs, and the first one's factors, ahead of it
    uint32_t pf[4][2][4];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (s <= own[j])
          ldsm4(pf[s][j], pt + block_of(own[j], s) * kBlock + row32_at(b_row, b_piece));
    float2 pi[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int col = 16 * own[j] + 8 * q + 2 * t;
        const float2 oq = *reinterpret_cast<const float2 *>(vec + kVecO * kC + col);
        pi[j][q] = *reinterpret_cast<const float2 *>(vec + kVecP * kC + col);
        O[j][q].top = mul2(mul2(O[j][q].top, both(most.x * kDown)), oq);
        O[j][q].low = mul2(mul2(O[j][q].low, both(most.y * kDown)), oq);
      }
    const uint32_t next_parity = next ? parity : parity ^ 1;
    if constexpr (!kLate) bring_next();
    if (fed > n + 1) wait_full(next, next_parity);
    bar_sync(bar_w, kGroup);
    if constexpr (kLate) bring_next();
    const float2 ui = mul2(gs.u_inv[lane], both(kDown));
    Acc I[2][2] = {};
    uint32_t uf[4][4];
#pragma unroll
    for (int s = 0; s < 4; ++s) get4(&gs.u_frag[s][lane], uf[s]);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (s <= own[j]) {
          mma16(I[j][0], uf[s], pf[s][j][0], pf[s][j][1]);
          mma16(I[j][1], uf[s], pf[s][j][2], pf[s][j][3]);
        }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float2 top = fma2(mul2(I[j][q].top, both(ui.x)), pi[j][q], O[j][q].top);
        const float2 low = fma2(mul2(I[j][q].low, both(ui.y)), pi[j][q], O[j][q].low);
        w[2 * q] = pack_bf16(top.x, top.y);
        w[2 * q + 1] = pack_bf16(low.x, low.y);
      }
      // transposed back: token rows of 16 channels
      stsm4_t(o_at + own[j] * 16 * 32, w[0], w[1], w[2], w[3]);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (16 * own[j] + my_row < now)
        *reinterpret_cast<uint4 *>(o_dst + 16 * own[j] * out_ld) =
            *reinterpret_cast<const uint4 *>(o_from + own[j] * 16 * 32);
    o_dst += kC * out_ld, now -= kC;
    if (now <= 0) begin_next();
    st = next, parity = next_parity;
    __syncwarp();
  }
  cp_async_wait<0>();
  // Copies in flight land before the CTA's shared memory is given up.  After a
  // wait that gave up, some of the four may have issued one more than the
  // others, whose arrivals its barrier then still waits for.
  if (copies) fed_by[copy] = fed;
  bar_sync(bar_out, 64 * groups_on);
  if (copies) {
    const int last = max(max(fed_by[0], fed_by[1]), max(fed_by[2], fed_by[3]));
    for (; fed < last; ++fed) ptx::mbar_arrive(&full[fed % kStages]);
    int ignore = 0;
    for (int c = max(0, fed - kStages); c < fed; ++c)
      ptx::mbar_wait(&full[c % kStages], (c / kStages) & 1, &ignore, ptx::kDrainBudgetNs);
    if (*reinterpret_cast<volatile int *>(abort_flag)) set_status(seq.status, MOE_DEV_TIMEOUT);
  }
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

template <int DK>
cudaError_t launch_chain(const moe_delta_dims &d, const moe_delta_inputs &in, const DeltaSeqs &seq,
                         uint8_t *ws, const int4 *list, const uint8_t *ws_key,
                         const uint8_t *ws_head, moe_bf16 *out, int64_t out_ld, cudaStream_t s) {
  using C = Chain<DK>;
  static_assert(C::kSmem <= 227 * 1024, "shared memory of one SM");
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(delta_chain_kernel<DK>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  const int pieces = seq.B * d.v_heads * (d.v_dim / 16), sms = tc_sm_count();
  return launch_early(delta_chain_kernel<DK>, dim3(pieces < sms ? pieces : sms), C::kThreads,
                      C::kSmem, s, d, in, seq, ws, list, ws_key, ws_head, out, out_ld,
                      tc_wait_budget_ns());
}

// The sequences' records, up to a whole 256 bytes.
size_t list_bytes(int B) { return (static_cast<size_t>(B) * sizeof(int4) + 255) / 256 * 256; }

template <int DK>
cudaError_t launch(const moe_delta_dims &d, const moe_delta_inputs &in, const DeltaSeqs &seq,
                   uint8_t *ws, moe_bf16 *out, int64_t out_ld, cudaStream_t s) {
  const ChunkSlots slots = chunk_slots(seq.N, seq.B);
  int4 *list = reinterpret_cast<int4 *>(ws + kHeader);
  uint8_t *ws_key = ws + kHeader + list_bytes(seq.B);
  uint8_t *ws_head = ws_key + slots.count * d.qk_heads * kKeyBlob<DK>;
  constexpr int kSmem = sizeof(PrepSmem<DK>);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(delta_prep_kernel<DK>, kSmem, done);
  if (e != cudaSuccess) return e;
  const int ratio = d.v_heads / d.qk_heads;
  // A CTA serves several of the value heads of its key head (and forms k k^T
  // and q k^T once for them) when there are enough to fill the SMs so: 8192
  // tokens take 312.5 us with two heads of 32 to a CTA, 328.7 with one, 13
  // sequences of 6007 tokens 240.5 and 253.6, 2048 tokens 89.6 and 90.5; where
  // there are not, 67 tokens take 20.0 and 16.4, 512 beside 32 of one 66.7 and
  // 61.4.
  int heads = 1;
  if (slots.count * d.qk_heads >= static_cast<size_t>(kPrepCtas * tc_sm_count()))
    for (int n = 2; n <= kPrepHeads; ++n)
      if (ratio % n == 0) heads = n;
  const dim3 grid(static_cast<unsigned>(slots.count) + 1, d.v_heads / heads);
  e = launch_early(delta_prep_kernel<DK>, grid, kPrepThreads, kSmem, s, d, in, seq, slots, heads,
                   tc_sm_count(), ws, list, ws_key, ws_head);
  if (e != cudaSuccess) return e;
  e = launch_chain<DK>(d, in, seq, ws, list, ws_key, ws_head, out, out_ld, s);
  if (e != cudaSuccess || !seq.cu_seqlens) return e;  // the one sequence is longer
  return launch_delta_recurrent(d, in, seq, kDeltaShort,
                                reinterpret_cast<const uint32_t *>(ws) + kFlagWord, out, out_ld, s);
}

}  // namespace

size_t delta_chunk_workspace(const moe_delta_dims &d, int N, int B) {
  const size_t slots = chunk_slots(N, B).count;
  const size_t key = d.qk_dim == 128 ? kKeyBlob<128> : kKeyBlob<64>;
  return kHeader + list_bytes(B) +
         slots * (d.qk_heads * key + static_cast<size_t>(d.v_heads) * kHeadBlob);
}

cudaError_t launch_delta_chunk(const moe_delta_dims &d, const moe_delta_inputs &in,
                               const DeltaSeqs &seq, void *ws, moe_bf16 *out, int64_t out_ld,
                               cudaStream_t s) {
  return d.qk_dim == 128 ? launch<128>(d, in, seq, static_cast<uint8_t *>(ws), out, out_ld, s)
                         : launch<64>(d, in, seq, static_cast<uint8_t *>(ws), out, out_ld, s);
}

}  // namespace moe
