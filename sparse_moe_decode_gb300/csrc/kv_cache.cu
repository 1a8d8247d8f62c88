// kv_cache.cu -- the paged cache's rows written (and quantised) and read back.
//
// A row is one token's D values of one head of k or v; D / 8 lanes take it, 16
// bytes of bf16 each, and find its scale by shuffles; the same lanes take k and v,
// whose place in the cache they look up once, and a block one head's rows of some
// tokens.  A row is read and written once: 8192 tokens of 8 heads of 128 in e4m3,
// written and read back, 19.8 us, 5.1 TB/s.  (Rows of all heads and of k and v one
// after another, each with its own look-up, were bound by their instructions: 25.8.)
//
// int8: c is x / s, the exact quotient, rounded to the nearest.  c1, x times the
// rounded inverse, rounded, is off by one at most, and d = x - c1 s is exact: it is
// a multiple of s's last place and no larger than s, or c1 is 0.  So c = c1 where
// |d| <= s / 2, else its neighbour towards d.  Where x / s lies in the middle c has
// to be even, and c1 is: (c + 1/2) s with s of 24 digits has the 8 of x only where s
// is a power of two (s = max / 127 rounded is one, or has no end within 24 digits),
// and then its inverse is exact.
// e4m3: s is a power of two, so x / s is exact and the conversion rounds once.
#include "attn.h"
#include "attn_sched.cuh"
#include "early.cuh"
#include "kernels.h"
#include "pair.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;

struct KvSide {  // of k or v
  const moe_bf16 *in;
  moe_bf16 *out;
  int64_t ld;
  void *store;
  float *scale;
};

// Where token t's row of `head` lies in the cache; -1: nowhere.
__device__ __forceinline__ int64_t kv_place(const AttnBatch &a, int t, int head, AttnSeq &s,
                                            int &b) {
  if (b < 0 || t < s.start || t >= s.start + s.n) {
    if (a.cu) {
      int low = 0, high = a.B;  // cu[low] <= t < cu[high]
      while (high - low > 1) {
        const int mid = (low + high) / 2;
        if (a.cu[mid] <= t) low = mid;
        else high = mid;
      }
      b = low;
    } else {
      b = t / a.T;
    }
    s = attn_seq(a, b, false);
    if (t < s.start || t >= s.start + s.n) {
      b = -1;
      return -1;
    }
  }
  const int pos = s.len - s.n + (t - s.start);
  const int page = a.table[b * a.table_ld + (pos >> a.page_shift)];
  if (page < 0 || page >= a.pages) {
    set_status(a.status, MOE_DEV_BAD_INDEX);
    return -1;
  }
  return ((static_cast<int64_t>(page) * a.kv_heads + head) << a.page_shift) +
         (pos & ((1 << a.page_shift) - 1));
}

// The scale of a row whose largest magnitude is `top`, and its inverse.
template <int KV>
__device__ __forceinline__ void kv_scale(float top, float &s, float &inv) {
  if (KV == MOE_KV_INT8) {
    s = fmaxf(__fdiv_rn(top, 127.0f), 0x1p-126f);
    inv = __frcp_rn(s);
  } else {
    // top = m 2^e, 448 = 1.75 * 2^8: s = 2^(e - 8), twice that where m > 1.75
    const int e = static_cast<int>((__float_as_uint(top) + 0x1FFFFFu) >> 23) - 8;
    const uint32_t f = static_cast<uint32_t>(max(e, 1));
    s = __uint_as_float(f << 23);
    inv = __uint_as_float((254u - f) << 23);
  }
}

__device__ __forceinline__ uint32_t int8_code(float x, float s, float inv) {
  // 1.5 * 2^23 + c: the low byte is c in two's complement
  constexpr float kPlace = 12582912.0f;
  const float c = fmaf(x, inv, kPlace), d = fmaf(kPlace - c, s, x);
  // (half of a scale next to 2^-126 may have no last place: d does not reach between)
  return __float_as_uint(fabsf(d) > __fmul_rz(0.5f, s) ? c + copysignf(1.0f, d) : c);
}

template <int KV>
__device__ __forceinline__ uint2 kv_codes(const float (&x)[8], float s, float inv) {
  uint32_t r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (KV == MOE_KV_INT8) {
      uint32_t c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = int8_code(x[4 * i + j], s, inv);
      r[i] = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
    } else {
      uint16_t lo, hi;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
          : "=h"(lo)
          : "f"(x[4 * i + 1] * inv), "f"(x[4 * i] * inv));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
          : "=h"(hi)
          : "f"(x[4 * i + 3] * inv), "f"(x[4 * i + 2] * inv));
      r[i] = lo | (static_cast<uint32_t>(hi) << 16);
    }
  }
  return make_uint2(r[0], r[1]);
}

template <int KV>
__device__ __forceinline__ void kv_values(uint2 c, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t v = i ? c.y : c.x;
    if (KV == MOE_KV_INT8) {
      const f4 f = i8x4_to_f32(v);
      x[4 * i] = f.x, x[4 * i + 1] = f.y, x[4 * i + 2] = f.z, x[4 * i + 3] = f.w;
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v >> (16 * j))));
        asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\t"
            "cvt.f32.f16 %1, u;\n\t}"
            : "=f"(x[4 * i + 2 * j]), "=f"(x[4 * i + 2 * j + 1])
            : "r"(h));
      }
    }
  }
}

// Block (x, y): kRows * EACH tokens' rows of k and v of head y.
template <int D, int KV, bool WRITE, int EACH>
__global__ void __launch_bounds__(kThreads)
kv_rows_kernel(const AttnBatch a, const KvSide k, const KvSide v) {
  constexpr int kLanes = D / 8, kRows = kThreads / kLanes;
  early_begin();
  if (blockIdx.x + blockIdx.y == 0)
    for (int b = threadIdx.x; b < a.B; b += kThreads) attn_seq(a, b, true);
  const int l = threadIdx.x % kLanes, head = blockIdx.y;
  const int first = blockIdx.x * (kRows * EACH) + threadIdx.x / kLanes;
  // (places and sides by constants: an index would put them into local memory)
  const auto side = [&](int i) -> const KvSide & { return i % 2 ? v : k; };
  uint4 data[2 * EACH];
  if (WRITE) {
#pragma unroll
    for (int i = 0; i < 2 * EACH; ++i) {
      const int t = first + i / 2 * kRows;
      if (t < a.N) data[i] = ld_nc(side(i).in + t * side(i).ld + head * D + l * 8);
    }
  }
  int64_t place[EACH];
  AttnSeq s;
  int b = -1;
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    const int t = first + e * kRows;
    place[e] = t < a.N ? kv_place(a, t, head, s, b) : -1;
  }
  if (WRITE) {
#pragma unroll
    for (int i = 0; i < 2 * EACH; ++i) {
      const int64_t at = place[i / 2];
      if (KV == MOE_KV_BF16) {
        if (at >= 0)
          *reinterpret_cast<uint4 *>(static_cast<moe_bf16 *>(side(i).store) + at * D + l * 8) =
              data[i];
        continue;
      }
      const uint32_t w[4] = {data[i].x, data[i].y, data[i].z, data[i].w};
      float x[8];
      // magnitudes order like their bits, inf and NaN above all; two at a time
      uint32_t both = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] = bf16_lo(w[j]), x[2 * j + 1] = bf16_hi(w[j]);
        both = __vmaxu2(both, w[j] & 0x7FFF7FFFu);
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1)
        both = __vmaxu2(both, __shfl_xor_sync(0xFFFFFFFFu, both, o));
      const uint32_t most = max(both << 16, both & 0xFFFF0000u);
      float scale, inv;
      kv_scale<KV>(__uint_as_float(most), scale, inv);
      uint2 c = kv_codes<KV>(x, scale, inv);
      if (most >= 0x7F800000u) c = make_uint2(0, 0), scale = __uint_as_float(0x7FC00000u);
      if (at >= 0) {
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(side(i).store) + at * D + l * 8) = c;
        if (l == 0) side(i).scale[at] = scale;
      }
    }
  } else {
    float scale[2 * EACH];
#pragma unroll
    for (int i = 0; i < 2 * EACH; ++i) {
      const int64_t at = place[i / 2];
      if (at < 0 || !side(i).out) continue;
      const uint8_t *from = static_cast<const uint8_t *>(side(i).store);
      if (KV == MOE_KV_BF16) {
        data[i] = *reinterpret_cast<const uint4 *>(from + (at * D + l * 8) * 2);
      } else {
        const uint2 c = *reinterpret_cast<const uint2 *>(from + at * D + l * 8);
        data[i].x = c.x, data[i].y = c.y;
        scale[i] = side(i).scale[at];
      }
    }
#pragma unroll
    for (int i = 0; i < 2 * EACH; ++i) {
      if (place[i / 2] < 0 || !side(i).out) continue;
      if (KV != MOE_KV_BF16) {
        float x[8];
        kv_values<KV>(make_uint2(data[i].x, data[i].y), x);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = pack_bf16(x[2 * j] * scale[i], x[2 * j + 1] * scale[i]);
        data[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      const int t = first + i / 2 * kRows;
      *reinterpret_cast<uint4 *>(side(i).out + t * side(i).ld + head * D + l * 8) = data[i];
    }
  }
}

template <int D, int KV, bool WRITE>
cudaError_t launch_rows(const AttnBatch &a, const KvSide (&io)[2], cudaStream_t s) {
  const auto go = [&](auto kernel, int tokens) {
    return launch_early(kernel, dim3((a.N + tokens - 1) / tokens, a.kv_heads), kThreads, 0, s, a,
                        io[0], io[1]);
  };
  // Two tokens a thread from 12 blocks an SM of one each (8 run at once): 4096 tokens of
  // 8 heads of 128 in e4m3 10.7 and 10.1 us, 16384 38.3 and 33.7; 1536 blocks 8.8 and
  // 9.3, 256 4.2 and 4.7.  (Four: 21.3 us where two take 19.8.)
  constexpr int kTokens = kThreads / (D / 8);
  if ((a.N + kTokens - 1) / kTokens * static_cast<int64_t>(a.kv_heads) < 12 * tc_sm_count())
    return go(kv_rows_kernel<D, KV, WRITE, 1>, kTokens);
  return go(kv_rows_kernel<D, KV, WRITE, 2>, 2 * kTokens);
}

template <int D, bool WRITE>
cudaError_t launch_rows_kv(int kv, const AttnBatch &a, const KvSide (&io)[2], cudaStream_t s) {
  if (kv == MOE_KV_BF16) return launch_rows<D, MOE_KV_BF16, WRITE>(a, io, s);
  if (kv == MOE_KV_INT8) return launch_rows<D, MOE_KV_INT8, WRITE>(a, io, s);
  return launch_rows<D, MOE_KV_E4M3, WRITE>(a, io, s);
}

template <bool WRITE>
cudaError_t launch_rows_any(const moe_attn_dims &d, const AttnBatch &a, const KvSide (&io)[2],
                            cudaStream_t s) {
  if (d.head_dim == 64) return launch_rows_kv<64, WRITE>(d.kv_type, a, io, s);
  if (d.head_dim == 128) return launch_rows_kv<128, WRITE>(d.kv_type, a, io, s);
  return launch_rows_kv<256, WRITE>(d.kv_type, a, io, s);
}

}  // namespace

cudaError_t launch_kv_write(const moe_attn_dims &d, const moe_kv_cache &c, const AttnBatch &a,
                            const moe_bf16 *k, int64_t k_ld, const moe_bf16 *v, int64_t v_ld,
                            cudaStream_t s) {
  const KvSide io[2] = {{k, nullptr, k_ld, c.k, c.k_scale}, {v, nullptr, v_ld, c.v, c.v_scale}};
  return launch_rows_any<true>(d, a, io, s);
}

cudaError_t launch_kv_read(const moe_attn_dims &d, const moe_kv_cache &c, const AttnBatch &a,
                           moe_bf16 *k, int64_t k_ld, moe_bf16 *v, int64_t v_ld, cudaStream_t s) {
  const KvSide io[2] = {{nullptr, k, k_ld, c.k, c.k_scale}, {nullptr, v, v_ld, c.v, c.v_scale}};
  return launch_rows_any<false>(d, a, io, s);
}

}  // namespace moe
