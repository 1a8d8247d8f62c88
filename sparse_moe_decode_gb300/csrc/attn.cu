// attn.cu -- paged attention: the choice of the kernel, its workspace, and the
// kernel that joins the tiles which several blocks worked on.
//
// Joining is bound by latency: a list of the tiles, their maxima and totals, then
// the sums, a few MB in the L2 (verification of 8 sequences of 4, 16 heads of 256 on
// 2 over 8192: 9.8 us of the 35 that the two kernels take one by one; in a stream,
// where its launch overlaps, 3 of 26).
#include "attn_launch.h"
#include "early.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kCombineThreads = 256, kCombineWarps = kCombineThreads / 32;

// Up to 32 of a tile's rows in 4 Q columns for each of the rest of the lanes:
// sum_i w_i o_i / sum_i w_i l_i with w_i = 2^(m_i - max m) over the blocks that
// worked on it.  A warp does it (Q = 8); where tiles are few and blocks per tile
// many, the warps of a block share the blocks out (Q = 2).
template <int Q, bool TOGETHER>
__device__ __forceinline__ void combine(const AttnBatch &a, const AttnArgs &p, int D, int count,
                                        const int *list, float4 (*part)[32], float2 *part_ml) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int R = p.parts.rows, side = R < 32 ? R : 32, subs = 32 / side;
  const int cols = 4 * Q * subs, row_tasks = R / side, tasks = row_tasks * (D / cols);
  const int total = count * tasks;
  for (int t = TOGETHER ? blockIdx.x : blockIdx.x + warp * gridDim.x; t < total;
       t += TOGETHER ? gridDim.x : gridDim.x * kCombineWarps) {
    const int b0 = list[t / tasks], in = t % tasks;
    const AttnOpen o = p.parts.open[b0];
    // (neighbouring tasks are columns of the same rows: a tile need not have them all)
    const int row0 = in / (D / cols) * side;
    if (row0 >= o.rows) continue;
    const int r = row0 + lane % side;
    const int d = in % (D / cols) * cols + lane / side * (4 * Q);
    const int n = o.last - b0 + 1;
    float m = -INFINITY, l = 0.0f;
    float4 v[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) v[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const auto add = [&](float2 ml, const float4 (&x)[Q]) {
      // a part that saw no key has no sums (one that saw keys of NaN alone has NaN of them)
      if (ml.x == -INFINITY && ml.y == 0.0f) return;
      const float top = fmaxf(m, ml.x);
      const float f = attn_exp2(m - top), g = attn_exp2(ml.x - top);
      m = top;
      l = l * f + ml.y * g;
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        v[q].x = v[q].x * f + x[q].x * g, v[q].y = v[q].y * f + x[q].y * g;
        v[q].z = v[q].z * f + x[q].z * g, v[q].w = v[q].w * f + x[q].w * g;
      }
    };
    if (r < o.rows) {
      constexpr int kAhead = TOGETHER ? 4 : 2;
      for (int i0 = TOGETHER ? warp : 0; i0 < n; i0 += kAhead * (TOGETHER ? kCombineWarps : 1)) {
        float2 ml[kAhead];
        float4 x[kAhead][Q];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int i = i0 + k * (TOGETHER ? kCombineWarps : 1);
          ml[k] = make_float2(-INFINITY, 0.0f);
          if (i < n) {
            const int64_t slot = i == 0 ? 2 * b0 + 1 : 2 * (b0 + i);
            ml[k] = p.parts.ml[slot * R + r];
#pragma unroll
            for (int q = 0; q < Q; ++q)
              x[k][q] = *reinterpret_cast<const float4 *>(p.parts.at(slot, D, d + 4 * q, r));
          }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) add(ml[k], x[k]);
      }
    }
    if (TOGETHER) {
#pragma unroll
      for (int q = 0; q < Q; ++q) part[warp * Q + q][lane] = v[q];
      part_ml[warp * 32 + lane] = make_float2(m, l);
      __syncthreads();
      if (warp == 0)
        for (int k = 1; k < kCombineWarps; ++k) {
          float4 x[Q];
#pragma unroll
          for (int q = 0; q < Q; ++q) x[q] = part[k * Q + q][lane];
          add(part_ml[k * 32 + lane], x);
        }
    }
    if ((!TOGETHER || warp == 0) && r < o.rows) {
      const int token = attn_token(a, o.row0 + r), h = o.row0 + r - token * a.group;
      moe_bf16 *dst = p.out + (o.start + token) * p.out_ld + (o.head * a.group + h) * D + d;
      const float f = 1.0f / l;
#pragma unroll
      for (int q = 0; q < Q; q += 2)
        *reinterpret_cast<uint4 *>(dst + 4 * q) =
            make_uint4(pack_bf16(v[q].x * f, v[q].y * f), pack_bf16(v[q].z * f, v[q].w * f),
                       pack_bf16(v[q + 1].x * f, v[q + 1].y * f),
                       pack_bf16(v[q + 1].z * f, v[q + 1].w * f));
    }
    if (TOGETHER) __syncthreads();
  }
}

__global__ void __launch_bounds__(kCombineThreads)
attn_combine_kernel(const AttnBatch a, const AttnArgs p, int D, int blocks) {
  __shared__ int list[kStreamMaxCtas];
  __shared__ int count;
  __shared__ float4 part[kCombineWarps * 2][32];
  __shared__ float2 part_ml[kCombineWarps * 32];
  early_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    bool has[kStreamMaxCtas / 32];
#pragma unroll
    for (int i = 0; i < kStreamMaxCtas / 32; ++i)
      has[i] = 32 * i + lane < blocks && p.parts.open[32 * i + lane].last >= 0;
    int n = 0;
#pragma unroll
    for (int i = 0; i < kStreamMaxCtas / 32; ++i) {
      const unsigned mask = __ballot_sync(0xFFFFFFFFu, has[i]);
      if (has[i]) list[n + __popc(mask & ((1u << lane) - 1))] = 32 * i + lane;
      n += __popc(mask);
    }
    if (lane == 0) count = n;
  }
  __syncthreads();
  if (count == 0) return;
  if (blocks > 6 * count) combine<2, true>(a, p, D, count, list, part, part_ml);
  else combine<8, false>(a, p, D, count, list, part, part_ml);
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

struct Layout {
  size_t open, ml, sums, total;
};

Layout layout(const moe_attn_dims &d) {
  // both kernels' parts: 2 a block
  const size_t tc = 2 * kTcMaxCtas * (d.head_dim == 256 ? 128 : 256);
  size_t rows = 2 * kStreamMaxCtas * kStreamRows;
  if (tc > rows) rows = tc;
  Layout l;
  l.open = 256;
  l.ml = l.open + align256(kStreamMaxCtas * sizeof(AttnOpen));
  l.sums = l.ml + align256(rows * sizeof(float2));
  l.total = l.sums + rows * d.head_dim * 4;
  return l;
}

}  // namespace

bool attn_map(CUtensorMap *m, const void *base, int d, int size, int64_t rows, int box) {
  const int bytes = d * size;
  const CUtensorMapDataType dt =
      size == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if (bytes == 64) {  // two positions a line
    const uint64_t dims[3] = {128, static_cast<uint64_t>(rows) / 2, 1}, strides[2] = {128, 128};
    const uint32_t bx[3] = {128, static_cast<uint32_t>(box) / 2, 1};
    return tc_make_map3(m, base, dt, size, dims, strides, bx);
  }
  const uint64_t cols = static_cast<uint64_t>(bytes) / 128, inner = 128 / static_cast<uint64_t>(size);
  const uint64_t dims[3] = {inner, static_cast<uint64_t>(rows), cols};
  const uint64_t strides[2] = {static_cast<uint64_t>(bytes), 128};
  const uint32_t bx[3] = {static_cast<uint32_t>(inner), static_cast<uint32_t>(box),
                          static_cast<uint32_t>(cols)};
  return tc_make_map3(m, base, dt, size, dims, strides, bx);
}

bool attn_tc_map(CUtensorMap *m, const void *base, int d, int size, int64_t rows, int box, int cols) {
  const uint64_t dims[3] = {64, static_cast<uint64_t>(rows), static_cast<uint64_t>(d) / 64};
  const uint64_t strides[2] = {static_cast<uint64_t>(d) * size, static_cast<uint64_t>(64) * size};
  const uint32_t bx[3] = {64, static_cast<uint32_t>(box), static_cast<uint32_t>(cols)};
  if (size == 2)
    return tc_make_map3(m, base, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, dims, strides, bx);
  return tc_make_map_nd(m, base, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, dims, strides, bx);
}

cudaError_t launch_attn_combine(const AttnBatch &a, const AttnArgs &p, int d, int blocks,
                                cudaStream_t s) {
  return launch_early(attn_combine_kernel, dim3(4 * tc_sm_count()), kCombineThreads, 0, s, a, p, d,
                      blocks);
}

size_t attn_workspace(const moe_attn_dims &d) { return layout(d).total; }

cudaError_t launch_attention(const moe_attn_dims &d, const moe_kv_cache &c, const AttnBatch &a,
                             const moe_bf16 *q, int64_t q_ld, moe_bf16 *out, int64_t out_ld,
                             void *ws, cudaStream_t s) {
  const Layout l = layout(d);
  uint8_t *base = static_cast<uint8_t *>(ws);
  AttnLaunch x;
  x.k = c.k, x.v = c.v;
  x.cache_rows = c.pages * d.kv_heads * d.page_size;
  x.page = d.page_size;
  x.batch = a;
  x.stream = s;
  x.args.q = q, x.args.out = out;
  x.args.q_ld = q_ld, x.args.out_ld = out_ld;
  x.args.k_scale = c.k_scale, x.args.v_scale = c.v_scale;
  x.args.parts.open = reinterpret_cast<AttnOpen *>(base + l.open);
  x.args.parts.ml = reinterpret_cast<float2 *>(base + l.ml);
  x.args.parts.sums = reinterpret_cast<float *>(base + l.sums);
  x.args.parts.rows = 0;
  x.args.scale_log2 = attn_scale_log2(d);
  x.args.budget = tc_wait_budget_ns();
  const auto stream = d.kv_type == MOE_KV_BF16   ? launch_stream_bf16
                      : d.kv_type == MOE_KV_INT8 ? launch_stream_int8
                                                 : launch_stream_e4m3;
  const auto tc = d.kv_type == MOE_KV_BF16   ? launch_tc_bf16
                  : d.kv_type == MOE_KV_INT8 ? launch_tc_int8
                                             : launch_tc_e4m3;
  // Sequences of up to 16 rows stream; the others go to the tensor cores' kernel
  // (8 sequences of 4 tokens, 32 rows each, take 26 us there and 37 us
  // streaming).  Lengths that only the device knows: both kernels look.
  const int64_t most = static_cast<int64_t>(a.cu ? a.N : a.T) * a.group;
  cudaError_t e = cudaSuccess;
  if ((a.cu && a.group <= kStreamRows) || most <= kStreamRows) {
    x.range.least = 0, x.range.most = kStreamRows;
    x.args.least_share = 2;
    e = stream(x, d.head_dim);
  }
  if (e == cudaSuccess && most > kStreamRows) {
    x.range.least = kStreamRows, x.range.most = INT32_MAX;
    x.args.least_share = 1;
    e = tc(x, d.head_dim);
  }
  return e;
}

}  // namespace moe
