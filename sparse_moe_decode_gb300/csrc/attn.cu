// attn.cu -- paged attention: the choice of the kernel, its workspace, and the
// kernel that joins the tiles which several blocks worked on.
#include "attn_launch.h"
#include "early.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kCombineThreads = 256, kCombineWarps = kCombineThreads / 32;

// A tile's row in 128 columns (a lane has four): sum_i w_i o_i / sum_i w_i l_i
// with w_i = 2^(m_i - max m) over the blocks that worked on it.  A warp does
// it, or where tiles are few and blocks per tile many, the warps of a block
// share the blocks out.
__global__ void __launch_bounds__(kCombineThreads)
attn_combine_kernel(const AttnBatch a, const AttnArgs p, int D, int blocks) {
  __shared__ int list[kStreamMaxCtas];
  __shared__ int count;
  __shared__ float4 part[kCombineWarps][32];
  __shared__ float part_l[kCombineWarps];
  early_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    int n = 0;
    for (int i0 = 0; i0 < blocks; i0 += 32) {
      const bool has = i0 + lane < blocks && p.parts.open[i0 + lane].last >= 0;
      const unsigned mask = __ballot_sync(0xFFFFFFFFu, has);
      if (has) list[n + __popc(mask & ((1u << lane) - 1))] = i0 + lane;
      n += __popc(mask);
    }
    if (lane == 0) count = n;
  }
  __syncthreads();
  if (count == 0) return;
  const int R = p.parts.rows, chunks = D > 128 ? D / 128 : 1;
  const bool together = blocks > 6 * count;
  const int64_t tasks = static_cast<int64_t>(count) * R * chunks;
  const int64_t step = together ? gridDim.x : static_cast<int64_t>(gridDim.x) * kCombineWarps;
  // (neighbouring tasks in different blocks)
  for (int64_t t = blockIdx.x + (together ? 0 : static_cast<int64_t>(warp) * gridDim.x); t < tasks;
       t += step) {
    const int b0 = list[t / (R * chunks)];
    const AttnOpen o = p.parts.open[b0];
    const int r = static_cast<int>(t % (R * chunks)) / chunks, d = static_cast<int>(t % chunks) * 128 + 4 * lane;
    if (r >= o.rows) continue;  // (the same for all warps that share a task)
    const int n = o.last - b0 + 1;
    const auto slot = [&](int i) {
      return static_cast<int64_t>(i == 0 ? 2 * b0 + 1 : 2 * (b0 + i)) * R + r;
    };
    float top = -INFINITY;
    for (int i = lane; i < n; i += 32) top = fmaxf(top, p.parts.ml[slot(i)].x);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float l = 0.0f;
#pragma unroll 4
    for (int i = together ? warp : 0; i < n; i += together ? kCombineWarps : 1) {
      const int64_t at = slot(i);
      const float2 ml = p.parts.ml[at];
      const float w = ml.x == -INFINITY ? 0.0f : attn_exp2(ml.x - top);
      l += w * ml.y;
      if (d < D && ml.x != -INFINITY) {  // (a part that saw no key has no sums)
        const float4 x = *reinterpret_cast<const float4 *>(p.parts.sums + at * D + d);
        v.x += w * x.x, v.y += w * x.y, v.z += w * x.z, v.w += w * x.w;
      }
    }
    if (together) {
      part[warp][lane] = v;
      if (lane == 0) part_l[warp] = l;
      __syncthreads();
      if (warp == 0) {
        for (int k = 1; k < kCombineWarps; ++k) {
          const float4 x = part[k][lane];
          v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
          l += part_l[k];
        }
      }
    }
    if ((!together || warp == 0) && d < D) {
      const int64_t at = static_cast<int64_t>(o.row0) + r;
      moe_bf16 *dst = p.out + (o.start + at / a.group) * p.out_ld +
                      (o.head * a.group + at % a.group) * D + d;
      const float f = 1.0f / l;
      *reinterpret_cast<uint2 *>(dst) =
          make_uint2(bf16x2(v.x * f, v.y * f), bf16x2(v.z * f, v.w * f));
    }
    if (together) __syncthreads();
  }
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

struct Layout {
  size_t open, ml, sums, total;
};

Layout layout(const moe_attn_dims &d) {
  // both kernels' parts: 2 a block
  const size_t tc = 2 * kTcMaxCtas * (d.head_dim == 256 ? 128 : 256);
  size_t rows = 2 * kStreamMaxCtas * kStreamMaxRows;
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
  return launch_early(attn_combine_kernel, dim3(2 * tc_sm_count()), kCombineThreads, 0, s, a, p, d,
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
  x.args.scale_log2 = d.scale * 1.44269504088896340736f;
  x.args.budget = tc_wait_budget_ns();
  const auto stream = d.kv_type == MOE_KV_BF16   ? launch_stream_bf16
                      : d.kv_type == MOE_KV_INT8 ? launch_stream_int8
                                                 : launch_stream_e4m3;
  const auto tc = d.kv_type == MOE_KV_BF16   ? launch_tc_bf16
                  : d.kv_type == MOE_KV_INT8 ? launch_tc_int8
                                             : launch_tc_e4m3;
  // Sequences of up to `few` rows stream; the others go to the tensor cores'
  // kernel.  Lengths that only the device knows: both kernels look.
  const int64_t most = static_cast<int64_t>(a.cu ? a.N : a.T) * a.group;
  const int few = a.cu ? (a.group <= 16 ? 16 : a.group <= 32 ? 32 : 64) : 64;
  cudaError_t e = cudaSuccess;
  if (a.cu || most <= few) {
    const int rows = static_cast<int>(most < few ? most : few);
    x.range.least = 0, x.range.most = few;
    x.args.least_share = 2;
    e = stream(x, d.head_dim, rows <= 16 ? 1 : rows <= 32 ? 2 : 4);
  }
  if (e == cudaSuccess && most > few) {
    x.range.least = few, x.range.most = INT32_MAX;
    x.args.least_share = 1;
    e = tc(x, d.head_dim);
  }
  return e;
}

}  // namespace moe
