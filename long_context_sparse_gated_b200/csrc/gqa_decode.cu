// gqa_decode_attn: the last T tokens of every sequence attend to the paged
// cache.
//
// One warp per (query row, head) walks the row's keys with a running maximum
// and sum; a lane holds d/32 dims of the query, the keys and the output.
#include "gqa.cuh"
#include "kernels.h"

namespace csa {

namespace {

using namespace gqa;

struct DecodeArgs {
  gqa_rows q, out;
  gqa_cache cache;
  const int32_t* table;
  int64_t table_cols;
  const int32_t* lens;
  const float* sink;
  int B, T, n_max, n_heads, n_kv, page, window;
  float scale;
  int32_t* err;
};

template <bool kBf16, bool kFp8, int kD>
__device__ __forceinline__ void load_row(const void* base, const float* scale, int64_t row, int lane, float (&x)[kD / 32]) {
  constexpr int n = kD / 32;
#pragma unroll
  for (int j = 0; j < n; j += 2) {
    if (kFp8) {
      const uint8_t* p = reinterpret_cast<const uint8_t*>(base) + row * kD + n * lane + j;
      x[j] = e4m3_to_f32(p[0]) * scale[row];
      x[j + 1] = e4m3_to_f32(p[1]) * scale[row];
    } else {
      const float2 f = unpack2<kBf16>(*reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint16_t*>(base) + row * kD + n * lane + j));
      x[j] = f.x;
      x[j + 1] = f.y;
    }
  }
}

template <bool kBf16, bool kFp8, int kD>
__global__ void __launch_bounds__(128) gqa_decode_kernel(const DecodeArgs a) {
  constexpr int n = kD / 32;
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (w >= (int64_t)a.B * a.T * a.n_heads) return;
  const int h = (int)(w % a.n_heads);
  const int row = (int)(w / a.n_heads), b = row / a.T, tau = row % a.T;
  int len = a.lens[b];
  if (len > a.n_max) {
    len = a.n_max;
    if (lane == 0) raise_err(a.err, CSA_DEV_ERR_RANGE);
  }
  const int t = len - a.T + tau;
  const int first = a.window > 0 ? max(0, t - a.window + 1) : 0;
  const int kvh = h / (a.n_heads / a.n_kv);
  float q[n], o[n] = {}, x[n];
#pragma unroll
  for (int j = 0; j < n; j += 2) {
    const float2 f = unpack2<kBf16>(*reinterpret_cast<const uint32_t*>(
        reinterpret_cast<const uint16_t*>(a.q.ptr) + row * a.q.row_stride + h * a.q.head_stride + n * lane + j));
    q[j] = f.x;
    q[j + 1] = f.y;
  }
  float m = a.sink ? a.sink[h] : -INFINITY, l = a.sink ? 1.f : 0.f;
  for (int j = first; j <= t; ++j) {
    const int id = a.table[(int64_t)b * a.table_cols + j / a.page];
    if (id < 0 || id >= a.cache.n_pages) {
      if (lane == 0) raise_err(a.err, CSA_DEV_ERR_INDEX);
      continue;
    }
    const int64_t r = ((int64_t)id * a.n_kv + kvh) * a.page + j % a.page;
    load_row<kBf16, kFp8, kD>(a.cache.k, a.cache.k_scale, r, lane, x);
    float z = 0.f;
#pragma unroll
    for (int e = 0; e < n; ++e) z = fmaf(q[e], x[e], z);
    z = warp_sum(z) * a.scale;
    const float mn = fmaxf(m, z), f = m == -INFINITY ? 0.f : expf(m - mn), p = expf(z - mn);
    load_row<kBf16, kFp8, kD>(a.cache.v, a.cache.v_scale, r, lane, x);
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < n; ++e) o[e] = fmaf(p, x[e], o[e] * f);
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < n; e += 2)
    *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(a.out.ptr) + row * a.out.row_stride +
                                 h * a.out.head_stride + n * lane + e) = pack2<kBf16>(o[e] * inv, o[e + 1] * inv);
}

}  // namespace

size_t gqa_decode_workspace_bytes(const gqa_params&, int, int) { return 0; }

cudaError_t launch_gqa_decode(const gqa_params& p, const gqa_rows& q, const gqa_cache& cache, const int32_t* table,
                              int64_t table_cols, const int32_t* lens, int T, int n_max, const float* sink,
                              const gqa_rows& out, void*, int32_t* err, cudaStream_t st) {
  const DecodeArgs a{q, out, cache, table, table_cols, lens, sink, p.B, T, n_max,
                     p.n_heads, p.n_kv_heads, p.page, p.window, p.softmax_scale, err};
  const bool bf = p.act_fmt == CSA_ACT_BF16, f8 = p.kv_fmt == CSA_KV_FP8;
  auto pick = [&](auto k128, auto k64) { return p.d == 128 ? k128 : k64; };
  auto fn = bf ? (f8 ? pick(gqa_decode_kernel<true, true, 128>, gqa_decode_kernel<true, true, 64>)
                     : pick(gqa_decode_kernel<true, false, 128>, gqa_decode_kernel<true, false, 64>))
               : (f8 ? pick(gqa_decode_kernel<false, true, 128>, gqa_decode_kernel<false, true, 64>)
                     : pick(gqa_decode_kernel<false, false, 128>, gqa_decode_kernel<false, false, 64>));
  const int64_t warps = (int64_t)p.B * T * p.n_heads;
  return launch_pdl(fn, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, st, a);
}

}  // namespace csa
