// gqa_prompt_attn: causal attention over packed prompts.
//
// One warp per (query row, head) walks the row's keys with a running maximum
// and sum; a lane holds d/32 dims of the query, the keys and the output.
#include "gqa.cuh"
#include "kernels.h"

namespace csa {

namespace {

using namespace gqa;

struct PromptArgs {
  gqa_rows q, k, v, out;
  int n_q, n_k;
  const int32_t* cu_q;
  const int32_t* cu_k;
  const float* sink;
  int B, n_heads, n_kv, window;
  float scale;
  int32_t* err;
};

template <bool kBf16, int kD>
__device__ __forceinline__ void load_row(const gqa_rows& s, int64_t row, int h, int lane, float (&x)[kD / 32]) {
  constexpr int n = kD / 32;
#pragma unroll
  for (int j = 0; j < n; j += 2) {
    const float2 f = unpack2<kBf16>(*reinterpret_cast<const uint32_t*>(
        reinterpret_cast<const uint16_t*>(s.ptr) + row * s.row_stride + h * s.head_stride + n * lane + j));
    x[j] = f.x;
    x[j + 1] = f.y;
  }
}

template <bool kBf16, int kD>
__global__ void __launch_bounds__(128) gqa_prompt_kernel(const PromptArgs a) {
  constexpr int n = kD / 32;
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (w >= (int64_t)a.n_q * a.n_heads) return;
  const int row = (int)(w / a.n_heads), h = (int)(w % a.n_heads);
  if (row >= a.cu_q[a.B]) return;
  int lo = 0, hi = a.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.cu_q[mid] <= row) lo = mid; else hi = mid - 1;
  }
  const int q0 = a.cu_q[lo], q1 = a.cu_q[lo + 1], k0 = a.cu_k[lo], k1 = a.cu_k[lo + 1];
  if (q0 < 0 || q1 > a.n_q || k0 < 0 || k1 > a.n_k || k1 < k0 || row < q0 || row >= q1) {
    if (lane == 0) raise_err(a.err, CSA_DEV_ERR_RANGE);
    return;
  }
  const int t = k1 - k0 - (q1 - q0) + (row - q0);
  const int first = a.window > 0 ? max(0, t - a.window + 1) : 0;
  const int kvh = h / (a.n_heads / a.n_kv);
  float q[n], o[n] = {}, x[n];
  load_row<kBf16, kD>(a.q, row, h, lane, q);
  float m = a.sink ? a.sink[h] : -INFINITY, l = a.sink ? 1.f : 0.f;
  for (int j = first; j <= t; ++j) {
    load_row<kBf16, kD>(a.k, k0 + j, kvh, lane, x);
    float z = 0.f;
#pragma unroll
    for (int e = 0; e < n; ++e) z = fmaf(q[e], x[e], z);
    z = warp_sum(z) * a.scale;
    const float mn = fmaxf(m, z), f = m == -INFINITY ? 0.f : expf(m - mn), p = expf(z - mn);
    load_row<kBf16, kD>(a.v, k0 + j, kvh, lane, x);
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

cudaError_t launch_gqa_prompt(const gqa_params& p, const gqa_rows& q, const gqa_rows& k, const gqa_rows& v,
                              int64_t n_q, int64_t n_k, const int32_t* cu_q, const int32_t* cu_k, const float* sink,
                              const gqa_rows& out, int32_t* err, cudaStream_t st) {
  const PromptArgs a{q, k, v, out, (int)n_q, (int)n_k, cu_q, cu_k, sink,
                     p.B, p.n_heads, p.n_kv_heads, p.window, p.softmax_scale, err};
  const bool bf = p.act_fmt == CSA_ACT_BF16;
  auto fn = bf ? (p.d == 128 ? gqa_prompt_kernel<true, 128> : gqa_prompt_kernel<true, 64>)
               : (p.d == 128 ? gqa_prompt_kernel<false, 128> : gqa_prompt_kernel<false, 64>);
  const int64_t warps = n_q * p.n_heads;
  return launch_pdl(fn, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, st, a);
}

}  // namespace csa
