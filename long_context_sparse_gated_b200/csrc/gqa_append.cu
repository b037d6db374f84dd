// gqa_cache_append: new tokens' keys and values into the paged cache, keys
// and queries turned by their positions on the way.
//
// One CTA per token.  The token's cosines and sines (one pair per rotated
// pair of dims, shared by all heads) go to shared memory once; a thread then
// carries 8 dims (16 bytes in) of one head at a time through the turn to all
// the places they are written to.
#include "gqa.cuh"
#include "kernels.h"

namespace csa {

namespace {

using namespace gqa;

constexpr int kThreads = 256;

struct AppendArgs {
  gqa_rows q, k, v, q_out, k_out;
  gqa_cache cache;
  const int32_t* cu;
  const int32_t* pos0;
  const int32_t* table;
  int64_t table_cols;
  int B, n_heads, n_kv, d, r, page;
  float theta;
  int32_t* err;
};

// The sequence that packed row i belongs to: the last b with cu[b] <= i (so
// that empty sequences are passed over), or -1 when i >= cu[B].
__device__ __forceinline__ int find_seq(const int32_t* cu, int B, int i) {
  if (i >= cu[B]) return -1;
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The larger, or NaN if one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <bool kBf16, bool kFp8>
__global__ void __launch_bounds__(kThreads) gqa_append_kernel(const AppendArgs a) {
  __shared__ float cs[64], sn[64];
  pdl_wait();
  const int i = blockIdx.x;
  const int b = find_seq(a.cu, a.B, i);
  if (b < 0) return;
  const int64_t pos = (int64_t)a.pos0[b] + (i - a.cu[b]);
  const int half = a.r / 2;
  if ((int)threadIdx.x < half) {
    float c, s;
    rope_cos_sin((double)pos, threadIdx.x, a.r, (double)a.theta, &c, &s);
    cs[threadIdx.x] = c;
    sn[threadIdx.x] = s;
  }
  __syncthreads();
  int64_t page = -1;
  int slot = 0;
  if (pos < 0 || pos >= a.table_cols * a.page) {
    if (threadIdx.x == 0) raise_err(a.err, CSA_DEV_ERR_RANGE);
  } else {
    page = a.table[(int64_t)b * a.table_cols + pos / a.page];
    slot = (int)(pos % a.page);
    if (page < 0 || page >= a.cache.n_pages) {
      if (threadIdx.x == 0) raise_err(a.err, CSA_DEV_ERR_INDEX);
      page = -1;
    }
  }
  const int pieces = a.d / 8;  // 16 or 8 lanes hold a row
  const int nq = a.q.ptr ? a.n_heads : 0;
  const int total = (nq + 2 * a.n_kv) * pieces;
  // whole warps take part in the shuffles: the bound is rounded up
  for (int e = threadIdx.x; e < ((total + 31) & ~31); e += kThreads) {
    const int c = e % pieces;
    int h = e / pieces;
    const bool live = e < total;
    const gqa_rows* src = &a.q;
    int kind = 0;
    if (h >= nq) {
      h -= nq;
      kind = 1;
      src = &a.k;
      if (h >= a.n_kv) {
        h -= a.n_kv;
        kind = 2;
        src = &a.v;
      }
    }
    float x[8] = {};
    if (live) {
      const uint16_t* p = reinterpret_cast<const uint16_t*>(src->ptr) + i * src->row_stride + h * src->head_stride + 8 * c;
      unpack8<kBf16>(*reinterpret_cast<const uint4*>(p), x);
    }
    const int at = 8 * c - (a.d - a.r);
    if (kind < 2 && at >= 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float co = cs[at / 2 + j], si = sn[at / 2 + j], u = x[2 * j], w = x[2 * j + 1];
        x[2 * j] = __fsub_rn(__fmul_rn(u, co), __fmul_rn(w, si));
        x[2 * j + 1] = __fadd_rn(__fmul_rn(u, si), __fmul_rn(w, co));
      }
    }
    const gqa_rows* dst = kind == 0 ? &a.q_out : &a.k_out;
    const uint4 y = pack8<kBf16>(x);
    if (live && kind < 2 && dst->ptr)
      *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(dst->ptr) + i * dst->row_stride + h * dst->head_stride +
                                8 * c) = y;
    const int64_t row = (page * a.n_kv + h) * a.page + slot;
    if (!kFp8) {
      if (live && kind > 0 && page >= 0)
        reinterpret_cast<uint4*>(kind == 1 ? a.cache.k : a.cache.v)[row * pieces + c] = y;
    } else {
      float am = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) am = max_nan(am, fabsf(x[j]));
      for (int o = pieces / 2; o > 0; o >>= 1) am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
      if (live && kind > 0 && page >= 0) {
        const float scale = am == 0.f ? 1.f : __fdiv_rn(am, kE4M3Max);  // NaN in a row: a NaN scale
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j / 4] |= f32_to_e4m3_sat(__fdiv_rn(x[j], scale)) << (8 * (j % 4));
        reinterpret_cast<uint2*>(kind == 1 ? a.cache.k : a.cache.v)[row * pieces + c] = make_uint2(w[0], w[1]);
        if (c == 0) (kind == 1 ? a.cache.k_scale : a.cache.v_scale)[row] = scale;
      }
    }
  }
}

}  // namespace

cudaError_t launch_gqa_append(const gqa_params& p, const gqa_rows& q, const gqa_rows& k, const gqa_rows& v,
                              int64_t n_tokens, const int32_t* cu, const int32_t* pos0, const gqa_cache& cache,
                              const int32_t* table, int64_t table_cols, const gqa_rows& q_out, const gqa_rows& k_out,
                              int32_t* err, cudaStream_t st) {
  const AppendArgs a{q, k, v, q_out, k_out, cache, cu, pos0, table, table_cols,
                     p.B, p.n_heads, p.n_kv_heads, p.d, p.r, p.page, p.rope_theta, err};
  const bool bf = p.act_fmt == CSA_ACT_BF16, f8 = p.kv_fmt == CSA_KV_FP8;
  auto fn = bf ? (f8 ? gqa_append_kernel<true, true> : gqa_append_kernel<true, false>)
               : (f8 ? gqa_append_kernel<false, true> : gqa_append_kernel<false, false>);
  return launch_pdl(fn, dim3((unsigned)n_tokens), dim3(kThreads), 0, st, a);
}

}  // namespace csa
