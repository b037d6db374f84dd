// gqa_cache_append: new tokens' keys and values into the paged cache, keys
// and queries turned by their positions on the way.
//
// Bound by bytes (each row read once, written once or twice), and by latency
// for a decode step.  A CTA takes one token, or several while their rows are
// few; a thread carries 16 dims (32 bytes in) of a head at a time.  The rows'
// addresses do not depend on positions, so the first four or six loads of a
// thread are on their way before one warp per token looks up its sequence, position
// and page and fills the token's cosines and sines (one pair per rotated pair
// of dims, shared by all heads) in shared memory.  22730 tokens of 32 + 16 heads
// of 128: 109 us through the binding, 86% of the copy rate; into an FP8 cache 105 us,
// 83%.
//
// Angles.  pos * theta^(-2j/r) in turns: the frequencies / 2 pi come from the
// host in fp64, the product is reduced to [-1/2, 1/2] turns in fp64 and only
// then rounded, so that an angle is off by 2^-25 turns at any position.
//
// FP8.  The lanes that hold a row agree on its largest magnitude.  The scale
// is amax * (1/448) and codes are those of value * (1 / scale): both differ from
// the quotients by an fp32 rounding or two (a code only where the quotient is
// that near a border).  Only rows whose 1 / scale is beyond fp32 are divided.
#include <cmath>
#include <cstring>

#include "gqa.cuh"
#include "kernels.h"

namespace csa {

namespace {

using namespace gqa;

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8; // per CTA, a warp each

struct AppendArgs {
  gqa_rows in[3];   // q, k, v
  gqa_rows out[2];  // q_out, k_out
  void* cache[3];   // -, k, v
  float* scale[3];
  int64_t n_pages;
  const int32_t* cu;
  const int32_t* pos0;
  const int32_t* table;
  int64_t table_cols;
  int n_tokens, tokens;  // all, per CTA
  int B, nq, n_kv, r, page, page_shift;
  int rows, per_token;   // rows (heads) of a CTA, of a token
  uint32_t token_magic;  // ceil(2^16 / per_token), with several tokens per CTA
  int32_t* err;
  double turns[64];  // theta^(-2j/r) / 2 pi
};

// The sequence that packed row i belongs to: the last b with cu[b] <= i (so
// that empty sequences are passed over), or -1 when i >= cu[B].  A warp
// narrows 32 ways at a time.
__device__ __forceinline__ int find_seq(const int32_t* cu, int B, int i, int lane) {
  int lo = 0, n = B + 1;  // cu[lo] <= i, and it is one of cu[lo .. lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32, at = lo + lane * step;
    const bool le = lane * step < n && cu[at] <= i;
    const unsigned hits = __ballot_sync(0xffffffffu, le) | 1u;
    const int last = 31 - __clz(hits);
    n = min(step, n - last * step);
    lo += last * step;
  }
  return lo < B ? lo : -1;
}

// kBatch: pieces of 16 dims that a thread has in flight.
template <bool kBf16, bool kFp8, int kD, int kBatch>
__global__ void __launch_bounds__(kThreads, kFp8 || kBatch == 3 ? 4 : 5) gqa_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kPieces = kD / 16;  // of a row: 8 or 4 neighbouring lanes
  __shared__ __align__(16) float2 turn[kMaxTokens][kD / 2];
  __shared__ int64_t row0[kMaxTokens];  // page * n_kv * page size + slot, -1: not stored, -2: no token
  pdl_wait();
  const int i0 = blockIdx.x * a.tokens;
  const int c = threadIdx.x % kPieces;
  const int pair0 = 8 * c - (kD - a.r) / 2;  // first of this thread's pairs
  constexpr int kRows = kThreads / kPieces;  // rows that the CTA's threads cover at once

  // A row of the CTA: its token and kind (0 q, 1 k, 2 v), and the head.
  auto locate = [&](int row, int& tok, int& kind, int& h) {
    tok = a.tokens > 1 ? (int)((uint32_t)row * a.token_magic >> 16) : 0;
    h = row - tok * a.per_token;
    kind = 0;
    if (h >= a.nq) {
      h -= a.nq;
      kind = h >= a.n_kv ? 2 : 1;
      h -= h >= a.n_kv ? a.n_kv : 0;
    }
  };
  uint4 w[kBatch][2];
  auto load = [&](int k, int row) {
    int tok, kind, h;
    locate(row, tok, kind, h);
    w[k][0] = w[k][1] = make_uint4(0, 0, 0, 0);
    if (row >= a.rows || i0 + tok >= a.n_tokens) return;
    const gqa_rows& s = a.in[kind];
    const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(s.ptr) + (i0 + tok) * s.row_stride +
                                                      h * s.head_stride + 16 * c);
    w[k][0] = src[0];
    w[k][1] = src[1];
  };
  const int row_t = threadIdx.x / kPieces;
#pragma unroll
  for (int k = 0; k < kBatch; ++k) load(k, row_t + k * kRows);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < a.tokens) {
    const int i = i0 + warp;
    const int b = i < a.n_tokens ? find_seq(a.cu, a.B, i, lane) : -1;
    int64_t at = -2;
    if (b >= 0) {
      const int64_t pos = (int64_t)a.pos0[b] + (i - a.cu[b]);
      for (int j = lane; 2 * j < a.r; j += 32) {
        double t = (double)pos * a.turns[j];
        t -= rint(t);
        float s, co;
        sincospif(2.f * (float)t, &s, &co);
        turn[warp][j] = make_float2(co, s);
      }
      at = -1;
      if (pos < 0 || pos >= a.table_cols << a.page_shift) {
        if (lane == 0) raise_err(a.err, CSA_DEV_ERR_RANGE);
      } else {
        const int64_t id = a.table[(int64_t)b * a.table_cols + (pos >> a.page_shift)];
        if (id < 0 || id >= a.n_pages) {
          if (lane == 0) raise_err(a.err, CSA_DEV_ERR_INDEX);
        } else {
          at = (id * a.n_kv << a.page_shift) + (pos & (a.page - 1));
        }
      }
    }
    if (lane == 0) row0[warp] = at;
  }
  __syncthreads();

  // whole warps stay for the shuffles
  constexpr int kWarpRows = 32 / kPieces;
  const int rows_up = (a.rows + kWarpRows - 1) / kWarpRows * kWarpRows;
  for (int row0_t = row_t; row0_t < rows_up; row0_t += kBatch * kRows) {
    if (row0_t != row_t) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) load(k, row0_t + k * kRows);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int row = row0_t + k * kRows;
      if (row >= rows_up) break;
      int tok, kind, h;
      locate(min(row, a.rows - 1), tok, kind, h);
      const int64_t at = row < a.rows ? row0[tok] : -2;
      float v[2][8];
      unpack8<kBf16>(w[k][0], v[0]);
      unpack8<kBf16>(w[k][1], v[1]);
      if (kind < 2) {
        // r is a multiple of 8: the rotated dims begin at either half
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (pair0 + 4 * e < 0) continue;
          const float4* t4 = reinterpret_cast<const float4*>(&turn[tok][pair0 + 4 * e]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float4 t = t4[j];  // (cos, sin) of two pairs
            const float p = v[e][4 * j], q = v[e][4 * j + 1], x = v[e][4 * j + 2], y = v[e][4 * j + 3];
            v[e][4 * j] = fmaf(p, t.x, -(q * t.y));
            v[e][4 * j + 1] = fmaf(p, t.y, q * t.x);
            v[e][4 * j + 2] = fmaf(x, t.z, -(y * t.w));
            v[e][4 * j + 3] = fmaf(x, t.w, y * t.z);
          }
        }
        w[k][0] = pack8<kBf16>(v[0]);
        w[k][1] = pack8<kBf16>(v[1]);
        const gqa_rows& dst = a.out[kind];
        if (at >= -1 && dst.ptr) {
          uint4* to = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(dst.ptr) + (i0 + tok) * dst.row_stride +
                                               h * dst.head_stride + 16 * c);
          to[0] = w[k][0];
          to[1] = w[k][1];
        }
      }
      const int64_t slot = at + ((int64_t)h << a.page_shift);
      if (!kFp8) {
        if (at >= 0 && kind > 0) {
          uint4* to = reinterpret_cast<uint4*>(a.cache[kind]) + (slot * kPieces + c) * 2;
          to[0] = w[k][0];
          to[1] = w[k][1];
        }
      } else if (__any_sync(0xffffffffu, kind > 0)) {
        float am = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) am = max_nan(am, fabsf(v[j / 8][j % 8]));
#pragma unroll
        for (int o = kPieces / 2; o > 0; o >>= 1) am = max_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
        if (at >= 0 && kind > 0) {
          const float s = am * (1.f / kE4M3Max);    // NaN in a row: a NaN scale
          const float scale = s == 0.f ? 1.f : s;   // zeros, and what is zero beside fp32's smallest step
          // a reciprocal beyond fp32 (rows below 2^-117): divide
          const float inv = rcp(scale);
          const bool tiny = !(inv < INFINITY);
          uint32_t u[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float x = v[j / 4][2 * (j % 4)], y = v[j / 4][2 * (j % 4) + 1];
            const float2 z = tiny ? make_float2(__fdiv_rn(x, scale), __fdiv_rn(y, scale)) : make_float2(x * inv, y * inv);
            u[j] = __nv_cvt_float2_to_fp8x2(z, __NV_SATFINITE, __NV_E4M3);
          }
          reinterpret_cast<uint4*>(a.cache[kind])[slot * kPieces + c] =
              make_uint4(u[0] | (u[1] << 16), u[2] | (u[3] << 16), u[4] | (u[5] << 16), u[6] | (u[7] << 16));
          if (c == 0) a.scale[kind][slot] = scale;
        }
      }
    }
  }
  pdl_trigger();
}

// The frequencies of a (theta, r), kept per host thread: 64 powers cost more
// than the rest of the call.
const double* turns_of(float theta, int r) {
  thread_local float t_theta = 0.f;
  thread_local int t_r = -1;
  thread_local double t_turns[64];
  if (t_theta != theta || t_r != r) {
    for (int j = 0; j < 64; ++j)
      t_turns[j] = 2 * j < r ? std::pow((double)theta, -2.0 * j / r) / 6.283185307179586476925 : 0.0;
    t_theta = theta;
    t_r = r;
  }
  return t_turns;
}

}  // namespace

cudaError_t launch_gqa_append(const gqa_params& p, const gqa_rows& q, const gqa_rows& k, const gqa_rows& v,
                              int64_t n_tokens, const int32_t* cu, const int32_t* pos0, const gqa_cache& cache,
                              const int32_t* table, int64_t table_cols, const gqa_rows& q_out, const gqa_rows& k_out,
                              int32_t* err, cudaStream_t st) {
  // tokens per CTA: as many as fill the threads' first batch of loads, but no
  // fewer CTAs than SMs.  Three pieces a thread where that leaves fewer threads
  // idle than two do (us with two / three, in short runs: 32 + 16 heads of 128 106 /
  // 103, FP8 122 / 101, of 64 60 / 56; 64 + 16 heads, as many idle either way, 157 / 162).
  const int nq = q.ptr ? p.n_heads : 0, per_token = nq + 2 * p.n_kv_heads, pieces = per_token * p.d / 16;
  const int64_t most = n_tokens / sm_count();
  auto tokens_of = [&](int batch) {
    int n = batch * kThreads / pieces;
    if (n > kMaxTokens) n = kMaxTokens;
    if (n > most) n = (int)most;
    return n < 1 ? 1 : n;
  };
  auto places = [&](int n) { return (n * pieces + kThreads - 1) / kThreads * kThreads; };
  const int two = tokens_of(2), three = tokens_of(3);
  const bool wide = three * places(two) > two * places(three);  // pieces by places, as a cross product
  const int tokens = wide ? three : two;
  int shift = 0;
  while ((1 << shift) < p.page) ++shift;
  AppendArgs a{{q, k, v}, {q_out, k_out}, {nullptr, cache.k, cache.v}, {nullptr, cache.k_scale, cache.v_scale},
               cache.n_pages, cu, pos0, table, table_cols, (int)n_tokens, tokens, p.B, nq, p.n_kv_heads, p.r, p.page,
               shift, tokens * per_token, per_token, (65536u + per_token - 1) / per_token, err, {}};
  std::memcpy(a.turns, turns_of(p.rope_theta, p.r), sizeof(a.turns));
  const bool bf = p.act_fmt == CSA_ACT_BF16, f8 = p.kv_fmt == CSA_KV_FP8;
#define GQA_PICK(BF, F8)                                                                            \
  (p.d == 128 ? (wide ? gqa_append_kernel<BF, F8, 128, 3> : gqa_append_kernel<BF, F8, 128, 2>) \
              : (wide ? gqa_append_kernel<BF, F8, 64, 3> : gqa_append_kernel<BF, F8, 64, 2>))
  auto fn = bf ? (f8 ? GQA_PICK(true, true) : GQA_PICK(true, false)) : (f8 ? GQA_PICK(false, true) : GQA_PICK(false, false));
#undef GQA_PICK
  return launch_pdl(fn, dim3((unsigned)((n_tokens + tokens - 1) / tokens)), dim3(kThreads), 0, st, a);
}

}  // namespace csa
