// gqa_prompt_attn: causal attention over packed prompts, on the 5th-generation
// tensor cores.
//
//   S = Q K^T,  P = exp(scale S - m),  O = P V / (exp(sink - m) + sum P)
//
// Work.  A unit is 128 query positions of one query head; units of a
// sequence and KV head are numbered position tile by position tile, the heads
// of a group inside, and a CTA takes two neighbours, which then mostly read
// the same keys.  Blocks are ordered from a sequence's last positions (most
// keys) to its first.
//
//   warp 8    loads: both Q tiles once, then K and V tiles of 128 keys into
//             rings of their own (TMA, 128-byte swizzle)
//   warp 9    issues the MMAs (tcgen05 kind::f16, M = 128, fp32 in TMEM):
//             S_i = Q_i K^T from shared memory; O_i += P_i V with P_i read
//             from TMEM, where it lies on top of S_i.  The two units take
//             turns: while one's S is turned into P, the tensor cores run
//             the other's products.
//   warps 0-3, 4-7   softmax of unit 0 / 1, a thread a row: the row's 128
//             logits in registers, running maximum, P in 16 bits back to
//             TMEM, in two halves, so that the product with the first 64 keys
//             begins while the second half is computed.  The maximum moves
//             only when a row exceeds it by 2^8 (FP16: 2^6), so O is hardly ever
//             rescaled; at the end the same threads normalise O and write it
//             out through shared memory.
//
// Exponentials.  A tile pair has 32768 of them: 2048 clocks of the 16-lane
// special-function pipe, as many as its four products take.  So kPoly of
// every 8 pairs of logits (3 for BF16, 2 for FP16; 16K tokens, one call from cold
// caches, take 452 us with 4, 422 with 3, 426 with 2, 442 with 1, 430 with none; FP16
// 442 with 3, 440 with 2, 455 with 1, 443 with none) go through the FMA pipe instead:
// 2^x = 2^n 2^f with n the nearest integer (by adding 1.5 * 2^23) and a polynomial in f,
// minimax for the relative error on [-1/2, 1/2]: degree 3, 7.5e-5, before P is
// rounded to BF16 (2^-8), degree 4, 2.6e-6, before FP16 (2^-11).  n is added to
// the exponent field; weights below 2^-126 (2^-112 of the row's largest and less)
// come out as about that.  Packed fp32 pairs (f32x2) throughout.
//
// Masks.  In tiles that some row does not see as a whole logits are selected,
// blocks of 32 keys that a warp's rows all see or all miss at once.  A value
// that is not finite where a row's weight is 0 would still reach the row's sum
// (0 * NaN is NaN): rows behind the sequence are cleared in shared memory, and
// rows that come out as something not finite are looked at again (rows_again).
// (Looking through the value tiles before the products cost 2700 clocks a tile.)
//
// TMEM: S_0, S_1 (128 columns each), O_0, O_1 (d columns each).
// Rounding: P to the activation type, since a product's operands are of one type:
// to BF16 (2^-8 of itself) or FP16 (2^-11, where FP16 has its full precision: down to
// 2^-23 of the row's largest weight, which is 2^9.5 at least; below that by up to
// 2^-34 of the largest).  The rest is fp32.
#include <cuda.h>

#include <cmath>

#include "gqa.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace csa {

namespace {

using namespace gqa;

constexpr int kTile = 128;  // query positions of a unit, keys of a tile
constexpr int kThreads = 384;
constexpr float kLog2e = 1.4426950408889634f;
// Weights are 2^(z - m + kTop) with m a running maximum, raised when a logit
// exceeds it by kLazy (base-2 units).  FP16 holds weights from 2^-14 (with fewer bits
// from 2^-24) to 2^16, so the largest are put near its top, the nearer the closer the
// maximum is followed (16K tokens, FP16, 8/1 heads of 128: by 2^8 438 us, 2^6 440, 2^4
// 461).  BF16 weights begin at 2^-14: sums of the type's largest values stay finite
// while the weights add up to less than 2^14 of the largest, and products with its
// smallest are still well above fp32's last bit.
template <bool kBf16>
struct Weights {
  static constexpr float kTop = kBf16 ? -14.f : 9.5f, kLazy = kBf16 ? 8.f : 6.f;
};

struct PromptArgs {
  gqa_rows q, k, v, out;
  int n_q, n_k;
  const int32_t* cu_q;
  const int32_t* cu_k;
  const float* sink;
  int B, n_heads, n_kv, window;
  float scale, step;  // softmax_scale * log2(e); kLazy in units of S
  int32_t* err;
};

template <int kD>
struct __align__(1024) PromptSmem {
  static constexpr int kOperand = kTile * kD * 2;
  static constexpr int kK = kD == 128 ? 3 : 4, kV = kD == 128 ? 2 : 4;  // stages
  uint8_t q[2][kOperand];  // later the staged output
  uint8_t k[kK][kOperand];
  uint8_t v[kV][kOperand];
  uint64_t q_full, k_full[kK], k_empty[kK], v_full[kV], v_empty[kV];
  uint64_t s_full[2], p_full[2][2], o_full;  // p_full: of a unit's half tile
  uint32_t tmem;
  int abort;
  int blocks[kThreads / 32];  // of a warp's sequences
  int item[6];  // sequence (-1: none), its block, first query, queries, first key, keys
};


__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, float (&r)[128], int at) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r) + at;
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr)
      : "memory");
}
// After tmem_ld_wait(): 32 registers count as produced here.
__device__ __forceinline__ void pin32(float (&r)[128], int at) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile(""
                 : "+f"(r[at + i]), "+f"(r[at + i + 1]), "+f"(r[at + i + 2]), "+f"(r[at + i + 3]), "+f"(r[at + i + 4]),
                   "+f"(r[at + i + 5]), "+f"(r[at + i + 6]), "+f"(r[at + i + 7]));
}
__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t (&u)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]), "r"(u[9]),
      "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(u[16]), "r"(u[17]), "r"(u[18]),
      "r"(u[19]), "r"(u[20]), "r"(u[21]), "r"(u[22]), "r"(u[23]), "r"(u[24]), "r"(u[25]), "r"(u[26]), "r"(u[27]),
      "r"(u[28]), "r"(u[29]), "r"(u[30]), "r"(u[31])
      : "memory");
}
// Whether this lane is the one of its warp that issues MMAs.  The rest of the
// warp runs along: issued from a branch on the lane index, an MMA took some 118
// clocks to issue, twice what it takes to run.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// D[tmem] (+)= A B, 16-bit operands, A in shared memory or TMEM.
template <bool kAdd>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
               "l"(a), "l"(b), "r"(idesc), "n"(kAdd ? 1 : 0)
               : "memory");
}
template <bool kAdd>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
               "r"(a), "l"(b), "r"(idesc), "n"(kAdd ? 1 : 0)
               : "memory");
}

struct True { static constexpr bool value = true; };
struct False { static constexpr bool value = false; };

// Pairs of fp32 in one register pair.
__device__ __forceinline__ uint64_t f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// 2^x of two numbers that are at most 127 (smaller ones than -126 count as -126).
template <bool kBf16>
__device__ __forceinline__ uint64_t exp2_poly(uint64_t x2) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
  float x, y;
  split2(x2, x, y);
  x2 = f32x2(fmaxf(x, -126.f), fmaxf(y, -126.f));
  const uint64_t t2 = add2(x2, f32x2(kMagic, kMagic));  // the low bits hold round(x)
  const uint64_t f2 = fma2(add2(t2, f32x2(-kMagic, -kMagic)), f32x2(-1.f, -1.f), x2);
  uint64_t p2;
  if (kBf16) {
    p2 = fma2(f2, f32x2(0.0551716685295105f, 0.0551716685295105f), f32x2(0.2426111251115799f, 0.2426111251115799f));
    p2 = fma2(f2, p2, f32x2(0.6932609677314758f, 0.6932609677314758f));
    p2 = fma2(f2, p2, f32x2(0.9999280571937561f, 0.9999280571937561f));
  } else {
    p2 = fma2(f2, f32x2(0.009570102207362652f, 0.009570102207362652f), f32x2(0.05591785907745361f, 0.05591785907745361f));
    p2 = fma2(f2, p2, f32x2(0.240247443318367f, 0.240247443318367f));
    p2 = fma2(f2, p2, f32x2(0.6931217908859253f, 0.6931217908859253f));
    p2 = fma2(f2, p2, f32x2(0.9999992847442627f, 0.9999992847442627f));
  }
  float tx, ty;
  split2(t2, tx, ty);
  split2(p2, x, y);
  return f32x2(__int_as_float(__float_as_int(x) + (__float_as_int(tx) << 23)),
              __int_as_float(__float_as_int(y) + (__float_as_int(ty) << 23)));
}

// Thread r of 128 clears its part of the rows from `first` on of a value tile.
template <int kD>
__device__ __forceinline__ void clear_rows(uint8_t* v, int r, int first) {
  for (int x = r; x < kTile * kD / 8; x += 128)
    if (((x >> 3) & (kTile - 1)) >= first) reinterpret_cast<uint4*>(v)[x] = make_uint4(0, 0, 0, 0);
  sm100::fence_proxy_async_smem();
}

// One unit: 128 positions of a query head.
struct Unit {
  int rows;        // its queries (0: no unit)
  int head, row0;  // query head, first packed query row
  int t0, t1;      // positions of its first and last query
  int j0, j1;      // key tiles [j0, j1)
};

// Whether one of eight values is an infinity or NaN.
template <bool kBf16>
__device__ __forceinline__ bool odd8(const uint4& v) {
  constexpr uint32_t e = kBf16 ? 0x7F80u : 0x7C00u, low = kBf16 ? 0x80u : 0x400u;
  // (an exponent of all ones carries into the sign's place)
  auto top = [](uint32_t x) { return (x & (e | e << 16)) + (low | low << 16); };
  return ((top(v.x) | top(v.y) | top(v.z) | top(v.w)) & 0x80008000u) != 0;
}

// Rows of a unit that came out as something not finite (those of `rows` of the 32 from
// packed query row row0, at position t0, on), looked at again by their warp.  They
// stay as they are unless a value that is not finite lies in one of the unit's tiles
// (keys [key0, key1)) where not all of them see it; it has then reached rows that do
// not see it as 0 * NaN.  Such rows are computed again, 16 rows by 16 keys at a time
// with mma.sync and operands straight from global memory; values that are not finite
// are taken out of blocks that a row does not see as a whole and given to the rows that
// see them.  6000 tokens of 8/1 heads of 128, us: 110 without such values, 111 with a
// NaN in the first, 2010 in the last (one unit a head, 32 rows each of its warps), 2170
// in every one; row by row and key by key the last three take 83000.
template <bool kBf16, int kD>
__device__ __noinline__ void blocks_again(const PromptArgs& a, unsigned rows, int row0, int t0, int head, int kvh, int k_begin,
                                        int key0, int key1, int lane) {
  constexpr float kTop = Weights<kBf16>::kTop;
  const uint16_t* qp = reinterpret_cast<const uint16_t*>(a.q.ptr) + row0 * a.q.row_stride + head * a.q.head_stride;
  const uint16_t* kp = reinterpret_cast<const uint16_t*>(a.k.ptr) + k_begin * a.k.row_stride + kvh * a.k.head_stride;
  const uint16_t* vp = reinterpret_cast<const uint16_t*>(a.v.ptr) + k_begin * a.v.row_stride + kvh * a.v.head_stride;
  const int r0 = __ffs(rows) - 1, r1 = 31 - __clz(rows), window = a.window;
  // ---- keys that the first of them does not see, or the last one does not any more
  bool some = false;
  auto look = [&](int from, int to) {
    for (int key = from + lane; key < to; key += 32)
      for (int i = 0; i < kD / 8; ++i) some |= odd8<kBf16>(reinterpret_cast<const uint4*>(vp + key * a.v.row_stride)[i]);
  };
  look(max(key0, t0 + r0 + 1), key1);
  if (window > 0) look(key0, min(key1, t0 + r1 - window + 1));
  if (!__any_sync(0xffffffffu, some)) return;

  const int g = lane >> 2, q4 = lane & 3;
#pragma unroll 1
  for (int half = 0; half < 32; half += 16) {
    const unsigned here = rows >> half & 0xFFFFu;
    if (!here) continue;
    // fragments' rows g and g + 8; rows that are not asked for count as the nearest
    // that are, so that none is read that is not there
    const int h0 = half + __ffs(here) - 1, h1 = half + 31 - __clz(here);
    int t[2];
    uint32_t qf[kD / 16][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = min(max(half + g + 8 * e, h0), h1);
      t[e] = t0 + row;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(qp + row * a.q.row_stride) + q4;
#pragma unroll
      for (int c = 0; c < kD / 16; ++c) {
        qf[c][e] = src[8 * c];
        qf[c][2 + e] = src[8 * c + 4];
      }
    }
    const int first = window > 0 ? max(0, t0 + h0 - window + 1) : 0;  // of their keys
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[kD / 8][4];
#pragma unroll
    for (int c = 0; c < kD / 8; ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
#pragma unroll 1
    for (int key = first & ~15; key <= t0 + h1; key += 16) {
      auto seen = [&](int j, int e) { return j <= t[e] && (window == 0 || j > t[e] - window); };
      auto at = [&](int j) { return (int64_t)min(max(j, first), t0 + h1); };  // a key that is there
      float s[2][4] = {};
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(kp + at(key + 8 * n + g) * a.k.row_stride) + q4;
#pragma unroll
        for (int c = 0; c < kD / 16; ++c) mma16816<kBf16>(s[n], qf[c], src[8 * c], src[8 * c + 4]);
      }
      bool edge = false;
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool see = seen(key + 8 * n + 2 * q4 + (e & 1), e >> 1);
          edge |= !see;
          if (!see) s[n][e] = -INFINITY;
          top[e >> 1] = fmaxf(top[e >> 1], s[n][e]);
        }
      edge = __any_sync(0xffffffffu, edge);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
        const float alpha = top[e] > m[e] ? ex2((m[e] - top[e]) * a.scale) : 1.f;
        m[e] = fmaxf(m[e], top[e]);
        l[e] *= alpha;
#pragma unroll
        for (int c = 0; c < kD / 8; ++c) {
          o[c][2 * e] *= alpha;
          o[c][2 * e + 1] *= alpha;
        }
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float mr = m[e >> 1] == -INFINITY ? 0.f : m[e >> 1];
          s[n][e] = ex2(fmaf(s[n][e] - mr, a.scale, kTop));
          l[e >> 1] += s[n][e];
        }
      const uint32_t pf[4] = {pack2<kBf16>(s[0][0], s[0][1]), pack2<kBf16>(s[0][2], s[0][3]),
                              pack2<kBf16>(s[1][0], s[1][1]), pack2<kBf16>(s[1][2], s[1][3])};
      const uint16_t* src[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) src[e] = vp + at(key + 2 * q4 + (e & 1) + 8 * (e >> 1)) * a.v.row_stride + g;
      bool odd = false;
#pragma unroll
      for (int c = 0; c < kD / 8; ++c) {
        uint32_t b[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          b[e] = (uint32_t)src[2 * e][8 * c] | (uint32_t)src[2 * e + 1][8 * c] << 16;
          if (edge) {
            const uint32_t bad = odd_halves<kBf16>(b[e]);
            odd |= bad != 0;
            b[e] &= ~bad;
          }
        }
        mma16816<kBf16>(o[c], pf, b[0], b[1]);
      }
      if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
        for (int j = key; j < key + 16; ++j) {
          const uint32_t* v = reinterpret_cast<const uint32_t*>(vp + at(j) * a.v.row_stride) + q4;
#pragma unroll
          for (int c = 0; c < kD / 8; ++c) {
            const float2 x = unpack2<kBf16>(v[4 * c]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (seen(j, e) && !(fabsf(x.x) < INFINITY)) o[c][2 * e] += x.x;
              if (seen(j, e) && !(fabsf(x.y) < INFINITY)) o[c][2 * e + 1] += x.y;
            }
          }
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      if (a.sink && m[e] != -INFINITY) l[e] += ex2(a.sink[head] * kLog2e - (m[e] * a.scale - kTop));
      const float f = l[e] != 0.f ? rcp(l[e]) : 0.f;
      if (here >> (g + 8 * e) & 1) {
        uint32_t* dst = reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(a.out.ptr) + (int64_t)(row0 + half + g + 8 * e) * a.out.row_stride +
                                                    head * a.out.head_stride) + q4;
#pragma unroll
        for (int c = 0; c < kD / 8; ++c) dst[4 * c] = pack2<kBf16>(o[c][2 * e] * f, o[c][2 * e + 1] * f);
      }
    }
  }
}

// A lone such row near a sequence's beginning is computed by itself, a lane with kD/32
// dims of it.  (32000 such rows of 8 keys take 0.39 ms, by blocks 0.47, of 44 keys 0.96
// and 1.04; and with this path the kernel around takes 416 us for 16K tokens, not 440:
// what registers the code out of line takes changes those of the softmax.)
template <bool kBf16, int kD>
__device__ __noinline__ void rows_again(const PromptArgs& a, unsigned odd, int key0, int key1, int row, int t, int head, int kvh,
                                        int k0, int lane) {
  constexpr float kTop = Weights<kBf16>::kTop;
  constexpr int n = kD / 32;
  auto load = [&](const gqa_rows& s, int64_t row, int h, float (&x)[n]) {
#pragma unroll
    for (int j = 0; j < n; j += 2) {
      const float2 f = unpack2<kBf16>(*reinterpret_cast<const uint32_t*>(
          reinterpret_cast<const uint16_t*>(s.ptr) + row * s.row_stride + h * s.head_stride + n * lane + j));
      x[j] = f.x;
      x[j + 1] = f.y;
    }
  };
  if ((odd & (odd - 1)) || t >= 16) {
    blocks_again<kBf16, kD>(a, odd, row, t, head, kvh, k0, key0, key1, lane);
    return;
  }
  row += __ffs(odd) - 1;
  t += __ffs(odd) - 1;
  const int first = a.window > 0 ? max(0, t - a.window + 1) : 0;
  float q[n], x[n], o[n] = {}, m = -INFINITY, l = 0.f;
  load(a.q, row, head, q);
  for (int j = first; j <= t; ++j) {
    load(a.k, k0 + j, kvh, x);
    float z = 0.f;
#pragma unroll
    for (int e = 0; e < n; ++e) z = fmaf(q[e], x[e], z);
    z = warp_sum(z) * a.scale;
    const float mn = fmaxf(m, z), f = m == -INFINITY ? 0.f : ex2(m - mn), p = ex2(z - mn + kTop);
    load(a.v, k0 + j, kvh, x);
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < n; ++e) o[e] = fmaf(p, x[e], o[e] * f);
    m = mn;
  }
  if (a.sink && m != -INFINITY) l += ex2(a.sink[head] * kLog2e - m + kTop);
  const float inv = l != 0.f ? rcp(l) : 0.f;
#pragma unroll
  for (int e = 0; e < n; e += 2)
    *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(a.out.ptr) + (int64_t)row * a.out.row_stride +
                                 head * a.out.head_stride + n * lane + e) = pack2<kBf16>(o[e] * inv, o[e + 1] * inv);
}

template <bool kBf16, int kD>
__global__ void __launch_bounds__(kThreads, 1)
    gqa_prompt_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_v, const __grid_constant__ PromptArgs a) {
  using Smem = PromptSmem<kD>;
  extern __shared__ uint8_t raw[];
  Smem& S = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &S.abort;

  if (warp == 8) {
    sm100::tmem_alloc(&S.tmem, 512);
    sm100::tmem_relinquish();
    sm100::tc_fence_before();
  }
  pdl_wait();
  // ---- which sequence, pair of units and KV head
  const int G = a.n_heads / a.n_kv;
  if (threadIdx.x == 0) {
    S.item[0] = -1;
    S.abort = 0;
    sm100::mbar_init(&S.q_full, 1);
    for (int i = 0; i < Smem::kK; ++i) {
      sm100::mbar_init(&S.k_full[i], 1);
      sm100::mbar_init(&S.k_empty[i], 1);
    }
    for (int i = 0; i < Smem::kV; ++i) {
      sm100::mbar_init(&S.v_full[i], 1);
      sm100::mbar_init(&S.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&S.s_full[i], 1);
      for (int x = 0; x < 2; ++x) sm100::mbar_init(&S.p_full[i][x], 4);
    }
    sm100::mbar_init(&S.o_full, 1);
    sm100::fence_mbar_init();
  }
  // a sequence per thread, kThreads of them at a time
  for (int b0 = 0, base = 0; b0 < a.B; b0 += kThreads) {
    int n = 0, q0 = 0, q1 = 0, k0 = 0, k1 = 0;
    const int b = b0 + threadIdx.x;
    if (b < a.B) {
      q0 = a.cu_q[b];
      q1 = a.cu_q[b + 1];
      k0 = a.cu_k[b];
      k1 = a.cu_k[b + 1];
      if (q0 < 0 || q1 < q0 || q1 > a.n_q || k0 < 0 || k1 < k0 || k1 > a.n_k) {
        raise_err(a.err, CSA_DEV_ERR_RANGE);
      } else {
        n = ((q1 - q0 + kTile - 1) / kTile * G + 1) / 2 * a.n_kv;
      }
    }
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (b0 > 0) __syncthreads();  // the last sums are read
    if (lane == 31) S.blocks[warp] = x;
    __syncthreads();
    int before = base;
    for (int w = 0; w < kThreads / 32; ++w) {
      base += S.blocks[w];
      if (w < warp) before += S.blocks[w];
    }
    const int at = (int)blockIdx.x - before - (x - n);
    if (at >= 0 && at < n) {
      S.item[0] = b;
      S.item[1] = at;
      S.item[2] = q0;
      S.item[3] = q1 - q0;
      S.item[4] = k0;
      S.item[5] = k1 - k0;
    }
    if ((int)blockIdx.x < base) break;  // (the same for all threads)
  }
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = S.tmem;
  if (S.item[0] < 0) {
    if (warp == 8) sm100::tmem_dealloc(tmem, 512);
    return;
  }
  const int q_begin = S.item[2], n_q = S.item[3], k_begin = S.item[4], n_k = S.item[5];
  const int tiles = (n_q + kTile - 1) / kTile, pairs = (tiles * G + 1) / 2;
  const int kvh = S.item[1] % a.n_kv, pair = pairs - 1 - S.item[1] / a.n_kv;
  Unit un[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int x = 2 * pair + i, tile = x / G;
    Unit& u = un[i];
    u.rows = tile < tiles ? min(kTile, n_q - tile * kTile) : 0;
    u.head = kvh * G + x % G;
    u.row0 = q_begin + tile * kTile;
    u.t0 = n_k - n_q + tile * kTile;
    u.t1 = u.rows > 0 ? u.t0 + u.rows - 1 : -1;
    const bool some = u.rows > 0 && u.t1 >= 0;
    u.j0 = some && a.window > 0 ? max(0, u.t0 - a.window + 1) / kTile : 0;
    u.j1 = some ? u.t1 / kTile + 1 : u.j0;
  }
  const int work0 = un[0].j1 - un[0].j0, work1 = un[1].j1 - un[1].j0;
  const int j_begin = work0 == 0 ? un[1].j0 : (work1 == 0 ? un[0].j0 : min(un[0].j0, un[1].j0));
  const int j_end = work0 == 0 ? un[1].j1 : (work1 == 0 ? un[0].j1 : max(un[0].j1, un[1].j1));
  // a tile that some row of the unit does not see as a whole
  auto edge_of = [&](const Unit& u, int j) {
    return j >= u.j0 && j < u.j1 && (j * kTile + kTile - 1 > u.t0 || (a.window > 0 && j * kTile <= u.t1 - a.window));
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8 && lane == 0) {
      // ---- loads
      int n_live = (work0 > 0) + (work1 > 0);
      if (n_live) sm100::mbar_arrive_expect_tx(&S.q_full, n_live * Smem::kOperand);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if ((i ? work1 : work0) > 0)
          for (int c = 0; c < kD / 64; ++c)
            sm100::tma_load_3d(S.q[i] + c * kTile * 128, &map_q, &S.q_full, 64 * c, un[i].row0, un[i].head);
      int n = 0;
      for (int j = j_begin; j < j_end; ++j, ++n) {
        const int ks = n % Smem::kK, vs = n % Smem::kV;
        if (n >= Smem::kK) sm100::mbar_wait(&S.k_empty[ks], (n / Smem::kK - 1) & 1, abort);
        if (*abort) break;
        sm100::mbar_arrive_expect_tx(&S.k_full[ks], Smem::kOperand);
        for (int c = 0; c < kD / 64; ++c)
          sm100::tma_load_3d(S.k[ks] + c * kTile * 128, &map_k, &S.k_full[ks], 64 * c, k_begin + j * kTile, kvh);
        if (n >= Smem::kV) sm100::mbar_wait(&S.v_empty[vs], (n / Smem::kV - 1) & 1, abort);
        if (*abort) {
          ++n;
          break;
        }
        sm100::mbar_arrive_expect_tx(&S.v_full[vs], Smem::kOperand);
        for (int c = 0; c < kD / 64; ++c)
          sm100::tma_load_3d(S.v[vs] + c * kTile * 128, &map_v, &S.v_full[vs], 64 * c, k_begin + j * kTile, kvh);
      }
      if (*abort) {
        // copies in flight land before the CTA goes (each wait bounded)
        auto drain = [&](uint64_t* bar, int parity) {
          const uint64_t t0 = sm100::globaltimer();
          while (!sm100::mbar_try_wait(bar, parity) && sm100::globaltimer() - t0 < sm100::kWaitNs) {
          }
        };
        if (n_live) drain(&S.q_full, 0);
        for (int i = max(0, n - Smem::kK); i < n; ++i) drain(&S.k_full[i % Smem::kK], (i / Smem::kK) & 1);
        for (int i = max(0, n - Smem::kV); i < n; ++i) drain(&S.v_full[i % Smem::kV], (i / Smem::kV) & 1);
      }
    } else if (warp == 9) {
      // ---- MMAs
      const uint32_t id_s = kBf16 ? sm100::idesc_bf16(kTile, kTile, 0, 0) : sm100::idesc_f16(kTile, kTile, 0, 0);
      const uint32_t id_o = kBf16 ? sm100::idesc_bf16(kTile, kD, 0, 1) : sm100::idesc_f16(kTile, kD, 0, 1);
      // Q and K K-major (8-row groups 1 KB apart, 64-dim halves 16 KB); V
      // MN-major: 64-dim halves 16 KB apart, groups of 8 keys 1 KB
      const uint64_t dq = sm100::smem_desc(sm100::smem_u32(S.q[0]), 16, 1024, 2);
      const uint64_t dk = sm100::smem_desc(sm100::smem_u32(S.k[0]), 16, 1024, 2);
      const uint64_t dv = sm100::smem_desc(sm100::smem_u32(S.v[0]), kTile * 128, 1024, 2);
      const bool leader = elect_one();
      auto active = [&](int i, int j) { return j >= un[i].j0 && j < un[i].j1; };
      auto issue_s = [&](int i, int ks) {  // S_i = Q_i K^T with the K tile of stage ks
        sm100::tc_fence_after();
        if (!*abort && leader) {
          const uint64_t q = dq + ((i * Smem::kOperand) >> 4), k = dk + ((ks * Smem::kOperand) >> 4);
          mma_ss<false>(tmem + 128 * i, q, k, id_s);
#pragma unroll
          for (int c = 1; c < kD / 16; ++c) {
            const uint32_t off = ((c >> 2) * kTile * 128 + (c & 3) * 32) >> 4;
            mma_ss<true>(tmem + 128 * i, q + off, k + off, id_s);
          }
        }
        if (leader) sm100::tc_commit(&S.s_full[i]);
        __syncwarp();
      };
      if (j_begin < j_end) {
        sm100::mbar_wait_poll(&S.q_full, 0, abort);
        sm100::mbar_wait_poll(&S.k_full[0], 0, abort);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (active(i, j_begin)) issue_s(i, 0);
        if (leader) sm100::tc_commit(&S.k_empty[0]);
      }
      int done[2] = {0, 0};
      int vs = 0, vph = 0, ks = 1, kph = 0;  // V tile j, K tile j + 1
      for (int j = j_begin; j < j_end; ++j) {
        sm100::mbar_wait_poll(&S.v_full[vs], vph, abort);
        if (j + 1 < j_end) sm100::mbar_wait_poll(&S.k_full[ks], kph, abort);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (active(i, j)) {
            const uint64_t v = dv + ((vs * Smem::kOperand) >> 4);
            const uint32_t o_col = tmem + 256 + kD * i, p_col = tmem + 128 * i;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              sm100::mbar_wait_poll(&S.p_full[i][half], done[i] & 1, abort);
              sm100::tc_fence_after();
              if (!*abort && leader) {
                if (half == 0) {
                  if (done[i] > 0) mma_ts<true>(o_col, p_col, v, id_o);
                  else mma_ts<false>(o_col, p_col, v, id_o);
                }
#pragma unroll
                for (int c = 4 * half + (half == 0); c < 4 * half + 4; ++c)
                  mma_ts<true>(o_col, p_col + 8 * c, v + ((c * 2048) >> 4), id_o);
              }
              __syncwarp();
            }
            ++done[i];
          }
          if (active(i, j + 1)) issue_s(i, ks);
        }
        if (leader) {
          sm100::tc_commit(&S.v_empty[vs]);
          if (j + 1 < j_end) sm100::tc_commit(&S.k_empty[ks]);
        }
        __syncwarp();
        if (++vs == Smem::kV) {
          vs = 0;
          vph ^= 1;
        }
        if (++ks == Smem::kK) {
          ks = 0;
          kph ^= 1;
        }
      }
      if (leader) {
        sm100::tc_commit(&S.o_full);
        if (*abort) {
          const uint64_t t0 = sm100::globaltimer();
          while (!sm100::mbar_try_wait(&S.o_full, 0) && sm100::globaltimer() - t0 < sm100::kWaitNs) {
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ---- softmax: unit i, row r
    const int i = warp >> 2, r = (warp & 3) * 32 + lane;
    const Unit u = i ? un[1] : un[0];
    constexpr int kPoly = kBf16 ? 3 : 2;
    constexpr float kTop = Weights<kBf16>::kTop;
    const int work = i ? work1 : work0;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + 128 * i + lanes, o_col = tmem + 256 + kD * i + lanes;
    const int t = u.t0 + r;
    float m = -INFINITY, l = 0.f;  // m in units of S
    bool far = false;              // some row's maximum is 2^20 or more away from 0
    for (int n = 0; n < work; ++n) {
      const int key0 = (u.j0 + n) * kTile;
      float s[128];
      sm100::mbar_wait(&S.s_full[i], n & 1, abort);
      sm100::tc_fence_after();
#pragma unroll
      for (int c = 0; c < 128; c += 32) tmem_ld_x32(s_col + c, s, c);
      sm100::tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < 128; c += 32) pin32(s, c);
      const bool edge = edge_of(u, u.j0 + n);
      uint32_t none = 0;  // blocks of 32 keys that no row of the warp sees
      if (edge) {
        // columns lo < c <= hi are seen; a warp's rows lie 31 apart at most, so
        // that most blocks are seen by all of them or by none
        const int hi = t - key0, lo = a.window > 0 ? t - a.window - key0 : INT32_MIN;
        const int hi0 = hi - lane, lo0 = a.window > 0 ? lo - lane : INT32_MIN, lo1 = a.window > 0 ? lo0 + 31 : INT32_MIN;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (32 * k > hi0 + 31 || 32 * k + 31 <= lo0) {
            none |= 1u << k;
#pragma unroll
            for (int c = 32 * k; c < 32 * k + 32; ++c) s[c] = -INFINITY;
          } else {
            if (32 * k + 31 > hi0) {
#pragma unroll
              for (int c = 32 * k; c < 32 * k + 32; ++c)
                if (c > hi) s[c] = -INFINITY;
            }
            if (32 * k <= lo1) {
#pragma unroll
              for (int c = 32 * k; c < 32 * k + 32; ++c)
                if (c <= lo) s[c] = -INFINITY;
            }
          }
        }
        if (key0 + kTile > n_k) {
          // rows behind the sequence: cleared, since 0 * NaN is NaN.  (S being
          // here says that the loads of all earlier tiles have been waited
          // for, so this parity cannot mean an earlier one)
          const int nu = u.j0 + n - j_begin, vs = nu % Smem::kV;
          sm100::mbar_wait(&S.v_full[vs], (nu / Smem::kV) & 1, abort);
          clear_rows<kD>(S.v[vs], r, n_k - key0);
        }
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int c = 4; c < 128; c += 4)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = max_nan(mx[e], s[c + e]);
      const float top = max_nan(max_nan(mx[0], mx[1]), max_nan(mx[2], mx[3]));
      const bool over = top - m > a.step;
      if (__any_sync(0xffffffffu, over)) {
        const float alpha = over ? ex2((m - top) * a.scale) : 1.f;  // 0 from -inf
        if (over) m = top;
        far = __any_sync(0xffffffffu, m != -INFINITY && fabsf(m * a.scale) > 1048576.f);
        l *= alpha;
        if (n > 0) {
          // S being here says that the products before it are done
#pragma unroll 1
          for (int c = 0; c < kD; c += 16) {
            uint32_t w[16];
            sm100::tmem_ld_x16(o_col + c, w);
            sm100::tmem_ld_wait();
            sm100::tmem_pin16(w);
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * alpha);
            sm100::tmem_st_x16(o_col + c, w);
          }
        }
      }
      float mc = m == -INFINITY ? 0.f : m * a.scale - kTop;
      if (far) {
        // the rounding of m * scale would move all weights of the row by a factor,
        // up to out of the type's range: differences first
        const float mr = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int c = 0; c < 128; ++c) s[c] -= mr;
        mc = m == -INFINITY ? 0.f : -kTop;
      }
      const uint64_t scale2 = f32x2(a.scale, a.scale), mc2 = f32x2(-mc, -mc);
      uint64_t sum2[2] = {0, 0};
      auto weights = [&](auto poly) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t p[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            if (!decltype(poly)::value && ((none >> (2 * half + c / 16)) & 1)) {
              p[c] = 0;
              continue;
            }
            const uint64_t x2 = fma2(f32x2(s[64 * half + 2 * c], s[64 * half + 2 * c + 1]), scale2, mc2);
            float x, y;
            if (decltype(poly)::value && (c * kPoly) % 8 < kPoly) {
              const uint64_t y2 = exp2_poly<kBf16>(x2);
              split2(y2, x, y);
              sum2[c & 1] = add2(sum2[c & 1], y2);
            } else {
              split2(x2, x, y);
              x = ex2(x);
              y = ex2(y);
              sum2[c & 1] = add2(sum2[c & 1], f32x2(x, y));
            }
            p[c] = pack2<kBf16>(x, y);
          }
          tmem_st_x32(s_col + 32 * half, p);
          sm100::tmem_st_wait();
          sm100::tc_fence_before();
          __syncwarp();
          if (lane == 0) sm100::mbar_arrive(&S.p_full[i][half]);
        }
      };
      if (edge) weights(False{});  // masked weights have to be zeros
      else weights(True{});
      float a0, a1, a2, a3;
      split2(sum2[0], a0, a1);
      split2(sum2[1], a2, a3);
      l += (a0 + a1) + (a2 + a3);
      // a logit that is NaN or +infinity makes the row NaN (the polynomial alone
      // would take it for a small weight)
      if (!(top < INFINITY)) l = NAN;
    }

    // ---- output
    if (work > 0) {
      sm100::mbar_wait(&S.o_full, 0, abort);
      sm100::tc_fence_after();
    }
    if (u.rows > 0) {
      if (a.sink && m != -INFINITY) l += ex2(a.sink[u.head] * kLog2e - (m * a.scale - kTop));
      const float f = l != 0.f ? rcp(l) : 0.f;
      uint32_t top = 0;  // largest magnitude of the row, as bits
      constexpr int kChunks = kD / 8;  // 16-byte pieces of a row
      uint4* stage = reinterpret_cast<uint4*>(S.q[i]) + (warp & 3) * 32 * kChunks;  // the warp's 32 rows
      // (rolled: it runs once, and instructions that are fetched for the first
      // time cost more than the loop)
#pragma unroll 1
      for (int c = 0; c < kD; c += 16) {
        uint32_t w[16];
        if (work > 0) {
          sm100::tmem_ld_x16(o_col + c, w);
          sm100::tmem_ld_wait();
          sm100::tmem_pin16(w);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = 0;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] = __uint_as_float(w[8 * h + e]) * f;
            top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
          }
          stage[lane * kChunks + ((c / 8 + h) ^ (lane & 7))] = pack8<kBf16>(x);
        }
      }
      __syncwarp();
      if (!*abort) {
#pragma unroll 4
        for (int x = lane; x < 32 * kChunks; x += 32) {
          const int row = x / kChunks, ch = x % kChunks;
          if ((warp & 3) * 32 + row < u.rows) {
            uint16_t* dst = reinterpret_cast<uint16_t*>(a.out.ptr) + (int64_t)(u.row0 + (warp & 3) * 32 + row) * a.out.row_stride +
                            (int64_t)u.head * a.out.head_stride + 8 * ch;
            *reinterpret_cast<uint4*>(dst) = stage[row * kChunks + (ch ^ (row & 7))];
          }
        }
        __syncwarp();
        const unsigned odd = __ballot_sync(0xffffffffu, r < u.rows && top >= 0x7F800000u);
        if (odd) rows_again<kBf16, kD>(a, odd, u.j0 * kTile, min(u.j1 * kTile, n_k), u.row0 + (warp & 3) * 32, t - lane, u.head, kvh, k_begin, lane);
      }
    }
  }
  __syncwarp();
  sm100::tc_fence_before();
  __syncthreads();
  if (S.abort && threadIdx.x == 0) raise_err(a.err, CSA_DEV_ERR_TIMEOUT);
  if (warp == 8) {
    sm100::tc_fence_after();
    sm100::tmem_dealloc(tmem, 512);
  }
  pdl_trigger();
}

template <bool kBf16, int kD>
cudaError_t launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const PromptArgs& a, int64_t blocks,
                   cudaStream_t st) {
  auto fn = gqa_prompt_kernel<kBf16, kD>;
  const size_t smem = sizeof(PromptSmem<kD>) + 1024;
  static_assert(sizeof(PromptSmem<kD>) + 1024 <= 232448, "shared memory of a CTA");
  const cudaError_t e = set_max_smem(reinterpret_cast<const void*>(fn), smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(fn, dim3((unsigned)blocks), dim3(kThreads), smem, st, mq, mk, mv, a);
}

}  // namespace

cudaError_t launch_gqa_prompt(const gqa_params& p, const gqa_rows& q, const gqa_rows& k, const gqa_rows& v,
                              int64_t n_q, int64_t n_k, const int32_t* cu_q, const int32_t* cu_k, const float* sink,
                              const gqa_rows& out, int32_t* err, cudaStream_t st) {
  const bool bf = p.act_fmt == CSA_ACT_BF16;
  const CUtensorMapDataType dt = bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  auto encode = [&](CUtensorMap* m, const gqa_rows& x, int64_t rows, int heads) {
    const uint64_t dims[3] = {(uint64_t)p.d, (uint64_t)rows, (uint64_t)heads};
    const uint64_t str[2] = {(uint64_t)x.row_stride * 2, (uint64_t)x.head_stride * 2};
    const uint32_t box[3] = {64, (uint32_t)kTile, 1};
    return encode_tensor_map(m, dt, 3, x.ptr, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  CUtensorMap mq, mk, mv;
  // without keys nothing is loaded: the queries' map stands in
  if (!encode(&mq, q, n_q, p.n_heads) || !encode(&mk, n_k ? k : q, n_k ? n_k : n_q, n_k ? p.n_kv_heads : p.n_heads) ||
      !encode(&mv, n_k ? v : q, n_k ? n_k : n_q, n_k ? p.n_kv_heads : p.n_heads))
    return cudaErrorInvalidValue;
  const float scale = p.softmax_scale * kLog2e;
  const PromptArgs a{q, k, v, out, (int)n_q, (int)n_k, cu_q, cu_k, sink, p.B, p.n_heads, p.n_kv_heads,
                     p.window < (1 << 30) ? p.window : 0, scale,
                     fminf((bf ? Weights<true>::kLazy : Weights<false>::kLazy) / scale, 3.0e38f), err};
  // the most pairs of units that B sequences of n_q queries can have
  const int64_t G = p.n_heads / p.n_kv_heads, tiles = n_q / kTile + (n_q < p.B ? n_q : p.B);
  const int64_t blocks = (tiles * G + p.B + 1) / 2 * p.n_kv_heads;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  return bf ? (p.d == 128 ? launch<true, 128>(mq, mk, mv, a, blocks, st) : launch<true, 64>(mq, mk, mv, a, blocks, st))
            : (p.d == 128 ? launch<false, 128>(mq, mk, mv, a, blocks, st) : launch<false, 64>(mq, mk, mv, a, blocks, st));
}

}  // namespace csa
