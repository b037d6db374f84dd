// gqa_decode_attn: the last T tokens of every sequence attend to the paged
// cache, split over the cache's length and joined.
//
//   z_j = scale q.k_j,  o = sum_j exp(z_j - m) v_j / (exp(sink - m) + sum_j exp(z_j - m))
//
// Every K and V row is read once for the G = n_heads / n_kv_heads query heads
// that share it, so with 16-bit rows a byte carries G flops: the cache's
// bytes bound the call up to about a hundred rows per KV head.
//
// Work.  An item is one sequence's split of its keys, one KV head and up to
// kNq of its T * G query rows.  Splits are a rule on the sequence's own tile
// count (split_tiles), so a query's bits do not depend on its batch.  The
// grid is persistent: CTA c takes items c, c + grid, ... and one producer
// warp runs ahead over item borders, so the stream of tiles never drains.
//
//   producer   one warp.  Reads page ids 32 at a time and moves a tile of 64
//              keys and values per stage with TMA (one box per page and
//              64 dims, a lane each, 128-byte swizzle), page by page, so
//              that pages of any size from 16 on fill a tile.
//   consumers  8 warps in two groups of four that take alternate tiles; a
//              warp owns 16 keys of a tile and keeps its own running maximum,
//              sum and output, so tiles need no barrier among warps:
//                S^T[16 keys, rows] = K Q^T     (mma m16n8k16, K by ldmatrix)
//                P^T = exp2(S^T - m), rounded to 16 bits, transposed in
//                registers by movmatrix
//                O^T[d, rows] += V^T P^T        (V by ldmatrix.trans)
//              With the keys as M, 8 query rows fill an MMA (m16n8k16 with
//              rows as M would waste half of it for the usual groups of 8).
//   item end   the eight warps' results are joined in shared memory in
//              warp order; a sequence with one split is finished here, the
//              others leave (m, l, O) in fp32 for gqa_join_kernel.
//
// FP8 cache.  E4M3 codes become FP16 exactly in registers; the dims of a
// 16-byte piece are dealt to MMA steps in an order that Q's fragments share,
// so no shuffles are needed.  A query row is brought into FP16 by a power of
// two of its own (largest magnitude in [2^14, 2^15); what is 2^29 below that
// loses bits that do not show in fp32).  The value's scale s_j joins the
// weight: w_j = exp2(z_j + log2 s_j - M) with M the running maximum of that
// sum, so weights stay in (0, 1] whatever the scales are, and the
// denominator sums exp2(z_j - M).
//
// Rounding.  Weights are rounded to the MMA's 16-bit type (relative 2^-9
// for BF16, 2^-12 for FP16), sums and partial outputs are fp32.
//
// Masks.  Tiles that a row does not see as a whole (the last one, a window's
// first, pages that are none) take a path of their own: logits are
// selected, and values that are not finite are taken out of the product and
// given to the rows that see them one by one, so that what a masked slot
// holds cannot reach a sum (0 * NaN is NaN).
#include <cuda.h>

#include "gqa.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace csa {

namespace {

using namespace gqa;

constexpr int kTile = 64;         // keys per stage
constexpr int kConsumers = 8;     // warps
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kObufPitch = 68;    // floats per row of the join buffer (a warp's stores hit 32 banks)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinLogScale = -90.f, kMaxLogScale = 90.f;

// Tiles per split for a sequence of n tiles: about 32 splits, of 2 to 16
// tiles (128 to 1024 keys).
__host__ __device__ inline int split_tiles(int n) {
  int c = 2;
  while (c < 16 && c * 32 < n) c *= 2;
  return c;
}
__host__ __device__ inline int n_splits(int n) {
  const int c = split_tiles(n);
  return n <= c ? 1 : (n + c - 1) / c;  // a sequence without keys has one empty split
}
// The most splits that any sequence of up to n tiles has.
inline int most_splits(int n) {
  int most = 1;
  for (int c = 2; c <= 16; c *= 2) {  // the rule's longest sequence for each c
    const int top = c < 16 ? (n < 32 * c ? n : 32 * c) : n;
    if (top > (c > 2 ? 16 * c : 0)) most = most > n_splits(top) ? most : n_splits(top);
  }
  return most;
}

struct DecodeArgs {
  gqa_rows q, out;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  int64_t table_cols;
  const int32_t* lens;
  const float* sink;
  float* part_o;   // [B][max_splits][T * n_heads][d]
  float2* part_ml; // [B][max_splits][T * n_heads]: (m, l), m in base-2 units
  int64_t n_pages;
  int B, T, n_max, n_heads, n_kv, page, page_shift, window, max_splits;
  float scale;  // softmax_scale * log2(e)
  int32_t* err;
};

// Keys [lo, hi) that some query of the sequence sees, and the tiles that
// hold them.
struct Span {
  int len, lo, t0, n;
};
__device__ __forceinline__ Span span_of(const DecodeArgs& a, int b) {
  Span s;
  s.len = max(0, min(a.lens[b], a.n_max));
  s.lo = a.window > 0 ? max(0, s.len - a.T - a.window + 1) : 0;
  s.t0 = s.lo / kTile;
  s.n = s.len > s.lo ? (s.len + kTile - 1) / kTile - s.t0 : 0;
  return s;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <bool kBf16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kBf16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two E4M3 codes (low 16 bits) -> two FP16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(v & 0xFFFFu), __NV_E4M3);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
}
// Halves of a register that are infinities or NaN, as a mask over them.
template <bool kBf16>
__device__ __forceinline__ uint32_t odd_halves(uint32_t v) {
  constexpr uint32_t e = kBf16 ? 0x7F80u : 0x7C00u;
  return ((v & e) == e ? 0xFFFFu : 0u) | ((v & (e << 16)) == (e << 16) ? 0xFFFF0000u : 0u);
}

template <bool kFp8, int kD>
struct Layout {
  static constexpr int kRowBytes = kFp8 ? kD : 2 * kD;
  static constexpr int kHalves = kFp8 ? 1 : kD / 64;           // boxes of 64 dims side by side
  static constexpr int kBoxBytes = kRowBytes / kHalves;        // inner box: 128 bytes (64 for 64-dim FP8)
  static constexpr int kOperand = kTile * kRowBytes;           // K or V of a tile
  static constexpr int kScales = kFp8 ? kTile * 4 : 0;         // K or V scales of a tile
  static constexpr int kStage = 2 * kOperand;
  static constexpr int kObuf = kConsumers * 8 * kObufPitch * 4;  // eight warps' outputs: 8 rows, 64 dims
  // even, so that a stage always belongs to the same group of warps: a group
  // then waits for every phase of its stages' barriers in turn (with an odd
  // count it would meet every second phase, which a parity cannot tell from
  // the one before it)
  static constexpr int kStages = kStage >= 32768 ? 6 : (kFp8 ? (kD == 128 ? 10 : 20) : 12);
  static_assert(kStages % 2 == 0, "a stage belongs to one group");
  static constexpr size_t kSmem = 1024 + (size_t)kStages * (kStage + 2 * kScales) + kObuf;
};

template <bool kBf16, bool kFp8, int kD, int kNq>
__global__ void __launch_bounds__(kThreads, 1)
    gqa_decode_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                      const DecodeArgs a) {
  using L = Layout<kFp8, kD>;
  constexpr bool kMmaBf16 = kBf16 && !kFp8;  // FP8 codes are exact in FP16
  constexpr int kNt = kNq / 8;
  extern __shared__ uint8_t raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  float* scales = reinterpret_cast<float*>(stages + L::kStages * L::kStage);  // [stage][K, V][64]
  float* obuf = reinterpret_cast<float*>(stages + L::kStages * (L::kStage + 2 * L::kScales));
  __shared__ uint64_t full[L::kStages], empty[L::kStages];
  __shared__ uint32_t pages_ok[L::kStages];
  __shared__ float red_m[2][kConsumers][kNq], red_l[2][kConsumers][kNq];
  __shared__ int first_item[2049];  // items before sequence b
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      sm100::mbar_init(&full[s], 1);
      sm100::mbar_init(&empty[s], 4);
    }
    abort_flag = 0;
    sm100::fence_mbar_init();
    sm100::prefetch_tmap(&map_k);
    sm100::prefetch_tmap(&map_v);
  }
  pdl_wait();
  const int G = a.n_heads / a.n_kv, rows = a.T * G;
  const int chunks = (rows + kNq - 1) / kNq;
  if (warp == 0) {
    int base = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      int n = 0;
      if (b0 + lane < a.B) {
        n = n_splits(span_of(a, b0 + lane).n) * a.n_kv * chunks;
        if (blockIdx.x == 0 && a.lens[b0 + lane] > a.n_max) raise_err(a.err, CSA_DEV_ERR_RANGE);
      }
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b0 + lane < a.B) first_item[b0 + lane] = base + x - n;
      base += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) first_item[a.B] = base;
  }
  __syncthreads();
  const int total = first_item[a.B];
  volatile int* abort = &abort_flag;

  // the sequence of an item, walking forward from sequence b
  auto seek = [&](int item, int b) {
    while (item >= first_item[b + 1]) ++b;
    return b;
  };

  if (warp == kConsumers) {
    // ---- producer ------------------------------------------------------------
    const int box_rows = min(a.page, kTile), boxes = kTile / box_rows;  // pages per tile
    int it = 0, b = 0;
    for (int item = blockIdx.x; item < total; item += gridDim.x) {
      b = seek(item, b);
      const Span s = span_of(a, b);
      const int x = (item - first_item[b]) / chunks, kvh = x % a.n_kv, split = x / a.n_kv;
      const int c = split_tiles(s.n);
      const int t_begin = s.t0 + split * c, t_end = min(t_begin + c, s.t0 + s.n);
      const int32_t* row = a.table + (int64_t)b * a.table_cols;
      const int last_page = (s.len - 1) >> a.page_shift, first_page = s.lo >> a.page_shift;
      int have = -1, ids = 0;  // this lane's page id of group `have` (32 pages)
      for (int t = t_begin; t < t_end; ++t, ++it) {
        const int st = it % L::kStages;
        const int p0 = (t * kTile) >> a.page_shift;  // first page of the tile (a group holds all of them)
        if ((p0 >> 5) != have) {
          have = p0 >> 5;
          const int p = 32 * have + lane;
          ids = (p >= first_page && p <= last_page) ? row[p] : -1;
          const bool bad = p >= first_page && p <= last_page && (ids < 0 || ids >= a.n_pages);
          if (bad) {
            ids = -1;
            if (p >= p0 && p <= ((t_end * kTile - 1) >> a.page_shift)) raise_err(a.err, CSA_DEV_ERR_INDEX);
          }
        }
        if (it >= L::kStages) sm100::mbar_wait(&empty[st], (it / L::kStages - 1) & 1, abort);
        if (*abort) break;
        const int id_l = __shfl_sync(0xffffffffu, ids, (p0 + (lane & 3)) & 31);
        const uint32_t ok = __ballot_sync(0xffffffffu, id_l >= 0) & ((1u << boxes) - 1);
        if (lane == 0) {
          pages_ok[st] = ok;
          sm100::mbar_arrive_expect_tx(&full[st], __popc(ok) * box_rows * 2 * (L::kRowBytes + (kFp8 ? 4 : 0)));
        }
        __syncwarp();
        // lane = box + 4 half + 8 (value) (+ 16: scales)
        const int box = lane & 3, half = (lane >> 2) & 1, val = (lane >> 3) & 1;
        if (box < boxes && id_l >= 0 && half < L::kHalves) {
          const int slot = (t * kTile) & (a.page - 1);
          const int64_t head_page = (int64_t)id_l * a.n_kv + kvh;
          if (lane < 16) {
            uint8_t* dst = stages + st * L::kStage + val * L::kOperand + half * kTile * 128 + box * box_rows * L::kBoxBytes;
            sm100::tma_load_3d(dst, val ? &map_v : &map_k, &full[st], half * 64, slot, (int)head_page);
          } else if (kFp8) {
            float* dst = scales + (st * 2 + val) * kTile + box * box_rows;
            sm100::bulk_load(dst, (val ? a.v_scale : a.k_scale) + head_page * a.page + slot, box_rows * 4, &full[st]);
          }
        }
        __syncwarp();
      }
      if (*abort) break;
    }
    // after a timeout: copies still in flight land before the CTA goes
    if (*abort)
      for (int i = max(0, it - L::kStages); i < it; ++i) {
        const uint64_t t0 = sm100::globaltimer();
        while (!sm100::mbar_try_wait(&full[i % L::kStages], (i / L::kStages) & 1) &&
               sm100::globaltimer() - t0 < sm100::kWaitNs) {
        }
      }
  } else {
    // ---- consumers -------------------------------------------------------------
    const int g = lane >> 2, q4 = lane & 3, grp = warp >> 2, w16 = (warp & 3) * 16;
    int it = 0, b = 0, par = 0;
    for (int item = blockIdx.x; item < total; item += gridDim.x, par ^= 1) {
      b = seek(item, b);
      const Span s = span_of(a, b);
      const int in_b = item - first_item[b];
      const int chunk = in_b % chunks, x = in_b / chunks, kvh = x % a.n_kv, split = x / a.n_kv;
      const int c = split_tiles(s.n);
      const int t_begin = s.t0 + split * c, t_end = min(t_begin + c, s.t0 + s.n);
      const bool single = s.n <= c;

      // query fragments: B operand, column g of n-tile nt is query row
      // chunk * kNq + 8 nt + g = tau * G + head
      uint32_t qf[kNt][kD / 16][2];
      float qs[kNt][2];      // logit factor of columns 2 q4, 2 q4 + 1
      int tq[kNt][2];        // their positions (INT_MIN: no row)
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) {
        const int r = chunk * kNq + 8 * nt + g;
        const bool live = r < rows;
        const int tau = live ? r / G : 0, h = kvh * G + (live ? r % G : 0);
        const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q.ptr) +
                              ((int64_t)b * a.T + tau) * a.q.row_stride + (int64_t)h * a.q.head_stride;
        if (!kFp8) {
#pragma unroll
          for (int kk = 0; kk < kD / 16; ++kk)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              qf[nt][kk][e] = live ? *reinterpret_cast<const uint32_t*>(src + 16 * kk + 8 * e + 2 * q4) : 0u;
          qs[nt][0] = qs[nt][1] = a.scale;
        } else {
          // this lane's dims: kD/4 consecutive ones from kD/4 * q4 on
          uint4 v[kD / 32];
          float am = 0.f;
#pragma unroll
          for (int i = 0; i < kD / 32; ++i) {
            v[i] = live ? reinterpret_cast<const uint4*>(src + kD / 4 * q4)[i] : make_uint4(0, 0, 0, 0);
            float f[8];
            unpack8<kBf16>(v[i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) am = fmaxf(am, fabsf(f[j]));
          }
          am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
          am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
          // 2^-e brings the largest magnitude into [2^14, 2^15)
          const int e = am > 0.f ? min(126, max(-112, (int)((__float_as_uint(am) >> 23) & 0xFFu) - 127 - 14)) : 0;
          const float down = __uint_as_float((uint32_t)(127 - e) << 23), up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
          for (int i = 0; i < kD / 32; ++i) {
            float f[8];
            unpack8<kBf16>(v[i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] *= down;
            const uint4 u = pack8<false>(f);
            qf[nt][2 * i][0] = u.x; qf[nt][2 * i][1] = u.y;
            qf[nt][2 * i + 1][0] = u.z; qf[nt][2 * i + 1][1] = u.w;
          }
          // column c's factor sits in lanes 4 c .. 4 c + 3
          qs[nt][0] = a.scale * __shfl_sync(0xffffffffu, up, 8 * q4);
          qs[nt][1] = a.scale * __shfl_sync(0xffffffffu, up, 8 * q4 + 4);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rc = chunk * kNq + 8 * nt + 2 * q4 + e;
          tq[nt][e] = rc < rows ? s.len - a.T + rc / G : INT32_MIN;
        }
      }

      float m[kNt][2], l[kNt][2], o[kD / 16][kNt][4];
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < kD / 16; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
      }

      for (int t = t_begin; t < t_end; ++t, ++it) {
        if ((it & 1) != grp) continue;
        const int st = it % L::kStages;
        sm100::mbar_wait(&full[st], (it / L::kStages) & 1, abort);
        const int key0 = t * kTile + w16;  // this warp's first key
        const uint32_t sk = sm100::smem_u32(stages + st * L::kStage), sv = sk + L::kOperand;
        const uint32_t all = (1u << (kTile / min(a.page, kTile))) - 1, okp = pages_ok[st];
        // seen by every row: keys up to the first query, from the last query's window on
        const bool edge = okp != all || key0 + 15 > s.len - a.T || (a.window > 0 && key0 < s.len - a.window);

        // S^T = K Q^T
        float z[kNt][4];
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt) z[nt][0] = z[nt][1] = z[nt][2] = z[nt][3] = 0.f;
        if (!kFp8) {
          const int r = w16 + (lane & 15);
#pragma unroll
          for (int kk = 0; kk < kD / 16; ++kk) {
            uint32_t af[4];
            const int ch = 2 * (kk & 3) + (lane >> 4);
            ldsm4(sk + (kk >> 2) * kTile * 128 + r * 128 + ((ch ^ (r & 7)) << 4), af);
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) mma16816<kMmaBf16>(z[nt], af, qf[nt][kk][0], qf[nt][kk][1]);
          }
        } else {
          // 16 codes of rows g and g + 8 at a time: four MMA steps, whose
          // dims are 4 s .. 4 s + 3 of this lane's piece
#pragma unroll
          for (int i = 0; i < kD / 64; ++i) {
            uint4 w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = w16 + g + 8 * e;
              const uint32_t at = kD == 128 ? (uint32_t)(r * 128 + (((2 * q4 + i) ^ (r & 7)) << 4))
                                            : (uint32_t)(r * 64 + ((q4 ^ ((r >> 1) & 3)) << 4));
              asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                           : "=r"(w[e].x), "=r"(w[e].y), "=r"(w[e].z), "=r"(w[e].w) : "r"(sk + at) : "memory");
            }
            const uint32_t w0[4] = {w[0].x, w[0].y, w[0].z, w[0].w}, w1[4] = {w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
            for (int sp = 0; sp < 4; ++sp) {
              const uint32_t af[4] = {e4m3x2_to_f16x2(w0[sp]), e4m3x2_to_f16x2(w1[sp]), e4m3x2_to_f16x2(w0[sp] >> 16),
                                      e4m3x2_to_f16x2(w1[sp] >> 16)};
#pragma unroll
              for (int nt = 0; nt < kNt; ++nt) mma16816<false>(z[nt], af, qf[nt][4 * i + sp][0], qf[nt][4 * i + sp][1]);
            }
          }
        }
        float ks[2] = {1.f, 1.f}, lv[2] = {0.f, 0.f};  // of keys g, g + 8
        if (kFp8) {
          const float* sc = scales + st * 2 * kTile + w16 + g;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            ks[e] = sc[8 * e];
            lv[e] = fminf(fmaxf(log2f(sc[kTile + 8 * e]), kMinLogScale), kMaxLogScale);
          }
        }
        // base-2 logits; masked ones -inf
        auto seen = [&](int key, int tcol) {
          const bool in_page = (okp >> ((key & (kTile - 1)) / min(a.page, kTile))) & 1u;
          return in_page && key <= tcol && (a.window == 0 || key > tcol - a.window);
        };
        float u[kNt][4];  // logit plus the value's log-scale
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            z[nt][e] *= kFp8 ? qs[nt][e & 1] * ks[e >> 1] : qs[nt][e & 1];
            if (edge && !seen(key0 + g + 8 * (e >> 1), tq[nt][e & 1])) z[nt][e] = -INFINITY;
            u[nt][e] = kFp8 ? (z[nt][e] == -INFINITY ? -INFINITY : z[nt][e] + lv[e >> 1]) : z[nt][e];
          }
        // running maxima over the 16 keys (lanes of equal q4)
        bool moved = false;
        float alpha[kNt][2];
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = fmaxf(u[nt][e], u[nt][e + 2]);
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            alpha[nt][e] = 1.f;
            if (v > m[nt][e]) {
              alpha[nt][e] = ex2(m[nt][e] - v);  // 0 from -inf
              m[nt][e] = v;
              moved = true;
            }
          }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt) {
            l[nt][0] *= alpha[nt][0];
            l[nt][1] *= alpha[nt][1];
#pragma unroll
            for (int mt = 0; mt < kD / 16; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[mt][nt][e] *= alpha[nt][e & 1];
          }
        }
        uint32_t pf[kNt][2];
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float mr = m[nt][e & 1] == -INFINITY ? 0.f : m[nt][e & 1];
            p[e] = ex2(u[nt][e] - mr);
            l[nt][e & 1] += kFp8 ? ex2(z[nt][e] - mr) : p[e];
          }
          pf[nt][0] = transpose8x8(pack2<kMmaBf16>(p[0], p[1]));
          pf[nt][1] = transpose8x8(pack2<kMmaBf16>(p[2], p[3]));
        }

        // O^T += V^T P^T.  Row g / g + 8 of m-tile mt is dim dim_of(mt, 0 / 1).
        uint32_t odd = 0;
        if (!kFp8) {
          const int i = lane >> 3, r = w16 + (lane & 7) + 8 * (i >> 1);
#pragma unroll
          for (int mt = 0; mt < kD / 16; ++mt) {
            uint32_t af[4];
            const int ch = 2 * (mt & 3) + (i & 1);
            ldsm4t(sv + (mt >> 2) * kTile * 128 + r * 128 + ((ch ^ (r & 7)) << 4), af);
            if (edge) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t bad = odd_halves<kMmaBf16>(af[e]);
                odd |= bad;
                af[e] &= ~bad;
              }
            }
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) mma16816<kMmaBf16>(o[mt][nt], af, pf[nt][0], pf[nt][1]);
          }
        } else {
          // kD/8 codes of keys 2 q4, 2 q4 + 1, + 8, + 9 from dim kD/8 * g on
          constexpr int kW = kD / 32;  // words per key
          uint32_t w[4][kW];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = w16 + 2 * q4 + (e & 1) + 8 * (e >> 1);
            if (kD == 128) {
              const uint32_t at = (uint32_t)(r * 128 + ((g ^ (r & 7)) << 4));
              asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                           : "=r"(w[e][0]), "=r"(w[e][1]), "=r"(w[e][kW - 2]), "=r"(w[e][kW - 1]) : "r"(sv + at) : "memory");
            } else {
              const uint32_t at = (uint32_t)(r * 64 + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + (g & 1) * 8);
              asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[e][0]), "=r"(w[e][1]) : "r"(sv + at) : "memory");
            }
          }
#pragma unroll
          for (int mt = 0; mt < kD / 16; ++mt) {
            const int wi = mt / 2;
            const uint32_t sel = (mt & 1) ? 0x7362u : 0x5140u;
            const uint32_t lo = __byte_perm(w[0][wi], w[1][wi], sel), hi = __byte_perm(w[2][wi], w[3][wi], sel);
            uint32_t af[4] = {e4m3x2_to_f16x2(lo), e4m3x2_to_f16x2(lo >> 16), e4m3x2_to_f16x2(hi), e4m3x2_to_f16x2(hi >> 16)};
            if (edge) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t bad = odd_halves<false>(af[e]);
                odd |= bad;
                af[e] &= ~bad;
              }
            }
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) mma16816<false>(o[mt][nt], af, pf[nt][0], pf[nt][1]);
          }
        }
        if (edge && __any_sync(0xffffffffu, odd != 0)) {
          // give each value that is not finite to the rows that see it
#pragma unroll
          for (int mt = 0; mt < kD / 16; ++mt)
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) {
              const int dim = kFp8 ? kD / 8 * g + 2 * mt + e2 : 16 * mt + g + 8 * e2;
#pragma unroll 1
              for (int k = 0; k < 16; ++k) {
                const int r = w16 + k;
                float v;
                if (!kFp8) {
                  const uint32_t at = (uint32_t)((dim >> 6) * kTile * 128 + r * 128 + ((((dim >> 3) & 7) ^ (r & 7)) << 4) + (dim & 7) * 2);
                  const uint32_t bits = *reinterpret_cast<const uint16_t*>(stages + st * L::kStage + L::kOperand + at);
                  v = unpack2<kBf16>(bits).x;
                } else {
                  const uint32_t at = kD == 128 ? (uint32_t)(r * 128 + (((dim >> 4) ^ (r & 7)) << 4) + (dim & 15))
                                                : (uint32_t)(r * 64 + (((dim >> 4) ^ ((r >> 1) & 3)) << 4) + (dim & 15));
                  v = e4m3_to_f32(stages[st * L::kStage + L::kOperand + at]);
                }
                if (!(fabsf(v) < INFINITY)) {
#pragma unroll
                  for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                      if (seen(key0 + k, tq[nt][e])) o[mt][nt][2 * e2 + e] += v;
                }
              }
            }
        }
        __syncwarp();
        if (lane == 0) sm100::mbar_arrive(&empty[st]);
      }

      // ---- join the eight warps ----
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = l[nt][e];
          v += __shfl_xor_sync(0xffffffffu, v, 4);
          v += __shfl_xor_sync(0xffffffffu, v, 8);
          v += __shfl_xor_sync(0xffffffffu, v, 16);
          if (g == 0) {
            red_m[par][warp][8 * nt + 2 * q4 + e] = m[nt][e];
            red_l[par][warp][8 * nt + 2 * q4 + e] = v;
          }
        }
      sm100::named_bar_sync(1, 32 * kConsumers);
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) {
        if (chunk * kNq + 8 * nt >= rows) break;
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float M = -INFINITY;
#pragma unroll
          for (int w = 0; w < kConsumers; ++w) M = fmaxf(M, red_m[par][w][8 * nt + 2 * q4 + e]);
          f[e] = M == -INFINITY ? 0.f : ex2(m[nt][e] - M);
        }
#pragma unroll
        for (int hh = 0; hh < kD / 64; ++hh) {  // 64 dims (four m-tiles) at a time
          if (nt + hh > 0) sm100::named_bar_sync(1, 32 * kConsumers);  // the last ones' sums are read
#pragma unroll
          for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int pos = kFp8 ? 8 * g + 2 * mt + (e >> 1) : 16 * mt + g + 8 * (e >> 1);
              obuf[(warp * 8 + 2 * q4 + (e & 1)) * kObufPitch + pos] =
                  f[e & 1] == 0.f ? 0.f : o[4 * hh + mt][nt][e] * f[e & 1];
            }
          sm100::named_bar_sync(1, 32 * kConsumers);
          // threads 0 .. 127: four dims of one row each
          const int col = threadIdx.x >> 4, pos = (threadIdx.x & 15) * 4, r = chunk * kNq + 8 * nt + col;
          if (col >= 8 || r >= rows) continue;
          const int dim = kFp8 ? kD / 8 * (pos >> 3) + 8 * hh + (pos & 7) : 64 * hh + pos;
          float M = -INFINITY, den = 0.f;
#pragma unroll
          for (int w = 0; w < kConsumers; ++w) M = fmaxf(M, red_m[par][w][8 * nt + col]);
          float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kConsumers; ++w) {
            const float4 v = *reinterpret_cast<const float4*>(obuf + (w * 8 + col) * kObufPitch + pos);
            sum.x += v.x; sum.y += v.y; sum.z += v.z; sum.w += v.w;
            if (M != -INFINITY) den += red_l[par][w][8 * nt + col] * ex2(red_m[par][w][8 * nt + col] - M);
          }
          const int tau = r / G, h = kvh * G + r % G;
          if (single) {
            if (a.sink && M != -INFINITY) den += ex2(a.sink[h] * kLog2e - M);
            const float inv = den != 0.f ? 1.f / den : 0.f;
            uint16_t* dst = reinterpret_cast<uint16_t*>(a.out.ptr) + ((int64_t)b * a.T + tau) * a.out.row_stride +
                            (int64_t)h * a.out.head_stride + dim;
            *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<kBf16>(sum.x * inv, sum.y * inv), pack2<kBf16>(sum.z * inv, sum.w * inv));
          } else {
            const int64_t slot = ((int64_t)b * a.max_splits + split) * a.T * a.n_heads + tau * a.n_heads + h;
            *reinterpret_cast<float4*>(a.part_o + slot * kD + dim) = sum;
            if (dim == 0) a.part_ml[slot] = make_float2(M, den);
          }
        }
      }
    }
  }
  __syncthreads();
  pdl_trigger();
  if (abort_flag && threadIdx.x == 0) raise_err(a.err, CSA_DEV_ERR_TIMEOUT);
}

// Joins the splits of one (query row, head): M = max m_s, o = sum_s
// exp2(m_s - M) O_s / (exp2(sink - M) + sum_s exp2(m_s - M) l_s).  One CTA
// per row; warp w takes splits w, w + 8, ... in order and the warps are added
// in order.
template <bool kBf16, int kD>
__global__ void __launch_bounds__(256) gqa_join_kernel(const DecodeArgs a) {
  __shared__ float red[8][kD];
  __shared__ float red_l[8], red_m[8];
  pdl_wait();
  const int row = blockIdx.x, h = blockIdx.y, b = row / a.T, tau = row % a.T;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = n_splits(span_of(a, b).n);
  if (n == 1) return;  // finished by gqa_decode_kernel
  const int64_t stride = (int64_t)a.T * a.n_heads;
  const int64_t slot = (int64_t)b * a.max_splits * stride + tau * a.n_heads + h;
  float M = -INFINITY;
  for (int s = threadIdx.x; s < n; s += 256) M = fmaxf(M, a.part_ml[slot + s * stride].x);
  M = warp_max(M);
  if (lane == 0) red_m[warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) M = fmaxf(M, red_m[w]);
  constexpr int kV = kD / 32;
  float acc[kV] = {}, den = 0.f;
  if (M != -INFINITY) {
#pragma unroll 4
    for (int s = warp; s < n; s += 8) {
      const float2 ml = a.part_ml[slot + s * stride];
      const float f = ex2(ml.x - M);
      den = fmaf(ml.y, f, den);
      const float* src = a.part_o + (slot + s * stride) * kD + kV * lane;
      if (kV == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        acc[0] = fmaf(v.x, f, acc[0]); acc[1] = fmaf(v.y, f, acc[1]);
        acc[kV - 2] = fmaf(v.z, f, acc[kV - 2]); acc[kV - 1] = fmaf(v.w, f, acc[kV - 1]);
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src);
        acc[0] = fmaf(v.x, f, acc[0]); acc[1] = fmaf(v.y, f, acc[1]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kV; ++i) red[warp][kV * lane + i] = acc[i];
  if (lane == 0) red_l[warp] = den;
  __syncthreads();
  if (threadIdx.x < kD / 2) {
    float x = 0.f, y = 0.f, l = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      x += red[w][2 * threadIdx.x];
      y += red[w][2 * threadIdx.x + 1];
      l += red_l[w];
    }
    if (a.sink && M != -INFINITY) l += ex2(a.sink[h] * kLog2e - M);
    const float inv = l != 0.f ? 1.f / l : 0.f;
    uint16_t* dst = reinterpret_cast<uint16_t*>(a.out.ptr) + (int64_t)row * a.out.row_stride +
                    (int64_t)h * a.out.head_stride + 2 * threadIdx.x;
    *reinterpret_cast<uint32_t*>(dst) = pack2<kBf16>(x * inv, y * inv);
  }
}

int most_tiles(const gqa_params& p, int T, int n_max) {
  int64_t keys = n_max;
  if (p.window > 0 && keys > (int64_t)p.window + T - 1) keys = (int64_t)p.window + T - 1 + kTile - 1;
  return (int)((keys + kTile - 1) / kTile);
}

template <bool kBf16, bool kFp8, int kD, int kNq>
cudaError_t launch(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeArgs& a, int64_t items, cudaStream_t st) {
  using L = Layout<kFp8, kD>;
  auto fn = gqa_decode_kernel<kBf16, kFp8, kD, kNq>;
  cudaError_t e = set_max_smem(reinterpret_cast<const void*>(fn), L::kSmem);
  if (e != cudaSuccess) return e;
  const int grid = (int)(items < sm_count() ? items : sm_count());
  e = launch_pdl(fn, dim3(grid), dim3(kThreads), L::kSmem, st, mk, mv, a);
  if (e != cudaSuccess || a.max_splits == 1) return e;
  return launch_pdl(gqa_join_kernel<kBf16, kD>, dim3(a.B * a.T, a.n_heads), dim3(256), 0, st, a);
}

}  // namespace

size_t gqa_decode_workspace_bytes(const gqa_params& p, int T, int n_max) {
  const int s = most_splits(most_tiles(p, T, n_max));
  if (s == 1) return 0;
  return (size_t)p.B * s * T * p.n_heads * (p.d + 2) * sizeof(float);
}

cudaError_t launch_gqa_decode(const gqa_params& p, const gqa_rows& q, const gqa_cache& cache, const int32_t* table,
                              int64_t table_cols, const int32_t* lens, int T, int n_max, const float* sink,
                              const gqa_rows& out, void* ws, int32_t* err, cudaStream_t st) {
  const bool bf = p.act_fmt == CSA_ACT_BF16, f8 = p.kv_fmt == CSA_KV_FP8;
  CUtensorMap mk, mv;
  const uint64_t es = f8 ? 1 : 2;
  const uint64_t dims[3] = {(uint64_t)p.d, (uint64_t)p.page, (uint64_t)cache.n_pages * p.n_kv_heads};
  const uint64_t str[2] = {p.d * es, (uint64_t)p.page * p.d * es};
  const uint32_t box[3] = {f8 ? (uint32_t)p.d : 64u, (uint32_t)(p.page < kTile ? p.page : kTile), 1};
  const CUtensorMapSwizzle sw = f8 && p.d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  const CUtensorMapDataType dt = f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!encode_tensor_map(&mk, dt, 3, cache.k, dims, str, box, sw) ||
      !encode_tensor_map(&mv, dt, 3, cache.v, dims, str, box, sw))
    return cudaErrorInvalidValue;
  const int splits = most_splits(most_tiles(p, T, n_max));
  const int64_t slots = (int64_t)p.B * splits * T * p.n_heads;
  float* part_o = reinterpret_cast<float*>(ws);
  int shift = 0;
  while ((1 << shift) < p.page) ++shift;
  const DecodeArgs a{q, out, cache.k_scale, cache.v_scale, table, table_cols, lens, sink, part_o,
                     splits > 1 ? reinterpret_cast<float2*>(part_o + slots * p.d) : nullptr, cache.n_pages, p.B, T,
                     n_max, p.n_heads, p.n_kv_heads, p.page, shift, p.window, splits, p.softmax_scale * kLog2e, err};
  // 8 query rows per item where they hold the whole group, else 16
  const int rows = T * (p.n_heads / p.n_kv_heads), nq = rows <= 8 ? 8 : 16;
  const int64_t items = (int64_t)p.B * splits * p.n_kv_heads * ((rows + nq - 1) / nq);
  if (items > INT32_MAX) return cudaErrorInvalidValue;
#define GQA_GO(BF, F8)                                                                                              \
  (p.d == 128 ? (nq == 8 ? launch<BF, F8, 128, 8>(mk, mv, a, items, st) : launch<BF, F8, 128, 16>(mk, mv, a, items, st)) \
              : (nq == 8 ? launch<BF, F8, 64, 8>(mk, mv, a, items, st) : launch<BF, F8, 64, 16>(mk, mv, a, items, st)))
  return bf ? (f8 ? GQA_GO(true, true) : GQA_GO(true, false)) : (f8 ? GQA_GO(false, true) : GQA_GO(false, false));
#undef GQA_GO
}

}  // namespace csa
