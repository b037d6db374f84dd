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
// count (split_tiles), so a query's bits do not depend on its batch.  Every
// warp works alone: worker w takes items w, w + workers, ... and leaves the
// item's (m, l, O) in fp32 for gqa_join_kernel, or the result where the
// sequence has one split.
//
//   tiles    16 keys and values, always inside one page.  A warp owns a ring
//            of stages and refills each with TMA as soon as it has read it;
//            the loading side runs ahead over item borders, so the stream of
//            tiles never drains.  No barrier among warps, no producer: a
//            first version joined eight warps' results per item in shared
//            memory and spent twice the instructions on short splits.
//   product  S^T[16 keys, rows] = K Q^T     (mma m16n8k16, K by ldmatrix)
//            P^T = exp2(S^T - m), rounded to 16 bits, transposed in
//            registers by movmatrix
//            O^T[d, rows] += V^T P^T        (V by ldmatrix.trans)
//            With the keys as M, 8 query rows fill an MMA (with rows as M
//            the usual groups of 8 would waste half of it).
//
// FP8 cache.  E4M3 codes become FP16 (of 2^-8 their value, exactly) in registers; the dims of a
// 16-byte piece are dealt to MMA steps in an order that Q's fragments share,
// so no shuffles are needed.  A query row is brought into FP16 by a power of
// two of its own (largest magnitude in [2^14, 2^15); what is 2^29 below that
// loses bits that do not show in fp32).  The value's scale s_j joins the
// weight: w_j = exp2(z_j + log2 s_j - M) with M the running maximum of that
// sum, so weights stay in (0, 1] whatever the scales are, and the
// denominator sums exp2(z_j - M).  Scales are read as within 2^-90 .. 2^90.
//
// Rounding.  Weights are rounded to the MMA's 16-bit type (relative 2^-9
// for BF16, 2^-12 for FP16), sums and partial outputs are fp32.
//
// Masks.  Tiles of pages that are none are passed over.  Tiles that a row
// does not see as a whole (the last ones, a window's first) take a path of
// their own: logits are selected, and values that are not finite are taken
// out of the product and given to the rows that see them one by one, so that
// what a masked slot holds cannot reach a sum (0 * NaN is NaN).
#include <cuda.h>

#include "gqa.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace csa {

namespace {

using namespace gqa;

constexpr int kTile = 16;  // keys per stage
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLazy = 8.f;      // base-2 units
constexpr float kMinLogScale = -90.f, kMaxLogScale = 90.f;

// Tiles per split for a sequence of n tiles: about 32 splits of 8 to 32 tiles
// (128 to 512 keys).
constexpr int kMinSplit = 8, kMaxSplit = 32, kSplits = 32;
__host__ __device__ inline int split_tiles(int n) {
  int c = kMinSplit;
  while (c < kMaxSplit && c * kSplits < n) c *= 2;
  return c;
}
__host__ __device__ inline int n_splits(int n) {
  const int c = split_tiles(n);
  return n <= c ? 1 : (n + c - 1) / c;  // a sequence without keys has one empty split
}
// The most splits that any sequence of up to n tiles has.
inline int most_splits(int n) {
  int most = n_splits(n);
  for (int c = kMinSplit; c < kMaxSplit; c *= 2)  // the longest sequence cut into c tiles
    if (c * kSplits < n && most < kSplits) most = kSplits;
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
// E4M3 codes in bytes 1 and 3 (bytes 0 and 2) -> two FP16 of 2^-8 their
// value: sign, four exponent and three mantissa bits move to FP16's places
// (its exponent bias is 8 larger), subnormals included.  Three or four ALU
// instructions for two codes; the conversion instruction goes through the
// 16-lane special-function pipe, which 128 codes a lane and 16 keys fill.
// `top` gathers the largest magnitudes, which tell whether a NaN code was
// among them (they come out as +-480 here).
__device__ __forceinline__ uint32_t codes13_to_f16x2(uint32_t v, uint32_t& top) {
  const uint32_t mag = (v >> 1) & 0x3F803F80u;
  top = __vmaxu2(top, mag);
  return (v & 0x80008000u) | mag;
}
__device__ __forceinline__ uint32_t codes02_to_f16x2(uint32_t v, uint32_t& top) { return codes13_to_f16x2(v << 8, top); }
__device__ __forceinline__ bool has_nan_code(uint32_t top) {
  return (top & 0xFFFFu) == 0x3F80u || (top >> 16) == 0x3F80u;
}
constexpr float kCodeExp = 8.f, kCodeFactor = 256.f;

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

// K or V of a tile: 16 rows of one page and head, the 64-dim halves of a
// 16-bit row one after the other.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::
          "r"(sm100::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(sm100::smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
// Halves of a register that are infinities or NaN, as a mask over them.
template <bool kBf16>
__device__ __forceinline__ uint32_t odd_halves(uint32_t v) {
  constexpr uint32_t e = kBf16 ? 0x7F80u : 0x7C00u;
  return ((v & e) == e ? 0xFFFFu : 0u) | ((v & (e << 16)) == (e << 16) ? 0xFFFF0000u : 0u);
}

template <bool kFp8, int kD, int kNq>
struct Layout {
  // 12 warps of up to 168 registers hold 8 query rows each, 8 warps 16 rows
  static constexpr int kWarps = kNq == 8 ? 12 : 8;
  static constexpr int kRowBytes = kFp8 ? kD : 2 * kD;
  static constexpr int kOperand = kTile * kRowBytes;          // K or V of a tile
  static constexpr int kScales = kFp8 ? 2 * kTile * 4 : 0;    // its scales, K then V
  static constexpr int kStage = 2 * kOperand;
  static constexpr int kStages = 196608 / kWarps / kStage;    // per warp: about 192 KB in flight on an SM
  static constexpr size_t kSmem = 1024 + (size_t)kWarps * kStages * (kStage + kScales);
};

// Where a worker stands: its item, and the tile in it.
struct Cursor {
  int item, b, kvh, split, chunk;  // chunk: which kNq of the query rows
  int t, t_end;                    // tiles of 16 keys from the sequence's start
  Span s;
};

template <bool kBf16, bool kFp8, int kD, int kNq>
__global__ void __launch_bounds__(32 * Layout<kFp8, kD, kNq>::kWarps, 1)
    gqa_decode_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                      const DecodeArgs a) {
  using L = Layout<kFp8, kD, kNq>;
  constexpr bool kMmaBf16 = kBf16 && !kFp8;  // FP8 codes are exact in FP16
  constexpr int kNt = kNq / 8;
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t full_bar[L::kWarps][L::kStages];
  __shared__ int first_item[2049];  // items before sequence b
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* all = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* ring = all + warp * L::kStages * L::kStage;
  float* scales = reinterpret_cast<float*>(all + L::kWarps * L::kStages * L::kStage + warp * L::kStages * L::kScales);
  uint64_t* full = full_bar[warp];

  if (lane == 0) {
    for (int s = 0; s < L::kStages; ++s) sm100::mbar_init(&full[s], 1);
    sm100::fence_mbar_init();
    if (warp == 0) {
      abort_flag = 0;
      sm100::prefetch_tmap(&map_k);
      sm100::prefetch_tmap(&map_v);
    }
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
  // workers are numbered across the SMs first
  const int worker = warp * gridDim.x + blockIdx.x, workers = L::kWarps * gridDim.x;
  volatile int* abort = &abort_flag;

  // Enters the cursor's item (or runs past the end).
  auto enter = [&](Cursor& c) {
    if (c.item >= total) return;
    while (c.item >= first_item[c.b + 1]) ++c.b;
    const int in_b = c.item - first_item[c.b], x = in_b / chunks;
    c.chunk = in_b - x * chunks;
    c.split = x / a.n_kv;
    c.kvh = x - c.split * a.n_kv;
    c.s = span_of(a, c.b);
    const int n = split_tiles(c.s.n);
    c.t = c.s.t0 + c.split * n;
    c.t_end = min(c.t + n, c.s.t0 + c.s.n);
  };

  // ---- loading side: page ids 32 at a time, then one tile per free stage
  Cursor ld;
  ld.item = worker;
  ld.b = 0;
  enter(ld);
  int ids = -1, group = -1;  // this lane's page id of 32-page group `group` of the item's sequence
  uint32_t issued = 0;       // tiles given a stage so far
  uint32_t none = 0;         // stages whose tile belongs to no page (nothing is loaded)
  // The next tile of the loading side goes to stage issued % kStages; false
  // at the end of the work.
  auto load_next = [&]() {
    while (ld.item < total) {
      if (ld.t >= ld.t_end) {
        ld.item += workers;
        enter(ld);
        group = -1;
        continue;
      }
      const int p = (ld.t * kTile) >> a.page_shift;
      if ((p >> 5) != group) {
        group = p >> 5;
        const int mine = 32 * group + lane;
        const int last = (min(ld.t_end * kTile, ld.s.len) - 1) >> a.page_shift;
        ids = -1;
        if (mine >= p && mine <= last) {
          const int id = a.table[(int64_t)ld.b * a.table_cols + mine];
          if (id >= 0 && id < a.n_pages) ids = id;
          else raise_err(a.err, CSA_DEV_ERR_INDEX);
        }
      }
      const int id = __shfl_sync(0xffffffffu, ids, p & 31);
      const int st = issued % L::kStages;
      none = id >= 0 ? none & ~(1u << st) : none | (1u << st);
      if (lane == 0) {
        if (id >= 0) {
          sm100::mbar_arrive_expect_tx(&full[st], L::kStage + L::kScales);
          uint8_t* dst = ring + st * L::kStage;
          const int slot = (ld.t * kTile) & (a.page - 1), head_page = id * a.n_kv + ld.kvh;
          tma_load_4d(dst, &map_k, &full[st], 0, slot, 0, head_page);
          tma_load_4d(dst + L::kOperand, &map_v, &full[st], 0, slot, 0, head_page);
          if (kFp8) {
            const int64_t at = (int64_t)head_page * a.page + slot;
            sm100::bulk_load(scales + st * 2 * kTile, a.k_scale + at, kTile * 4, &full[st]);
            sm100::bulk_load(scales + st * 2 * kTile + kTile, a.v_scale + at, kTile * 4, &full[st]);
          }
        } else {
          sm100::mbar_arrive(&full[st]);
        }
      }
      ++ld.t;
      ++issued;
      return;
    }
  };
  for (int i = 0; i < L::kStages; ++i) load_next();

  // ---- computing side
  const int g = lane >> 2, q4 = lane & 3;
  uint32_t done = 0;
  bool lost = false;
  Cursor c;
  c.b = 0;
  for (c.item = worker; c.item < total && !lost; c.item += workers) {
    enter(c);
    const bool single = c.s.n <= split_tiles(c.s.n);

    // query fragments: B operand, column g of n-tile nt is query row
    // chunk * kNq + 8 nt + g = tau * G + head
    uint32_t qf[kNt][kD / 16][2];
    float qs[kNt][2];  // logit factor of columns 2 q4, 2 q4 + 1
    int tq[kNt][2];    // their positions (INT_MIN: no row)
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) {
      const int r = c.chunk * kNq + 8 * nt + g;
      const bool live = r < rows;
      const int tau = live ? r / G : 0, h = c.kvh * G + (live ? r % G : 0);
      const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q.ptr) + ((int64_t)c.b * a.T + tau) * a.q.row_stride +
                            (int64_t)h * a.q.head_stride;
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
          // dims 0, 2 and 1, 3 of each four, as the codes of a word come out
          qf[nt][2 * i][0] = __byte_perm(u.x, u.y, 0x5410);
          qf[nt][2 * i][1] = __byte_perm(u.x, u.y, 0x7632);
          qf[nt][2 * i + 1][0] = __byte_perm(u.z, u.w, 0x5410);
          qf[nt][2 * i + 1][1] = __byte_perm(u.z, u.w, 0x7632);
        }
        // column c's factor sits in lanes 4 c .. 4 c + 3
        qs[nt][0] = kCodeFactor * a.scale * __shfl_sync(0xffffffffu, up, 8 * q4);
        qs[nt][1] = kCodeFactor * a.scale * __shfl_sync(0xffffffffu, up, 8 * q4 + 4);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rc = c.chunk * kNq + 8 * nt + 2 * q4 + e;
        tq[nt][e] = rc < rows ? c.s.len - a.T + rc / G : INT32_MIN;
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

    for (; c.t < c.t_end; ++c.t, ++done) {
      const int st = done % L::kStages;
      lost = __any_sync(0xffffffffu, !sm100::mbar_wait(&full[st], (done / L::kStages) & 1, abort));
      if (lost) break;
      if (!((none >> st) & 1)) {
        const int key0 = c.t * kTile;
        const uint32_t sk = sm100::smem_u32(ring + st * L::kStage), sv = sk + L::kOperand;
        // not seen by every row: keys after the first query, before the last query's window
        const bool edge = key0 + kTile - 1 > c.s.len - a.T || (a.window > 0 && key0 < c.s.len - a.window);
        auto seen = [&](int key, int tcol) { return key <= tcol && (a.window == 0 || key > tcol - a.window); };

        // S^T = K Q^T, in two chains of MMAs
        float z[kNt][4], z2[kNt][4];
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[nt][e] = z2[nt][e] = 0.f;
        uint32_t top_k[2] = {0, 0};  // largest magnitudes of the codes of keys g, g + 8
        if (!kFp8) {
          const int r = lane & 15;
#pragma unroll
          for (int kk = 0; kk < kD / 16; ++kk) {
            uint32_t af[4];
            const int ch = 2 * (kk & 3) + (lane >> 4);
            ldsm4(sk + (kk >> 2) * kTile * 128 + r * 128 + ((ch ^ (r & 7)) << 4), af);
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) mma16816<kMmaBf16>((kk & 1) ? z2[nt] : z[nt], af, qf[nt][kk][0], qf[nt][kk][1]);
          }
        } else {
          // 16 codes of keys g and g + 8 at a time: four MMA steps, whose dims
          // are 4 s .. 4 s + 3 of this lane's piece
#pragma unroll
          for (int i = 0; i < kD / 64; ++i) {
            uint4 w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = g + 8 * e;
              w[e] = lds128(sk + (kD == 128 ? r * 128 + (((2 * q4 + i) ^ (r & 7)) << 4) : r * 64 + ((q4 ^ ((r >> 1) & 3)) << 4)));
            }
            const uint32_t w0[4] = {w[0].x, w[0].y, w[0].z, w[0].w}, w1[4] = {w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
            for (int sp = 0; sp < 4; ++sp) {
              const uint32_t af[4] = {codes02_to_f16x2(w0[sp], top_k[0]), codes02_to_f16x2(w1[sp], top_k[1]),
                                      codes13_to_f16x2(w0[sp], top_k[0]), codes13_to_f16x2(w1[sp], top_k[1])};
#pragma unroll
              for (int nt = 0; nt < kNt; ++nt)
                mma16816<false>((sp & 1) ? z2[nt] : z[nt], af, qf[nt][4 * i + sp][0], qf[nt][4 * i + sp][1]);
            }
          }
        }
        // of keys g, g + 8: K scale, log2 of the V scale (codes come as 2^-8 of
        // their value) and 2^ of its negative
        float ks[2] = {1.f, 1.f}, lv[2] = {0.f, 0.f}, rv[2] = {1.f, 1.f};
        if (kFp8) {
          const float* sc = scales + st * 2 * kTile + g;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            ks[e] = sc[8 * e];
            const float x = sc[kTile + 8 * e];
            lv[e] = x != x ? x : fminf(fmaxf(lg2(x), kMinLogScale), kMaxLogScale) + kCodeExp;
            rv[e] = ex2(-lv[e]);
          }
          const bool nan_k = has_nan_code(top_k[0]) || has_nan_code(top_k[1]);
          if (__any_sync(0xffffffffu, nan_k)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              int bad = has_nan_code(top_k[e]);
              bad |= __shfl_xor_sync(0xffffffffu, bad, 1);
              bad |= __shfl_xor_sync(0xffffffffu, bad, 2);
              if (bad) ks[e] = __int_as_float(0x7FC00000);
            }
          }
        }
        float u[kNt][4];  // base-2 logit plus the value's log-scale; masked ones -inf
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float zz = (z[nt][e] + z2[nt][e]) * (kFp8 ? qs[nt][e & 1] * ks[e >> 1] : qs[nt][e & 1]);
            u[nt][e] = kFp8 ? zz + lv[e >> 1] : zz;
            if (edge && !seen(key0 + g + 8 * (e >> 1), tq[nt][e & 1])) u[nt][e] = -INFINITY;
            over |= u[nt][e] > m[nt][e & 1] + kLazy;
          }
        // The running maxima move only when a logit exceeds them by kLazy
        // (weights then stay below 2^kLazy): mostly one vote instead of
        // shuffles over the 16 keys and a pass over O.
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt) {
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float v = fmaxf(u[nt][e], u[nt][e + 2]);
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
              alpha[e] = 1.f;
              if (v > m[nt][e]) {
                alpha[e] = ex2(m[nt][e] - v);  // 0 from -inf
                m[nt][e] = v;
              }
              l[nt][e] *= alpha[e];
            }
#pragma unroll
            for (int mt = 0; mt < kD / 16; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[mt][nt][e] *= alpha[e & 1];
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
            if (!kFp8) l[nt][e & 1] += p[e];
            else if (!edge || u[nt][e] != -INFINITY) l[nt][e & 1] = fmaf(p[e], rv[e >> 1], l[nt][e & 1]);
          }
          pf[nt][0] = transpose8x8(pack2<kMmaBf16>(p[0], p[1]));
          pf[nt][1] = transpose8x8(pack2<kMmaBf16>(p[2], p[3]));
        }

        // O^T += V^T P^T.  Rows g, g + 8 of m-tile mt are dims dim_of(mt, 0),
        // dim_of(mt, 1).
        bool odd = false;  // values that are not finite, taken out
        if (!kFp8) {
          const int i = lane >> 3, r = (lane & 7) + 8 * (i >> 1);
#pragma unroll
          for (int mt = 0; mt < kD / 16; ++mt) {
            uint32_t af[4];
            const int ch = 2 * (mt & 3) + (i & 1);
            ldsm4t(sv + (mt >> 2) * kTile * 128 + r * 128 + ((ch ^ (r & 7)) << 4), af);
            if (edge) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t bad = odd_halves<kMmaBf16>(af[e]);
                odd |= bad != 0;
                af[e] &= ~bad;
              }
            }
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) mma16816<kMmaBf16>(o[mt][nt], af, pf[nt][0], pf[nt][1]);
          }
        } else {
          // kD/8 codes of keys 2 q4, 2 q4 + 1, + 8, + 9 from dim kD/8 * g on
          uint32_t w[4][kD / 32], top_v = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 2 * q4 + (e & 1) + 8 * (e >> 1);
            if (kD == 128) {
              const uint4 x = lds128(sv + r * 128 + ((g ^ (r & 7)) << 4));
              w[e][0] = x.x;
              w[e][1] = x.y;
              w[e][kD / 32 - 2] = x.z;
              w[e][kD / 32 - 1] = x.w;
            } else {
              const uint2 x = lds64(sv + r * 64 + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + (g & 1) * 8);
              w[e][0] = x.x;
              w[e][1] = x.y;
            }
          }
#pragma unroll
          for (int mt = 0; mt < kD / 16; ++mt) {
            // dims 2 mt, 2 mt + 1 of the piece, of two keys each
            const uint32_t sel = (mt & 1) ? 0x7632u : 0x5410u;
            const uint32_t lo = __byte_perm(w[0][mt / 2], w[1][mt / 2], sel), hi = __byte_perm(w[2][mt / 2], w[3][mt / 2], sel);
            const uint32_t af[4] = {codes02_to_f16x2(lo, top_v), codes13_to_f16x2(lo, top_v), codes02_to_f16x2(hi, top_v),
                                    codes13_to_f16x2(hi, top_v)};
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) mma16816<false>(o[mt][nt], af, pf[nt][0], pf[nt][1]);
          }
          odd = has_nan_code(top_v);
        }
        if (__any_sync(0xffffffffu, odd)) {
          // give each value that is not finite to the rows that see it
#pragma unroll
          for (int mt = 0; mt < kD / 16; ++mt)
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2) {
              const int dim = kFp8 ? kD / 8 * g + 2 * mt + e2 : 16 * mt + g + 8 * e2;
#pragma unroll 1
              for (int k = 0; k < kTile; ++k) {
                const uint8_t* vs = ring + st * L::kStage + L::kOperand;
                float v;
                if (!kFp8)
                  v = unpack2<kBf16>(*reinterpret_cast<const uint16_t*>(
                      vs + (dim >> 6) * kTile * 128 + k * 128 + ((((dim >> 3) & 7) ^ (k & 7)) << 4) + (dim & 7) * 2)).x;
                else
                  v = e4m3_to_f32(vs[kD == 128 ? k * 128 + (((dim >> 4) ^ (k & 7)) << 4) + (dim & 15)
                                               : k * 64 + (((dim >> 4) ^ ((k >> 1) & 3)) << 4) + (dim & 15)]);
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
      }
      __syncwarp();  // every lane has read the stage
      load_next();
    }
    if (lost) break;

    // ---- the item's result: sums over the keys of a column sit in its 8 lanes
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) {
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = l[nt][e];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        l[nt][e] = v;
        f[e] = 1.f;
        if (single) {
          const int r = c.chunk * kNq + 8 * nt + 2 * q4 + e;
          if (a.sink && r < rows && m[nt][e] != -INFINITY) v += ex2(a.sink[c.kvh * G + r % G] * kLog2e - m[nt][e]);
          f[e] = v != 0.f ? 1.f / v : 0.f;
        }
      }
      // Pieces of rows: a lane takes column 2 q4 + (g & 1) of itself and its
      // neighbour lane ^ 4 (16-bit cache: two dims from 16 mt + 8 e2 + (g & 6)),
      // or both columns, four dims each (FP8 cache: from kD/8 g + 4 j).
      auto put = [&](int col, int dim, const float* x, int n) {
        const int r = c.chunk * kNq + 8 * nt + col;
        if (r >= rows) return;
        const int tau = r / G, h = c.kvh * G + r - tau * G;
        if (single) {
          uint16_t* dst = reinterpret_cast<uint16_t*>(a.out.ptr) + ((int64_t)c.b * a.T + tau) * a.out.row_stride +
                          (int64_t)h * a.out.head_stride + dim;
          if (n == 2) *reinterpret_cast<uint32_t*>(dst) = pack2<kBf16>(x[0], x[1]);
          else *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<kBf16>(x[0], x[1]), pack2<kBf16>(x[2], x[3]));
        } else {
          const int64_t slot = (((int64_t)c.b * a.max_splits + c.split) * a.T + tau) * a.n_heads + h;
          float* dst = a.part_o + slot * kD + dim;
          if (n == 2) *reinterpret_cast<float2*>(dst) = make_float2(x[0], x[1]);
          else *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
        }
      };
      if (!kFp8) {
        const bool hi = g & 1;
#pragma unroll
        for (int mt = 0; mt < kD / 16; ++mt)
#pragma unroll
          for (int e2 = 0; e2 < 2; ++e2) {
            const float x0 = o[mt][nt][2 * e2] * f[0], x1 = o[mt][nt][2 * e2 + 1] * f[1];
            const float y = __shfl_xor_sync(0xffffffffu, hi ? x0 : x1, 4);
            const float x[2] = {hi ? y : x0, hi ? x1 : y};
            put(2 * q4 + hi, 16 * mt + 8 * e2 + (g & 6), x, 2);
          }
      } else {
#pragma unroll
        for (int j = 0; j < kD / 32; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x[4] = {o[2 * j][nt][e] * f[e], o[2 * j][nt][2 + e] * f[e], o[2 * j + 1][nt][e] * f[e],
                                o[2 * j + 1][nt][2 + e] * f[e]};
            put(2 * q4 + e, kD / 8 * g + 4 * j, x, 4);
          }
      }
      if (!single && g == 0) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = c.chunk * kNq + 8 * nt + 2 * q4 + e;
          if (r < rows) {
            const int tau = r / G, h = c.kvh * G + r - tau * G;
            a.part_ml[(((int64_t)c.b * a.max_splits + c.split) * a.T + tau) * a.n_heads + h] = make_float2(m[nt][e], l[nt][e]);
          }
        }
      }
    }
  }
  if (lost) {
    // a wait gave up: copies in flight land before the CTA goes
    for (; done < issued; ++done) {
      const uint64_t t0 = sm100::globaltimer();
      while (!sm100::mbar_try_wait(&full[done % L::kStages], (done / L::kStages) & 1) && sm100::globaltimer() - t0 < sm100::kWaitNs) {
      }
    }
    if (lane == 0) raise_err(a.err, CSA_DEV_ERR_TIMEOUT);
  }
  pdl_trigger();
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
  const float mr = M == -INFINITY ? 0.f : M;
#pragma unroll 4
  for (int s = warp; s < n; s += 8) {
    const float2 ml = a.part_ml[slot + s * stride];
    const float f = ex2(ml.x - mr);
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
  using L = Layout<kFp8, kD, kNq>;
  auto fn = gqa_decode_kernel<kBf16, kFp8, kD, kNq>;
  cudaError_t e = set_max_smem(reinterpret_cast<const void*>(fn), L::kSmem);
  if (e != cudaSuccess) return e;
  const int grid = (int)(items < sm_count() ? items : sm_count());
  e = launch_pdl(fn, dim3(grid), dim3(32 * L::kWarps), L::kSmem, st, mk, mv, a);
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
  // [pages * heads][halves of a row][page slots][64 dims (a whole FP8 row)]
  const uint32_t inner = f8 ? (uint32_t)p.d : 64u, halves = (uint32_t)p.d / inner;
  const uint64_t dims[4] = {inner, (uint64_t)p.page, halves, (uint64_t)cache.n_pages * p.n_kv_heads};
  const uint64_t str[3] = {p.d * es, inner * es, (uint64_t)p.page * p.d * es};
  const uint32_t box[4] = {inner, (uint32_t)kTile, halves, 1};
  const CUtensorMapSwizzle sw = f8 && p.d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  const CUtensorMapDataType dt = f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!encode_tensor_map(&mk, dt, 4, cache.k, dims, str, box, sw) ||
      !encode_tensor_map(&mv, dt, 4, cache.v, dims, str, box, sw))
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
