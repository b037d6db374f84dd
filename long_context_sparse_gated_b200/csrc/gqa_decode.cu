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
// kNq of its T * G query rows.  Splits are a rule on the sequence's own length
// (split_blocks), so a query's bits do not depend on its batch.  A team of
// four warps takes an item, its tiles in turn, and joins the four results in
// shared memory; teams take items t, t + teams, ..., the largest splits first,
// and leave an item's (m, l, O) in fp32 for gqa_join_kernel, or the result where
// the sequence has one split.  (A warp needs some 0.9 us a tile when it is
// alone, so one warp an item makes short contexts slow: 15.4 us for 777 keys;
// all eight warps of a CTA an item costs long ones their join.)
//
//   tiles    16 keys and values, always inside one page, loaded by TMA.  A warp
//            owns a ring of stages and refills each as soon as it has read it; the
//            loading side runs ahead over item borders, so the stream of
//            tiles never drains, and there is no producer to wait for.  With
//            fewer items than teams, fewer teams have deeper rings.
//   product  S^T[keys, rows] = K Q^T, P^T = exp2(S^T - m), O^T[d, rows] += V^T P^T
//            by mma.sync.  With the keys as M, 8 query rows fill an MMA (with
//            rows as M the usual groups of 8 would waste half of it).
//   rows     8, 16 or 32 an item, so that several tokens and large groups do not
//            read the cache twice. With 32 the sums leave no registers for the
//            queries, whose fragments and positions wait in shared memory.  40
//            sequences of up to 1152 keys, 4 tokens, 40 / 8 heads: 43 us, in items
//            of 16 rows 48; 8 of up to 20000, 64 / 8 heads: 110 and 122, FP8 119 and
//            151.  (Two warps a scheduler then wait for their own instructions, some
//            4000 clocks a tile: 110 us are 62% of the copy rate.)
//
// 16-bit cache.  m16n8k16; K by ldmatrix, V by ldmatrix.trans, P^T rounded to
// 16 bits and transposed in registers by movmatrix.
//
// FP8 cache.  E4M3 codes become FP16 in registers by the packed conversion
// instruction (moving the bits by hand took 163 us instead of 129 for 24
// sequences of up to 32K keys, m16n8k32 on the codes and weights split into E5M2 pieces
// 263 to 358; now 134).  The dims of a 16-byte piece
// are dealt to MMA steps in an order that Q's fragments share, so no shuffles
// are needed.  A query row is brought into FP16 by a power of two of its own
// (largest magnitude in [2^14, 2^15); what is 2^29 below that loses bits that do
// not show in fp32).  The value's scale s_j joins the weight: w_j = exp2(z_j +
// log2 s_j - M) with M following the running maximum of that sum, so weights
// stay in (0, 2^15] whatever the scales are, and the denominator sums w_j / s_j.
// Value scales are read as within 2^-90 .. 2^90.  (Weights below fp32's 2^-126 are lost to
// the denominator: with scales 2^90 apart at most those are of keys whose exp(z_j) is
// below 2^-32 of the largest.  Looking for them took 3% in every call.)
//
// Rounding.  Weights are rounded to 16 bits, since that is what the product
// takes: to BF16 for a BF16 cache (2^-8 of themselves), else to FP16 (2^-11, where
// FP16 has its full precision: down to 2^-25 of the largest weight, which is 2^11
// at least; below that by up to 2^-36 of the largest).  The maximum is followed
// closer for that than for BF16 (by 2^4 instead of 2^8).  Sums and partial outputs
// are fp32.
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

constexpr int kTile = 16;   // keys per stage
constexpr int kBlock = 32;  // keys: splits begin at multiples of it
constexpr int kMaxStages = 16;
constexpr float kLog2e = 1.4426950408889634f;
// Weights are 2^(z - m) with m = a running maximum - kTop, raised when a logit
// exceeds the maximum by kLazy (base-2 units).  FP16 holds weights from 2^-14
// (with fewer bits from 2^-24) to 2^16, so the largest are put near its top.  BF16
// weights begin at 2^-14: sums of the type's largest values stay finite while the
// weights add up to less than 2^14 of the largest, and products with its smallest
// are still well above fp32's last bit.
template <bool kBf16>
struct Weights {
  static constexpr float kTop = kBf16 ? -14.f : 11.f, kLazy = kBf16 ? 8.f : 4.f;
};
constexpr float kNone = -3.0e38f;  // a running maximum before the first key
struct Edge { static constexpr bool value = true; };
struct Whole { static constexpr bool value = false; };
constexpr float kMinLogScale = -90.f, kMaxLogScale = 90.f;

// Blocks per split for a sequence of n blocks: 8, 16 or 32 blocks, so that
// there are about 12 splits (256 to 1024 keys), and 64 for more than 64K keys.
// Measured (32 mixed up to 16K / 4 of 128K / 24 FP8 up to 32K / 16 x 4 drafted
// tokens / 777 keys alone, us, one call from cold caches): this 172 / 342 / 143 / 20 /
// 14; 4 to 16 blocks and 32 splits 180 / 371 / 152 / 25 / 14; never 64 blocks 172 / 362 /
// 141 / 20 / 14; 4 blocks at least 174 / 342 / 143 / 25 / 14; 16 at least 169 / 342 / 141 /
// 20 / 16.
constexpr int kMinSplit = 8, kMidSplit = 32, kMaxSplit = 64, kSplits = 12, kLong = 2048;
__host__ __device__ inline int split_blocks(int n) {
  if (n > kLong) return kMaxSplit;
  int c = kMinSplit;
  while (c < kMidSplit && c * kSplits < n) c *= 2;
  return c;
}
__host__ __device__ inline int n_splits(int n) {
  const int c = split_blocks(n);
  return n <= c ? 1 : (n + c - 1) / c;  // a sequence without keys has one empty split
}
// The most splits that any sequence of up to n blocks has.
inline int most_splits(int n) {
  int most = n_splits(n);
  for (int top : {kMinSplit * kSplits, 2 * kMinSplit * kSplits, kLong})  // the longest of their kind
    if (top < n && most < n_splits(top)) most = n_splits(top);
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
  int B, T, n_max, n_heads, n_kv, kv_shift, page, page_shift, window, max_splits;  // kv_shift: log2 n_kv, or -1
  float scale;  // softmax_scale * log2(e)
  int32_t* err;
};

// The keys [lo, len) that some query of the sequence sees, and the n blocks
// from block b0 on that hold them.
struct Span {
  int len, lo, b0, n;
};
__device__ __forceinline__ Span span_of(const DecodeArgs& a, int len) {
  Span s;
  s.len = max(0, min(len, a.n_max));
  s.lo = a.window > 0 ? max(0, s.len - a.T - a.window + 1) : 0;
  s.b0 = s.lo / kBlock;
  s.n = s.len > s.lo ? (s.len + kBlock - 1) / kBlock - s.b0 : 0;
  return s;
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
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// Four E4M3 codes -> FP16, bytes 0, 1 and 2, 3.
__device__ __forceinline__ void cvt_codes(uint32_t v, uint32_t& a, uint32_t& b) {
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(v));
}

constexpr int kTeam = 4;  // warps
constexpr int kMaxB = 1024, kNear = 256;

template <bool kFp8, int kD, int kNq>
struct Layout {
  // 8 query rows: three teams of up to 168 registers a thread, or four of 128 for
  // an FP8 cache, whose work is in the instructions (142 us with three, 128 with
  // four); 16 rows: two of up to 255
  static constexpr int kTeams = kNq == 8 ? (kFp8 ? 4 : 3) : 2, kWarps = kTeam * kTeams;
  static constexpr int kRowBytes = kFp8 ? kD : 2 * kD;
  static constexpr int kOperand = kTile * kRowBytes;       // K or V of a tile
  static constexpr int kStage = 2 * kOperand;
  static constexpr int kScales = kFp8 ? 2 * kTile * 4 : 0;  // its scales, K then V
  static constexpr int kSlots = kFp8 ? (kD == 128 ? 32 : 64) : (kD == 128 ? 24 : 48);  // stages of all warps
  static constexpr int kJoin = 2 * kD * 8 * 4;              // a team's buffer: two warps' 8 rows
  static constexpr size_t kSmem = 1024 + (size_t)kSlots * (kStage + kScales) + kTeams * kJoin;
  static_assert(kSmem + 8192 + 72 * kTeams * kNq <= 232448, "shared memory of a CTA");
};

// An item and the stretch of keys in it that has to be read.
struct Item {
  int at;                  // in the order of sequences
  int b, kvh, split, chunk;  // chunk: which kNq of the query rows
  int t, t_end;            // this warp's tiles: t, t + kTeam, ... of the sequence's
  Span s;
};

template <bool kBf16, bool kFp8, int kD, int kNq>
__global__ void __launch_bounds__(32 * Layout<kFp8, kD, kNq>::kWarps, 1)
    gqa_decode_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                      const __grid_constant__ DecodeArgs a) {
  using L = Layout<kFp8, kD, kNq>;
  constexpr int kNt = kNq / 8;
  constexpr bool kShared = kNq == 32;  // the queries' fragments in shared memory
  static_assert(!kShared || kNt == kTeam, "a warp brings one n-tile's");
  constexpr bool kMmaBf16 = kBf16 && !kFp8;
  constexpr float kTop = Weights<kMmaBf16>::kTop, kOver = kTop + Weights<kMmaBf16>::kLazy;
  extern __shared__ uint8_t raw[];
  __shared__ uint64_t full_bar[L::kSlots];
  __shared__ int first_item[kMaxB + 1];  // items before the i-th sequence of the order
  __shared__ uint16_t order[kMaxB];      // sequences, those with the largest splits first
  __shared__ float red_m[L::kTeams][2][kTeam][kNq], red_l[L::kTeams][2][kTeam][kNq];
  __shared__ float red_q[L::kTeams][kShared ? kNq : 1];  // logit factors of the rows
  __shared__ int red_t[L::kTeams][kShared ? kNq : 1];    // and their positions
  __shared__ int near_lens[kNear];       // lengths of the first sequences
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* all = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);

  for (int s = threadIdx.x; s < L::kSlots; s += blockDim.x) sm100::mbar_init(&full_bar[s], 1);
  sm100::fence_mbar_init();
  if (threadIdx.x == 0) {
    abort_flag = 0;
    sm100::prefetch_tmap(&map_k);
    sm100::prefetch_tmap(&map_v);
  }
  pdl_wait();
  pdl_trigger();  // gqa_join_kernel may take its place; it waits for this kernel's end
  const int G = a.n_heads / a.n_kv, rows = a.T * G;
  const int chunks = (rows + kNq - 1) / kNq;
  // ---- the order of the sequences and their items.  (The ring's memory holds
  // the counts until the first loads.)
  int* counts = reinterpret_cast<int*>(all);
  for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
    const int len = a.lens[b], n = span_of(a, len).n;
    counts[b] = n_splits(n) * 128 + split_blocks(n);
    if (b < kNear) near_lens[b] = len;
    if (blockIdx.x == 0 && len > a.n_max) raise_err(a.err, CSA_DEV_ERR_RANGE);
  }
  __syncthreads();
  if (warp == 0) {
    int items = 0, place = 0;
#pragma unroll 1
    for (int c = kMaxSplit; c >= kMinSplit; c /= 2)
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int x = b0 + lane < a.B ? counts[b0 + lane] : 0;
        const bool mine = (x & 127) == c;
        const unsigned who = __ballot_sync(0xffffffffu, mine);
        if (!who) continue;
        const int n = mine ? (x >> 7) * a.n_kv * chunks : 0;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const int y = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += y;
        }
        if (mine) {
          const int i = place + __popc(who & ((1u << lane) - 1));
          first_item[i] = items + sum - n;
          order[i] = (uint16_t)(b0 + lane);
        }
        items += __shfl_sync(0xffffffffu, sum, 31);
        place += __popc(who);
      }
    if (lane == 0) first_item[a.B] = items;
    sm100::fence_proxy_async_smem();  // the counts' place is loaded over
  }
  __syncthreads();
  const int total = first_item[a.B];
  // teams with work, numbered across the SMs first
  const int team = warp / kTeam, w4 = warp % kTeam;
  const int teams = max(1, min(L::kTeams, (total - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x));
  const int item0 = team * gridDim.x + blockIdx.x, step = L::kTeams * gridDim.x;
  if (team >= teams) return;
  // ---- this warp's ring
  const int n_st = min(kMaxStages, L::kSlots / (kTeam * teams));
  uint8_t* ring = all + warp * n_st * L::kStage;
  float* scales = reinterpret_cast<float*>(all + L::kSlots * L::kStage + warp * n_st * L::kScales);
  float4* join = reinterpret_cast<float4*>(all + L::kSlots * (L::kStage + L::kScales) + team * L::kJoin);
  uint64_t* full = full_bar + warp * n_st;
  const uint32_t ring_u32 = sm100::smem_u32(ring), scales_u32 = sm100::smem_u32(scales), join_u32 = sm100::smem_u32(join), full_u32 = sm100::smem_u32(full);
  volatile int* abort = &abort_flag;

  auto enter = [&](Item& c, int item) {
    while (item >= first_item[c.at + 1]) ++c.at;
    c.b = order[c.at];
    const int in_b = item - first_item[c.at], x = chunks == 1 ? in_b : in_b / chunks;
    c.chunk = in_b - x * chunks;
    c.split = a.kv_shift >= 0 ? x >> a.kv_shift : x / a.n_kv;
    c.kvh = x - c.split * a.n_kv;
    c.s = span_of(a, c.b < kNear ? near_lens[c.b] : a.lens[c.b]);
    const int n = split_blocks(c.s.n), b0 = c.s.b0 + c.split * n;
    c.t = max(b0 * kBlock, c.s.lo) / kTile + w4;
    c.t_end = c.s.n == 0 ? 0 : (min((b0 + n) * kBlock, c.s.len) + kTile - 1) / kTile;
  };

  // ---- loading side: page ids 32 at a time, then tiles as long as stages are
  // free
  Item ld;
  ld.at = 0;
  ld.t = ld.t_end = 0;
  int next = item0;           // the next item to load
  uint32_t issued = 0, done = 0;
  int st_ld = 0;              // issued % n_st
  int ids = -1, group = -1;   // this lane's page id of 32-page group `group`
  uint32_t none = 0;          // stages whose tile belongs to no page (nothing is loaded)
  auto fill = [&]() {
    while (issued - done < (uint32_t)n_st) {
      if (ld.t >= ld.t_end) {
        if (next >= total) return;
        enter(ld, next);
        next += step;
        group = -1;
        continue;
      }
      const int key = ld.t * kTile, p = key >> a.page_shift;
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
      const int st = st_ld;
      none = id >= 0 ? none & ~(1u << st) : none | (1u << st);
      if (lane == 0) {
        const uint32_t bar = full_u32 + 8 * st;
        if (id >= 0) {
          expect_tx(bar, L::kStage + L::kScales);
          const uint32_t dst = ring_u32 + st * L::kStage;
          const int slot = key & (a.page - 1), head_page = id * a.n_kv + ld.kvh;
          tma_load_4d(dst, &map_k, bar, 0, slot, 0, head_page);
          tma_load_4d(dst + L::kOperand, &map_v, bar, 0, slot, 0, head_page);
          if (kFp8) {
            const int64_t at = ((int64_t)head_page << a.page_shift) + slot;
            const uint32_t sc = scales_u32 + st * L::kScales;
            bulk_load(sc, a.k_scale + at, kTile * 4, bar);
            bulk_load(sc + kTile * 4, a.v_scale + at, kTile * 4, bar);
          }
        } else {
          sm100::mbar_arrive(&full[st]);
        }
      }
      ld.t += kTeam;
      ++issued;
      if (++st_ld == n_st) st_ld = 0;
    }
  };
  fill();

  // ---- computing side
  const int g = lane >> 2, q4 = lane & 3;
  bool lost = false;
  int st = 0;            // done % n_st
  uint32_t phase = 0;    // of the stage
  int par = 0;
  Item c;
  c.at = 0;
  for (int item = item0; item < total; item += step, par ^= 1) {
    enter(c, item);
    const bool single = c.s.n <= split_blocks(c.s.n);

    // query fragments: B operand, column g of n-tile nt is query row
    // chunk * kNq + 8 nt + g = tau * G + head
    uint32_t qf[kShared ? 1 : kNt][kD / 8];
    float qs[kNt][2];  // logit factor of columns 2 q4, 2 q4 + 1
    int tq[kShared ? 1 : kNt][2];  // their positions (INT_MIN: no row)
#pragma unroll
    for (int x = 0; x < (kShared ? 1 : kNt); ++x) {
      const int nt = kShared ? w4 : x;
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
            qf[x][2 * kk + e] = live ? *reinterpret_cast<const uint32_t*>(src + 16 * kk + 8 * e + 2 * q4) : 0u;
        if (!kShared) qs[x][0] = qs[x][1] = a.scale;
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
          qf[x][4 * i] = u.x;
          qf[x][4 * i + 1] = u.y;
          qf[x][4 * i + 2] = u.z;
          qf[x][4 * i + 3] = u.w;
        }
        // column c's factor sits in lanes 4 c .. 4 c + 3
        if (kShared) {
          if (q4 == 0) red_q[team][kShared ? 8 * nt + g : 0] = a.scale * up;
        } else {
          qs[x][0] = a.scale * __shfl_sync(0xffffffffu, up, 8 * q4);
          qs[x][1] = a.scale * __shfl_sync(0xffffffffu, up, 8 * q4 + 4);
        }
      }
    }
    auto position = [&](int r) { return r < rows ? c.s.len - a.T + r / G : INT32_MIN; };
    if (kShared) {
      if (q4 == 0) red_t[team][kShared ? 8 * w4 + g : 0] = position(c.chunk * kNq + 8 * w4 + g);
      sm100::named_bar_sync(1 + team, 32 * kTeam);  // the last item's join has read the place
#pragma unroll
      for (int j = 0; j < kD / 32; ++j)
        reinterpret_cast<uint4*>(join)[(w4 * kD / 32 + j) * 32 + lane] =
            make_uint4(qf[0][4 * j], qf[0][4 * j + 1], qf[0][4 * j + 2], qf[0][4 * j + 3]);
      sm100::named_bar_sync(1 + team, 32 * kTeam);
    }
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (kShared) qs[nt][e] = kFp8 ? red_q[team][kShared ? 8 * nt + 2 * q4 + e : 0] : a.scale;
        if (!kShared) tq[kShared ? 0 : nt][e] = position(c.chunk * kNq + 8 * nt + 2 * q4 + e);
      }
    }

    // the queries' fragments 4 j .. 4 j + 3
    auto q_at = [&](int nt, int j, uint32_t (&b)[4]) {
      if (kShared) {
        const uint4 v = lds128(join_u32 + ((nt * kD / 32 + j) * 32 + lane) * 16);
        b[0] = v.x, b[1] = v.y, b[2] = v.z, b[3] = v.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = qf[kShared ? 0 : nt][4 * j + e];
      }
    };

    float m[kNt][2], l[kNt][2], o[kD / 16][kNt][4];
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) {
      m[nt][0] = m[nt][1] = kNone;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int mt = 0; mt < kD / 16; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
    }

    for (; c.t < c.t_end && !lost; c.t += kTeam) {
      lost = __any_sync(0xffffffffu, !sm100::mbar_wait(&full[st], phase, abort));
      if (lost) break;
      if (!((none >> st) & 1)) {
        const int key0 = c.t * kTile;
        const uint32_t sk = sm100::smem_u32(ring + st * L::kStage), sv = sk + L::kOperand;
        // some row does not see it as a whole: keys after the first query, or
        // before the last query's window
        const bool at_edge = key0 + kTile - 1 > c.s.len - a.T || (a.window > 0 && key0 < c.s.len - a.window);
        auto seen = [&](int k, int nt, int e) {  // the tile's k-th key by column e of an n-tile
          const int key = key0 + k, tcol = kShared ? red_t[team][kShared ? 8 * nt + 2 * q4 + e : 0] : tq[kShared ? 0 : nt][e];
          return key <= tcol && (a.window == 0 || key > tcol - a.window);
        };

        auto tile = [&](auto kind) {
        constexpr bool edge = decltype(kind)::value;
        // S^T = K Q^T (keys g, g + 8), in two chains of MMAs or more
        float z[kNt][4], z2[kNt][4];
        uint32_t qb[kNt][4];
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) z[nt][e] = z2[nt][e] = 0.f;
        if (!kFp8) {
          const int r = lane & 15;
#pragma unroll
          for (int kk = 0; kk < kD / 16; ++kk) {
            if (!(kk & 1)) {
#pragma unroll
              for (int nt = 0; nt < kNt; ++nt) q_at(nt, kk / 2, qb[nt]);
            }
            uint32_t af[4];
            const int ch = 2 * (kk & 3) + (lane >> 4);
            ldsm4(sk + (kk >> 2) * kTile * 128 + r * 128 + ((ch ^ (r & 7)) << 4), af);
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) 
              mma16816<kMmaBf16>((kk & 1) && !kShared ? z2[nt] : z[nt], af, qb[nt][2 * (kk & 1)], qb[nt][2 * (kk & 1) + 1]);
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
              if (!(sp & 1)) {
#pragma unroll
                for (int nt = 0; nt < kNt; ++nt) q_at(nt, 2 * i + sp / 2, qb[nt]);
              }
              uint32_t af[4];
              cvt_codes(w0[sp], af[0], af[2]);
              cvt_codes(w1[sp], af[1], af[3]);
#pragma unroll
              for (int nt = 0; nt < kNt; ++nt)
                mma16816<false>((sp & 1) && !kShared ? z2[nt] : z[nt], af, qb[nt][2 * (sp & 1)], qb[nt][2 * (sp & 1) + 1]);
            }
          }
        }
        // of keys g, g + 8: K scale, log2 of the V scale and 2^ of its negative
        float ks[2] = {1.f, 1.f}, lv[2] = {0.f, 0.f}, rv[2] = {1.f, 1.f};
        if (kFp8) {
          const float* sc = scales + st * 2 * kTile + g;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            ks[e] = sc[8 * e];
            const float x = sc[kTile + 8 * e];
            lv[e] = x < INFINITY ? fminf(fmaxf(lg2(x), kMinLogScale), kMaxLogScale) : NAN;
            rv[e] = ex2(-lv[e]);
          }
        }
        // base-2 logit plus the value's log-scale; masked ones -inf
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float& u = z[nt][e];
            if (!kShared) u += z2[nt][e];
            u = kFp8 ? fmaf(u, qs[nt][e & 1] * ks[e >> 1], lv[e >> 1]) : u * qs[nt][e & 1];
            if (edge && !seen(g + 8 * (e >> 1), nt, e & 1)) u = -INFINITY;
            over |= u - m[nt][e & 1] > kOver;
          }
        // The references move only when a logit exceeds its maximum by kLazy
        // (weights then stay below 2^kOver): mostly one vote instead of
        // shuffles over the keys and a pass over O.
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int nt = 0; nt < kNt; ++nt) {
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float v = fmaxf(z[nt][e], z[nt][e + 2]);
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
              // (where fp32's step is larger than kTop, to the maximum itself)
              v = kTop < 0.f ? __fadd_rd(v, -kTop) : __fadd_ru(v, -kTop);
              alpha[e] = 1.f;
              if (v > m[nt][e]) {
                alpha[e] = ex2(m[nt][e] - v);  // 0 from kNone
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
        // weights, transposed: B operand of the second product
        uint32_t pf[kNt][2];
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float u = z[nt][e];
            p[e] = ex2(u - m[nt][e & 1]);
            if (!kFp8) l[nt][e & 1] += p[e];
            else if (!edge || u != -INFINITY) l[nt][e & 1] = fmaf(p[e], rv[e >> 1], l[nt][e & 1]);
          }
          pf[nt][0] = transpose8x8(pack2<kMmaBf16>(p[0], p[1]));
          pf[nt][1] = transpose8x8(pack2<kMmaBf16>(p[2], p[3]));
        }

        // O^T += V^T P^T
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
          // kD/8 codes of keys 2 q4, 2 q4 + 1, + 8, + 9 from dim kD/8 * g on: rows
          // g and g + 8 of m-tile mt are dims 2 mt and 2 mt + 1 of that piece
          uint32_t w[4][kD / 32];
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
            const uint32_t sel = (mt & 1) ? 0x7362u : 0x5140u;
            uint32_t af[4];
            cvt_codes(__byte_perm(w[0][mt / 2], w[1][mt / 2], sel), af[0], af[1]);
            cvt_codes(__byte_perm(w[2][mt / 2], w[3][mt / 2], sel), af[2], af[3]);
            if (edge) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint32_t bad = odd_halves<false>(af[e]);
                odd |= bad != 0;
                af[e] &= ~bad;
              }
            }
#pragma unroll
            for (int nt = 0; nt < kNt; ++nt) mma16816<false>(o[mt][nt], af, pf[nt][0], pf[nt][1]);
          }
        }
        if (edge && __any_sync(0xffffffffu, odd)) {
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
                      if (seen(k, nt, e)) o[mt][nt][2 * e2 + e] += v;
                }
              }
            }
        }
        };
        if (at_edge) tile(Edge{});
        else tile(Whole{});
      }
      __syncwarp();  // every lane has read the stage
      ++done;
      if (++st == n_st) {
        st = 0;
        phase ^= 1;
      }
      fill();
    }

    // ---- the team's result (after a lost wait the barriers are still met):
    // sums over the keys of a column sit in its 8 lanes
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (m[nt][e] == kNone) m[nt][e] = -INFINITY;
        float v = l[nt][e];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        l[nt][e] = v;
        if (g == 0) {
          red_m[team][par][w4][8 * nt + 2 * q4 + e] = m[nt][e];
          red_l[team][par][w4][8 * nt + 2 * q4 + e] = v;
        }
      }
    sm100::named_bar_sync(1 + team, 32 * kTeam);
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) {
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = 8 * nt + 2 * q4 + e;
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kTeam; ++w) top = fmaxf(top, red_m[team][par][w][col]);
        const float mr = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int w = 0; w < kTeam; ++w) sum = fmaf(red_l[team][par][w][col], ex2(red_m[team][par][w][col] - mr), sum);
        f[e] = ex2(m[nt][e] - mr);
        m[nt][e] = top;
        l[nt][e] = sum;
      }
#pragma unroll
      for (int mt = 0; mt < kD / 16; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[mt][nt][e] *= f[e & 1];
      // warp nt takes an n-tile over: of the warps in turn from it, the third
      // and fourth give to it and the second, then the second to it, a lane's
      // registers to the same lane
      const int turn = (w4 - nt) & 3;
      if (nt > 0) sm100::named_bar_sync(1 + team, 32 * kTeam);  // the buffer is read
      auto give = [&](int buf) {
#pragma unroll
        for (int mt = 0; mt < kD / 16; ++mt)
          join[(buf * kD / 16 + mt) * 32 + lane] = make_float4(o[mt][nt][0], o[mt][nt][1], o[mt][nt][2], o[mt][nt][3]);
      };
      auto take = [&](int buf) {
#pragma unroll
        for (int mt = 0; mt < kD / 16; ++mt) {
          const float4 v = join[(buf * kD / 16 + mt) * 32 + lane];
          o[mt][nt][0] += v.x;
          o[mt][nt][1] += v.y;
          o[mt][nt][2] += v.z;
          o[mt][nt][3] += v.w;
        }
      };
      if (turn >= 2) give(turn & 1);
      sm100::named_bar_sync(1 + team, 32 * kTeam);
      if (turn < 2) take(turn);
      if (turn == 1) give(1);
      sm100::named_bar_sync(1 + team, 32 * kTeam);
      if (turn == 0) take(1);
    }
#pragma unroll
    for (int nt = 0; nt < kNt; ++nt) {
      if (w4 != nt) continue;
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        f[e] = 1.f;
        if (single) {
          const int r = c.chunk * kNq + 8 * nt + 2 * q4 + e;
          float v = l[nt][e];
          if (a.sink && r < rows && m[nt][e] != -INFINITY) v += ex2(a.sink[c.kvh * G + r % G] * kLog2e - m[nt][e]);
          f[e] = v != 0.f ? rcp(v) : 0.f;
        }
      }
      // Pieces of rows.  16-bit cache: a lane takes column 2 q4 + (g & 1) of itself
      // and its neighbour lane ^ 4, two dims from 16 mt + 8 e2 + (g & 6); FP8 cache:
      // both its columns, four dims each from kD/8 g + 4 j.
      int64_t at[2] = {-1, -1};  // of the columns' rows: in the output, or in the partial results
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = c.chunk * kNq + 8 * nt + 2 * q4 + (kFp8 ? e : g & 1);
        if (r < rows) {
          const int tau = r / G, h = c.kvh * G + r - tau * G;
          at[e] = single ? ((int64_t)c.b * a.T + tau) * a.out.row_stride + (int64_t)h * a.out.head_stride
                         : ((((int64_t)c.b * a.max_splits + c.split) * a.T + tau) * a.n_heads + h) * kD;
        }
        if (!kFp8) break;
      }
      if (!kFp8) {
        const bool hi = g & 1;
        uint16_t* dst = reinterpret_cast<uint16_t*>(a.out.ptr) + at[0] + (g & 6);
        float* part = a.part_o + at[0] + (g & 6);
#pragma unroll
        for (int mt = 0; mt < kD / 16; ++mt)
#pragma unroll
          for (int e2 = 0; e2 < 2; ++e2) {
            const float x0 = o[mt][nt][2 * e2] * f[0], x1 = o[mt][nt][2 * e2 + 1] * f[1];
            const float y = __shfl_xor_sync(0xffffffffu, hi ? x0 : x1, 4);
            o[mt][nt][2 * e2] = hi ? y : x0;
            o[mt][nt][2 * e2 + 1] = hi ? x1 : y;
          }
        if (at[0] >= 0) {
          if (single) {
#pragma unroll
            for (int mt = 0; mt < kD / 16; ++mt)
#pragma unroll
              for (int e2 = 0; e2 < 2; ++e2)
                *reinterpret_cast<uint32_t*>(dst + 16 * mt + 8 * e2) = pack2<kBf16>(o[mt][nt][2 * e2], o[mt][nt][2 * e2 + 1]);
          } else {
#pragma unroll
            for (int mt = 0; mt < kD / 16; ++mt)
#pragma unroll
              for (int e2 = 0; e2 < 2; ++e2)
                *reinterpret_cast<float2*>(part + 16 * mt + 8 * e2) = make_float2(o[mt][nt][2 * e2], o[mt][nt][2 * e2 + 1]);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (at[e] < 0) continue;
          uint16_t* dst = reinterpret_cast<uint16_t*>(a.out.ptr) + at[e] + kD / 8 * g;
          float* part = a.part_o + at[e] + kD / 8 * g;
#pragma unroll
          for (int j = 0; j < kD / 32; ++j) {
            const float4 x = make_float4(o[2 * j][nt][e] * f[e], o[2 * j][nt][2 + e] * f[e], o[2 * j + 1][nt][e] * f[e],
                                         o[2 * j + 1][nt][2 + e] * f[e]);
            if (single) *reinterpret_cast<uint2*>(dst + 4 * j) = make_uint2(pack2<kBf16>(x.x, x.y), pack2<kBf16>(x.z, x.w));
            else *reinterpret_cast<float4*>(part + 4 * j) = x;
          }
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
    // a wait gave up: copies in flight land before the warp goes
    for (; done < issued; ++done) {
      const uint64_t t0 = sm100::globaltimer();
      while (!sm100::mbar_try_wait(&full[st], phase) && sm100::globaltimer() - t0 < sm100::kWaitNs) {
      }
      if (++st == n_st) {
        st = 0;
        phase ^= 1;
      }
    }
    if (lane == 0) raise_err(a.err, CSA_DEV_ERR_TIMEOUT);
  }
}

// Joins the splits of one (query row, head): M = max m_s, o = sum_s
// exp2(m_s - M) O_s / (exp2(sink - M) + sum_s exp2(m_s - M) l_s).  Up to kFew
// splits are a warp's work, a CTA then takes eight heads (160 x 40 rows of few
// splits: 15.5 us with a CTA each).  More are a CTA's: warp w takes splits w, w + 8,
// ..., 32 at a time: a lane reads one split's (m, l) while the outputs are
// already on their way; the warps' results are then added in order.
constexpr int kFew = kSplits;  // at most a warp's lanes
template <bool kBf16, int kD>
__global__ void __launch_bounds__(256) gqa_join_kernel(const __grid_constant__ DecodeArgs a) {
  constexpr int kV = kD / 32;
  __shared__ float red[8][kD];
  __shared__ float red_l[8], red_m[8];
  const int row = blockIdx.x, b = row / a.T, tau = row % a.T;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (lens was complete before gqa_decode_kernel let this kernel begin)
  const int n = n_splits(span_of(a, a.lens[b]).n);
  // (the grid has eight heads a CTA where no sequence can have more than kFew)
  const bool few = n <= kFew;
  const int heads8 = a.max_splits <= kFew ? 8 * blockIdx.y : blockIdx.y;
  const int h = few ? heads8 + warp : heads8;
  pdl_wait();
  if (n == 1) return;  // finished by gqa_decode_kernel
  if (few && ((heads8 & 7) || h >= a.n_heads)) return;
  const float sink = a.sink ? a.sink[h] * kLog2e : -INFINITY;
  const int64_t stride = (int64_t)a.T * a.n_heads;
  const int64_t slot = (int64_t)b * a.max_splits * stride + tau * a.n_heads + h;
  float acc[kV] = {}, M = -INFINITY, den = 0.f;
  const int every = few ? 1 : 8;
  for (int s0 = few ? 0 : warp; s0 < n; s0 += 32 * every) {
    const int mine = s0 + every * lane, count = min(32, (n - s0 + every - 1) / every);
    const float2 ml = mine < n ? a.part_ml[slot + mine * stride] : make_float2(-INFINITY, 0.f);
    const float* src = a.part_o + (slot + s0 * stride) * kD + kV * lane;
    float buf[4][kV];
    auto load = [&](int i, float (&v)[kV]) {
      const float* p = src + every * i * stride * kD;
      if (kV == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        v[0] = x.x; v[1] = x.y; v[kV - 2] = x.z; v[kV - 1] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(p);
        v[0] = x.x; v[1] = x.y;
      }
    };
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < count) load(i, buf[i]);
    const float top = fmaxf(M, warp_max(ml.x)), mr = top == -INFINITY ? 0.f : top;
    const float down = ex2(M - mr);  // 0 from -inf
    M = top;
    const float f = ex2(ml.x - mr);
    den = den * down + warp_sum(ml.y * f);
#pragma unroll
    for (int j = 0; j < kV; ++j) acc[j] *= down;
    for (int i0 = 0; i0 < count; i0 += 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i0 + i < count) {
          const float w = __shfl_sync(0xffffffffu, f, i0 + i);
#pragma unroll
          for (int j = 0; j < kV; ++j) acc[j] = fmaf(buf[i][j], w, acc[j]);
          if (i0 + 4 + i < count) load(i0 + 4 + i, buf[i]);
        }
    }
  }
  if (few) {
    if (M != -INFINITY) den += ex2(sink - M);
    const float inv = den != 0.f ? rcp(den) : 0.f;
    uint16_t* dst = reinterpret_cast<uint16_t*>(a.out.ptr) + (int64_t)row * a.out.row_stride +
                    (int64_t)h * a.out.head_stride + kV * lane;
#pragma unroll
    for (int j = 0; j < kV; j += 2)
      *reinterpret_cast<uint32_t*>(dst + j) = pack2<kBf16>(acc[j] * inv, acc[j + 1] * inv);
    return;
  }
#pragma unroll
  for (int j = 0; j < kV; ++j) red[warp][kV * lane + j] = acc[j];
  if (lane == 0) {
    red_l[warp] = den;
    red_m[warp] = M;
  }
  __syncthreads();
  if (threadIdx.x < kD / 2) {
    float top = -INFINITY, x = 0.f, y = 0.f, l = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) top = fmaxf(top, red_m[w]);
    const float mr = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      const float f = ex2(red_m[w] - mr);
      x = fmaf(red[w][2 * threadIdx.x], f, x);
      y = fmaf(red[w][2 * threadIdx.x + 1], f, y);
      l = fmaf(red_l[w], f, l);
    }
    if (top != -INFINITY) l += ex2(sink - top);
    const float inv = l != 0.f ? rcp(l) : 0.f;
    uint16_t* dst = reinterpret_cast<uint16_t*>(a.out.ptr) + (int64_t)row * a.out.row_stride +
                    (int64_t)h * a.out.head_stride + 2 * threadIdx.x;
    *reinterpret_cast<uint32_t*>(dst) = pack2<kBf16>(x * inv, y * inv);
  }
}

int most_blocks(const gqa_params& p, int T, int n_max) {
  int64_t keys = n_max;
  if (p.window > 0 && keys > (int64_t)p.window + T - 1) keys = (int64_t)p.window + T - 1 + kBlock - 1;
  return (int)((keys + kBlock - 1) / kBlock);
}

// 8 or 16 query rows per item where they hold the whole group, else 32.
int rows_per_item(const gqa_params& p, int T) {
  const int rows = T * (p.n_heads / p.n_kv_heads);
  return rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
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
  const int heads = a.max_splits <= kFew ? (a.n_heads + 7) / 8 : a.n_heads;
  return launch_pdl(gqa_join_kernel<kBf16, kD>, dim3(a.B * a.T, heads), dim3(256), 0, st, a);
}

}  // namespace

int64_t gqa_decode_items(const gqa_params& p, int T, int n_max) {
  const int rows = T * (p.n_heads / p.n_kv_heads), nq = rows_per_item(p, T);
  return (int64_t)p.B * most_splits(most_blocks(p, T, n_max)) * p.n_kv_heads * ((rows + nq - 1) / nq);
}

size_t gqa_decode_workspace_bytes(const gqa_params& p, int T, int n_max) {
  const int s = most_splits(most_blocks(p, T, n_max));
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
  const int splits = most_splits(most_blocks(p, T, n_max));
  const int64_t slots = (int64_t)p.B * splits * T * p.n_heads;
  float* part_o = reinterpret_cast<float*>(ws);
  int shift = 0;
  while ((1 << shift) < p.page) ++shift;
  int kv_shift = 0;
  while ((1 << kv_shift) < p.n_kv_heads) ++kv_shift;
  if ((1 << kv_shift) != p.n_kv_heads) kv_shift = -1;
  const DecodeArgs a{q, out, cache.k_scale, cache.v_scale, table, table_cols, lens, sink, part_o,
                     splits > 1 ? reinterpret_cast<float2*>(part_o + slots * p.d) : nullptr, cache.n_pages, p.B, T,
                     n_max, p.n_heads, p.n_kv_heads, kv_shift, p.page, shift, p.window < (1 << 30) ? p.window : 0, splits, p.softmax_scale * kLog2e, err};
  const int nq = rows_per_item(p, T);
  const int64_t items = gqa_decode_items(p, T, n_max);
#define GQA_ROWS(BF, F8, D)                              \
  (nq == 8    ? launch<BF, F8, D, 8>(mk, mv, a, items, st)  \
   : nq == 16 ? launch<BF, F8, D, 16>(mk, mv, a, items, st) \
              : launch<BF, F8, D, 32>(mk, mv, a, items, st))
#define GQA_GO(BF, F8) (p.d == 128 ? GQA_ROWS(BF, F8, 128) : GQA_ROWS(BF, F8, 64))
  return bf ? (f8 ? GQA_GO(true, true) : GQA_GO(true, false)) : (f8 ? GQA_GO(false, true) : GQA_GO(false, false));
#undef GQA_GO
#undef GQA_ROWS
}

}  // namespace csa
