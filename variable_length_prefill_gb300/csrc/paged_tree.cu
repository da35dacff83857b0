// Attention of drafted tokens over a paged cache for sm_103a
// (include/paged_attn_tree.h has what is computed).
//
// The rows that read the same keys are stacked: a row tile is up to 128 of the
// (draft, query head of one KV head) pairs of a sequence, so that every key
// and value page is read once for all of them (more than 128 rows: once per
// row tile, from L2 for all but the first).  With r rows a key costs 4 D bytes
// and 4 D r operations; below about 280 rows the stream of pages bounds the
// call, and the design keeps bytes in flight while tcgen05 does the products.
//
// Both caches go to the tensor cores in the layout they have in memory:
//   keys    a page of one head is [D/8][16 tokens][8]: no-swizzle core
//           matrices of 8 tokens x 16 bytes.  One bulk copy per page; the two
//           8-token halves of a page's 16 tokens are 128 bytes apart, the
//           pages of a tile one page apart, so S = Q K^T runs as two products:
//           the first halves of all pages of the tile, then the second halves
//           (a fixed permutation of the tile's tokens).
//   values  a page is [D][16 tokens], 32 bytes a row: the K-major operand of one
//           16-token step of O += P V in the 32-byte swizzle, but for the
//           swizzle itself, which exchanges the two halves of the rows d with
//           bit 2 set.  One bulk copy per page, and a warp exchanges those
//           halves in shared memory.  (A tiled copy can do the swizzle, in
//           32-byte rows; it held the 64 x 4096 case to 322 us.)
// P is rounded to the cache type and written to TMEM over its scores, in token
// order, for the value product.  Weights are at most 2^8 of a row's running
// maximum, so fp16 would leave seven powers of two above them unused and lose
// those below 2^-25, which a long context has many of: fp16 weights, and with
// them the sums, are held 2^7 times as large.
//
// A persistent CTA per SM takes an equal share of all (sequence, KV head, row
// tile, key tile) units in that order (paged_walk.cuh), so a long sequence is
// split over many CTAs without the host knowing a length.  Row tiles that begin
// and end in one CTA are written to `out`; the others leave unnormalised partial
// results in the workspace for tree_join_kernel, which adds them in CTA order:
// results do not depend on timing.  Warps of a CTA:
//   key producer  walks the CTA's range, publishes its segments (a row tile's
//                 key tiles in this CTA) and streams their keys through a ring;
//   value producer  does the same for the values (a page's copy takes a warp 182
//                 clocks to issue, whatever its size; one warp for both took
//                 137 us instead of 113 for 64 x 4096 tokens at D = 64);
//   value warp    readies the values (below) and builds the table of ancestors
//                 (two warps for D = 256);
//   MMA issuer    one elected lane;
//   softmax       NG groups of four warps, one thread per row.
// For D <= 128 the two groups take the key tiles in turn, each with its own
// score buffer, running maximum, sum and accumulator (TMEM: S0 S1 O0 O1), so
// that one group's exponentials run under the other's products; they are added
// at the end of the segment.  For D = 256 one group works on both score buffers
// (two 256-column accumulators do not fit).
//
// Few rows would leave most softmax warps idle while the pages stream.  A tile
// of at most 64 (32) rows therefore holds each row twice (four times), and each
// copy takes the weights of its own half (quarter) of the keys, zeros for the
// others: all four warps share the exponentials, and the copies are added like
// the groups.  The softmax works on 32 keys at a time, twice over the scores
// (maximum, then weights), reading them from TMEM again: with all 128 scores of
// a row in registers the kernel spilled, and its code passed the instruction
// cache; a tile's softmax took 4000 clocks instead of 1300.
//
// A weight of 0 does not silence a NaN or an infinity in the values, so in a
// tile that holds drafts or slots past the last token, the warp that readies the
// values clears those slots, and the non-finite values of drafts; rows that see
// one get it back at the end, in a pass of its own over what was written
// (mend_non_finite).
//
// Measured (both kernels of a call, captured; 32 query and 8 KV heads, D = 128
// unless said): 64 x 4096 tokens, 16 drafts 186 us, 5.9 TB/s, 87 % of a copy's
// bandwidth (D = 64: 113 us, 71 %: the issue of 2 KB copies); one token each 179
// us (D = 64: 101).  3 sequences of up to 131071, 33 drafts, 40 query heads 216
// us, 5.3 TB/s: tiles of 128 rows take about 2000 clocks, scores, softmax and
// value product one behind the other, tensor pipe 40 % busy.
// 16 of up to 2112, 64 drafts, 4 KV heads, D = 256 50 us, tensor pipe 25 %
// busy: 1800 clocks a 64-key tile (1060 of products) and 20000 for a row tile's
// start and end.  4 x 128 tokens, 8 drafts 12.9 us, all latency.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "attn_varlen_device.cuh"
#include "packed_slice.h"
#include "paged_tree_internal.h"
#include "paged_walk.cuh"
#include "ptx.cuh"

namespace avp {
namespace {

constexpr int kMaxDevices = 64;
constexpr int kAncWords = kTreeMaxDrafts / 32;
constexpr int kAncStride = kAncWords + 1;  // words between rows of the ancestor table
constexpr int kMaskDepth = 8;              // key tiles whose page masks are kept
constexpr int kSegDepth = 4;               // published segments
constexpr int kStageCols = 32;             // columns of an output step

// A CTA's part of one row tile: key tiles [t0, t1) of nt.
struct Segment {
  int lo, n;    // packed rows of the sequence
  int len;      // tokens in the table (0 with too many drafts)
  int base;     // position of draft 0 (may be negative)
  int seq, g, mt;
  int t0, t1, nt;
  long long u;  // first unit of the row tile
  int valid;    // 0: the CTA's range is done
  int pad;
  __device__ bool whole() const { return t0 == 0 && t1 == nt; }
};

template <int D>
struct TreeCfg {
  static constexpr int NG = D == 256 ? 1 : 2;     // softmax groups
  static constexpr int NT = D == 256 ? 64 : 128;  // keys per tile
  static constexpr int BLK = NT / kPageTokens;    // pages per tile
  static constexpr int CHUNKS = NT / 32;
  static constexpr uint32_t PAGE = D * kPageTokens * 2;  // bytes of one head's keys (or values)
  static constexpr uint32_t UNIT = BLK * PAGE;           // a key or value tile
  // Slots of the rings of keys and of values, which are held longer (D = 128, 3
  // and 2: the long case takes 221 us instead of 216; D = 256, 4 and 2: 64 drafts
  // 54 us instead of 51).
  static constexpr int KS = D == 64 ? 5 : (D == 128 ? 2 : 3), VS = D == 64 ? 5 : 3;
  static constexpr int SOFTMAX = 128 * NG;  // softmax threads
  // A row tile's fixed cost (query rows in, filling the pipeline, output) in key
  // tiles, for the CTAs' equal shares.  Counted as 5 / 7 / 8 / 10 tiles, 16
  // ragged sequences of up to 2112 tokens and 64 drafts, 32 query and 4 KV heads
  // of 256, fp16, took 51.8 / 47.7 / 48.4 / 48.2 us; counted as 3 / 4 / 5 / 6, the
  // same with 8 KV heads of 128, bf16, 47.8 / 41.2 / 43.2 / 40.9, and 5 of up to
  // 3239 tokens and 20 drafts, 8 query heads on one of 128, bf16, 16.5 / 16.5 /
  // 16.3 / 19.1 (64 x 4096 tokens: no difference).
  static constexpr int OVERHEAD = D == 256 ? 8 : 4;
  // No share is smaller than this, nor than least(): more CTAs on a row tile
  // leave more partial results to join.  At D = 128 a first turn (4 x 128 tokens,
  // 8 drafts, 32 query and 8 KV heads, fp16) took 12.6 us with 2 and 13.0 with 4,
  // the 5 of up to 3239 tokens 16.5 and 17.8.
  static constexpr int LEAST = D == 256 ? 4 : 2;
  // s units a share take time as s, and the parts of a row tile of m units as
  // m / s, least together at s ~ sqrt(m).  One token on 20000 / 100000, 8 query
  // heads on one of 64, bf16: 16.9 / 27.6 us with m / 5 under the root, 17.0 / 26.3 with m / 10, 18.3 /
  // 25.7 with m / 20, 16.6 / 34 with 4 units for both.
  __device__ static int least(int longest) {
    return max(LEAST, (int)sqrtf(0.1f * (float)longest));
  }
  // Warps that ready the values.  (One, at D = 256: 16 sequences of up to 2112
  // tokens and 64 drafts 52.6 us, not 49.5 (four: 50.5); two, at D <= 128, leave
  // too few registers.)
  static constexpr int NFIX = NG == 1 ? 2 : 1;
  static constexpr int THREADS = SOFTMAX + 32 * (NFIX + 3);
  // Warps past the softmax groups
  static constexpr int FIX = 4 * NG, VPROD = FIX + NFIX, KPROD = VPROD + 1, MMA = VPROD + 2;
  // The page mask of tile t is overwritten by tile t + kMaskDepth, whose keys
  // are loaded behind the scores of tile t + kMaskDepth - KS, which are issued
  // behind the value product two tiles before them: t's has read the mask.
  static_assert(kMaskDepth >= KS + 2, "mask depth");
  // TMEM columns
  __host__ __device__ static constexpr uint32_t S(int b) { return (uint32_t)(b * NT); }
  __host__ __device__ static constexpr uint32_t O(int g) { return (uint32_t)(2 * NT + g * D); }
  // The query rows are the products' first operand.  In TMEM, where it has
  // room for them, they cost no shared-memory reads (D = 256: 38 to 17 clocks
  // a product); for D = 128 they are in shared memory.
  static constexpr bool Q_TMEM = D != 128;
  __host__ __device__ static constexpr uint32_t QT() { return (uint32_t)(2 * NT + NG * D); }
  static_assert(2 * NT + NG * D + (Q_TMEM ? D / 2 : 0) <= 512, "TMEM columns");
  // A group's part of a query row, in 16-byte pieces; a warp reads QP pieces of
  // 32 / QP rows at a time
  static constexpr int QN = D / 8 / NG;
  static constexpr int QP = Q_TMEM && QN >= 8 ? 8 : 4;
  // shared memory, from a 1024-byte aligned base
  static constexpr uint32_t RING = 0;
  // query rows for D = 128, [D / 8][128 rows][16 bytes]; at the end of a segment
  // the place where copies of a row meet, [NG][kStageCols][128 rows] floats
  static constexpr uint32_t Q = RING + (KS + VS) * UNIT;
  static constexpr uint32_t STAGE = kStageCols * kTreeRows * 4;
  static constexpr uint32_t ANC = Q + NG * STAGE;  // [2][128][kAncStride]
  static_assert(Q_TMEM || kTreeRows * D * 2 <= NG * STAGE, "query rows");
  static constexpr uint32_t ODD = ANC + 2 * kTreeRows * kAncStride * 4;  // [2][2]
  static constexpr uint32_t PARENT = ODD + 16;
  static constexpr uint32_t ML = PARENT + NFIX * kTreeMaxDrafts * 4;  // [NG][2][128] max (unscaled), sum
  static constexpr uint32_t SEG = ML + NG * 2 * kTreeRows * 4;
  static_assert(SEG % 8 == 0, "segments");
  static constexpr uint32_t MASK = SEG + kSegDepth * (uint32_t)sizeof(Segment);
  static constexpr uint32_t BAR = (MASK + kMaskDepth * 4 + 7) & ~7u;
  // Barriers.  A parity wait only tells a phase from the one before it, so a
  // waiter has to see every phase of its barrier, or know that it is over: keys
  // (waited for by the MMA issuer) and values (by the value warp) have rings,
  // and barriers, of their own.
  static constexpr int K_FULL = 0, K_EMPTY = KS, V_FULL = 2 * KS, V_READY = V_FULL + VS,
                       V_EMPTY = V_READY + VS, S_FULL = V_EMPTY + VS,
                       P_READY = S_FULL + 2, PV_DONE = P_READY + 2, Q_READY = PV_DONE + 2,
                       ANC_FULL = Q_READY + 1, ANC_EMPTY = ANC_FULL + 2, SEG_FULL = ANC_EMPTY + 2,
                       SEG_EMPTY = SEG_FULL + kSegDepth, DRAIN = SEG_EMPTY + kSegDepth,
                       NBAR = DRAIN + 1;
  static constexpr uint32_t TMEM_SLOT = BAR + NBAR * 8;
  static constexpr uint32_t ABORT = TMEM_SLOT + 4;
  static constexpr uint32_t GO = ABORT + 4;
  static constexpr uint32_t BYTES = GO + 4 + 1024;  // + alignment slack
  static_assert(BYTES + 512 <= 232448, "one CTA per SM");
};

// The two 16-bit types: packing, the exponent that marks a NaN or an infinity,
// the unit of softmax weights (2^7 times the largest, 2^8, fits fp16) and the
// operand format of the instruction descriptor.
template <typename T>
struct Half16;
template <>
struct Half16<__nv_bfloat16> {
  static constexpr uint32_t kExp = 0x7F80u, kFormat = 1;
  static constexpr float kWeightLog2 = 0.f;  // log2 of the unit that weights are held in
  __device__ static uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
  __device__ static float widen(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
};
template <>
struct Half16<__half> {
  static constexpr uint32_t kExp = 0x7C00u, kFormat = 0;
  static constexpr float kWeightLog2 = 7.f;
  __device__ static uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  __device__ static float widen(uint16_t x) { return __half2float(__ushort_as_half(x)); }
};

// Instruction descriptor: fp32 D, A and B of one 16-bit type, both K-major.
template <typename T>
__host__ __device__ constexpr uint32_t idesc(uint32_t m, uint32_t n) {
  return (1u << 4) | (Half16<T>::kFormat << 7) | (Half16<T>::kFormat << 10) | ((n >> 3) << 17) |
         ((m >> 4) << 24);
}

struct SeqInfo {
  int lo, n, len, base;  // as in Segment
  int mts, nt;           // row tiles, key tiles (at least 1)
};

template <int D>
__device__ __forceinline__ SeqInfo seq_info(const TreeParams& p, int group, int i) {
  SeqInfo s;
  const PackedSlice rows = packed_slice(__ldg(p.cu + i), __ldg(p.cu + i + 1), p.total_q);
  s.lo = rows.lo;
  s.n = rows.n;
  const int len = max(__ldg(p.seq_lens + i), 0);
  s.base = len - s.n;
  s.len = (int)min((long long)len, (long long)p.c.max_blocks * kPageTokens);
  if (s.n > kTreeMaxDrafts) s.len = 0;
  s.mts = (int)(((long long)s.n * group + kTreeRows - 1) / kTreeRows);
  s.nt = max(1, (s.len + TreeCfg<D>::NT - 1) / TreeCfg<D>::NT);
  return s;
}

// The producer's walk over its CTA's range.
template <int D>
struct Walker {
  long long u, end, off;
  int seq, known;  // `s` holds the numbers of sequence `known`
  SeqInfo s;
  __device__ bool next(const TreeParams& p, int group, Segment& x) {
    x.valid = 0;
    while (u < end) {
      if (seq >= p.c.num_seqs) return false;  // only if the lengths changed under the kernel
      if (known != seq) {
        s = seq_info<D>(p, group, seq);
        known = seq;
      }
      const int per = s.nt + TreeCfg<D>::OVERHEAD;  // units of a row tile: the overhead, then its tiles
      if (off >= (long long)s.mts * p.c.num_kv_heads * per) {
        ++seq;
        off = 0;
        continue;
      }
      const long long tile = off / per;
      const int from = (int)(off - tile * per), take = (int)min((long long)per - from, end - u);
      x.t0 = max(0, from - TreeCfg<D>::OVERHEAD);
      x.t1 = from + take - TreeCfg<D>::OVERHEAD;
      x.u = u - from;
      u += take;
      off += take;
      if (x.t1 <= x.t0) continue;  // a share that ends in the overhead: no tile
      x.lo = s.lo;
      x.n = s.n;
      x.len = s.len;
      x.base = s.base;
      x.nt = s.nt;
      x.seq = seq;
      x.g = (int)(tile / s.mts);
      x.mt = (int)(tile - (long long)x.g * s.mts);
      x.valid = 1;
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
}

// Barrier among softmax warps.  Like the tcgen05 loads and stores it wants the
// whole warp at once, which lane-dependent branches before it do not promise.
// No warp leaves its loop but by what all of them read behind such a barrier.
__device__ __forceinline__ void softmax_barrier(int id, int threads) {
  __syncwarp();
  named_bar_sync(id, threads);
}

// Sums of the non-finite values that a lane's row sees at dimensions c .. c + 7
// among the positions [from, to), 0 where there are none.  The whole warp calls,
// for one c.  Every row sees the whole context, so where a lane asks for it
// (`wild`) the lanes share it, 8 tokens of a dimension a load, and add up; the
// drafts (`branch`), at most 256, are each row's own.
template <int D, typename T>
__device__ __forceinline__ void non_finite_sums(const TreeParams& p, int seq, int g, int from, int to,
                                             int base, const uint32_t* anc, int c, bool wild,
                                             bool branch, float (&sum)[8]) {
  const int lane = threadIdx.x & 31;
  const int32_t* table = p.block_tables + (size_t)seq * p.c.max_blocks;
  const uint16_t* values = static_cast<const uint16_t*>(p.c.v_cache);
  // adds those of the 8 tokens from pos on that `bits` names
  auto add = [&](int id, int pos, uint32_t bits, float (&s)[8]) {
    if (id < 0 || id >= p.c.num_blocks) return;
    const uint4* v = reinterpret_cast<const uint4*>(
        values + (((size_t)id * p.c.num_kv_heads + g) * D + c) * kPageTokens + pos % kPageTokens);
    uint4 e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = __ldg(v + i * (kPageTokens / 8));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t w[4] = {e[i].x, e[i].y, e[i].z, e[i].w};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint16_t h = (uint16_t)(w[k / 2] >> (16 * (k & 1)));
        if ((h & Half16<T>::kExp) == Half16<T>::kExp && (bits >> k & 1u)) s[i] += Half16<T>::widen(h);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.f;
  if (__any_sync(0xffffffffu, wild)) {
    const int end = min(base, to);
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = 0.f;
    int pos = from + 8 * lane;
    int id = pos < end ? __ldg(table + pos / kPageTokens) : -1;
#pragma unroll 1
    while (pos < end) {
      const int ahead = pos + 256;
      const int next = ahead < end ? __ldg(table + ahead / kPageTokens) : -1;
      add(id, pos, low_bits(end - pos), s);
      pos = ahead;
      id = next;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s[i] += __shfl_xor_sync(0xffffffffu, s[i], d);
      if (wild) sum[i] = s[i];
    }
  }
  if (branch) {
#pragma unroll 1
    for (int pos = max(from, base) & ~7; pos < to; pos += 8) {
      const int a = pos - base;  // draft of the first of 8 tokens, from -7 on
      uint32_t bits = a < 0 ? anc[0] << -a
                            : __funnelshift_r(anc[a >> 5], a + 32 < kTreeMaxDrafts ? anc[(a >> 5) + 1] : 0u,
                                              a & 31);
      bits &= low_bits(to - pos) & 0xffu;
      if (bits) add(__ldg(table + pos / kPageTokens), pos, bits, sum);
    }
  }
  __syncwarp();
}

// Writes the non-finite sums of a lane's row over what stands at its columns, of
// every output step `width` from c0 on: in the output row `dst`, or in partial
// results.  `wild`: the steps (a bit each) where the context may hold some.  The
// whole warp calls; rows without any have wild 0 and branch false.
//
// Bound by the latency of its loads.  A CTA that holds three row tiles of 131072
// tokens each (3 drafts, 2 query heads, bf16) takes 5.2 ms at D = 256
// without such values, 5.2 with some in the drafts, 11.7 with four in the context,
// 33 with one in every dimension; at D = 128 3.0, 3.0, 5.7 and 8.7.  (Each row
// reading all positions for itself took 190 ms for 24000 tokens, in which waits
// of other warps could run out.)
template <int D, typename T>
__device__ __forceinline__ void mend_non_finite(const TreeParams& p, int seq, int g, int from, int to,
                                             int base, const uint32_t* anc, int c0, int width,
                                             uint32_t wild, bool branch, float scale, T* dst,
                                             float* part) {
#pragma unroll 1
  for (int i = 0; i < D / TreeCfg<D>::NG / kStageCols * width; i += 8) {
    const int step = i / width, c = c0 + step * kStageCols + i % width;
    float sum[8];
    non_finite_sums<D, T>(p, seq, g, from, to, base, anc, c, wild >> step & 1u, branch, sum);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (sum[k] - sum[k] == 0.f) continue;
      if (part)
        part[(c + k) * kTreeRows] = sum[k];
      else
        reinterpret_cast<uint16_t*>(dst)[c + k] = (uint16_t)Half16<T>::pack(sum[k] * scale, 0.f);
    }
  }
}

template <int D, typename T>
__global__ void __launch_bounds__(TreeCfg<D>::THREADS, 1)
    tree_kernel(const __grid_constant__ TreeParams p) {
  using C = TreeCfg<D>;
  constexpr int NT = C::NT, NG = C::NG, BLK = C::BLK;
  extern __shared__ uint8_t smem_raw[];
  __shared__ UnitScratch scratch;
  __shared__ long long s_total;  // of the range, for the end of a segment
  __shared__ int s_used;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* bp = smem_raw + (base - raw);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bp + C::ABORT);
  volatile uint32_t* page_mask = reinterpret_cast<volatile uint32_t*>(bp + C::MASK);
  Segment* segs = reinterpret_cast<Segment*>(bp + C::SEG);
  auto bar = [&](int i) { return base + C::BAR + 8u * (uint32_t)i; };
  auto k_slot = [&](uint32_t s) { return base + C::RING + s * C::UNIT; };
  auto v_slot = [&](uint32_t s) { return base + C::RING + (C::KS + s) * C::UNIT; };
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    for (int i = C::K_FULL; i < C::S_FULL; ++i)  // the rings'
      mbar_init(bar(i), i >= C::V_READY && i < C::V_EMPTY ? C::NFIX : 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(C::S_FULL + b), 1);
      mbar_init(bar(C::P_READY + b), 4);
      mbar_init(bar(C::PV_DONE + b), 1);
      mbar_init(bar(C::ANC_FULL + b), C::NFIX);
      mbar_init(bar(C::ANC_EMPTY + b), 4 * NG);
    }
    for (int s = 0; s < kSegDepth; ++s) {
      mbar_init(bar(C::SEG_FULL + s), 1);
      mbar_init(bar(C::SEG_EMPTY + s), C::NFIX + 3);  // all readers (the softmax as one)
    }
    mbar_init(bar(C::Q_READY), 4 * NG);
    mbar_init(bar(C::DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncwarp();
  if (warp == 0) {
    tmem_alloc(base + C::TMEM_SLOT, 512);
    tmem_relinquish();
  }
  const int group = p.num_query_heads / p.c.num_kv_heads;
  const UnitRange range = locate_units<C::THREADS>(
      p.c.num_seqs, blockIdx.x, gridDim.x, scratch,
      [&](int i) -> Units {
        const SeqInfo s = seq_info<D>(p, group, i);
        const int per = s.nt + C::OVERHEAD;
        return {(long long)s.mts * p.c.num_kv_heads * per, s.mts ? per : 0};
      },
      [](int longest) { return C::least(longest); });
  if (tid == 0) {
    s_total = range.total;
    s_used = range.used;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(bp + C::TMEM_SLOT);
  grid_launch_dependents();
  Segment x;
  uint32_t tiles = 0, count = 0;  // key tiles and segments before the current segment
  auto wait = [&](int b, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu,
                      wait_bounded(bar(b), parity, abort_flag, p.c.status, kPageStatusTimeout));
  };
  // wait on a slot's barrier of the array b; `phases` has a bit per slot
  auto wait_slot = [&](int b, uint32_t s, uint32_t& phases) -> bool {
    const bool ok = wait(b + s, phases >> s & 1u);
    phases ^= 1u << s;
    return ok;
  };
  // the next published segment into x; false at the end, or when given up.  Its
  // place may be used again once every reader has released it.
  auto segment_there = [&](uint32_t i) -> bool {
    return wait(C::SEG_FULL + i % kSegDepth, (i / kSegDepth) & 1u) && segs[i % kSegDepth].valid;
  };
  auto next_segment = [&]() -> bool {
    if (!segment_there(count)) return false;
    x = segs[count % kSegDepth];
    return true;
  };
  auto release_segment = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::SEG_EMPTY + count % kSegDepth));
  };
  // do key tiles of the segment hold drafts that a row may or may not see?
  auto has_drafts = [&]() -> bool {
    return (long long)x.t1 * NT > x.base && x.n <= kTreeMaxDrafts;
  };

  // For the producers: page ids come 32 at a time, one read ahead of their use;
  // lane b of the warp copies page b of a tile.
  constexpr int TPC = 32 / BLK;  // key tiles per read of ids
  auto read_ids = [&](const Segment& y, int chunk) -> int {
    const int i = y.t0 * BLK + chunk * 32 + lane;
    return chunk * TPC < y.t1 - y.t0 && i < (y.len + kPageTokens - 1) / kPageTokens
               ? __ldg(p.block_tables + (size_t)y.seq * p.c.max_blocks + i)
               : -1;
  };
  // announces the pages of a tile on `full`, then copies them to `dst`; returns
  // a bit per page that is there
  auto copy_pages = [&](const void* cache, int page, uint32_t dst, uint32_t full,
                        volatile uint32_t* mask_out) {
    const bool there = lane < BLK && page >= 0 && page < p.c.num_blocks;
    const uint32_t mask = __ballot_sync(0xffffffffu, there);
    if (lane == 0) {
      if (mask_out) *mask_out = mask;
      mbar_arrive_expect_tx(full, __popc(mask) * C::PAGE);
    }
    __syncwarp();
    if (there)
      bulk_copy_g2s(dst + lane * C::PAGE,
                    static_cast<const T*>(cache) +
                        ((size_t)page * p.c.num_kv_heads + x.g) * (D * kPageTokens),
                    C::PAGE, full);
    __syncwarp();
  };
  // every announced copy has landed before the CTA can exit (also where others
  // gave up); `phases` has a bit per slot
  auto drain = [&](int full, int slots, uint32_t phases) {
    for (int s = 0; s < slots; ++s) wait_drain(bar(full + s), (phases >> s & 1u) ^ 1u);
  };

  if (warp == C::KPROD) {
    // -------------------------------------------------------- key producer
    Walker<D> walk{range.u0, range.u1, range.off, range.seq, -1, {}};
    uint32_t phases = 0;
    // a segment that is published soon: its query rows to L2
    auto prefetch_query = [&](const Segment& y) {
      const int r0 = y.mt * kTreeRows;
      const int rows = (int)min((long long)kTreeRows, (long long)y.n * group - r0);
      for (int i = lane; i < rows; i += 32) {
        const int j = (r0 + i) / group;
        const T* q = static_cast<const T*>(p.query) +
                     ((size_t)(y.lo + j) * p.num_query_heads + y.g * group + (r0 + i - j * group)) * D;
#pragma unroll
        for (int d = 0; d < D; d += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + d));
      }
      __syncwarp();
    };
    auto publish = [&](const Segment& y) -> bool {
      const uint32_t s = count % kSegDepth;
      if (!wait(C::SEG_EMPTY + s, ((count / kSegDepth) & 1u) ^ 1u)) return false;
      if (lane == 0) {
        segs[s] = y;
        mbar_arrive(bar(C::SEG_FULL + s));
      }
      __syncwarp();
      ++count;
      return true;
    };
    bool more = walk.next(p, group, x);
    bool ok = publish(x);
    int ids = -1, next = -1;
    if (more) {
      ids = read_ids(x, 0);
      next = read_ids(x, 1);
    }
    while (ok && more) {
      const int nt = x.t1 - x.t0;
      const int pages = (x.len + kPageTokens - 1) / kPageTokens;
      if (lane == 0 && x.n > kTreeMaxDrafts) atomicOr(p.c.status, kPageStatusBadDraft);
      __syncwarp();
      for (int t = 0; t < nt; ++t) {
        if (t && t % TPC == 0) {
          ids = next;
          next = read_ids(x, t / TPC + 1);
        }
        const int mine = __shfl_sync(0xffffffffu, ids, (t % TPC) * BLK + lane % BLK);
        if (lane < BLK && (x.t0 + t) * BLK + lane < pages && (mine < 0 || mine >= p.c.num_blocks))
          atomicOr(p.c.status, kPageStatusBadBlock);
        __syncwarp();
        const uint32_t u = tiles + t, s = u % C::KS;
        if (!(ok = wait(C::K_EMPTY + s, ((u / C::KS) & 1u) ^ 1u))) break;
#if ATTN_VARLEN_TEST_HOOKS
        if (p.test_withhold && x.u == 0 && x.t0 + t == 0 && u == 0) continue;  // never announced
#endif
        copy_pages(p.c.k_cache, mine, k_slot(s), bar(C::K_FULL + s), page_mask + u % kMaskDepth);
        phases ^= 1u << s;
      }
      if (!ok) break;
      tiles += nt;
      more = walk.next(p, group, x);
      if (more) {
        ids = read_ids(x, 0);
        next = read_ids(x, 1);
        prefetch_query(x);
      }
      ok = publish(x);
    }
    drain(C::K_FULL, C::KS, phases);
  } else if (warp == C::VPROD) {
    // ------------------------------------------------------ value producer
    uint32_t phases = 0;
    bool ok = true;
    while (ok && next_segment()) {
      release_segment();
      const int nt = x.t1 - x.t0;
      int ids = read_ids(x, 0), next = read_ids(x, 1);
      for (int t = 0; t < nt; ++t) {
        if (t && t % TPC == 0) {
          ids = next;
          next = read_ids(x, t / TPC + 1);
        }
        const int mine = __shfl_sync(0xffffffffu, ids, (t % TPC) * BLK + lane % BLK);
        const uint32_t u = tiles + t, s = u % C::VS;
        if (!(ok = wait(C::V_EMPTY + s, ((u / C::VS) & 1u) ^ 1u))) break;
        copy_pages(p.c.v_cache, mine, v_slot(s), bar(C::V_FULL + s), nullptr);
        phases ^= 1u << s;
      }
      tiles += nt;
      ++count;
    }
    drain(C::V_FULL, C::VS, phases);
  } else if (warp == C::MMA) {
    // ---------------------------------------------------------- MMA issuer
    const uint32_t leader = elect_one();
    constexpr uint32_t id_s = idesc<T>(128, NT / 2), id_o = idesc<T>(128, D);
    const uint64_t aq = smem_desc(base + C::Q, 16 * kTreeRows, 128, kSwizzleNone);
    uint32_t p_phase = 0;  // a bit per score buffer
    uint32_t k_phase = 0, v_phase = 0;  // a bit per ring slot
    bool ok = true;
    while (ok && next_segment()) {
      release_segment();
      const int nt = x.t1 - x.t0;
      uint32_t started = 0;  // a bit per accumulator that holds something
      auto scores = [&](int t) -> bool {
        const uint32_t ks = (tiles + t) % C::KS;
        if (!wait_slot(C::K_FULL, ks, k_phase)) return false;
        tc_fence_after();
        const uint64_t bk = smem_desc(k_slot(ks), 256, C::PAGE, kSwizzleNone);
        const uint32_t d = tmem + C::S(t & 1);
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            if constexpr (C::Q_TMEM)
              mma_ts_if(leader, d + half * (NT / 2), tmem + C::QT() + 8 * k,
                        bk + ((half * 128 + k * 512) >> 4), id_s, k > 0 ? 1u : 0u);
            else
              mma_ss_if(leader, d + half * (NT / 2), aq + ((k * 2 * 16 * kTreeRows) >> 4),
                        bk + ((half * 128 + k * 512) >> 4), id_s, k > 0 ? 1u : 0u);
        mma_commit_if(leader, bar(C::K_EMPTY + ks));
        mma_commit_if(leader, bar(C::S_FULL + (t & 1)));
        return true;
      };
      ok = wait(C::Q_READY, count & 1u);
      if (ok) tc_fence_after();
      ok = ok && scores(0) && (nt < 2 || scores(1));
      for (int t = 0; ok && t < nt; ++t) {
        const int b = t & 1, a = NG == 2 ? b : 0;
        const uint32_t vs = (tiles + t) % C::VS;
        ok = wait(C::P_READY + b, p_phase >> b & 1u) && wait_slot(C::V_READY, vs, v_phase);
        if (!ok) break;
        p_phase ^= 1u << b;
        tc_fence_after();
        const uint32_t mask = page_mask[(tiles + t) % kMaskDepth];
        const uint64_t bv = smem_desc(v_slot(vs), 16, 256, kSwizzle32B);
        const uint32_t d = tmem + C::O(a), ps = tmem + C::S(b);
        if (mask == (1u << BLK) - 1u) {
          mma_ts_if(leader, d, ps, bv, id_o, started >> a & 1u);
#pragma unroll
          for (int j = 1; j < BLK; ++j)
            mma_ts_if(leader, d, ps + 8u * j, bv + ((j * C::PAGE) >> 4), id_o, 1u);
          started |= 1u << a;
        } else {
#pragma unroll 1
          for (int j = 0; j < BLK; ++j) {
            if (!(mask >> j & 1)) continue;
            mma_ts_if(leader, d, ps + 8u * j, bv + ((j * C::PAGE) >> 4), id_o, started >> a & 1u);
            started |= 1u << a;
          }
        }
        mma_commit_if(leader, bar(C::V_EMPTY + vs));
        mma_commit_if(leader, bar(C::PV_DONE + b));
        if (t + 2 < nt) ok = scores(t + 2);
      }
      tiles += nt;
      ++count;
    }
    // every MMA of this warp has finished before TMEM is freed
    mma_commit_if(leader, bar(C::DRAIN));
    wait_drain(bar(C::DRAIN), 0);
  } else if (warp >= C::FIX && warp < C::FIX + C::NFIX) {
    // ---------------------------------------------- values made operands
    // A row of a tile is one dimension of one page, 32 bytes.  Rows with bit 2
    // of the dimension set exchange their halves.  Each warp has its pages.
    const int f = warp - C::FIX;
    volatile int* s_odd = reinterpret_cast<volatile int*>(bp + C::ODD);
    int* s_parent = reinterpret_cast<int*>(bp + C::PARENT) + f * kTreeMaxDrafts;
    constexpr int PAGES = BLK / C::NFIX, ROWS = PAGES * D;
    uint32_t uses = 0;  // segments with drafts before this one
    uint32_t v_phase = 0;
    bool ok = true;
    while (ok && next_segment()) {
      release_segment();
      const int nt = x.t1 - x.t0;
      const int edge = min(x.base, x.len);
      const bool drafts = has_drafts();
      const uint32_t a2 = uses & 1u;
      if (drafts) {
        // who sees whom: a bit per draft for every draft that has a row in the
        // tile, by a walk up the tree (parents are below their children).  A
        // few thousand clocks, so before the values, not when the drafts' tile
        // needs it.
        if (!(ok = wait(C::ANC_EMPTY + a2, ((uses >> 1) & 1u) ^ 1u))) break;
        if (lane == 0) s_odd[2 * a2 + f] = 0;
        for (int a = lane; a < x.n; a += 32) {
          int up = p.parents ? __ldg(p.parents + x.lo + a) : a - 1;
          if (up < -1 || up >= a) {
            up = -1;
            atomicOr(p.c.status, kPageStatusBadDraft);
          }
          s_parent[a] = up;
        }
        __syncwarp();
        const int r0 = x.mt * kTreeRows, j0 = r0 / group;
        const int last =
            (int)min((long long)r0 + kTreeRows - 1, (long long)x.n * group - 1) / group;
        uint32_t* table =
            reinterpret_cast<uint32_t*>(bp + C::ANC) + a2 * kTreeRows * kAncStride;
        // two drafts a lane at a time: a step of a walk is a wait for the parent
#pragma unroll 1
        for (int j = j0 + f * 64 + lane; j <= last; j += 64 * C::NFIX) {
          uint32_t word[2] = {0, 0};
          int up[2] = {j, j + 32 <= last ? j + 32 : -1}, at[2] = {j >> 5, (j + 32) >> 5};
          uint32_t* mine[2] = {table + (j - j0) * kAncStride, table + (j + 32 - j0) * kAncStride};
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int w = 0; w < kAncWords; ++w)
              if (up[i] >= 0) mine[i][w] = 0;
          const bool both = up[1] >= 0;
          while (up[0] >= 0 || up[1] >= 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int a = up[i];
              if (a < 0) continue;
              if (a >> 5 != at[i]) {
                mine[i][at[i]] = word[i];
                word[i] = 0;
                at[i] = a >> 5;
              }
              word[i] |= 1u << (a & 31);
              up[i] = s_parent[a];
            }
          }
          mine[0][at[0]] = word[0];
          if (both) mine[1][at[1]] = word[1];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::ANC_FULL + a2));
      }
      for (int t = 0; t < nt; ++t) {
        const int p0 = (x.t0 + t) * NT;
        const uint32_t vs = (tiles + t) % C::VS;
        if (!(ok = wait_slot(C::V_FULL, vs, v_phase))) break;
        uint8_t* v = bp + C::RING + (C::KS + vs) * C::UNIT + f * ROWS * 32;
        // 16-byte pieces of the rows 4 .. 7 of every 8: 8 lanes on 128 bytes
        uint8_t* at = v + (lane >> 3) * 256 + 128 + (lane & 7) * 16;
        uint8_t* to = v + (lane >> 3) * 256 + 128 + ((lane & 7) ^ 1) * 16;
#pragma unroll 1
        for (int i = 0; i < ROWS / 32; i += 8) {
          uint4 e[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) e[k] = *reinterpret_cast<uint4*>(at + (i + k) * 1024);
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(to + (i + k) * 1024) = e[k];
        }
        if (p0 + NT > edge) {
          // slots past the last token, and non-finite values of drafts, must
          // not meet a weight of 0
          __syncwarp();
          uint32_t odd = 0;
#pragma unroll 1
          for (int pg = 0; pg < PAGES; ++pg) {
            const int q0 = p0 + (f * PAGES + pg) * kPageTokens;
            if (q0 + kPageTokens <= edge || q0 >= x.len) continue;
            // the words of a row: tokens past the last, and drafts (sign bits)
            uint32_t past[8], draft[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int pos = q0 + 2 * k;
              past[k] = (pos >= x.len ? 0xffffu : 0u) | (pos + 1 >= x.len ? 0xffff0000u : 0u);
              draft[k] = ((pos >= x.base ? 0x8000u : 0u) | (pos + 1 >= x.base ? 0x80000000u : 0u)) &
                         ~past[k];
            }
#pragma unroll 2
            for (int d = lane; d < D; d += 32) {
              uint8_t* at = v + (pg * D + d) * 32;
              uint4* piece[2] = {reinterpret_cast<uint4*>(at + (d >> 2 & 1) * 16),
                                 reinterpret_cast<uint4*>(at + ((d >> 2 & 1) ^ 1) * 16)};
              const uint4 e[2] = {*piece[0], *piece[1]};
              uint32_t w[8] = {e[0].x, e[0].y, e[0].z, e[0].w, e[1].x, e[1].y, e[1].z, e[1].w};
              // adding the distance from the least non-finite magnitude to the
              // sign bit sets that bit for those that reach it, in both halves
              constexpr uint32_t kToSign = (0x8000u - Half16<T>::kExp) * 0x10001u;
              uint32_t wild[8], any = 0;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                wild[k] = ((w[k] & 0x7fff7fffu) + kToSign) & draft[k];
                any |= wild[k];
                w[k] &= ~past[k];
              }
              if (any) {
#pragma unroll
                for (int k = 0; k < 8; ++k) w[k] &= ~((wild[k] >> 15) * 0xffffu);
              }
              odd |= any;
              if (any || q0 + kPageTokens > x.len) {
                *piece[0] = make_uint4(w[0], w[1], w[2], w[3]);
                *piece[1] = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
          }
          if (odd) s_odd[2 * a2 + f] = 1;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::V_READY + vs));
      }
      tiles += nt;
      ++count;
      if (drafts) ++uses;
    }
  } else {
    // ------------------------------------------------------ softmax groups
    // One thread per row of the tile.  Control flow around the named barriers
    // is the same in every warp; a warp whose wait gave up only skips its
    // arithmetic.
    const int grp = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    float* s_ml = reinterpret_cast<float*>(bp + C::ML);
    volatile int* s_go = reinterpret_cast<volatile int*>(bp + C::GO);
    const volatile int* s_odd = reinterpret_cast<const volatile int*>(bp + C::ODD);
    float* stage = reinterpret_cast<float*>(bp + C::Q + grp * C::STAGE);
    const uint32_t s_tmem[2] = {tmem + lanes + C::S(0), tmem + lanes + C::S(1)};
    const uint32_t o_tmem = tmem + lanes + C::O(grp);
    uint32_t s_count = 0, pv_count = 0;  // parities: bit b for buffer b
    uint32_t uses = 0;
    bool ok = true;
    TreeOpen open{};
    // lanes per copy of a tile's rows
    auto span_of = [&](int rows) {
      return rows <= 32 && C::CHUNKS == 4 ? 32 : (rows <= 64 ? 64 : kTreeRows);
    };
    auto rows_of = [&](const Segment& y) {
      return (int)min((long long)kTreeRows, (long long)y.n * group - (long long)y.mt * kTreeRows);
    };
    // element offset of row r of a segment's tile in query and out (rows past
    // the last: some row of the sequence)
    auto row_at = [&](const Segment& y, int r) -> size_t {
      const int r0 = y.mt * kTreeRows, j = min(r0 + r, y.n * group - 1) / group;
      return ((size_t)(y.lo + j) * p.num_query_heads + y.g * group + (r0 + r - j * group)) * D;
    };
    // A warp fetches the group's part of its 32 query rows, zeros past the last
    // row, in loads that cover 32 / QP rows each: a thread that reads its own
    // row touches 32 lines with every load (D = 256: 5000 clocks between row
    // tiles instead of 3400).  Load i: pieces QP (i / QP) on, rows i % QP on.
    const int q_piece = C::QP == 8 ? lane & 7 : lane >> 3;
    const int q_row = C::QP == 8 ? lane >> 3 : lane & 7;
    constexpr uint32_t kNoRow = 0xffffffffu;  // (as many rows do not fit the memory)
    auto load_query = [&](const Segment& y, uint4 (&e)[C::QN]) {
      const int rows = rows_of(y), r = row % span_of(rows);
      const uint32_t mine = r < rows ? (uint32_t)(row_at(y, r) / D) : kNoRow;
      const uint4* q = static_cast<const uint4*>(p.query) + grp * C::QN + q_piece;
      __syncwarp();
#pragma unroll
      for (int k = 0; k < C::QP; ++k) {
        const uint32_t at = __shfl_sync(0xffffffffu, mine, k * (32 / C::QP) + q_row);
#pragma unroll
        for (int i = k; i < C::QN; i += C::QP)
          e[i] = at != kNoRow ? __ldg(q + (size_t)at * (D / 8) + i / C::QP * C::QP)
                              : make_uint4(0, 0, 0, 0);
      }
    };
    auto store_query = [&](const uint4 (&e)[C::QN]) {
      if constexpr (C::Q_TMEM) {
        // Rows meet their threads in the group's stage, each in the words that
        // it alone writes there later (128 bytes of every 512, pieces exchanged
        // against bank conflicts).
        uint8_t* at = reinterpret_cast<uint8_t*>(stage) + (warp & 3) * 128;
#pragma unroll
        for (int i0 = 0; i0 < C::QN; i0 += C::QP) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < C::QP; ++i) {
            const int q = i * (32 / C::QP) + q_row;
            *reinterpret_cast<uint4*>(at + q * 512 + ((q_piece ^ q) & 7) * 16) = e[i0 + i];
          }
          __syncwarp();
          uint4 o[C::QP];
#pragma unroll
          for (int i = 0; i < C::QP; ++i)
            o[i] = *reinterpret_cast<const uint4*>(at + lane * 512 + ((i ^ lane) & 7) * 16);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < C::QP; i += 4) {
            const uint32_t w[16] = {o[i].x,     o[i].y,     o[i].z,     o[i].w,
                                    o[i + 1].x, o[i + 1].y, o[i + 1].z, o[i + 1].w,
                                    o[i + 2].x, o[i + 2].y, o[i + 2].z, o[i + 2].w,
                                    o[i + 3].x, o[i + 3].y, o[i + 3].z, o[i + 3].w};
            tmem_st16(tmem + lanes + C::QT() + 4 * (grp * C::QN + i0 + i), w);
          }
        }
        __syncwarp();
      } else {
        uint4* dst = reinterpret_cast<uint4*>(bp + C::Q) + (row & ~31);
#pragma unroll
        for (int i = 0; i < C::QN; ++i)
          dst[(grp * C::QN + i / C::QP * C::QP + q_piece) * kTreeRows +
              (i % C::QP) * (32 / C::QP) + q_row] = e[i];
      }
    };
    auto query_ready = [&]() {
      if constexpr (C::Q_TMEM) {
        tmem_wait_st();
        tc_fence_before();
      } else {
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::Q_READY));
    };
    // A segment is taken by one warp and handed on at a barrier, so that all go
    // on or stop together.
    auto take_segment = [&](uint32_t i) {
      if (warp == 0) {
        const bool go = segment_there(i);
        if (lane == 0) *s_go = go ? 1 : 0;
      }
    };
    uint4 query[C::QN];
    take_segment(0);
    softmax_barrier(1, C::SOFTMAX);
    bool more = *s_go != 0;
    if (more) {
      load_query(segs[0], query);
      if (C::Q_TMEM) {
        store_query(query);
        query_ready();
      }
    }
    while (more) {
      x = segs[count % kSegDepth];
      if (!C::Q_TMEM) {
        store_query(query);
        query_ready();
      }
      const int nt = x.t1 - x.t0;
      const int r0 = x.mt * kTreeRows;  // row r of the tile is row r0 + r of the sequence
      const int rows = rows_of(x);
      const int span = span_of(rows), copies = kTreeRows / span;
      const int copy = row / span, r = row % span;  // this thread's copy and row
      const int j0 = r0 / group;
      const int j = min(r0 + r, x.n * group - 1) / group;
      // first position that is not context (every position below it is seen)
      const int edge = min(x.base, x.len);
      const bool drafts = has_drafts();
      const uint32_t a2 = uses & 1u;
      const uint32_t* anc = reinterpret_cast<const uint32_t*>(bp + C::ANC) +
                            (a2 * kTreeRows + (j - j0)) * kAncStride;
      bool built = false;
      float m = -INFINITY, l = 0.f;
      bool seen = false;
#pragma unroll 1
      for (int t = grp; t < nt; t += NG) {
        const int b = t & 1;
        const int p0 = (x.t0 + t) * NT;
        const uint32_t st = b ? s_tmem[1] : s_tmem[0];
        if (ok) ok = wait(C::S_FULL + b, s_count >> b & 1u);
        s_count ^= 1u << b;
        const uint32_t mask = page_mask[(tiles + t) % kMaskDepth];
        const bool masked = p0 + NT > edge || mask != (1u << BLK) - 1u;
        if (masked && drafts && !built) {
          if (ok) ok = wait(C::ANC_FULL + a2, uses >> 1 & 1u);
          built = true;
        }
        if (ok) {
          tc_fence_after();
          // Keys 32 i .. 32 i + 31 of the tile (pages 2 i, 2 i + 1): their
          // scores are columns 16 i .. 16 i + 15 (first halves of the pages)
          // and NT / 2 + 16 i .. + 15 of the buffer, their weights go to
          // columns 16 i .. 16 i + 15.  s[8 half + 16 page + k] below.
          auto load = [&](int i, uint32_t (&s)[32]) {
            __syncwarp();
            tmem_ld16(st + 16 * i, *reinterpret_cast<uint32_t(*)[16]>(&s[0]));
            tmem_ld16(st + NT / 2 + 16 * i, *reinterpret_cast<uint32_t(*)[16]>(&s[16]));
          };
          auto sees = [&](int i) -> uint32_t {  // a bit per key
            const int q0 = p0 + 32 * i;
            const int o = q0 - x.base;  // draft of the first key
            uint32_t w = low_bits(edge - q0);
            if (drafts && o > -32 && o < kTreeMaxDrafts) {
              if (o < 0) {
                w |= anc[0] << -o;
              } else {
                const int k = o >> 5;
                w |= __funnelshift_r(anc[k], k + 1 < kAncWords ? anc[k + 1] : 0u, o & 31);
              }
            }
            w &= low_bits(x.len - q0);
            const uint32_t two = mask >> (2 * i);
            return w & ((two & 1u ? 0xffffu : 0u) | (two & 2u ? 0xffff0000u : 0u));
          };
          auto hide = [&](int i, uint32_t (&s)[32]) {  // scores not seen become -inf
            const uint32_t w = sees(i);
            seen |= w != 0;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              // register k: half k / 16, page k % 16 / 8, token k % 8 + 8 half
              const int key = k % 16 / 8 * 16 + k / 16 * 8 + k % 8;
              if (!(w >> key & 1u)) s[k] = 0xff800000u;
            }
          };
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          auto most = [&](const uint32_t (&s)[32]) {
#pragma unroll
            for (int k = 0; k < 32; k += 8)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                mx[q] = fmax3(mx[q], __uint_as_float(s[k + 2 * q]), __uint_as_float(s[k + 2 * q + 1]));
          };
          // A copy owns the chunks copy, copy + copies, ...: one, two, or (one
          // copy of 128 keys) four, of which the second pair stays in registers
          // between the passes.
          const bool four = C::CHUNKS / copies == 4, two = C::CHUNKS / copies >= 2;
          const int i0 = four ? 2 : copy, i1 = four ? 3 : copy + copies;
          uint32_t s0[32], s1[32];
          auto load_pair = [&](int a, int b2) {
            load(a, s0);
            if (two) load(b2, s1);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) asm volatile("" : "+r"(s0[k]), "+r"(s1[k]));
            if (masked) {
              hide(a, s0);
              if (two) hide(b2, s1);
            }
          };
          if (four) {
            load_pair(0, 1);
            most(s0);
            most(s1);
          }
          load_pair(i0, i1);
          most(s0);
          if (two) most(s1);
          if (!masked) seen = true;
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          // the maximum (of unscaled scores) is only raised where that makes
          // weights more than 2^8 times smaller (weights stay <= 2^8)
          const bool raise = (top - m) * p.scale_log2 > kRescaleThreshold;
          const float alpha = raise ? ex2((m - top) * p.scale_log2) : 1.f;  // m = -inf: 0
          if (raise) {
            m = top;
            l *= alpha;
          }
          if (t >= NG && __any_sync(0xffffffffu, raise)) {
            // With one group the accumulator's last product may still run; with
            // two, S of this tile was issued behind it.  (Not to wait for a
            // product loses no phase: S of the next tile is issued behind it.)
            if (NG == 1) {
              ok = wait(C::PV_DONE + (b ^ 1), pv_count >> (b ^ 1) & 1u);
              tc_fence_after();
            }
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              __syncwarp();
              tmem_ld32(o_tmem + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(o_tmem + c, o);
            }
            tmem_wait_st();
          }
          // A weight is 2^(scale score + off) with off the unit's less scale m.
          // Where scale m passes 2^23, 32 bits hold scores to about 1, and what
          // rounding leaves of scale m could be a weight that overflows.  There a
          // power of two below the scale takes its place, whose product with m is
          // exact (2^100 at most: scores that differ are then 2^76 apart).
          const float ms = m * p.scale_log2;
          float mul = p.scale_log2, off = Half16<T>::kWeightLog2 - ms;
          if (!(fabsf(ms) < 0x1p23f)) {
            const int e = max(1, min(__float_as_int(p.scale_log2) >> 23,
                                     127 + 227 - (__float_as_int(m) >> 23 & 255)));
            mul = __int_as_float(e << 23);
            off = m == -INFINITY ? 0.f : __fadd_rd(Half16<T>::kWeightLog2, -(m * mul));
          }
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          auto weights = [&](int i, const uint32_t (&s)[32]) {
            uint32_t pk[16];
#pragma unroll
            for (int w = 0; w < 16; ++w) {
              // word w of the weights: keys 2 (w % 8), + 1 of page w / 8
              const int k = w % 8 / 4 * 16 + w / 8 * 8 + w % 4 * 2;
              const float a = ex2(fmaf(__uint_as_float(s[k]), mul, off));
              const float e = ex2(fmaf(__uint_as_float(s[k + 1]), mul, off));
              sum[w % 4] += a + e;
              pk[w] = Half16<T>::pack(a, e);
            }
            __syncwarp();
            tmem_st16(st + 16 * i, pk);
          };
          weights(i0, s0);
          if (two) weights(i1, s1);
          if (four) {
            load_pair(0, 1);
            weights(0, s0);
            weights(1, s1);
          }
          if (copies > 1) {  // the other copies' keys
            uint32_t zero[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) zero[i] = 0;
#pragma unroll 1
            for (int i = 0; i < C::CHUNKS; ++i) {
              if (i % copies == copy) continue;
              __syncwarp();
              tmem_st16(st + 16 * i, zero);
            }
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_wait_st();
        }
        if (NG == 1 && t > 0) pv_count ^= 1u << (b ^ 1);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::P_READY + b));
      }
      // -1 marks a row that sees keys, all with a score of -inf
      if (m == -INFINITY && l == 0.f && seen) l = -1.f;
      s_ml[(grp * 2 + 0) * kTreeRows + row] = m;
      s_ml[(grp * 2 + 1) * kTreeRows + row] = l;
      take_segment(count + 1);
      softmax_barrier(1, C::SOFTMAX);
      if (warp == 0) release_segment();  // all have read x
      more = *s_go != 0;
      if (more) {
        // All scores of this segment are there, so the next one's query rows
        // can go to TMEM: its first products run under this one's output.
        load_query(segs[(count + 1) % kSegDepth], query);
        if (C::Q_TMEM) {
          tc_fence_after();
          store_query(query);
          query_ready();
        }
      }
      // The last products.  Those of one buffer finish in order, and all but
      // its last are known to be over (see above).
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int those = (nt - b + 1) / 2;  // the buffer's tiles
        if (NG == 1 ? b != ((nt - 1) & 1) : those == 0) continue;
        if (NG == 2) pv_count ^= (uint32_t)((those - 1) & 1) << b;
        if (ok) ok = wait(C::PV_DONE + b, pv_count >> b & 1u);
        pv_count ^= 1u << b;
      }
      // m, l of the row over groups and copies, and this thread's factors
      float mm = -INFINITY, ll = 0.f, f[NG];
      bool nan = false, weightless = false;
#pragma unroll 1
      for (int i = r; i < kTreeRows; i += span)
#pragma unroll
        for (int a = 0; a < NG; ++a) mm = fmaxf(mm, s_ml[2 * a * kTreeRows + i]);
#pragma unroll 1
      for (int i = r; i < kTreeRows; i += span)
#pragma unroll
        for (int a = 0; a < NG; ++a) {
          const float gm = s_ml[2 * a * kTreeRows + i], gl = s_ml[(2 * a + 1) * kTreeRows + i];
          const float e = gm == -INFINITY ? 0.f : ex2((gm - mm) * p.scale_log2);
          if (e > 0.f) ll += e * gl;
          nan |= !(gl == gl);
          weightless |= gl == -1.f;
          if (i == row) f[a] = gm == -INFINITY ? -1.f : e;  // -1: nothing seen
        }
      if (nan) ll = __uint_as_float(0x7fc00000u);
      if (mm == -INFINITY && !nan) ll = weightless ? -1.f : 0.f;
      // (the segment's value products are over, so its values were looked at)
      const bool odd = drafts && (s_odd[2 * a2] | (C::NFIX == 2 ? s_odd[2 * a2 + 1] : 0)) != 0;
      const bool whole = x.whole();
      float scale = 1.f / ll;
      if (mm == -INFINITY) scale = ll == 0.f ? 0.f : __uint_as_float(0x7fc00000u);
      float* part = reinterpret_cast<float*>(p.workspace + tree_parts_offset()) +
                    (size_t)(2 * blockIdx.x + (x.t0 == 0)) * tree_part_floats(D) + r;
      T* dst = static_cast<T*>(p.out) + row_at(x, r);
      if (ok && !whole && row < rows && grp == 0) {
        part[D * kTreeRows] = mm;
        part[(D + 1) * kTreeRows] = ll;
      }
      // Output steps (a bit each) that are not finite, to be mended at the end
      uint32_t wild = 0;
      tc_fence_after();
#pragma unroll 1
      for (int c = grp * (D / NG); c < (grp + 1) * (D / NG); c += kStageCols) {
        float o[kStageCols];
#pragma unroll
        for (int i = 0; i < kStageCols; ++i) o[i] = 0.f;
        if (ok) {
          uint32_t e[NG][kStageCols];
          __syncwarp();
#pragma unroll
          for (int a = 0; a < NG; ++a) tmem_ld32(tmem + lanes + C::O(a) + c, e[a]);
          tmem_wait_ld();
          // an accumulator that saw no key of the row may hold anything
#pragma unroll
          for (int a = 0; a < NG; ++a)
#pragma unroll
            for (int i = 0; i < kStageCols; ++i)
              o[i] = f[a] < 0.f ? o[i] : fmaf(f[a], __uint_as_float(e[a][i]), o[i]);
        }
        // The copies of a row meet in shared memory, and each goes on with its
        // share of the columns: o[0 .. width).
        int c0 = c, width = kStageCols;
        if (copies > 1) {
#pragma unroll
          for (int i = 0; i < kStageCols; ++i) stage[i * kTreeRows + row] = o[i];
          softmax_barrier(2 + grp, 128);
          width = kStageCols / copies;
          c0 += copy * width;
          const float* at = stage + copy * width * kTreeRows + r;
          if (copies == 2) {
#pragma unroll
            for (int i = 0; i < kStageCols / 2; ++i)
              o[i] = at[i * kTreeRows] + at[i * kTreeRows + kTreeRows / 2];
          } else {
#pragma unroll
            for (int i = 0; i < kStageCols / 4; ++i)
              o[i] = (at[i * kTreeRows] + at[i * kTreeRows + kTreeRows / 4]) +
                     (at[i * kTreeRows + kTreeRows / 2] + at[i * kTreeRows + kTreeRows / 4 * 3]);
          }
          softmax_barrier(2 + grp, 128);
        }
        if (r >= rows || !ok) continue;
        float apart[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kStageCols; ++i)
          if (i < width) apart[i % 4] += o[i] - o[i];
        if (!((apart[0] + apart[1]) + (apart[2] + apart[3]) == 0.f))
          wild |= 1u << ((c - grp * (D / NG)) / kStageCols);
        if (!whole) {
#pragma unroll
          for (int i = 0; i < kStageCols; ++i)
            if (i < width) part[(c0 + i) * kTreeRows] = o[i];
        } else {
#pragma unroll
          for (int i = 0; i < kStageCols; i += 8)
            if (i < width)
              *reinterpret_cast<uint4*>(dst + c0 + i) =
                  make_uint4(Half16<T>::pack(o[i] * scale, o[i + 1] * scale),
                             Half16<T>::pack(o[i + 2] * scale, o[i + 3] * scale),
                             Half16<T>::pack(o[i + 4] * scale, o[i + 5] * scale),
                             Half16<T>::pack(o[i + 6] * scale, o[i + 7] * scale));
        }
      }
      __syncwarp();
      tc_fence_before();
      // The values of drafts were looked at; weights of 0 (a copy's for the keys
      // of the others, a factor's) turn an infinity of the context into a NaN.
      // Where either shows, the sum of the non-finite values that the row sees
      // in this segment is the result (a NaN of the scores is one anyway).
      const bool branch = odd && r < rows && ok && !nan;
      if (nan) wild = 0;
      if (__any_sync(0xffffffffu, wild != 0 || branch)) {
        const int width = kStageCols / copies;
        mend_non_finite<D, T>(p, x.seq, x.g, x.t0 * NT, (int)min((long long)x.len, (long long)x.t1 * NT),
                              x.base, anc, grp * (D / NG) + copy * width, width, wild, branch, scale,
                              dst, whole ? nullptr : part);
      }
      if (drafts) {
        if (lane == 0) mbar_arrive(bar(C::ANC_EMPTY + a2));
        ++uses;
      }
      if (x.t1 < x.nt) {
        // the CTAs that hold the row tile's first key tile and its last unit
        const long long total = s_total, used = s_used;
        auto holder = [&](long long u) { return (int)(((u + 1) * used + total - 1) / total) - 1; };
        open = {1, x.lo, x.n, x.g, x.mt, holder(x.u + C::OVERHEAD + x.nt - 1),
                holder(x.u + C::OVERHEAD), 0};
      }
      tiles += nt;
      ++count;
      // what the next segment overwrites is read
      if (more) softmax_barrier(1, C::SOFTMAX);
    }
    if (tid == 0) {
      if (!ok) open.valid = 0;
      reinterpret_cast<TreeOpen*>(p.workspace)[blockIdx.x] = open;
    }
  }

  // all roles done (or given up, with their async work drained): free TMEM
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// Joins the partial results of the row tiles that no CTA holds whole.  A row tile
// of two or three parts is bound by L2; one of a hundred (a long sequence by
// itself) by latency, so what counts is loads in flight.  A CTA joins 32 rows (a
// row a lane) and 64 columns, 8 columns a warp, or 1 / 2, 1 / 4, 1 / 8 of the
// columns with the parts dealt out to as many groups of warps, so that no warp
// reads more than a few rounds of kJoinParts parts: then CTAs that stand for
// the attention CTAs in the middle of the row tile join the other columns.  The
// parts of a group are added in CTA order and the groups in theirs.  (One token
// on one sequence of 100000: 89 us without groups, 37 with them.)
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinParts = 4;

// groups of warps that share the parts of a row tile: fewer than parts
__device__ __forceinline__ int join_groups(int parts) {
  return parts <= kJoinParts ? 1 : (parts <= 2 * kJoinParts ? 2 : (parts <= 4 * kJoinParts ? 4 : 8));
}

template <int D, typename T>
__global__ void __launch_bounds__(kJoinThreads, 4) tree_join_kernel(const __grid_constant__ TreeParams p) {
  __shared__ float s_m[kJoinWarps][32], s_l[kJoinWarps][32];
  __shared__ float s_f[kTreeMaxCtas][32];
  __shared__ float s_o[kJoinWarps][8][32];
  grid_wait_prerequisite();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = p.num_query_heads / p.c.num_kv_heads;
  const TreeOpen open = reinterpret_cast<const TreeOpen*>(p.workspace)[blockIdx.x];
  if (!open.valid) return;
  const int rows = min(kTreeRows, open.n * group - open.mt * kTreeRows);
  const int cta = open.first, count = open.last - cta + 1, groups = join_groups(count);
  const int share = blockIdx.x - cta;  // of this CTA's columns
  if (32 * (int)blockIdx.y >= rows || share >= groups) return;
  const float* parts = reinterpret_cast<const float*>(p.workspace + tree_parts_offset());
  const int across = kJoinWarps / groups;  // warps side by side on columns
  const int row = 32 * blockIdx.y + lane;
  const int c = ((blockIdx.z * groups + share) * across + warp % across) * 8, mine = warp / across;
  const bool live = row < rows;  // rows past the last have no partial results
  auto part = [&](int k) {
    return parts + (size_t)(k == 0 ? 2 * cta + 1 : 2 * (cta + k)) * tree_part_floats(D) + row;
  };
  float e[kJoinParts][8];
  auto read = [&](int k0) {
#pragma unroll
    for (int x = 0; x < kJoinParts; ++x) {
      const int k = k0 + x * groups;
      const bool there = live && k < count;
      const float* src = part(there ? k : 0) + c * kTreeRows;
#pragma unroll
      for (int i = 0; i < 8; ++i) e[x][i] = there ? src[i * kTreeRows] : 0.f;
    }
  };
  read(mine);
  // the row's maximum, and the parts' factors and sums
  float mm = -INFINITY, l0 = 0.f;  // l0: the sum of this warp's first part
  for (int k = warp; k < count; k += kJoinWarps) {
    const float m = live ? part(k)[D * kTreeRows] : -INFINITY;
    if (k == warp) l0 = live ? part(k)[(D + 1) * kTreeRows] : 0.f;
    s_f[k][lane] = m;
    mm = fmaxf(mm, m);
  }
  s_m[warp][lane] = mm;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) mm = fmaxf(mm, s_m[w][lane]);
  float ll = 0.f;
  bool nan = false, weightless = false;
  for (int k = warp; k < count; k += kJoinWarps) {
    const float m = s_f[k][lane];
    const float l = k == warp ? l0 : (live ? part(k)[(D + 1) * kTreeRows] : 0.f);
    const float f = m == -INFINITY ? 0.f : ex2((m - mm) * p.scale_log2);
    if (f > 0.f) ll += f * l;
    nan |= !(l == l);
    weightless |= l == -1.f;
    s_f[k][lane] = f;
  }
  __syncthreads();  // s_m is read
  s_m[warp][lane] = ll;
  s_l[warp][lane] = nan ? 2.f : (weightless ? 1.f : 0.f);
  __syncthreads();
  float o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = 0.f;
  for (int k0 = mine; k0 < count; k0 += kJoinParts * groups) {
    if (k0 != mine) read(k0);
#pragma unroll
    for (int x = 0; x < kJoinParts; ++x) {
      const int k = k0 + x * groups;
      if (k >= count) break;
      const float f = s_f[k][lane];
      // a factor of 0 does not silence a value that is not finite
#pragma unroll
      for (int i = 0; i < 8; ++i)
        o[i] += f != 0.f ? f * e[x][i] : (e[x][i] - e[x][i] == 0.f ? 0.f : e[x][i]);
    }
  }
  if (groups > 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s_o[warp][i][lane] = o[i];
    __syncthreads();
    if (mine == 0)
      for (int w = warp + across; w < kJoinWarps; w += across)
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] += s_o[w][i][lane];
  }
  if (mine == 0 && live) {
    float state = 0.f;
    ll = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      ll += s_m[w][lane];
      state = fmaxf(state, s_l[w][lane]);
    }
    float scale = 1.f / ll;
    if (state == 2.f || (mm == -INFINITY && state == 1.f)) scale = __uint_as_float(0x7fc00000u);
    else if (mm == -INFINITY) scale = 0.f;
    const int r = open.mt * kTreeRows + row, j = r / group;
    T* dst = static_cast<T*>(p.out) +
             ((size_t)(open.lo + j) * p.num_query_heads + open.g * group + (r - j * group)) * D + c;
    *reinterpret_cast<uint4*>(dst) = make_uint4(
        Half16<T>::pack(o[0] * scale, o[1] * scale), Half16<T>::pack(o[2] * scale, o[3] * scale),
        Half16<T>::pack(o[4] * scale, o[5] * scale), Half16<T>::pack(o[6] * scale, o[7] * scale));
  }
}

template <int D, typename T>
cudaError_t launch_dt(const TreeParams& p, cudaStream_t stream) {
  using C = TreeCfg<D>;
  // per device: the shared-memory opt-in; read by callers of several threads
  static std::atomic<bool> prepared[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!prepared[dev]) {
    e = cudaFuncSetAttribute(tree_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)C::BYTES);
    if (e != cudaSuccess) return e;
    prepared[dev] = true;
  }
  const int grid = std::min(p.c.sm_count, kTreeMaxCtas);
  tree_kernel<D, T><<<grid, C::THREADS, C::BYTES, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, kTreeRows / 32, D / 64);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_join_kernel<D, T>, p);
}

template <int D>
cudaError_t launch_d(const TreeParams& p, bool fp16, cudaStream_t stream) {
  return fp16 ? launch_dt<D, __half>(p, stream) : launch_dt<D, __nv_bfloat16>(p, stream);
}

}  // namespace

cudaError_t launch_tree(const TreeParams& p, bool fp16, cudaStream_t stream) {
  switch (p.c.head_size) {
    case 64: return launch_d<64>(p, fp16, stream);
    case 128: return launch_d<128>(p, fp16, stream);
    case 256: return launch_d<256>(p, fp16, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace avp
