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
//           bit 2 set.  One bulk copy per page, and two warps exchange those
//           halves in shared memory.  (A tiled copy can do the swizzle, in
//           32-byte rows; it held the 64 x 4096 case to 322 us.)
// P is rounded to the cache type and written to TMEM over its scores, in token
// order, for the value product.
//
// A persistent CTA per SM (NG softmax groups of four warps, a producer, an MMA
// issuer, two warps that ready the values) takes an equal share of all (sequence, KV head, row tile, key tile)
// units in that order (paged_walk.cuh), so a long sequence is split over many
// CTAs without the host knowing a length.  Row tiles that begin and end in one
// CTA are written to `out`; the others leave unnormalised partial results in
// the workspace for tree_join_kernel, which adds them in CTA order: results do
// not depend on timing.
//
// For D <= 128 the two groups take the key tiles in turn, each with its own
// score buffer, running maximum, sum and accumulator (TMEM: S0 S1 O0 O1), so
// that one group's exponentials run under the other's products; they are added
// at the end of the row tile.  For D = 256 one group works on both score
// buffers (two 256-column accumulators do not fit).
//
// A weight of 0 does not silence a NaN or an infinity in the values, so in a
// tile that holds drafts or slots past the last token, the warps that ready the
// values clear those slots, and the non-finite values of drafts; the latter are
// added at the end to the rows that see them.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "attn_varlen_device.cuh"
#include "paged_tree_internal.h"
#include "paged_walk.cuh"
#include "ptx.cuh"

namespace avp {
namespace {

constexpr int kMaxDevices = 64;
constexpr int kAncWords = kTreeMaxDrafts / 32;
constexpr int kAncStride = kAncWords + 1;  // words between rows of the ancestor table
constexpr int kMaskDepth = 8;              // key tiles whose page masks are kept
constexpr int kFlagDepth = 8;              // segments whose flags are kept

template <int D>
struct TreeCfg {
  static constexpr int NG = D == 256 ? 1 : 2;     // softmax groups
  static constexpr int NT = D == 256 ? 64 : 128;  // keys per tile
  static constexpr int BLK = NT / kPageTokens;    // pages per tile
  static constexpr uint32_t PAGE = D * kPageTokens * 2;  // bytes of one head's keys (or values)
  static constexpr uint32_t UNIT = BLK * PAGE;           // a key or value tile
  static constexpr int STAGES = D == 64 ? 10 : (D == 128 ? 5 : 4);
  static constexpr int SOFTMAX = 128 * NG;  // softmax threads
  static constexpr int THREADS = SOFTMAX + 128;
  // Warps past the softmax groups.  The MMA issuer comes last: it then shares
  // its scheduler with the groups' last warps, which have no rows below 97.
  static constexpr int FIX = 4 * NG, PROD = 4 * NG + 2, MMA = 4 * NG + 3;
  // the page masks of tile t are overwritten by tile t + kMaskDepth, whose
  // keys cannot be loaded before t's values are released
  static_assert(2 * kMaskDepth - 3 >= STAGES, "mask depth");
  // TMEM columns
  __host__ __device__ static constexpr uint32_t S(int b) { return (uint32_t)(b * NT); }
  __host__ __device__ static constexpr uint32_t O(int g) { return (uint32_t)(2 * NT + g * D); }
  static_assert(2 * NT + NG * D <= 512, "TMEM columns");
  // shared memory, from a 1024-byte aligned base
  static constexpr uint32_t RING = 0;
  static constexpr uint32_t Q = RING + STAGES * UNIT;  // [D / 8][128 rows][16 bytes]
  static constexpr uint32_t ANC = Q + kTreeRows * D * 2;
  static constexpr uint32_t PARENT = ANC + kTreeRows * kAncStride * 4;
  static constexpr uint32_t ML = PARENT + kTreeMaxDrafts * 4;  // [NG][2][128] max, sum
  static constexpr uint32_t MASK = ML + NG * 2 * kTreeRows * 4;
  static constexpr uint32_t BAR = (MASK + kMaskDepth * 4 + 7) & ~7u;
  // barriers
  static constexpr int FULL = 0, EMPTY = STAGES, S_FULL = 2 * STAGES, P_READY = S_FULL + 2,
                       PV_DONE = P_READY + 2, Q_READY = PV_DONE + 2, V_READY = Q_READY + 1,
                       DRAIN = V_READY + STAGES, NBAR = DRAIN + 1;
  static constexpr uint32_t TMEM_SLOT = BAR + NBAR * 8;
  static constexpr uint32_t ABORT = TMEM_SLOT + 4;
  static constexpr uint32_t ODD = ABORT + 4;  // [kFlagDepth][2]
  static constexpr uint32_t BYTES = ODD + kFlagDepth * 8 + 1024;  // + alignment slack
  // a segment has at least two units, so the warps that ready values are at
  // most STAGES / 2 segments ahead of the softmax groups
  static_assert(kFlagDepth > STAGES / 2, "flag depth");
  static_assert(BYTES + 512 <= 232448, "one CTA per SM");
};

// The two 16-bit types: packing, the exponent that marks a NaN or an infinity,
// and the operand format of the instruction descriptor.
template <typename T>
struct Half16;
template <>
struct Half16<__nv_bfloat16> {
  static constexpr uint32_t kExp = 0x7F80u, kFormat = 1;
  __device__ static uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
  __device__ static float widen(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
};
template <>
struct Half16<__half> {
  static constexpr uint32_t kExp = 0x7C00u, kFormat = 0;
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
  int lo, n;    // packed rows
  int len;      // tokens in the table (0 with too many drafts)
  int base;     // position of draft 0 (may be negative)
  int mts, nt;  // row tiles, key tiles (at least 1)
};

template <int D>
__device__ __forceinline__ SeqInfo seq_info(const TreeParams& p, int group, int i) {
  SeqInfo s;
  s.lo = max(__ldg(p.cu + i), 0);
  s.n = max(min(__ldg(p.cu + i + 1), p.total_q) - s.lo, 0);
  const int len = max(__ldg(p.seq_lens + i), 0);
  s.base = len - s.n;
  s.len = (int)min((long long)len, (long long)p.c.max_blocks * kPageTokens);
  if (s.n > kTreeMaxDrafts) s.len = 0;
  s.mts = (int)(((long long)s.n * group + kTreeRows - 1) / kTreeRows);
  s.nt = max(1, (s.len + TreeCfg<D>::NT - 1) / TreeCfg<D>::NT);
  return s;
}

// A CTA's part of one row tile: key tiles [t0, t1).
struct Segment {
  SeqInfo s;
  int seq, g, mt, t0, t1;
  long long u;  // unit number of t0
  __device__ bool whole() const { return t0 == 0 && t1 == s.nt; }
};

// Every role walks its CTA's range on its own.
template <int D>
struct Walker {
  long long u, end, off;
  int seq;
  __device__ bool next(const TreeParams& p, int group, Segment& x) {
    if (u >= end) return false;
    for (;; ++seq, off = 0) {
      if (seq >= p.c.num_seqs) return false;  // only if the lengths changed under the kernel
      x.s = seq_info<D>(p, group, seq);
      const long long units = (long long)x.s.mts * p.c.num_kv_heads * x.s.nt;
      if (off < units) break;
    }
    x.seq = seq;
    const long long tile = off / x.s.nt;
    x.t0 = (int)(off - tile * x.s.nt);
    x.t1 = (int)min((long long)x.s.nt, x.t0 + (end - u));
    x.g = (int)(tile / x.s.mts);
    x.mt = (int)(tile - (long long)x.g * x.s.mts);
    x.u = u;
    u += x.t1 - x.t0;
    off += x.t1 - x.t0;
    return true;
  }
};

// Ring units of a segment with nt key tiles, in the order they are used:
// K0 K1 V0 K2 V1 K3 ... V(nt-1).
__device__ __forceinline__ int unit_k(int t) { return t < 2 ? t : 2 * t - 1; }
__device__ __forceinline__ int unit_v(int t, int nt) { return t == nt - 1 ? 2 * nt - 1 : 2 * t + 2; }

__device__ __forceinline__ uint32_t low_bits(int n) {
  return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
}

// Barrier among the softmax warps.  Like the tcgen05 loads and stores it wants
// the whole warp at once, which lane-dependent branches before it do not promise.
__device__ __forceinline__ void softmax_barrier(int threads) {
  __syncwarp();
  named_bar_sync(1, threads);
}

template <int D, typename T>
__global__ void __launch_bounds__(TreeCfg<D>::THREADS, 1)
    tree_kernel(const __grid_constant__ TreeParams p) {
  using C = TreeCfg<D>;
  constexpr int NT = C::NT, NG = C::NG, BLK = C::BLK;
  extern __shared__ uint8_t smem_raw[];
  __shared__ UnitScratch scratch;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* bp = smem_raw + (base - raw);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bp + C::ABORT);
  volatile uint32_t* page_mask = reinterpret_cast<volatile uint32_t*>(bp + C::MASK);
  auto bar = [&](int i) { return base + C::BAR + 8u * (uint32_t)i; };
  auto slot = [&](uint32_t unit) { return base + C::RING + (unit % C::STAGES) * C::UNIT; };
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(bar(C::FULL + s), 1);
      mbar_init(bar(C::EMPTY + s), 1);
      mbar_init(bar(C::V_READY + s), 2);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(C::S_FULL + b), 1);
      mbar_init(bar(C::P_READY + b), 4);
      mbar_init(bar(C::PV_DONE + b), 1);
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
      p.c.num_seqs, blockIdx.x, gridDim.x, scratch, [&](int i) -> long long {
        const SeqInfo s = seq_info<D>(p, group, i);
        return (long long)s.mts * p.c.num_kv_heads * s.nt;
      });
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(bp + C::TMEM_SLOT);
  grid_launch_dependents();
  Walker<D> walk{range.u0, range.u1, range.off, range.seq};
  Segment x;
  uint32_t units = 0, tiles = 0;  // ring units and key tiles of the segments before this one
  auto wait = [&](int b, uint32_t parity, int code) -> bool {
    return __all_sync(0xffffffffu, wait_bounded(bar(b), parity, abort_flag, p.c.status, code));
  };
  auto wait_unit = [&](uint32_t u) -> bool {
    return wait(C::FULL + u % C::STAGES, (u / C::STAGES) & 1u, kPageStatusTimeout);
  };

  if (warp == C::PROD) {
    // ------------------------------------------------------------ producer
    // Page ids come 32 at a time, one read ahead of their use; lane b of the
    // warp copies page b of a tile.
    constexpr int TPC = 32 / BLK;  // key tiles per read of ids
    uint32_t issued = 0;
    bool ok = true;
    while (ok && walk.next(p, group, x)) {
      const int nt = x.t1 - x.t0;
      const int pages = (x.s.len + kPageTokens - 1) / kPageTokens;
      const int32_t* table = p.block_tables + (size_t)x.seq * p.c.max_blocks;
      auto read_ids = [&](int chunk) -> int {
        const int i = x.t0 * BLK + chunk * 32 + lane;
        return chunk * TPC < nt && i < pages ? __ldg(table + i) : -1;
      };
      int ids = read_ids(0), next = read_ids(1);
      int id[2] = {-1, -1};  // this lane's page of the last two key tiles
      auto issue = [&](int t, bool value) {
        const uint32_t u = issued, s = u % C::STAGES;
        if (!wait(C::EMPTY + s, ((u / C::STAGES) & 1u) ^ 1u, kPageStatusTimeout)) return false;
        const int page = t & 1 ? id[1] : id[0];
        const bool there = lane < BLK && page >= 0 && page < p.c.num_blocks;
        const uint32_t mask = __ballot_sync(0xffffffffu, there);
        const uint32_t full = bar(C::FULL + s);
        if (lane == 0) {
          if (!value) page_mask[(tiles + t) % kMaskDepth] = mask;
          mbar_arrive_expect_tx(full, __popc(mask) * C::PAGE);
        }
        __syncwarp();
        if (there)
          bulk_copy_g2s(slot(u) + lane * C::PAGE,
                        static_cast<const T*>(value ? p.c.v_cache : p.c.k_cache) +
                            ((size_t)page * p.c.num_kv_heads + x.g) * (D * kPageTokens),
                        C::PAGE, full);
        ++issued;
        return true;
      };
      auto load_k = [&](int t) {
        if (t && t % TPC == 0) {
          ids = next;
          next = read_ids(t / TPC + 1);
        }
        const int mine = __shfl_sync(0xffffffffu, ids, (t % TPC) * BLK + lane % BLK);
        if (t & 1) id[1] = mine; else id[0] = mine;
        if (lane < BLK && (x.t0 + t) * BLK + lane < pages &&
            (mine < 0 || mine >= p.c.num_blocks))
          atomicOr(p.c.status, kPageStatusBadBlock);
        return issue(t, false);
      };
      ok = load_k(0) && (nt < 2 || load_k(1));
      for (int t = 0; ok && t < nt; ++t) {
        ok = issue(t, true);
        if (ok && t + 2 < nt) ok = load_k(t + 2);
      }
      tiles += nt;
    }
    if (!ok) {
      // let every copy already issued land before the CTA can exit
      const uint32_t first = issued > (uint32_t)C::STAGES ? issued - C::STAGES : 0;
      for (uint32_t u = first; u < issued; ++u)
        wait_drain(bar(C::FULL + u % C::STAGES), (u / C::STAGES) & 1u);
    }
  } else if (warp == C::MMA) {
    // ---------------------------------------------------------- MMA issuer
    const uint32_t leader = elect_one();
    constexpr uint32_t id_s = idesc<T>(128, NT / 2), id_o = idesc<T>(128, D);
    const uint64_t aq = smem_desc(base + C::Q, 16 * kTreeRows, 128, kSwizzleNone);
    uint32_t p_count[2] = {0, 0}, segments = 0;
    uint32_t v_parity = 0;  // a bit per ring slot
    bool ok = true;
    while (ok && walk.next(p, group, x)) {
      const int nt = x.t1 - x.t0;
      bool started[2] = {false, false};  // the accumulators hold something
      auto scores = [&](int t) {
        const uint32_t u = units + unit_k(t);
        if (!wait_unit(u)) return false;
        tc_fence_after();
        const uint64_t bk = smem_desc(slot(u), 256, C::PAGE, kSwizzleNone);
        const uint32_t d = tmem + C::S(t & 1);
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss_if(leader, d + half * (NT / 2), aq + ((k * 2 * 16 * kTreeRows) >> 4),
                      bk + ((half * 128 + k * 512) >> 4), id_s, k > 0 ? 1u : 0u);
        mma_commit_if(leader, bar(C::EMPTY + u % C::STAGES));
        mma_commit_if(leader, bar(C::S_FULL + (t & 1)));
        return true;
      };
      ok = wait(C::Q_READY, segments++ & 1u, kPageStatusTimeout);
      if (ok) tc_fence_after();
      ok = ok && scores(0) && (nt < 2 || scores(1));
      for (int t = 0; ok && t < nt; ++t) {
        const int b = t & 1, a = NG == 2 ? b : 0;
        const uint32_t u = units + unit_v(t, nt);
        const uint32_t vs = u % C::STAGES;
        ok = wait(C::P_READY + b, p_count[b]++ & 1u, kPageStatusTimeout) &&
             wait(C::V_READY + vs, v_parity >> vs & 1u, kPageStatusTimeout);
        if (!ok) break;
        v_parity ^= 1u << vs;
        tc_fence_after();
        const uint32_t mask = page_mask[(tiles + t) % kMaskDepth];
        const uint64_t bv = smem_desc(slot(u), 16, 256, kSwizzle32B);
        const uint32_t d = tmem + C::O(a), ps = tmem + C::S(b);
        if (mask == (1u << BLK) - 1u) {
          mma_ts_if(leader, d, ps, bv, id_o, started[a] ? 1u : 0u);
#pragma unroll
          for (int j = 1; j < BLK; ++j)
            mma_ts_if(leader, d, ps + 8u * j, bv + ((j * C::PAGE) >> 4), id_o, 1u);
          started[a] = true;
        } else {
          for (int j = 0; j < BLK; ++j) {
            if (!(mask >> j & 1)) continue;
            mma_ts_if(leader, d, ps + 8u * j, bv + ((j * C::PAGE) >> 4), id_o,
                      started[a] ? 1u : 0u);
            started[a] = true;
          }
        }
        mma_commit_if(leader, bar(C::EMPTY + u % C::STAGES));
        mma_commit_if(leader, bar(C::PV_DONE + b));
        if (t + 2 < nt) ok = scores(t + 2);
      }
      units += 2 * nt;
      tiles += nt;
    }
    // every MMA of this warp has finished before TMEM is freed
    mma_commit_if(leader, bar(C::DRAIN));
    wait_drain(bar(C::DRAIN), 0);
  } else if (warp >= C::FIX && warp < C::FIX + 2) {
    // ---------------------------------------------- values made operands
    // Each warp takes half of a tile's rows (a row: one dimension of one page,
    // 32 bytes).  Rows with bit 2 of the dimension set exchange their halves.
    const int f = warp - C::FIX;
    volatile int* flags = reinterpret_cast<volatile int*>(bp + C::ODD);
    constexpr int ROWS = BLK * D / 2;
    uint32_t segments = 0;
    bool ok = true;
    while (ok && walk.next(p, group, x)) {
      const int nt = x.t1 - x.t0;
      const int edge = min(x.s.base, x.s.len);
      if (lane == 0) flags[2 * (segments % kFlagDepth) + f] = 0;
      __syncwarp();
      for (int t = 0; t < nt; ++t) {
        const uint32_t u = units + unit_v(t, nt);
        if (!(ok = wait_unit(u))) break;
        uint8_t* v = bp + C::RING + (u % C::STAGES) * C::UNIT + f * ROWS * 32;
        // 16-byte pieces of the rows 4 .. 7 of every 8: 8 lanes on 128 bytes
        uint8_t* at = v + (lane >> 3) * 256 + 128 + (lane & 7) * 16;
        uint8_t* to = v + (lane >> 3) * 256 + 128 + ((lane & 7) ^ 1) * 16;
#pragma unroll
        for (int i = 0; i < ROWS / 32; i += 8) {
          uint4 e[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (i + k < ROWS / 32) e[k] = *reinterpret_cast<uint4*>(at + (i + k) * 1024);
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (i + k < ROWS / 32) *reinterpret_cast<uint4*>(to + (i + k) * 1024) = e[k];
        }
        const int p0 = (x.t0 + t) * NT;
        if (p0 + NT > edge) {
          // slots past the last token, and non-finite values of drafts, must
          // not meet a weight of 0
          __syncwarp();
          bool odd = false;
          for (int i = lane; i < ROWS; i += 32) {
            const int page = (f * ROWS + i) / D, d = (f * ROWS + i) % D;
            const int q0 = p0 + page * kPageTokens;
            if (q0 + kPageTokens <= edge) continue;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint4* piece =
                  reinterpret_cast<uint4*>(v + i * 32 + ((half ^ (d >> 2 & 1)) * 16));
              uint4 e = *piece;
              uint32_t* w = reinterpret_cast<uint32_t*>(&e);
              bool change = false;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const int pos = q0 + half * 8 + k;
                const uint32_t sh = 16 * (k & 1);
                const bool past = pos >= x.s.len;
                const bool wild =
                    pos >= x.s.base && (w[k >> 1] >> sh & Half16<T>::kExp) == Half16<T>::kExp;
                odd |= wild && !past;
                if (past || wild) {
                  w[k >> 1] &= ~(0xffffu << sh);
                  change = true;
                }
              }
              if (change) *piece = e;
            }
          }
          if (odd) flags[2 * (segments % kFlagDepth) + f] = 1;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::V_READY + u % C::STAGES));
      }
      units += 2 * nt;
      ++segments;
    }
  } else {
    // ------------------------------------------------------ softmax groups
    // One thread per row.  Control flow around the named barriers is the same
    // in every warp; a warp whose wait gave up only skips its arithmetic.
    const int grp = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    uint32_t* s_anc = reinterpret_cast<uint32_t*>(bp + C::ANC);
    int* s_parent = reinterpret_cast<int*>(bp + C::PARENT);
    float* s_ml = reinterpret_cast<float*>(bp + C::ML);
    const volatile int* s_odd = reinterpret_cast<const volatile int*>(bp + C::ODD);
    const T* query = static_cast<const T*>(p.query);
    T* out = static_cast<T*>(p.out);
    float* parts = reinterpret_cast<float*>(p.workspace + tree_parts_offset());
    uint32_t s_count[2] = {0, 0}, pv_count[2] = {0, 0}, segments = 0;
    bool ok = true;
    TreeOpen open{};
    while (walk.next(p, group, x)) {
      const int nt = x.t1 - x.t0;
      const int rows = (int)min((long long)kTreeRows,
                                (long long)x.s.n * group - (long long)x.mt * kTreeRows);
      const int r0 = x.mt * kTreeRows;  // row r of the tile is row r0 + r of the sequence
      const int j0 = r0 / group;
      const int j = min(r0 + row, x.s.n * group - 1) / group;
      // first position that is not context (every position below it is seen)
      const int edge = min(x.s.base, x.s.len);
      softmax_barrier(C::SOFTMAX);  // the last segment's shared tables are read
      // the query rows, zeros past the last
      {
        const T* src = query + ((size_t)(x.s.lo + j) * p.num_query_heads + x.g * group +
                                (r0 + row - j * group)) * D;
#pragma unroll 4
        for (int c = grp; c < D / 8; c += NG) {
          uint4 e = make_uint4(0, 0, 0, 0);
          if (row < rows) e = __ldg(reinterpret_cast<const uint4*>(src + c * 8));
          *reinterpret_cast<uint4*>(bp + C::Q + (c * kTreeRows + row) * 16) = e;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::Q_READY));
      const bool drafts = (long long)x.t1 * NT > x.s.base && x.s.n <= kTreeMaxDrafts;
      if (tid == 0 && x.s.n > kTreeMaxDrafts) atomicOr(p.c.status, kPageStatusBadDraft);
      if (drafts) {
        for (int a = tid; a < x.s.n; a += C::SOFTMAX) {
          int up = p.parents ? __ldg(p.parents + x.s.lo + a) : a - 1;
          if (up < -1 || up >= a) {
            up = -1;
            atomicOr(p.c.status, kPageStatusBadDraft);
          }
          s_parent[a] = up;
        }
        softmax_barrier(C::SOFTMAX);
        const int last = min(r0 + rows - 1, x.s.n * group - 1) / group;
        if (tid <= last - j0) {  // at most 128 drafts have a row in the tile
          uint32_t* mine = s_anc + tid * kAncStride;
#pragma unroll
          for (int w = 0; w < kAncWords; ++w) mine[w] = 0;
          for (int a = j0 + tid; a >= 0; a = s_parent[a]) mine[a >> 5] |= 1u << (a & 31);
        }
      }
      softmax_barrier(C::SOFTMAX);
      const uint32_t* anc = s_anc + (j - j0) * kAncStride;
      const bool live_warp = 32 * (warp & 3) < rows;
      float m = -INFINITY, l = 0.f;
      bool seen = false;
      for (int t = grp; t < nt; t += NG) {
        const int b = t & 1;
        const int p0 = (x.t0 + t) * NT;
        if (ok) ok = wait(C::S_FULL + b, s_count[b] & 1u, kPageStatusTimeout);
        ++s_count[b];
        const uint32_t mask = page_mask[(tiles + t) % kMaskDepth];
        if (ok && live_warp) {
          tc_fence_after();
          uint32_t s[NT];
          __syncwarp();
          tmem_ld_cols<NT>(tmem + lanes + C::S(b), s);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < NT; ++i) asm volatile("" : "+r"(s[i]));
          // scores the row does not see become -inf; column c of the buffer is
          // token (c % 8) + 8 half of page (c % (NT / 2)) / 8
          if (p0 + NT > edge || mask != (1u << BLK) - 1u) {
#pragma unroll
            for (int w = 0; w < NT / 32; ++w) {
              const int q0 = p0 + 32 * w;
              const int o = q0 - x.s.base;  // draft of the word's first token
              uint32_t sees = low_bits(edge - q0);
              if (drafts && o > -32 && o < kTreeMaxDrafts) {
                if (o < 0) {
                  sees |= anc[0] << -o;
                } else {
                  const int k = o >> 5;
                  sees |= __funnelshift_r(anc[k], k + 1 < kAncWords ? anc[k + 1] : 0u, o & 31);
                }
              }
              sees &= low_bits(x.s.len - q0);
              const uint32_t two = mask >> (2 * w);
              sees &= (two & 1u ? 0xffffu : 0u) | (two & 2u ? 0xffff0000u : 0u);
              seen |= sees != 0;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const int page = 2 * w + i / 16, half = i % 16 / 8;
                const int c = half * (NT / 2) + page * 8 + i % 8;
                if (!(sees >> i & 1u)) s[c] = 0xff800000u;
              }
            }
          } else {
            seen = true;
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < NT; i += 8) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              mx[q] = fmax3(mx[q], __uint_as_float(s[i + 2 * q]), __uint_as_float(s[i + 2 * q + 1]));
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
          // with one group the last product of the accumulator may still run;
          // with two, S of this tile was issued behind it
          if (NG == 1 && t > 0) {
            ok = wait(C::PV_DONE + (b ^ 1), pv_count[b ^ 1] & 1u, kPageStatusTimeout);
            ++pv_count[b ^ 1];
            tc_fence_after();
          }
          // the maximum is only raised by more than 2^8 (weights stay <= 2^8)
          const bool raise = top > m + kRescaleThreshold;
          const float alpha = raise ? ex2(m - top) : 1.f;  // m = -inf: 0
          if (raise) {
            m = top;
            l *= alpha;
          }
          if (t >= NG && __any_sync(0xffffffffu, raise)) {
            __syncwarp();
#pragma unroll
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(tmem + lanes + C::O(grp) + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(tmem + lanes + C::O(grp) + c, o);
            }
            tmem_wait_st();
          }
          const float off = m == -INFINITY ? 0.f : -m;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          uint32_t pk[NT / 2];
#pragma unroll
          for (int i = 0; i < NT / 2; ++i) {
            // word i of P: tokens 2 (i % 8) and the next of page i / 8
            const int c = (i % 8 / 4) * (NT / 2) + i / 8 * 8 + i % 4 * 2;
            const float a = ex2(fmaf(__uint_as_float(s[c]), p.scale_log2, off));
            const float e = ex2(fmaf(__uint_as_float(s[c + 1]), p.scale_log2, off));
            sum[i % 4] += a + e;
            pk[i] = Half16<T>::pack(a, e);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          __syncwarp();
          tmem_st_cols<NT / 2>(tmem + lanes + C::S(b), pk);
          tmem_wait_st();
        } else if (NG == 1 && t > 0) {
          if (ok) ok = wait(C::PV_DONE + (b ^ 1), pv_count[b ^ 1] & 1u, kPageStatusTimeout);
          ++pv_count[b ^ 1];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::P_READY + b));
      }
      // the group's last product (with one group also the last of the other
      // buffer, which the loop has waited for)
      {
        const int t = nt - 1 - (NG == 2 && ((nt - 1) & 1) != grp ? 1 : 0);
        if (NG == 2) {
          if (t >= 0) {
            // products of one buffer finish in order: the phases before the
            // last are known to be over (see above)
            pv_count[grp] += (t - grp) / 2;
            if (ok) ok = wait(C::PV_DONE + grp, pv_count[grp] & 1u, kPageStatusTimeout);
            ++pv_count[grp];
          }
        } else {
          if (ok) ok = wait(C::PV_DONE + (t & 1), pv_count[t & 1] & 1u, kPageStatusTimeout);
          ++pv_count[t & 1];
        }
      }
      // -1 marks a row that sees keys, all with a score of -inf
      if (m == -INFINITY && l == 0.f && seen) l = -1.f;
      s_ml[(grp * 2 + 0) * kTreeRows + row] = m;
      s_ml[(grp * 2 + 1) * kTreeRows + row] = l;
      softmax_barrier(C::SOFTMAX);
      // m, l of the row over the groups, and each group's factor
      float gm[NG], gl[NG], f[NG], mm = -INFINITY, ll = 0.f;
      bool nan = false, weightless = false;
#pragma unroll
      for (int a = 0; a < NG; ++a) {
        gm[a] = s_ml[(a * 2 + 0) * kTreeRows + row];
        gl[a] = s_ml[(a * 2 + 1) * kTreeRows + row];
        mm = fmaxf(mm, gm[a]);
        nan |= !(gl[a] == gl[a]);
        weightless |= gl[a] == -1.f;
      }
#pragma unroll
      for (int a = 0; a < NG; ++a) {
        f[a] = gm[a] == -INFINITY ? 0.f : ex2(gm[a] - mm);
        if (f[a] > 0.f) ll += f[a] * gl[a];
      }
      if (nan) ll = __uint_as_float(0x7fc00000u);
      if (mm == -INFINITY && !nan) ll = weightless ? -1.f : 0.f;
      // (the tile's value products are over, so its values have been looked at)
      const bool odd = (s_odd[2 * (segments % kFlagDepth)] | s_odd[2 * (segments % kFlagDepth) + 1]) != 0;
      const bool whole = x.whole();
      if (ok && live_warp) {
        tc_fence_after();
        const float scale = mm == -INFINITY ? (ll == 0.f ? 0.f : __uint_as_float(0x7fc00000u))
                                            : 1.f / ll;
        float* part = parts + (size_t)(2 * blockIdx.x + (x.t0 == 0)) * tree_part_floats(D);
        if (!whole && grp == 0) {
          part[D * kTreeRows + row] = mm;
          part[(D + 1) * kTreeRows + row] = ll;
        }
        T* dst = out + ((size_t)(x.s.lo + j) * p.num_query_heads + x.g * group +
                        (r0 + row - j * group)) * D;
#pragma unroll 1
        for (int c = grp * (D / NG); c < (grp + 1) * (D / NG); c += 32) {
          float o[32];
          {
            uint32_t e[NG][32];
            __syncwarp();
#pragma unroll
            for (int a = 0; a < NG; ++a) tmem_ld32(tmem + lanes + C::O(a) + c, e[a]);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              o[i] = 0.f;
#pragma unroll
              for (int a = 0; a < NG; ++a) {
                // a group that saw no key of the row may hold anything
                const float y = __uint_as_float(e[a][i]);
                if (f[a] != 0.f) o[i] += f[a] * y;
                else if (gm[a] != -INFINITY && !(y - y == 0.f)) o[i] += y;
              }
            }
          }
          if (odd && drafts && row < rows) {
            // the non-finite values of the drafts the row sees in this segment
            const int from = max(x.t0 * NT, max(x.s.base, 0));
            const int to = (int)min((long long)x.s.len, (long long)x.t1 * NT);
            for (int pos = from; pos < to; ++pos) {
              const int a = pos - x.s.base;
              if (!(anc[a >> 5] >> (a & 31) & 1u)) continue;
              const int id =
                  __ldg(p.block_tables + (size_t)x.seq * p.c.max_blocks + pos / kPageTokens);
              if (id < 0 || id >= p.c.num_blocks) continue;
              const uint16_t* v = static_cast<const uint16_t*>(p.c.v_cache) +
                                  (((size_t)id * p.c.num_kv_heads + x.g) * D + c) * kPageTokens +
                                  pos % kPageTokens;
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const uint16_t e = v[i * kPageTokens];
                if ((e & Half16<T>::kExp) == Half16<T>::kExp) o[i] += Half16<T>::widen(e);
              }
            }
          }
          if (whole) {
            if (row < rows) {
#pragma unroll
              for (int i = 0; i < 32; i += 8) {
                uint4 w;
                w.x = Half16<T>::pack(o[i] * scale, o[i + 1] * scale);
                w.y = Half16<T>::pack(o[i + 2] * scale, o[i + 3] * scale);
                w.z = Half16<T>::pack(o[i + 4] * scale, o[i + 5] * scale);
                w.w = Half16<T>::pack(o[i + 6] * scale, o[i + 7] * scale);
                *reinterpret_cast<uint4*>(dst + c + i) = w;
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) part[(c + i) * kTreeRows + row] = o[i];
          }
        }
        tc_fence_before();
      }
      if (!whole && x.t0 == 0) {
        const long long used = range.total < gridDim.x ? range.total : gridDim.x;
        const long long next = x.u + x.s.nt;  // the unit behind the row tile
        open = {1, x.s.lo, x.s.n, x.g, x.mt,
                (int)((next * used + range.total - 1) / range.total) - 1, {0, 0}};
      }
      units += 2 * nt;
      tiles += nt;
      ++segments;
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

// Joins the partial results of the row tile that CTA blockIdx.x began and
// others went on with: 32 rows a CTA (blockIdx.y), a row a lane, D / 8 columns
// a warp, the parts in CTA order.
constexpr int kJoinThreads = 256;

template <int D, typename T>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const __grid_constant__ TreeParams p) {
  constexpr int COLS = D / 8;
  grid_wait_prerequisite();
  const int cta = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const TreeOpen open = reinterpret_cast<const TreeOpen*>(p.workspace)[cta];
  const int group = p.num_query_heads / p.c.num_kv_heads;
  const int r0 = open.mt * kTreeRows, row = 32 * blockIdx.y + lane;
  if (!open.valid || open.n * group - r0 <= 32 * (int)blockIdx.y) return;
  const float* parts = reinterpret_cast<const float*>(p.workspace + tree_parts_offset());
  auto part = [&](int k) {
    return parts + (size_t)(k == cta ? 2 * cta + 1 : 2 * k) * tree_part_floats(D) + row;
  };
  float mm = -INFINITY;
  bool nan = false, weightless = false;
  for (int k = cta; k <= open.last; ++k) {
    const float* a = part(k);
    const float m = a[D * kTreeRows], l = a[(D + 1) * kTreeRows];
    mm = fmaxf(mm, m);
    nan |= !(l == l);
    weightless |= l == -1.f;
  }
  float o[COLS], ll = 0.f;
#pragma unroll
  for (int i = 0; i < COLS; ++i) o[i] = 0.f;
  for (int k = cta; k <= open.last; ++k) {
    const float* a = part(k);
    const float m = a[D * kTreeRows];
    const float f = m == -INFINITY ? 0.f : ex2(m - mm);
    if (f > 0.f) ll += f * a[(D + 1) * kTreeRows];
#pragma unroll
    for (int i = 0; i < COLS; ++i) {
      const float e = a[(warp * COLS + i) * kTreeRows];
      // part of a row without weight: nothing but non-finite values of drafts
      o[i] += f != 0.f ? f * e : (e - e == 0.f ? 0.f : e);
    }
  }
  float scale = 1.f / ll;
  if (nan || (mm == -INFINITY && weightless)) scale = __uint_as_float(0x7fc00000u);
  else if (mm == -INFINITY) scale = 0.f;
  if (r0 + row >= open.n * group) return;
  const int j = (r0 + row) / group;
  T* dst = static_cast<T*>(p.out) +
           ((size_t)(open.lo + j) * p.num_query_heads + open.g * group + (r0 + row - j * group)) * D +
           warp * COLS;
#pragma unroll
  for (int i = 0; i < COLS; i += 8) {
    uint4 w;
    w.x = Half16<T>::pack(o[i] * scale, o[i + 1] * scale);
    w.y = Half16<T>::pack(o[i + 2] * scale, o[i + 3] * scale);
    w.z = Half16<T>::pack(o[i + 4] * scale, o[i + 5] * scale);
    w.w = Half16<T>::pack(o[i + 6] * scale, o[i + 7] * scale);
    *reinterpret_cast<uint4*>(dst + i) = w;
  }
}

template <int D, typename T>
cudaError_t launch_dt(const TreeParams& p, cudaStream_t stream) {
  using C = TreeCfg<D>;
  static bool prepared[kMaxDevices] = {};  // per device: the shared-memory opt-in
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
  cfg.gridDim = dim3(grid, kTreeRows / 32);
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
