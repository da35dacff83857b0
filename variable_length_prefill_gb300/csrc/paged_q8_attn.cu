// Attention of each sequence's last tokens over an 8-bit paged cache
// (include/paged_attn_q8.h has what is computed).
//
// Bound by HBM where few query rows read a key: D bytes of keys and D of values
// for each token and KV head against 4 D operations a row.  So the codes go from
// HBM to registers once, and what is done on the way has to keep up with 24 bytes
// a clock and SM:
//
// - Half of a CTA's 16 warps copy, half compute, one for one: a copying warp keeps a ring
//   of pages in shared memory full for its computing warp, by bulk copies of a page's
//   keys and of its values.  A bulk copy costs the thread that issues it about 350
//   clocks, as much as a page's products, and copies of 16 bytes a lane hold up the
//   load pipe that the products' operands need while HBM is saturated (114 us instead
//   of 101 for the batch below), so copying is nobody's business but the copying warps'.
//   They give their registers to the others.
// - Products are warp-level ones of 16 x 8 x 16 with the tokens (or the value's
//   dimensions) as the 16 rows and eight query rows as the columns: S^T = K Q^T,
//   O^T = V^T P^T.  A decoding step has 1 to 16 query rows for a KV head; a
//   128-row tensor-memory tile would be empty for the most part, and would need the
//   codes widened through shared memory first, where here a lane's four codes are
//   two instructions away from being an operand (codes are exact in fp16).
// - The order of a page's tokens and of a piece's dimensions within a product is
//   free, as long as both operands agree.  It is chosen so that the 8 x 16-byte matrix
//   load gives a lane its operands from the cache as it lies, keys and values alike.
// - Pages that every row sees in full, all but the last few, go two at a time (one where
//   O leaves no registers) through code without masks.  The running maxima are left
//   behind by up to 2^6 before the lanes agree on new ones: one vote a page, no
//   reductions.
//
// Softmax, per query row: m is the running maximum of the scores (times log2 e), l
// the sum of 2^(s - m).  The values' scales differ from page to page and can be
// any number, so the weights of the value product are 2^(s - m + log2 v_scale - x)
// with a running maximum of their own, m + x: neither a large scale that has no
// weight nor a small one can take the others' bits.  O is the sum of weight times
// code, the row O 2^x / l.  Weights are at most 2^14 in fp16, the products' sums 32 bits.
//
// Two forms.  Few pages for each warp: it takes whole (sequence, KV head) pairs, one
// launch, nothing shared.  Else the pages of all sequences are laid end to end and cut
// into equal ranges, one for each computing warp.  A row tile inside a range is
// finished by its warp; what a range leaves open is a partial result, which at the end
// takes the place of the warp's ring.  A CTA joins those of its own warps, and a second
// launch joins what is then still open, at most two results of each CTA.
//
// Measured (captured calls; 32 query and 8 KV heads of 128, bf16, unless said): one token
// on 64 contexts of 4096, 100 us with e4m3 codes (5.4 TB/s, 79 % of a copy's bandwidth)
// and 97 with int8 ones, whose conversion is quicker; 128 contexts 187 us (85 %).  The
// start and the joins take about 12 us, and SMs differ in what they get from HBM by up
// to a third, which equal ranges do not know.  3 contexts of up to 131072, 4 tokens
// each, 40 query heads (20 rows): 151 us, bound by a page's chain of products and
// softmax at two warps a scheduler (2300 clocks for 24 rows, 450 for 8).  Four contexts of
// 128: 7.3 us, latency.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cstdint>

#include "attn_varlen_device.cuh"
#include "packed_slice.h"
#include "paged_q8_codes.cuh"
#include "paged_q8_internal.h"
#include "paged_walk.cuh"  // warp_inclusive
#include "ptx.cuh"

namespace avp {
namespace {

constexpr int kPage = kPageTokens;
constexpr float kNone = -3.0e38f;    // maximum of a row that has seen nothing
constexpr float kLeast = -200.f;     // least exponent of O (scales are 2^-149 at least)
constexpr float kSlack = 6.f;        // a maximum may be passed by this much before O is rescaled
constexpr float kBase = 8.f;         // weights are held 2^8 times as large: 2^14 at most
// Rows up to kMostRow (a query's power of two) under a softmax scale (times log2 e) up to
// kMostScale have all scores of a page below 2^kLinear if its key scale is up to
// kMostKeyScale: products of fp16 and codes are below 2^33.  What is past one of the three
// may still be an ordinary score; it takes the way of settle_scores.
constexpr int kLinear = 100;
constexpr float kMostRow = 0x1p10f, kMostScale = 0x1p20f, kMostKeyScale = 0x1p36f;
// What a row tile costs beside its pages, in pages, and a warp's range at least, in pages
// and kPartCost: 3 and 6 are the best of (1 to 4, 4 to 12) over contexts of 400 to 4096
// (2, 4: 10 % slower on 16 x 8 drafts of head size 256; 3, 8: 10 % on 2 x 4096).
constexpr int kPartCost = 3;
constexpr int kLeastUnits = 6;

constexpr int kTakers = kQ8Warps;          // warps that compute, each with a ring of its own
constexpr int kTakeThreads = 32 * kTakers;
constexpr int kThreads = 2 * kTakeThreads;  // and as many that copy, one for each

template <int D, int NT>
struct Cfg {
  static constexpr int ROWS = 8 * NT;
  static constexpr int SLOT = 2 * kPage * D;  // a page's keys, values
  static constexpr int BUDGET = 218 * 1024;
  // maxima, exponents and sums of the warps' partial results
  static constexpr int JOIN = 4 * 3 * 2 * kTakers * ROWS;
  // Registers of a thread that computes and of one that copies, 256 of each; the 512
  // start with 128.  32 rows of O want all that the copying ones can spare (8 drafts
  // of 4 heads on 64 contexts of 4096: 184 us with 224, 193 with 216), the others are
  // held up by copying threads that spill (one token each: 99 us with 216, 106 with 224).
  static constexpr int TAKE_REGS = NT == 4 ? 224 : 216, COPY_REGS = 256 - TAKE_REGS;
  // query rows as operands stay in registers, or in shared memory where O needs those
  static constexpr bool KEPT = D * NT < 512;
  static constexpr int ROWS_BYTES = KEPT ? 0 : kTakers * (D / 16) * NT * 256;
  static constexpr int PAGES = D <= 128 && D * NT <= 256 ? 2 : 1;  // that a warp takes at a time
  // a ring's stages hold that many pages each
  static constexpr int STAGE = PAGES * SLOT;
  static constexpr int FIT = (BUDGET - JOIN - ROWS_BYTES) / (kTakers * (STAGE + 16 * PAGES + 16));
  static constexpr int STAGES = FIT < 12 / PAGES ? FIT : 12 / PAGES;
  static constexpr int RING = kTakers * STAGES * STAGE;
  // of a page: two scales and whether it is there; of a stage: two barriers
  static constexpr int META = kTakers * STAGES * PAGES * 16, BARS = kTakers * STAGES * 16;
  static constexpr int BYTES = RING + ROWS_BYTES + META + BARS + JOIN;
  static_assert(STAGES >= 2, "stages");
  static_assert(ROWS <= q8_max_rows(D), "rows");
  static_assert(STAGES * STAGE >= ROWS * D * 4, "a partial result takes a ring's place");
};

// ----------------------------------------------------------------- primitives
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Bytes that `bar`'s phase is to wait for, beside its arrivals.
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Arrive on `bar` once this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copies_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// A wait that gives up after kWaitLimitNs, or when another warp of the CTA has.  The
// warp's lanes agree on what came of it.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  bool ok = mbar_try_wait(bar, parity);
  if (!__all_sync(0xffffffffu, ok)) {
    const uint64_t from = global_timer_ns();
    while (!(ok = mbar_try_wait(bar, parity))) {
      if (*abort_flag) break;
      if (global_timer_ns() - from > kWaitLimitNs) {
        atomicOr(status, kPageStatusTimeout);
        *abort_flag = 1;
        break;
      }
    }
    ok = __all_sync(0xffffffffu, ok);
  }
  return ok;
}
// Four 8 x 16-byte matrices, lane i having the address of row i % 8 of matrix i / 8:
// of each, lane i gets bytes 4 (i % 4) on of row i / 4.
__device__ __forceinline__ uint4 load_matrices(uint32_t a) {
  uint4 v;
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ float lds_float(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}

// c[16 x 8] += a[16 x 16] b[16 x 8], fp16 operands, 32-bit sums.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit elements, turned over.
__device__ __forceinline__ uint32_t turned(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t out2_of(bool fp16, float lo, float hi) {
  return fp16 ? half2_of(lo, hi) : pack_bf16x2(lo, hi);
}
__device__ __forceinline__ float nan_f() { return __uint_as_float(0x7fffffffu); }
__device__ __forceinline__ float valid_scale(float s) {
  return s >= 0.f && s <= 3.402823466e38f ? s : nan_f();
}
// 2^e for e in [-126, 127]
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// x 2^e for e in [-400, 400], without a factor that leaves 32 bits
__device__ __forceinline__ float times_exp2(float x, float e) {
  const float h = exp2f(0.5f * e);
  return x * h * h;
}

// -------------------------------------------------------------------- the walk
// A sequence's rows and tokens.
struct Seq {
  int lo, n, base, len, tiles, pages;  // base: position of its first row
};

template <int ROWS>
__device__ __forceinline__ Seq seq_of(const Q8AttnParams& p, int i, int group) {
  Seq s;
  if (p.cu) {
    const PackedSlice rows = packed_slice(__ldg(p.cu + i), __ldg(p.cu + i + 1), p.total_q);
    s.lo = rows.lo, s.n = rows.n;
  } else {
    s.lo = i, s.n = 1;
  }
  const int len = max(__ldg(p.seq_lens + i), 0);
  s.base = len - s.n;
  s.len = (int)min((long long)len, (long long)p.c.max_blocks * kPage);
  s.tiles = (s.n * group + ROWS - 1) / ROWS;
  // rows that see nothing are written too
  s.pages = max((s.len - 1) / kPage + 1, 1);
  return s;
}

// Pages [a, b) of a row tile of a sequence's KV head, of `pages` in all.
struct Part {
  Seq s;
  int seq, g, tile, a, b;
  // of the tile's rows: positions that all of them see, positions that any does
  int all, any;
  int stop;  // pages [a, stop) hold what is seen
};

template <int ROWS>
__device__ __forceinline__ void settle(Part& t, int group) {
  const int first = t.tile * ROWS / group;
  const int last = min(t.s.n - 1, (t.tile * ROWS + ROWS - 1) / group);
  t.any = min(t.s.len, t.s.base + last + 1);
  // rows past the last are as good as seeing everything: they are not written
  t.all = min(t.s.len, t.s.base + first + 1);
  t.stop = min(t.b, t.any > 0 ? (t.any - 1) / kPage + 1 : 0);
}

// A warp's range of units, part by part.  A row tile is kPartCost units that stand
// for its fixed cost, then its pages; it belongs to the range with its first page.
template <int ROWS>
struct RangeWalk {
  long long off, left;
  int seq;
  __device__ __forceinline__ bool next(const Q8AttnParams& p, int group, Part& t) {
    while (left > 0 && seq < p.c.num_seqs) {
      t.s = seq_of<ROWS>(p, seq, group);
      const int each = t.s.pages + kPartCost;
      const long long here = t.s.n > 0 ? (long long)p.c.num_kv_heads * t.s.tiles * each : 0;
      if (off >= here) {
        ++seq, off = 0;
        continue;
      }
      t.seq = seq;
      int which;  // KV head and row tile
      if (off <= INT_MAX)
        which = (int)((unsigned)off / (unsigned)each);
      else
        which = (int)(off / each);
      const int from = (int)(off - (long long)which * each);
      t.g = t.s.tiles == 1 ? which : (int)((unsigned)which / (unsigned)t.s.tiles);
      t.tile = which - t.g * t.s.tiles;
      const int to = (int)min((long long)each, from + left);
      off += to - from;
      left -= to - from;
      t.a = max(from - kPartCost, 0), t.b = max(to - kPartCost, 0);
      if (t.b == 0) continue;  // no page of it: the next range begins it
      settle<ROWS>(t, group);
      return true;
    }
    return false;
  }
};

// Whole (sequence, KV head) pairs, `step` apart, row tile by row tile.
template <int ROWS>
struct PairWalk {
  long long at, step;
  int tile;
  __device__ __forceinline__ bool next(const Q8AttnParams& p, int group, Part& t) {
    const int heads = p.c.num_kv_heads;
    for (; at < (long long)p.c.num_seqs * heads; at += step, tile = 0) {
      t.seq = at <= UINT_MAX ? (int)((unsigned)at / (unsigned)heads) : (int)(at / heads);
      t.g = (int)(at - (long long)t.seq * heads);
      t.s = seq_of<ROWS>(p, t.seq, group);
      if (t.s.n <= 0 || tile >= t.s.tiles) continue;
      t.tile = tile++;
      t.a = 0, t.b = t.s.pages;
      settle<ROWS>(t, group);
      return true;
    }
    return false;
  }
};

// ------------------------------------------------------------------ the kernel
template <int D, int NT>
struct Rows {
  static constexpr bool KEPT = Cfg<D, NT>::KEPT;
  uint32_t kept[KEPT ? NT : 1][D / 16][2];  // query rows as operands
  uint4* lane_q;                            // or where this lane has them: two operands' worth each
  float qf[NT][2];            // powers of two that the operands were divided by, rows 2 t, 2 t + 1
  float most;                 // key scales up to this leave all scores below 2^kLinear
  float m[NT][2], x[NT][2], l[NT][2];
  float o[NT][D / 16][4];
};

// The tile's query rows: lane (r = lane / 4, t = lane % 4) gets, of row r, dimensions
// 4 t to 4 t + 3 of each 16, in fp16.
template <int D, int NT>
__device__ __forceinline__ void load_rows(const Q8AttnParams& p, const Part& part, int group,
                                          Rows<D, NT>& w) {
  const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
  const uint32_t inf = p.fp16 ? 0x7c00u : 0x7f80u;
  bool large = p.scale_log2 > kMostScale;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = part.tile * (8 * NT) + nt * 8 + r, j = row / group;
    float qf = 0.f;
    uint32_t(&q)[D / 16][2] = w.kept[w.KEPT ? nt : 0];
    if (j < part.s.n) {
      const uint2* src = reinterpret_cast<const uint2*>(
          static_cast<const uint16_t*>(p.query) +
          ((size_t)(part.s.lo + j) * p.num_query_heads + part.g * group + row % group) * D);
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint2 v = __ldg(src + 4 * k + t);
        q[k][0] = v.x, q[k][1] = v.y;
        const uint32_t m = __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu);
        top = max(top, max(m & 0xffffu, m >> 16));
      }
      const uint32_t mask = 0xfu << (lane & 28);
      top = max(top, __shfl_xor_sync(mask, top, 1));
      top = max(top, __shfl_xor_sync(mask, top, 2));
      if (p.fp16) {
        qf = 1.f;
      } else {
        // the row's largest becomes 2^14 to 2^15
        const int e = max((int)(top >> 7) - 127, -110);
        const float f = __uint_as_float((uint32_t)(14 - e + 127) << 23);
        qf = __uint_as_float((uint32_t)(e - 14 + 127) << 23);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t v = q[k][h];
            q[k][h] = half2_of(__uint_as_float(v << 16) * f, __uint_as_float(v & 0xffff0000u) * f);
          }
      }
      if (top >= inf) qf = nan_f();
    } else {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) q[k][0] = q[k][1] = 0;
    }
    if constexpr (!w.KEPT) {
#pragma unroll
      for (int k = 0; k < D / 32; ++k)
        w.lane_q[(k * NT + nt) * 32] = make_uint4(q[2 * k][0], q[2 * k][1], q[2 * k + 1][0], q[2 * k + 1][1]);
    }
    __syncwarp();
    large |= qf > kMostRow;
    w.qf[nt][0] = __shfl_sync(0xffffffffu, qf, t * 8);
    w.qf[nt][1] = __shfl_sync(0xffffffffu, qf, t * 8 + 4);
#pragma unroll
    for (int e = 0; e < 2; ++e) w.m[nt][e] = kNone, w.x[nt][e] = kLeast, w.l[nt][e] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) w.o[nt][k][e] = 0.f;
  }
  w.most = __any_sync(0xffffffffu, large) ? -1.f : kMostKeyScale;
}

// x >= 0 (or NaN) as m 2^e with m below 4, added to e.
__device__ __forceinline__ float split(float x, int& e) {
  if (x < 0x1p-126f) x *= 0x1p24f, e -= 24;
  const int k = min(max((int)(__float_as_uint(x) >> 23) - 127, -126), 126);
  e += k;
  return x * power_of_two(-k);
}

// The scores of a page's products for two rows, where the row's power of two, the softmax
// scale and the key scale may be any: their exponents meet as integers, so that none is
// cut or lost before the others make up for it.  Scores past 2^kLinear in magnitude, of
// which the largest has all the weight, are folded, sixteen powers of two into one: 32 bits
// hold the order of all there can be (2^407), to 2^-19 of a score.  Beside the other
// pages' way this code costs 256 short contexts 7 % (19.4 us against 18.0 without it),
// four contexts of 128 and batches of 4096 nothing.
__device__ __forceinline__ void settle_scores(const Q8AttnParams& p, float ks, const float (&qf)[2], const float (&s)[4],
                                              float (&t)[4]) {
  constexpr uint32_t kBorder = (uint32_t)(kLinear + 127) << 23;
  int from = p.scale_exp - 127;
  const float frac = split(ks, from) * p.scale_frac;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    // in two steps: neither leaves 32 bits unless the score does.  A product is 0 or from
    // 2^-33 (fp16 times codes) to 2^33, so exponents past 240 say as much as 240
    const int exp = max(from + (int)(__float_as_uint(qf[e]) >> 23), -240), near = min(exp, 240);
    const float half = power_of_two(near >> 1), rest = power_of_two(near - (near >> 1));
    const float m = frac + (qf[e] - qf[e]);  // NaN stays
#pragma unroll
    for (int h = e; h < 4; h += 2) {
      const float x = s[h] * m, y = x * half * rest;
      // x 2^exp as bits of a number with a wider exponent, past the border's
      const uint32_t past = (__float_as_uint(x) & 0x7fffffffu) + ((uint32_t)exp << 23) - kBorder;
      const uint32_t folded = (kBorder + (past >> 4)) | (__float_as_uint(x) & 0x80000000u);
      t[h] = fabsf(y) >= __uint_as_float(kBorder) ? __uint_as_float(folded) : y;
    }
  }
}

// Of a word of e4m3 codes, bit 7 of each that is NaN.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// A product's key rows r and r + 8 are tokens token_of(r, 0) and token_of(r, 1): those of
// rows 2 t, 2 t + 1, 2 t + 8 and 2 t + 9 are tokens 4 t to 4 t + 3, and eight rows' 16-byte
// pieces lie in different banks.
__device__ __forceinline__ int token_of(int r, int upper) {
  const int u = r >> 1;
  return 4 * u + (r & 1) + 2 * (upper ^ (u >> 1));
}

// NP pages in shared memory (`slot`: their addresses, `meta`: those of their scales),
// page, page + 1, ...
// MASKED: not every row sees every token of them.
template <bool MASKED, int NP, int D, int NT, bool INT8>
__device__ __forceinline__ void take_pages(const Q8AttnParams& p, const uint32_t (&slot)[NP],
                                           const uint32_t (&meta)[NP], int page, const Part& part, int group,
                                           Rows<D, NT>& w) {
  const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
  // the products of a page's dimensions in two sums where little else is in flight
  constexpr int CHAINS = NP * NT == 1 ? 2 : 1;
  float s[NP][NT][4], s2[NP][NT][4];
#pragma unroll
  for (int i = 0; i < NP; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][nt][e] = s2[i][nt][e] = 0.f;
  // rows of two pieces: this lane's of matrix lane / 8
  const uint32_t key_row = token_of(lane & 7, (lane >> 3) & 1) * 16 + (lane >> 4) * (kPage * 16);
#pragma unroll
  for (int h = 0; h < D / 32; ++h) {
    uint4 q[NT];  // operands of two products
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if constexpr (w.KEPT)
        q[nt] = make_uint4(w.kept[nt][2 * h][0], w.kept[nt][2 * h][1], w.kept[nt][2 * h + 1][0], w.kept[nt][2 * h + 1][1]);
      else
        q[nt] = w.lane_q[(h * NT + nt) * 32];
    }
    uint4 x[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) x[i] = load_matrices(slot[i] + key_row + h * (2 * kPage * 16));
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        uint32_t f[4];
        codes_to_half<INT8>(k ? x[i].z : x[i].x, f[0], f[2]);
        codes_to_half<INT8>(k ? x[i].w : x[i].y, f[1], f[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma16816(CHAINS == 2 && k ? s2[i][nt] : s[i][nt], f, k ? q[nt].z : q[nt].x, k ? q[nt].w : q[nt].y);
      }
  }
  if constexpr (CHAINS == 2) {
#pragma unroll
    for (int e = 0; e < 4; ++e) s[0][0][e] += s2[0][0][e];
  }
  float ks[NP], lv[NP];  // the keys' scale times the softmax's
  bool extreme = false;  // factors or scores may leave 32 bits
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const float k = valid_scale(lds_float(meta[i]));
    extreme |= k > w.most;
    ks[i] = k * p.scale_log2;
    lv[i] = __log2f(valid_scale(lds_float(meta[i] + 4)));
  }
  uint32_t seen[NP];  // bit 4 nt + e: that score counts
#pragma unroll
  for (int i = 0; i < NP; ++i) seen[i] = 0;
  if constexpr (MASKED) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = (part.tile * (8 * NT) + nt * 8 + 2 * t + e) / group;
        const int limit = j < part.s.n ? min(part.s.len, part.s.base + j + 1) : 0;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int pos = (page + i) * kPage;
          seen[i] |= (pos + token_of(r, 0) < limit ? 1u : 0u) << (4 * nt + e) |
                     (pos + token_of(r, 1) < limit ? 4u : 0u) << (4 * nt + e);
        }
      }
  }
  uint32_t pw[NP][NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float f[NP][2], d[NP][4];
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) f[i][e] = ks[i] * w.qf[nt][e];
    auto unseen = [&](int i, int e) { return MASKED && !(seen[i] >> (4 * nt + e) & 1); };
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        d[i][e] = fmaf(s[i][nt][e], f[i][e & 1], -w.m[nt][e & 1]);
        if (unseen(i, e)) d[i][e] = -INFINITY;
      }
    // A maximum may be passed by kSlack before anything is rescaled, so that the
    // lanes need not agree on one for every page.
    bool up = extreme;
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float over = fmaxf(d[i][e], d[i][e + 2]);
        up |= over > kSlack || over + lv[i] > w.x[nt][e] + kSlack;
      }
    if (__any_sync(0xffffffffu, up)) {
      // The scores as rounded products, as the maxima are: what the rounding cuts, half
      // a last bit, passes any slack from 2^27 on.
      float t[NP][4];
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) t[i][e] = __fmul_rn(s[i][nt][e], f[i][e & 1]);
      if (extreme) {
#pragma unroll
        for (int i = 0; i < NP; ++i) settle_scores(p, valid_scale(lds_float(meta[i])), w.qf[nt], s[i][nt], t[i]);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // of the scores themselves: they may vanish beside the first maximum, kNone
        float top[NP], m = w.m[nt][e];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const float a = unseen(i, e) ? -INFINITY : t[i][e];
          const float b = unseen(i, e + 2) ? -INFINITY : t[i][e + 2];
          top[i] = fmaxf(a, b);
#pragma unroll
          for (int h = 4; h < 32; h <<= 1) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], h));
          m = fmaxf(m, top[i]);
        }
        const float down = w.m[nt][e] - m;
        float x = fmaxf(w.x[nt][e] + down, kLeast);
#pragma unroll
        for (int i = 0; i < NP; ++i) x = fmaxf(x, (top[i] - m) + lv[i]);
        const float fo = ex2((w.x[nt][e] + down) - x);
        w.l[nt][e] *= ex2(down);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) w.o[nt][k][e] *= fo, w.o[nt][k][e + 2] *= fo;
        w.m[nt][e] = m;
        w.x[nt][e] = x;
      }
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          d[i][e] = unseen(i, e) ? -INFINITY : t[i][e] - w.m[nt][e & 1];
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      float pv[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w.l[nt][e & 1] += ex2(d[i][e]);
        pv[e] = ex2(d[i][e] + (lv[i] - w.x[nt][e & 1] + kBase));
        if (unseen(i, e)) pv[e] = 0.f;
      }
      // rows 2 t, 2 t + 1 and 2 t + 8, 2 t + 9 of this lane's column, as tokens 4 t on
      const uint32_t lower = turned(half2_of(pv[0], pv[1])), upper = turned(half2_of(pv[2], pv[3]));
      pw[i][nt][0] = t < 2 ? lower : upper;
      pw[i][nt][1] = t < 2 ? upper : lower;
    }
  }
  const uint32_t value_row = kPage * D + lane * kPage;  // of 32 dimensions
  if constexpr (!MASKED) {
#pragma unroll
    for (int k = 0; k < D / 16; k += 2)
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const uint4 x = load_matrices(slot[i] + value_row + k * 256);
        uint32_t f[4];
        codes_to_half<INT8>(x.x, f[0], f[2]);
        codes_to_half<INT8>(x.y, f[1], f[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(w.o[nt][k], f, pw[i][nt][0], pw[i][nt][1]);
        codes_to_half<INT8>(x.z, f[0], f[2]);
        codes_to_half<INT8>(x.w, f[1], f[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(w.o[nt][k + 1], f, pw[i][nt][0], pw[i][nt][1]);
      }
  } else {
    // Tokens that no row sees are cleared.  A weight of 0 does not silence a NaN, so
    // NaN codes are cleared as well, and a product of their places with who sees
    // what tells which results they reach.
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int live = min(max(part.any - (page + i) * kPage - 4 * t, 0), 4);
      const uint32_t live_mask = live == 4 ? 0xffffffffu : (1u << (8 * live)) - 1u;
      uint32_t who[NT][2];
      if constexpr (!INT8) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t bits = seen[i] >> (4 * nt);
          const uint32_t lower = turned((bits & 1 ? 0x3c00u : 0u) | (bits & 2 ? 0x3c000000u : 0u));
          const uint32_t upper = turned((bits & 4 ? 0x3c00u : 0u) | (bits & 8 ? 0x3c000000u : 0u));
          who[nt][0] = t < 2 ? lower : upper;
          who[nt][1] = t < 2 ? upper : lower;
        }
      }
#pragma unroll
      for (int k2 = 0; k2 < D / 32; ++k2) {
        const uint4 x = load_matrices(slot[i] + value_row + k2 * 512);
#pragma unroll
        for (int k1 = 0; k1 < 2; ++k1) {
          const int k = 2 * k2 + k1;
          uint32_t a = (k1 ? x.z : x.x) & live_mask, b = (k1 ? x.w : x.y) & live_mask;
          uint32_t f[4];
          if constexpr (!INT8) {
            const uint32_t na = nan_codes(a), nb = nan_codes(b);
            if (__any_sync(0xffffffffu, (na | nb) != 0u)) {
              codes_to_half<false>((na >> 7) * 0x38u, f[0], f[2]);  // 0x38 is 1
              codes_to_half<false>((nb >> 7) * 0x38u, f[1], f[3]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float c[4] = {0.f, 0.f, 0.f, 0.f};
                mma16816(c, f, who[nt][0], who[nt][1]);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (c[e] > 0.f) w.o[nt][k][e] = nan_f();
              }
              a &= ~((na >> 7) * 0xffu);
              b &= ~((nb >> 7) * 0xffu);
            }
          }
          codes_to_half<INT8>(a, f[0], f[2]);
          codes_to_half<INT8>(b, f[1], f[3]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(w.o[nt][k], f, pw[i][nt][0], pw[i][nt][1]);
        }
      }
    }
  }
}

// What a copying warp does: the pages of its walk in order, into the stages of one
// computing warp's ring as they come free.  Ids are read 32 at a time.  Returns how
// many stages it filled.
template <int D, int NT, class Walk>
__device__ __forceinline__ int copy_pages(const Q8AttnParams& p, Walk walk, int group, uint32_t ring, uint32_t metas,
                                           uint32_t bars, volatile int* abort_flag) {
  using C = Cfg<D, NT>;
  const int lane = threadIdx.x & 31;
  const uint8_t* const keys = static_cast<const uint8_t*>(p.c.k_cache);
  const uint8_t* const values = static_cast<const uint8_t*>(p.c.v_cache);
  const float* const scales = lane ? p.v_scale : p.k_scale;
  int stage = 0, issued = 0;
  uint32_t parity = 1;  // of the stages' empty phases: the first time round they are
  Part part;
  while (walk.next(p, group, part)) {
    const int32_t* table = p.block_tables + (size_t)part.seq * p.c.max_blocks;
    int ids = 0, known = 0;  // pages of the part whose ids the lanes have (32 from a multiple of 32 on)
    for (int page = part.a; page < part.stop; page += C::PAGES) {
      const uint32_t full = bars + 16 * stage;
      const uint32_t meta = metas + 16 * C::PAGES * stage, at = ring + stage * C::STAGE;
      bool waited = false;
#pragma unroll
      for (int i = 0; i < C::PAGES; ++i) {
        const int n = page - part.a + i;
        if (page + i >= part.stop) break;
        if (n >= known) {
          ids = part.a + n + lane < part.stop ? __ldg(table + part.a + n + lane) : 0;
          known = n + 32;
        }
        const int id = __shfl_sync(0xffffffffu, ids, n & 31);
        const bool good = id >= 0 && id < p.c.num_blocks;
        if (!waited && !wait_for(full + 8, parity, abort_flag, p.c.status)) return issued;
        waited = true;
#if ATTN_VARLEN_TEST_HOOKS
        if (p.test_withhold && blockIdx.x == 0 && page == part.a) return issued;  // never announced
#endif
        if (lane == 0)
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(meta + 16 * i + 8), "r"((uint32_t)good) : "memory");
        if (good) {
          const size_t which = (size_t)id * p.c.num_kv_heads + part.g;
          if (lane == 0) {
            mbar_expect_tx(full, C::SLOT);
            bulk_copy_g2s(at + i * C::SLOT, keys + which * (kPage * D), kPage * D, full);
            bulk_copy_g2s(at + i * C::SLOT + kPage * D, values + which * (kPage * D), kPage * D, full);
          }
          if (lane < 2) copy4(meta + 16 * i + lane * 4, scales + which);
        } else if (lane == 0) {
          atomicOr(p.c.status, kPageStatusBadBlock);
        }
      }
      if (lane < 2) copies_arrive(full);
      if (lane == 0) mbar_arrive(full);  // the marks above are there
      ++issued;
      if (++stage == C::STAGES) stage = 0, parity ^= 1;
    }
  }
  return issued;
}

// A row tile's rows, finished by one warp.
template <int D, int NT>
__device__ __forceinline__ void write_rows(const Q8AttnParams& p, const Part& part, int group,
                                           Rows<D, NT>& w) {
  const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float f[2], x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = w.l[nt][e];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
      f[e] = l == 0.f ? 0.f : 1.f / l;  // NaN passes
      x[e] = w.x[nt][e] - kBase;
    }
    const int row = part.tile * (8 * NT) + nt * 8 + r, j = row / group;
    uint32_t* dst = reinterpret_cast<uint32_t*>(
        static_cast<uint16_t*>(p.out) +
        ((size_t)(part.s.lo + j) * p.num_query_heads + part.g * group + row % group) * D);
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t v = turned(out2_of(p.fp16, times_exp2(w.o[nt][k][2 * h] * f[0], x[0]),
                                                times_exp2(w.o[nt][k][2 * h + 1] * f[1], x[1])));
        if (j < part.s.n) dst[k * 8 + h * 4 + t] = v;
      }
  }
}

// -------------------------------------------------------------- partial results
// What a warp's range leaves open: the row tile that it goes on with (head), and the
// one that it begins and does not end (tail).
struct Pieces {
  int head, head_ends;  // the head, and whether the row tile ends in this range
  int tail;
  int last_piece;       // 0: the head, 1: the tail is in the place of the warp's ring
  int lo, n, g, tile;   // the tail's row tile
  int last;             // and the CTA that holds its end
};

// Shared memory for it, after the rings: maxima, exponents and sums of piece 2 warp +
// (0: head, 1: tail).
template <int D, int NT>
struct PieceSums {
  static constexpr int N = 2 * kTakers, ROWS = 8 * NT;
  float m[N][ROWS], x[N][ROWS], l[N][ROWS];
};

// Piece `i` of CTA `cta` in the workspace: O [rows][D] after the three numbers of each row.
template <int D, int ROWS>
__device__ __forceinline__ float* piece_at(const Q8AttnParams& p, int cta, int i) {
  return reinterpret_cast<float*>(p.workspace + q8_parts_offset()) +
         ((size_t)cta * (2 * kTakers) + i) * q8_part_floats(D, ROWS);
}

// Where element d of a row's O is, in floats, for a piece in the place of a ring: the
// lanes that put it down, 8 dimensions of every other row, meet no bank twice.
template <int D>
__device__ __forceinline__ int ring_place(int row, int d) {
  return row * D + (d ^ ((row >> 1 & 3) * 8));
}

// The piece goes to the workspace while the ring is in use, and to the ring (`own`)
// at the end of the warp's range.
template <int D, int NT>
__device__ __forceinline__ void put_piece(const Q8AttnParams& p, int i, Rows<D, NT>& w,
                                          PieceSums<D, NT>& sums, float* own) {
  const int lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
  float* o = piece_at<D, 8 * NT>(p, blockIdx.x, i) + 4 * 8 * NT;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float l = w.l[nt][e];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
      if (r == 0) {
        const int row = nt * 8 + 2 * t + e;
        sums.m[i][row] = w.m[nt][e], sums.x[i][row] = w.x[nt][e], sums.l[i][row] = l;
      }
    }
    if (own) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          own[ring_place<D>(nt * 8 + 2 * t + (e & 1), k * 16 + (e >> 1) * 8 + r)] = w.o[nt][k][e];
    } else {
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[(nt * 8 + 2 * t + (e & 1)) * D + k * 16 + (e >> 1) * 8 + r] = w.o[nt][k][e];
    }
  }
}

// A lane's D / 32 neighbouring elements of a row of O.
template <int D>
__device__ __forceinline__ void load_part(const float* row, float (&v)[D / 32]) {
  constexpr int E = D / 32;
  const float* at = row + (threadIdx.x & 31) * E;
  if constexpr (E == 2) {
    const float2 a = *reinterpret_cast<const float2*>(at);
    v[0] = a.x, v[1] = a.y;
  } else {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      const float4 a = reinterpret_cast<const float4*>(at)[i];
      v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = a.z, v[4 * i + 3] = a.w;
    }
  }
}

// A finished row: O 2^x / l in 16 bits.
template <int D>
__device__ __forceinline__ void write_row(const Q8AttnParams& p, int lo, int g, int group, int at,
                                          const float (&o)[D / 32], float x, float l) {
  constexpr int E = D / 32;
  const float f = l == 0.f ? 0.f : 1.f / l;  // NaN passes
  uint32_t* dst = reinterpret_cast<uint32_t*>(
                      static_cast<uint16_t*>(p.out) +
                      ((size_t)(lo + at / group) * p.num_query_heads + g * group + at % group) * D) +
                  (threadIdx.x & 31) * (E / 2);
#pragma unroll
  for (int e = 0; e < E; e += 2)
    dst[e / 2] = out2_of(p.fp16, times_exp2(o[e] * f, x - kBase), times_exp2(o[e + 1] * f, x - kBase));
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

// The CTA's warps have put down their pieces.  In the order head of warp 0, tail of
// warp 0, head of warp 1, ..., the pieces of one row tile are neighbours: a tail and
// the heads behind it, or the first heads of the CTA.  They are joined; a row tile
// that begins and ends here is written, another leaves one piece, in the place of its
// first, and a record for the second launch.
template <int D, int NT>
__device__ __forceinline__ void join_pieces(const Q8AttnParams& p, int group, const Pieces* pieces,
                                            PieceSums<D, NT>& sums, const uint8_t* rings) {
  constexpr int ROWS = 8 * NT, N = 2 * kTakers;
  constexpr int EACH = (N * ROWS + kTakeThreads - 1) / kTakeThreads;
  using C = Cfg<D, NT>;
  const int tid = threadIdx.x, lane = tid & 31;
  // bits of pieces: those there are, those that begin a row tile here, heads that end
  // one, those in the place of a ring
  const Pieces& mine = pieces[(lane & 15) >> 1];
  const bool is = lane < N && (lane & 1 ? mine.tail : mine.head);
  const uint32_t there = __ballot_sync(0xffffffffu, is);
  const uint32_t begins = __ballot_sync(0xffffffffu, is && (lane & 1)) | (there & (0u - there));
  const uint32_t ends = __ballot_sync(0xffffffffu, is && !(lane & 1) && mine.head_ends);
  const uint32_t in_ring = __ballot_sync(0xffffffffu, is && mine.last_piece == (lane & 1));
  // the pieces of piece i's row tile
  auto tile_of = [&](int i) {
    const uint32_t upto = (2u << i) - 1u;
    const int first = 31 - __clz(begins & upto);
    const uint32_t behind = begins & ~upto;
    const uint32_t until = behind ? (behind & (0u - behind)) - 1u : ~0u;
    return there & until & ~((1u << first) - 1u);
  };
  if (tid == 0) {
    Q8Open open = {};
    // a tail whose row tile does not end here is the last that begins
    const int i = there ? 31 - __clz(begins) : 0;
    if (there && (i & 1) && !(tile_of(i) & ends)) {
      const Pieces& q = pieces[i >> 1];
      open.valid = 1;
      open.lo = q.lo, open.n = q.n, open.g = q.g, open.tile = q.tile;
      open.last = q.last;
      open.tail_piece = i;
    }
    reinterpret_cast<Q8Open*>(p.workspace)[blockIdx.x] = open;
  }
  // Of a piece and a row: the factor that brings it to its row tile's maximum and
  // exponent takes the place of x; at a row tile's first piece these, and the sum, take
  // the places of m and l, and go to the workspace with a piece that stays.
  float factor[EACH], top[EACH], exponent[EACH], total[EACH];
#pragma unroll
  for (int j = 0; j < EACH; ++j) {
    const int item = j * kTakeThreads + tid, i = item / ROWS, row = item % ROWS;
    factor[j] = top[j] = exponent[j] = total[j] = 0.f;
    if (item >= N * ROWS || !(there >> i & 1)) continue;
    const uint32_t tile = tile_of(i);
    float m = kNone, x = kLeast, l = 0.f;
    for (uint32_t left = tile; left; left &= left - 1) m = fmaxf(m, sums.m[__ffs(left) - 1][row]);
    for (uint32_t left = tile; left; left &= left - 1) {
      const int k = __ffs(left) - 1;
      const float down = sums.m[k][row] - m;
      x = fmaxf(x, sums.x[k][row] + down);
      l += sums.l[k][row] * ex2(down);
    }
    factor[j] = ex2((sums.x[i][row] + (sums.m[i][row] - m)) - x);
    top[j] = m, exponent[j] = x, total[j] = l;
  }
  named_bar_sync(1, kTakeThreads);
#pragma unroll
  for (int j = 0; j < EACH; ++j) {
    const int item = j * kTakeThreads + tid, i = item / ROWS, row = item % ROWS;
    if (item >= N * ROWS || !(there >> i & 1)) continue;
    sums.x[i][row] = factor[j];
    if (begins >> i & 1) {
      sums.m[i][row] = exponent[j], sums.l[i][row] = total[j];
      float* to = piece_at<D, ROWS>(p, blockIdx.x, i);
      to[row] = top[j], to[ROWS + row] = exponent[j], to[2 * ROWS + row] = total[j];
    }
  }
  named_bar_sync(1, kTakeThreads);
  // row tile by row tile, four neighbouring elements of O for each thread and item, the
  // loads of four pieces at a time (this code runs once and comes from memory: short
  // loops, not unrolled ones)
  constexpr int ALL = ROWS * D / 4, ITEMS = (ALL + kTakeThreads - 1) / kTakeThreads;
  auto none = [&](int j) { return ALL % kTakeThreads != 0 && j * kTakeThreads + tid >= ALL; };
  float* const base = piece_at<D, ROWS>(p, blockIdx.x, 0) + 4 * ROWS + tid * 4;
#pragma unroll 1
  for (uint32_t firsts = begins; firsts; firsts &= firsts - 1) {
    const int first = __ffs(firsts) - 1;
    const uint32_t tile = tile_of(first);
    float4 sum[ITEMS];
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) sum[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (uint32_t left = tile; left;) {
      int at[4];
      float4 v[4][ITEMS];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        at[k] = __ffs(left) - 1;
        left &= left - 1;
        if (at[k] < 0) continue;
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
          const int item = j * kTakeThreads + tid;
          if (none(j)) continue;
          v[k][j] = *reinterpret_cast<const float4*>(
              in_ring >> at[k] & 1
                  ? reinterpret_cast<const float*>(rings + (at[k] >> 1) * (C::STAGES * C::STAGE)) +
                        ring_place<D>(item / (D / 4), item % (D / 4) * 4)
                  : base + at[k] * q8_part_floats(D, ROWS) + j * kTakeThreads * 4);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (at[k] < 0) continue;
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
          if (none(j)) continue;
          const float f = sums.x[at[k]][(j * kTakeThreads + tid) / (D / 4)];
          sum[j].x += f * v[k][j].x, sum[j].y += f * v[k][j].y;
          sum[j].z += f * v[k][j].z, sum[j].w += f * v[k][j].w;
        }
      }
    }
    const bool whole = (first & 1) && (tile & ends);
    const bool moved = (tile & (tile - 1)) != 0 || (in_ring >> first & 1);  // from where it was put
    const Pieces& q = pieces[first >> 1];
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      const int item = j * kTakeThreads + tid, row = item / (D / 4), d = item % (D / 4) * 4;
      if (none(j)) continue;
      if (!whole) {
        if (moved) *reinterpret_cast<float4*>(base + first * q8_part_floats(D, ROWS) + j * kTakeThreads * 4) = sum[j];
        continue;
      }
      const int tile_row = q.tile * ROWS + row, n = tile_row / group;
      if (n >= q.n) continue;
      const float l = sums.l[first][row], h = exp2f(0.5f * (sums.m[first][row] - kBase));
      const float g = l == 0.f ? 0.f : h / l;  // NaN passes
      uint2 r;
      r.x = out2_of(p.fp16, sum[j].x * g * h, sum[j].y * g * h);
      r.y = out2_of(p.fp16, sum[j].z * g * h, sum[j].w * g * h);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) +
                                ((size_t)(q.lo + n) * p.num_query_heads + q.g * group + tile_row % group) * D + d) = r;
    }
  }
}

// ------------------------------------------------------------------ the kernel
struct RangeScratch {
  long long sum[kThreads / 32];
  long long off[kTakers];
  int seq[kTakers];
};

// Units cut into `parts` ranges that differ by one unit at most: the first `more` of
// them have `each` + 1, the others `each`.
struct Cut {
  long long each;
  int more, parts;
  __device__ __forceinline__ long long begin(int i) const { return i * each + min(i, more); }
  // the range that holds unit u
  __device__ __forceinline__ int holder(long long u) const {
    const long long longer = more * (each + 1);
    return u < longer ? (int)(u / (each + 1)) : more + (int)((u - longer) / each);
  }
};

// The units of all sequences in equal ranges, one for each CTA (as far as there are
// kLeastUnits for each), and a CTA's in equal ranges for its warps, or for a half, a
// quarter, ... of them.
template <int ROWS>
__device__ __forceinline__ void locate_ranges(const Q8AttnParams& p, int group, RangeScratch& s,
                                              Cut& cut, long long& stop, RangeWalk<ROWS>& walk) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = p.c.num_seqs;
  const int run = (n + kThreads - 1) / kThreads;
  const int a = min(n, tid * run), b = min(n, a + run);
  auto units = [&](int i) -> long long {
    const Seq q = seq_of<ROWS>(p, i, group);
    return q.n > 0 ? (long long)p.c.num_kv_heads * q.tiles * (q.pages + kPartCost) : 0;
  };
  long long sum = 0;
  for (int i = a; i < b; ++i) sum += units(i);
  const long long inc = warp_inclusive(sum, lane);
  if (lane == 31) s.sum[warp] = inc;
  if (tid < kTakers) s.seq[tid] = n, s.off[tid] = 0;
  __syncthreads();
  long long before = inc - sum, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += s.sum[w];
    total += s.sum[w];
  }
  cut.parts = (int)min((long long)gridDim.x, max(total / kLeastUnits, min(total, 1LL)));
  if (cut.parts == 0) cut.parts = 1;
  // both fit 32 bits for all but the largest calls
  cut.each = total <= UINT_MAX ? (unsigned)total / (unsigned)cut.parts : total / cut.parts;
  cut.more = (int)(total - cut.each * cut.parts);
  const int c = blockIdx.x;
  const long long begin = c < cut.parts ? cut.begin(c) : total;
  const long long length = c < cut.parts ? cut.begin(c + 1) - begin : 0;
  int shift = 3;
  while (shift > 0 && length < (long long)kLeastUnits << shift) --shift;
  auto start = [&](int w) { return begin + (w >> shift ? length : length * w >> shift); };
  if (before < begin + length && begin < before + sum) {  // some start may lie in this thread's run
    for (int w = 0; w < 1 << shift; ++w) {
      const long long u = start(w);
      if (before <= u && u < before + sum) {
        long long at = before;
        for (int i = a; i < b; ++i) {
          const long long here = units(i);
          if (u < at + here) {
            s.seq[w] = i;
            s.off[w] = u - at;
            break;
          }
          at += here;
        }
      }
    }
  }
  __syncthreads();
  const int mine = warp % kTakers;
  walk.seq = s.seq[mine], walk.off = s.off[mine];
  stop = start(mine + 1);
  walk.left = stop - start(mine);
}

template <int D, int NT, bool INT8, bool RANGES>
__global__ void __launch_bounds__(kThreads, 1) q8_attn_kernel(const __grid_constant__ Q8AttnParams p) {
  using C = Cfg<D, NT>;
  using Walk = typename std::conditional<RANGES, RangeWalk<C::ROWS>, PairWalk<C::ROWS>>::type;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ RangeScratch scratch;
  __shared__ Pieces pieces[kTakers];
  __shared__ volatile int abort_flag;
  __shared__ volatile int issued[kTakers];  // stages that were filled, once that is known
  const int lane = threadIdx.x & 31, role = threadIdx.x / kTakeThreads, warp = (threadIdx.x >> 5) % kTakers;
  const int group = p.group;
  const uint32_t ring = smem_u32(smem) + warp * (C::STAGES * C::STAGE);
  const uint32_t metas = smem_u32(smem) + C::RING + C::ROWS_BYTES + warp * (C::STAGES * C::PAGES * 16);
  const uint32_t bars = smem_u32(smem) + C::RING + C::ROWS_BYTES + C::META + warp * (C::STAGES * 16);  // of each slot: full, empty
  if (threadIdx.x == 0) abort_flag = 0;
  if (role == 0 && lane == 0) {
    for (int i = 0; i < C::STAGES; ++i) mbar_init(bars + 16 * i, 3), mbar_init(bars + 16 * i + 8, 1);
    fence_mbar_init();
    pieces[warp] = Pieces{};
    pieces[warp].last_piece = -1;
    issued[warp] = -1;
  }
  __syncthreads();
  Walk walk;
  Cut cut = {};
  long long end = 0;  // of the warp's range
  // launched while the kernel before it ends: nothing is read or written before this
  grid_wait_prerequisite();
  if constexpr (RANGES) {
    grid_launch_dependents();
    locate_ranges<C::ROWS>(p, group, scratch, cut, end, walk);
  } else {
    walk.at = (long long)warp * gridDim.x + blockIdx.x;  // few pairs: on different SMs
    walk.step = (long long)gridDim.x * kTakers;
    walk.tile = 0;
  }
  if (role == 1) {
    fewer_registers<C::COPY_REGS>();
    const int n = copy_pages<D, NT, Walk>(p, walk, group, ring, metas, bars, &abort_flag);
    if (lane == 0) issued[warp] = n;
    copies_wait_all();
    return;
  }
  more_registers<C::TAKE_REGS>();
  PieceSums<D, NT>& sums = *reinterpret_cast<PieceSums<D, NT>*>(smem + C::RING + C::ROWS_BYTES + C::META + C::BARS);
  int stage = 0;
  uint32_t parity = 0;  // of the stages' full phases
  int taken = 0;        // stages
  bool dead = false;
  Part part;
  Rows<D, NT> w;
  float* const own = reinterpret_cast<float*>(smem + warp * (C::STAGES * C::STAGE));
  w.lane_q = reinterpret_cast<uint4*>(smem + C::RING) + warp * ((D / 32) * NT * 32) + lane;
  while (!dead && walk.next(p, group, part)) {
    load_rows<D, NT>(p, part, group, w);
    for (int page = part.a; page < part.stop; page += C::PAGES) {
      const uint32_t bar = bars + 16 * stage;
      if (!wait_for(bar, parity, &abort_flag, p.c.status)) {
        dead = true;
        break;
      }
      uint32_t slots[C::PAGES], meta[C::PAGES], there[C::PAGES];
      bool all = page + C::PAGES <= part.stop;
#pragma unroll
      for (int i = 0; i < C::PAGES; ++i) {
        slots[i] = ring + stage * C::STAGE + i * C::SLOT, meta[i] = metas + 16 * (C::PAGES * stage + i);
        there[i] = page + i < part.stop ? __float_as_uint(lds_float(meta[i] + 8)) : 0u;
      }
#pragma unroll
      for (int i = 0; i < C::PAGES; ++i) all = all && there[i];
      if (all && (page + C::PAGES) * kPage <= part.all) {
        take_pages<false, C::PAGES, D, NT, INT8>(p, slots, meta, page, part, group, w);
      } else {
#pragma unroll 1
        for (int i = 0; i < C::PAGES; ++i) {
          const uint32_t one_slot[1] = {slots[0] + i * C::SLOT}, one_meta[1] = {meta[0] + 16 * i};
          if (i == 0 ? there[0] : there[C::PAGES - 1])
            take_pages<true, 1, D, NT, INT8>(p, one_slot, one_meta, page + i, part, group, w);
        }
      }
      fence_proxy_async_smem();  // the stage is read before copies write it again
      __syncwarp();
      if (lane == 0) mbar_arrive(bar + 8);
      ++taken;
      if (++stage == C::STAGES) stage = 0, parity ^= 1;
    }
    if (dead) break;
    if constexpr (RANGES) {
      const bool ends = part.b == part.s.pages;
      if (part.a > 0) {
        const bool last = walk.left <= 0;
        put_piece<D, NT>(p, 2 * warp, w, sums, last ? own : nullptr);
        if (lane == 0) pieces[warp].head = 1, pieces[warp].head_ends = ends, pieces[warp].last_piece = last ? 0 : -1;
      } else if (!ends) {
        put_piece<D, NT>(p, 2 * warp + 1, w, sums, own);
        if (lane == 0) {
          Pieces& q = pieces[warp];
          q.tail = 1, q.last_piece = 1;
          q.lo = part.s.lo, q.n = part.s.n, q.g = part.g, q.tile = part.tile;
          q.last = cut.holder(end + (part.s.pages - part.b) - 1);  // of its last unit
        }
      } else {
        write_rows<D, NT>(p, part, group, w);
      }
    } else {
      write_rows<D, NT>(p, part, group, w);
    }
  }
  if (dead) {  // a wait ran out: copies that are under way end before the CTA does
    const uint64_t from = global_timer_ns();
    auto late = [&] { return global_timer_ns() - from > kWaitLimitNs; };
    while (issued[warp] < 0 && !late()) {
    }
    for (const int all = issued[warp]; taken < all; ++taken) {
      while (!mbar_try_wait(bars + 16 * stage, parity) && !late()) {
      }
      if (++stage == C::STAGES) stage = 0, parity ^= 1;
    }
  }
  if constexpr (RANGES) {
    named_bar_sync(1, kTakeThreads);
    join_pieces<D, NT>(p, group, pieces, sums, smem);
  }
}

// ------------------------------------------------------------ the second launch
// A row tile that CTA b left open: its tail, and the heads of the CTAs behind it up to
// `last`.  A CTA joins four rows, two warps share the pieces of each (there are two,
// unless a row tile is longer than a CTA's range).  Bound by latency: the record, then
// everything else at once.
constexpr int kJoinRows = 4, kJoinWays = 2;
constexpr int kJoinThreads = 32 * kJoinRows * kJoinWays;

template <int D, int NT>
__global__ void __launch_bounds__(kJoinThreads, 4) q8_join_kernel(const __grid_constant__ Q8AttnParams p) {
  constexpr int ROWS = 8 * NT, E = D / 32;
  __shared__ float s_o[kJoinWays][kJoinRows][D];
  grid_launch_dependents();
  grid_wait_prerequisite();
  const Q8Open* opens = reinterpret_cast<const Q8Open*>(p.workspace);
  const Q8Open o = opens[blockIdx.x];
  const int group = p.group;
  if (!o.valid) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = warp % kJoinRows, way = warp / kJoinRows;
  const int row = blockIdx.y * kJoinRows + r, at = o.tile * ROWS + row;
  const int count = o.last - (int)blockIdx.x + 1;
  auto piece = [&](int i) -> const float* {
    return i == 0 ? piece_at<D, ROWS>(p, blockIdx.x, o.tail_piece)
                  : piece_at<D, ROWS>(p, blockIdx.x + i, 0);
  };
  float top = kNone, exponent = kLeast, l = 0.f;
  float sum[E];
#pragma unroll
  for (int e = 0; e < E; ++e) sum[e] = 0.f;
  if (at / group < o.n) {
    float v[E];  // this warp's first piece, on its way while the factors are found
    if (way < count) load_part<D>(piece(way) + 4 * ROWS + row * D, v);
    for (int i = lane; i < count; i += 32) {
      const float* q = piece(i);
      // a running join of this lane's pieces
      const float m = fmaxf(top, q[row]), down = top - m, other = q[row] - m;
      exponent = fmaxf(fmaxf(exponent + down, q[ROWS + row] + other), kLeast);
      l = l * ex2(down) + q[2 * ROWS + row] * ex2(other);
      top = m;
    }
    const float m = warp_max(top);
    exponent = warp_max(fmaxf(exponent + (top - m), kLeast));
    l = warp_sum(l * ex2(top - m));
    top = m;
#pragma unroll 4
    for (int i = way; i < count; i += kJoinWays) {
      const float* q = piece(i);
      const float by = ex2((q[ROWS + row] + (q[row] - top)) - exponent);
      if (i != way) load_part<D>(q + 4 * ROWS + row * D, v);
#pragma unroll
      for (int e = 0; e < E; ++e) sum[e] += by * v[e];
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[way][r][lane * E + e] = sum[e];
  __syncthreads();
  if (way == 0 && at / group < o.n) {
#pragma unroll
    for (int i = 1; i < kJoinWays; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) sum[e] += s_o[i][r][lane * E + e];
    write_row<D>(p, o.lo, o.g, group, at, sum, exponent, l);
  }
}

// ------------------------------------------------------------------ launches
constexpr int kMaxDevices = 64;

// `prepared`, by device, is read by callers of several threads; two may both set the attribute.
template <class K>
cudaError_t opt_in(K kernel, int bytes, std::atomic<bool>* prepared) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!prepared[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    prepared[dev] = true;
  }
  return cudaSuccess;
}

// Whether whole pairs are quicker than ranges, from what the host knows: counts and the
// table's width, no lengths.  A pair's row tiles are one warp's, each about 6 pages' time
// beside its pages (those of the longest table row); warps go round the pairs, and one
// sequence may have all the rows that cu_seqlens hands out.  Ranges cost 24 pages' time for
// two launches and the joins, and 3 a row tile.  A page alone takes a warp 0.44 us.
//
// Both sides take the table for full, so a context that is much longer than the others
// would be one warp's alone behind a wide table: kPairPages is where batches of 1 token to
// the table's width turn.  Measured, one token each, 8 KV heads, pairs | ranges, us: 152
// contexts of 1 to 1024 tokens 41 | 52, to 1536 59 | 65, to 2048 76 | 73; 304 of them 76 |
// 80, 110 | 103, 144 | 123; one of 1024, 1536 or 2048 among 151 of 100 32 | 23, 46 | 23, 60 |
// 23, and one of 65536 1786 | 48.  256 x 16 pairs of up to 4 pages 19 | 31, 64 x 8 of up to 25
// 15 | 20, 4 x 8 of 9 7.7 | 11; the same behind tables of 64 pages and more, and the first
// with cu_seqlens, take ranges.
constexpr int kPairPages = 96;

bool pairs_are_quicker(const Q8AttnParams& p, long long rows, int tile_rows) {
  const long long pairs = (long long)p.c.num_seqs * p.c.num_kv_heads, pages = p.c.max_blocks;
  if (pages > kPairPages) return false;
  const long long warps = (long long)kTakers * p.c.sm_count;
  const long long tiles = (rows + tile_rows - 1) / tile_rows;  // of a pair, on average
  const long long most = ((p.cu ? (long long)p.total_q : 1) * p.group + tile_rows - 1) / tile_rows;
  return std::max((pairs + warps - 1) / warps * tiles, most) * (pages + 6) <=
         24 + pairs * tiles * (pages + 3) / warps;
}

// Behind what is on the stream, started while that ends (the kernels wait for it).
template <class K>
cudaError_t launch_behind(K kernel, dim3 grid, int threads, int bytes, const Q8AttnParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, int NT, bool INT8>
cudaError_t launch_nt(const Q8AttnParams& p, long long rows, cudaStream_t stream) {
  using C = Cfg<D, NT>;
  if (pairs_are_quicker(p, rows, C::ROWS)) {
    static std::atomic<bool> prepared[kMaxDevices] = {};
    const cudaError_t e = opt_in(q8_attn_kernel<D, NT, INT8, false>, C::BYTES, prepared);
    if (e != cudaSuccess) return e;
    const long long pairs = (long long)p.c.num_seqs * p.c.num_kv_heads;
    const int grid = (int)std::min<long long>(pairs, p.c.sm_count);
    return launch_behind(q8_attn_kernel<D, NT, INT8, false>, dim3(grid), kThreads, C::BYTES, p, stream);
  }
  static std::atomic<bool> prepared[kMaxDevices] = {};
  cudaError_t e = opt_in(q8_attn_kernel<D, NT, INT8, true>, C::BYTES, prepared);
  if (e != cudaSuccess) return e;
  const int grid = std::min(p.c.sm_count, kQ8MaxSms);
  e = launch_behind(q8_attn_kernel<D, NT, INT8, true>, dim3(grid), kThreads, C::BYTES, p, stream);
  if (e != cudaSuccess) return e;
  return launch_behind(q8_join_kernel<D, NT>, dim3(grid, C::ROWS / kJoinRows), kJoinThreads, 0, p, stream);
}

template <int D, bool INT8>
cudaError_t launch_d(const Q8AttnParams& p, cudaStream_t stream) {
  // rows of a sequence's KV head, on average
  const long long group = p.num_query_heads / p.c.num_kv_heads;
  const long long rows = (p.total_q + p.c.num_seqs - 1LL) / p.c.num_seqs * group;
  if (rows <= 8) return launch_nt<D, 1, INT8>(p, rows, stream);
  if constexpr (D == 256) {
    return launch_nt<D, 2, INT8>(p, rows, stream);
  } else {
    if (rows <= 16) return launch_nt<D, 2, INT8>(p, rows, stream);
    return rows <= 24 ? launch_nt<D, 3, INT8>(p, rows, stream) : launch_nt<D, 4, INT8>(p, rows, stream);
  }
}

template <bool INT8>
cudaError_t launch_type(const Q8AttnParams& p, cudaStream_t stream) {
  switch (p.c.head_size) {
    case 64: return launch_d<64, INT8>(p, stream);
    case 128: return launch_d<128, INT8>(p, stream);
    default: return launch_d<256, INT8>(p, stream);
  }
}

}  // namespace

cudaError_t launch_q8_attn(const Q8AttnParams& p, bool int8, cudaStream_t stream) {
  return int8 ? launch_type<true>(p, stream) : launch_type<false>(p, stream);
}

}  // namespace avp
