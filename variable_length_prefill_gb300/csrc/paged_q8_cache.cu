// The operators that write an 8-bit paged cache and read it back
// (include/paged_attn_q8.h has what each computes).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "packed_slice.h"
#include "paged_q8_codes.cuh"
#include "paged_q8_internal.h"
#include "paged_walk.cuh"
#include "ptx.cuh"

namespace avp {
namespace {

constexpr int kPage = kPageTokens;
constexpr int kMoveThreads = 256;
constexpr int kMoveWarps = kMoveThreads / 32;

// A sequence's packed rows and the positions they stand for.
struct Tokens {
  int lo, n, len;
  int begin, end;    // positions that are moved
  int first, pages;  // their pages
};

__device__ __forceinline__ Tokens tokens_of(const Q8MoveParams& p, int i) {
  Tokens t;
  const PackedSlice rows = packed_slice(__ldg(p.cu + i), __ldg(p.cu + i + 1), p.total_tokens);
  t.lo = rows.lo;
  t.n = rows.n;
  t.len = max(__ldg(p.seq_lens + i), 0);
  t.begin = max(t.len - t.n, 0);
  t.end = (int)min((long long)t.len, (long long)p.c.max_blocks * kPage);
  t.first = t.begin / kPage;
  t.pages = t.n > 0 && t.end > t.begin ? (t.end - 1) / kPage - t.first + 1 : 0;
  return t;
}

// One page of one KV head, keys or values: slots [s0, s1) are packed rows row0 +
// slot, `held` slots before them hold tokens of the sequence.
struct PageTask {
  size_t page_head;  // page * heads + head
  int g, s0, s1;
  long long row0;
  bool values;
  bool held;
};

// f(task) for the tasks of sequence i that are `at`, `at + step`, ... of its
// pages x heads x {keys, values}, below `until`.
template <class F>
__device__ __forceinline__ void page_tasks(const Q8MoveParams& p, int i, const Tokens& t,
                                           long long at, long long until, int step, F f) {
  const int per_page = p.c.num_kv_heads * 2;
  const int32_t* table = p.block_tables + (size_t)i * p.c.max_blocks + t.first;
  // pages x heads of a sequence may pass 32 bits only where no cache could hold them
  auto page_of = [&](long long x) { return (int)((unsigned)x / (unsigned)per_page); };
  int next = at < until ? __ldg(table + page_of(at)) : 0;
  for (; at < until; at += step) {
    const int off = page_of(at), page = t.first + off, rest = (int)((unsigned)at - (unsigned)off * per_page);
    const int id = next;
    if (at + step < until) next = __ldg(table + page_of(at + step));
    if (id < 0 || id >= p.c.num_blocks) {
      if ((threadIdx.x & 31) == 0) atomicOr(p.c.status, kPageStatusBadBlock);
      continue;
    }
    PageTask k;
    k.g = rest >> 1;
    k.values = rest & 1;
    k.page_head = (size_t)id * p.c.num_kv_heads + k.g;
    k.s0 = max(t.begin - page * kPage, 0);
    k.s1 = min(t.end - page * kPage, kPage);
    k.row0 = (long long)t.lo + page * kPage - (t.len - t.n);
    k.held = k.s0 > 0;
    f(k);
  }
}

// The tasks of this warp: those of all sequences are cut into one equal range per CTA,
// whose warps take turns.
template <class F>
__device__ __forceinline__ void move_tasks(const Q8MoveParams& p, UnitScratch& scratch, F f) {
  const int warp = threadIdx.x >> 5;
  // launched while the kernel before it ends: nothing is read or written before this
  grid_wait_prerequisite();
  grid_launch_dependents();
  const UnitRange range = locate_units<kMoveThreads>(
      p.c.num_seqs, blockIdx.x, gridDim.x, scratch,
      [&](int i) -> Units {
        const Tokens t = tokens_of(p, i);
        if (blockIdx.x == 0 && t.n > 0 && t.len > t.end) atomicOr(p.c.status, kPageStatusBadBlock);
        return {(long long)t.pages * p.c.num_kv_heads * 2, 1};
      },
      [](int) { return 1; });
  long long at = range.off, left = range.u1 - range.u0;
  for (int i = range.seq; left > 0 && i < p.c.num_seqs; ++i, at = 0) {
    const Tokens t = tokens_of(p, i);
    const long long here = min((long long)t.pages * p.c.num_kv_heads * 2 - at, left);
    if (here <= 0) continue;
    // the warps take turns over the CTA's whole range
    const long long done = (range.u1 - range.u0) - left;
    const int first = (int)((warp - done % kMoveWarps + kMoveWarps) % kMoveWarps);
    page_tasks(p, i, t, at + first, at + here, kMoveWarps, f);
    left -= here;
  }
}

template <bool FP16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
  if constexpr (FP16) return half2_bits_to_float2(w);
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// N consecutive words, of 4, 8, 16 or 32 bytes.
template <int N>
__device__ __forceinline__ void load_words(const void* src, uint32_t* w) {
  if constexpr (N == 1) {
    w[0] = *static_cast<const uint32_t*>(src);
  } else if constexpr (N == 2) {
    const uint2 v = *static_cast<const uint2*>(src);
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = static_cast<const uint4*>(src)[i];
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  }
}

template <int N>
__device__ __forceinline__ void store_words(void* dst, const uint32_t* w) {
  if constexpr (N == 1) {
    *static_cast<uint32_t*>(dst) = w[0];
  } else if constexpr (N == 2) {
    *static_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      static_cast<uint4*>(dst)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
}

// 32 bytes of a sector, in one store where they begin one (a cache's base may be 16 bytes
// past: then in two).
__device__ __forceinline__ void store_sector(uint8_t* dst, const uint32_t (&w)[8]) {
  if ((reinterpret_cast<uintptr_t>(dst) & 31u) == 0)
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  else
    store_words<8>(dst, w);
}

// --------------------------------------------------------------------- write
// The larger magnitudes of two pairs; NaN wins.
template <bool FP16>
__device__ __forceinline__ uint32_t max_pair(uint32_t m, uint32_t w) {
  uint32_t r;
  w &= 0x7fff7fffu;
  if constexpr (FP16)
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(w));
  else
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(w));
  return r;
}

// The largest finite magnitude of a warp's words of 16-bit pairs, and whether
// there are non-finite ones.  Magnitudes compare as their bits do.
template <bool FP16, int N>
__device__ __forceinline__ float largest_of(const uint32_t (&w)[N], bool& odd) {
  constexpr uint32_t kInf = FP16 ? 0x7c00u : 0x7f80u;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max_pair<FP16>(m, w[i]);
  uint32_t top = __reduce_max_sync(0xffffffffu, max(m & 0x7fffu, (m >> 16) & 0x7fffu));
  odd = top >= kInf;
  if (odd) {
    top = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t a = w[i] & 0x7fffu, b = (w[i] >> 16) & 0x7fffu;
      top = max(top, max(a < kInf ? a : 0u, b < kInf ? b : 0u));
    }
    top = __reduce_max_sync(0xffffffffu, top);
  }
  return unpack16<FP16>(top).x;
}

// A page's codes of tokens before the new ones, rounded anew: slots [0, s0).
template <int D, bool INT8>
__device__ __noinline__ void round_anew(uint8_t* page, bool values, int s0, float by) {
  for (int item = threadIdx.x & 31; item < D; item += 32) {
    if (!values && item % kPage >= s0) continue;
    uint4* at = reinterpret_cast<uint4*>(page) + item;
    uint4 v = *at;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[4];
      codes_to_float<INT8>(w[i], f);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] *= by;
      if constexpr (!INT8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = fabsf(f[j]) <= 3.4e38f ? f[j] : __uint_as_float(0x7fffffffu);
      }
      const uint32_t c = float_to_codes<INT8>(f[0], f[1], f[2], f[3]);
      // of values, this word's four bytes are tokens 4 i on
      const int keep = values ? min(max(s0 - 4 * i, 0), 4) : 4;
      const uint32_t mask = keep == 4 ? 0xffffffffu : (1u << (8 * keep)) - 1u;
      w[i] = (c & mask) | (w[i] & ~mask);
    }
    *at = v;
  }
}

// Settles the page's scale; returns its reciprocal (both are powers of two, the
// product below is exact).
template <int D, bool INT8>
__device__ __forceinline__ float settle_scale(float* scale, uint8_t* page, const PageTask& k,
                                              float largest) {
  float now = scale_for<INT8>(largest);
  const int lane = threadIdx.x & 31;
  if (k.held) {
    const float old = *scale;
    if (finite_positive(old)) now = fmaxf(now, power_at_least(old));
    __syncwarp();  // every lane has read it
    if (old != now) round_anew<D, INT8>(page, k.values, k.s0, old / now);
    __syncwarp();  // what is rounded anew comes before the new tokens' bytes
  }
  if (lane == 0) *scale = now;
  const uint32_t e = 0x7f000000u - __float_as_uint(now);
  return __uint_as_float(e ? e : 0x00400000u);  // of 2^127: 2^-127
}

// A page that gets one or two tokens (decoding): one at a time.  A lane has D / 32
// elements of a token; all but the last are read again after the scale is known.
template <int D, bool FP16, bool INT8>
__device__ __forceinline__ void write_few(const PageTask& k, const uint16_t* src, long long token, uint8_t* page,
                                          float* scale) {
  const int lane = threadIdx.x & 31;
  constexpr int E = D / 32, W = E / 2;
  src += lane * E;
  uint32_t w[W];
  float largest = 0.f;
  bool odd = false;
#pragma unroll 1
  for (int slot = k.s0; slot < k.s1; ++slot) {
    load_words<W>(src + slot * token, w);
    bool some;
    largest = fmaxf(largest, largest_of<FP16>(w, some));
    odd |= some;
  }
  const float by = settle_scale<D, INT8>(scale, page, k, largest);
  const float nan = __uint_as_float(0x7fffffffu);
#pragma unroll 1
  for (int slot = k.s1 - 1; slot >= k.s0; --slot) {
    if (slot != k.s1 - 1) load_words<W>(src + slot * token, w);
    uint32_t o[(E + 3) / 4];
#pragma unroll
    for (int j = 0; j < (E + 3) / 4; ++j) {
      float2 a = unpack16<FP16>(w[2 * j]), b = 2 * j + 1 < W ? unpack16<FP16>(w[2 * j + 1]) : make_float2(0.f, 0.f);
      a.x *= by, a.y *= by, b.x *= by, b.y *= by;
      if (!INT8 && odd) {
        a.x = isinf(a.x) ? nan : a.x, a.y = isinf(a.y) ? nan : a.y;
        b.x = isinf(b.x) ? nan : b.x, b.y = isinf(b.y) ? nan : b.y;
      }
      o[j] = float_to_codes<INT8>(a.x, a.y, b.x, b.y);
    }
    if (!k.values) {
      uint8_t* dst = page + (lane * E / 16) * (kPage * 16) + slot * 16 + lane * E % 16;
      if constexpr (E == 2)
        *reinterpret_cast<uint16_t*>(dst) = (uint16_t)o[0];
      else
        store_words<E / 4>(dst, o);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) page[(lane * E + e) * kPage + slot] = (uint8_t)(o[e / 4] >> (8 * (e % 4)));
    }
  }
}

// Bound by HBM: 2 bytes of each new element are read and 1 written.  A warp takes
// the keys or the values of one page and head, so that the page's largest
// magnitude needs no more than a reduction of the warp, and holds them in
// registers from the reduction to the rounding: one pass over the data.  Keys: a
// lane loads D / 16 elements of every other token, and stores their bytes, so
// that two lanes with neighbouring tokens fill each 32-byte sector.  Values: a
// lane loads D / 32 elements of all 16 tokens and stores two rows of tokens, a
// sector, at a time.
//
// Measured (captured calls): 12 prompts of up to 4195 tokens, 8 heads of 128, 39.2 us,
// 4.4 TB/s, 65 % of a copy's bandwidth: a warp has nothing in flight between its
// loads and the next task's, at three CTAs an SM (two 44 us; four spill, 52).  One token
// for each of 256 sequences, 16 heads of 128: 9.0 us, latency.  The walk over all
// lengths costs the latter 2 us; without it (a CTA a sequence) a prompt among many
// single tokens would have all of its pages to one CTA.
// FULL: all 16 tokens of the page are new.
template <bool FULL, int D, bool FP16, bool INT8>
__device__ __forceinline__ void write_page(const PageTask& k, const uint16_t* src, long long token, uint8_t* page,
                                           float* scale) {
  const int lane = threadIdx.x & 31;
  const float nan = __uint_as_float(0x7fffffffu);
  auto in = [&](int slot) { return FULL || (slot >= k.s0 && slot < k.s1); };
  bool odd;
  if (!k.values) {
    constexpr int C = D / 16, W = C / 2;  // elements and words of a lane's token
    const int c = (lane >> 1) * C, parity = lane & 1;
    uint32_t w[8 * W];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int slot = 2 * i + parity;
      if (in(slot)) {
        load_words<W>(src + slot * token + c, w + i * W);
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j) w[i * W + j] = 0;
      }
    }
    const float largest = largest_of<FP16>(w, odd);
    const float by = settle_scale<D, INT8>(scale, page, k, largest);
    uint8_t* dst = page + (c / 16) * (kPage * 16) + c % 16;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int slot = 2 * i + parity;
      uint32_t o[C / 4];
#pragma unroll
      for (int j = 0; j < C / 4; ++j) {
        float2 a = unpack16<FP16>(w[i * W + 2 * j]), b = unpack16<FP16>(w[i * W + 2 * j + 1]);
        a.x *= by, a.y *= by, b.x *= by, b.y *= by;
        if (!INT8 && odd) {
          a.x = isinf(a.x) ? nan : a.x, a.y = isinf(a.y) ? nan : a.y;
          b.x = isinf(b.x) ? nan : b.x, b.y = isinf(b.y) ? nan : b.y;
        }
        o[j] = float_to_codes<INT8>(a.x, a.y, b.x, b.y);
      }
      if (in(slot)) store_words<C / 4>(dst + slot * 16, o);
    }
  } else {
    constexpr int E = D / 32, W = E / 2;
    uint32_t w[16 * W];
#pragma unroll
    for (int i = 0; i < kPage; ++i) {
      if (in(i)) {
        load_words<W>(src + i * token + lane * E, w + i * W);
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j) w[i * W + j] = 0;
      }
    }
    const float largest = largest_of<FP16>(w, odd);
    const float by = settle_scale<D, INT8>(scale, page, k, largest);
    uint8_t* dst = page + lane * E * kPage;
#pragma unroll
    for (int e = 0; e < E; e += 2) {  // two rows, which are one 32-byte sector
      uint32_t o[8];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float f[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float2 v = unpack16<FP16>(w[(4 * j + x) * W + e / 2]);
            f[x] = (h ? v.y : v.x) * by;
            if (!INT8 && odd) f[x] = isinf(f[x]) ? nan : f[x];
          }
          o[4 * h + j] = float_to_codes<INT8>(f[0], f[1], f[2], f[3]);
        }
      if constexpr (FULL) {
        store_sector(dst + e * kPage, o);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < kPage; ++i)
            if (in(i)) dst[(e + h) * kPage + i] = (uint8_t)(o[4 * h + i / 4] >> (8 * (i % 4)));
      }
    }
  }
}

template <int D, bool FP16, bool INT8>
__global__ void __launch_bounds__(kMoveThreads, D == 256 ? 2 : 3) q8_write_kernel(const __grid_constant__ Q8MoveParams p) {
  __shared__ UnitScratch scratch;
  move_tasks(p, scratch, [&](const PageTask& k) {
    const uint16_t* src = static_cast<const uint16_t*>(k.values ? p.value : p.key);
    const long long token = k.values ? p.value_token : p.key_token;
    src += k.row0 * token + k.g * (k.values ? p.value_head : p.key_head);
    uint8_t* page = static_cast<uint8_t*>(k.values ? p.c.v_cache : p.c.k_cache) + k.page_head * (D * kPage);
    float* scale = (k.values ? p.v_scale : p.k_scale) + k.page_head;
    if (k.s1 - k.s0 <= 2) {
      write_few<D, FP16, INT8>(k, src, token, page, scale);
      return;
    }
    if (k.s0 == 0 && k.s1 == kPage)
      write_page<true, D, FP16, INT8>(k, src, token, page, scale);
    else
      write_page<false, D, FP16, INT8>(k, src, token, page, scale);
  });
}

// ---------------------------------------------------------------------- read
// scale * codes in 16 bits, cut to the finite range.
template <bool FP16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  const float most = FP16 ? 65504.f : 3.3895314e38f;
  // NaN passes: both comparisons are false
  a = a > most ? most : a < -most ? -most : a;
  b = b > most ? most : b < -most ? -most : b;
  uint32_t r;
  if constexpr (FP16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// The write's mirror, with its layout of lanes: bound by HBM, 1 byte read and 2
// written for each element.  The prompts above: 33 us, 5.2 TB/s, 76 % of a copy's
// bandwidth.
template <int D, bool FP16, bool INT8>
__global__ void __launch_bounds__(kMoveThreads, D == 256 ? 2 : 3) q8_read_kernel(const __grid_constant__ Q8MoveParams p) {
  __shared__ UnitScratch scratch;
  const int lane = threadIdx.x & 31;
  move_tasks(p, scratch, [&](const PageTask& k) {
    uint16_t* dst = static_cast<uint16_t*>(k.values ? p.value : p.key);
    const long long token = k.values ? p.value_token : p.key_token;
    dst += k.row0 * token + k.g * (k.values ? p.value_head : p.key_head);
    const uint8_t* page =
        static_cast<const uint8_t*>(k.values ? p.c.v_cache : p.c.k_cache) + k.page_head * (D * kPage);
    float scale = __ldg((k.values ? p.v_scale : p.k_scale) + k.page_head);
    if (!(scale >= 0.f && scale <= 3.402823466e38f)) scale = __uint_as_float(0x7fffffffu);
    if (!k.values) {
      constexpr int C = D / 16;
      const int c = (lane >> 1) * C, parity = lane & 1;
      const uint8_t* src = page + (c / 16) * (kPage * 16) + c % 16;
      uint32_t w[8][C / 4];
#pragma unroll
      for (int i = 0; i < 8; ++i) load_words<C / 4>(src + (2 * i + parity) * 16, w[i]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int slot = 2 * i + parity;
        uint32_t o[C / 2];
#pragma unroll
        for (int j = 0; j < C / 4; ++j) {
          float f[4];
          codes_to_float<INT8>(w[i][j], f);
          o[2 * j] = pack16<FP16>(f[0] * scale, f[1] * scale);
          o[2 * j + 1] = pack16<FP16>(f[2] * scale, f[3] * scale);
        }
        if (slot >= k.s0 && slot < k.s1) store_words<C / 2>(dst + slot * token + c, o);
      }
    } else {
      constexpr int E = D / 32;
      uint32_t w[E][4];
#pragma unroll
      for (int e = 0; e < E; ++e) load_words<4>(page + (lane * E + e) * kPage, w[e]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float f[E][4];
#pragma unroll
        for (int e = 0; e < E; ++e) codes_to_float<INT8>(w[e][j], f[e]);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int slot = 4 * j + x;
          uint32_t o[E / 2];
#pragma unroll
          for (int e = 0; e < E; e += 2) o[e / 2] = pack16<FP16>(f[e][x] * scale, f[e + 1][x] * scale);
          if (slot >= k.s0 && slot < k.s1) store_words<E / 2>(dst + slot * token + lane * E, o);
        }
      }
    }
  });
}

// ------------------------------------------------------------------ launches
// Behind what is on the stream, started while that ends (the kernels wait for it).
template <class K>
cudaError_t launch_behind(K kernel, int grid, const Q8MoveParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, bool FP16, bool INT8>
cudaError_t launch_move(const Q8MoveParams& p, bool write, cudaStream_t stream) {
  // n tokens touch at most n / 16 + 2 pages, and no more than n
  const long long pages = std::min<long long>(p.total_tokens, p.total_tokens / kPage + 2LL * p.c.num_seqs);
  const long long most = (pages * 2 * p.c.num_kv_heads + kMoveWarps - 1) / kMoveWarps;
  const int grid = (int)std::min<long long>(most, p.c.sm_count * (D == 256 ? 2LL : 3LL));
  return launch_behind(write ? q8_write_kernel<D, FP16, INT8> : q8_read_kernel<D, FP16, INT8>, grid, p, stream);
}

template <int D>
cudaError_t launch_move_d(const Q8MoveParams& p, bool fp16, bool int8, bool write, cudaStream_t stream) {
  if (fp16)
    return int8 ? launch_move<D, true, true>(p, write, stream) : launch_move<D, true, false>(p, write, stream);
  return int8 ? launch_move<D, false, true>(p, write, stream) : launch_move<D, false, false>(p, write, stream);
}

cudaError_t launch_move_any(const Q8MoveParams& p, bool fp16, bool int8, bool write, cudaStream_t stream) {
  switch (p.c.head_size) {
    case 64: return launch_move_d<64>(p, fp16, int8, write, stream);
    case 128: return launch_move_d<128>(p, fp16, int8, write, stream);
    default: return launch_move_d<256>(p, fp16, int8, write, stream);
  }
}

}  // namespace

cudaError_t launch_q8_write(const Q8MoveParams& p, bool fp16, bool int8, cudaStream_t stream) {
  return launch_move_any(p, fp16, int8, true, stream);
}

cudaError_t launch_q8_read(const Q8MoveParams& p, bool fp16, bool int8, cudaStream_t stream) {
  return launch_move_any(p, fp16, int8, false, stream);
}

}  // namespace avp
