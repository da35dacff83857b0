// The operators that fill and manage the paged key/value cache: write, accept,
// free, fork, compact (include/paged_attn_cache.h has what each computes).
// They move 2-byte elements and count pages; no floating-point arithmetic.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <mutex>

#include "packed_slice.h"
#include "paged_cache_internal.h"
#include "paged_walk.cuh"
#include "ptx.cuh"

namespace avp {
namespace {

constexpr int kPage = kPageTokens;

// A sequence's new tokens: packed rows [lo, lo + n), the last n positions of
// its len tokens.  A negative slice is empty, rows outside the packed tensor
// are never read, a negative length is 0.
struct NewTokens {
  int lo, n, len;
};

__device__ __forceinline__ NewTokens new_tokens(const int32_t* __restrict__ cu,
                                                const int32_t* __restrict__ seq_lens, int i,
                                                int total) {
  NewTokens t;
  const PackedSlice rows = packed_slice(__ldg(cu + i), __ldg(cu + i + 1), total);
  t.lo = rows.lo;
  t.n = rows.n;
  t.len = max(__ldg(seq_lens + i), 0);
  return t;
}

// --------------------------------------------------------------------- write
// Bound by HBM: every new element is read once and written once.  A unit is
// one page of one sequence for a group of heads, so that the tokens of a page
// meet in one CTA: the value cache is token-fastest, and a thread that holds 8
// tokens of 8 dimensions turns them over in registers and writes whole 16-byte
// pieces of 8 tokens (32 bytes with its neighbour).  Keys keep their 8-element
// pieces: 16 lanes write 16 tokens of a piece, 256 bytes in a row.  Eight loads
// a thread are out at a time, with four CTAs on an SM (three of more registers:
// 50 us instead of 46 for the prompts below).
//
// Measured (captured calls): 12 prompts of up to 4195 tokens, 8 heads of 128,
// 46.4 us, 4.9 TB/s of reads and writes, 72 % of a copy's bandwidth.  One token
// for each of 256 sequences, 16 heads of 128: 10.5 us, bound by latency and by
// the value cache: a token's 2-byte values each have a 32-byte sector to
// themselves.
constexpr int kWriteThreads = 256;
constexpr int kWriteKeys = 8;  // key pieces a thread moves per page of a full head group

struct WritePages {
  int begin, end;    // positions that are written
  int first, pages;  // their pages
};

__device__ __forceinline__ WritePages write_pages(const NewTokens& t, int max_blocks) {
  WritePages w;
  w.begin = max(t.len - t.n, 0);
  w.end = (int)min((long long)t.len, (long long)max_blocks * kPage);
  w.first = w.begin / kPage;
  w.pages = t.n > 0 && w.end > w.begin ? (w.end - 1) / kPage - w.first + 1 : 0;
  return w;
}

__global__ void __launch_bounds__(kWriteThreads, 4) cache_write_kernel(
    const __grid_constant__ CacheWriteParams p, int head_group) {
  __shared__ UnitScratch scratch;
  const int groups = (p.c.num_kv_heads + head_group - 1) / head_group;
  const UnitRange range = locate_units<kWriteThreads>(
      p.c.num_seqs, blockIdx.x, gridDim.x, scratch,
      [&](int i) -> Units {
        const NewTokens t = new_tokens(p.cu, p.seq_lens, i, p.total_tokens);
        const WritePages w = write_pages(t, p.c.max_blocks);
        // here, not at a page: all of a sequence's tokens may lie past its table
        if (blockIdx.x == 0 && t.n > 0 && t.len > w.end) atomicOr(p.c.status, kPageStatusBadBlock);
        return {(long long)w.pages * groups, 1};
      },
      [](int) { return 1; });
  const int tid = threadIdx.x;
  const int pieces = p.c.head_size / 8;  // 16-byte pieces of a head's elements, a power of two
  const int shift = __ffs(pieces) - 1;
  const uint16_t* key = static_cast<const uint16_t*>(p.key);
  const uint16_t* value = static_cast<const uint16_t*>(p.value);
  uint16_t* kc = static_cast<uint16_t*>(p.c.k_cache);
  uint16_t* vc = static_cast<uint16_t*>(p.c.v_cache);
  // a thread's items: values (head, 8 dimensions, 8 slots), one; keys (head,
  // piece, slot), kWriteKeys
  const int half = tid & 1, vpiece = (tid >> 1) & (pieces - 1), vh = tid >> (1 + shift);
  const int slot = tid & (kPage - 1);
  int seq = range.seq;
  long long off = range.off;
  NewTokens t;
  WritePages w;
  bool known = false;
  for (long long u = range.u0; u < range.u1; ++u, ++off) {
    for (;; ++seq, off = 0, known = false) {
      if (seq >= p.c.num_seqs) return;  // only if the lengths changed under the kernel
      if (!known) {
        t = new_tokens(p.cu, p.seq_lens, seq, p.total_tokens);
        w = write_pages(t, p.c.max_blocks);
        known = true;
      }
      if (off < (long long)w.pages * groups) break;
    }
    const int page = w.first + (int)(off / groups), g0 = (int)(off % groups) * head_group;
    const int heads = min(head_group, p.c.num_kv_heads - g0);
    const int id = __ldg(p.block_tables + (size_t)seq * p.c.max_blocks + page);
    if (id < 0 || id >= p.c.num_blocks) {
      if (tid == 0) atomicOr(p.c.status, kPageStatusBadBlock);
      continue;
    }
    // slots [s0, s1) of the page take packed rows row0 + slot
    const int s0 = max(w.begin - page * kPage, 0), s1 = min(w.end - page * kPage, kPage);
    const long long row0 = (long long)t.lo + page * kPage - (t.len - t.n);
    const size_t head0 = (size_t)id * p.c.num_kv_heads + g0;
    if (slot >= s0 && slot < s1) {
      const uint16_t* src = key + (row0 + slot) * p.key_token + (long long)g0 * p.key_head;
      uint16_t* dst = kc + head0 * pieces * (kPage * 8) + slot * 8;
      const int x0 = tid / kPage, items = heads * pieces;
      uint4 e[kWriteKeys];
#pragma unroll
      for (int i = 0; i < kWriteKeys; ++i) {
        const int x = x0 + i * (kWriteThreads / kPage);
        if (x < items)
          e[i] = *reinterpret_cast<const uint4*>(src + (x >> shift) * p.key_head +
                                                 (x & (pieces - 1)) * 8);
      }
#pragma unroll
      for (int i = 0; i < kWriteKeys; ++i) {
        const int x = x0 + i * (kWriteThreads / kPage);
        if (x < items) *reinterpret_cast<uint4*>(dst + x * (kPage * 8)) = e[i];
      }
    }
    const int lo = max(s0 - half * 8, 0), hi = min(s1 - half * 8, 8);
    if (vh >= heads || lo >= hi) continue;
    const uint16_t* src = value + (row0 + half * 8) * p.value_token +
                          (long long)(g0 + vh) * p.value_head + vpiece * 8;
    uint16_t* dst = vc + ((head0 + vh) * p.c.head_size + vpiece * 8) * kPage + half * 8;
    if (hi - lo == 8) {
      uint32_t e[8][4];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 v = *reinterpret_cast<const uint4*>(src + i * p.value_token);
        e[i][0] = v.x, e[i][1] = v.y, e[i][2] = v.z, e[i][3] = v.w;
      }
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        // tokens 2 j, 2 j + 1 of dimension d in one word
        const uint32_t sel = d & 1 ? 0x7632u : 0x5410u;
        uint4 o;
        o.x = __byte_perm(e[0][d >> 1], e[1][d >> 1], sel);
        o.y = __byte_perm(e[2][d >> 1], e[3][d >> 1], sel);
        o.z = __byte_perm(e[4][d >> 1], e[5][d >> 1], sel);
        o.w = __byte_perm(e[6][d >> 1], e[7][d >> 1], sel);
        *reinterpret_cast<uint4*>(dst + d * kPage) = o;
      }
    } else {
#pragma unroll 1
      for (int i = lo; i < hi; ++i) {
        const uint4 v = *reinterpret_cast<const uint4*>(src + i * p.value_token);
        const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int d = 0; d < 8; ++d) dst[d * kPage + i] = (uint16_t)(e[d >> 1] >> (16 * (d & 1)));
      }
    }
  }
}

// -------------------------------------------------------------------- accept
// Draft a_m moves to slot m of the drafts, and a_m >= m with a increasing, so
// a move never overwrites a draft that a later one reads.  Each thread owns
// one element position (a value dimension, or an 8-element piece of a key) and
// moves it for every accepted draft in order, eight loads ahead of their
// stores: threads never touch one another's elements, so no barrier is needed
// between moves.
//
// Bound by the form of the work, not by a memory: 256 sequences, up to 12 of 64
// drafts, 8 heads of 128 take 14.5 us with DRAM at a fifth.  A value moves as 2
// bytes of a sector of its own, 44 MB of sectors touched each way, of which 17
// MB read and 10 MB written are distinct (5 us with the keys at a copy's
// bandwidth), by up to two batches of loads and stores that wait for each other.
// 4 sequences, up to 4 of 8: 3.2 us.
constexpr int kAcceptThreads = 128;
constexpr int kAcceptBatch = 128;  // moves resolved through the table at a time

__global__ void __launch_bounds__(kAcceptThreads) cache_accept_kernel(
    const __grid_constant__ CacheAcceptParams p) {
  __shared__ int s_from[kAcceptBatch], s_to[kAcceptBatch];            // page ids, -1: not moved
  __shared__ uint8_t s_fslot[kAcceptBatch], s_tslot[kAcceptBatch];
  __shared__ int s_stop;
  const int seq = blockIdx.x, tid = threadIdx.x;
  const NewTokens t = new_tokens(p.cu, p.seq_lens, seq, INT_MAX);
  const int base = t.len - t.n;
  const int asked = __ldg(p.num_accepted + seq);
  int take = max(min(asked, min(p.max_accepted, t.n)), 0);
  bool bad = take != asked;
  const int32_t* list = p.accepted + (size_t)seq * p.max_accepted;
  const int32_t* table = p.block_tables + (size_t)seq * p.c.max_blocks;
  const int pieces = p.c.head_size / 8;
  const int values = p.c.num_kv_heads * p.c.head_size, keys = p.c.num_kv_heads * pieces;
  const int item = blockIdx.y * kAcceptThreads + tid;  // value elements, then key pieces
  for (int m0 = 0; m0 < take; m0 += kAcceptBatch) {
    if (tid == 0) s_stop = kAcceptBatch;
    __syncthreads();
    const int n = min(kAcceptBatch, take - m0);
    if (tid < n) {
      const int m = m0 + tid;
      const int a = __ldg(list + m);
      const int prev = m ? __ldg(list + m - 1) : -1;
      // increasing entries from 0 on have a >= m
      const bool holds = a > prev && a >= m && a < t.n;
      if (!holds) atomicMin(&s_stop, tid);
      const long long src = (long long)base + a, dst = (long long)base + m;
      int from = -1, to = -1;
      if (holds && a != m && dst >= 0) {  // dst < src
        if (src < (long long)p.c.max_blocks * kPage) {
          from = __ldg(table + src / kPage);
          to = __ldg(table + dst / kPage);
        }
        if (from < 0 || from >= p.c.num_blocks || to < 0 || to >= p.c.num_blocks) {
          atomicOr(p.c.status, kPageStatusBadBlock);
          from = -1;
        }
      }
      s_from[tid] = from;
      s_to[tid] = to;
      s_fslot[tid] = (uint8_t)(src & (kPage - 1));
      s_tslot[tid] = (uint8_t)(dst & (kPage - 1));
    }
    __syncthreads();
    const int stop = min(n, s_stop);
    if (item < values) {
      uint16_t* vc = static_cast<uint16_t*>(p.c.v_cache) + (size_t)item * kPage;
      const size_t page = (size_t)values * kPage;
      for (int m = 0; m < stop; m += 8) {
        uint16_t e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (m + i < stop && s_from[m + i] >= 0) e[i] = vc[s_from[m + i] * page + s_fslot[m + i]];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (m + i < stop && s_from[m + i] >= 0) vc[s_to[m + i] * page + s_tslot[m + i]] = e[i];
      }
    } else if (item < values + keys) {
      uint4* kc = static_cast<uint4*>(p.c.k_cache) + (size_t)(item - values) * kPage;
      const size_t page = (size_t)keys * kPage;
      for (int m = 0; m < stop; m += 8) {
        uint4 e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (m + i < stop && s_from[m + i] >= 0) e[i] = kc[s_from[m + i] * page + s_fslot[m + i]];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (m + i < stop && s_from[m + i] >= 0) kc[s_to[m + i] * page + s_tslot[m + i]] = e[i];
      }
    }
    __syncthreads();  // the batch's lists are read
    if (stop < n) {   // out of order: acceptance ends here
      take = m0 + stop;
      bad = true;
    }
  }
  if (blockIdx.y == 0 && tid == 0) {
    p.new_lens[seq] = max(base + take, 0);
    if (bad) atomicOr(p.c.status, kPageStatusBadDraft);
  }
}

// ---------------------------------------------------------------------- free
// One CTA per named row.  The exchange of the length with 0 makes one of
// several frees of a row the one that counts; counts only go down by integer
// atomics, so the result does not depend on their order.
constexpr int kFreeThreads = 128;

__global__ void __launch_bounds__(kFreeThreads) cache_free_kernel(
    const __grid_constant__ CacheFreeParams p) {
  __shared__ int s_len;
  const int row = __ldg(p.rows + blockIdx.x);
  if (row < 0 || row >= p.c.num_seqs) {
    if (threadIdx.x == 0) atomicOr(p.c.status, kPageStatusBadRow);
    return;
  }
  if (threadIdx.x == 0) s_len = atomicExch(p.seq_lens + row, 0);
  __syncthreads();
  const int len = s_len;
  const int pages = len > 0 ? min((len - 1) / kPage + 1, p.c.max_blocks) : 0;
  const int32_t* table = p.block_tables + (size_t)row * p.c.max_blocks;
  for (int i = threadIdx.x; i < pages; i += kFreeThreads) {
    const int id = __ldg(table + i);
    if (id < 0 || id >= p.c.num_blocks) {
      atomicOr(p.c.status, kPageStatusBadBlock);
    } else if (atomicSub(p.refs + id, 1) <= 0) {
      atomicAdd(p.refs + id, 1);
      atomicOr(p.c.status, kPageStatusBadRow);
    }
  }
}

// ---------------------------------------------------------------------- fork
// A plan (one CTA) decides which forks hold, which of them need a page and
// which page each gets; the forks themselves then run side by side.  The plan
// reads counts and lengths before any fork changes them.  Bound by latency:
// with the free before it, three short launches, 8.3 us for a few beams and
// 15.1 us for a full server (captured).
constexpr int kPlanThreads = 1024;
constexpr int kForkThreads = 256;
constexpr int kForkParts = 4;  // CTAs per fork
constexpr int kRefused = -2, kNoPage = -1;

// Exclusive scan over the CTA's threads; `total` gets the sum.
__device__ __forceinline__ int block_exclusive(int x, int& total, int* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += y;
  }
  __syncthreads();  // s_warp's last readers are done
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  int w = s_warp[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return inc - x + (warp ? before : 0);
}

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(
    const __grid_constant__ CacheForkParams p) {
  __shared__ int s_warp[32];
  const int tid = threadIdx.x;
  grid_launch_dependents();
  for (int r = tid; r < p.c.num_seqs; r += kPlanThreads) {
    p.owner[r] = INT_MAX;
    p.is_src[r] = 0;
  }
  __syncthreads();
  auto inside = [&](int r) { return r >= 0 && r < p.c.num_seqs; };
  for (int j = tid; j < p.num_forks; j += kPlanThreads) {
    const int s = __ldg(p.src + j), d = __ldg(p.dst + j);
    if (inside(s) && inside(d)) {
      p.is_src[s] = 1;
      atomicMin(p.owner + d, j);
    }
  }
  __syncthreads();
  int need = 0;  // pages the forks so far take
  for (int j0 = 0; j0 < p.num_forks; j0 += kPlanThreads) {
    const int j = j0 + tid;
    bool holds = false, part = false;
    if (j < p.num_forks) {
      const int s = __ldg(p.src + j), d = __ldg(p.dst + j);
      holds = inside(s) && inside(d) && __ldcg(p.owner + d) == j && !p.is_src[d] &&
              p.seq_lens[d] <= 0;
      if (!holds) atomicOr(p.c.status, kPageStatusBadRow);
      // a row longer than its table has no page past the table to copy
      part = holds && p.seq_lens[s] > 0 && p.seq_lens[s] % kPage != 0 &&
             p.seq_lens[s] < p.c.max_blocks * (long long)kPage;
      if (part) {  // nor has a last id that is no page
        const int id = p.block_tables[(size_t)s * p.c.max_blocks + p.seq_lens[s] / kPage];
        part = id >= 0 && id < p.c.num_blocks;
      }
    }
    int total;
    const int rank = need + block_exclusive(part ? 1 : 0, total, s_warp);
    if (j < p.num_forks) p.state[j] = !holds ? kRefused : (part ? rank : kNoPage);
    need += total;
  }
  // the `need` lowest free pages
  int found = 0;
  for (long long b0 = 0; b0 < p.c.num_blocks && found < need; b0 += 4 * kPlanThreads) {
    const long long b = b0 + 4 * tid;
    int free_mask = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (b + i < p.c.num_blocks && __ldcg(p.refs + b + i) <= 0) free_mask |= 1 << i;
    int total;
    int at = found + block_exclusive(__popc(free_mask), total, s_warp);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (free_mask >> i & 1) {
        if (at < need) p.pages[at] = (int)b + i;
        ++at;
      }
    found += total;
  }
  __syncthreads();
  for (int j = tid; j < p.num_forks; j += kPlanThreads) {
    const int rank = p.state[j];
    if (rank < 0) continue;
    if (rank < found) {
      p.state[j] = p.pages[rank];
    } else {
      p.state[j] = kRefused;
      atomicOr(p.c.status, kPageStatusNoBlock);
    }
  }
}

// Copies 16-byte pieces [a, b) of one page to another, four in flight a thread.
template <int THREADS>
__device__ __forceinline__ void copy_pieces(const uint4* __restrict__ src, uint4* __restrict__ dst,
                                            int a, int b) {
  int i = a + (int)threadIdx.x;
  for (; i + 3 * THREADS < b; i += 4 * THREADS) {
    uint4 e[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) e[x] = __ldcs(src + i + x * THREADS);
#pragma unroll
    for (int x = 0; x < 4; ++x) dst[i + x * THREADS] = e[x];
  }
  for (; i < b; i += THREADS) dst[i] = __ldcs(src + i);
}

__global__ void __launch_bounds__(kForkThreads) fork_apply_kernel(
    const __grid_constant__ CacheForkParams p) {
  const int j = blockIdx.x, part = blockIdx.y;
  grid_wait_prerequisite();
  const int fresh = p.state[j];
  if (fresh == kRefused) return;
  const int s = __ldg(p.src + j), d = __ldg(p.dst + j);
  const int len = max(p.seq_lens[s], 0);
  const int32_t* from = p.block_tables + (size_t)s * p.c.max_blocks;
  int32_t* to = p.block_tables + (size_t)d * p.c.max_blocks;
  const int full = min(len / kPage, p.c.max_blocks);
  // a last page without a fresh one in its place is a bad id, which is copied
  const int ids = fresh >= 0 ? full : (int)min((len + kPage - 1LL) / kPage, (long long)p.c.max_blocks);
  for (int i = part * kForkThreads + threadIdx.x; i < ids; i += kForkParts * kForkThreads) {
    const int id = from[i];
    to[i] = id;
    if (id < 0 || id >= p.c.num_blocks)
      atomicOr(p.c.status, kPageStatusBadBlock);
    else
      atomicAdd(p.refs + id, 1);
  }
  if (part == 0 && threadIdx.x == 0) {
    p.seq_lens[d] = len;
    if (fresh >= 0) {
      to[full] = fresh;
      p.refs[fresh] = 1;
    }
  }
  if (fresh < 0) return;
  const int last = from[full];
  if (last < 0 || last >= p.c.num_blocks) return;  // only if the table changed under the kernel
  const int page = p.c.num_kv_heads * p.c.head_size * 2;  // 16-byte pieces
  const int a = (int)((long long)page * part / kForkParts);
  const int b = (int)((long long)page * (part + 1) / kForkParts);
  const uint4* k = static_cast<const uint4*>(p.c.k_cache);
  const uint4* v = static_cast<const uint4*>(p.c.v_cache);
  copy_pieces<kForkThreads>(k + (size_t)last * page,
                            static_cast<uint4*>(p.c.k_cache) + (size_t)fresh * page, a, b);
  copy_pieces<kForkThreads>(v + (size_t)last * page,
                            static_cast<uint4*>(p.c.v_cache) + (size_t)fresh * page, a, b);
}

// ------------------------------------------------------------------- compact
// A plan (one CTA) counts the used pages, U, and lists the moves: the i-th
// lowest hole below U receives the i-th highest used page.  Both indexes
// follow from one scan u(p) = used pages below p: a hole p is number p - u(p),
// a used page p >= U is number U - u(p) - 1.  Then pages are copied, counts
// moved and table entries renamed side by side: an entry below U stays, one at
// or past it asks its page's number i (checked against the list, so an entry
// that no count backs stays as it is).
//
// The copies are bound by HBM; the plan is bound by latency, so each of its
// threads takes 16 pages at a time, in registers between the count and the
// scan where the pool has at most 16384.  A large pool (258 MB moved) takes
// 92 us, 78 of them the copies: 5.6 TB/s of reads and writes, 83 % of a copy's
// bandwidth; a small one 7.6 us.
constexpr int kCompactThreads = 256;
constexpr int kPieceGroup = 1024;  // 16-byte pieces of a page one CTA copies at a time
constexpr int kPlanPages = 16;     // pages a plan thread takes at a time

__device__ __forceinline__ void load_counts(const int32_t* refs, long long b, int blocks,
                                            int (&ref)[kPlanPages]) {
  if ((reinterpret_cast<uintptr_t>(refs) & 15u) == 0 && b + kPlanPages <= blocks) {
#pragma unroll
    for (int i = 0; i < kPlanPages; i += 4) {
      const int4 v = *reinterpret_cast<const int4*>(refs + b + i);
      ref[i] = v.x, ref[i + 1] = v.y, ref[i + 2] = v.z, ref[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPlanPages; ++i) ref[i] = b + i < blocks ? refs[b + i] : 0;
  }
}

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(
    const __grid_constant__ CacheCompactParams p) {
  __shared__ int s_warp[32];
  const int tid = threadIdx.x, blocks = p.c.num_blocks;
  constexpr int kStep = kPlanPages * kPlanThreads;
  grid_launch_dependents();
  int ref[kPlanPages], mine = 0;
  for (long long b0 = 0; b0 < blocks; b0 += kStep) {
    load_counts(p.refs, b0 + kPlanPages * tid, blocks, ref);
#pragma unroll
    for (int i = 0; i < kPlanPages; ++i) mine += ref[i] > 0;
  }
  int used;
  int below = block_exclusive(mine, used, s_warp);  // used pages of lower threads
  if (tid == 0) {
    p.head[0] = 0;
    p.head[1] = used;
  }
  __syncthreads();
  int before = 0;  // used pages below b0
  for (long long b0 = 0; b0 < blocks; b0 += kStep) {
    const long long b = b0 + kPlanPages * tid;
    if (blocks > kStep) {
      load_counts(p.refs, b, blocks, ref);
      int n = 0;
#pragma unroll
      for (int i = 0; i < kPlanPages; ++i) n += ref[i] > 0;
      int total;
      below = before + block_exclusive(n, total, s_warp);
      before += total;
    }
    int u = below;
#pragma unroll
    for (int i = 0; i < kPlanPages; ++i) {
      const int id = (int)b + i;
      if (b + i >= blocks) break;
      if (id == used) p.head[0] = used - u;  // holes below `used`
      if (ref[i] <= 0 && id < used) p.to[id - u] = id;
      if (ref[i] > 0 && id >= used) {
        p.from[used - u - 1] = id;
        p.number[id] = used - u - 1;
      }
      u += ref[i] > 0;
    }
  }
}

__global__ void __launch_bounds__(kCompactThreads) compact_apply_kernel(
    const __grid_constant__ CacheCompactParams p) {
  grid_wait_prerequisite();
  const int moves = __ldcg(p.head), used = __ldcg(p.head + 1);
  const int page = p.c.num_kv_heads * p.c.head_size * 2;  // 16-byte pieces
  const int groups = (page + kPieceGroup - 1) / kPieceGroup;
  const long long tasks = (long long)moves * groups * 2;
  for (long long x = blockIdx.x; x < tasks; x += gridDim.x) {
    const bool value = x & 1;
    const int g = (int)((x >> 1) % groups), i = (int)((x >> 1) / groups);
    const size_t from = (size_t)__ldcg(p.from + i) * page, to = (size_t)__ldcg(p.to + i) * page;
    uint4* c = static_cast<uint4*>(value ? p.c.v_cache : p.c.k_cache);
    copy_pieces<kCompactThreads>(c + from, c + to, g * kPieceGroup,
                                 min(page, (g + 1) * kPieceGroup));
  }
  const long long first = (long long)blockIdx.x * kCompactThreads + threadIdx.x;
  const long long step = (long long)gridDim.x * kCompactThreads;
  // counts: every page is one move's source or target, or keeps its own.  (In
  // place the last is nothing to do, so nothing else reads what a move writes.)
  for (long long i = first; i < moves; i += step) {
    const int from = __ldcg(p.from + i), to = __ldcg(p.to + i);
    p.refs_out[to] = p.refs[from];
    p.refs_out[from] = 0;
  }
  if (p.refs_out != p.refs)
    for (long long b = first; b < p.c.num_blocks; b += step) {
      const int ref = p.refs[b];
      if ((ref > 0) == (b < used)) p.refs_out[b] = ref;
    }
  const long long entries = (long long)p.c.num_seqs * p.c.max_blocks;
  for (long long e = first; e < entries; e += step) {
    const int row = (int)(e / p.c.max_blocks), col = (int)(e - (long long)row * p.c.max_blocks);
    int id = p.block_tables[e];
    if ((long long)col * kPage < __ldg(p.seq_lens + row)) {
      if (id < 0 || id >= p.c.num_blocks) {
        atomicOr(p.c.status, kPageStatusBadBlock);
      } else if (id >= used) {
        const int i = __ldcg(p.number + id);
        if (i >= 0 && i < moves && __ldcg(p.from + i) == id) id = __ldcg(p.to + i);
      }
    }
    p.block_tables_out[e] = id;
  }
}

// Launches a kernel that may start while the one before it on the stream still
// runs (it waits for that one's end before it reads anything).
template <class Params>
cudaError_t launch_behind(void (*kernel)(Params), dim3 grid, int threads, const Params& p,
                          cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// A fork and a compaction are a plan and what carries it out: no other call that
// changes counts, lengths or tables may come between the two on their stream,
// also from another thread.
std::mutex g_plan_mu;

}  // namespace

cudaError_t launch_cache_write(const CacheWriteParams& p, cudaStream_t stream) {
  // a page's heads in groups that give each thread one value item
  const int pieces = p.c.head_size / 8;
  const int group = std::min(p.c.num_kv_heads, kWriteThreads / (2 * pieces));
  const long long groups = (p.c.num_kv_heads + group - 1) / group;
  // n tokens touch at most n / 16 + 2 pages
  const long long most = (p.total_tokens / kPage + 2LL * p.c.num_seqs) * groups;
  const int grid = (int)std::min<long long>(most, p.c.sm_count * 4LL);
  cache_write_kernel<<<grid, kWriteThreads, 0, stream>>>(p, group);
  return cudaGetLastError();
}

cudaError_t launch_cache_accept(const CacheAcceptParams& p, cudaStream_t stream) {
  const long long items = (long long)p.c.num_kv_heads * p.c.head_size * 9 / 8;
  const long long y = (items + kAcceptThreads - 1) / kAcceptThreads;
  if (y > 65535) return cudaErrorInvalidConfiguration;
  cache_accept_kernel<<<dim3(p.c.num_seqs, (unsigned)y), kAcceptThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_cache_free(const CacheFreeParams& p, cudaStream_t stream) {
  std::lock_guard<std::mutex> lock(g_plan_mu);
  cache_free_kernel<<<p.num_rows, kFreeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_cache_fork(const CacheForkParams& p, cudaStream_t stream) {
  std::lock_guard<std::mutex> lock(g_plan_mu);
  fork_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_behind(fork_apply_kernel, dim3(p.num_forks, kForkParts), kForkThreads, p, stream);
}

cudaError_t launch_cache_compact(const CacheCompactParams& p, cudaStream_t stream) {
  std::lock_guard<std::mutex> lock(g_plan_mu);
  compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_behind(compact_apply_kernel, dim3(p.c.sm_count * 4), kCompactThreads, p, stream);
}

}  // namespace avp
