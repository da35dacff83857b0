// Work that the host cannot count: every sequence has a number of units that
// follows from its lengths on the device.  The units of all sequences, laid
// end to end, are cut into one equal range per CTA.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace avp {
namespace {

// A CTA's range: units [u0, u1) of `total`; unit u0 is unit `off` of sequence
// `seq`.  Empty when u0 == u1.
struct UnitRange {
  long long u0, u1, total;
  int used;  // ranges that the units are cut into
  long long off;
  int seq;
};

// The units of a sequence, and how many of them its longest piece of work has
// (pieces are the caller's: what a range that ends inside one costs extra for).
struct Units {
  long long count;
  int longest;
};

struct UnitScratch {
  long long warp_sum[32];
  int warp_longest[32];
  long long off;
  int seq;
};

__device__ __forceinline__ long long warp_inclusive(long long x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// Range `part` of at most `parts`, none shorter than least(longest piece of all)
// units unless there are fewer; every thread of the CTA takes part.  units(i)
// is the Units of sequence i.  Thread t sums a run of consecutive sequences, a
// scan over the threads gives the total, and the thread whose run holds unit
// u0 walks it.
template <int THREADS, class Count, class Least>
__device__ __forceinline__ UnitRange locate_units(int n, int part, int parts, UnitScratch& s,
                                                  Count units, Least least) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (n + THREADS - 1) / THREADS;
  const int a = min(n, tid * run), b = min(n, a + run);
  long long sum = 0;
  int longest = 0;
  for (int i = a; i < b; ++i) {
    const Units x = units(i);
    sum += x.count;
    longest = max(longest, x.longest);
  }
  const long long inc = warp_inclusive(sum, lane);
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 31) {
    s.warp_sum[warp] = inc;
    s.warp_longest[warp] = longest;
  }
  if (tid == 0) {
    s.seq = n;
    s.off = 0;
  }
  __syncthreads();
  long long before = inc - sum, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += s.warp_sum[w];
    total += s.warp_sum[w];
    longest = max(longest, s.warp_longest[w]);
  }
  // ranges that hold units
  const int used = (int)min((long long)parts, max(total / least(longest), min(total, 1LL)));
  UnitRange r;
  r.total = total;
  r.used = used;
  r.u0 = part < used ? total * part / used : total;
  r.u1 = part < used ? total * (part + 1) / used : total;
  if (r.u0 < r.u1 && before <= r.u0 && r.u0 < before + sum) {
    long long at = before;
    for (int i = a; i < b; ++i) {
      const long long c = units(i).count;
      if (r.u0 < at + c) {
        s.seq = i;
        s.off = r.u0 - at;
        break;
      }
      at += c;
    }
  }
  __syncthreads();
  r.seq = s.seq;
  r.off = s.off;
  return r;
}

}  // namespace
}  // namespace avp
