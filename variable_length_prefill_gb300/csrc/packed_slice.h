// A sequence's rows in a packed tensor.  Plain arithmetic, for the host as well.
#pragma once

#ifdef __CUDACC__
#define AVP_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define AVP_HOST_DEVICE inline
#endif

namespace avp {

struct PackedSlice {
  int lo, n;  // rows [lo, lo + n) of [0, total); n is 0 where the slice is empty
};

// The slice between two neighbours of cu_seqlens, of any value.  Both are cut to
// [0, total] before they are subtracted: the difference of what they hold may
// not fit 32 bits.
AVP_HOST_DEVICE PackedSlice packed_slice(int first, int next, int total) {
  const int lo = first < 0 ? 0 : (first < total ? first : total);
  const int hi = next < 0 ? 0 : (next < total ? next : total);
  return {lo, hi > lo ? hi - lo : 0};
}

}  // namespace avp
