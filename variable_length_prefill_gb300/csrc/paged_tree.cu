// Attention of drafted tokens over a paged cache (include/paged_attn_tree.h).
//
// The plain form: one CTA per (packed row, query head) walks the row's keys in
// tiles of 128, one key a thread, with a running maximum and sum.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "paged_tree_internal.h"
#include "ptx.cuh"

namespace avp {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) tree_plain_kernel(const __grid_constant__ TreeParams p) {
  __shared__ float s_q[D], s_p[kThreads], s_red[4];
  __shared__ uint32_t s_sees[kTreeMaxDrafts / 32];
  const int row = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
  const int group = p.num_query_heads / p.c.num_kv_heads, g = h / group;
  for (int seq = 0; seq < p.c.num_seqs; ++seq) {
    const int lo = max(__ldg(p.cu + seq), 0);
    const int n = max(min(__ldg(p.cu + seq + 1), p.total_q) - lo, 0);
    if (row < lo || row >= lo + n) continue;
    const int j = row - lo;
    int len = max(__ldg(p.seq_lens + seq), 0);
    const int base = len - n;
    len = (int)min((long long)len, (long long)p.c.max_blocks * kPageTokens);
    if (n > kTreeMaxDrafts) {
      len = 0;
      if (tid == 0) atomicOr(p.c.status, kPageStatusBadDraft);
    }
    const size_t at = ((size_t)row * p.num_query_heads + h) * D;
    __syncthreads();
    for (int d = tid; d < D; d += kThreads) s_q[d] = to_f32(static_cast<const T*>(p.query)[at + d]);
    if (tid == 0 && n <= kTreeMaxDrafts) {
      for (int w = 0; w < kTreeMaxDrafts / 32; ++w) s_sees[w] = 0;
      for (int a = j; a >= 0;) {
        s_sees[a >> 5] |= 1u << (a & 31);
        int up = p.parents ? __ldg(p.parents + lo + a) : a - 1;
        if (up < -1 || up >= a) {
          up = -1;
          atomicOr(p.c.status, kPageStatusBadDraft);
        }
        a = up;
      }
    }
    __syncthreads();
    float m = -INFINITY, l = 0.f, o[(D + kThreads - 1) / kThreads] = {};
    bool seen_any = false;
    for (int p0 = 0; p0 < len; p0 += kThreads) {
      const int pos = p0 + tid;
      bool sees = pos < len;
      if (sees && pos >= base) sees = s_sees[(pos - base) >> 5] >> ((pos - base) & 31) & 1;
      float sc = -INFINITY;
      if (pos < len) {
        const int id = __ldg(p.block_tables + (size_t)seq * p.c.max_blocks + pos / kPageTokens);
        if (id < 0 || id >= p.c.num_blocks) {
          sees = false;
          atomicOr(p.c.status, kPageStatusBadBlock);
        }
        if (sees) {
          const T* k = static_cast<const T*>(p.c.k_cache) +
                       ((size_t)id * p.c.num_kv_heads + g) * D * kPageTokens +
                       (pos % kPageTokens) * 8;
          sc = 0.f;
          for (int d = 0; d < D; ++d)
            sc = fmaf(s_q[d], to_f32(k[(d / 8) * kPageTokens * 8 + d % 8]), sc);
          sc *= p.scale_log2;
        }
      }
      seen_any |= __syncthreads_or(sees);
      float top = sc;
      for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      if (tid % 32 == 0) s_red[tid / 32] = top;
      __syncthreads();
      top = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
      const float mn = fmaxf(m, top), alpha = mn == -INFINITY ? 1.f : ex2(m - mn);
      m = mn;
      // a negative weight marks what the row does not see
      s_p[tid] = sees ? (mn == -INFINITY ? 0.f : ex2(sc - mn)) : -1.f;
      __syncthreads();
      l *= alpha;
      for (int t = 0; t < kThreads; ++t) l += fmaxf(s_p[t], 0.f);
      for (int e = 0; e < (D + kThreads - 1) / kThreads; ++e) {
        const int d = e * kThreads + tid;
        if (d >= D) break;
        o[e] *= alpha;
        for (int t = 0; t < kThreads; ++t) {
          if (s_p[t] < 0.f) continue;
          const int id =
              __ldg(p.block_tables + (size_t)seq * p.c.max_blocks + (p0 + t) / kPageTokens);
          o[e] = fmaf(s_p[t],
                      to_f32(static_cast<const T*>(
                          p.c.v_cache)[(((size_t)id * p.c.num_kv_heads + g) * D + d) * kPageTokens +
                                       (p0 + t) % kPageTokens]),
                      o[e]);
        }
      }
      __syncthreads();
    }
    for (int e = 0; e < (D + kThreads - 1) / kThreads; ++e)
      if (e * kThreads + tid < D)
        static_cast<T*>(p.out)[at + e * kThreads + tid] = from_f32<T>(seen_any ? o[e] / l : 0.f);
  }
}

}  // namespace

size_t tree_workspace_bytes(int) { return 16; }

template <int D>
static cudaError_t launch_d(const TreeParams& p, bool fp16, cudaStream_t stream) {
  const dim3 grid(p.total_q, p.num_query_heads);
  if (fp16)
    tree_plain_kernel<D, __half><<<grid, kThreads, 0, stream>>>(p);
  else
    tree_plain_kernel<D, __nv_bfloat16><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_tree(const TreeParams& p, bool fp16, EncodeTiledFn, cudaStream_t stream) {
  switch (p.c.head_size) {
    case 64: return launch_d<64>(p, fp16, stream);
    case 128: return launch_d<128>(p, fp16, stream);
    case 256: return launch_d<256>(p, fp16, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace avp
