// Attention of new tokens over a shared prefix and each request's own pages (contract in include/fa.h).
//
// Row (n, h) sees the prefix's keys and its request's own keys up to its place; with s_j the
// scaled scores, O = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m) and LSE = m + ln sum_j e^(s_j - m),
// formed in one pass with the running maximum m.
#include <math.h>

#include "fa_pages.h"
#include "ptx.cuh"

namespace fa {

static __device__ unsigned int g_prefix_status;  // kStatus* bits

// One warp per row; lane l holds columns l * D/32 .. of q and o.
template <int D>
__global__ void __launch_bounds__(256) fa_prefix_row_kernel(const PrefixParams p) {
  constexpr int C = D / 32;
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * 8 + threadIdx.x / 32;
  if (row >= static_cast<long long>(p.N) * p.H) return;
  const int n = static_cast<int>(row / p.H), h = static_cast<int>(row % p.H), g = h / p.group;
  if (n >= p.cu_new[p.B]) return;
  int b = 0, hi = p.B;
  while (hi - b > 1) {
    const int mid = (b + hi) >> 1;
    if (p.cu_new[mid] <= n)
      b = mid;
    else
      hi = mid;
  }
  const int first = p.cu_new[b], end = p.cu_new[b + 1], added = min(end, p.N) - first;
  if (end > p.N && lane == 0) atomicOr(&g_prefix_status, kStatusBadLength);
  int len = p.seq_lens[b];
  if (len < 0 || len > p.max_pages * kPage) {
    if (lane == 0) atomicOr(&g_prefix_status, kStatusBadLength);
    len = len < 0 ? 0 : p.max_pages * kPage;
  }
  const int own = p.causal ? max(0, min(len, len - added + (n - first) + 1)) : len;
  float q[C], o[C], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    q[c] = __bfloat162float(p.q[row * D + lane * C + c]) * p.scale_log2;
    o[c] = 0.f;
  }
  for (int part = 0; part < 2; ++part) {
    const int* table = part ? p.block_table + static_cast<size_t>(b) * p.max_pages : p.prefix_table;
    const int keys = part ? own : p.prefix_len;
    for (int j = 0; j < keys; ++j) {
      const int page = table[j / kPage];
      const bool in = page >= 0 && page < p.num_pages;
      if (!in && lane == 0) atomicOr(&g_prefix_status, kStatusBadPage);
      const size_t at = in ? ((static_cast<size_t>(page) * p.Hkv + g) * kPage + j % kPage) * D + lane * C : 0;
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < C; ++c) s += q[c] * (in ? __bfloat162float(p.k_pages[at + c]) : 0.f);
#pragma unroll
      for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
      const float m2 = fmaxf(m, s), r = exp2f(m - m2), e = exp2f(s - m2);
      m = m2;
      l = l * r + e;
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] = o[c] * r + e * (in ? __bfloat162float(p.v_pages[at + c]) : 0.f);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;  // no visible key: O = 0 (a NaN sum stays one)
#pragma unroll
  for (int c = 0; c < C; ++c) p.o[row * D + lane * C + c] = __float2bfloat16(o[c] * inv);
  if (lane == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}

cudaError_t launch_fa_fwd_prefix(int d, const PrefixParams& p, cudaStream_t stream) {
  const long long rows = static_cast<long long>(p.N) * p.H;
  const unsigned int grid = static_cast<unsigned int>((rows + 7) / 8);
  if (d == 64)
    fa_prefix_row_kernel<64><<<grid, 256, 0, stream>>>(p);
  else
    fa_prefix_row_kernel<128><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t read_and_clear_prefix_status(cudaStream_t stream, unsigned int* out) {
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return e;
  e = cudaMemcpyFromSymbol(out, g_prefix_status, sizeof(unsigned int));
  if (e != cudaSuccess || *out == 0) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_prefix_status, &zero, sizeof(unsigned int));
}

}  // namespace fa
