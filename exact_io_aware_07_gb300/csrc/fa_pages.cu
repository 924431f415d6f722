// Page plan and append for paged K/V caches (contracts in include/fa.h).
#include "fa_pages.h"

namespace fa {

static __device__ unsigned int g_pages_status;  // kStatus* bits

// ---------------------------------------------------------------- page plan
// With c_b, n_b the cached and new tokens of request b and s_b = c_b + n_b, the requests'
// first new token and first new page are running sums of n_b and ceil(s_b/128) - ceil(c_b/128).
// Every block forms both sums for all requests, 1024 requests at a time in one packed 64-bit
// scan, and keeps them in shared memory; the blocks share out the tokens and the new pages of
// those requests, each thread finding its request by bisection.  Blocks need nothing from one
// another: a kept table entry (read for the tokens that fill up a page) is never written.
//
// Bound by latency, not by its bytes (310 KB for 2 000 requests, 0.05 us at the rate of the memory): lengths, scan and
// barriers, a bisection in shared memory, one dependent load of a page, stores.  In a graph 2.8 us for 64 decoding requests,
// 3.2 for 7 prompts of up to 9 000 tokens, 6.9 for 2 000 requests with 62 000 tokens.  A thread takes one request, so those
// 2 000 are two scans of 1024 one behind the other; a thread with two or more would need one, and more shared memory (not
// built).  One kernel, every block with the whole scan: a scan over blocks would add a launch or a wait between blocks (2 us).
constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int pages_of(int n) { return (n >> 7) + ((n & 127) != 0); }

// Index of the last of the ascending first[0 .. n-1] that is <= x (first[0] <= x).
__device__ __forceinline__ int last_not_above(const int* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) fa_page_plan_kernel(const PlanParams p) {
  __shared__ int s_tok[kPlanThreads + 1], s_page[kPlanThreads + 1], s_ctx[kPlanThreads];
  __shared__ unsigned long long s_warp[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int stride = gridDim.x * kPlanThreads, me = blockIdx.x * kPlanThreads + tid;
  unsigned int bad = 0;
  const int head = *p.free_head;
  // page of the f-th page this step takes; -1 (and an error) past the list or outside the pool
  auto fresh_page = [&](int f) -> int {
    const long long at = static_cast<long long>(head) + f;
    if (at < 0 || at >= p.num_free) {
      bad |= kStatusNoPages;
      return -1;
    }
    const int pg = p.free_pages[at];
    if (pg >= 0 && pg < p.num_pages) return pg;
    bad |= kStatusBadPage;
    return -1;
  };
  unsigned long long carry = 0;  // tokens (low half) and new pages (high half) of the requests so far
  int next_c = tid < p.B ? p.ctx_lens[tid] : 0, next_n = tid < p.B ? p.new_lens[tid] : 0;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + tid, count = min(kPlanThreads, p.B - b0);
    int c = next_c, n = next_n;
    if (p.B - b > kPlanThreads) {  // the next requests' lengths load while these are scanned
      next_c = p.ctx_lens[b + kPlanThreads];
      next_n = p.new_lens[b + kPlanThreads];
    }
    if (b < p.B) {
      if (c < 0 || n < 0 || static_cast<long long>(c) + n > static_cast<long long>(p.max_pages) * kPage) {
        bad |= kStatusBadLength;
        c = min(max(c, 0), p.max_pages * kPage);
        n = 0;
      }
    }
    if (b >= p.B) c = n = 0;
    const unsigned long long mine =
        static_cast<unsigned int>(n) | static_cast<unsigned long long>(pages_of(c + n) - pages_of(c)) << 32;
    unsigned long long sum = mine;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
      const unsigned long long t = __shfl_up_sync(0xffffffffu, sum, w);
      if (lane >= w) sum += t;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      unsigned long long t = s_warp[lane];
#pragma unroll
      for (int w = 1; w < 32; w <<= 1) {
        const unsigned long long u = __shfl_up_sync(0xffffffffu, t, w);
        if (lane >= w) t += u;
      }
      s_warp[lane] = t;
    }
    __syncthreads();
    const unsigned long long incl = carry + (warp ? s_warp[warp - 1] : 0) + sum, excl = incl - mine;
    s_tok[tid] = static_cast<int>(static_cast<unsigned int>(excl));
    s_page[tid] = static_cast<int>(excl >> 32);
    s_ctx[tid] = c;
    if (tid == kPlanThreads - 1) {
      s_tok[kPlanThreads] = static_cast<int>(static_cast<unsigned int>(incl));
      s_page[kPlanThreads] = static_cast<int>(incl >> 32);
    }
    if (b < p.B && blockIdx.x == 0) {
      p.seq_lens[b] = c + n;
      p.cu_new[b] = static_cast<int>(static_cast<unsigned int>(excl));
    }
    carry += s_warp[31];
    __syncthreads();
    const int tok0 = s_tok[0], tok1 = s_tok[kPlanThreads], page0 = s_page[0], page1 = s_page[kPlanThreads];
    for (int f = page0 + me; f < page1; f += stride) {
      const int r = last_not_above(s_page, count, f);
      p.block_table[static_cast<size_t>(b0 + r) * p.max_pages + pages_of(s_ctx[r]) + (f - s_page[r])] = fresh_page(f);
    }
    const int stop = min(tok1, p.max_tokens);
    for (unsigned int at = static_cast<unsigned int>(tok0) + me; at < static_cast<unsigned int>(stop); at += stride) {
      const int t = static_cast<int>(at);
      const int r = last_not_above(s_tok, count, t);
      const int pos = s_ctx[r] + (t - s_tok[r]), lp = pos >> 7, held = pages_of(s_ctx[r]);
      int pg;
      if (lp < held) {
        pg = p.block_table[static_cast<size_t>(b0 + r) * p.max_pages + lp];
        if (pg < 0 || pg >= p.num_pages) {
          bad |= kStatusBadPage;
          pg = -1;
        }
      } else {
        pg = fresh_page(s_page[r] + lp - held);
      }
      p.slot_map[t] = pg < 0 ? -1 : pg * kPage + (pos & 127);
    }
    __syncthreads();  // the next requests overwrite the sums
  }
  const int total = static_cast<int>(static_cast<unsigned int>(carry)), taken = static_cast<int>(carry >> 32);
  for (long long t = static_cast<long long>(total) + me; t < p.max_tokens; t += stride) p.slot_map[t] = -1;
  if (blockIdx.x == 0 && tid == 0) {
    p.cu_new[p.B] = total;
    const long long h = static_cast<long long>(head) + taken;
    *p.free_head_out = static_cast<int>(h < 0 ? 0 : h > p.num_free ? p.num_free : h);
    if (total > p.max_tokens) bad |= kStatusBadLength;
  }
  if (bad) atomicOr(&g_pages_status, bad);
}

cudaError_t launch_page_plan(const PlanParams& p, int num_sms, cudaStream_t stream) {
  // a thread per place of the slot map (8.9 -> 7.0 us for 62 000 tokens against four places one behind the other)
  const long long want = (static_cast<long long>(p.max_tokens) + kPlanThreads - 1) / kPlanThreads;
  const int grid = static_cast<int>(want < 1 ? 1 : want > num_sms ? num_sms : want);
  fa_page_plan_kernel<<<grid, kPlanThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- append
// One thread moves 16 bytes of one token's K row and the same 16 bytes of its V row: a head's 128 or 256 bytes are whole
// sectors on both sides, whatever the slots.  Bound by HBM, each byte read and written once: 16 384 tokens of 8 heads of 128
// take 21.6 us in a graph over three sets of inputs, 6.2 TB/s (92 % of the measured copy rate), 24.2 us launched one by one
// (5.6 TB/s); 64 tokens 1.7 us, which is a launch's latency.  Blocks of 128 threads (21.6 against 21.4 us in turn with 256, 22.1
// with 512; 64 tokens 1.6 and 1.8 against 1.5).  Stores that go first from L2 would save 0.4 us here, but the
// attention that follows reads these rows.
__global__ void __launch_bounds__(128) fa_kv_append_kernel(const AppendParams p) {
  const int chunks = p.Hkv * p.d / 8, per_head = p.d / 8;
  const long long at = static_cast<long long>(blockIdx.x) * 128 + threadIdx.x;
  const long long t = at / chunks;
  if (t >= p.N) return;
  const int c = static_cast<int>(at - t * chunks);
  const int slot = p.slot_map[t];
  if (slot < 0) return;
  const int page = slot / kPage;
  if (page >= p.num_pages) {
    if (c == 0) atomicOr(&g_pages_status, kStatusBadPage);
    return;
  }
  const int g = c / per_head, x = c - g * per_head;
  const size_t dst = (static_cast<size_t>(page) * p.Hkv + g) * kPage * p.d + static_cast<size_t>(slot % kPage) * p.d + x * 8;
  const uint4 k = *reinterpret_cast<const uint4*>(p.k_new + t * p.k_stride + c * 8);
  const uint4 v = *reinterpret_cast<const uint4*>(p.v_new + t * p.v_stride + c * 8);
  *reinterpret_cast<uint4*>(p.k_pages + dst) = k;
  *reinterpret_cast<uint4*>(p.v_pages + dst) = v;
}

cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t stream) {
  const long long threads = static_cast<long long>(p.N) * (p.Hkv * p.d / 8);
  fa_kv_append_kernel<<<static_cast<unsigned int>((threads + 127) / 128), 128, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t read_pages_status(unsigned int* out) {
  return cudaMemcpyFromSymbolAsync(out, g_pages_status, sizeof(unsigned int), 0, cudaMemcpyDeviceToHost, cudaStreamLegacy);
}
cudaError_t clear_pages_status() {
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_pages_status, &zero, sizeof(unsigned int));
}

}  // namespace fa
