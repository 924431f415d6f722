// Internal interface of the paged-cache step: page plan and append (fa_pages.cu), attention over
// a shared prefix and paged caches (fa_prefix.cu).
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace fa {

constexpr int kPage = 128;  // keys per page

// Bits of the device status words.
constexpr unsigned int kStatusTimeout = 1u, kStatusBadPage = 2u, kStatusBadLength = 4u, kStatusNoPages = 8u;

struct PlanParams {
  const int* ctx_lens;
  const int* new_lens;
  const int* free_pages;
  const int* free_head;
  int* block_table;
  int* seq_lens;
  int* cu_new;
  int* slot_map;
  int* free_head_out;
  int B, max_pages, num_pages, num_free, max_tokens;
};
cudaError_t launch_page_plan(const PlanParams& p, int num_sms, cudaStream_t stream);

struct AppendParams {
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  const int* slot_map;
  __nv_bfloat16* k_pages;
  __nv_bfloat16* v_pages;
  long long k_stride, v_stride;  // elements from one token to the next
  int N, Hkv, d, num_pages;
};
cudaError_t launch_kv_append(const AppendParams& p, int num_sms, cudaStream_t stream);
// Reads and clears the status word of fa_pages.cu.
cudaError_t read_and_clear_pages_status(cudaStream_t stream, unsigned int* out);

struct PrefixParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k_pages;
  const __nv_bfloat16* v_pages;
  const int* prefix_table;
  const int* block_table;
  const int* seq_lens;
  const int* cu_new;
  __nv_bfloat16* o;
  float* lse;
  int N, B, H, Hkv, group;
  int prefix_len, causal;
  int num_pages, max_pages;
  float scale_log2;  // scale * log2(e)
};
cudaError_t launch_fa_fwd_prefix(int d, const PrefixParams& p, cudaStream_t stream);
cudaError_t read_and_clear_prefix_status(cudaStream_t stream, unsigned int* out);

}  // namespace fa
