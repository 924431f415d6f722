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
cudaError_t launch_kv_append(const AppendParams& p, cudaStream_t stream);
// The status word of fa_pages.cu (see fa_kernel.h).
cudaError_t read_pages_status(unsigned int* out);
cudaError_t clear_pages_status();

struct PrefixParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;  // the page pools
  const __nv_bfloat16* v;
  const int* prefix_table;
  const int* block_table;
  const int* seq_lens;
  const int* cu_new;
  __nv_bfloat16* o;
  float* lse;
  int N, B, H, Hkv, group;
  int prefix_len, causal;
  int num_pages, max_pages;
  float scale_log2;               // scale * log2(e)
  unsigned long long timeout_ns;  // bound on every in-kernel wait
  int ctas;      // blocks of the attention kernel: one per SM, at most kPrefixMaxCtas
  int few_rows;  // rows of a few-row item at most: 8 or 16
  int head_bytes;  // of a key's row: 2 d
  int step;      // keys per few-row step: 16 (d = 128) or 32
  int tiles_p;   // 128-key tiles of the prefix
  int tp;        // tokens of a 128-row tile
  // workspace
  int* hdr;           // kHdr* words
  int4* tok;          // [N] place of the token's own item (K/V head 0), its units, the units that the token's row
                      // tile sees, the token's number in the item | kTokFew | places of a unit << 16
  int* rank;          // [N] the token's item of the prefix (K/V head 0); -1: none
  int slab_rows;      // rows of a many-row slab
  float* slab_o;      // [ctas][2][slab_rows][d], then [ctas * kFewWarps][2][few_rows][d]: parts of cut items
  float* slab_lse;    // the same rows, base-2
  float* own_o;       // [N * H][d] parts of whole items of own keys
  float* own_lse;
  float* prefix_o;    // the same of the prefix
  float* prefix_lse;
};
constexpr int kPrefixMaxCtas = 160;
constexpr int kFewWarps = 8;  // warps of a block that work few rows
// q: bf16 (d, H, N) with boxes of 64 columns x group heads x tp tokens; k, v: the page pools as (64, 128 rows, d / 64,
// num_pages * Hkv) in boxes of whole pages, k16, v16: of `step` rows.
struct PrefixMaps {
  CUtensorMap q, k, v, k16, v16;
};
unsigned int prefix_page_cost();  // the most places a page and an item take on a line (see fa_prefix.cu)
unsigned int prefix_item_cost();
cudaError_t launch_fa_fwd_prefix(int d, const PrefixMaps& t, const PrefixParams& p, cudaStream_t stream);
cudaError_t read_prefix_status(unsigned int* out);
cudaError_t clear_prefix_status();

}  // namespace fa
