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
  int ctas;     // blocks of the attention kernel: one per SM, at most kPrefixMaxCtas
  int tiles_p;  // 128-key tiles of the prefix
  int tp, ts;   // tokens of a 128-row tile over the prefix / over own keys
  // workspace
  int* hdr;             // kHdr* words
  int* start;           // [ctas] the request a block's own keys begin with
  unsigned int* cum;    // [B] place of the request's first item
  int4* tok;            // [N] place of the token's own item (K/V head 0), its tiles, the tiles the token's row
                        // tile sees, the token's number within the item
  int slab_rows;        // rows of a slab
  float4* slab_o;       // [ctas][2][d / 4][slab_rows] parts of cut items, four columns each
  float* slab_lse;      // [ctas][2][slab_rows], base-2
  float4* own_o;        // [Hkv][d / 4][N * group] parts of whole items of own keys
  float* own_lse;       // [Hkv][N * group]
  float4* prefix_o;     // the same of the prefix
  float* prefix_lse;
};
constexpr int kPrefixMaxCtas = 160;
unsigned int prefix_tile_cost();  // places a key tile and an item take (see fa_prefix.cu)
unsigned int prefix_item_cost();
// qp, qs: bf16 (d, H, N) with boxes of 64 columns x group heads x tp / ts tokens; k, v: the page pools.
cudaError_t launch_fa_fwd_prefix(int d, const CUtensorMap& qp, const CUtensorMap& qs, const CUtensorMap& k,
                                 const CUtensorMap& v, const PrefixParams& p, cudaStream_t stream);
cudaError_t read_and_clear_prefix_status(cudaStream_t stream, unsigned int* out);

}  // namespace fa
