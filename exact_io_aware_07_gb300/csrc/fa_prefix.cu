// Attention of new tokens over a shared prefix and each request's own pages (contract in include/fa.h).
//
// Row (n, h) sees the prefix's keys and its request's own keys up to its place; with s_j the scaled
// scores, O = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m) and LSE = m + ln sum_j e^(s_j - m).  The keys of a
// row are cut into parts that run on different SMs, each giving (O_p, LSE_p); a row's parts join as
//   LSE = ln sum_p e^LSE_p,   O = sum_p e^(LSE_p - LSE) O_p,
// which is the softmax over all keys, so that the prefix can be worked once for the rows of the whole
// batch and the own keys request by request.
//
// Three kernels on the stream, each starting its set-up while the one before it ends:
//   fa_prefix_plan_kernel  lays out the work from the device lengths,
//   fa_prefix_kernel       one block per SM, tcgen05 products over its share of the key tiles,
//   fa_prefix_join_kernel  joins the parts of every row.
//
// The work is a list of items: (K/V head, up to two row tiles of 128 rows, the 128-key tiles of one
// source).  The items of the prefix come first: rows are the (token, query head) pairs of the whole
// batch, `group` rows per token, so a K/V tile is loaded once for up to 256 rows.  Then the items of
// every request's own keys.  Every key tile takes kTileCost places on a line, every item kItemCost
// more, and SM c works the tiles whose places begin in [c Q, (c + 1) Q), Q = the line's length over
// the number of SMs: all SMs get the same share whatever the lengths, and at most two items of an SM
// are cut (its first and its last).
#include <math.h>

#include "fa_pages.h"
#include "ptx.cuh"

namespace fa {

static __device__ unsigned int g_prefix_status;  // kStatus* bits

constexpr unsigned int kTileCost = 4, kItemCost = 4;
enum { kHdrTotal, kHdrShare, kHdrPrefix, kHdrBlocks, kHdrTokens };  // words of p.hdr

__device__ __forceinline__ unsigned int item_cost(int tiles) { return tiles ? kItemCost + kTileCost * tiles : 0u; }
// First tile of an item of `tiles` tiles beginning at c0 whose place is not before x.
__device__ __forceinline__ int tile_from(unsigned int x, unsigned int c0, int tiles) {
  if (x <= c0 + kItemCost) return 0;
  const unsigned int j = (x - c0 - kItemCost + kTileCost - 1) / kTileCost;
  return j < static_cast<unsigned int>(tiles) ? static_cast<int>(j) : tiles;
}

struct Request {
  int first, added, len;  // first new token, new tokens, own keys
};
__device__ __forceinline__ Request make_request(const PrefixParams& p, int cu0, int cu1, int seq) {
  Request r;
  r.first = min(max(cu0, 0), p.N);
  r.added = min(max(cu1, r.first), p.N) - r.first;
  r.len = min(max(seq, 0), p.max_pages * kPage);
  return r;
}
__device__ __forceinline__ int tiles_of(int keys) { return (keys + kPage - 1) / kPage; }
// Own keys that the tokens before the request's token `end` (exclusive) can see at most.
__device__ __forceinline__ int visible(const PrefixParams& p, const Request& r, int end) {
  return p.causal ? max(0, min(r.len, r.len - r.added + end)) : r.len;
}
__device__ __forceinline__ int block_tiles(const PrefixParams& p, const Request& r, int blk) {
  return tiles_of(visible(p, r, min(r.added, (blk + 1) * 2 * p.ts)));
}

// ---------------------------------------------------------------- plan
// Every block forms the running sum of the requests' costs, kPlanThreads requests at a time; block 0
// writes it out with the share Q and the request each SM begins with, and the blocks share out the
// tokens, whose item (place, cost, visible tiles, row) the join needs.
constexpr int kPlanThreads = 512;

__global__ void __launch_bounds__(kPlanThreads) fa_prefix_plan_kernel(const PrefixParams p) {
  __shared__ unsigned int s_cum[kPlanThreads + 1];
  __shared__ int s_first[kPlanThreads], s_added[kPlanThreads], s_len[kPlanThreads];
  __shared__ unsigned int s_warp[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_launch_dependents();
  pdl_wait();
  const int end = p.cu_new[p.B], tokens = min(max(end, 0), p.N);
  const int blocks = (tokens + 2 * p.tp - 1) / (2 * p.tp);
  const unsigned int prefix_cost = static_cast<unsigned int>(p.Hkv) * blocks * item_cost(p.tiles_p);
  bool bad = end > p.N || end < 0 || p.cu_new[0] != 0;
  const bool one = p.B <= kPlanThreads;  // a single round: the sum is known before it is used
  unsigned int total = 0, share = 1;
  for (int pass = one ? 1 : 0; pass < 2; ++pass) {  // pass 0 only sums
    unsigned int carry = prefix_cost;
    for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
      const int b = b0 + tid, count = min(kPlanThreads, p.B - b0);
      Request r{0, 0, 0};
      unsigned int mine = 0;
      if (b < p.B) {
        const int c0 = p.cu_new[b], c1 = p.cu_new[b + 1], seq = p.seq_lens[b];
        bad |= c1 < c0 || seq < 0 || seq > p.max_pages * kPage;
        r = make_request(p, c0, c1, seq);
        for (int blk = 0; blk * 2 * p.ts < r.added; ++blk) mine += item_cost(block_tiles(p, r, blk));
        mine *= p.Hkv;
      }
      unsigned int sum = mine;
#pragma unroll
      for (int w = 1; w < 32; w <<= 1) {
        const unsigned int t = __shfl_up_sync(0xffffffffu, sum, w);
        if (lane >= w) sum += t;
      }
      if (lane == 31) s_warp[warp] = sum;
      __syncthreads();
      unsigned int before = 0, all = 0;
#pragma unroll
      for (int w = 0; w < kPlanThreads / 32; ++w) {
        const unsigned int t = s_warp[w];
        before += w < warp ? t : 0u;
        all += t;
      }
      const unsigned int cum = carry + before + sum - mine;
      carry += all;
      if (pass == 1) {
        s_cum[tid] = cum;
        s_first[tid] = r.first;
        s_added[tid] = r.added;
        s_len[tid] = r.len;
        if (blockIdx.x == 0 && b < p.B) p.cum[b] = cum;
        if (one) {
          total = carry;
          share = max(1u, (total + p.ctas - 1) / p.ctas);
        }
      }
      __syncthreads();
      if (pass == 0) continue;
      const unsigned int c_begin = s_cum[0];
      if (blockIdx.x == 0)  // the request that holds place max(c * share, prefix_cost) of SM c
        for (int c = tid; c < p.ctas; c += kPlanThreads) {
          const unsigned int x = max(static_cast<unsigned int>(c) * share, prefix_cost);
          if (x < c_begin || x >= carry) continue;
          int lo = 0, hi = count;  // the last request beginning at or before x
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_cum[mid] <= x)
              lo = mid;
            else
              hi = mid;
          }
          p.start[c] = b0 + lo;
        }
      const int n_begin = b0 == 0 ? 0 : s_first[0], n_end = s_first[count - 1] + s_added[count - 1];
      for (int n = n_begin + blockIdx.x * kPlanThreads + tid; n < n_end; n += gridDim.x * kPlanThreads) {
        int lo = 0, hi = count;  // the last request whose first token is at or before n
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (s_first[mid] <= n)
            lo = mid;
          else
            hi = mid;
        }
        const Request q{s_first[lo], s_added[lo], s_len[lo]};
        const int i = n - q.first;
        int4 t = make_int4(0, 0, 0, 0);  // no own key
        if (i >= 0 && i < q.added) {
          const int blk = i / (2 * p.ts);
          unsigned int c0 = s_cum[lo];
          for (int k = 0; k < blk; ++k) c0 += p.Hkv * item_cost(block_tiles(p, q, k));
          const int tile = i / p.ts;
          t = make_int4(static_cast<int>(c0), block_tiles(p, q, blk),
                        tiles_of(visible(p, q, min(q.added, (tile + 1) * p.ts))), i - blk * 2 * p.ts);
        }
        p.tok[n] = t;
      }
      __syncthreads();
    }
    total = carry;
    share = max(1u, (total + p.ctas - 1) / p.ctas);
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.hdr[kHdrTotal] = static_cast<int>(total);
    p.hdr[kHdrShare] = static_cast<int>(share);
    p.hdr[kHdrPrefix] = static_cast<int>(prefix_cost);
    p.hdr[kHdrBlocks] = blocks;
    p.hdr[kHdrTokens] = tokens;
  }
  if (bad && blockIdx.x == 0) atomicOr(&g_prefix_status, kStatusBadLength);
}

// ---------------------------------------------------------------- attention
// Roles (one block per SM): warps 0-3 and 4-7 the softmax of slot 0 and slot 1 (a thread has one of
// 128 rows), warp 8 the producer (lays out the SM's pieces, issues the TMA loads), warp 9 the
// tcgen05.mma issuer.  A piece is the SM's share of an item, in one of two forms:
//   two row tiles: each slot holds one, both visit every key tile (a tile is loaded once);
//   one row tile (a decoding request has `group` rows): the slots take its key tiles in turn, so that
//   one's softmax overlaps the other's products, and slot 0 joins both results at the end.
// Tensor Memory (512 columns): S_0 [0,128), S_1 [128,256), O_0, O_1 from 256; P_i (bf16 pairs) over S_i.
constexpr int BM = 128, BN = 128;
constexpr int PRODUCER_WARP = 8, MMA_WARP = 9, THREADS = 320;
constexpr int BOX_BYTES = 128 * 128;  // 128 rows x 64 bf16, 128-byte swizzle
constexpr float LN2 = 0.693147180559945309f;
constexpr int kPieceSlots = 3;

struct __align__(16) Piece {
  int mode;          // 0: no more pieces, 1: one row tile, 2: two row tiles
  int n, n0, n1;     // key tiles of the piece; visited by slot 0 / slot 1
  int j0;            // first key tile
  int keys;          // keys of the source
  int lim0, step;    // the item's token i sees min(keys, lim0 + i * step) of them
  int t0;            // the item's first token
  int rows0, rows1;  // rows of tile 0 / tile 1
  int g;             // K/V head
  int dst;           // where the part goes: kDst*
  int tile_rows;     // rows of a full row tile
  int pad0, pad1;
};
enum { kDstOutput, kDstSlab0, kDstSlab1, kDstOwn, kDstPrefix };

template <int D>
struct PLayout {
  static constexpr int TILE_BYTES = BM * D * 2;
  static constexpr int BOXES = D / 64;
  static constexpr int STAGES = D == 128 ? 5 : 10;
  static constexpr int KV_OFF = 2 * TILE_BYTES;  // after the two query tiles
  static constexpr int XCH_OFF = KV_OFF + STAGES * TILE_BYTES;  // slot 1's (m, l, lr) of one-tile pieces
  static constexpr int PIECE_OFF = XCH_OFF + 128 * 12;
  static constexpr int BAR_OFF = PIECE_OFF + kPieceSlots * int(sizeof(Piece));
  // q_full, q_empty, kv_full[S], kv_empty[S], s_full[2], p_full[2], o_full[2], o_empty[2], x_full[4], done,
  // piece_full[], piece_empty[]
  static constexpr int NUM_BARS = 2 + 2 * STAGES + 8 + 4 + 1 + 2 * kPieceSlots;
  static constexpr int MISC_OFF = BAR_OFF + NUM_BARS * 8;  // TMEM base, abort flag
  static constexpr int SMEM_BYTES = MISC_OFF + 16 + 1024;
};
static_assert(PLayout<64>::SMEM_BYTES <= 232448 && PLayout<128>::SMEM_BYTES <= 232448, "shared memory");

__device__ __forceinline__ float u2f(uint32_t x) { return __uint_as_float(x); }
__device__ __forceinline__ uint32_t f2u(float x) { return __float_as_uint(x); }

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
fa_prefix_kernel(const __grid_constant__ CUtensorMap tmQp, const __grid_constant__ CUtensorMap tmQs,
                 const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                 const PrefixParams p) {
  using L = PLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t kv_smem = sbase + L::KV_OFF;
  const uint32_t bar = sbase + L::BAR_OFF;
  const uint32_t bar_q_full = bar, bar_q_empty = bar + 8;
  const uint32_t bar_kv_full = bar + 16, bar_kv_empty = bar_kv_full + 8 * L::STAGES;
  const uint32_t bar_s_full = bar_kv_empty + 8 * L::STAGES, bar_p_full = bar_s_full + 16;
  const uint32_t bar_o_full = bar_s_full + 32, bar_o_empty = bar_s_full + 48;
  const uint32_t bar_x_full = bar_s_full + 64, bar_done = bar_x_full + 32;
  const uint32_t bar_piece_full = bar_done + 8, bar_piece_empty = bar_piece_full + 8 * kPieceSlots;
  volatile Piece* pieces = reinterpret_cast<volatile Piece*>(smem + L::PIECE_OFF);
  volatile float* xch = reinterpret_cast<volatile float*>(smem + L::XCH_OFF);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::MISC_OFF + 4);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    mbar_init(bar_q_full, 1);
    mbar_init(bar_q_empty, 1);
    for (int s = 0; s < L::STAGES; ++s) {
      mbar_init(bar_kv_full + 8 * s, 1);
      mbar_init(bar_kv_empty + 8 * s, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_s_full + 8 * i, 1);
      mbar_init(bar_p_full + 8 * i, 4);
      mbar_init(bar_o_full + 8 * i, 1);
      mbar_init(bar_o_empty + 8 * i, 4);
    }
    for (int w = 0; w < 4; ++w) mbar_init(bar_x_full + 8 * w, 1);
    mbar_init(bar_done, 1);
    for (int s = 0; s < kPieceSlots; ++s) {
      mbar_init(bar_piece_full + 8 * s, 1);
      mbar_init(bar_piece_empty + 8 * s, 9);  // every softmax warp and the MMA warp reads each piece
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == MMA_WARP) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  if (warp == PRODUCER_WARP && lane == 0) {
    tma_prefetch_desc(&tmQp);
    tma_prefetch_desc(&tmQs);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Waiter W{abort_flag, p.timeout_ns, &g_prefix_status};
  pdl_launch_dependents();
  pdl_wait();

  if (warp == PRODUCER_WARP) {
    const unsigned int total = p.hdr[kHdrTotal], share = p.hdr[kHdrShare], prefix_cost = p.hdr[kHdrPrefix];
    const int blocks = p.hdr[kHdrBlocks], tokens = p.hdr[kHdrTokens];
    const unsigned int x0 = blockIdx.x * share, x1 = min(total, x0 + share);
    int stage = 0, np = 0;
    uint32_t phase = 0, issued = 0, issued_parity = 0;
    bool ok = true;
    // page numbers of 32 tiles of one table row, one per lane
    const int* held_table = nullptr;
    int held_base = -1, held_page = 0;
    auto kv_load = [&](const CUtensorMap* map, const int* table, int tile, int g) -> bool {
      if (table != held_table || (tile & ~31) != held_base) {
        held_table = table;
        held_base = tile & ~31;
        const int limit = table == p.prefix_table ? p.tiles_p : p.max_pages;
        held_page = held_base + lane < limit ? table[held_base + lane] : 0;
      }
      int pg = __shfl_sync(0xffffffffu, held_page, tile & 31);
      if (pg < 0 || pg >= p.num_pages) {  // out of the pool: reads zeros and is reported
        if (lane == 0) atomicOr(&g_prefix_status, kStatusBadPage);
        pg = p.num_pages;
      }
      if (!wait_all(W, bar_kv_empty + 8 * stage, phase ^ 1)) return false;
      mbar_arrive_expect_tx_elect(bar_kv_full + 8 * stage, L::TILE_BYTES);
#pragma unroll
      for (int b = 0; b < L::BOXES; ++b)
        tma_load_3d_elect(kv_smem + stage * L::TILE_BYTES + b * BOX_BYTES, map, b * 64, 0, pg * p.Hkv + g,
                          bar_kv_full + 8 * stage);
      issued |= 1u << stage;
      issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
      if (++stage == L::STAGES) {
        stage = 0;
        phase ^= 1;
      }
      return true;
    };
    auto publish = [&](const Piece& q) -> bool {
      const int s = np % kPieceSlots;
      if (!wait_all(W, bar_piece_empty + 8 * s, ((np / kPieceSlots) & 1) ^ 1)) return false;
      if (lane == 0) {
        const int* src = reinterpret_cast<const int*>(&q);
        volatile int* dst = reinterpret_cast<volatile int*>(pieces + s);
#pragma unroll
        for (int w = 0; w < 14; ++w) dst[w] = src[w];
        mbar_arrive(bar_piece_full + 8 * s);
      }
      __syncwarp();
      ++np;
      return true;
    };
    // Emits this SM's tiles [j0, j1) of an item: tokens [t0, t0 + count) in row tiles of tile_tokens.
    auto emit = [&](bool own, const int* table, int g, int t0, int count, int tile_tokens, int tiles, int tiles0, int j0,
                    int j1, int keys, int lim0, int step) -> bool {
      Piece q;
      q.n = j1 - j0;
      q.mode = count > tile_tokens ? 2 : 1;
      q.n0 = q.mode == 2 ? max(0, min(tiles0, j1) - j0) : (q.n + 1) / 2;
      q.n1 = q.mode == 2 ? q.n : q.n / 2;
      q.j0 = j0;
      q.keys = keys;
      q.lim0 = lim0;
      q.step = step;
      q.t0 = t0;
      q.tile_rows = tile_tokens * p.group;
      q.rows0 = min(count, tile_tokens) * p.group;
      q.rows1 = max(0, count - tile_tokens) * p.group;
      q.g = g;
      q.dst = j0 > 0 ? kDstSlab0 : j1 < tiles ? kDstSlab1 : !own ? kDstPrefix : p.tiles_p > 0 ? kDstOwn : kDstOutput;
      const int k = np;
      if (!publish(q)) return false;
      if (!wait_all(W, bar_q_empty, (k & 1) ^ 1)) return false;
      const CUtensorMap* qm = own ? &tmQs : &tmQp;
      const uint32_t box = static_cast<uint32_t>(q.tile_rows) * 128;
      mbar_arrive_expect_tx_elect(bar_q_full, box * L::BOXES * q.mode);
      for (int i = 0; i < q.mode; ++i)
#pragma unroll
        for (int b = 0; b < L::BOXES; ++b)
          tma_load_3d_elect(sbase + i * L::TILE_BYTES + b * BOX_BYTES, qm, b * 64, g * p.group, t0 + i * tile_tokens,
                            bar_q_full);
      if (q.mode == 1) {  // K_0 K_1 V_0 K_2 V_1 K_3 ...
        if (!kv_load(&tmK, table, j0, g) || (q.n > 1 && !kv_load(&tmK, table, j0 + 1, g))) return false;
        for (int j = j0; j < j1; ++j)
          if (!kv_load(&tmV, table, j, g) || (j + 2 < j1 && !kv_load(&tmK, table, j + 2, g))) return false;
      } else {
        for (int j = j0; j < j1; ++j)
          if (!kv_load(&tmK, table, j, g) || !kv_load(&tmV, table, j, g)) return false;
      }
      return true;
    };

    if (x0 < x1 && x0 < prefix_cost) {  // items of the prefix: head by head, block of rows by block
      const unsigned int cost = item_cost(p.tiles_p);
      const int items = p.Hkv * blocks;
      for (int it = x0 / cost; ok && it < items && it * cost < x1; ++it) {
        const unsigned int c0 = it * cost;
        const int j0 = tile_from(x0, c0, p.tiles_p), j1 = tile_from(x1, c0, p.tiles_p);
        if (j0 >= j1) continue;
        const int g = it / blocks, t0 = (it - g * blocks) * 2 * p.tp;
        ok = emit(false, p.prefix_table, g, t0, min(2 * p.tp, tokens - t0), p.tp, p.tiles_p, p.tiles_p, j0, j1,
                  p.prefix_len, p.prefix_len, 0);
      }
    }
    if (ok && x0 < x1 && x1 > prefix_cost) {  // items of own keys: requests, blocks of tokens, heads
      int b = p.start[blockIdx.x], base = b - 32;
      int r_cu0 = 0, r_cu1 = 0, r_seq = 0;
      unsigned int r_cum = 0;
      for (bool more = true; ok && more && b < p.B; ++b) {
        if (b >= base + 32) {  // 32 requests at a time, one per lane
          base = b;
          const int l = min(b + lane, p.B - 1);
          r_cu0 = p.cu_new[l];
          r_cu1 = p.cu_new[l + 1];
          r_seq = p.seq_lens[l];
          r_cum = p.cum[l];
        }
        const Request r = make_request(p, __shfl_sync(0xffffffffu, r_cu0, b - base), __shfl_sync(0xffffffffu, r_cu1, b - base),
                                       __shfl_sync(0xffffffffu, r_seq, b - base));
        unsigned int c0 = __shfl_sync(0xffffffffu, r_cum, b - base);
        if (c0 >= x1) break;
        const int* table = p.block_table + static_cast<size_t>(b) * p.max_pages;
        for (int t = 0; ok && t < r.added; t += 2 * p.ts) {
          const int count = min(2 * p.ts, r.added - t), tiles = tiles_of(visible(p, r, t + count));
          const unsigned int cost = item_cost(tiles);
          if (c0 >= x1) {
            more = false;
            break;
          }
          if (tiles == 0 || c0 + p.Hkv * cost <= x0) {
            c0 += p.Hkv * cost;
            continue;
          }
          const int tiles0 = tiles_of(visible(p, r, min(r.added, t + p.ts)));
          for (int g = x0 > c0 ? (x0 - c0) / cost : 0; ok && g < p.Hkv && c0 + g * cost < x1; ++g) {
            const int j0 = tile_from(x0, c0 + g * cost, tiles), j1 = tile_from(x1, c0 + g * cost, tiles);
            if (j0 < j1)
              ok = emit(true, table, g, r.first + t, count, p.ts, tiles, tiles0, j0, j1, r.len,
                        p.causal ? r.len - r.added + t + 1 : r.len, p.causal);
          }
          c0 += p.Hkv * cost;
        }
      }
    }
    if (ok) {
      Piece q;
      q.mode = 0;
      q.n = q.n0 = q.n1 = q.j0 = q.keys = q.lim0 = q.step = q.t0 = q.rows0 = q.rows1 = q.g = q.dst = q.tile_rows = 0;
      ok = publish(q);
    }
    if (!ok) {  // let every copy already issued land before the block exits
      if (np > 0) drain_all(W, bar_q_full, (np - 1) & 1);
      for (int s = 0; s < L::STAGES; ++s)
        if (issued & (1u << s)) drain_all(W, bar_kv_full + 8 * s, (issued_parity >> s) & 1u);
    }
    __syncwarp();
  } else if (warp == MMA_WARP) {
    constexpr uint32_t IDESC_S = make_idesc_bf16(BM, BN, 0);  // S = Q K^T: both K-major
    constexpr uint32_t IDESC_PV = make_idesc_bf16(BM, D, 1);  // O += P V: V is MN-major
    const uint64_t dqk = make_sdesc_sw128(sbase, 16, 1024), dvv = make_sdesc_sw128(sbase, BOX_BYTES, 1024);
    const uint32_t dqk_lo = uint32_t(dqk), dqk_hi = uint32_t(dqk >> 32);
    const uint32_t dv_lo = uint32_t(dvv), dv_hi = uint32_t(dvv >> 32);
    int stage = 0;
    uint32_t phase = 0, pf = 0, oe = 0;  // bit i: slot i's next parity of p_full, o_empty
    bool ok = true;
    auto take = [&](int& slot) -> bool {  // the ring's next tile
      slot = stage;
      if (!wait_all(W, bar_kv_full + 8 * stage, phase)) return false;
      if (++stage == L::STAGES) {
        stage = 0;
        phase ^= 1;
      }
      tc_fence_after();
      return true;
    };
    auto issue_s = [&](int slot, int qtile, int ks) {  // S_slot = Q_qtile K^T, d in steps of 16
      const uint32_t a0 = dqk_lo + ((qtile * L::TILE_BYTES) >> 4);
      const uint32_t b0 = dqk_lo + ((L::KV_OFF + ks * L::TILE_BYTES) >> 4);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk / 4) * BOX_BYTES + (kk % 4) * 32) >> 4;
        mma_ss_elect(tmem + slot * 128, a0 + off, dqk_hi, b0 + off, dqk_hi, IDESC_S, kk > 0 ? 1u : 0u);
      }
      mma_commit_elect(bar_s_full + 8 * slot);
    };
    // The last tile of a source holds fewer than 128 keys, and what its page holds behind them may be
    // anything.  Their weights are 0, but 0 times an infinity or NaN is not: the product runs over the keys
    // in steps of 16 as far as there are keys, and the value rows behind the last key in its last step are
    // set to 0.  Returns the steps.
    auto value_steps = [&](const Piece& q, int tile, int vs) -> int {
      const int valid = q.keys - tile * BN;
      if (valid >= BN) return BN / 16;
      const int steps = (valid + 15) / 16, words = (steps * 16 - valid) * 8;  // 16-byte words per box
      for (int w = lane; w < words * L::BOXES; w += 32) {
        const int box = w / words, at = w - box * words;
        st_shared_v4(kv_smem + vs * L::TILE_BYTES + box * BOX_BYTES + valid * 128 + at * 16, 0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      return steps;
    };
    auto issue_pv = [&](int slot, int vs, int steps, bool acc) {  // O_slot (+)= P_slot V, keys in steps of 16
      const uint32_t b0 = dv_lo + ((L::KV_OFF + vs * L::TILE_BYTES) >> 4);
#pragma unroll
      for (int kk = 0; kk < BN / 16; ++kk)
        if (kk < steps)
          mma_ts_elect(tmem + 256 + slot * D, tmem + slot * 128 + kk * 8, b0 + ((kk * 2048) >> 4), dv_hi, IDESC_PV,
                       (acc || kk > 0) ? 1u : 0u);
    };
    auto ready_pv = [&](int slot, bool first) -> bool {  // P_slot written; O_slot free at a piece's first product
      if (first) {
        if (!wait_all(W, bar_o_empty + 8 * slot, ((oe >> slot) & 1) ^ 1)) return false;
        oe ^= 1u << slot;
      }
      if (!wait_all(W, bar_p_full + 8 * slot, (pf >> slot) & 1)) return false;
      pf ^= 1u << slot;
      tc_fence_after();
      return true;
    };
    for (int k = 0; ok; ++k) {
      const int s = k % kPieceSlots;
      if (!(ok = wait_all(W, bar_piece_full + 8 * s, (k / kPieceSlots) & 1))) break;
      Piece q;
      q.mode = pieces[s].mode;
      q.n = pieces[s].n;
      q.n0 = pieces[s].n0;
      q.n1 = pieces[s].n1;
      q.j0 = pieces[s].j0;
      q.keys = pieces[s].keys;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_piece_empty + 8 * s);
      if (q.mode == 0) break;
      if (!(ok = wait_all(W, bar_q_full, k & 1))) break;
      tc_fence_after();
      int ks = 0, vs = 0;
      if (q.mode == 1) {
        for (int x = 0; ok && x < min(q.n, 2); ++x) {
          if (!(ok = take(ks))) break;
          issue_s(x, 0, ks);
          if (x + 1 == q.n) mma_commit_elect(bar_q_empty);
          mma_commit_elect(bar_kv_empty + 8 * ks);
        }
        for (int x = 0; ok && x < q.n; ++x) {
          const int slot = x & 1;
          if (!(ok = take(vs))) break;
          const int steps = value_steps(q, q.j0 + x, vs);
          if (!(ok = ready_pv(slot, x < 2))) break;
          issue_pv(slot, vs, steps, x >= 2);
          if (x + 2 >= q.n) mma_commit_elect(bar_o_full + 8 * slot);
          mma_commit_elect(bar_kv_empty + 8 * vs);
          if (x + 2 < q.n) {
            if (!(ok = take(ks))) break;
            issue_s(slot, 0, ks);
            if (x + 3 == q.n) mma_commit_elect(bar_q_empty);
            mma_commit_elect(bar_kv_empty + 8 * ks);
          }
        }
      } else {  // slot 1 visits every tile (n1 = n), slot 0 the first n0
        if (!(ok = take(ks))) break;
        if (q.n0 > 0) issue_s(0, 0, ks);
        issue_s(1, 1, ks);
        if (q.n == 1) mma_commit_elect(bar_q_empty);
        mma_commit_elect(bar_kv_empty + 8 * ks);
        for (int j = 0; j < q.n; ++j) {
          bool next = false;
          if (!(ok = take(vs))) break;
          const int steps = value_steps(q, q.j0 + j, vs);
          if (j < q.n0) {
            if (!(ok = ready_pv(0, j == 0))) break;
            issue_pv(0, vs, steps, j > 0);
            if (j + 1 == q.n0) mma_commit_elect(bar_o_full);
            if (j + 1 < q.n0) {
              if (!(ok = take(ks))) break;
              next = true;
              issue_s(0, 0, ks);
            }
          }
          if (!(ok = ready_pv(1, j == 0))) break;
          issue_pv(1, vs, steps, j > 0);
          if (j + 1 == q.n) mma_commit_elect(bar_o_full + 8);
          mma_commit_elect(bar_kv_empty + 8 * vs);
          if (j + 1 < q.n) {
            if (!next && !(ok = take(ks))) break;
            issue_s(1, 1, ks);
            if (j + 2 == q.n) mma_commit_elect(bar_q_empty);
            mma_commit_elect(bar_kv_empty + 8 * ks);
          }
        }
      }
    }
    // every MMA and every commit arrival has landed before TMEM is freed
    mma_commit_elect(bar_done);
    drain_all(W, bar_done, 0);
    __syncwarp();
  } else {
    const int i = warp / 4, wq = warp % 4, rt = wq * 32 + lane;
    const uint32_t lane_off = uint32_t(wq * 32) << 16;
    const uint32_t t_s = tmem + lane_off + i * 128, t_o = tmem + lane_off + 256 + i * D;
    const uint32_t my_s_full = bar_s_full + 8 * i, my_p_full = bar_p_full + 8 * i;
    const uint32_t my_o_full = bar_o_full + 8 * i;
    const int tok = rt / p.group, hh = rt - tok * p.group;  // the row's token within its tile, its head within the group
    const float sl2 = p.scale_log2;
    uint32_t sf_phase = 0, of_phase = 0, x_phase = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int s = k % kPieceSlots;
      if (!(ok = wait_all(W, bar_piece_full + 8 * s, (k / kPieceSlots) & 1))) break;
      const int mode = pieces[s].mode, n = pieces[s].n, n_mine = i ? pieces[s].n1 : pieces[s].n0, j0 = pieces[s].j0;
      const int rows = (mode == 2 && i) ? pieces[s].rows1 : pieces[s].rows0, g = pieces[s].g, dst = pieces[s].dst;
      const int tile_rows = pieces[s].tile_rows, t0 = pieces[s].t0;
      const int row0 = mode == 2 ? i * tile_rows : 0;  // the tile's first row within the item
      int lim = min(pieces[s].keys, pieces[s].lim0 + pieces[s].step * (row0 / p.group + tok));  // keys the row sees
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_piece_empty + 8 * s);
      if (mode == 0) break;
      if (n_mine == 0) continue;
      const bool live = rt < rows, live_warp = wq * 32 < rows;
      if (!live) lim = 0;
      float m_run = -INFINITY;  // reference max, base-2 units of the scaled score
      float l = 0.f, lr = 0.f;  // sums of the fp32 weights (LSE) and of the bf16 weights the product uses (divides O)
      for (int x = 0; x < n_mine; ++x) {
        if (!(ok = wait_all(W, my_s_full, sf_phase))) break;
        sf_phase ^= 1;
        tc_fence_after();
        if (live_warp) {
          uint32_t sr[BN];
          tmem_ld128_wait(t_s, sr);
          const int left = lim - (j0 + (mode == 1 ? 2 * x + i : x)) * BN;  // keys of this tile the row sees
          if (__any_sync(0xffffffffu, left < BN)) {
#pragma unroll
            for (int c = 0; c < BN; ++c)
              if (c >= left) sr[c] = f2u(-INFINITY);
          }
          float m8[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) m8[e] = u2f(sr[e]);
#pragma unroll
          for (int c = 8; c < BN; c += 8)
#pragma unroll
            for (int e = 0; e < 8; ++e) m8[e] = fmaxf(m8[e], u2f(sr[c + e]));
#pragma unroll
          for (int w = 4; w >= 1; w >>= 1)
#pragma unroll
            for (int e = 0; e < w; ++e) m8[e] = fmaxf(m8[e], m8[e + w]);
          const float mx = m8[0] * sl2;
          // the reference is moved, and l, lr and O rescaled, only when the maximum grows by more than 2^8
          float r = 1.f;
          bool rescale = false;
          if (x == 0) {
            m_run = mx;
          } else if (__any_sync(0xffffffffu, mx > m_run + 8.f)) {
            const float m_new = (mx > m_run + 8.f) ? mx : m_run;
            r = m_new == -INFINITY ? 1.f : ex2_approx(m_run - m_new);
            m_run = m_new;
            l *= r;
            lr *= r;
            rescale = true;
          }
          const float nm = m_run == -INFINITY ? 0.f : -m_run;  // no key seen yet: every weight is 2^(-inf) = 0
          float la0 = 0.f, la1 = 0.f, lb0 = 0.f, lb1 = 0.f, lr0 = 0.f, lr1 = 0.f;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float x0, x1;
              ffma2(x0, x1, u2f(sr[32 * c + 2 * e]), u2f(sr[32 * c + 2 * e + 1]), sl2, nm);
              const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
              if (e & 1)
                fadd2(lb0, lb1, p0, p1);
              else
                fadd2(la0, la1, p0, p1);
              pk[e] = pack_bf16x2(p0, p1);
              add_bf16x2_f32(pk[e], lr0, lr1);
            }
            tmem_st16(t_s + c * 16, pk);
          }
          l += (la0 + la1) + (lb0 + lb1);
          lr += lr0 + lr1;
          if (rescale) {  // this slot's last product was issued before S, so O is complete
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t ov[32];
              tmem_ld32_wait(t_o + c * 32, ov);
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] = f2u(u2f(ov[e]) * r);
              tmem_st32(t_o + c * 32, ov);
            }
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(my_p_full);
      }
      if (!ok) break;
      if (!(ok = wait_all(W, my_o_full, of_phase))) break;
      of_phase ^= 1;
      tc_fence_after();
      const bool pair = mode == 1 && n > 1;  // slot 0 joins both slots' results
      if (pair && i == 1) {
        xch[rt * 3] = m_run;
        xch[rt * 3 + 1] = l;
        xch[rt * 3 + 2] = lr;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_x_full + 8 * wq);
        continue;
      }
      float a0 = 1.f, a1 = 0.f;
      if (pair) {
        if (!(ok = wait_all(W, bar_x_full + 8 * wq, x_phase))) break;
        x_phase ^= 1;
        tc_fence_after();
        const float m1 = xch[rt * 3], l1 = xch[rt * 3 + 1], lr1 = xch[rt * 3 + 2];
        const float m = fmaxf(m_run, m1);
        a0 = m_run == -INFINITY ? 0.f : ex2_approx(m_run - m);
        a1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - m);
        m_run = m;
        l = a0 * l + a1 * l1;
        lr = a0 * lr + a1 * lr1;
      }
      if (live_warp) {
        const float inv = lr == 0.f ? 0.f : 1.f / lr;  // no key seen: O = 0 (a NaN sum stays one)
        const float lse2 = l == 0.f ? -INFINITY : m_run + log2f(l);
        a0 *= inv;
        a1 *= inv;
        const int row = row0 + rt;  // within the item
        float4* part = nullptr;     // the row's first four columns; the next four `stride` further on
        size_t stride = 0;
        __nv_bfloat16* out = nullptr;
        if (dst == kDstOutput) {
          const size_t orow = static_cast<size_t>(t0 + row0 / p.group + tok) * p.H + g * p.group + hh;
          out = p.o + orow * D;
          if (live) p.lse[orow] = lse2 * LN2;
        } else if (dst == kDstSlab0 || dst == kDstSlab1) {
          const size_t slab = blockIdx.x * 2 + (dst - kDstSlab0);
          stride = p.slab_rows;
          part = p.slab_o + slab * (D / 4) * stride + row;
          if (live) p.slab_lse[slab * stride + row] = lse2;
        } else {
          stride = static_cast<size_t>(p.N) * p.group;
          const size_t at = static_cast<size_t>(t0) * p.group + row;
          part = (dst == kDstOwn ? p.own_o : p.prefix_o) + static_cast<size_t>(g) * (D / 4) * stride + at;
          if (live) (dst == kDstOwn ? p.own_lse : p.prefix_lse)[g * stride + at] = lse2;
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          tmem_ld32_wait(t_o + c * 32, ov);
          if (pair) {
            uint32_t o1[32];
            tmem_ld32_wait(t_o + D + c * 32, o1);
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = f2u(u2f(ov[e]) * a0 + u2f(o1[e]) * a1);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = f2u(u2f(ov[e]) * a0);
          }
          if (!live) continue;
          if (out) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint4*>(out + c * 32 + e * 8) =
                  make_uint4(pack_bf16x2(u2f(ov[8 * e]), u2f(ov[8 * e + 1])), pack_bf16x2(u2f(ov[8 * e + 2]), u2f(ov[8 * e + 3])),
                             pack_bf16x2(u2f(ov[8 * e + 4]), u2f(ov[8 * e + 5])), pack_bf16x2(u2f(ov[8 * e + 6]), u2f(ov[8 * e + 7])));
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              part[(c * 8 + e) * stride] =
                  make_float4(u2f(ov[4 * e]), u2f(ov[4 * e + 1]), u2f(ov[4 * e + 2]), u2f(ov[4 * e + 3]));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar_o_empty + 8 * i);
        if (pair) mbar_arrive(bar_o_empty + 8);
      }
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- join
// A block joins 32 rows of one K/V head: lane = row, every warp 8 columns.  The parts of a row follow
// from the places of its two items: an item inside one SM's share has one part, in the buffer of its
// source; one that is cut has a part in a slab of every SM that worked some of its tiles.
template <int D>
__global__ void __launch_bounds__(D * 4) fa_prefix_join_kernel(const PrefixParams p) {
  const int lane = threadIdx.x & 31, col = threadIdx.x >> 5;  // columns 8 col .. 8 col + 7
  const int blocks_per_head = (p.N * p.group + 31) / 32;
  const int g = blockIdx.x / blocks_per_head;
  const long long r = static_cast<long long>(blockIdx.x - g * blocks_per_head) * 32 + lane;  // row of head g
  pdl_wait();
  const int tokens = p.hdr[kHdrTokens];
  const int n = static_cast<int>(r / p.group);
  if (n >= tokens) return;
  const unsigned int share = p.hdr[kHdrShare];
  const int4 t = p.tok[n];
  const size_t rows = static_cast<size_t>(p.N) * p.group;
  float m = -INFINITY, sum = 0.f, acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  auto add = [&](float lse2, const float4* part, size_t stride) {
    const float4 a = part[2 * col * stride], b = part[(2 * col + 1) * stride];
    if (lse2 == -INFINITY) return;
    const float m2 = fmaxf(m, lse2), f = exp2f(m - m2), w = exp2f(lse2 - m2);
    m = m2;
    sum = sum * f + w;
    acc[0] = acc[0] * f + w * a.x;
    acc[1] = acc[1] * f + w * a.y;
    acc[2] = acc[2] * f + w * a.z;
    acc[3] = acc[3] * f + w * a.w;
    acc[4] = acc[4] * f + w * b.x;
    acc[5] = acc[5] * f + w * b.y;
    acc[6] = acc[6] * f + w * b.z;
    acc[7] = acc[7] * f + w * b.w;
  };
  // parts of the item at c0 with `tiles` tiles, `seen` of them visible to this row, row `at` of the item
  auto join = [&](unsigned int c0, int tiles, int seen, int at, const float4* whole, const float* whole_lse) {
    const int c_first = (c0 + kItemCost) / share, c_last = (c0 + kItemCost + kTileCost * (tiles - 1)) / share;
    if (c_first == c_last) {
      add(whole_lse[g * rows + r], whole + static_cast<size_t>(g) * (D / 4) * rows + r, rows);
      return;
    }
    for (int c = c_first; c <= c_last; ++c) {
      const int j0 = tile_from(c * share, c0, tiles), j1 = tile_from((c + 1) * share, c0, tiles);
      if (j0 >= seen) break;
      if (j0 >= j1) continue;
      const size_t slab = c * 2 + (j0 == 0);
      add(p.slab_lse[slab * p.slab_rows + at], p.slab_o + slab * (D / 4) * p.slab_rows + at, p.slab_rows);
    }
  };
  const int hh = static_cast<int>(r - static_cast<long long>(n) * p.group);
  if (p.tiles_p > 0) {
    const int blk = n / (2 * p.tp), blocks = p.hdr[kHdrBlocks];
    join((static_cast<unsigned int>(g) * blocks + blk) * item_cost(p.tiles_p), p.tiles_p, p.tiles_p,
         (n - blk * 2 * p.tp) * p.group + hh, p.prefix_o, p.prefix_lse);
  }
  if (t.z > 0) {
    const unsigned int c0 = static_cast<unsigned int>(t.x) + g * item_cost(t.y);
    if (p.tiles_p == 0 && (c0 + kItemCost) / share == (c0 + kItemCost + kTileCost * (t.y - 1)) / share)
      return;  // the attention kernel wrote this row
    join(c0, t.y, t.z, t.w * p.group + hh, p.own_o, p.own_lse);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const size_t orow = static_cast<size_t>(n) * p.H + g * p.group + hh;
  *reinterpret_cast<uint4*>(p.o + orow * D + col * 8) =
      make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                 pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
  if (col == 0) p.lse[orow] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * LN2;
}

template <int D>
static cudaError_t launch(const CUtensorMap& qp, const CUtensorMap& qs, const CUtensorMap& k, const CUtensorMap& v,
                          const PrefixParams& p, cudaStream_t stream) {
  using L = PLayout<D>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && !attr_set[dev]) {
    e = cudaFuncSetAttribute(fa_prefix_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int plan_blocks = (p.N + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
  cfg.gridDim = dim3(plan_blocks < 64 ? plan_blocks : 64);
  cfg.blockDim = dim3(kPlanThreads);
  if ((e = cudaLaunchKernelEx(&cfg, fa_prefix_plan_kernel, p)) != cudaSuccess) return e;
  cfg.gridDim = dim3(p.ctas);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = L::SMEM_BYTES;
  if ((e = cudaLaunchKernelEx(&cfg, fa_prefix_kernel<D>, qp, qs, k, v, p)) != cudaSuccess) return e;
  cfg.gridDim = dim3(p.Hkv * ((p.N * p.group + 31) / 32));
  cfg.blockDim = dim3(D * 4);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, fa_prefix_join_kernel<D>, p);
}

cudaError_t launch_fa_fwd_prefix(int d, const CUtensorMap& qp, const CUtensorMap& qs, const CUtensorMap& k,
                                 const CUtensorMap& v, const PrefixParams& p, cudaStream_t stream) {
  return d == 64 ? launch<64>(qp, qs, k, v, p, stream) : launch<128>(qp, qs, k, v, p, stream);
}

unsigned int prefix_tile_cost() { return kTileCost; }
unsigned int prefix_item_cost() { return kItemCost; }

cudaError_t read_and_clear_prefix_status(cudaStream_t stream, unsigned int* out) {
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return e;
  e = cudaMemcpyFromSymbol(out, g_prefix_status, sizeof(unsigned int));
  if (e != cudaSuccess || *out == 0) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_prefix_status, &zero, sizeof(unsigned int));
}

}  // namespace fa
