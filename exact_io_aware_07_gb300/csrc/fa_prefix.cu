// Attention of new tokens over a shared prefix and each request's own pages (contract in include/fa.h).
//
// Row (n, h) sees the prefix's keys and its request's own keys up to its place; with s_j the scaled
// scores, O = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m) and LSE = m + ln sum_j e^(s_j - m).  The keys of a
// row are cut into parts that run on different SMs, each giving (O_p, LSE_p); a row's parts join as
//   LSE = ln sum_p e^LSE_p,   O = sum_p e^(LSE_p - LSE) O_p,
// which is the softmax over all keys, so that the prefix can be worked once for the rows of the whole
// batch and the own keys request by request.  Scores, maxima, sums and parts are fp32.  The weights e^(s_j - m) are
// rounded to bf16 for the product with V, the operand type of the tensor core; the sum that divides O is that of the
// rounded weights, so that the roundings move O by at most 2^-8 of its values' spread, not of their size.  O is rounded once more.
//
// Two kernels on the stream: fa_prefix_kernel, one block per SM, lays out the work from the device lengths
// (every block for itself) and works its share of the keys; fa_prefix_join_kernel joins the parts of the rows
// that have several.
//
// The work is a list of items: (K/V head, rows, keys), rows being (token, query head) pairs, `group` of them
// per token.  A request is few (up to 8 rows, or 16 at d = 64: a decoding request, a few drafted tokens), big (from
// kBigRows rows on: a prompt chunk) or between.  The items are
//   the prefix for blocks of up to 256 rows of any requests (a key tile is loaded once for all of them),
//   the own keys of a few or between request,
//   the prefix and then the own keys of up to 256 rows of a big request (it fills row tiles by itself, so its
//   rows need no second item and no join: 130 us against 148 for a batch of prompt chunks).
// There are two kinds of them, and every block works one of them:
//   many rows: up to 256 rows on tcgen05 products, keys in tiles of 128 (bound by the tensor core);
//   few rows:  the items of few requests (and the prefix, when all rows together are few) on warp-level
//              products, keys in steps of 16 or 32, by the block's eight warps one by one (bound by loading the keys).
// The items of a kind stand on a line, a key tile or step and an item taking so many places each, and the
// kind's workers (blocks, or warps) get equal stretches of it: worker w the tiles whose places begin in
// [w Q, (w + 1) Q).  So all workers have the same share whatever the lengths, and at most two items of a
// worker are cut, its first and its last.  The blocks are shared out between the kinds by their cost.
//
// What a call takes (GB300, in a graph, keys not in L2): one request behind 256 keys 12.8 us, which is two kernels' latency
// (the work's layout 3, a piece 5, the boundary between the kernels 1.5, the join 3); 64 requests with up to 1 024 own keys behind
// 4 096 shared ones 39 to 41 us (151 MB: 22 us at the measured copy rate); 128 behind 32 768 76 us (69 GFLOP: 36 us at the
// measured tensor rate, and 40 us of loading); 8 prompt chunks of up to 600 tokens 130 us (125 GFLOP: 65 us); one prompt of 8 192
// tokens 450 us (550 GFLOP: 284 us).
//
// 168 registers a thread (ten warps of 32); nvcc spills 32 bytes of them at d = 128, at d = 64 36 with few-row items of 8 rows and
// 180 of 16, the eight-lane join of d = 128 4.
#include <float.h>
#include <limits.h>
#include <math.h>

#include "fa_pages.h"
#include "ptx.cuh"

namespace fa {

static __device__ unsigned int g_prefix_status;  // kStatus* bits

// Places on the lines.  Many rows: an item, and a key tile of an item with up to 128 and more rows; few rows: an
// item, and one per step.  For sharing out the SMs, in microseconds and bytes per microsecond, fitted to the best
// shares of six batches (64 to 256 requests, prefixes of 1 024 to 32 768 keys): a place of either kind on one SM; what the
// many-row kind takes longer at its ends; the part of the loading time that its work is to fill; the rate of loading.
// The same constants do for both head sizes and few-row kinds: of 16 batches of 1 to 8 new tokens at d = 64 and 128 with 1 to 8
// query heads to a K/V head, a time 20 % up or down gains 5 % at most (45.3 -> 43.1 us) and costs up to a fourth (55 -> 69).
constexpr unsigned int kItemCost = 20, kTileCost128 = 6, kTileCost256 = 8;
constexpr unsigned int kFewItemCost = 4, kFewLeast = 4;  // (at least kFewLeast places for a warp)
constexpr float kManyTime = 0.19f, kFewTime = 0.12f, kManyStart = 2.6f, kManyShare = 0.4f, kLoadRate = 6.5e6f;
constexpr int kBigRows = 128;   // rows from which a request is big
// Row blocks of the batch whose need of the prefix is looked at one by one.  Of more, all count as needed: the prefix is
// then worked for the rows of big requests too, whose items have it already, and what comes of it is not read (40 000 new
// tokens with 8 query heads to a K/V head behind 4 096 keys take 6.0 ms, 32 000 take 3.2).
constexpr int kMaxFlags = 1024;
// words of p.hdr: both lines' shares, needed row blocks, tokens
enum { kHdrShare = 0, kHdrItems = 2, kHdrTokens };
constexpr int kTokFew = 1 << 15;  // in a token's fourth word: its item is on the few-row line

constexpr int THREADS = 320;
constexpr int BM = 128, BN = 128;
constexpr int BOX_BYTES = 128 * 128;  // 128 rows x 64 bf16, 128-byte swizzle
constexpr float LN2 = 0.693147180559945309f;

// A line's item: its first place, places before its first unit (tile or step), places per unit, units.
struct Item {
  unsigned int c0, lead, unit;
  int units;
  __device__ __forceinline__ unsigned int cost() const { return units ? lead + unit * units : 0u; }
  // first unit whose place is not before x
  __device__ __forceinline__ int from(unsigned int x) const {
    if (x <= c0 + lead) return 0;
    const unsigned int y = x - c0 - lead + unit - 1;  // (units are of three sizes: no division by a variable)
    const unsigned int j = unit == 1u ? y : unit == kTileCost256 ? y / kTileCost256 : y / kTileCost128;
    return j < static_cast<unsigned int>(units) ? static_cast<int>(j) : units;
  }
  __device__ __forceinline__ unsigned int worker(int unit_index, unsigned int share) const {
    return (c0 + lead + unit * unit_index) / share;
  }
};
__device__ __forceinline__ Item many_item(unsigned int c0, int tiles, int rows) {
  return Item{c0, kItemCost, rows <= 128 ? kTileCost128 : kTileCost256, tiles};
}
// Keys per step of the few-row kind: 8 KB of K and V.
template <int D>
constexpr int kStep = D == 64 ? 32 : 16;
__device__ __forceinline__ Item few_item(const PrefixParams& p, unsigned int c0, int keys) {
  return Item{c0, kFewItemCost, 1u, (keys + p.step - 1) >> (p.step == 32 ? 5 : 4)};
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
__device__ __forceinline__ bool is_few(const PrefixParams& p, const Request& r) { return r.added * p.group <= p.few_rows; }
__device__ __forceinline__ bool is_big(const PrefixParams& p, const Request& r) { return r.added * p.group >= kBigRows; }
__device__ __forceinline__ int tiles_of(int keys) { return (keys + kPage - 1) / kPage; }
// Own keys that the tokens before the request's token `end` (exclusive) can see at most.
__device__ __forceinline__ int visible(const PrefixParams& p, const Request& r, int end) {
  return p.causal ? max(0, min(r.len, r.len - r.added + end)) : r.len;
}
// The item (of K/V head 0, at c0) of a many-row request's block of 2 tp tokens; a big request's begins with the prefix.
__device__ __forceinline__ Item block_item(const PrefixParams& p, const Request& r, int blk, unsigned int c0) {
  const int end = min(r.added, (blk + 1) * 2 * p.tp);
  return many_item(c0, (is_big(p, r) ? p.tiles_p : 0) + tiles_of(visible(p, r, end)), (end - blk * 2 * p.tp) * p.group);
}
// A request's places on its line.
__device__ __forceinline__ unsigned int request_cost(const PrefixParams& p, const Request& r) {
  if (r.added == 0) return 0u;
  if (is_few(p, r)) return few_item(p, 0, visible(p, r, r.added)).cost() * p.Hkv;
  unsigned int sum = 0;
#pragma unroll 1
  for (int blk = 0; blk * 2 * p.tp < r.added; ++blk) sum += block_item(p, r, blk, 0).cost();
  return sum * p.Hkv;
}
// The prefix's items: per K/V head one few-row item when all rows of the batch together are few, else one of each
// needed block of 2 tp tokens (each counted as a full one unless the batch is smaller).
__device__ __forceinline__ bool few_prefix(const PrefixParams& p, int tokens) { return tokens * p.group <= p.few_rows; }
__device__ __forceinline__ Item prefix_item(const PrefixParams& p, int tokens, unsigned int index) {
  Item it = few_prefix(p, tokens) ? few_item(p, 0, p.prefix_len) : many_item(0, p.tiles_p, min(2 * p.tp, tokens) * p.group);
  it.c0 = index * it.cost();
  return it;
}

// ---------------------------------------------------------------- layout of the work
// Every block forms the running sums of the requests' places on both lines (a thread has a run of requests), finds
// the requests that its own workers begin with, and the blocks share out the tokens, whose item the join needs.
// (Up to 320 requests a thread has one.  Of more it has several and asks for their lengths one after another: 2 000
// requests of up to 60 keys take 84 us, 41 of them the loading of their keys at the measured copy rate; 320 take 25 and 7.)
struct Layout {                // in shared memory until the roles begin
  unsigned long long cum[THREADS];  // places before the thread's first request: many rows, few rows << 32
  int first[THREADS];               // the first new token of it
  unsigned long long warp[THREADS / 32];
  unsigned int need[kMaxFlags / 32];  // bit: a block of 2 tp tokens has tokens of requests that are not big
};
struct Begin {  // what a worker begins with
  int b;             // request
  unsigned int c0;   // its first place
};
struct Plan {
  unsigned int total[2], share[2], lead[2];  // lead: the prefix's places
  int many, tokens, blocks, items;           // blocks that work many rows; new tokens; row blocks; needed ones
  int few, worker;                           // whether this block works few rows; its number among the blocks of its kind
};

__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ bool flagged(const PrefixParams& p, int blocks) { return blocks <= kMaxFlags; }
// The needed block with `rank` needed ones before it.
__device__ __forceinline__ int needed_block(const PrefixParams& p, const volatile unsigned int* need, int blocks, int rank) {
  if (!flagged(p, blocks)) return rank;
#pragma unroll 1
  for (int w = 0; w < kMaxFlags / 32; ++w) {
    unsigned int bits = need[w];
    const int n = __popc(bits);
    if (rank < n) {
#pragma unroll 1
      for (; rank; --rank) bits &= bits - 1;
      return w * 32 + __ffs(bits) - 1;
    }
    rank -= n;
  }
  return 0;  // (never: rank is below the number of needed blocks)
}

__device__ __forceinline__ Plan make_plan(const PrefixParams& p, Layout& s, volatile unsigned int* need, Begin* begin) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (p.B + THREADS - 1) / THREADS, b_lo = min(p.B, tid * run), b_hi = min(p.B, b_lo + run);
  Plan l;
  const int end = p.cu_new[p.B];
  l.tokens = min(max(end, 0), p.N);
  const bool few = few_prefix(p, l.tokens);
  l.blocks = few ? 1 : (l.tokens + 2 * p.tp - 1) / (2 * p.tp);
  bool bad = end > p.N || end < 0;
  unsigned long long mine = 0;
  int first = p.N;
#pragma unroll 1
  for (int b = b_lo; b < b_hi; ++b) {
    const int c0 = p.cu_new[b], c1 = p.cu_new[b + 1], seq = p.seq_lens[b];
    bad |= c1 < c0 || seq < 0 || seq > p.max_pages * kPage || (b == 0 && c0 != 0);
    const Request r = make_request(p, c0, c1, seq);
    if (b == b_lo) first = r.first;
    mine += static_cast<unsigned long long>(request_cost(p, r)) << (is_few(p, r) ? 32 : 0);
    if (r.added > 0 && !is_big(p, r) && flagged(p, l.blocks))
#pragma unroll 1
      for (int k = r.first / (2 * p.tp); k <= (r.first + r.added - 1) / (2 * p.tp) && k < l.blocks; ++k)
        atomicOr(const_cast<unsigned int*>(need) + k / 32, 1u << (k % 32));
  }
  unsigned long long sum = mine;
#pragma unroll
  for (int w = 1; w < 32; w <<= 1) {
    const unsigned long long t = __shfl_up_sync(0xffffffffu, sum, w);
    if (lane >= w) sum += t;
  }
  if (lane == 31) s.warp[warp] = sum;
  __syncthreads();
  l.items = l.blocks;
  if (few)
    l.items = 1;
  else if (flagged(p, l.blocks)) {
    l.items = 0;
#pragma unroll 1
    for (int w = 0; w * 32 < l.blocks; ++w) l.items += __popc(need[w]);
  }
  if (l.tokens == 0) l.items = 0;
  const unsigned int prefix = l.items == 0 ? 0u : static_cast<unsigned int>(p.Hkv) * l.items * prefix_item(p, l.tokens, 0).cost();
  l.lead[0] = few ? 0u : prefix;
  l.lead[1] = few ? prefix : 0u;
  unsigned long long before = l.lead[0] | static_cast<unsigned long long>(l.lead[1]) << 32, all = before;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const unsigned long long t = s.warp[w];
    before += w < warp ? t : 0u;
    all += t;
  }
  l.total[0] = static_cast<unsigned int>(all);
  l.total[1] = static_cast<unsigned int>(all >> 32);
  s.cum[tid] = before + sum - mine;
  s.first[tid] = first;
  // Blocks for the many-row line.  m1 of them end it together with the few-row line, kManyStart + A / m1 = B / (G - m1);
  // where loading all keys takes longer than that, more do no harm to the few rows until their own work takes as long,
  // and the many-row blocks, which wait for their keys behind the others', are given time for kManyShare of the loading.
  const float a = kManyTime * l.total[0], b = kFewTime * l.total[1], g = p.ctas, d = kManyStart * g - a - b;
  float m = (d + sqrt_approx(d * d + 4.f * kManyStart * a * g)) * (0.5f / kManyStart);
  const float load = (l.total[1] * 8192.f + p.Hkv * p.tiles_p * 2.f * kPage * p.head_bytes) / kLoadRate;
  m = max(m, min(__fdividef(a, kManyShare * load), g - __fdividef(b, load)));
  l.many = l.total[0] == 0 ? 0 : l.total[1] == 0 ? p.ctas : max(1, min(p.ctas - 1, __float2int_rn(m)));
  l.share[0] = max(1u, (l.total[0] + max(l.many, 1) - 1) / max(l.many, 1));
  // Only the prefix on the many-row line: every item in the same whole number of stretches, so that the row blocks of a
  // head come to a key tile at the same time and all but the first read it from L2 (76 against 85 us for 128 requests
  // behind 32 768 keys, 71 against 77 for 256 behind 16 384).
  const int items = p.Hkv * l.items, each = items == 0 ? 0 : (2 * l.many + items) / (2 * items);
  if (l.total[0] > 0 && l.total[0] == l.lead[0] && each > 0 && each * items <= p.ctas - (l.total[1] > 0)) {
    l.many = each * items;
    l.share[0] = (l.total[0] / items + each - 1) / each;
  }
  const unsigned int warps = max(1, (p.ctas - l.many) * kFewWarps);
  l.share[1] = max(kFewLeast, (l.total[1] + warps - 1) / warps);
  __syncthreads();
  // the last thread with requests whose key is not above x
  auto owner = [&](auto key, unsigned int x) {
    int lo = 0, hi = (p.B + run - 1) / run;
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (key(mid) <= x)
        lo = mid;
      else
        hi = mid;
    }
    return lo;
  };
  auto request = [&](int b) { return make_request(p, p.cu_new[b], p.cu_new[b + 1], p.seq_lens[b]); };
  l.few = static_cast<int>(blockIdx.x) >= l.many;
  l.worker = l.few ? blockIdx.x - l.many : blockIdx.x;
  const int kind = l.few;
  if (tid < (kind ? kFewWarps : 1)) {  // the request that holds this block's worker's first own place
    const unsigned long long at =
        static_cast<unsigned long long>(kind ? l.worker * kFewWarps + tid : l.worker) * l.share[kind];
    if (at < l.total[kind]) {
      const unsigned int x = max(static_cast<unsigned int>(at), l.lead[kind]);
      auto place = [&](int t) { return static_cast<unsigned int>(s.cum[t] >> (32 * kind)); };
      const int t = owner(place, x);
      Begin w{t * run, place(t)};
#pragma unroll 1
      for (const int last = min(p.B, (t + 1) * run) - 1; w.b < last; ++w.b) {
        const Request r = request(w.b);
        const unsigned int c = is_few(p, r) == static_cast<bool>(kind) ? request_cost(p, r) : 0u;
        if (w.c0 + c > x) break;
        w.c0 += c;
      }
      begin[tid] = w;
    }
  }
#pragma unroll 1
  // (the first warp is at `begin` meanwhile)
  for (int n = blockIdx.x + gridDim.x * (tid - 32); n >= 0 && n < l.tokens; n += gridDim.x * (THREADS - 32)) {
    const int t = owner([&](int k) { return static_cast<unsigned int>(s.first[k]); }, n);
    unsigned int c0[2] = {static_cast<unsigned int>(s.cum[t]), static_cast<unsigned int>(s.cum[t] >> 32)};
    int b = t * run;
    Request r = request(b);
#pragma unroll 1
    for (const int last = min(p.B, (t + 1) * run) - 1; b < last; ++b) {
      const Request next = request(b + 1);
      if (next.first > n) break;
      c0[is_few(p, r)] += request_cost(p, r);
      r = next;
    }
    const int i = n - r.first;
    int4 tok = make_int4(0, 0, 0, 0);  // no own key
    int rank = -1;                     // no item of the prefix
    if (i >= 0 && i < r.added) {
      if (is_few(p, r)) {
        const Item it = few_item(p, c0[1], visible(p, r, r.added));
        tok = make_int4(static_cast<int>(it.c0), it.units, it.units, i | kTokFew);
      } else {
        const int blk = i / (2 * p.tp);
        unsigned int c = c0[0];
#pragma unroll 1
        for (int k = 0; k < blk; ++k) c += p.Hkv * block_item(p, r, k, 0).cost();
        const Item it = block_item(p, r, blk, c);
        tok = make_int4(static_cast<int>(c), it.units,
                        (is_big(p, r) ? p.tiles_p : 0) + tiles_of(visible(p, r, min(r.added, (i / p.tp + 1) * p.tp))),
                        (i - blk * 2 * p.tp) | static_cast<int>(it.unit) << 16);
      }
      if (p.tiles_p > 0 && !is_big(p, r)) {
        rank = few ? 0 : n / (2 * p.tp);
        if (!few && flagged(p, l.blocks)) {
          const int blk = rank;
          rank = __popc(need[blk / 32] & ((1u << (blk % 32)) - 1));
#pragma unroll 1
          for (int w = 0; w < blk / 32; ++w) rank += __popc(need[w]);
        }
      }
    }
    p.tok[n] = tok;
    p.rank[n] = rank;
  }
  if (blockIdx.x == 0) {
    if (tid == 0) {
      p.hdr[kHdrShare] = static_cast<int>(l.share[0]);
      p.hdr[kHdrShare + 1] = static_cast<int>(l.share[1]);
      p.hdr[kHdrItems] = l.items;
      p.hdr[kHdrTokens] = l.tokens;
    }
    if (bad) atomicOr(&g_prefix_status, kStatusBadLength);
  }
  fence_proxy_async_smem();  // the tiles will be loaded over what the layout wrote
  __syncthreads();
  return l;
}

// ---------------------------------------------------------------- parts
// Where a row's part goes: `out` (the row itself, in bf16) or `part`, and the LSE at `lse` (natural for the row
// itself, base-2 for a part).
enum { kDstOutput, kDstSlab0, kDstSlab1, kDstOwn, kDstPrefix };
// First slab row of worker `w` of a kind for its first (0) or last (1) cut item.
__device__ __forceinline__ size_t many_slab(const PrefixParams& p, int w, int which) {
  return (static_cast<size_t>(w) * 2 + which) * p.slab_rows;
}
__device__ __forceinline__ size_t few_slab(const PrefixParams& p, int w, int which) {
  return static_cast<size_t>(p.ctas) * 2 * p.slab_rows + (static_cast<size_t>(w) * 2 + which) * p.few_rows;
}
struct RowOut {
  __nv_bfloat16* out;
  float* part;
  float* lse;
};
// Row `row` of an item at token t0 and K/V head g; `slab`: the slab's first row.
template <int D>
__device__ __forceinline__ RowOut row_out(const PrefixParams& p, int dst, size_t slab, int g, int t0, int row) {
  if (dst == kDstSlab0 || dst == kDstSlab1) return RowOut{nullptr, p.slab_o + (slab + row) * D, p.slab_lse + slab + row};
  const int t = row / p.group;
  const size_t orow = static_cast<size_t>(t0 + t) * p.H + g * p.group + (row - t * p.group);
  if (dst == kDstOutput) return RowOut{p.o + orow * D, nullptr, p.lse + orow};
  if (dst == kDstOwn) return RowOut{nullptr, p.own_o + orow * D, p.own_lse + orow};
  return RowOut{nullptr, p.prefix_o + orow * D, p.prefix_lse + orow};
}

__device__ __forceinline__ float u2f(uint32_t x) { return __uint_as_float(x); }
__device__ __forceinline__ uint32_t f2u(float x) { return __float_as_uint(x); }
// 16 lanes x 64 columns of Tensor Memory: of every eight columns lane l gets columns 2 (l % 4) and the next, of rows l / 4
// (two registers) and l / 4 + 8 (two more).
__device__ __forceinline__ void tmem_ld_16x256b_x8_wait(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr) : "memory");
}
// The value of lane 0, known to be the same for the whole warp (tensor-core and TMA operands are warp-uniform).
__device__ __forceinline__ int uni(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// ---------------------------------------------------------------- values that are not finite
// The weight of an own key that causality hides from a row is 0, but 0 times an infinity or NaN is not, and a product's tile
// (or step) on the diagonal has keys that only some of its rows see: a new token whose value is not finite puts a NaN into
// the rows of the earlier new tokens beside it.  The products know nothing of it, but a block notes whether any of its
// results is not finite, and mends them at its end if so:
//   many rows: the block works its pieces once more with such values of keys that not all rows see set to 0 (`finite`), and
//   adds those to the rows that see them; a row's sum has them with a weight above 0, so that it is that infinity or NaN,
//   whatever the weight and the divisor;
//   few rows: rows that show a NaN and hide such a value are worked again key by key as they see them.
// The note costs 0 to 3 % (128 requests behind 32 768 keys 75.2 and 75.7 us, 256 requests of 60 keys 31.0 and 31.8, prompts of 600
// tokens 74.5 and 75.2); a look at the diagonal's values before the products cost prompts 3 to 5 %, on whichever warp, and 400
// requests of 60 keys 5 %.  A prompt of 8 192 tokens with a NaN in its last value takes 1.1 ms in place of 0.45, with one in every
// value 3.9; 48 requests of up to 8 drafted tokens with an infinity in each 0.8 ms in place of 0.06.
__device__ __forceinline__ uint32_t finite(uint32_t x) {  // of two bf16, those that are
  const uint32_t t = x & 0x7F807F80u;
  return ((t & 0x7F80u) == 0x7F80u ? 0u : x & 0xFFFFu) | ((t >> 16) == 0x7F80u ? 0u : x & 0xFFFF0000u);
}

// ---------------------------------------------------------------- many rows
// One lane loads a box of a page pool ((64, 128 rows, d / 64, planes) view: the 64-column halves of the box's rows one
// behind the other) and adds its bytes to what `bar` expects.
__device__ __forceinline__ void load_rows_elect(uint32_t dst, const void* tmap, int row, int plane, uint32_t bar, uint32_t bytes,
                                                uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b64 st;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 st, [%4], %5;\n\t"
      "@e cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {0, %2, 0, %3}], [%4], %6;\n\t}"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(row), "r"(plane), "r"(bar), "r"(bytes), "l"(policy) : "memory");
}
// The same rows of two pools, to dst and dst + half, with an L2 cache policy.
__device__ __forceinline__ void load_rows2_elect(uint32_t dst, uint32_t half, const void* tmap0, const void* tmap1, int row,
                                                 int plane, uint32_t bar, uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b64 st;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 st, [%6], %7;\n\t"
      "@e cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%2, {0, %4, 0, %5}], [%6], %8;\n\t"
      "@e cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%1], [%3, {0, %4, 0, %5}], [%6], %8;\n\t}"
      :: "r"(dst), "r"(dst + half), "l"(reinterpret_cast<uint64_t>(tmap0)), "l"(reinterpret_cast<uint64_t>(tmap1)),
         "r"(row), "r"(plane), "r"(bar), "r"(2 * half), "l"(policy) : "memory");
}
// Four tcgen05.mma, 64 deep: D (+)= A B with both from shared memory, 128-byte rows (a step of 16 is 32 bytes on), or with A
// from Tensor Memory and B's rows 2 048 bytes a step on.  One election for all four keeps a
// step's code short.
__device__ __forceinline__ void mma_ss4_elect(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q, e;\n\t.reg .b64 da, db;\n\t.reg .b32 a, b;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "setp.eq.b32 q, 0, 0;\n\t"
      "mov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, p;\n\t"
      "add.u32 a, %1, 2;\n\tadd.u32 b, %3, 2;\n\tmov.b64 da, {a, %2};\n\tmov.b64 db, {b, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, q;\n\t"
      "add.u32 a, %1, 4;\n\tadd.u32 b, %3, 4;\n\tmov.b64 da, {a, %2};\n\tmov.b64 db, {b, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, q;\n\t"
      "add.u32 a, %1, 6;\n\tadd.u32 b, %3, 6;\n\tmov.b64 da, {a, %2};\n\tmov.b64 db, {b, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, q;\n\t}"
      :: "r"(d_tmem), "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void mma_ts4_elect(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q, e;\n\t.reg .b64 db;\n\t.reg .b32 a, b;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.eq.b32 q, 0, 0;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t"
      "add.u32 a, %1, 8;\n\tadd.u32 b, %2, 128;\n\tmov.b64 db, {b, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %4, q;\n\t"
      "add.u32 a, %1, 16;\n\tadd.u32 b, %2, 256;\n\tmov.b64 db, {b, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %4, q;\n\t"
      "add.u32 a, %1, 24;\n\tadd.u32 b, %2, 384;\n\tmov.b64 db, {b, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], db, %4, q;\n\t}"
      :: "r"(d_tmem), "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate) : "memory");
}

// Many rows.  Roles: warps 0-3 and 4-7 the softmax of slot 0 and slot 1 (a thread has one of 128 rows),
// warp 8 the producer (lays out the block's pieces, issues the TMA loads), warp 9 the tcgen05.mma
// issuer.  A piece is the block's share of an item, in one of two forms:
//   two row tiles: each slot holds one, both visit every key tile (a tile is loaded once);
//   one row tile: the slots take its key tiles in turn, so that one's softmax overlaps the other's
//   products, and slot 0 joins both results at the end.
// Tensor Memory (512 columns): S_0 [0,128), S_1 [128,256), O_0, O_1 from 256; P_i (bf16 pairs) over S_i.
constexpr int PRODUCER_WARP = 8, MMA_WARP = 9;
constexpr int kPieceSlots = 3;

struct __align__(16) Piece {
  int mode;          // 0: no more pieces, 1: one row tile, 2: two row tiles
  int n, n0, n1;     // key tiles of the piece; visited by slot 0 / slot 1
  int j0;            // first key tile
  int ptiles;        // tiles below are the prefix's, the rest own keys from tile 0 on
  int keys;          // own keys
  int lim0, step;    // the item's token i sees min(keys, lim0 + i * step) of them
  int t0;            // the item's first token
  int rows0, rows1;  // rows of tile 0 / tile 1
  int g;             // K/V head
  int dst;           // where the part goes: kDst*
  int tile_rows;     // rows of a full row tile
  int turn;          // the slot that begins a piece of one row tile
};

template <int D>
struct PLayout {
  static constexpr int TILE_BYTES = BM * D * 2;
  static constexpr int BOXES = D / 64;
  static constexpr int STAGES = D == 128 ? 5 : 10;
  static constexpr int KV_OFF = 2 * TILE_BYTES;  // after the two query tiles
  static constexpr int XCH_OFF = 224 * 1024;  // behind both kinds' rings: slot 1's (m, l, lr) of one-tile pieces
  static_assert(KV_OFF + STAGES * TILE_BYTES <= XCH_OFF, "the ring reaches into what follows it");
  static constexpr int PIECE_OFF = XCH_OFF + 128 * 12;
  static constexpr int BAR_OFF = PIECE_OFF + kPieceSlots * int(sizeof(Piece));
  // q_full, q_empty, kv_full[S], kv_empty[S], s_full[2], p_full[2], o_full[2], o_empty[2], x_full[4], done,
  // piece_full[], piece_empty[]
  static constexpr int NUM_BARS = 2 + 2 * STAGES + 8 + 4 + 1 + 2 * kPieceSlots;
  static constexpr int MISC_OFF = BAR_OFF + NUM_BARS * 8;  // TMEM base, abort flag, whether a result is not finite
  static constexpr int END = MISC_OFF + 16;

  // Initialises barrier `t` (threads 0 .. NUM_BARS - 1, one each).
  static __device__ __forceinline__ void init(uint32_t sbase, int t) {
    const int u = t - (2 + 2 * STAGES);  // from s_full on
    int count = 1;
    if (u >= 0 && u < 8 && (u / 2 == 1 || u / 2 == 3)) count = 4;                      // p_full, o_empty: a slot's warps
    if (t >= NUM_BARS - kPieceSlots) count = 9;  // piece_empty: every softmax warp and the MMA warp reads each piece
    mbar_init(sbase + BAR_OFF + 8 * t, count);
  }
};
// Kept from laying out the work until the end: the plan, the needed row blocks and what the block's workers begin with.
constexpr int SMEM_BYTES = 232448;  // 227 KB opt-in dynamic shared memory per block on sm_103
constexpr int BEGIN_OFF = SMEM_BYTES - 8 * int(sizeof(Begin)), NEED_OFF = BEGIN_OFF - kMaxFlags / 8;
constexpr int PLAN_OFF = NEED_OFF - (int(sizeof(Plan)) + 15) / 16 * 16;
static_assert(PLayout<64>::END <= PLAN_OFF && PLayout<128>::END <= PLAN_OFF && sizeof(Layout) <= PLayout<64>::XCH_OFF, "shared memory");

template <int D, bool CLEAN>
__device__ __forceinline__ void many_rows(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                          const PrefixParams& p, const Plan& l, uint8_t* smem) {
  using L = PLayout<D>;
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
  volatile int* off_flag = reinterpret_cast<volatile int*>(smem + L::MISC_OFF + 8);
  const int warp = uni(threadIdx.x / 32), lane = threadIdx.x % 32;

  const uint32_t tmem = *tmem_slot;
  const Waiter W{abort_flag, p.timeout_ns, &g_prefix_status};

  if (warp == PRODUCER_WARP) {
    const unsigned int share = uni(l.share[0]), total = uni(l.total[0]), lead = uni(l.lead[0]);
    const unsigned int x0 = uni(l.worker) * share, x1 = min(total, x0 + share);
    const uint64_t once = l2_policy_evict_first();  // (see fa_prefix_kernel)
    int stage = 0, np = 0, turn = 0;
    uint32_t phase = 0, issued = 0, issued_parity = 0;
    bool ok = true;
    // page numbers of 32 tiles of one table row, one per lane (the row of a request may also be the prefix's)
    const int* held_table = nullptr;
    int held_base = -1, held_limit = 0, held_page = 0;
    auto kv_load = [&](const CUtensorMap* map, const int* own_table, int j, int ptiles, int g) -> bool {
      const bool of_prefix = j < ptiles;
      const int* table = of_prefix ? p.prefix_table : own_table;
      const int tile = of_prefix ? j : j - ptiles, limit = of_prefix ? p.tiles_p : p.max_pages;
      if (table != held_table || (tile & ~31) != held_base || limit != held_limit) {
        held_table = table;
        held_base = tile & ~31;
        held_limit = limit;
        held_page = held_base + lane < limit ? table[held_base + lane] : 0;
      }
      int pg = __shfl_sync(0xffffffffu, held_page, tile & 31);
      if (pg < 0 || pg >= p.num_pages) {  // out of the pool: reads zeros and is reported
        if (lane == 0) atomicOr(&g_prefix_status, kStatusBadPage);
        pg = p.num_pages;
      }
      if (!wait_all(W, bar_kv_empty + 8 * stage, phase ^ 1)) return false;
      load_rows_elect(kv_smem + stage * L::TILE_BYTES, map, 0, pg * p.Hkv + g, bar_kv_full + 8 * stage, L::TILE_BYTES, once);
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
        for (int w = 0; w < 16; ++w) dst[w] = src[w];
        mbar_arrive(bar_piece_full + 8 * s);
      }
      __syncwarp();
      ++np;
      return true;
    };
    // Emits this block's tiles [j0, j1) of an item: tokens [t0, t0 + count) in row tiles of tp tokens, the first of
    // which sees tiles0 of its tiles.
    auto emit = [&](const int* table, int g, int t0, int count, int tiles, int tiles0, int j0, int j1, int ptiles, int keys,
                    int lim0, int step, int whole) -> bool {
      Piece q;
      q.n = j1 - j0;
      q.mode = count > p.tp ? 2 : 1;
      // pieces of a single tile take the slots in turn: one's end overlaps the next one's scores and softmax (62 against
      // 73 us for 300 requests of 32 rows with 100 keys)
      q.turn = q.n == 1 && q.mode == 1 ? turn : 0;
      if (q.n == 1 && q.mode == 1) turn ^= 1;
      q.n0 = q.mode == 2 ? max(0, min(tiles0, j1) - j0) : (q.n + 1 - q.turn) / 2;
      q.n1 = q.mode == 2 ? q.n : (q.n + q.turn) / 2;
      q.j0 = j0;
      q.ptiles = ptiles;
      q.keys = keys;
      q.lim0 = lim0;
      q.step = step;
      q.t0 = t0;
      q.tile_rows = p.tp * p.group;
      q.rows0 = min(count, p.tp) * p.group;
      q.rows1 = max(0, count - p.tp) * p.group;
      q.g = g;
      q.dst = j0 > 0 ? kDstSlab0 : j1 < tiles ? kDstSlab1 : whole;
      const int k = np;
      if (!publish(q)) return false;
      if (!wait_all(W, bar_q_empty, (k & 1) ^ 1)) return false;
      const uint32_t box = static_cast<uint32_t>(q.tile_rows) * 128;
      mbar_arrive_expect_tx_elect(bar_q_full, box * L::BOXES * q.mode);
#pragma unroll 1
      for (int i = 0; i < q.mode; ++i)
#pragma unroll
        for (int b = 0; b < L::BOXES; ++b)
          tma_load_3d_elect(sbase + i * L::TILE_BYTES + b * BOX_BYTES, &tmQ, b * 64, g * p.group, t0 + i * p.tp,
                            bar_q_full);
      // two row tiles: K_0 V_0 K_1 V_1 ...; one: K_0 K_1 V_0 K_2 V_1 K_3 ... V_(n-1)
#pragma unroll 1
      for (int i = 0; i < 2 * q.n; ++i) {
        const bool k = q.mode == 2 ? !(i & 1) : i == 0 || ((i & 1) && i < 2 * q.n - 1);
        const int j = q.mode == 2 ? i >> 1 : k ? (i + 1) >> 1 : i < 2 * q.n - 1 ? (i >> 1) - 1 : q.n - 1;
        if (!kv_load(k ? &tmK : &tmV, table, j0 + j, ptiles, g)) return false;
      }
      return true;
    };

    if (x0 < x1 && x0 < lead) {  // items of the prefix: head by head, needed block of rows by block
      const volatile unsigned int* need = reinterpret_cast<const volatile unsigned int*>(smem + NEED_OFF);
      const int tokens = uni(l.tokens), blocks = uni(l.blocks), per_head = uni(l.items), items = p.Hkv * per_head;
#pragma unroll 1
      for (int at = x0 / prefix_item(p, tokens, 0).cost(); ok && at < items; ++at) {
        const Item it = prefix_item(p, tokens, at);
        if (it.c0 >= x1) break;
        const int j0 = it.from(x0), j1 = it.from(x1);
        if (j0 >= j1) continue;
        const int g = at / per_head, t0 = uni(needed_block(p, need, blocks, at - g * per_head)) * 2 * p.tp;
        ok = emit(nullptr, g, t0, min(2 * p.tp, tokens - t0), p.tiles_p, p.tiles_p, j0, j1, p.tiles_p, 0, 0, 0, kDstPrefix);
      }
    }
    if (ok && x0 < x1 && x1 > lead) {  // items of requests, blocks of tokens, heads
      const volatile Begin* begin = reinterpret_cast<const volatile Begin*>(smem + BEGIN_OFF);
      int b = uni(begin->b), base = b - 32;
      unsigned int c0 = uni(begin->c0);
      int r_cu0 = 0, r_cu1 = 0, r_seq = 0;
#pragma unroll 1
      for (; ok && b < p.B && c0 < x1; ++b) {
        if (b >= base + 32) {  // 32 requests at a time, one per lane
          base = b;
          const int at = min(b + lane, p.B - 1);
          r_cu0 = p.cu_new[at];
          r_cu1 = p.cu_new[at + 1];
          r_seq = p.seq_lens[at];
        }
        const Request r = make_request(p, __shfl_sync(0xffffffffu, r_cu0, b - base), __shfl_sync(0xffffffffu, r_cu1, b - base),
                                       __shfl_sync(0xffffffffu, r_seq, b - base));
        if (is_few(p, r)) continue;
        const int* table = p.block_table + static_cast<size_t>(b) * p.max_pages;
        const int ptiles = is_big(p, r) ? p.tiles_p : 0;
#pragma unroll 1
        for (int blk = 0; ok && blk * 2 * p.tp < r.added && c0 < x1; ++blk) {
          Item it = block_item(p, r, blk, c0);
          const unsigned int cost = it.cost();
          c0 += p.Hkv * cost;
          if (it.units == 0 || c0 <= x0) continue;
          const int t = blk * 2 * p.tp, count = min(2 * p.tp, r.added - t);
          const int tiles0 = ptiles + tiles_of(visible(p, r, min(r.added, t + p.tp)));
          const int g0 = x0 > it.c0 ? (x0 - it.c0) / cost : 0;
          it.c0 += g0 * cost;
#pragma unroll 1
          for (int g = g0; ok && g < p.Hkv && it.c0 < x1; ++g, it.c0 += cost) {
            const int j0 = it.from(x0), j1 = it.from(x1);
            if (j0 < j1)
              ok = emit(table, g, r.first + t, count, it.units, tiles0, j0, j1, ptiles, r.len,
                        p.causal ? r.len - r.added + t + 1 : r.len, p.causal,
                        p.tiles_p == ptiles ? kDstOutput : kDstOwn);
          }
        }
      }
    }
    if (ok) {
      Piece q;
      q.mode = 0;
      q.n = q.n0 = q.n1 = q.j0 = q.ptiles = q.keys = q.lim0 = q.step = q.t0 = q.rows0 = q.rows1 = q.g = q.dst = q.tile_rows = q.turn = 0;
      ok = publish(q);
    }
    if (!ok) {  // let every copy already issued land before the block exits
      if (np > 0) drain_all(W, bar_q_full, (np - 1) & 1);
#pragma unroll 1
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
      for (int c = 0; c < D / 64; ++c)
        mma_ss4_elect(tmem + slot * 128, a0 + c * (BOX_BYTES >> 4), dqk_hi, b0 + c * (BOX_BYTES >> 4), dqk_hi, IDESC_S, c);
      mma_commit_elect(bar_s_full + 8 * slot);
    };
    // The last tile of a source holds fewer than 128 keys, and what its page holds behind them may be
    // anything.  Their weights are 0, but 0 times an infinity or NaN is not: the product runs over the keys
    // in steps of 16 as far as there are keys, and the value rows behind the last key in its last step are
    // set to 0.  Returns the steps.  (CLEAN: values of a tile on the diagonal that are not finite are set to 0 too.)
    auto value_steps = [&](const Piece& q, int tile, int vs) -> int {
      const int valid = tile < q.ptiles ? p.prefix_len - tile * BN : q.keys - (tile - q.ptiles) * BN;
      if (CLEAN && tile >= q.ptiles && q.lim0 < q.keys) {
        const int words = min(valid, BN) * 8;  // per box, from the first key that not all rows see
#pragma unroll 1
        for (int w = max(0, q.lim0 - (tile - q.ptiles) * BN) * 8 + lane; w < words; w += 32)
#pragma unroll 1
          for (int box = 0; box < L::BOXES; ++box) {
            const uint32_t at = kv_smem + vs * L::TILE_BYTES + box * BOX_BYTES + w * 16;
            const float4 x = ld_shared_v4f(at);
            st_shared_v4(at, finite(f2u(x.x)), finite(f2u(x.y)), finite(f2u(x.z)), finite(f2u(x.w)));
          }
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (valid >= BN) return BN / 16;
      const int steps = (valid + 15) / 16, words = (steps * 16 - valid) * 8;  // 16-byte words per box
#pragma unroll 1
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
      if (steps == BN / 16) {
        mma_ts4_elect(tmem + 256 + slot * D, tmem + slot * 128, b0, dv_hi, IDESC_PV, acc ? 1u : 0u);
        mma_ts4_elect(tmem + 256 + slot * D, tmem + slot * 128 + 32, b0 + (8192 >> 4), dv_hi, IDESC_PV, 1u);
      } else {
#pragma unroll 1
        for (int kk = 0; kk < steps; ++kk)
          mma_ts_elect(tmem + 256 + slot * D, tmem + slot * 128 + kk * 8, b0 + ((kk * 2048) >> 4), dv_hi, IDESC_PV,
                       (acc || kk > 0) ? 1u : 0u);
      }
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
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      const int s = k % kPieceSlots;
      if (!(ok = wait_all(W, bar_piece_full + 8 * s, (k / kPieceSlots) & 1))) break;
      Piece q;
      q.mode = uni(pieces[s].mode);
      q.n = uni(pieces[s].n);
      q.n0 = uni(pieces[s].n0);
      q.n1 = uni(pieces[s].n1);
      q.j0 = uni(pieces[s].j0);
      q.keys = uni(pieces[s].keys);
      q.ptiles = uni(pieces[s].ptiles);
      if (CLEAN) q.lim0 = uni(pieces[s].lim0);
      q.turn = uni(pieces[s].turn);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_piece_empty + 8 * s);
      if (q.mode == 0) break;
      if (!(ok = wait_all(W, bar_q_full, k & 1))) break;
      tc_fence_after();
      int ks = 0, vs = 0;
      if (q.mode == 1) {
#pragma unroll 1
        for (int x = 0; ok && x < min(q.n, 2); ++x) {
          if (!(ok = take(ks))) break;
          issue_s(x ^ q.turn, 0, ks);
          if (x + 1 == q.n) mma_commit_elect(bar_q_empty);
          mma_commit_elect(bar_kv_empty + 8 * ks);
        }
#pragma unroll 1
        for (int x = 0; ok && x < q.n; ++x) {
          const int slot = (x & 1) ^ q.turn;
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
#pragma unroll 1
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
    const int tok = rt / p.group;  // the row's token within its tile
    const int l_worker = l.worker;  // (l is the sum below)
    const float sl2 = p.scale_log2;
    uint32_t sf_phase = 0, of_phase = 0, x_phase = 0;
    bool ok = true;
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      const int s = k % kPieceSlots;
      if (!(ok = wait_all(W, bar_piece_full + 8 * s, (k / kPieceSlots) & 1))) break;
      const int mode = pieces[s].mode, n = pieces[s].n, n_mine = i ? pieces[s].n1 : pieces[s].n0, j0 = pieces[s].j0;
      const int rows = (mode == 2 && i) ? pieces[s].rows1 : pieces[s].rows0, g = pieces[s].g, dst = pieces[s].dst;
      const int ptiles = pieces[s].ptiles;
      const int tile_rows = pieces[s].tile_rows, t0 = pieces[s].t0;
      const int row0 = mode == 2 ? i * tile_rows : 0;  // the tile's first row within the item
      int lim = min(pieces[s].keys, pieces[s].lim0 + pieces[s].step * (row0 / p.group + tok));  // keys the row sees
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_piece_empty + 8 * s);
      if (mode == 0) break;
      if (n_mine == 0) continue;
      const bool live = rt < rows, live_warp = wq * 32 < rows;
      const int lim_p = live ? p.prefix_len : 0;  // of the prefix's keys
      if (!live) lim = 0;
      float m_run = -INFINITY;  // reference max, base-2 units of the scaled score
      float l = 0.f, lr = 0.f;  // sums of the fp32 weights (LSE) and of the bf16 weights the product uses (divides O)
#pragma unroll 1
      for (int x = 0; x < n_mine; ++x) {
        if (!(ok = wait_all(W, my_s_full, sf_phase))) break;
        sf_phase ^= 1;
        tc_fence_after();
        if (live_warp) {
          uint32_t sr[BN];
          tmem_ld128_wait(t_s, sr);
          const int tile = j0 + (mode == 1 && n > 1 ? 2 * x + i : x);
          const int left = tile < ptiles ? lim_p - tile * BN : lim - (tile - ptiles) * BN;  // keys of the tile the row sees
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
        const RowOut to = row_out<D>(p, dst, many_slab(p, l_worker, dst == kDstSlab1), g, t0, row0 + rt);
        if (live) *to.lse = to.out ? lse2 * LN2 : lse2;
        // O leaves 16 rows at a time in the layout in which four lanes have eight columns of a row (a whole 32-byte
        // sector of a part): lane l has columns 2 (l % 4), + 1 of every eight, rows l / 4 and l / 4 + 8
        const unsigned long long mine = live ? reinterpret_cast<unsigned long long>(to.out ? static_cast<void*>(to.out) : to.part) : 0;
        bool off = false;  // whether a result is not finite
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const int r_lo = h * 16 + lane / 4, r_hi = r_lo + 8;
          const unsigned long long at_lo = __shfl_sync(0xffffffffu, mine, r_lo), at_hi = __shfl_sync(0xffffffffu, mine, r_hi);
          const float a0_lo = __shfl_sync(0xffffffffu, a0, r_lo), a0_hi = __shfl_sync(0xffffffffu, a0, r_hi);
          const float a1_lo = __shfl_sync(0xffffffffu, a1, r_lo), a1_hi = __shfl_sync(0xffffffffu, a1, r_hi);
#pragma unroll 1
          for (int c = 0; c < D / 64; ++c) {
            uint32_t ov[32];
            tmem_ld_16x256b_x8_wait(t_o + (uint32_t(h * 16) << 16) + c * 64, ov);
            if (pair) {
              uint32_t o1[32];
              tmem_ld_16x256b_x8_wait(t_o + D + (uint32_t(h * 16) << 16) + c * 64, o1);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                ov[e] = f2u(u2f(ov[e]) * (e & 2 ? a0_hi : a0_lo) + u2f(o1[e]) * (e & 2 ? a1_hi : a1_lo));
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e) ov[e] = f2u(u2f(ov[e]) * (e & 2 ? a0_hi : a0_lo));
            }
            float x_lo = 0.f, x_hi = 0.f;  // 0, or NaN with one that is not
#pragma unroll
            for (int e = 0; e < 32; ++e) (e & 2 ? x_hi : x_lo) = fmaf(u2f(ov[e]), 0.f, e & 2 ? x_hi : x_lo);
            off |= (at_lo && x_lo != 0.f) || (at_hi && x_hi != 0.f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int col = c * 64 + e * 8 + 2 * (lane & 3);
              if (dst == kDstOutput) {
                if (at_lo) reinterpret_cast<uint32_t*>(at_lo)[col / 2] = pack_bf16x2(u2f(ov[4 * e]), u2f(ov[4 * e + 1]));
                if (at_hi) reinterpret_cast<uint32_t*>(at_hi)[col / 2] = pack_bf16x2(u2f(ov[4 * e + 2]), u2f(ov[4 * e + 3]));
              } else {
                if (at_lo) reinterpret_cast<float2*>(at_lo)[col / 2] = make_float2(u2f(ov[4 * e]), u2f(ov[4 * e + 1]));
                if (at_hi) reinterpret_cast<float2*>(at_hi)[col / 2] = make_float2(u2f(ov[4 * e + 2]), u2f(ov[4 * e + 3]));
              }
            }
          }
        }
        if (p.causal && off) *off_flag = 1;  // (see `finite`)
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

}

// The block's pieces once more: a function of its own, so that the code of the first time is as if there were no second.
template <int D>
__device__ __noinline__ void many_rows_clean(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                             const PrefixParams& p, uint8_t* smem) {
  many_rows<D, true>(tmQ, tmK, tmV, p, *reinterpret_cast<const Plan*>(smem + PLAN_OFF), smem);
}

// ---------------------------------------------------------------- few rows
// A warp works items of up to 8 NT rows, keys in steps of 16 or 32 (8 KB of K and V).  A 128-row tcgen05 tile would spend
// its softmax on empty rows; here the products are warp-level and transposed, keys (or columns of V) as the 16 rows of
// mma.sync m16n8k16 and query rows as its 8 columns:
//   S^T (16 keys x 8 rows) = K Q^T,   O^T (16 columns x 8 rows) += V^T P^T,
// so that eight rows cost one product per 16 x 16 of K and V and half the accumulators that rows as M would.  P^T
// becomes the second product's operand by an 8 x 8 transpose in registers (movmatrix); the softmax state stays in
// registers too, and a warp meets no other: each fills its own ring of K/V steps by TMA, and one's item start (request,
// table and query loads) and end hide behind the others' keys in flight.
//
// Bound by loading the keys with 8 rows: 32 requests with 1 000 to 32 768 keys (2.2 GB) take 340 us, 6.5 TB/s, 96 % of the
// measured copy rate.  With 16 rows the warp-level products and exponentials take twice as long and are the bound at d = 128, and the
// tcgen05 kind is better from some 100 keys on (64 requests of 16 rows: 54 against 81 us with 1 024 keys, 31 against 35 with
// 200, 24 against 18 with 20).  At d = 64 a step has half the work per key: 12 rows take 60 us against 76 with 1 000 keys and 16
// against 31 with 40, but 24 rows, as two warps, 91 against 77.  So the few are up to 8 rows at d = 128, up to 16 at d = 64.
template <int D>
struct FLayout {
  static constexpr int STEP = kStep<D>;
  static constexpr int STEP_BYTES = 2 * STEP * D * 2;  // K, then V; 64 columns per box of STEP rows x 128 bytes
  static constexpr int BOX = STEP * 128;
  static constexpr int STAGES = PLayout<D>::XCH_OFF / (kFewWarps * STEP_BYTES);
  static constexpr int BAR_OFF = PLayout<D>::END;  // full[kFewWarps][STAGES]
  static constexpr int NUM_BARS = kFewWarps * STAGES;
  static_assert(STAGES >= 3 && BAR_OFF % 8 == 0 && BAR_OFF + NUM_BARS * 8 <= PLAN_OFF && NUM_BARS <= THREADS, "barriers");
  static_assert(kFewWarps * STAGES * STEP_BYTES <= PLayout<D>::XCH_OFF, "the rings reach into what follows them");
};

// Warp-level products: D (16 x 8) += A (16 x 16) B (16 x 8), bf16 in, fp32 out.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four 8 x 8 matrices of 16-bit values; lane l gives the address of row l % 8 of matrix l / 8.
__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// Transpose of an 8 x 8 matrix of 16-bit values (lane l: row l / 4, columns 2 (l % 4) and the next).
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

struct FewPiece {
  const int* table;
  int entries;              // of the table
  int g, t0, rows, j0, j1;  // K/V head, first token, rows, steps
  int keys, lim0, step;     // keys of the source; token i sees min(keys, lim0 + i * step) of them
  int dst;
};

// The pieces of a stretch [x0, x1) of the few-row line, in order (all lanes of a warp together).
struct FewWalk {
  unsigned int x0, x1, lead, cost, c0;  // c0: first place of request b
  int tokens, at, items;                // items of the prefix on this line
  int b, base, g;
  bool have;
  Request r;
  Item it;
  int cu0, cu1, seq;  // of request base + lane

  __device__ __forceinline__ void start(const PrefixParams& p, const Plan& l, unsigned int from, unsigned int to, int first,
                                        unsigned int first_place) {
    x0 = from;
    x1 = to;
    lead = l.lead[1];
    tokens = l.tokens;
    items = lead > 0 ? p.Hkv : 0;
    at = x0 < lead ? static_cast<int>(x0 / (lead / p.Hkv)) : items;
    b = first;
    c0 = first_place;
    base = b - 32;
    have = false;
  }
  __device__ __forceinline__ bool next(const PrefixParams& p, int lane, FewPiece& q) {
#pragma unroll 1
    while (at < items) {
      const Item i = prefix_item(p, tokens, at);
      const int j0 = i.from(x0), j1 = i.from(x1);
      if (i.c0 >= x1) return false;
      const int head = at++;
      if (j0 >= j1) continue;
      q = FewPiece{p.prefix_table, p.tiles_p, head, 0, tokens * p.group, j0, j1, p.prefix_len, p.prefix_len, 0,
                   j0 > 0 ? kDstSlab0 : j1 < i.units ? kDstSlab1 : kDstPrefix};
      return true;
    }
    if (x1 <= lead) return false;
#pragma unroll 1
    for (;;) {
      if (have) {
        if (g < p.Hkv) {
          if (it.c0 >= x1) return false;
          const int j0 = it.from(x0), j1 = it.from(x1), head = g++;
          it.c0 += cost;
          if (j0 >= j1) continue;
          q = FewPiece{p.block_table + static_cast<size_t>(b) * p.max_pages, p.max_pages, head, r.first, r.added * p.group,
                       j0, j1, r.len, p.causal ? r.len - r.added + 1 : r.len, p.causal,
                       j0 > 0 ? kDstSlab0 : j1 < it.units ? kDstSlab1 : p.tiles_p > 0 ? kDstOwn : kDstOutput};
          return true;
        }
        c0 += p.Hkv * cost;
        ++b;
        have = false;
      }
#pragma unroll 1
      for (;; ++b) {
        if (b >= p.B || c0 >= x1) return false;
        if (b >= base + 32) {  // 32 requests at a time, one per lane
          base = b;
          const int l = min(b + lane, p.B - 1);
          cu0 = p.cu_new[l];
          cu1 = p.cu_new[l + 1];
          seq = p.seq_lens[l];
        }
        r = make_request(p, __shfl_sync(0xffffffffu, cu0, b - base), __shfl_sync(0xffffffffu, cu1, b - base),
                         __shfl_sync(0xffffffffu, seq, b - base));
        if (r.added == 0 || !is_few(p, r)) continue;
        it = few_item(p, c0, visible(p, r, r.added));
        cost = it.cost();
        if (c0 + p.Hkv * cost > x0 && cost > 0) break;
        c0 += p.Hkv * cost;
      }
      g = x0 > c0 ? static_cast<int>((x0 - c0) / cost) : 0;
      it.c0 = c0 + g * cost;
      have = true;
    }
  }
};

template <int D, int NT>
__device__ __forceinline__ void few_rows(const CUtensorMap& tmK, const CUtensorMap& tmV, const PrefixParams& p,
                                         const Plan& l, uint8_t* smem) {
  using L = FLayout<D>;
  const uint32_t sbase = smem_u32(smem);
  const int warp = uni(threadIdx.x / 32), lane = threadIdx.x % 32;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + PLayout<D>::MISC_OFF + 4);
  volatile int* off_flag = reinterpret_cast<volatile int*>(smem + PLayout<D>::MISC_OFF + 8);
  if (warp >= kFewWarps) return;
  const Waiter W{abort_flag, p.timeout_ns, &g_prefix_status};
  const uint32_t ring = sbase + warp * L::STAGES * L::STEP_BYTES;
  const uint32_t bar_full = sbase + L::BAR_OFF + 8 * warp * L::STAGES;
  const int worker = uni(l.worker) * kFewWarps + warp;
  const unsigned int total = uni(l.total[1]), share = uni(l.share[1]);
  const unsigned long long from = static_cast<unsigned long long>(worker) * share;
  if (from >= total) return;
  const unsigned int x0 = static_cast<unsigned int>(from);
  const unsigned int x1 = static_cast<unsigned int>(min(from + share, static_cast<unsigned long long>(total)));
  const volatile Begin* begin = reinterpret_cast<const volatile Begin*>(smem + BEGIN_OFF) + warp;
  const int first = uni(begin->b);
  const unsigned int first_place = uni(begin->c0);

  // The ring's filling side stands a piece ahead: the next piece's pages (32 tiles', one per
  // lane) and query rows are asked for when the piece before it begins.
  FewWalk walk, load;
  FewPiece q, lp, ahead;
  int lj = 0, issued = 0, lstage = 0, page = 0, base = 0, ahead_page = 0;
  walk.start(p, l, x0, x1, first, first_place);
  bool have = walk.next(p, lane, q), more = true, any = have;
  auto ask = [&] {  // for the piece ahead's pages and query rows
    const int first_tile = ahead.j0 / (kPage / L::STEP) & ~31;
    ahead_page = first_tile + lane < ahead.entries ? ahead.table[first_tile + lane] : 0;
#pragma unroll 1
    for (int r = lane; r < ahead.rows; r += 32) {
      const int tok = r / p.group;
      const __nv_bfloat16* src = p.q + (static_cast<size_t>(ahead.t0 + tok) * p.H + ahead.g * p.group + (r - tok * p.group)) * D;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
      if (D == 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + 64));
    }
  };
  load = walk;
  ahead = q;
  lp.j1 = 0;
  if (any) ask();
  const uint64_t once = l2_policy_evict_first();
  auto fill = [&] {  // loads the stretch's next step, if there is one
    if (lj >= lp.j1) {
      if (!any) {
        more = false;
        return;
      }
      lp = ahead;
      lj = lp.j0;
      page = ahead_page;
      base = lj / (kPage / L::STEP) & ~31;
      if ((any = load.next(p, lane, ahead))) ask();
    }
    const int tile = lj / (kPage / L::STEP);
    if ((tile & ~31) != base) {
      base = tile & ~31;
      page = base + lane < lp.entries ? lp.table[base + lane] : 0;
    }
    int pg = __shfl_sync(0xffffffffu, page, tile & 31);
    if (pg < 0 || pg >= p.num_pages) {  // out of the pool: reads zeros and is reported
      if (lane == 0) atomicOr(&g_prefix_status, kStatusBadPage);
      pg = p.num_pages;
    }
    load_rows2_elect(ring + lstage * L::STEP_BYTES, L::STEP_BYTES / 2, &tmK, &tmV, (lj % (kPage / L::STEP)) * L::STEP,
                     pg * p.Hkv + lp.g, bar_full + 8 * lstage, once);
    ++lj;
    ++issued;
    if (++lstage == L::STAGES) lstage = 0;
  };
#pragma unroll 1
  for (int t = 0; more && t < L::STAGES; ++t) fill();
  bool ok = true;

  const int c0 = 2 * (lane & 3);  // a thread's columns of a product are c0 and c0 + 1
  const float sl2 = p.scale_log2;
  // shared-memory words of a 16 x 16 block of K (rows as they are) and of V (transposed), within a step
  const int k_row = lane & 15, v_row = ((lane >> 4) << 3) + (lane & 7);
  uint32_t k_at[4], v_at[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    k_at[c] = ring + k_row * 128 + (((2 * c + (lane >> 4)) ^ (k_row & 7)) << 4);
    v_at[c] = ring + L::STEP_BYTES / 2 + v_row * 128 + (((2 * c + ((lane >> 3) & 1)) ^ (v_row & 7)) << 4);
  }
  const uint32_t ones[4] = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  int stage = 0;
  uint32_t full_par = 0;
#pragma unroll 1
  for (; ok && have; have = walk.next(p, lane, q)) {
    uint32_t qf[D / 16][NT][2];  // Q^T
    int lim[NT][2], lim_min = q.keys;  // keys the thread's rows see (rows past the last one: all, they are not used)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = 8 * t + lane / 4, tok = r / p.group;
      const __nv_bfloat16* src = p.q + (static_cast<size_t>(q.t0 + tok) * p.H + q.g * p.group + (r - tok * p.group)) * D + c0;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qf[kk][t][0] = r < q.rows ? *reinterpret_cast<const uint32_t*>(src + kk * 16) : 0u;
        qf[kk][t][1] = r < q.rows ? *reinterpret_cast<const uint32_t*>(src + kk * 16 + 8) : 0u;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * t + c0 + e;
        lim[t][e] = row < q.rows ? min(q.keys, q.lim0 + q.step * (row / p.group)) : q.keys;
        lim_min = min(lim_min, lim[t][e]);
      }
    }
    lim_min = __reduce_min_sync(0xffffffffu, lim_min);
    // per row: the reference (base-2 units of the scaled score); the sum of the fp32 weights (LSE; this thread's keys);
    // the sum of the bf16 weights that the product uses (divides O), kept by a product with ones
    float o[D / 16][NT][4], m[NT][2], lw[NT][2], lr[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[t][e] = -INFINITY;
        lw[t][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        lr[t][e] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) o[c][t][e] = 0.f;
      }
    }
#pragma unroll 1
    for (int j = q.j0; j < q.j1; ++j) {
      if (!(ok = wait_all(W, bar_full + 8 * stage, (full_par >> stage) & 1))) break;
      full_par ^= 1u << stage;
      const uint32_t at = stage * L::STEP_BYTES;
      const int k0 = j * L::STEP;
      constexpr int U = L::STEP / 16, CHAINS = U == 1 ? 2 : 1;  // sixteens of keys; chains of products for each
      float s[U][NT][4], s2[NT][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s2[t][e] = 0.f;
#pragma unroll
          for (int u = 0; u < U; ++u) s[u][t][e] = 0.f;
        }
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          uint32_t a[4];
          ldmatrix_x4(a, k_at[kk % 4] + at + (kk / 4) * L::BOX + u * 2048);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma_16816(CHAINS == 2 && (kk & 1) ? s2[t] : s[u][t], a, qf[kk][t][0], qf[kk][t][1]);
        }
      if (CHAINS == 2)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[0][t][e] += s2[t][e];
      if (k0 + L::STEP > lim_min) {  // some row does not see all of these keys
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int key = k0 + u * 16 + lane / 4;
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              if (key >= lim[t][e]) s[u][t][e] = -INFINITY;
              if (key + 8 >= lim[t][e]) s[u][t][2 + e] = -INFINITY;
            }
        }
      }
      float x[NT][2];
      bool grows = false;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x[t][e] = fmaxf(s[0][t][e], s[0][t][2 + e]);
#pragma unroll
          for (int u = 1; u < U; ++u) x[t][e] = fmaxf(x[t][e], fmaxf(s[u][t][e], s[u][t][2 + e]));
#pragma unroll
          for (int w = 4; w <= 16; w <<= 1) x[t][e] = fmaxf(x[t][e], __shfl_xor_sync(0xffffffffu, x[t][e], w));
          x[t][e] *= sl2;
          grows |= x[t][e] > m[t][e] + 8.f;
        }
      // the references are moved, and the sums and O rescaled, only when a maximum grows by more than 2^8
      if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float top = x[t][e] > m[t][e] + 8.f ? x[t][e] : m[t][e];
            const float f = top == -INFINITY ? 1.f : ex2_approx(m[t][e] - top);
            m[t][e] = top;
            lw[t][e] *= f;
            lr[t][e] *= f;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              o[c][t][e] *= f;
              o[c][t][2 + e] *= f;
            }
          }
      }
      uint32_t pt[U][NT][2];  // P^T
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float z0 = m[t][0] == -INFINITY ? 0.f : -m[t][0], z1 = m[t][1] == -INFINITY ? 0.f : -m[t][1];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float p0 = ex2_approx(fmaf(s[u][t][0], sl2, z0)), p1 = ex2_approx(fmaf(s[u][t][1], sl2, z1));
          const float p2 = ex2_approx(fmaf(s[u][t][2], sl2, z0)), p3 = ex2_approx(fmaf(s[u][t][3], sl2, z1));
          lw[t][0] += p0 + p2;
          lw[t][1] += p1 + p3;
          pt[u][t][0] = transpose_8x8(pack_bf16x2(p0, p1));
          pt[u][t][1] = transpose_8x8(pack_bf16x2(p2, p3));
          mma_16816(lr[t], ones, pt[u][t][0], pt[u][t][1]);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int left = q.keys - k0 - u * 16;
        // value rows behind the source's last key may hold anything: they count as 0 (their weights are 0 too)
        uint32_t v0 = 0xFFFFFFFFu, v1 = 0xFFFFFFFFu;
        if (left < 16) {
          v0 = (c0 < left ? 0xFFFFu : 0u) | (c0 + 1 < left ? 0xFFFF0000u : 0u);
          v1 = (c0 + 8 < left ? 0xFFFFu : 0u) | (c0 + 9 < left ? 0xFFFF0000u : 0u);
        }
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t a[4];
          ldmatrix_x4_trans(a, v_at[c % 4] + at + (c / 4) * L::BOX + u * 2048);
          if (left < 16) {
            a[0] &= v0;
            a[1] &= v0;
            a[2] &= v1;
            a[3] &= v1;
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) mma_16816(o[c][t], a, pt[u][t][0], pt[u][t][1]);
        }
      }
      __syncwarp();
      if (++stage == L::STAGES) stage = 0;
      if (more) fill();
    }
    if (!ok) break;
    const size_t slab = few_slab(p, worker, q.dst == kDstSlab1);
    bool off = false;  // whether a result is not finite
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int w = 4; w <= 16; w <<= 1) lw[t][e] += __shfl_xor_sync(0xffffffffu, lw[t][e], w);
        const int r = 8 * t + c0 + e;
        if (r >= q.rows) continue;
        const float inv = lr[t][e] == 0.f ? 0.f : 1.f / lr[t][e];  // no key seen: O = 0 (a NaN sum stays one)
        const RowOut to = row_out<D>(p, q.dst, slab, q.g, q.t0, r);
        float x = 0.f;  // 0, or NaN with one that is not
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int col = 16 * c + 8 * h + lane / 4;
            const float y = o[c][t][2 * h + e] * inv;
            x = fmaf(y, 0.f, x);
            if (to.out)
              to.out[col] = __float2bfloat16_rn(y);
            else
              to.part[col] = y;
          }
        off |= x != 0.f;
        if (lane < 4) {
          const float lse2 = lw[t][e] == 0.f ? -INFINITY : m[t][e] + log2f(lw[t][e]);
          *to.lse = to.out ? lse2 * LN2 : lse2;
        }
      }
    if (lim_min < q.keys && off) *off_flag = 1;  // (see `finite`)
  }
  if (!ok)  // let every copy already issued land before the block exits
#pragma unroll 1
    for (int t = 0; t < L::STAGES && t < issued; ++t)
      drain_all(W, bar_full + 8 * t, ((issued - 1 - t) / L::STAGES) & 1);
}

// ---------------------------------------------------------------- values that are not finite: the block's end
// Lane r's row is at `to` (nowhere: none) and sees the keys of `own` below `lim`: adds to it those values of the keys from k0 to
// k1 that are not finite.  (What the product has taken already changes nothing when it is added again.)
template <int D>
__device__ __noinline__ void add_not_finite(const PrefixParams& p, const int* own, int g, const RowOut& to, int k0, int k1, int lim) {
  const int lane = threadIdx.x & 31;
  const bool out = to.out != nullptr;
  const unsigned long long row = reinterpret_cast<unsigned long long>(out ? static_cast<void*>(to.out) : to.part);
  float sum[D / 32];  // of columns lane, lane + 32 ..: what the keys so far add
#pragma unroll
  for (int c = 0; c < D / 32; ++c) sum[c] = 0.f;
  int next = 0;  // the rows see more keys from one to the next: those before `next` are done
  auto add_below = [&](int k) {  // to the rows that see no key from k on
#pragma unroll 1
    for (; next < 32 && __shfl_sync(0xffffffffu, lim, next) <= k; ++next) {
      const unsigned long long at = __shfl_sync(0xffffffffu, row, next);
      const bool bf16 = __shfl_sync(0xffffffffu, out, next);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        if (!at || sum[c] == 0.f) continue;
        if (bf16) {
          __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(at) + lane + 32 * c;
          *o = __float2bfloat16_rn(__bfloat162float(*o) + sum[c]);
        } else {
          reinterpret_cast<float*>(at)[lane + 32 * c] += sum[c];
        }
      }
    }
  };
#pragma unroll 1
  for (; k0 < k1; k0 += 32) {  // a key per lane first: which have such values
    const uint32_t* mine = nullptr;
    bool any = false;
    if (k0 + lane < k1) {
      const int page = own[(k0 + lane) / kPage];
      if (page >= 0 && page < p.num_pages) {  // (another reads as zeros)
        mine = reinterpret_cast<const uint32_t*>(p.v + ((static_cast<size_t>(page) * p.Hkv + g) * kPage + (k0 + lane) % kPage) * D);
#pragma unroll 4
        for (int c = 0; c < D / 2; ++c) any |= finite(mine[c]) != mine[c];
      }
    }
#pragma unroll 1
    for (unsigned int keys = __ballot_sync(0xffffffffu, any); keys; keys &= keys - 1) {
      const int k = __ffs(keys) - 1;
      const uint32_t* v = reinterpret_cast<const uint32_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), k));
      add_below(k0 + k);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        const uint32_t x = v[(lane + 32 * c) / 2];
        const float y = __uint_as_float(lane & 1 ? x & 0xFFFF0000u : x << 16);
        if (!isfinite(y)) sum[c] += y;
      }
    }
  }
  add_below(INT_MAX);
}

// Lane r's row: `query`, written to `to` (to.lse nullptr: no row), seeing the keys from k0 to k1 of `own` below `lim`.  g: K/V head.
template <int D>
__device__ __noinline__ void rework_rows(const PrefixParams& p, uint8_t* smem, const int* own, int g, const __nv_bfloat16* query,
                                         const RowOut& to, int k0, int k1, int lim) {
  constexpr unsigned int kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  auto place = [&](int key) -> long long {  // of a key's row in the pools; -1: reads as zeros
    const int page = own[key / kPage];
    return page < 0 || page >= p.num_pages ? -1 : (static_cast<long long>(page) * p.Hkv + g) * kPage + key % kPage;
  };
  bool again = false;
  if (to.lse) {
#pragma unroll 1
    for (int c = 0; c < D; ++c) again |= isnan(to.out ? __bfloat162float(to.out[c]) : to.part[c]);
    again &= !isnan(*to.lse);  // (a key that the row sees gives it a NaN)
  }
  // the last key whose value is not finite: hidden ones are a request's last new tokens, 16 at most
  const long long mine = k1 - 1 - lane >= k0 ? place(k1 - 1 - lane) : -1;
  bool off = false;
  if (mine >= 0) {
    const uint32_t* v = reinterpret_cast<const uint32_t*>(p.v + mine * D);
#pragma unroll 4
    for (int c = 0; c < D / 2; ++c) off |= finite(v[c]) != v[c];
  }
  const int last = k1 - __ffs(__ballot_sync(kAll, off));  // (k1 without one)
  again &= last >= lim && last < k1;
  if (!__any_sync(kAll, again)) return;
  const int end = __reduce_max_sync(kAll, again ? min(lim, k1) : 0);
  const float ref = again ? (to.out ? *to.lse / LN2 : *to.lse) : 0.f;  // -infinity: sees none of these keys
  // The rows' queries and 16 keys and values at a time in shared memory, which no one uses any more: a lane works its row, and
  // the lanes read a key's words together.
  constexpr int KEYS = 16, ROW = D * 2, QROW = ROW + 16;  // (a query's bytes in other banks than its neighbours')
  constexpr int AREA = 2 * KEYS * ROW + 32 * QROW;
  static_assert(THREADS / 32 * AREA <= PLayout<D>::XCH_OFF, "the areas reach into what is still needed");
  char* area = reinterpret_cast<char*>(smem) + threadIdx.x / 32 * AREA;
  char* queries = area + 2 * KEYS * ROW;
  if (again)
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c)
      reinterpret_cast<uint4*>(queries + lane * QROW)[c] = reinterpret_cast<const uint4*>(query)[c];
#pragma unroll 1
  for (int half = 0; half < D / 64; ++half) {
    float sum = 0.f, acc[64];
#pragma unroll
    for (int c = 0; c < 64; ++c) acc[c] = 0.f;
#pragma unroll 1
    for (int k = k0; k < end; k += KEYS) {
      __syncwarp();  // the keys before are done with
#pragma unroll 8
      for (int w = lane; w < KEYS * D / 4; w += 32) {  // 16-byte words: the keys', then the values'
        const int key = w / (D / 8) % KEYS;
        const long long at = k + key < end ? place(k + key) : -1;
        const __nv_bfloat16* pool = w < KEYS * D / 8 ? p.k : p.v;
        reinterpret_cast<uint4*>(area)[w] =
            at < 0 ? make_uint4(0, 0, 0, 0) : reinterpret_cast<const uint4*>(pool + at * D)[w % (D / 8)];
      }
      __syncwarp();
      const int count = again ? min(min(KEYS, end - k), lim - k) : 0;
#pragma unroll 1
      for (int e = 0; e < count; ++e) {
        const uint4* key = reinterpret_cast<const uint4*>(area + e * ROW);
        const uint4* q = reinterpret_cast<const uint4*>(queries + lane * QROW);
        float s0 = 0.f, s1 = 0.f;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          const uint4 x = key[c], y = q[c];
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            s0 = fmaf(u2f(xs[b] << 16), u2f(ys[b] << 16), s0);
            s1 = fmaf(u2f(xs[b] & 0xFFFF0000u), u2f(ys[b] & 0xFFFF0000u), s1);
          }
        }
        const float w = ref == -INFINITY ? 0.f : exp2f(fmaf(s0 + s1, p.scale_log2, -ref));
        sum += w;
        const uint4* v = reinterpret_cast<const uint4*>(area + (KEYS + e) * ROW + 128 * half);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 x = v[c];
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            acc[8 * c + 2 * b] = fmaf(w, u2f(xs[b] << 16), acc[8 * c + 2 * b]);
            acc[8 * c + 2 * b + 1] = fmaf(w, u2f(xs[b] & 0xFFFF0000u), acc[8 * c + 2 * b + 1]);
          }
        }
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (again)
#pragma unroll
      for (int c = 0; c < 64; ++c) {
        if (to.out)
          to.out[64 * half + c] = __float2bfloat16_rn(acc[c] * inv);
        else
          to.part[64 * half + c] = acc[c] * inv;
      }
  }
}

// Through the block's pieces once more, after a note: no warp waits for another any more, and the rows and parts are written.
template <int D>
__device__ __noinline__ void mend_block(const PrefixParams& p, uint8_t* smem) {
  const Plan& l = *reinterpret_cast<const Plan*>(smem + PLAN_OFF);
  const Begin* begin = reinterpret_cast<const Begin*>(smem + BEGIN_OFF);
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const unsigned int worker = l.few ? l.worker * kFewWarps + warp : l.worker;
  const unsigned long long from = static_cast<unsigned long long>(worker) * l.share[l.few];
  if ((l.few && warp >= kFewWarps) || from >= l.total[l.few]) return;
  const unsigned int x0 = static_cast<unsigned int>(from);
  const unsigned int x1 = static_cast<unsigned int>(min(from + l.share[l.few], static_cast<unsigned long long>(l.total[l.few])));
  if (l.few) {
    FewWalk walk;
    FewPiece q;
    walk.start(p, l, x0, x1, begin[warp].b, begin[warp].c0);
#pragma unroll 1
    while (walk.next(p, lane, q))
      if (q.step)  // (else all rows see all its keys)
        rework_rows<D>(p, smem, q.table, q.g,
                       p.q + (static_cast<size_t>(q.t0 + lane / p.group) * p.H + q.g * p.group + lane % p.group) * D,
                       lane < q.rows ? row_out<D>(p, q.dst, few_slab(p, worker, q.dst == kDstSlab1), q.g, q.t0, lane) : RowOut{},
                       q.j0 * kStep<D>, min(q.keys, q.j1 * kStep<D>), q.lim0 + lane / p.group);
    return;
  }
  if (x1 <= l.lead[0]) return;  // the prefix's items alone
  unsigned int c0 = begin->c0;
#pragma unroll 1
  for (int b = begin->b; b < p.B && c0 < x1; ++b) {
    const Request r = make_request(p, p.cu_new[b], p.cu_new[b + 1], p.seq_lens[b]);
    if (is_few(p, r)) continue;
    const int ptiles = is_big(p, r) ? p.tiles_p : 0;
#pragma unroll 1
    for (int blk = 0; blk * 2 * p.tp < r.added && c0 < x1; ++blk) {
      Item it = block_item(p, r, blk, c0);
      const unsigned int cost = it.cost();
      c0 += p.Hkv * cost;
      if (it.units == 0) continue;
      const int t = blk * 2 * p.tp, rows = min(2 * p.tp, r.added - t) * p.group;
#pragma unroll 1
      for (int g = 0; g < p.Hkv && it.c0 < x1; ++g, it.c0 += cost) {
        const int j0 = it.from(x0), j1 = it.from(x1);
        if (j0 >= j1 || j1 <= ptiles) continue;
        const int dst = j0 > 0 ? kDstSlab0 : j1 < it.units ? kDstSlab1 : p.tiles_p == ptiles ? kDstOutput : kDstOwn;
#pragma unroll 1
        for (int row = warp * 32 + lane; row - lane < rows; row += THREADS)
          add_not_finite<D>(p, p.block_table + static_cast<size_t>(b) * p.max_pages, g,
                            row < rows ? row_out<D>(p, dst, many_slab(p, worker, dst == kDstSlab1), g, r.first + t, row) : RowOut{},
                            max(max(0, j0 - ptiles) * BN, max(0, r.len - r.added + t + 1)), min(r.len, (j1 - ptiles) * BN),
                            row < rows ? min(r.len, r.len - r.added + t + 1 + row / p.group) : 0);
      }
    }
  }
}

// All keys are loaded to go first from L2: a key tile is read again, by the other row blocks of its head, within
// microseconds, while the kernel's code, which every block waits for as it starts, has to live until the next call (55
// against 61 us for 64 requests behind 16 384 keys, 73 against 84 for 256).  For the same reason loops of run-time length
// stay rolled, and the many-row code comes first: what is further behind the kernel's start arrives later (80 against
// 82 us for 128 requests behind 32 768 keys).
template <int D, int NT>
__global__ void __launch_bounds__(THREADS, 1)
fa_prefix_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmK16,
                 const __grid_constant__ CUtensorMap tmV16, const __grid_constant__ PrefixParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    tma_prefetch_desc(&tmK16);
    tma_prefetch_desc(&tmV16);
    if (smem_u32(smem) % 1024 != 0) atomicOr(&g_prefix_status, kStatusTimeout);  // (the tiles' swizzle needs it)
  }
  volatile unsigned int* need = reinterpret_cast<volatile unsigned int*>(smem + NEED_OFF);
  if (threadIdx.x < kMaxFlags / 32) need[threadIdx.x] = 0;
  // both kinds' barriers and the Tensor Memory: which kind the block works is known only after the wait
  using M = PLayout<D>;
  using F = FLayout<D>;
  const uint32_t sbase = smem_u32(smem);
  if (threadIdx.x < M::NUM_BARS) M::init(sbase, threadIdx.x);
  if (threadIdx.x < F::NUM_BARS) mbar_init(sbase + F::BAR_OFF + 8 * threadIdx.x, 1);
  if (threadIdx.x < 2) reinterpret_cast<volatile int*>(smem + M::MISC_OFF + 4)[threadIdx.x] = 0;
  fence_mbar_init();
  const int warp = uni(threadIdx.x / 32);
  if (warp == MMA_WARP) {
    tmem_alloc(sbase + M::MISC_OFF, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  const Plan l = make_plan(p, *reinterpret_cast<Layout*>(smem), need, reinterpret_cast<Begin*>(smem + BEGIN_OFF));
  if (threadIdx.x == 0) *reinterpret_cast<Plan*>(smem + PLAN_OFF) = l;
  volatile int* flags = reinterpret_cast<volatile int*>(smem + M::MISC_OFF + 4);  // abort, a result is not finite
  if (!l.few) {
    many_rows<D, false>(tmQ, tmK, tmV, p, l, smem);
    if (p.causal) {
      __syncthreads();
      if (__builtin_expect(flags[0] == 0 && flags[1] != 0, 0)) {
        if (threadIdx.x < M::NUM_BARS) {
          asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(sbase + M::BAR_OFF + 8 * threadIdx.x) : "memory");
          M::init(sbase, threadIdx.x);
        }
        fence_mbar_init();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        many_rows_clean<D>(tmQ, tmK, tmV, p, smem);
      }
    }
  } else {
    few_rows<D, NT>(tmK16, tmV16, p, l, smem);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(*reinterpret_cast<volatile uint32_t*>(smem + M::MISC_OFF), 512);
  }
  if (__builtin_expect(p.causal && flags[1] != 0, 0)) {
    __syncwarp();
    mend_block<D>(p, smem);
  }
}

// ---------------------------------------------------------------- join
// The parts of a row follow from the places of its items: an item inside one worker's stretch has one part, with the
// rows of its source; one that is cut has a part in a slab of every worker that worked some of its units.
struct Parts {
  Item it;
  bool few;
  unsigned int share;
  int first, count, seen, at;  // first worker, workers; units visible to the row; the row's number within the item
  __device__ __forceinline__ void locate(const PrefixParams& p, const Plan& l) {
    share = few ? l.share[1] : l.share[0];
    // (places past the last worker come only of a cu_new that decreases, which is reported)
    const unsigned int last = (few ? p.ctas * kFewWarps : p.ctas) - 1;
    const unsigned int w0 = min(it.worker(0, share), last), w1 = min(it.worker(it.units - 1, share), last);
    first = static_cast<int>(w0);
    count = w1 < w0 ? 1 : static_cast<int>(w1 - w0) + 1;
  }
  // Row of the slabs that worker `first + i` wrote the part to; -1 if it had none of the row's units.
  __device__ __forceinline__ long long slab_row(const PrefixParams& p, int i) const {
    const int w = first + i, j0 = it.from(w * share), j1 = it.from((w + 1) * share);
    if (j0 >= j1 || j0 >= seen) return -1;
    return static_cast<long long>((few ? few_slab(p, w, j0 == 0) : many_slab(p, w, j0 == 0)) + at);
  }
};

// A lane's columns of a part.
template <int C, int G>
__device__ __forceinline__ void load_columns(const float* src, int sub, float (&v)[C]) {
  if (C >= 4) {
#pragma unroll
    for (int e = 0; e < C / 4; ++e) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(src + 4 * G * e + 4 * sub));
      v[4 * e] = x.x;
      v[(4 * e + 1) % C] = x.y;
      v[(4 * e + 2) % C] = x.z;
      v[(4 * e + 3) % C] = x.w;
    }
  } else {
    const float2 x = __ldg(reinterpret_cast<const float2*>(src + 2 * sub));
    v[0] = x.x;
    v[1 % C] = x.y;
  }
}

// Joins row h of token n if it needs it: if it has no, or several parts (a row with one item and that inside one worker's
// stretch is written already).  t and rank are the token's.  G lanes of a warp (`mask`, this one the `sub`-th) or, W > 1, W
// whole warps together; every lane has D / G columns.  The lanes look up G parts at a time (warp w of W every W-th), weight
// them by their LSE and add them several loads at a time.
template <int D, int W, int G>
__device__ __forceinline__ void join_row(const PrefixParams& p, const Plan& l, int n, int h, int4 t, int rank, int warp, int sub,
                                         unsigned int mask, float* smem) {
  constexpr int C = D / G;  // columns 4 G e + 4 sub .. of the e-th four, or (C < 4) C sub ..
  const size_t orow = static_cast<size_t>(n) * p.H + h;
  const int g = h / p.group, hh = h - g * p.group;
  Parts pre, own;
  pre.count = own.count = 0;
  if (t.z > 0) {
    own.few = t.w & kTokFew;
    own.it = Item{static_cast<unsigned int>(t.x), own.few ? kFewItemCost : kItemCost,
                  own.few ? 1u : static_cast<unsigned int>(t.w) >> 16, t.y};
    own.it.c0 += g * own.it.cost();
    own.seen = t.z;
    own.at = (t.w & (kTokFew - 1)) * p.group + hh;
    own.locate(p, l);
    if (rank < 0 && own.count == 1) return;
  }
  if (rank >= 0) {
    pre.few = few_prefix(p, l.tokens);
    pre.it = prefix_item(p, l.tokens, g * l.items + rank);
    pre.seen = INT_MAX;
    pre.at = (pre.few ? n : n % (2 * p.tp)) * p.group + hh;
    pre.locate(p, l);
  }
  float m = -INFINITY, sum = 0.f, acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = 0.f;
  const int parts = pre.count + own.count;
#pragma unroll 1
  for (int i0 = 0; i0 < parts; i0 += G * W) {
    const int i = i0 + sub * W + (W > 1 ? warp : 0);
    float lse2 = -INFINITY;
    const float* o = p.slab_o;
    if (i < parts) {
      const bool is_own = i >= pre.count;
      if ((is_own ? own.count : pre.count) == 1) {
        o = (is_own ? p.own_o : p.prefix_o) + orow * D;
        lse2 = __ldg((is_own ? p.own_lse : p.prefix_lse) + orow);
      } else {
        const Parts part = is_own ? own : pre;
        const long long row = part.slab_row(p, is_own ? i - pre.count : i);
        if (row >= 0) {
          o = p.slab_o + row * D;
          lse2 = __ldg(p.slab_lse + row);
        }
      }
    }
    float top = lse2;
#pragma unroll
    for (int w = G / 2; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(mask, top, w, G));
    top = fmaxf(top, m);
    const float f = m == -INFINITY ? 0.f : exp2f(m - top);
    float mine = lse2 == -INFINITY ? 0.f : exp2f(lse2 - top);
    if (lse2 != -INFINITY && mine < FLT_MIN) mine = FLT_MIN;  // not 0: what is not finite in a part stays in the sum
    m = top;
    float all = mine;
#pragma unroll
    for (int w = G / 2; w; w >>= 1) all += __shfl_xor_sync(mask, all, w, G);
    sum = sum * f + all;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] *= f;
    const int here = min(G, (parts - i0 + W - 1) / W);
    // (lanes without a part have weight 0 and the address of some other: loaded all the same, so that the loads of several
    // parts are under way together, and not added)
#pragma unroll 4 / (C > 4 ? C / 4 : 1)
    for (int k = 0; k < here; ++k) {
      const float w = __shfl_sync(mask, mine, k, G);
      const float* src = reinterpret_cast<const float*>(__shfl_sync(mask, reinterpret_cast<unsigned long long>(o), k, G));
      float v[C];
      load_columns<C, G>(src, sub, v);
      if (w != 0.f)
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] += w * v[c];
    }
  }
  if (W > 1) {  // the warps' sums, always in the same order
    float(*s_acc)[D] = reinterpret_cast<float(*)[D]>(smem);
    float* s_m = smem + W * D;
    float* s_sum = s_m + W;
    s_m[warp] = m;
    s_sum[warp] = sum;
#pragma unroll
    for (int c = 0; c < C; ++c) s_acc[warp][sub * C + c] = acc[c];  // (G = 32: C <= 4)
    __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < W; ++w) top = fmaxf(top, s_m[w]);
    sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = s_m[w] == -INFINITY ? s_sum[w] : exp2f(s_m[w] - top);  // (no part: 0; a NaN sum stays one)
      sum += f * s_sum[w];
#pragma unroll
      for (int c = 0; c < C; ++c) acc[c] += f * s_acc[w][sub * C + c];
    }
    m = top;
    if (warp > 0) return;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  __nv_bfloat16* out = p.o + orow * D;
  if (C >= 4) {
#pragma unroll
    for (int e = 0; e < C / 4; ++e)
      *reinterpret_cast<uint2*>(out + 4 * G * e + 4 * sub) =
          make_uint2(pack_bf16x2(acc[4 * e] * inv, acc[4 * e + 1] * inv), pack_bf16x2(acc[4 * e + 2] * inv, acc[4 * e + 3] * inv));
  } else {
    *reinterpret_cast<uint32_t*>(out + 2 * sub) = pack_bf16x2(acc[0] * inv, acc[1 % C] * inv);
  }
  if (sub == 0) p.lse[orow] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * LN2;
}

// Joins the rows that need it.  W = 8: a row per block (few rows, perhaps of many parts); else a warp or, of many rows,
// eight lanes a row (prompt chunks: two rows of five have two parts, and the time is that of their loads one after another).
constexpr int kJoinThreads = 128;
template <int D, int W, int G>
__global__ void __launch_bounds__(W > 1 ? 32 * W : kJoinThreads) fa_prefix_join_kernel(const __grid_constant__ PrefixParams p) {
  __shared__ float smem[W > 1 ? W * D + 2 * W : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % G;
  const unsigned int mask = G == 32 ? 0xffffffffu : 0xffu << (lane & 24);
  pdl_launch_dependents();  // a following call's blocks may set themselves up
  const unsigned int all = static_cast<unsigned int>(p.N) * p.H;  // (N H is below 2^31)
  const unsigned int stride = W > 1 ? gridDim.x : gridDim.x * (kJoinThreads / G);
  unsigned int row = W > 1 ? blockIdx.x : blockIdx.x * (kJoinThreads / G) + threadIdx.x / G;
  if (row >= all) return;
  Plan l;
  l.share[0] = p.hdr[kHdrShare];
  l.share[1] = p.hdr[kHdrShare + 1];
  l.items = p.hdr[kHdrItems];
  l.tokens = p.hdr[kHdrTokens];
#pragma unroll 1
  for (; row < all; row += stride) {
    const int n = static_cast<int>(row / p.H), h = static_cast<int>(row) - n * p.H;
    const int4 t = __ldg(p.tok + n);  // (past the last token: whatever, not used)
    const int rank = __ldg(p.rank + n);
    if (n < l.tokens) join_row<D, W, G>(p, l, n, h, t, rank, warp, sub, mask, smem);
  }
}

template <int D, int NT>
static cudaError_t launch(const PrefixMaps& t, const PrefixParams& p, cudaStream_t stream) {
  static bool attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && !attr_set[dev]) {
    e = cudaFuncSetAttribute(fa_prefix_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const long long rows = static_cast<long long>(p.N) * p.H;
  // Few rows, perhaps of many parts: the join takes a block for each.  Against a warp for each, with 32 heads of 128: one
  // request with 30 000 keys 35 and 63 us, 18 requests (576 rows) behind 4 096 keys 21.0 and 22.7, with 100 keys behind 256 16.0
  // and 15.7; 20 requests (640 rows) 22.9 and 23.8, 17.0 and 16.1; 32 requests 27.5 and 25.4, 19.1 and 16.3.
  const bool wide = rows < 4 * p.ctas;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.stream = stream;
  cfg.attrs = attr;
  // Launched early (its blocks set themselves up while the kernel before it ends) only when there are few rows.  Early and
  // not, in a graph: 12.9 and 13.5 us for one request, 15.6 and 16.2 for 20 with 100 keys behind 256 (18.7 and 20.7 launched one
  // by one), 25.5 and 25.4 for 32 (1 024 rows) behind 4 096 keys (28.2 and 29.6), 32.1 and 30.8 for 64.  Blocks that start as
  // the preceding kernel's end land on the SMs in any order, and the last block numbers, which stream the requests' own
  // keys, gather on neighbouring SMs and starve the others there (76 -> 88 us for 128 requests behind 32 768 keys).
  cfg.numAttrs = rows < 8 * p.ctas ? 1 : 0;
  cfg.gridDim = dim3(p.ctas);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  if ((e = cudaLaunchKernelEx(&cfg, fa_prefix_kernel<D, NT>, t.q, t.k, t.v, t.k16, t.v16, p)) != cudaSuccess) return e;
  // A warp a row, or of more rows eight lanes, 12 blocks per SM at most.  Behind 4 096 keys with 300 of their own: 64 requests
  // (2 048 rows) 30.5 us with a warp and 32.6 with eight lanes, 128 requests 40.3 and 40.3, 200 requests 54.4 and 52.0; a prompt of 200
  // tokens (6 400 rows) 22.1 and 20.1; prompt chunks with 77 568 rows 149 and 130.
  const int lanes = rows <= 27ll * p.ctas ? 32 : 8;
  const long long blocks = (rows * lanes + kJoinThreads - 1) / kJoinThreads;
  // not launched early: its blocks would gather on the SMs whose attention block ends first (46 -> 63 us for 64
  // requests behind 16 384 keys)
  cfg.numAttrs = 0;
  cfg.gridDim = dim3(static_cast<unsigned int>(wide ? rows : blocks < 12 * p.ctas ? blocks : 12 * p.ctas));
  cfg.blockDim = dim3(wide ? 256 : kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return wide          ? cudaLaunchKernelEx(&cfg, fa_prefix_join_kernel<D, 8, 32>, p)
         : lanes == 32 ? cudaLaunchKernelEx(&cfg, fa_prefix_join_kernel<D, 1, 32>, p)
                       : cudaLaunchKernelEx(&cfg, fa_prefix_join_kernel<D, 1, 8>, p);
}

cudaError_t launch_fa_fwd_prefix(int d, const PrefixMaps& t, const PrefixParams& p, cudaStream_t stream) {
  if (d == 128) return launch<128, 1>(t, p, stream);
  return p.few_rows == 8 ? launch<64, 1>(t, p, stream) : launch<64, 2>(t, p, stream);
}

unsigned int prefix_page_cost() { return kTileCost256; }
unsigned int prefix_item_cost() { return kItemCost; }
static_assert(kTileCost256 >= kPage / kStep<128> && kItemCost >= kFewItemCost, "prefix_page_cost, prefix_item_cost");

cudaError_t read_prefix_status(unsigned int* out) {
  return cudaMemcpyFromSymbolAsync(out, g_prefix_status, sizeof(unsigned int), 0, cudaMemcpyDeviceToHost, cudaStreamLegacy);
}
cudaError_t clear_prefix_status() {
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_prefix_status, &zero, sizeof(unsigned int));
}

}  // namespace fa
