// Dense attention for prompt rows on the 5th-generation tensor cores: rows of
// one request that follow one another share each tile of keys and values.
//
// The mathematics is dense_attn.cu's.  dense_plan_kernel cuts every run of
// consecutive rows of one request into chunks of at most 2 * (128 / G) rows
// (G query heads per KV head), at least kMinRows, unless all of them are
// little work; other CTAs of the same launch take the other rows.  A chunk and a KV head
// are one or two query tiles of 128 (query = row * G + head), and a unit of
// work is one tile of 128 positions for them.  All units form one sequence,
// cut into equal shares by cost, one per CTA; a (chunk, head) inside one share
// is finished there, one that crosses shares leaves partial states that
// dense_merge_kernel joins.  Where whole (chunk, head)s balance well enough,
// shares end with them.
//
// dense_prompt_kernel (persistent, one CTA per SM, 12 warps; the first CTAs, as
// many as the plan gives them):
//  * warp 0 streams the K tiles and warp 2 the V tiles (TMA, whole pages of
//    one head, 128-byte swizzle) into rings of 2 stages, warp 2 also each
//    segment's queries once the one before has had its last S;
//  * warp 1 issues the MMAs: S_w = Q_w K^T for the query tiles w = 0, 1, then
//    O_w += P_w V with P_w read from tensor memory, and the next tile's S_w
//    right behind it, so that while one query tile's softmax runs, the other
//    one's two products do;
//  * warps 4..7 and 8..11 are the softmax of query tile 0 and 1, thread =
//    query: the row of S in registers, masked where the tile crosses the row's
//    length, window or sinks, maximum (moves only when exceeded by more than
//    2^8, then O_w is rescaled), p = 2^(x - m), sum in fp32, P to tensor
//    memory over S; outputs go through shared memory in whole lines.
// P is rounded to bf16 here (the sum l takes it unrounded): its error is that
// of the output's own rounding, relative 2^-8 a term at most (against 64 bits
// the outputs of a prompt are 0.0021 to 0.0023 off, 2-norm, where unrounded ones
// are 0.0016 to 0.0017).  A second term as in the per-row kernel adds a half to
// the tensor work and lengthens the chain: with it the windowed prompt's call
// takes 211 us instead of 158, and 48 decode rows beside 512 tokens 593 instead
// of 573.
// A masked position has p = 0, and 0 times an infinity or NaN in V would reach
// rows that do not see it: V rows past the chunk's longest length are zeroed in
// shared memory, and a row whose output is not finite for any other reason is
// done again by the per-row kernel, which reads visible positions only.
//
// What bounds it: the chain of one query tile, S -> softmax -> P V -> next S,
// some 3,500 cycles a key tile where both query tiles' 32 products take 2,080
// (65 cycles a 128 x 128 x 16 MMA, measured alone).  512 tokens behind 8192 with
// 64 / 8 heads: 114-116 us, 1.22-1.24 PFLOP/s of products that a row sees; a
// 4095-token prompt under a window of 1024: 129 us.  Tried and no faster, by the
// first of these cases (120 us then): two softmax warps a row 126, P in two
// halves 127, an issuing warp a query tile 147.  Registers split by setmaxnreg: not timed, the
// compiler spilled.
#include <algorithm>

#include "dense_rows.cuh"

namespace dsa {
namespace {

constexpr int kPT = 128;                          // positions per tile
constexpr int kPKStages = 2, kPVStages = 2;
constexpr int kSoftWarps = 8;                     // 4 a query tile, 32 rows each
constexpr int kPWarps = 4 + kSoftWarps;
constexpr int kStageB = 4096;                     // a softmax warp's staging: 128 bytes of each of its rows
constexpr int kPThreads = kPWarps * 32;
constexpr int kPOk = 8;                           // page-validity ring, more than the K ring's tiles in flight
constexpr long long kPWaitBudget = 2000000000LL;  // SM cycles (about 1 s)
constexpr int kPlanThreads = 1024;
constexpr int kMinRows = 2;                       // fewer rows: the per-row kernel reads as much and computes less
constexpr int kMinCost = 8;                       // cost units (query tiles x key tiles) per CTA at least

// tensor-memory columns: S_w [128 x 128] fp32 at 128 w (P_w, bf16, over its
// first 64), O_w [128 x D] fp32 at 256 + 128 w
constexpr uint32_t kPColS = 0, kPColO = 256, kPTmemCols = 512;

// ---------------------------------------------------------------- tiles
// The pages that rows of lengths lmin .. lmax see, n tiles of 128 / P of them:
// ns pages with their sinks, then those from page w0 to the longest row's end.
// A tile's pages need not follow one another.
struct TileSpan {
  int ns, w0, pages, n;
  __device__ __forceinline__ int page(int j) const { return j < ns ? j : j - ns + w0; }
};
__device__ __forceinline__ TileSpan tile_span(const DenseParams &p, int lmin, int lmax) {
  TileSpan s;
  const int sink_end = p.window > 0 ? min(p.sinks, lmax) : 0;
  const int lo = p.window > 0 ? max(0, lmin - p.window) : 0;
  const int P = p.page_size, sh = p.page_shift;
  s.ns = (sink_end + P - 1) >> sh;
  s.w0 = max(s.ns, lo >> sh);
  s.pages = s.ns + ((lmax + P - 1) >> sh) - s.w0;
  s.n = ((s.pages << sh) + kPT - 1) / kPT;
  return s;
}
__device__ __forceinline__ int rows_per_tile(const DenseParams &p) { return 128 / (p.num_q_heads / p.num_kv_heads); }

// Cost of n tiles of one (chunk, KV head) with 1 or 2 query tiles: a unit a
// product pair, and kSegCost a query tile for what a segment takes besides
// (queries to load, the pipeline to fill and drain, outputs to write).  A pair
// alone is priced at half of two by its products, though its chain is as long
// (see above): where calls mix chunks of both kinds, those of one query tile get
// too few CTAs (64 requests of 4 rows each behind 8192 tokens take 375 us, of
// one row each, the same keys, 324).
constexpr int kSegCost = 3;
__device__ __forceinline__ int segment_cost(int n, int tiles) { return (n + kSegCost) * tiles; }
// Shares end at segments' ends (no partial states, no join) unless that makes
// the largest share this much larger than the mean: what a share's two partial
// segments and the join behind take: estimated at 10,000 cycles for the former
// and 10 to 13 us, the join's measured time, for the latter, in units of a query
// tile's 1,700 cycles.
constexpr int kSplitCost = 20;
// The first of its tiles whose cost lies at or past `at`.
__device__ __forceinline__ int tile_at(int at, int tiles) {
  return max(0, (at - kSegCost * tiles + tiles - 1) / tiles);
}

// Rows whose K and V, read row by row, come to less than this in all are left
// to the per-row kernel: the tiles' launches take some 12 us however little
// they do.
constexpr long long kLeastBytes = 32 << 20;

// Tiles and single rows run side by side, each on CTAs of its own, so that
// the former's chains and the latter's reads overlap (48 rows of up to 32768
// keys beside 512 tokens behind 8192: 516 to 529 us, one after the other 627; in
// other processes 565 to 588, and why is not known).  Their
// times, in SM cycles: a cost unit takes 1,700, and up to 800 more as the
// single rows near HBM's rate; single rows stream 36 (D 64: 22) bytes a cycle
// and CTA up to that rate.  Fitted, D 128, 64 / 8 heads beside the same tokens:
// rates of 28, 32 and 42 take 724, 588 and 559 us; without the 800, 200 rows of
// up to 4096 keys take 411 us instead of 355, and 24 rows beside 2000 tokens 934
// instead of 894; with a flat 2,600 a unit, 8 rows take 222 instead of 185.  A
// unit's times are those of D 128; D 64's are some 0.8 of them (512 tokens behind
// 8192: the call takes 106 us, 128 with D 128).
constexpr float kTileClk = 1700.f, kTileBusyClk = 800.f, kRowRate128 = 36.f, kRowRate64 = 22.f, kMemRate = 3450.f;

// ----------------------------------------------------------------- plan
// Bits of the rows where a run (of one request, its rows' windows touching)
// begins or a pad row lies, and
// of the words that hold any; the nearest such row at or below r, above r.
struct RowBits {
  const uint32_t *w, *any;  // [128] a bit a row, [4] a bit a word
  __device__ __forceinline__ int below(int r) const {  // row 0 is always set
    int k = r >> 5;
    uint32_t v = w[k] & (0xFFFFFFFFu >> (31 - (r & 31)));
    if (v == 0u) {
      int j = (k - 1) >> 5;
      uint32_t u = any[j] & (0xFFFFFFFFu >> (31 - ((k - 1) & 31)));
      while (u == 0u) u = any[--j];
      k = j * 32 + 31 - __clz(static_cast<int>(u));
      v = w[k];
    }
    return k * 32 + 31 - __clz(static_cast<int>(v));
  }
  __device__ __forceinline__ int above(int r, int R) const {
    if (r + 1 >= R) return R;
    int k = (r + 1) >> 5;
    uint32_t v = w[k] & (0xFFFFFFFFu << ((r + 1) & 31));
    if (v == 0u) {
      int j = (k + 1) >> 5;
      uint32_t u = j < 4 ? any[j] & (0xFFFFFFFFu << ((k + 1) & 31)) : 0u;
      while (u == 0u && j + 1 < 4) u = any[++j];
      if (u == 0u) return R;
      k = j * 32 + __ffs(static_cast<int>(u)) - 1;
      v = w[k];
    }
    return min(R, k * 32 + __ffs(static_cast<int>(v)) - 1);
  }
};

__global__ void __launch_bounds__(kPlanThreads)
    dense_plan_kernel(const DenseParams p, const DensePromptParams t, int head_dim, int all_ctas) {
  __shared__ uint32_t bits[128], words[4];  // max_rows <= 4096
  __shared__ int len_s[4096], req_s[4096];
  __shared__ int sum_n[32], sum_c[32];
  __shared__ int total_n, total_c, most, empty_n;
  __shared__ unsigned long long seen_s, all_s;  // positions that the chunks' rows see, and all rows
  __shared__ unsigned long long best_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, R = p.max_rows;
  pdl_launch_dependents();
  if (tid == 0) {
    seen_s = all_s = 0;
    best_s = ~0ull;
    empty_n = 0;
  }
  pdl_wait();
  if (tid < (R + 31) / 32) t.redo[tid] = 0u;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int r = e * kPlanThreads + tid;
    int L = 0, req = -1;
    if (r < R) {
      L = p.row_len[r];
      req = p.row_req[r];
      if (L < 0 || L > p.max_len || (L > 0 && (req < 0 || req >= p.max_reqs))) {
        flag_status(p.status, DSA_DEV_BAD_ROW);
        L = 0;
      }
    }
    len_s[r] = L;
    req_s[r] = req;
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int r = e * kPlanThreads + tid;
    // under a window, lengths further apart than it leave positions between that neither row sees, and whose
    // pages may be gone: the run ends there, so that a chunk's tiles are pages that its rows see
    const bool same = r > 0 && len_s[r] > 0 && len_s[r - 1] > 0 && req_s[r - 1] == req_s[r] &&
                      (p.window == 0 || abs(len_s[r] - len_s[r - 1]) <= p.window);
    const uint32_t b = __ballot_sync(0xFFFFFFFFu, !same);
    if (lane == 0) bits[r >> 5] = b;
  }
  __syncthreads();
  if (warp < 4) {
    const uint32_t b = __ballot_sync(0xFFFFFFFFu, bits[warp * 32 + lane] != 0u);
    if (lane == 0) words[warp] = b;
  }
  __syncthreads();
  const RowBits runs{bits, words};
  // a chunk's shortest and longest row, at half its first row (chunks have two
  // rows at least); the requests are done with
  int *lmin_s = req_s, *lmax_s = req_s + 2048;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    lmin_s[e * kPlanThreads + tid] = 0x7FFFFFFF;
    lmax_s[e * kPlanThreads + tid] = 0;
  }
  __syncthreads();
  const int step = 2 * rows_per_tile(p);
  // thread = rows 4 tid .. 4 tid + 3, so chunks are numbered in row order
  int rows[4], cost[4], n = 0, c = 0;
  uint32_t in_chunk = 0u;  // a bit a row
  long long seen = 0, all = 0;
  {
    // the chunk of the row before is this row's too until it is full or its
    // run ends; its rows here are joined before they meet the other threads'
    int head = 0, size = 0, end = 0, lo = 0x7FFFFFFF, hi = 0;
    auto flush = [&] {
      if (hi > 0) {
        atomicMin(lmin_s + (head >> 1), lo);
        atomicMax(lmax_s + (head >> 1), hi);
      }
      lo = 0x7FFFFFFF;
      hi = 0;
    };
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 4 * tid + e;
      rows[e] = 0;
      const int L = r < R ? len_s[r] : 0;
      if (e == 0 || r >= end || r >= head + size) {
        flush();
        if (e == 0 || r >= end) {
          const int start = r < R ? runs.below(r) : r;
          end = r < R ? runs.above(r, R) : r + 1;
          head = start + (r - start) / step * step;  // the chunk's first row
        } else {
          head = r;
        }
        size = min(step, end - head);
      }
      const long long sees =
          p.window > 0 && L > p.window ? static_cast<long long>(p.window) + min(p.sinks, L - p.window) : L;
      all += sees;
      if (L == 0 || size < kMinRows) continue;
      in_chunk |= 1u << e;
      if (head == r) rows[e] = size;
      lo = min(lo, L);
      hi = max(hi, L);
      seen += sees;
    }
    flush();
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    seen += __shfl_xor_sync(0xFFFFFFFFu, seen, o);
    all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
  }
  if (lane == 0 && all > 0) {
    atomicAdd(&seen_s, static_cast<unsigned long long>(seen));
    atomicAdd(&all_s, static_cast<unsigned long long>(all));
  }
  __syncthreads();
  const bool none = static_cast<long long>(seen_s) * p.num_kv_heads * head_dim * 4 < kLeastBytes || all_ctas < 2;
  {
    // 8 threads' rows are a word of the bitmaps
    uint32_t alone = 0u, empty = 0u;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = 4 * tid + e;
      if (r < R && len_s[r] == 0) empty |= 1u << e;
      else if (r < R && (none || !((in_chunk >> e) & 1u))) alone |= 1u << e;
    }
    const uint32_t pads = __reduce_add_sync(0xFFFFFFFFu, static_cast<unsigned>(__popc(empty)));
    if (lane == 0 && pads != 0u) atomicAdd(&empty_n, static_cast<int>(pads));
    alone <<= 4 * (lane & 7);
    empty <<= 4 * (lane & 7);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      alone |= __shfl_xor_sync(0xFFFFFFFFu, alone, o);
      empty |= __shfl_xor_sync(0xFFFFFFFFu, empty, o);
    }
    if ((lane & 7) == 0 && 4 * tid < R) {
      t.alone[tid >> 3] = alone;
      t.empty[tid >> 3] = empty;
    }
  }
  DenseChunk ch[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int r = 4 * tid + e;
    cost[e] = 0;
    if (none) rows[e] = 0;
    if (r >= R) continue;
    if (rows[e] > 0) {
      ch[e].first = r;
      ch[e].rows = rows[e];
      ch[e].lmin = lmin_s[r >> 1];
      ch[e].lmax = lmax_s[r >> 1];
      const int tiles = rows[e] > step / 2 ? 2 : 1;
      cost[e] = segment_cost(tile_span(p, ch[e].lmin, ch[e].lmax).n, tiles) * p.num_kv_heads;
      ++n;
      c += cost[e];
    }
  }
  int in_n = n, in_c = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, in_n, o), y = __shfl_up_sync(0xFFFFFFFFu, in_c, o);
    if (lane >= o) {
      in_n += x;
      in_c += y;
    }
  }
  if (lane == 31) {
    sum_n[warp] = in_n;
    sum_c[warp] = in_c;
  }
  __syncthreads();
  int at = in_n - n, before = in_c - c;
  for (int w = 0; w < warp; ++w) {
    at += sum_n[w];
    before += sum_c[w];
  }
  int *before_s = len_s;  // the lengths are done with
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (rows[e] > 0) {
      t.chunks[at] = ch[e];
      t.before[at] = before_s[at] = before;
      ++at;
      before += cost[e];
    }
  if (tid == kPlanThreads - 1) {
    *t.nchunks = at;
    t.before[at] = before_s[at] = before;
    total_n = at;
    total_c = before;
    most = 0;
  }
  __syncthreads();
  // ---- CTAs for the tiles and for the single rows: the split whose longer
  // side is shortest
  const int U = total_c;
  const long long alone_seen = static_cast<long long>(none ? all_s : all_s - seen_s);
  const float rows_bytes = static_cast<float>(alone_seen) * (4.f * p.num_kv_heads * head_dim) +
                           static_cast<float>(empty_n) * (2.f * p.num_q_heads * head_dim);
  if (tid < 256) {
    unsigned long long v = ~0ull;
    if (tid >= 1 && tid < all_ctas) {
      const float rate = fminf(tid * (head_dim == 128 ? kRowRate128 : kRowRate64), kMemRate);
      const float unit = kTileClk + kTileBusyClk * (rate / kMemRate);
      const float time = fmaxf(U * unit / (all_ctas - tid), rows_bytes / rate);
      v = static_cast<unsigned long long>(__float_as_uint(time)) << 32 | tid;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if (lane == 0) atomicMin(&best_s, v);
  }
  __syncthreads();
  const int ctas = U == 0 ? 0 : rows_bytes == 0.f ? all_ctas : all_ctas - static_cast<int>(best_s & 0xFFFFFFFFu);
  if (tid == 0) t.nchunks[1] = ctas;
  // whole segments or equal shares: thread c finds where CTA c's share of
  // whole segments begins, and how large it is
  const int nchunks = total_n;
  const Shares shares(U, ctas, kMinCost);
  const int x = tid < shares.A ? shares.begin(tid) : U;
  int2 at_seg = make_int2(nchunks * p.num_kv_heads, U);
  if (tid < shares.A) {
    int lo = 0, hi = nchunks;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before_s[mid] <= x) lo = mid;
      else hi = mid;
    }
    const int base = before_s[lo], per = (before_s[lo + 1] - base) / p.num_kv_heads, g = (x - base + per - 1) / per;
    at_seg = make_int2(lo * p.num_kv_heads + g, base + g * per);  // the first segment that starts at x or past it
  }
  if (tid <= ctas) req_s[tid] = at_seg.y;
  __syncthreads();
  if (tid < shares.A) atomicMax(&most, req_s[tid + 1] - req_s[tid]);
  __syncthreads();
  const bool whole = shares.A > 0 && most - shares.q <= kSplitCost;
  if (!whole && at_seg.y != x) {  // x lies inside the segment before
    --at_seg.x;
    at_seg.y = x;
  }
  if (tid <= ctas) t.shares[tid] = at_seg;
}

// ------------------------------------------------------------- segments
// One (chunk, KV head)'s tiles [t0, t1) of its n in a CTA's share.
struct Segment {
  DenseChunk c;
  int id, g, req, tiles;  // id: chunk * Hkv + g; tiles: query tiles (1 or 2)
  int cost0;              // cost before this (chunk, head)
  int t0, t1;
  TileSpan span;
  bool begins, ends;
};
// A CTA's segments follow one another: segment k is KV head k % Hkv of chunk
// k / Hkv.  Every role walks them, so the first kSegCache are worked out once,
// a thread each, into shared memory; the rest where they are needed.
constexpr int kSegCache = 24;
struct SegCache {
  DenseChunk c[kSegCache];
  int4 at[kSegCache];  // request, cost before the segment, first and last tile
};
__device__ __forceinline__ void locate(const DenseParams &p, const DensePromptParams &t, int k, int x0, int x1,
                                       DenseChunk &c, int4 &at) {
  const int chunk = k / p.num_kv_heads, g = k - chunk * p.num_kv_heads;
  c = t.chunks[chunk];
  const int tiles = c.rows > rows_per_tile(p) ? 2 : 1, per = segment_cost(tile_span(p, c.lmin, c.lmax).n, tiles);
  at.x = p.row_req[c.first];
  at.y = t.before[chunk] + g * per;
  at.z = tile_at(max(x0, at.y) - at.y, tiles);  // a tile belongs to the share its first cost unit is in
  at.w = tile_at(min(x1, at.y + per) - at.y, tiles);
}
struct Walk {
  const SegCache *cache;
  int x0, x1;         // the share, in cost
  int k0, k1, k;      // its segments, the next one
  __device__ __forceinline__ bool next(const DenseParams &p, const DensePromptParams &t, Segment &s) {
    while (k < k1) {
      int4 at;
      if (k - k0 < kSegCache) {
        s.c = cache->c[k - k0];
        at = cache->at[k - k0];
      } else {
        locate(p, t, k, x0, x1, s.c, at);
      }
      s.id = k++;
      if (at.z >= at.w) continue;
      s.req = at.x;
      s.cost0 = at.y;
      s.t0 = at.z;
      s.t1 = at.w;
      s.g = s.id % p.num_kv_heads;
      s.tiles = s.c.rows > rows_per_tile(p) ? 2 : 1;
      s.span = tile_span(p, s.c.lmin, s.c.lmax);
      s.begins = s.t0 == 0;
      s.ends = s.t1 == s.span.n;
      return true;
    }
    return false;
  }
};

struct PromptLayout {
  uint32_t off_q, off_k, off_v, off_stage, off_ok, off_bar, off_cache, off_misc;
};

__device__ __forceinline__ bool pwarp_wait(uint32_t bar, uint32_t parity, const volatile int *abort_flag) {
  const bool ok = tc::mbar_wait(bar, parity, abort_flag, kPWaitBudget);
  return __all_sync(0xFFFFFFFFu, ok);
}
// Two fp32 values in one 64-bit register: a product-sum and a sum of both in
// one instruction, and the largest of three.
__device__ __forceinline__ uint64_t pack2u(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) { return pack2u(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ void unpack2(uint64_t r, float &a, float &b) {
  uint32_t x, y;
  asm("mov.b64 {%0, %1}, %2;\n" : "=r"(x), "=r"(y) : "l"(r));
  a = __uint_as_float(x);
  b = __uint_as_float(y);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u; }

// CTA `me` of the `ctas` that take tiles.
template <int D>
__device__ __forceinline__ void prompt_tiles(const DenseParams &p, const DensePromptParams &t, const PromptLayout &lay,
                                             const CUtensorMap &kmap, const CUtensorMap &vmap, const CUtensorMap &qmap,
                                             uint8_t *sb, uint32_t base, int me, int ctas) {
  constexpr int kAtoms = D / 64;
  constexpr uint32_t kTileB = kPT * D * 2u, kAtomB = kPT * 128u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int Hq = p.num_q_heads, Hkv = p.num_kv_heads, G = Hq / Hkv, RT = rows_per_tile(p);
  const uint32_t bar0 = base + lay.off_bar;
  auto KFULL = [&](int s) { return bar0 + 8u * s; };
  auto KEMPTY = [&](int s) { return bar0 + 8u * (kPKStages + s); };
  auto VFULL = [&](int s) { return bar0 + 8u * (2 * kPKStages + s); };
  auto VEMPTY = [&](int s) { return bar0 + 8u * (2 * kPKStages + kPVStages + s); };
  constexpr int kB = 2 * (kPKStages + kPVStages);
  auto SFULL = [&](int w) { return bar0 + 8u * (kB + w); };
  auto PFULL = [&](int w) { return bar0 + 8u * (kB + 2 + w); };
  auto OFULL = [&](int w) { return bar0 + 8u * (kB + 4 + w); };
  auto OEMPTY = [&](int w) { return bar0 + 8u * (kB + 6 + w); };
  const uint32_t QFULL = bar0 + 8u * (kB + 8), QEMPTY = QFULL + 8;
  const uint32_t DONE = bar0 + 8u * (kB + 10);
  volatile uint32_t *ok_s = reinterpret_cast<uint32_t *>(sb + lay.off_ok);  // [kPOk] a bit a page of the tile
  int *misc = reinterpret_cast<int *>(sb + lay.off_misc);  // [0] tmem base [1] abort
  volatile int *abort_flag = misc + 1;

  if (tid == 0) {
    for (int s = 0; s < kPKStages; ++s) {
      tc::mbar_init(KFULL(s), 1);
      tc::mbar_init(KEMPTY(s), 1);
    }
    for (int s = 0; s < kPVStages; ++s) {
      tc::mbar_init(VFULL(s), 1);
      tc::mbar_init(VEMPTY(s), 1);
    }
    for (int w = 0; w < 2; ++w) {
      tc::mbar_init(SFULL(w), 2);  // the MMAs' commit, and the issuing thread (it has seen the page bits)
      tc::mbar_init(PFULL(w), 4);  // the query tile's 4 warps
      tc::mbar_init(OFULL(w), 1);
      tc::mbar_init(OEMPTY(w), 4);
    }
    tc::mbar_init(QFULL, 1);
    tc::mbar_init(QEMPTY, 1);
    tc::mbar_init(DONE, 1);
    misc[1] = 0;
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&kmap);
    tc::tma_prefetch_desc(&vmap);
    tc::tma_prefetch_desc(&qmap);
  }
  if (warp == 1) {
    tc::tmem_alloc(smem_u32(&misc[0]), kPTmemCols);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);
  pdl_launch_dependents();  // only now: no later kernel may take the tensor memory that this one waits for

  const int nchunks = *t.nchunks;
  const Shares shares(t.before[nchunks], ctas, kMinCost);
  SegCache *cache = reinterpret_cast<SegCache *>(sb + lay.off_cache);
  Walk walk;
  walk.cache = cache;
  {
    const int2 from = t.shares[me], to = t.shares[me + 1];
    walk.k0 = walk.k = from.x;
    walk.x0 = from.y;
    walk.k1 = to.y > from.y ? to.x + 1 : from.x;  // the last may end where it begins: it has no tile here then
    walk.x1 = to.y;
    if (walk.k1 > nchunks * Hkv) walk.k1 = nchunks * Hkv;
  }
  if (tid < kSegCache && walk.k0 + tid < walk.k1)
    locate(p, t, walk.k0 + tid, walk.x0, walk.x1, cache->c[tid], cache->at[tid]);
  __syncthreads();
  Segment s;

  if (warp == 0 || warp == 2) {
    // ================================== producers: K; V and the queries
    const bool vrole = warp == 2;
    const uint64_t policy = tc::l2_evict_last_policy();  // a request's other tiles and heads' CTAs read the same pages
    const uint64_t qpolicy = tc::l2_evict_first_policy();
    const int P = p.page_size, npg = kPT / P;
    int n = 0, qn = 0;
    bool stop = false;
    auto wait = [&](uint32_t bar, int parity) {
      if (!pwarp_wait(bar, static_cast<uint32_t>(parity), abort_flag)) {
        if (lane == 0) { *abort_flag = 1; flag_status(p.status, DSA_DEV_TIMEOUT); }
        stop = true;
      }
      return !stop;
    };
    while (!stop && walk.next(p, t, s)) {
      const int32_t *pt = p.page_table + static_cast<size_t>(s.req) * p.max_pages_per_req;
      if (vrole) {
        // query tile w: rows first + w RT .., heads of g, as [row * G + head][64] per atom
        if (!wait(QEMPTY, (qn & 1) ^ 1)) break;
        if (lane == 0) tc::mbar_arrive_expect_tx(QFULL, static_cast<uint32_t>(s.tiles * kAtoms * RT * G) * 128u);
        __syncwarp();
        if (lane < s.tiles * kAtoms) {
          const int w = lane / kAtoms, a = lane % kAtoms;
          tma_load_3d(base + lay.off_q + w * kTileB + a * kAtomB, &qmap, a * 64, s.g * G, s.c.first + w * RT, QFULL,
                      qpolicy);
        }
        ++qn;
      }
      for (int i = s.t0; i < s.t1; ++i) {
        // lane kAtoms k + a: the tile's page k, rows of head g, 64-element atom a
        const int k = lane / kAtoms, a = lane % kAtoms, page = i * npg + k;
        int rowc = -P;  // past the last page, or a page outside the pool: zeros
        bool there = false;
        if (k < npg && page < s.span.pages) {
          const int pg = pt[s.span.page(page)];
          there = pg >= 0 && pg < p.num_pages;
          if (there) rowc = pg * P;
          else if (!vrole) flag_status(p.status, DSA_DEV_BAD_PAGE);
        }
        const int st = n % (vrole ? kPVStages : kPKStages), ph = n / (vrole ? kPVStages : kPKStages);
        const uint32_t full = vrole ? VFULL(st) : KFULL(st);
        if (!wait(vrole ? VEMPTY(st) : KEMPTY(st), (ph & 1) ^ 1)) break;
        uint32_t okb = 0u;  // bit k: page k may be read
        if (!vrole) {
          uint32_t b = __ballot_sync(0xFFFFFFFFu, a == 0 && there);
          for (int e = 0; e < npg; ++e) okb |= ((b >> (e * kAtoms)) & 1u) << e;
        }
        if (lane == 0) {
          if (!vrole) ok_s[n % kPOk] = okb;
          tc::mbar_arrive_expect_tx(full, kTileB);
        }
        __syncwarp();
        if (k < npg)
          tc::tma_load_2d(base + (vrole ? lay.off_v : lay.off_k) + st * kTileB + a * kAtomB + k * P * 128u,
                          vrole ? &vmap : &kmap, s.g * D + a * 64, rowc, full, policy);
        ++n;
      }
    }
    // no copy may land after the CTA exits
    if (lane == 0) {
      const int S = vrole ? kPVStages : kPKStages;
      for (int i = max(0, n - S); i < n; ++i)
        tc::mbar_wait(vrole ? VFULL(i % S) : KFULL(i % S), (i / S) & 1, nullptr, kPWaitBudget);
      if (qn > 0) tc::mbar_wait(QFULL, (qn - 1) & 1, nullptr, kPWaitBudget);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ============================================================== MMA
    // One warp issues both query tiles' products (one elected lane): tile w's
    // two, P V and the next S, go out together, so that the tiles take turns
    // on the tensor cores; issued apart by two warps the kernel was slower
    // (147 us where it took 120).
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    const uint32_t idesc_qk = tc::idesc_m128(kPT, false);
    const uint32_t idesc_pv = tc::idesc_m128(D, false) | (1u << 16);  // B (V) MN-major
    const uint64_t dq0 = tc::desc_kmajor(base + lay.off_q), dk0 = tc::desc_kmajor(base + lay.off_k),
                   dv0 = tc::desc_mnmajor(base + lay.off_v, kAtomB, 1024u);
    constexpr uint64_t kAtomD = kAtomB >> 4, kTileD = kTileB >> 4;  // descriptor address units
    int kn = 0, vn = 0, qn = 0, pn[2] = {0, 0}, on[2] = {0, 0};
    bool stop = false, any = false;
    auto wait = [&](uint32_t bar, int parity) {
      if (!pwarp_wait(bar, static_cast<uint32_t>(parity), abort_flag)) stop = true;
      return !stop;
    };
    auto kwait = [&] { return wait(KFULL(kn % kPKStages), (kn / kPKStages) & 1); };
    // V of the segment's tile i; its rows past the longest row are zeroed
    auto vwait = [&](int i) {
      const int vs = vn % kPVStages;
      if (!wait(VFULL(vs), (vn / kPVStages) & 1)) return false;
      // the longest row's end in its last page; pages behind were zero-filled
      const int end = (s.span.pages << p.page_shift) - i * kPT;
      const int stale = end - ((s.span.page(s.span.pages - 1) + 1) * p.page_size - s.c.lmax);
      if (i + 1 == s.span.n && stale < end) {
        uint8_t *v = sb + lay.off_v + vs * kTileB;
        for (int e = lane; e < (end - stale) * kAtoms * 8; e += 32) {
          const int row = stale + e / (kAtoms * 8), c16 = e % (kAtoms * 8);
          *reinterpret_cast<uint4 *>(v + (c16 >> 3) * kAtomB + row * 128 + (c16 & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
      }
      return true;
    };
    // Issued by the elected lane: S_w = Q_w K^T of the K tile in stage ks,
    // with what waits for it: the softmax, the stage (after its last reader),
    // the queries (after the segment's last S)
    auto qk = [&](int w, int ks, bool last, bool final) {
      const uint64_t dk = dk0 + ks * kTileD, dq = dq0 + w * kTileD;
#pragma unroll
      for (int a = 0; a < kAtoms; ++a)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc::mma<false>(tm + kPColS + w * 128, dq + a * kAtomD + k * 2, dk + a * kAtomD + k * 2, idesc_qk,
                         (a | k) != 0 ? 1u : 0u);
      tc::mma_commit(SFULL(w));
      tc::mbar_arrive(SFULL(w));
      if (last) tc::mma_commit(KEMPTY(ks));
      if (last && final) tc::mma_commit(QEMPTY);
    };
    while (!stop && walk.next(p, t, s)) {
      const int W = s.tiles;
      if (!wait(QFULL, qn & 1)) break;
      ++qn;
      if (!kwait()) break;
      any = true;
      if (tc::elect_one())
        for (int w = 0; w < W; ++w) qk(w, kn % kPKStages, w == W - 1, s.t1 - s.t0 == 1);
      __syncwarp();
      ++kn;
      if (!vwait(s.t0) || (s.t0 + 1 < s.t1 && !kwait())) break;
      for (int i = s.t0; i < s.t1 && !stop; ++i) {
        const bool more = i + 1 < s.t1;
        const int vs = vn % kPVStages, ks = kn % kPKStages;
        const uint64_t dv = dv0 + vs * kTileD;
        for (int w = 0; w < W; ++w) {
          if (i == s.t0 && !wait(OEMPTY(w), (on[w] & 1) ^ 1)) break;  // the last segment's O_w is read
          if (!wait(PFULL(w), pn[w] & 1)) break;
          ++pn[w];
          tc::tc_fence_after();
          if (tc::elect_one()) {
#pragma unroll
            for (int k = 0; k < kPT / 16; ++k)  // O_w += P_w V
              tc::mma_tmem_a(tm + kPColO + w * 128, tm + kPColS + w * 128 + k * 8, dv + k * ((16u * 128u) >> 4), idesc_pv,
                             (i > s.t0 || k > 0) ? 1u : 0u);
            // S_w is free: the product that reads P_w there is issued before, and MMAs run in issue order
            if (more) qk(w, ks, w == W - 1, i + 2 == s.t1);
            else tc::mma_commit(OFULL(w));
            if (w == W - 1) tc::mma_commit(VEMPTY(vs));
          }
          __syncwarp();
          if (!more) ++on[w];
          if (w == 0) {  // what the next tile needs is awaited under the other query tile's softmax
            ++vn;
            if (more) {
              ++kn;
              if (!vwait(i + 1) || (i + 2 < s.t1 && !kwait())) break;
            }
          }
        }
      }
    }
    if (stop && lane == 0) {
      *abort_flag = 1;
      flag_status(p.status, DSA_DEV_TIMEOUT);
    }
    if (any) {  // every MMA issued here has completed before tensor memory is freed
      if (tc::elect_one()) {
        tc::mma_commit(DONE);
        tc::mbar_wait(DONE, 0, nullptr, kPWaitBudget);
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ========================================================== softmax
    const int idx = warp - 4, w = idx >> 2, quarter = warp & 3;
    const int q = quarter * 32 + lane;  // this thread's query of tile w
    const int j = q / G, hh = q - j * G;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t colS = tmem + lane_off + kPColS + w * 128, colO = tmem + lane_off + kPColO + w * 128;
    const float c = p.sm_scale_log2;
    const uint64_t c2 = pack2(c, c);
    const int npg = kPT >> p.page_shift;
    const uint32_t ok_all = low_bits(npg);
    uint8_t *stage = sb + lay.off_stage + idx * kStageB;
    int kn = 0, sn = 0, on = 0;  // K tiles (of the CTA), S tiles and segments taken
    bool stop = false;
    int2 tail = make_int2(-1, 0);
    auto wait = [&](uint32_t bar, int parity) {
      if (!pwarp_wait(bar, static_cast<uint32_t>(parity), abort_flag)) {
        if (lane == 0) { *abort_flag = 1; flag_status(p.status, DSA_DEV_TIMEOUT); }
        stop = true;
      }
      return !stop;
    };
    // the next segment with rows of this query tile, its row's length
    bool mine = false;
    int row = 0, L = 0;
    auto take = [&] {
      while (walk.next(p, t, s)) {
        if (!s.ends) {
          // the shares of its last and its first tile
          const int last = shares.of(s.cost0 + segment_cost(s.span.n, s.tiles) - s.tiles);
          tail = s.begins ? make_int2(s.id, last) : tail_inside(s.id, shares.of(s.cost0 + kSegCost * s.tiles), last);
        }
        if (w < s.tiles) {
          const int in_chunk = w * RT + j;
          mine = j < RT && in_chunk < s.c.rows;
          row = s.c.first + in_chunk;
          // queries past the chunk's rows take no mask (and are not written): they do not slow their warp
          L = mine ? p.row_len[row] : 0x7FFFFFFF;
          return true;
        }
        kn += s.t1 - s.t0;
      }
      return false;
    };
    bool have = take();
    while (have && !stop) {
      const int sink_end = p.window > 0 ? min(p.sinks, L) : 0, lo = p.window > 0 && mine ? max(0, L - p.window) : 0;
      float m = -INFINITY, l = 0.f;
      for (int i = s.t0; i < s.t1; ++i, ++kn) {
        // a tile of pages that follow one another and that every query of the
        // warp sees whole needs no mask
        const int page0 = i * npg, t0 = s.span.page(page0) << p.page_shift;
        const bool run = page0 >= s.span.ns || page0 + npg <= s.span.ns;
        const bool whole =
            __all_sync(0xFFFFFFFFu, run && t0 + kPT <= L && (t0 >= lo || t0 + kPT <= sink_end));
        if (!wait(SFULL(w), sn & 1)) break;
        ++sn;
        tc::tc_fence_after();
        uint32_t v[4][32];
#pragma unroll
        for (int e = 0; e < 4; ++e) tc::tmem_ld32_nowait(colS + 32 * e, v[e]);
        const uint32_t okb = ok_s[kn % kPOk];
        tc::tmem_wait_ld32(v[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) tc::tmem_fence_regs32(v[e]);
        if (!whole || okb != ok_all) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // the word's first position, and at 16-token pages its second half's
            const int b = (s.span.page(page0 + ((32 * e) >> p.page_shift)) << p.page_shift) + ((32 * e) & (p.page_size - 1));
            const int b2 = p.page_shift == 4 ? (s.span.page(page0 + 2 * e + 1) - 1) << 4 : b;
            auto sees = [&](int at) { return low_bits(L - at) & (~low_bits(lo - at) | low_bits(sink_end - at)); };
            uint32_t see = (sees(b) & 0x0000FFFFu) | (sees(b2) & 0xFFFF0000u);
            const uint32_t pages = okb >> ((32 * e) >> p.page_shift);
            if (p.page_shift == 4)
              see &= (pages & 1u ? 0x0000FFFFu : 0u) | (pages & 2u ? 0xFFFF0000u : 0u);
            else if (!(pages & 1u))
              see = 0u;
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!((see >> k) & 1u)) v[e][k] = 0xFF800000u;  // -inf
          }
        }
        float mx[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t *x = v[e >> 1] + 16 * (e & 1);
          mx[e] = max3(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]));
#pragma unroll
          for (int k = 3; k + 1 < 16; k += 2) mx[e] = max3(mx[e], __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
          mx[e] = fmaxf(mx[e], __uint_as_float(x[15]));
        }
        const float mn = fmaxf(max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), mx[6]), mx[7]) * c;  // c > 0
        float alpha = 1.f;
        if (m == -INFINITY) {
          m = mn;  // the first finite score: O_w holds no share of this row yet
        } else if (mn > m + 8.f) {
          alpha = ex2(m - mn);
          l *= alpha;
          m = mn;
        }
        if (__any_sync(0xFFFFFFFFu, alpha != 1.f)) {
          // O_w += P V of the tile before was issued before this S_w and has completed with it
#pragma unroll 1
          for (int d0 = 0; d0 < D; d0 += 16) {
            float o[16];
            tc::tmem_ld16_sync(colO + d0, o);
            uint32_t ob[16];
#pragma unroll
            for (int d = 0; d < 16; ++d) ob[d] = __float_as_uint(o[d] * alpha);
            tc::tmem_st16(colO + d0, ob);
          }
        }
        const float mb = m == -INFINITY ? 0.f : -m;
        const uint64_t mb2 = pack2(mb, mb);
        uint64_t la[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float p0, p1;
            unpack2(fma2(pack2u(v[e][2 * k], v[e][2 * k + 1]), c2, mb2), p0, p1);
            p0 = ex2(p0);
            p1 = ex2(p1);
            la[k & 1] = add2(la[k & 1], pack2(p0, p1));
            const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
            pk[k] = *reinterpret_cast<const uint32_t *>(&h);
          }
          tc::tmem_st16(colS + 16 * e, pk);
        }
        tc::tmem_st_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(PFULL(w));
        float l0, l1;
        unpack2(add2(la[0], la[1]), l0, l1);
        l += l0 + l1;
      }
      if (stop) break;
      // ---- the segment's state of this query.  What does not need O_w, and
      // the next segment's start, is worked out while the last product runs.
      const bool done = s.begins && s.ends, to_me = mine;
      const float inv = l == 0.f ? 0.f : done ? 1.f / l : 1.f;  // no finite score: O_w holds zeros times V
      const int at_row = row;
      const size_t rh = static_cast<size_t>(row) * Hq + s.g * G + hh;
      const size_t part = (static_cast<size_t>(me) * 2 + (s.begins ? 1 : 0)) * 256 + w * 128 + q;
      char *to = done ? reinterpret_cast<char *>(p.out) + rh * D * 2 : reinterpret_cast<char *>(t.part_o) + part * D * 4;
      const long long place = to_me ? reinterpret_cast<long long>(to) : 0;
      if (to_me) {
        if (!done) t.part_ml[part] = make_float2(m, l);
        else if (p.lse != nullptr) p.lse[rh] = l != 0.f ? m * kLn2D + logf(l) : -INFINITY;
      }
      have = take();
      if (!wait(OFULL(w), on & 1)) break;
      ++on;
      tc::tc_fence_after();
      float zero = 0.f;  // becomes NaN with any output that is not finite
#pragma unroll 1
      for (int d0 = 0; d0 < D; d0 += 64) {
        uint32_t o[2][32];
        tc::tmem_ld32_nowait(colO + d0, o[0]);
        tc::tmem_ld32_nowait(colO + d0 + 32, o[1]);
        tc::tmem_wait_ld32(o[0]);
        tc::tmem_fence_regs32(o[1]);
        if (d0 + 64 == D) {  // O_w is in registers
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(OEMPTY(w));
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int d = 0; d < 32; ++d) {
            const float x = __uint_as_float(o[e][d]);
            zero = fmaf(x, 0.f, zero);
            o[e][d] = __float_as_uint(x * inv);
          }
        // through the staging, 128 bytes a row at a time (64 elements as
        // bf16, 32 as fp32), so that a store covers whole lines
        const int pieces = done ? 1 : 2;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (e >= pieces) break;
          uint32_t h[32];
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(o[x >> 4][2 * x & 31]),
                                                           __uint_as_float(o[x >> 4][(2 * x & 31) + 1]));
            h[x] = done ? *reinterpret_cast<const uint32_t *>(&b) : o[e][x];
          }
          __syncwarp();
#pragma unroll
          for (int x = 0; x < 8; ++x)
            *reinterpret_cast<uint4 *>(stage + lane * 128 + ((x ^ (lane & 7)) << 4)) =
                make_uint4(h[4 * x], h[4 * x + 1], h[4 * x + 2], h[4 * x + 3]);
          __syncwarp();
          const int off = (done ? d0 * 2 : d0 * 4 + 128 * e) + (lane & 7) * 16;
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const int r = 4 * x + (lane >> 3);
            const long long at = __shfl_sync(0xFFFFFFFFu, place, r);
            const uint4 b = *reinterpret_cast<const uint4 *>(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
            if (at != 0) *reinterpret_cast<uint4 *>(reinterpret_cast<char *>(at) + off) = b;
          }
        }
      }
      if (to_me && !(zero == 0.f)) atomicOr(t.redo + (at_row >> 5), 1u << (at_row & 31));
    }
    if (tid == 128) t.tail[me] = stop ? make_int2(-1, 0) : tail;
  }

  // ---- teardown: every role is out of its loop and its async work is done
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  if (warp == 1) tc::tmem_dealloc(tmem, kPTmemCols);
}

// The first CTAs take tiles, the others single rows (see the plan).
template <int D>
__global__ void __launch_bounds__(kPThreads, 1)
    dense_prompt_kernel(const DenseParams p, const DensePromptParams t, const PromptLayout lay, const DenseLayout rows,
                        const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap rkmap,
                        const __grid_constant__ CUtensorMap rvmap) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *sb = smem_raw + (base - raw);
  pdl_wait();  // the chunks come from the plan kernel
  const int c = blockIdx.x, ctas = static_cast<int>(gridDim.x), np = t.nchunks[1];
  if (c < np) {
    prompt_tiles<D>(p, t, lay, kmap, vmap, qmap, sb, base, c, np);
    if (threadIdx.x == 0) p.tail[ctas - np + c] = make_int2(-1, 0);  // no share of single rows
  } else {
    pdl_launch_dependents();
    rows_init(p, rows, rkmap, rvmap, sb, base);
    attend_rows<D, kPThreads>(p, rows, rkmap, rvmap, sb, base, c - np, ctas - np);
    if (threadIdx.x == 0) t.tail[c] = make_int2(-1, 0);
  }
}

template <int D>
cudaError_t launch_prompt(const dsa_config_t &cfg, const DenseParams &p, const DensePromptParams &t,
                          const DenseLayout &rows, size_t rows_smem, const CUtensorMap (&row_maps)[2],
                          const void *k_cache, const void *v_cache, cudaStream_t st) {
  auto encode = tensor_map_encoder();
  if (encode == nullptr) return cudaErrorNotSupported;
  constexpr uint32_t kTileB = kPT * D * 2u;
  PromptLayout lay;
  uint32_t off = 0;
  lay.off_q = off;
  off += 2 * kTileB;
  lay.off_k = off;
  off += kPKStages * kTileB;
  lay.off_v = off;
  off += kPVStages * kTileB;
  lay.off_stage = off;
  off += kSoftWarps * kStageB;
  lay.off_ok = off;
  off += kPOk * 4;
  lay.off_bar = off;
  off += (2 * (kPKStages + kPVStages) + 11) * 8;
  lay.off_cache = off = (off + 15u) & ~15u;
  off += sizeof(SegCache);
  lay.off_misc = off;
  off += 16;
  const size_t smem = std::max<size_t>(off + 1024, rows_smem);
  static_assert((2 + kPKStages + kPVStages) * kTileB + kSoftWarps * kStageB + kPOk * 4 + 32 * 8 + sizeof(SegCache) + 32 +
                        1024 <= 227 * 1024, "shared memory");
  // K and V rows as [tokens of the pool][row elements], a box = 64 elements
  // of one page's rows; queries as [R][Hq][D], a box = 64 elements of G heads
  // of one tile's rows
  const bool inter = (cfg.flags & DSA_FLAG_KV_INTERLEAVED) != 0;
  const cuuint64_t row_elems = static_cast<cuuint64_t>(cfg.num_kv_heads) * D;
  const cuuint64_t gdim[2] = {row_elems, static_cast<cuuint64_t>(cfg.num_pages) * cfg.page_size};
  const cuuint64_t gstride[1] = {row_elems * 2 * (inter ? 2 : 1)};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(cfg.page_size)};
  const cuuint32_t es[3] = {1, 1, 1};
  CUtensorMap maps[3];
  for (int kv = 0; kv < 2; ++kv)
    if (encode(&maps[kv], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(kv ? v_cache : k_cache), gdim,
               gstride, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  const cuuint32_t G = static_cast<cuuint32_t>(cfg.num_q_heads / cfg.num_kv_heads);
  const cuuint64_t qdim[3] = {D, static_cast<cuuint64_t>(cfg.num_q_heads), static_cast<cuuint64_t>(cfg.max_rows)};
  const cuuint64_t qstride[2] = {D * 2, static_cast<cuuint64_t>(cfg.num_q_heads) * D * 2};
  const cuuint32_t qbox[3] = {64, G, 128 / G};
  if (encode(&maps[2], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint8_t *>(p.q), qdim, qstride, qbox, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  auto k = dense_prompt_kernel<D>;
  static SmemLimit limit;
  cudaError_t e = allow_smem(k, static_cast<int>(smem), limit);
  if (e != cudaSuccess) return e;
  int sms = 0;
  if ((e = sm_count(&sms)) != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(std::min(sms, kDenseMaxCtas));
  if ((e = launch_pdl(dense_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, 1u, p, t, D, static_cast<int>(grid))) != cudaSuccess) return e;
  return launch_pdl(k, dim3(grid), dim3(kPThreads), smem, st, 1u, p, t, lay, rows, maps[0], maps[1], maps[2], row_maps[0],
                    row_maps[1]);
}

}  // namespace

bool dense_prompt_enabled(const dsa_config_t &cfg) {
  // a config whose rows cannot come to kLeastBytes launches no tiles
  const long long most = static_cast<long long>(cfg.max_rows) * cfg.score_width * cfg.num_kv_heads * cfg.head_dim * 4;
  return (cfg.flags & DSA_FLAG_NO_PREFILL_GROUPS) == 0 && cfg.block_rows > 1 && cfg.max_rows >= kMinRows &&
         most >= kLeastBytes;
}

cudaError_t launch_dense_prompt(const dsa_config_t &cfg, const DenseParams &p, const DensePromptParams &t,
                                const DenseLayout &rows, size_t rows_smem, const CUtensorMap (&row_maps)[2],
                                const void *k_cache, const void *v_cache, cudaStream_t st) {
  return cfg.head_dim == 128 ? launch_prompt<128>(cfg, p, t, rows, rows_smem, row_maps, k_cache, v_cache, st)
                             : launch_prompt<64>(cfg, p, t, rows, rows_smem, row_maps, k_cache, v_cache, st);
}

}  // namespace dsa
