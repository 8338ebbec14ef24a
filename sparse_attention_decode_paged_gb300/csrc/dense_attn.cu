// Dense GQA attention over the paged K/V cache, whole prefix or sliding
// window with sinks, split over the cache's length and merged.
//
// For row r of length L a position t is visible when t < L and (no window,
// or t >= L - window, or t < sinks).  With x_t = scale q . k_t over the
// visible t: m = max x, l = sum e^(x - m), out = sum e^(x - m) v_t / l.
//
// Rows of prompts go to dense_prompt.cu's tiles when the config has more than
// one row a score block; its kernel then takes the other rows beside them, and
// the kernel here only what the tiles hand back.
//
// attend_rows (dense_rows.cuh; one persistent CTA per SM): a unit is T consecutive
// positions of one row, all KV heads; the units of all rows form one
// sequence that is cut into equal contiguous shares, one per CTA, so ragged
// lengths balance without a split count.  A row inside one share is finished
// there; a row that crosses shares leaves one partial state (m, l, O) per
// share and dense_merge_kernel joins them in share order.
//  * warp 0 (producer): for each unit two ring slots, its K and its V rows,
//    each one TMA box per page of [tokens x all heads] as 64-element columns
//    (128-byte swizzle); page ids are read a batch of 32 boxes ahead.  Pages
//    without a visible position are neither looked up nor read;
//  * warps 1..8 (consumers): warp = (KV head, group of 16 of the unit's
//    tokens).  S = Q K^T by mma.sync m16n8k16 (A: the group's <= 8 query
//    heads, B: 16 keys), softmax in the log2 domain in fp32, O^T += V^T P^T
//    with P as two bf16 terms hi + lo (their sum is p to about 2^-17).  The
//    running maximum moves only when exceeded by more than 2^8, so O is
//    rarely rescaled.
// Bound: HBM.  4 Hkv D bytes and 4 Hq D flops per position: at 8 query heads
// per KV head 8 flops a byte, far under what mma.sync sustains.  64 rows of
// 32768 keys, 8 KV heads, D = 128: 1224-1248 us, 6.9-7.0 TB/s; 16 rows of
// 1024 to 131072 keys: 632-649 us, 6.7-6.9 TB/s; 64 rows under a window of 4096:
// 162-165 us, 6.2-6.3 TB/s.  A call on two short rows takes 6.1-6.2 us: one
// launch, one CTA a row.
#include <algorithm>
#include <type_traits>

#include "dense_rows.cuh"

namespace dsa {
namespace {

template <int D>
__global__ void __launch_bounds__(kDThreads, 1)
    dense_attn_kernel(const DenseParams p, const DenseLayout lay, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *sb = smem_raw + (base - raw);
  rows_init(p, lay, kmap, vmap, sb, base);
  pdl_launch_dependents();
  pdl_wait();  // the step's rows, queries and cache may come from the kernel before
  attend_rows<D, kDThreads>(p, lay, kmap, vmap, sb, base, blockIdx.x, gridDim.x);
}

constexpr int kJoin = 4, kFewStates = 8;
struct MergeShared {
  long long rh[kJoin];  // each output's place among the (row, head) pairs, -1: not written
  float w[kDenseMaxCtas][kJoin], l[kJoin];
  float acc[8][kJoin][128];  // [warp][output][d]
};
// The partial states of what begins in CTA c0's share: c0's last and the first
// of c0 + 1, ..; state k of output i lies at (c0 + k) 2 + [k = 0] times `stride`,
// plus first + i.
struct States {
  const float2 *ml;
  const float *acc;
  int c0, n, stride, first;
  __device__ __forceinline__ size_t at(int k, int i) const {
    return (static_cast<size_t>(c0 + k) * 2 + (k == 0 ? 1 : 0)) * stride + first + i;
  }
  template <int D>
  __device__ __forceinline__ void load(int k, int i, int lane, float (&v)[D / 32]) const {
    using Vec = typename std::conditional<D == 128, float4, float2>::type;
    const Vec x = __ldcg(reinterpret_cast<const Vec *>(acc + at(k, i) * D) + lane);
    v[0] = x.x;
    v[1] = x.y;
    if constexpr (D == 128) {
      v[2] = x.z;
      v[3] = x.w;
    }
  }
};
template <int D>
__device__ __forceinline__ void store_joined(uint8_t *out, long long rh, int lane, const float *v, float l) {
  constexpr int VN = D / 32;
  const float inv = l != 0.f ? 1.f / l : 0.f;
  __nv_bfloat162 *dst = reinterpret_cast<__nv_bfloat162 *>(out) + (rh * D + lane * VN) / 2;
#pragma unroll
  for (int d = 0; d < VN; d += 2) dst[d / 2] = __floats2bfloat162_rn(v[d] * inv, v[d + 1] * inv);
}

// A block joins the at most kFewStates states of each of `outputs` outputs, in
// an order that their number alone sets (most joins: a share's end falls inside
// a row).  A warp takes 4 outputs, lane 8 j + k weighs state k of output j, and
// the states' loads are in flight together, 2 of each output at a time.  place(i)
// is output i's place among the (row, head) pairs, -1: not written.
template <int D, typename Place>
__device__ __forceinline__ void join_few(const DenseParams &p, const States &s, int outputs, Place place) {
  constexpr int VN = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = s.n;
  for (int i0 = warp * 4; i0 < outputs; i0 += 32) {
    const int k = lane & 7, i = i0 + (lane >> 3);
    float2 st = make_float2(-INFINITY, 0.f);
    if (k < n && i < outputs) st = __ldcg(s.ml + s.at(k, i));
    float mx = st.y != 0.f ? st.x : -INFINITY;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
    const float f = st.y != 0.f ? exp2f(st.x - mx) : 0.f;
    float l = st.y * f;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    const long long rh = i < outputs ? place(i) : -1;
    if (p.lse != nullptr && k == 0 && rh >= 0) p.lse[rh] = l != 0.f ? mx * kLn2D + logf(l) : -INFINITY;
    float a[4][VN];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int d = 0; d < VN; ++d) a[j][d] = 0.f;
    for (int k0 = 0; k0 < n; k0 += 2) {
      float v[4][2][VN];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (k0 + e < n && i0 + j < outputs) s.load<D>(k0 + e, i0 + j, lane, v[j][e]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float fk = __shfl_sync(0xFFFFFFFFu, f, 8 * j + ((k0 + e) & 7));
          if (k0 + e < n && i0 + j < outputs && fk != 0.f) {
#pragma unroll
            for (int d = 0; d < VN; ++d) a[j][d] = fmaf(v[j][e][d], fk, a[j][d]);
          }
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long to = __shfl_sync(0xFFFFFFFFu, rh, 8 * j);
      const float lj = __shfl_sync(0xFFFFFFFFu, l, 8 * j);
      if (to >= 0) store_joined<D>(p.out, to, lane, a[j], lj);
    }
  }
}

// The same of more states (a long row alone): the block takes J outputs at a
// time; warp i weighs output i's states, then every warp sums its k = warp,
// warp + 8, .. for all J, 4 loads in flight, and the warps' sums are added in
// order.  A function of its own, so that its registers are not the other join's
// (inlined beside it: 64 rows of up to 256 keys 20.8 us instead of 19.9).
template <int D, int J>
__device__ __noinline__ void join_many(MergeShared &sm, const States s, int outputs, uint8_t *out, float *lse) {
  constexpr int VN = D / 32, KU = 4 / J;  // KU states in flight a warp, of J outputs each
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = s.n;
  for (int i0 = 0; i0 < outputs; i0 += J) {
    const int m = min(J, outputs - i0);
    if (warp < m) {
      constexpr int kEach = kDenseMaxCtas / 32;  // states a lane
      float2 v[kEach];
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const int k = lane + 32 * e;
        v[e] = k < n ? __ldcg(s.ml + s.at(k, i0 + warp)) : make_float2(-INFINITY, 0.f);
      }
      float mx = -INFINITY, l = 0.f;
#pragma unroll
      for (int e = 0; e < kEach; ++e)
        if (v[e].y != 0.f) mx = fmaxf(mx, v[e].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const float f = v[e].y != 0.f ? exp2f(v[e].x - mx) : 0.f;
        sm.w[lane + 32 * e][warp] = f;
        l += v[e].y * f;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
      if (lane == 0) {
        sm.l[warp] = l;
        const long long rh = sm.rh[i0 + warp];
        if (lse != nullptr && rh >= 0) lse[rh] = l != 0.f ? mx * kLn2D + logf(l) : -INFINITY;
      }
    }
    __syncthreads();
    float a[J][VN];
#pragma unroll
    for (int i = 0; i < J; ++i)
#pragma unroll
      for (int d = 0; d < VN; ++d) a[i][d] = 0.f;
    for (int k0 = warp; k0 < n; k0 += 8 * KU) {
      float v[KU][J][VN];
#pragma unroll
      for (int e = 0; e < KU; ++e)
#pragma unroll
        for (int i = 0; i < J; ++i)
          if (k0 + 8 * e < n && i < m) s.load<D>(k0 + 8 * e, i0 + i, lane, v[e][i]);
#pragma unroll
      for (int e = 0; e < KU; ++e)
#pragma unroll
        for (int i = 0; i < J; ++i)
          if (k0 + 8 * e < n && i < m) {
            const float f = sm.w[k0 + 8 * e][i];
#pragma unroll
            for (int d = 0; d < VN; ++d) a[i][d] += f != 0.f ? v[e][i][d] * f : 0.f;
          }
    }
#pragma unroll
    for (int i = 0; i < J; ++i)
#pragma unroll
      for (int d = 0; d < VN; ++d) sm.acc[warp][i][lane * VN + d] = a[i][d];
    __syncthreads();
    if (warp < m) {  // warp i: output i
      const long long rh = sm.rh[i0 + warp];
      float v[VN];
#pragma unroll
      for (int d = 0; d < VN; ++d) {
        v[d] = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) v[d] += sm.acc[w][warp][lane * VN + d];
      }
      if (rh >= 0) store_joined<D>(out, rh, lane, v, sm.l[warp]);
    }
    __syncthreads();
  }
}

// Joins the partial states of what crosses shares; block (c, y) takes what
// begins in CTA c's share and goes on: 4 heads of a row, or (kPrompt, the first
// kPromptBlocks blocks of a CTA) 32 of a prompt segment's 256 queries.  What has
// more than kFewStates states is shared with the next CTAs' blocks, which lie
// inside it and have nothing of their own: a head a block, or 4 queries (one
// row of 32768 keys, 64 heads: join 20.3 -> 10.4 us, call 38.8 -> 33.5).
constexpr int kPromptBlocks = 8;

// What block c joins, as which of the CTAs in it: its own tail, or one that it
// lies inside of (see tail_inside).
__device__ __forceinline__ bool join_task(int2 tail, int c, int &id, int &c0, int &n) {
  if (tail.x == -1) return false;
  const bool inside = tail.x < 0;
  id = inside ? -2 - tail.x : tail.x;
  c0 = inside ? tail.y & 0xFFFF : c;
  n = (inside ? tail.y >> 16 : tail.y) - c0 + 1;
  return !inside || n > kFewStates;
}

template <int D, bool kPrompt>
__global__ void __launch_bounds__(256, 4) dense_merge_kernel(const DenseParams p, const DensePromptParams t) {
  __shared__ MergeShared sm;
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x, Hq = p.num_q_heads, y = static_cast<int>(blockIdx.y) - (kPrompt ? kPromptBlocks : 0);
  int id, c0, n;
  if (y >= 0) {
    if (!join_task(p.tail[c], c, id, c0, n)) return;
    const int h0 = y * kJoin;
    if (n <= kFewStates) {
      join_few<D>(p, States{p.part_ml, p.part_o, c0, n, Hq, h0}, min(kJoin, Hq - h0),
                  [&](int i) { return static_cast<long long>(id) * Hq + h0 + i; });
    } else if (c - c0 < kJoin && h0 + c - c0 < Hq) {
      const int h = h0 + c - c0;
      if (threadIdx.x == 0) sm.rh[0] = static_cast<long long>(id) * Hq + h;
      __syncthreads();
      join_many<D, 1>(sm, States{p.part_ml, p.part_o, c0, n, Hq, h}, 1, p.out, p.lse);
    }
  } else if constexpr (kPrompt) {
    if (!join_task(t.tail[c], c, id, c0, n)) return;
    const int Hkv = p.num_kv_heads, G = Hq / Hkv, RT = 128 / G, g = id % Hkv;
    const DenseChunk ch = t.chunks[id / Hkv];
    constexpr int kEach = 256 / kPromptBlocks;
    auto place = [&](int q) {  // no row's query, or a row that is done again: -1
      const int j = (q & 127) / G, in_chunk = (q >> 7) * RT + j, row = ch.first + in_chunk;
      if (j >= RT || in_chunk >= ch.rows || ((__ldcg(t.redo + (row >> 5)) >> (row & 31)) & 1u)) return -1LL;
      return static_cast<long long>(row) * Hq + g * G + (q & 127) - j * G;
    };
    const int q0 = static_cast<int>(blockIdx.y) * kEach;
    if (n <= kFewStates) {
      join_few<D>(p, States{t.part_ml, t.part_o, c0, n, 256, q0}, kEach, [&](int i) { return place(q0 + i); });
    } else if (c - c0 < kEach / kJoin) {
      const int q = q0 + (c - c0) * kJoin;
      if (threadIdx.x < kJoin) sm.rh[threadIdx.x] = place(q + threadIdx.x);
      __syncthreads();
      join_many<D, kJoin>(sm, States{t.part_ml, t.part_o, c0, n, 256, q}, kJoin, p.out, p.lse);
    }
  }
}

template <int D>
cudaError_t launch_dense(const dsa_config_t &cfg, const DenseParams &p, const DensePromptParams &t,
                         const void *k_cache, const void *v_cache, cudaStream_t st) {
  DenseLayout lay;
  const bool tiles = p.alone != nullptr;
  const size_t smem = rows_layout(cfg, tiles, lay);
  CUtensorMap maps[2];
  cudaError_t e = rows_maps(cfg, lay, k_cache, v_cache, maps);
  if (e != cudaSuccess) return e;
  auto k = dense_attn_kernel<D>;
  static SmemLimit limit;
  if ((e = allow_smem(k, static_cast<int>(smem), limit)) != cudaSuccess) return e;
  int sms = 0;
  if ((e = sm_count(&sms)) != cudaSuccess) return e;
  const unsigned grid = static_cast<unsigned>(std::min(sms, kDenseMaxCtas));
  const unsigned hy = lay.whole ? 0u : static_cast<unsigned>((cfg.num_q_heads + kJoin - 1) / kJoin);
  if (!tiles) {
    e = launch_pdl(k, dim3(grid), dim3(kDThreads), smem, st, 1u, p, lay, maps[0], maps[1]);
    if (e != cudaSuccess || hy == 0) return e;
    return launch_pdl(dense_merge_kernel<D, false>, dim3(grid, hy), dim3(256), 0, st, 1u, p, t);
  }
  if ((e = launch_dense_prompt(cfg, p, t, lay, smem, maps, k_cache, v_cache, st)) != cudaSuccess) return e;
  e = launch_pdl(dense_merge_kernel<D, true>, dim3(grid, kPromptBlocks + hy), dim3(256), 0, st, 1u, p, t);
  if (e != cudaSuccess) return e;
  // the rows that the tiles handed back, each by one CTA
  DenseParams again = p;
  again.alone = t.redo;
  again.empty = nullptr;
  lay.whole = 1;
  return launch_pdl(k, dim3(grid), dim3(kDThreads), smem, st, 1u, again, lay, maps[0], maps[1]);
}

}  // namespace

cudaError_t launch_dense_attn(const dsa_config_t &cfg, const DenseParams &p, const DensePromptParams &t,
                              const void *k_cache, const void *v_cache, cudaStream_t st) {
  return cfg.head_dim == 128 ? launch_dense<128>(cfg, p, t, k_cache, v_cache, st)
                             : launch_dense<64>(cfg, p, t, k_cache, v_cache, st);
}

}  // namespace dsa
