// Dense attention of single rows (the mathematics: dense_attn.cu) as a
// function of a CTA: a kernel of its own, and one of the two roles of a kernel
// that has prompt tiles beside it (dense_prompt.cu).
#pragma once

#include <algorithm>

#include "dense_common.cuh"

namespace dsa {

constexpr int kDWarps = 8;                        // consumer warps
constexpr int kDThreads = 32 * (1 + kDWarps);
constexpr int kDMaxSlots = 16;
constexpr long long kDWaitBudget = 2000000000LL;  // SM cycles (about 1 s)

struct DenseLayout {
  int T, tg;         // positions per unit, groups of 16 of them (T = 16 tg)
  int box_rows;      // positions per TMA box (one page's share of a unit)
  int slots;         // ring slots (a unit takes two: K, V)
  int whole;         // 1: no row is shared between CTAs
  uint32_t slot_bytes, off_pf, off_empty, off_list, off_rows, off_xch, off_ok, off_bar, off_misc;
};

// (x0, x1) as two bf16x2 terms hi + lo, their sum the pair to about 2^-17.
__device__ __forceinline__ void split2(float x0, float x1, uint32_t &hi, uint32_t &lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
  const float2 hf = __bfloat1622float2(h);
  const __nv_bfloat162 r = __floats2bfloat162_rn(x0 - hf.x, x1 - hf.y);
  hi = *reinterpret_cast<const uint32_t *>(&h);
  lo = *reinterpret_cast<const uint32_t *>(&r);
}

// The units of a row of length L: [0, ns) cover its sinks, the rest start at
// position unit w0 (of T positions) and end with the row.
struct RowSpan {
  int L, sink_end, lo;  // visible: [0, sink_end) and [lo, L)
  int ns, w0, n;        // n units
  __device__ __forceinline__ int base(int i, int T) const { return (i < ns ? i : i - ns + w0) * T; }
  __device__ __forceinline__ bool sees(int t) const { return t < L && (t >= lo || t < sink_end); }
  __device__ __forceinline__ bool sees_all(int a, int b) const { return b <= L && (a >= lo || b <= sink_end); }
  __device__ __forceinline__ bool sees_any(int a, int b) const { return a < sink_end || (a < L && b > lo); }
};
__device__ __forceinline__ RowSpan row_span(const DenseParams &p, int L, int T) {
  RowSpan s;
  s.L = L;
  s.lo = p.window > 0 ? max(0, L - p.window) : 0;
  s.sink_end = p.window > 0 ? min(p.sinks, L) : 0;
  s.ns = (s.sink_end + T - 1) / T;
  s.w0 = max(s.ns, s.lo / T);
  s.n = s.ns + (L + T - 1) / T - s.w0;
  return s;
}
__device__ __forceinline__ int find_row(const int *pf, int rows, int u) {
  int lo = 0, hi = rows;  // pf[lo] <= u < pf[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pf[mid] <= u) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ bool dwarp_wait(uint32_t bar, uint32_t parity, const volatile int *abort_flag) {
  const bool ok = tc::mbar_wait(bar, parity, abort_flag, kDWaitBudget);
  return __all_sync(0xFFFFFFFFu, ok);
}
__device__ __forceinline__ void consumer_barrier() {
  asm volatile("bar.sync 1, %0;\n" ::"n"(kDWarps * 32) : "memory");
}
// The same, true for every warp if `v` is true for one.
__device__ __forceinline__ bool consumer_barrier_any(bool v) {
  uint32_t any;
  asm volatile(
      "{\n .reg .pred a, b;\n setp.ne.b32 a, %1, 0;\n bar.red.or.pred b, 1, %2, a;\n selp.b32 %0, 1, 0, b;\n}\n"
      : "=r"(any)
      : "r"(v ? 1u : 0u), "n"(kDWarps * 32)
      : "memory");
  return any != 0;
}

// Units per CTA at least: shorter shares read faster and leave more states to
// join (with 4, one row of 1024 keys, 8 KV heads, takes 12.7 us instead of 11.4
// and 4 rows of 2048, 2 KV heads, 14.0 instead of 11.9; one row of 4096 keys 14.5
// instead of 14.9).
constexpr int kMinShare = 2;
constexpr int kRowsHere = 1024;                                // rows whose length and request are kept on chip
// Rows of at most this many bytes of K and V are never shared: no merge (with
// a limit of 1 MB, 8 rows of 256 keys and 8 KV heads take 17.9 us, not 13.6).
constexpr int kWholeBytes = 256 * 1024;

// The barriers of a CTA's ring; a block-wide barrier before they are used.
__device__ __forceinline__ void rows_init(const DenseParams &p, const DenseLayout &lay, const CUtensorMap &kmap,
                                          const CUtensorMap &vmap, uint8_t *sb, uint32_t base) {
  if (threadIdx.x == 0) {
    const int NS = lay.slots;
    const uint32_t bar0 = base + lay.off_bar;
    for (int s = 0; s < NS; ++s) {
      tc::mbar_init(bar0 + 8u * s, 1);
      tc::mbar_init(bar0 + 8u * (NS + s), static_cast<uint32_t>(p.num_kv_heads * lay.tg));
    }
    *reinterpret_cast<int *>(sb + lay.off_misc) = 0;
    tc::fence_mbar_init();
    tc::tma_prefetch_desc(&kmap);
    tc::tma_prefetch_desc(&vmap);
  }
}

// CTA `me` of `ctas`, NT threads each (9 warps work), over the rows that
// p.alone lists (null: all).  Called by every thread, after rows_init.
template <int D, int NT>
__device__ __forceinline__ void attend_rows(const DenseParams &p, const DenseLayout &lay, const CUtensorMap &kmap,
                                            const CUtensorMap &vmap, uint8_t *sb, uint32_t base, int me, int ctas) {
  constexpr int kIters = (4096 + NT - 1) / NT;  // max_rows <= 4096
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int T = lay.T, NS = lay.slots;
  const int Hq = p.num_q_heads, Hkv = p.num_kv_heads, G = Hq / Hkv;
  int *pf = reinterpret_cast<int *>(sb + lay.off_pf);            // [R + 1] units before each row
  uint32_t *ok_s = reinterpret_cast<uint32_t *>(sb + lay.off_ok);  // [slots] boxes loaded, a bit each
  const uint32_t bar0 = base + lay.off_bar;
  auto FULL = [&](int s) { return bar0 + 8u * s; };
  auto EMPTY = [&](int s) { return bar0 + 8u * (NS + s); };
  int *misc = reinterpret_cast<int *>(sb + lay.off_misc);  // [0] abort, [1..] scan scratch
  volatile int *abort_flag = misc;

  // the rows this kernel takes: all, or those that no prompt tile has, listed
  // in order from their bits
  const bool listed = p.alone != nullptr;
  uint32_t *empty = reinterpret_cast<uint32_t *>(sb + lay.off_empty);  // a bit a row: without a visible position
  uint16_t *list = reinterpret_cast<uint16_t *>(sb + lay.off_list);  // [R]
  int R = p.max_rows;
  if (listed) {
    uint32_t bits = 0u;
    if (tid < (R + 31) / 32) {  // 128 words at most: warps 0 .. 3
      bits = __ldcg(p.alone + tid);
      empty[tid] = p.empty != nullptr ? __ldcg(p.empty + tid) : 0u;
    }
    int inc = __popc(bits);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) misc[1 + warp] = inc;
    __syncthreads();
    int at = inc - __popc(bits);
    R = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      at += w < warp ? misc[1 + w] : 0;
      R += misc[1 + w];
    }
    for (; bits != 0u; bits &= bits - 1) list[at++] = static_cast<uint16_t>(tid * 32 + __ffs(static_cast<int>(bits)) - 1);
    __syncthreads();
    if (R == 0 && p.empty == nullptr) return;  // nothing to do again
  }
  auto row_id = [&](int i) { return listed ? static_cast<int>(list[i]) : i; };
  // units before each row: counted row by row with all rows' loads in flight,
  // then thread t sums its rows [t * per, (t + 1) * per)
  int2 *row_s = reinterpret_cast<int2 *>(sb + lay.off_rows);           // [R] length, request (R <= kRowsHere)
  auto count_row = [&](int i, int L, int req) {
    const bool bad = L < 0 || L > p.max_len || (L > 0 && (req < 0 || req >= p.max_reqs));
    if (bad && me == 0) flag_status(p.status, DSA_DEV_BAD_ROW);
    const int len = bad ? 0 : L, n = row_span(p, len, T).n;
    if (i < R) {
      pf[i] = n;
      if (R <= kRowsHere) row_s[i] = make_int2(len, req);
    }
    const uint32_t none = __ballot_sync(0xFFFFFFFFu, i < R && n == 0);
    if (lane == 0 && i < R && !listed) empty[i >> 5] = none;
  };
  auto load_row = [&](int i, int &L, int &req) {
    const int r = i < R ? row_id(i) : 0;
    L = i < R ? p.row_len[r] : 0;
    req = i < R ? p.row_req[r] : 0;
  };
  if (R <= NT) {  // one row a thread: little code to fetch where the call is short
    int L, req;
    load_row(tid, L, req);
    count_row(tid, L, req);
  } else {
    int L[kIters], req[kIters];
#pragma unroll
    for (int e = 0; e < kIters; ++e) load_row(e * NT + tid, L[e], req[e]);
#pragma unroll
    for (int e = 0; e < kIters; ++e)
      if (e * NT < R) count_row(e * NT + tid, L[e], req[e]);
  }
  // the sum before this thread's rows: one row a thread where they suffice
  const int per = R <= NT ? 1 : (R + NT - 1) / NT;
  const int first_row = min(R, tid * per), last_row = min(R, first_row + per);
  if (per > 1) __syncthreads();
  {
    int sum = 0;
    for (int r = first_row; r < last_row; ++r) sum += pf[r];
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) misc[1 + warp] = inc;
    __syncthreads();
    int before = inc - sum;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) before += w < warp ? misc[1 + w] : 0;
    for (int r = first_row; r < last_row; ++r) {
      const int n = pf[r];
      pf[r] = before;
      before += n;
    }
    if (last_row == R && (first_row < last_row || (R == 0 && tid == 0))) pf[R] = before;
  }
  __syncthreads();
  const int U = pf[R];
  const Shares shares(U, ctas, lay.whole ? 1 : kMinShare);
  // where a share begins: anywhere, or (whole rows) at the next row's first unit
  auto begin_of = [&](int c) {
    const int u = shares.begin(c);
    if (!lay.whole || u >= U) return u;
    const int r = find_row(pf, R, u);
    return pf[r] == u ? u : pf[r + 1];
  };
  const int u0 = me < shares.A ? begin_of(me) : 0, u1 = me < shares.A ? begin_of(me + 1) : 0;
  // length (0 where it was refused above) and request of the i-th row
  auto row_at = [&](int i) {
    return R <= kRowsHere ? row_s[i] : make_int2(checked_len(p, row_id(i), false), p.row_req[row_id(i)]);
  };

  if (warp == 0) {
    // ====================================================== producer
    const uint64_t policy = tc::l2_evict_first_policy();
    const int BR = lay.box_rows, nbox = T / BR, UB = 32 / nbox;  // units per batch of 32 boxes
    const uint32_t box_bytes = static_cast<uint32_t>(BR) * Hkv * D * 2;
    // this lane's box of the batch that starts with unit ub: first cache row,
    // -1 for none (no visible position, or a page outside the pool)
    auto lookup = [&](int ub) {
      const int u = ub + lane / nbox;
      if (lane >= UB * nbox || u >= u1) return -1LL;
      const int r = find_row(pf, R, u);
      const int2 row = row_at(r);
      const RowSpan s = row_span(p, row.x, T);
      const int t = s.base(u - pf[r], T) + (lane % nbox) * BR;
      if (!s.sees_any(t, t + BR)) return -1LL;
      const int pg = p.page_table[static_cast<size_t>(row.y) * p.max_pages_per_req + (t >> p.page_shift)];
      if (pg < 0 || pg >= p.num_pages) {
        flag_status(p.status, DSA_DEV_BAD_PAGE);
        return -1LL;
      }
      return static_cast<long long>(pg) * p.page_size + (t & (p.page_size - 1));
    };
    int slot = 0, phase = 0, issued = 0;
    bool stop = false;
    long long cur = lookup(u0);
    for (int ub = u0; ub < u1 && !stop; ub += UB) {
      const long long next = lookup(ub + UB);
      for (int i = 0; i < UB && ub + i < u1 && !stop; ++i) {
        const bool mine = lane / nbox == i && cur >= 0;
        const uint32_t have = __ballot_sync(0xFFFFFFFFu, mine);
        const uint32_t bits = have >> (i * nbox);
        for (int kv = 0; kv < 2; ++kv) {
          if (!dwarp_wait(EMPTY(slot), phase ^ 1, abort_flag)) {
            if (lane == 0) { *abort_flag = 1; flag_status(p.status, DSA_DEV_TIMEOUT); }
            stop = true;
            break;
          }
          if (lane == 0) {
            ok_s[slot] = bits;
            tc::mbar_arrive_expect_tx(FULL(slot), static_cast<uint32_t>(__popc(have)) * box_bytes);
          }
          __syncwarp();
          if (mine)
            tma_load_3d(base + slot * lay.slot_bytes + (lane % nbox) * box_bytes, kv ? &vmap : &kmap, 0,
                        static_cast<int>(cur), 0, FULL(slot), policy);
          ++issued;
          if (++slot == NS) { slot = 0; phase ^= 1; }
        }
      }
      cur = next;
    }
    // no copy may land after the CTA exits
    if (lane == 0)
      for (int c = max(0, issued - NS); c < issued; ++c)
        tc::mbar_wait(FULL(c % NS), (c / NS) & 1, nullptr, kDWaitBudget);
    __syncwarp();
  } else if (warp <= kDWarps) {
    // ===================================================== consumers
    const int cw = warp - 1, g = cw % Hkv, tg = cw / Hkv;  // KV head, token group
    const bool works = tg < lay.tg;
    const int c4 = lane & 3, g4 = lane >> 2;  // g4: query head of the KV group
    const int mat = lane >> 3, mrow = (lane & 7) + (mat >> 1) * 8;  // this lane's ldmatrix row (token)
    // byte offset in a slot of this lane's ldmatrix row, 16-byte chunk (mat & 1)
    const int BR = lay.box_rows, tok0 = tg * 16;
    const uint32_t atom = static_cast<uint32_t>(BR) * 128u;  // one 64-element column of a box
    const uint32_t lane_off = static_cast<uint32_t>(tok0 / BR) * (atom * (Hkv * D / 64)) + g * (D / 64) * atom +
                              static_cast<uint32_t>(tok0 % BR + mrow) * 128u +
                              static_cast<uint32_t>(((mat & 1) ^ (mrow & 7)) << 4);
    float *xch = reinterpret_cast<float *>(sb + lay.off_xch);  // token groups' states
    const float c = p.sm_scale_log2;
    int slot = 0, phase = 0;
    bool aborted = false;
    int2 tail = make_int2(-1, 0);

    // pad rows, and refused ones: empty outputs; a word of rows without any is
    // passed over at once, which counts where few CTAs take all the rows
    for (int r = me; r < p.max_rows;) {
      const uint32_t ahead = empty[r >> 5] >> (r & 31);
      if (ahead & 1u) {
        __nv_bfloat162 *dst = reinterpret_cast<__nv_bfloat162 *>(p.out) + static_cast<size_t>(r) * Hq * D / 2;
        for (int i = tid - 32; i < Hq * D / 2; i += kDWarps * 32) dst[i] = __floats2bfloat162_rn(0.f, 0.f);
        if (p.lse != nullptr)
          for (int i = tid - 32; i < Hq; i += kDWarps * 32) p.lse[static_cast<size_t>(r) * Hq + i] = -INFINITY;
      }
      r += ahead != 0u || ctas >= 32 ? ctas : (32 - (r & 31) + ctas - 1) / ctas * ctas;
    }

    int i = u0 < u1 ? find_row(pf, R, u0) : 0;
    const int first_i = i;
    for (int u = u0; u < u1 && !aborted;) {
      while (pf[i + 1] <= u) ++i;  // the row of unit u
      const RowSpan s = row_span(p, row_at(i).x, T);
      const int r = row_id(i), uend = min(u1, pf[i + 1]);
      uint32_t qa[D / 16][2];
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        qa[ks][0] = qa[ks][1] = 0u;
        if (works && g4 < G) {
          const uint8_t *qrow = p.q + ((static_cast<size_t>(r) * Hq + g * G + g4) * D + ks * 16 + 2 * c4) * 2;
          qa[ks][0] = *reinterpret_cast<const uint32_t *>(qrow);
          qa[ks][1] = *reinterpret_cast<const uint32_t *>(qrow + 16);
        }
      }
      float m = -INFINITY, l = 0.f;  // head g4, log2 domain; l: this lane's keys
      float o[D / 16][4];            // O^T: dims 16 mt + g4 (+8), heads 2 c4, 2 c4 + 1
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
      const int first = u;
      for (; works && u < uend; ++u) {
        const int t0 = s.base(u - pf[i], T) + tok0;
        // ---- S = Q K^T of 16 keys
        if (!dwarp_wait(FULL(slot), phase, abort_flag)) { aborted = true; break; }
        const bool box = (ok_s[slot] >> (tok0 / BR)) & 1u;
        const bool any = box && s.sees_any(t0, t0 + 16);
        float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb4[4] = {0.f, 0.f, 0.f, 0.f};
        if (any) {
          const uint32_t ka = base + slot * lay.slot_bytes + lane_off;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t b0, b1, b2, b3;
            ldmatrix_x4((ka ^ ((ks & 3) << 5)) + (ks >> 2) * atom, b0, b1, b2, b3);
            mma_bf16_16816(sa, qa[ks][0], 0u, qa[ks][1], 0u, b0, b1);
            mma_bf16_16816(sb4, qa[ks][0], 0u, qa[ks][1], 0u, b2, b3);
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(EMPTY(slot));
        if (++slot == NS) { slot = 0; phase ^= 1; }
        // ---- softmax; this lane's keys t0 + 2 c4, + 1, + 8, + 9
        float x0 = sa[0] * c, x1 = sa[1] * c, x2 = sb4[0] * c, x3 = sb4[1] * c;
        const bool full = box && s.sees_all(t0, t0 + 16);
        uint32_t vm0 = 0xFFFFFFFFu, vm1 = 0xFFFFFFFFu;  // V rows of keys that are not visible are zeroed
        if (any && !full) {
          const int t = t0 + 2 * c4;
          const bool v0 = s.sees(t), v1 = s.sees(t + 1), v2 = s.sees(t + 8), v3 = s.sees(t + 9);
          x0 = v0 ? x0 : -INFINITY;
          x1 = v1 ? x1 : -INFINITY;
          x2 = v2 ? x2 : -INFINITY;
          x3 = v3 ? x3 : -INFINITY;
          vm0 = (v0 ? 0x0000FFFFu : 0u) | (v1 ? 0xFFFF0000u : 0u);
          vm1 = (v2 ? 0x0000FFFFu : 0u) | (v3 ? 0xFFFF0000u : 0u);
        }
        uint32_t ph0 = 0u, pl0 = 0u, ph1 = 0u, pl1 = 0u;
        if (any) {
          float mx = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
          const bool move = mx > m + 8.f || (m == -INFINITY && mx > -INFINITY);
          if (__any_sync(0xFFFFFFFFu, move)) {
            const float al = move ? (m == -INFINITY ? 0.f : exp2f(m - mx)) : 1.f;
            if (move) m = mx;
            l *= al;
            const float al_a = __shfl_sync(0xFFFFFFFFu, al, 8 * c4), al_b = __shfl_sync(0xFFFFFFFFu, al, 8 * c4 + 4);
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
              o[mt][0] *= al_a;
              o[mt][1] *= al_b;
              o[mt][2] *= al_a;
              o[mt][3] *= al_b;
            }
          }
          const float mb = m == -INFINITY ? 0.f : m;  // no finite score yet: every p is 0
          const float p0 = ex2(x0 - mb), p1 = ex2(x1 - mb), p2 = ex2(x2 - mb), p3 = ex2(x3 - mb);
          l += (p0 + p1) + (p2 + p3);
          split2(p0, p1, ph0, pl0);
          split2(p2, p3, ph1, pl1);
        }
        // ---- O^T += V^T P^T
        if (!dwarp_wait(FULL(slot), phase, abort_flag)) { aborted = true; break; }
        if (any) {
          const uint32_t va = base + slot * lay.slot_bytes + lane_off;
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt) {
            uint32_t a0, a1, a2, a3;
            ldmatrix_x4_trans((va ^ ((mt & 3) << 5)) + (mt >> 2) * atom, a0, a1, a2, a3);
            a0 &= vm0;
            a1 &= vm0;
            a2 &= vm1;
            a3 &= vm1;
            mma_bf16_16816(o[mt], a0, a1, a2, a3, ph0, ph1);
            mma_bf16_16816(o[mt], a0, a1, a2, a3, pl0, pl1);
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(EMPTY(slot));
        if (++slot == NS) { slot = 0; phase ^= 1; }
      }
      u = uend;
      if (aborted && lane == 0) { *abort_flag = 1; flag_status(p.status, DSA_DEV_TIMEOUT); }
      if (lay.tg == 1 && aborted) break;
      // ---- the row's state on this CTA
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
      if (lay.tg > 1) {
        // token groups: every warp leaves (m, l, O) in shared memory, then
        // each of a KV head's warps joins them, in group order, for its share
        // of the dims and all 8 heads
        constexpr int kHead = D + 4, kState = 16 + 8 * kHead;  // 4 words of padding a head: no bank conflicts
        float *mine = xch + cw * kState;
        if (i > first_i) consumer_barrier();  // the last row's states are read
        if (works) {
          if (c4 == 0) {
            mine[g4] = m;
            mine[8 + g4] = l;
          }
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) mine[16 + (2 * c4 + (e & 1)) * kHead + 16 * mt + g4 + 8 * (e >> 1)] = o[mt][e];
        }
        // every warp leaves after the same row when one of them gave up, so none waits here alone
        aborted = consumer_barrier_any(aborted);
        if (works && !aborted) {
          // lane 4 h + j weighs head h's groups j and j + 4
          const int TG = lay.tg;
          float mk[2], lk[2], f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int k = c4 + 4 * e;
            const float *st = xch + (g + k * Hkv) * kState;
            lk[e] = k < TG ? st[8 + g4] : 0.f;
            mk[e] = lk[e] != 0.f ? st[g4] : -INFINITY;
          }
          m = fmaxf(mk[0], mk[1]);
          m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
          m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
#pragma unroll
          for (int e = 0; e < 2; ++e) f[e] = lk[e] != 0.f ? ex2(mk[e] - m) : 0.f;
          l = lk[0] * f[0] + lk[1] * f[1];
          l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
          l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
          const bool whole = first == pf[i] && uend == pf[i + 1];
          const float inv = !whole ? 1.f : l != 0.f ? 1.f / l : 0.f;
          const int sh = (D == 128 ? 7 : 6) - (TG == 8 ? 3 : TG == 4 ? 2 : 1);  // this warp's dims: 2^sh, 8 at least
          const int share = 1 << sh, d0 = tg << sh;
          const size_t rh = static_cast<size_t>(r) * Hq + g * G;
          const size_t ph = (static_cast<size_t>(me) * 2 + (first == pf[i] ? 1 : 0)) * Hq + g * G;
          for (int e = lane; e < 8 * share; e += 32) {
            const int h = e >> sh, d = d0 + (e & (share - 1));
            float v = 0.f;
#pragma unroll 4
            for (int k = 0; k < TG; ++k) {
              const float fk = __shfl_sync(0xFFFFFFFFu, (k & 4) ? f[1] : f[0], 4 * h + (k & 3));
              const float x = xch[(g + k * Hkv) * kState + 16 + h * kHead + d];
              v += fk != 0.f ? x * fk : 0.f;
            }
            v *= __shfl_sync(0xFFFFFFFFu, inv, 4 * h);
            if (h < G) {
              if (whole) reinterpret_cast<__nv_bfloat16 *>(p.out)[(rh + h) * D + d] = __float2bfloat16_rn(v);
              else p.part_o[(ph + h) * D + d] = v;
            }
          }
          if (tg == 0 && c4 == 0 && g4 < G) {
            if (!whole) p.part_ml[ph + g4] = make_float2(m, l);
            else if (p.lse != nullptr) p.lse[rh + g4] = l != 0.f ? m * kLn2D + logf(l) : -INFINITY;
          }
        }
      }
      const bool begins = first == pf[i], ends = uend == pf[i + 1];
      if (works && lay.tg == 1) {
        if (begins && ends) {  // the whole row: normalised, rounded to bf16
          const float inv = l != 0.f ? 1.f / l : 0.f;
          const float ia = __shfl_sync(0xFFFFFFFFu, inv, 8 * c4), ib = __shfl_sync(0xFFFFFFFFu, inv, 8 * c4 + 4);
          const size_t rh = static_cast<size_t>(r) * Hq + g * G;
          __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(p.out) + rh * D + g4;
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (2 * c4 + e < G) {
              const float f = e ? ib : ia;
#pragma unroll
              for (int mt = 0; mt < D / 16; ++mt) {
                dst[(2 * c4 + e) * D + 16 * mt] = __float2bfloat16_rn(o[mt][e] * f);
                dst[(2 * c4 + e) * D + 16 * mt + 8] = __float2bfloat16_rn(o[mt][2 + e] * f);
              }
            }
          if (p.lse != nullptr && c4 == 0 && g4 < G)
            p.lse[rh + g4] = l != 0.f ? m * kLn2D + logf(l) : -INFINITY;
        } else {  // this CTA's share of the row
          const size_t ph = (static_cast<size_t>(me) * 2 + (begins ? 1 : 0)) * Hq + g * G;
          if (c4 == 0 && g4 < G) p.part_ml[ph + g4] = make_float2(m, l);
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (2 * c4 + e < G) {
              float *dst = p.part_o + (ph + 2 * c4 + e) * D + g4;
#pragma unroll
              for (int mt = 0; mt < D / 16; ++mt) {
                dst[16 * mt] = o[mt][e];
                dst[16 * mt + 8] = o[mt][2 + e];
              }
            }
        }
      }
      if (!ends)
        tail = begins ? make_int2(r, shares.of(pf[i + 1] - 1))
                      : tail_inside(r, shares.of(pf[i]), shares.of(pf[i + 1] - 1));
    }
    if (tid == 32) p.tail[me] = aborted ? make_int2(-1, 0) : tail;
  }
  __syncthreads();
}

// Where a config's ring and tables lie, and the shared memory they take.
inline size_t rows_layout(const dsa_config_t &cfg, bool listed, DenseLayout &lay) {
  const int Hkv = cfg.num_kv_heads, D = cfg.head_dim;
  lay.tg = Hkv == 1 ? 8 : Hkv == 2 ? 4 : Hkv <= 4 ? 2 : 1;
  lay.T = 16 * lay.tg;
  lay.box_rows = std::min<int>(lay.T, cfg.page_size);
  lay.slot_bytes = static_cast<uint32_t>(lay.T) * Hkv * D * 2;  // a multiple of 1024: T >= 16, D >= 64
  lay.whole = static_cast<long long>((cfg.score_width + lay.T - 1) / lay.T) * 2 * lay.slot_bytes <= kWholeBytes;
  const uint32_t pf = ((static_cast<uint32_t>(cfg.max_rows) + 1) * 4 + 15u) & ~15u;
  const uint32_t empty = ((static_cast<uint32_t>(cfg.max_rows) + 31) / 32 * 4 + 15u) & ~15u;
  const uint32_t rows = (static_cast<uint32_t>(std::min(cfg.max_rows, kRowsHere)) * 8 + 15u) & ~15u;
  const uint32_t list = listed ? (static_cast<uint32_t>(cfg.max_rows) * 2 + 15u) & ~15u : 0u;
  const uint32_t xch = lay.tg > 1 ? kDWarps * (8 * (D + 4) + 16) * 4u : 0u;
  const uint32_t rest = pf + empty + rows + list + xch + kDMaxSlots * 4 + 2 * kDMaxSlots * 8 + 64 + 1024;
  constexpr uint32_t kSmem = 227 * 1024;
  lay.slots = std::min<int>(kDMaxSlots, static_cast<int>((kSmem - rest) / lay.slot_bytes));
  uint32_t off = static_cast<uint32_t>(lay.slots) * lay.slot_bytes;
  lay.off_pf = off;
  off += pf;
  lay.off_empty = off;
  off += empty;
  lay.off_list = off;
  off += list;
  lay.off_rows = off;
  off += rows;
  lay.off_xch = off;
  off += xch;
  lay.off_ok = off;
  off += kDMaxSlots * 4;
  lay.off_bar = off;
  off += 2 * kDMaxSlots * 8;
  lay.off_misc = off;
  off += 64;
  return off + 1024;
}

// Tensor maps of K and V for attend_rows.
inline cudaError_t rows_maps(const dsa_config_t &cfg, const DenseLayout &lay, const void *k_cache, const void *v_cache,
                             CUtensorMap (&maps)[2]) {
  auto encode = tensor_map_encoder();
  if (encode == nullptr) return cudaErrorNotSupported;
  const int Hkv = cfg.num_kv_heads, D = cfg.head_dim;
  // K and V as [columns of 64 elements][tokens of the pool][64]; one box is
  // box_rows tokens of one page, all columns (the interleaved cache: every
  // second row of tokens, V's columns behind K's)
  const bool inter = (cfg.flags & DSA_FLAG_KV_INTERLEAVED) != 0;
  const cuuint64_t row_bytes = static_cast<cuuint64_t>(Hkv) * D * 2;
  const cuuint64_t gdim[3] = {64, static_cast<cuuint64_t>(cfg.num_pages) * cfg.page_size,
                              static_cast<cuuint64_t>(Hkv) * D / 64};
  const cuuint64_t gstride[2] = {row_bytes * (inter ? 2 : 1), 128};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(lay.box_rows), static_cast<cuuint32_t>(Hkv * D / 64)};
  const cuuint32_t es[3] = {1, 1, 1};
  for (int kv = 0; kv < 2; ++kv) {
    void *ptr = const_cast<void *>(kv ? v_cache : k_cache);
    if (encode(&maps[kv], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, ptr, gdim, gstride, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  return cudaSuccess;
}

// Prompt tiles and single rows; rows, rows_smem, row_maps: the latter's layout,
// shared memory and tensor maps.
cudaError_t launch_dense_prompt(const dsa_config_t &cfg, const DenseParams &p, const DensePromptParams &t,
                                const DenseLayout &rows, size_t rows_smem, const CUtensorMap (&row_maps)[2],
                                const void *k_cache, const void *v_cache, cudaStream_t st);

}  // namespace dsa
