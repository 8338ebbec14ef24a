// Shared by the two dense attention kernels: single rows (dense_attn.cu) and
// prompt tiles (dense_prompt.cu).
#pragma once



#include "dsa_common.cuh"
#include "tc_ptx.cuh"

namespace dsa {

constexpr float kLn2D = 0.69314718055994530942f;

// 3-D tiled load of one box into shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, int x, int y, int z, uint32_t bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
      : "memory");
}

// 2^x by the hardware's approximation (relative error about 2^-22; 2^-inf = 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// A row's length, 0 for a pad row and for one whose request or length is out
// of range (flagged).
__device__ __forceinline__ int checked_len(const DenseParams &p, int r, bool flag) {
  const int L = p.row_len[r];
  const int req = p.row_req[r];
  if (L >= 0 && L <= p.max_len && (L == 0 || (req >= 0 && req < p.max_reqs))) return L;
  if (flag) flag_status(p.status, DSA_DEV_BAD_ROW);
  return 0;
}

// U units cut into A shares, the first U % A of them one unit longer.
struct Shares {
  int A, q, rem;
  __device__ __forceinline__ Shares(int U, int ctas, int least) {
    A = min(ctas, (U + least - 1) / least);
    q = A > 0 ? U / A : 0;
    rem = U - q * A;
  }
  __device__ __forceinline__ int begin(int c) const { return c * q + min(c, rem); }
  __device__ __forceinline__ int of(int u) const {  // the share of unit u
    const int longer = rem * (q + 1);
    return u < longer ? u / (q + 1) : rem + (u - longer) / q;
  }
};

// Tail of CTA c's share, for the join: (id, last) of a row or segment that
// begins in it and goes on up to CTA `last`; (-2 - id, first | last << 16) where
// the whole share lies inside one that begins in CTA `first`; (-1, 0) else.
__device__ __forceinline__ int2 tail_inside(int id, int first, int last) { return make_int2(-2 - id, first | last << 16); }

}  // namespace dsa
