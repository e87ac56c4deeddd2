// Attention over packed sequences with a sliding window and visible first
// tokens, and its gradient ("ultragraph -- when the graph is the 1-bit LLM, part
// 2", section "attention, as graph ops": softmax(Q K^T / sqrt(d) + mask) V).
#pragma once

#include <type_traits>

#include "attn_common.cuh"

namespace bl {

struct AttnArgs {
  const void *q, *k, *v;
  int64_t ldq, ldk, ldv, Tq, Tk;
  const int32_t *cu_q, *cu_k;
  int Hq, Hkv, D, B, max_q, max_k, window, sinks;
  float scale;
  void* out;
  float* lse;
  const void *dout, *o;
  float* delta;
  void *dq, *dk, *dv;
  int splits, split_heads;    // dK/dV: CTAs that share a key block's query heads, heads of each
  float* part;                // [splits][dK, dV][B, max_k, Hkv, D], where splits > 1
  int clear;                  // BL_CLEAR_*: outputs whose rows of no sequence become zero (lse: -inf)
  int work;                   // CTAs before those that clear
  int parts;                  // float16 row sums: CTAs of a sequence and key head
};

struct Seq {
  int q0, nq, k0, nk;
};
// The place of key j of sequence b and key head hk in the part that CTA z of those that share its
// heads takes of dK (which = 0) or dV (1).
__device__ __forceinline__ float* part_row(const AttnArgs& a, int z, int which, int b, int j, int hk) {
  const int64_t keys = int64_t(a.B) * a.max_k;
  return a.part + (((2 * z + which) * keys + int64_t(b) * a.max_k + j) * a.Hkv + hk) * a.D;
}
// Sequence b's rows; false (and the range flag) if its bounds cannot be.
__device__ __forceinline__ bool load_seq(const AttnArgs& a, int b, Seq& s, bool keys) {
  s.q0 = a.cu_q[b];
  s.k0 = a.cu_k[b];
  const int q1 = a.cu_q[b + 1], k1 = a.cu_k[b + 1];
  s.nq = q1 - s.q0;
  s.nk = k1 - s.k0;
  const bool ok = s.q0 >= 0 && s.k0 >= 0 && q1 >= s.q0 && k1 >= s.k0 && q1 <= a.Tq && k1 <= a.Tk && s.nq <= a.max_q &&
                  (!keys || s.nk <= a.max_k);
  if (!ok) raise_status(kDevRange);
  return ok;
}

// The rows that belong to no sequence: those before the first one's and behind the last one's.
struct Rest {
  int64_t lo, n;              // rows 0 .. lo - 1, and n - lo behind row lo + owned - 1
  int64_t owned;
};
__device__ __forceinline__ Rest rest_of(const int32_t* cu, int B, int64_t rows) {
  Rest r;
  r.lo = B > 0 ? min(int64_t(max(cu[0], 0)), rows) : 0;
  r.owned = B > 0 ? max(min(int64_t(cu[B]), rows), r.lo) - r.lo : 0;
  r.n = rows - r.owned;
  return r;
}
// Clears those rows of an output [rows, width] of 16-byte units; thread `at` of `all`.
__device__ __forceinline__ void clear_rows(void* out, const Rest& r, int64_t width, int64_t at, int64_t all) {
  for (int64_t i = at; i < r.n * width; i += all)
    static_cast<uint4*>(out)[i < r.lo * width ? i : i + r.owned * width] = make_uint4(0, 0, 0, 0);
}
// What is asked for of that, by the CTAs of a grid behind its first a.work ones (16-bit rows are
// whole 16-byte units).  CTAs of their own: a look at the bounds in every CTA and the registers
// it took cost the forward 5% (8192 tokens, 32/8 heads of 64: 381 -> 400 us).
__device__ __forceinline__ void clear_rest(const AttnArgs& a, int threads) {
  const int64_t at = int64_t(blockIdx.x - unsigned(a.work)) * threads + threadIdx.x;
  const int64_t all = int64_t(gridDim.x - unsigned(a.work)) * threads;
  const Rest q = rest_of(a.cu_q, a.B, a.Tq);
  if (q.n > 0) {
    const int64_t width = int64_t(a.Hq) * a.D / 8;
    if (a.clear & BL_CLEAR_OUT) clear_rows(a.out, q, width, at, all);
    if (a.clear & BL_CLEAR_DQ) clear_rows(a.dq, q, width, at, all);
    if (a.clear & BL_CLEAR_LSE)
      for (int64_t i = at; i < q.n * a.Hq; i += all) {
        const int64_t h = i / q.n, e = i - h * q.n;
        a.lse[h * a.Tq + (e < q.lo ? e : e + q.owned)] = -INFINITY;
      }
  }
  if ((a.clear & (BL_CLEAR_DK | BL_CLEAR_DV)) == 0) return;
  const Rest k = rest_of(a.cu_k, a.B, a.Tk);
  const int64_t width = int64_t(a.Hkv) * a.D / 8;
  if (a.clear & BL_CLEAR_DK) clear_rows(a.dk, k, width, at, all);
  if (a.clear & BL_CLEAR_DV) clear_rows(a.dv, k, width, at, all);
}
constexpr int kClearCtas = 32;                         // 1.8 TB/s of stores beside the work; 148 of them cost a small call 0.6 us of 8.6, these 0.35
// Alone (a.work = 0), where no other kernel does it: no sequences, or no queries.
__global__ void __launch_bounds__(256) attn_clear_kernel(const AttnArgs a) { clear_rest(a, 256); }

// Bits of the columns u of 32 with u < n.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
// Bits of the 32 columns from `first` on that are seen: u <= top and (u >= bot or u < lead).
// One word and a bit test per column instead of three comparisons.
__device__ __forceinline__ uint32_t seen_bits(int first, int top, int bot, int lead) {
  return low_bits(top + 1 - first) & (~low_bits(bot - first) | low_bits(lead - first));
}

}  // namespace bl
