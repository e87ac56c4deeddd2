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
  float* part;                // [splits][dK, dV][Tk, Hkv, D], where splits > 1
};

struct Seq {
  int q0, nq, k0, nk;
};
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

// Bits of the columns u of 32 with u < n.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
// Bits of the 32 columns from `first` on that are seen: u <= top and (u >= bot or u < lead).
// One word and a bit test per column instead of three comparisons.
__device__ __forceinline__ uint32_t seen_bits(int first, int top, int bot, int lead) {
  return low_bits(top + 1 - first) & (~low_bits(bot - first) | low_bits(lead - first));
}

}  // namespace bl
