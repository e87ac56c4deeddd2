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

constexpr int kSimpleWarps = 4;

// delta = rowsum(dO O): one warp per row and head.
template <typename T>
__global__ void __launch_bounds__(128)
attn_delta_kernel(const AttnArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t r = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (r >= a.Tq * a.Hq) return;
  const T* o = static_cast<const T*>(a.o) + r * a.D;
  const T* d = static_cast<const T*>(a.dout) + r * a.D;
  float s = 0.f;
  for (int i = lane; i < a.D; i += 32) s = fmaf(to_f32(o[i]), to_f32(d[i]), s);
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if (lane == 0) a.delta[(r % a.Hq) * a.Tq + r / a.Hq] = s;
}

// dQ: one warp per query row and head.
template <typename T>
__global__ void __launch_bounds__(32 * kSimpleWarps)
attn_dq_simple_kernel(const AttnArgs a) {
  __shared__ float sq[kSimpleWarps][128], sd[kSimpleWarps][128];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Seq s;
  if (!load_seq(a, blockIdx.z, s, true)) return;
  const int i = blockIdx.x * kSimpleWarps + w, h = blockIdx.y;
  if (i >= s.nq) return;
  const int hk = h / (a.Hq / a.Hkv), p = i + s.nk - s.nq;
  const T* q = static_cast<const T*>(a.q) + int64_t(s.q0 + i) * a.ldq + int64_t(h) * a.D;
  const T* g = static_cast<const T*>(a.dout) + (int64_t(s.q0 + i) * a.Hq + h) * a.D;
  for (int d = lane; d < a.D; d += 32) {
    sq[w][d] = to_f32(q[d]);
    sd[w][d] = to_f32(g[d]);
  }
  __syncwarp();
  const float c = a.scale * kLog2e;
  const float l = a.lse[int64_t(h) * a.Tq + s.q0 + i] * kLog2e, delta = a.delta[int64_t(h) * a.Tq + s.q0 + i];
  float o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 <= p; j0 += 32) {
    const int j = j0 + lane;
    const bool see = j < s.nk && sees(p, j, a.window, a.sinks);
    if (!__any_sync(0xffffffffu, see)) continue;
    float ds = 0.f;
    if (see) {
      const T* k = static_cast<const T*>(a.k) + int64_t(s.k0 + j) * a.ldk + int64_t(hk) * a.D;
      const T* v = static_cast<const T*>(a.v) + int64_t(s.k0 + j) * a.ldv + int64_t(hk) * a.D;
      float t = 0.f, dp = 0.f;
      for (int d = 0; d < a.D; ++d) {
        t = fmaf(sq[w][d], to_f32(k[d]), t);
        dp = fmaf(sd[w][d], to_f32(v[d]), dp);
      }
      ds = exp2_approx(fmaf(t, c, -l)) * (dp - delta) * a.scale;
    }
    for (int t = 0; t < 32 && j0 + t < s.nk; ++t) {
      const float pt = __shfl_sync(0xffffffffu, ds, t);
      if (!__shfl_sync(0xffffffffu, int(see), t)) continue;
      const T* k = static_cast<const T*>(a.k) + int64_t(s.k0 + j0 + t) * a.ldk + int64_t(hk) * a.D;
      for (int u = 0; u < 4; ++u)
        if (lane + 32 * u < a.D) o[u] = fmaf(pt, to_f32(k[lane + 32 * u]), o[u]);
    }
  }
  T* out = static_cast<T*>(a.dq) + (int64_t(s.q0 + i) * a.Hq + h) * a.D;
  bool bad = false;
  for (int u = 0; u < 4; ++u)
    if (lane + 32 * u < a.D) {
      if (!(fabsf(o[u]) < INFINITY)) bad = true;
      out[lane + 32 * u] = from_f32<T>(o[u]);
    }
  if (bad) raise_status(kDevNonFinite);
}

// dK, dV: one warp per key row and key head, 32 queries a turn, the group's heads in order.
template <typename T>
__global__ void __launch_bounds__(32 * kSimpleWarps)
attn_dkv_simple_kernel(const AttnArgs a) {
  __shared__ float sk[kSimpleWarps][128], sv[kSimpleWarps][128];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Seq s;
  if (!load_seq(a, blockIdx.z, s, true)) return;
  const int j = blockIdx.x * kSimpleWarps + w, hk = blockIdx.y, group = a.Hq / a.Hkv;
  if (j >= s.nk) return;
  const T* k = static_cast<const T*>(a.k) + int64_t(s.k0 + j) * a.ldk + int64_t(hk) * a.D;
  const T* v = static_cast<const T*>(a.v) + int64_t(s.k0 + j) * a.ldv + int64_t(hk) * a.D;
  for (int d = lane; d < a.D; d += 32) {
    sk[w][d] = to_f32(k[d]);
    sv[w][d] = to_f32(v[d]);
  }
  __syncwarp();
  const float c = a.scale * kLog2e;
  const int off = s.nk - s.nq;
  float gk[4] = {0.f, 0.f, 0.f, 0.f}, gv[4] = {0.f, 0.f, 0.f, 0.f};
  for (int h = hk * group; h < (hk + 1) * group; ++h)
    for (int i0 = max(0, j - off); i0 < s.nq; i0 += 32) {
      const int i = i0 + lane;
      const bool see = i < s.nq && sees(i + off, j, a.window, a.sinks);
      if (!__any_sync(0xffffffffu, see)) continue;
      float p = 0.f, ds = 0.f;
      if (see) {
        const T* q = static_cast<const T*>(a.q) + int64_t(s.q0 + i) * a.ldq + int64_t(h) * a.D;
        const T* g = static_cast<const T*>(a.dout) + (int64_t(s.q0 + i) * a.Hq + h) * a.D;
        float t = 0.f, dp = 0.f;
        for (int d = 0; d < a.D; ++d) {
          t = fmaf(sk[w][d], to_f32(q[d]), t);
          dp = fmaf(sv[w][d], to_f32(g[d]), dp);
        }
        const int64_t r = int64_t(h) * a.Tq + s.q0 + i;
        p = exp2_approx(fmaf(t, c, -a.lse[r] * kLog2e));
        ds = p * (dp - a.delta[r]) * a.scale;
      }
      for (int t = 0; t < 32 && i0 + t < s.nq; ++t) {
        const float pt = __shfl_sync(0xffffffffu, p, t), dt = __shfl_sync(0xffffffffu, ds, t);
        if (!__shfl_sync(0xffffffffu, int(see), t)) continue;
        const T* q = static_cast<const T*>(a.q) + int64_t(s.q0 + i0 + t) * a.ldq + int64_t(h) * a.D;
        const T* g = static_cast<const T*>(a.dout) + (int64_t(s.q0 + i0 + t) * a.Hq + h) * a.D;
        for (int u = 0; u < 4; ++u)
          if (lane + 32 * u < a.D) {
            gk[u] = fmaf(dt, to_f32(q[lane + 32 * u]), gk[u]);
            gv[u] = fmaf(pt, to_f32(g[lane + 32 * u]), gv[u]);
          }
      }
    }
  T* dk = static_cast<T*>(a.dk) + (int64_t(s.k0 + j) * a.Hkv + hk) * a.D;
  T* dv = static_cast<T*>(a.dv) + (int64_t(s.k0 + j) * a.Hkv + hk) * a.D;
  bool bad = false;
  for (int u = 0; u < 4; ++u)
    if (lane + 32 * u < a.D) {
      if (!(fabsf(gk[u]) + fabsf(gv[u]) < INFINITY)) bad = true;
      dk[lane + 32 * u] = from_f32<T>(gk[u]);
      dv[lane + 32 * u] = from_f32<T>(gv[u]);
    }
  if (bad) raise_status(kDevNonFinite);
}

}  // namespace bl
