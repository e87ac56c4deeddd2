// Per-head RMSNorm of queries and keys with the position rotation in one pass,
// and its gradient.
//
// "ultragraph -- when the graph is the 1-bit LLM, part 2", section "attention,
// as graph ops" (RMSNorm, heads) and RoPE of "ultragraph-1bit 0.12.0" (PyPI):
//   r = 1 / sqrt(mean(x^2) + eps),  y = x r g,
//   (a, b) -> (a cos - b sin, a sin + b cos) on the pairs of the first R elements.
// Backward: dy = the transposed rotation of dz, dg = sum dy x r,
//   dx = r (g dy - x r^2 mean(x g dy)).
//
// Bound by memory: 4 bytes in and 2 or 4 out per element, nothing read twice (the
// table's rows are shared by a token's heads through L1/L2).  A head is split over
// D/8 lanes, each holding both members of its four pairs (two float4 loads), so
// the rotation needs no exchange between lanes and the sum of squares a few
// shuffles.
#pragma once

#include "attn_common.cuh"

namespace bl {

constexpr int kQrThreads = 256;

struct QrArgs {
  int64_t M;
  int Hq, Hkv, D;
  const float *q, *k, *v;
  int64_t ldq, ldk, ldv;
  const int32_t* pos;
  const float* table;
  int64_t P;
  int R, interleaved;
  const float *gq, *gk;
  float eps;
  // forward
  void *oq, *ok, *ov;
  const int64_t* slots;     // append: ok, ov are the caches
  int64_t nslots;           // pages * page
  int page;
  // backward
  const void *dq, *dk, *dv;
  float *dxq, *dxk, *dxv;
  int64_t lddq, lddk, lddv;
  float* part;              // [grid, 2, D] partial gain gradients
  int lanes;                // lanes per head: the power of two >= D / 8
};

__global__ void __launch_bounds__(256)
rope_table_kernel(float* __restrict__ table, int64_t P, int half, double base) {
  const int64_t n = P * half;
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x) {
    const int64_t p = i / half;
    const int j = int(i - p * half);
    double s, c;
    sincos(double(p) * pow(base, -double(j) / double(half)), &s, &c);
    table[p * 2 * half + j] = float(c);
    table[p * 2 * half + half + j] = float(s);
  }
}

// Sum over the `lanes` (power of two) lanes that share a head.
__device__ __forceinline__ float head_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}
__device__ __forceinline__ float4 mul4(float4 a, float4 b) { return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w); }
__device__ __forceinline__ float4 scale4(float4 a, float s) { return make_float4(a.x * s, a.y * s, a.z * s, a.w * s); }

// Rotates the pairs of (lo, hi) by (c, s): split pairs are (lo.x, hi.x) ...,
// interleaved ones (lo.x, lo.y) ... with c, s of four consecutive pairs.
__device__ __forceinline__ void rotate(float4& lo, float4& hi, float4 c, float4 s, bool interleaved) {
  float4 a, b;
  if (interleaved) {
    a = make_float4(lo.x, lo.z, hi.x, hi.z);
    b = make_float4(lo.y, lo.w, hi.y, hi.w);
  } else {
    a = lo;
    b = hi;
  }
  const float4 x = make_float4(fmaf(a.x, c.x, -(b.x * s.x)), fmaf(a.y, c.y, -(b.y * s.y)), fmaf(a.z, c.z, -(b.z * s.z)),
                               fmaf(a.w, c.w, -(b.w * s.w)));
  const float4 y = make_float4(fmaf(a.x, s.x, b.x * c.x), fmaf(a.y, s.y, b.y * c.y), fmaf(a.z, s.z, b.z * c.z),
                               fmaf(a.w, s.w, b.w * c.w));
  if (interleaved) {
    lo = make_float4(x.x, y.x, x.y, y.y);
    hi = make_float4(x.z, y.z, x.w, y.w);
  } else {
    lo = x;
    hi = y;
  }
}

// Item i of the work is a token and up to kHeads consecutive heads of its
// Hq + 2 Hkv (queries, keys, values).
template <typename T, bool kAppend, int kHeads>
__global__ void __launch_bounds__(kQrThreads)
qk_norm_rope_kernel(const QrArgs a) {
  const int lanes = a.lanes, u = threadIdx.x & (lanes - 1);
  const int per_block = kQrThreads / lanes;
  const int heads = a.Hq + 2 * a.Hkv, chunks = (heads + kHeads - 1) / kHeads;
  const int64_t items = a.M * chunks, step = int64_t(gridDim.x) * per_block;
  const bool on = u < (a.D >> 3);                    // this lane holds elements
  const bool turned = on && u < (a.R >> 3);          // ... of rotated pairs
  const bool split = turned && !a.interleaved;
  const int lo = on ? (split ? 4 * u : 8 * u) : 0, hi = on ? (split ? (a.R >> 1) + 4 * u : 8 * u + 4) : 0;
  const float inv_d = 1.f / float(a.D);
  bool bad = false, range = false;
  // whole warps take every turn together: the shuffles need all lanes
  const int64_t first = int64_t(blockIdx.x) * per_block, mine = threadIdx.x / lanes;
  // the token, its position and slot are asked for an item ahead: the table's row follows the position
  int64_t m_next = 0, c_next = 0, p_next = 0, at_next = -1;
  auto ask = [&](int64_t i) {
    if (i >= items) return;
    split_index(i, chunks, items < (int64_t(1) << 31), m_next, c_next);
    p_next = a.R ? a.pos[m_next] : 0;
    if (kAppend) at_next = a.slots[m_next];
  };
  ask(first + mine);
  for (int64_t base = first; base < items; base += step) {
    const int64_t i = base + mine;
    const bool live = i < items;
    const int64_t m = m_next, p = p_next, at = at_next;
    const int h0 = int(c_next) * kHeads;
    float4 x[kHeads], y[kHeads];
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const int h = h0 + j;
      x[j] = y[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!live || !on || h >= heads) continue;
      const float* row = h < a.Hq ? a.q + m * a.ldq + int64_t(h) * a.D
                         : h < a.Hq + a.Hkv ? a.k + m * a.ldk + int64_t(h - a.Hq) * a.D
                                            : a.v + m * a.ldv + int64_t(h - a.Hq - a.Hkv) * a.D;
      const bool value = h >= a.Hq + a.Hkv;
      x[j] = ld_stream_f4(reinterpret_cast<const float4*>(row + (value ? 8 * u : lo)));
      y[j] = ld_stream_f4(reinterpret_cast<const float4*>(row + (value ? 8 * u + 4 : hi)));
    }
    const bool ok = p >= 0 && (a.R == 0 || p < a.P);
    if (live && !ok) range = true;
    float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
    if (turned && ok) {
      cs = *reinterpret_cast<const float4*>(a.table + p * a.R + 4 * u);
      sn = *reinterpret_cast<const float4*>(a.table + p * a.R + (a.R >> 1) + 4 * u);
    }
    ask(i + step);
    int64_t page = 0, in = 0;
    bool store = true;
    if (kAppend) {
      store = live && at >= 0 && at < a.nslots;
      if (live && at >= a.nslots) range = true;
      split_index(store ? at : 0, a.page, a.nslots < (int64_t(1) << 31), page, in);
    }
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const int h = h0 + j;
      const float ss = head_sum(dot4(x[j], x[j], dot4(y[j], y[j], 0.f)), lanes);
      const bool value = h >= a.Hq + a.Hkv;
      if (!live || h >= heads || !ok || !on) continue;
      if (value) {
        if (!(dot4(x[j], make_float4(0, 0, 0, 0), dot4(y[j], make_float4(0, 0, 0, 0), 0.f)) == 0.f)) bad = true;
      } else {
        if (!(ss <= 3.4028235e38f)) bad = true;
        const float r = 1.f / sqrtf(fmaf(ss, inv_d, a.eps));
        const float* g = h < a.Hq ? a.gq : a.gk;
        x[j] = scale4(x[j], r);
        y[j] = scale4(y[j], r);
        if (g) {
          x[j] = mul4(x[j], *reinterpret_cast<const float4*>(g + lo));
          y[j] = mul4(y[j], *reinterpret_cast<const float4*>(g + hi));
        }
        if (turned) rotate(x[j], y[j], cs, sn, a.interleaved != 0);
      }
      T* out;
      if (h < a.Hq) {
        out = static_cast<T*>(a.oq) + (m * a.Hq + h) * a.D;
      } else {
        const int hk = value ? h - a.Hq - a.Hkv : h - a.Hq;
        T* o = static_cast<T*>(value ? a.ov : a.ok);
        if (kAppend) {
          if (!store) continue;
          out = o + ((page * a.Hkv + hk) * a.page + in) * a.D;
        } else {
          out = o + (m * a.Hkv + hk) * a.D;
        }
      }
      st4(out + (value ? 8 * u : lo), x[j]);
      st4(out + (value ? 8 * u + 4 : hi), y[j]);
    }
  }
  if (bad) raise_status(kDevNonFinite);
  if (range) raise_status(kDevRange);
}

// The gradient.  A group of lanes keeps the same columns throughout, so the gains'
// gradients stay in its registers until the end; then the CTA adds its groups in
// order and writes one partial row, and gain_sum_kernel adds those in order.
template <typename T, int kHeads>
__global__ void __launch_bounds__(kQrThreads, 2)
qk_norm_rope_backward_kernel(const QrArgs a) {
  extern __shared__ float sums[];                    // [per_block, 2, D]
  const int lanes = a.lanes, u = threadIdx.x & (lanes - 1), grp = threadIdx.x / lanes;
  const int per_block = kQrThreads / lanes;
  const int heads = a.Hq + 2 * a.Hkv, chunks = (heads + kHeads - 1) / kHeads;
  const int64_t items = a.M * chunks, step = int64_t(gridDim.x) * per_block;
  const bool on = u < (a.D >> 3), turned = on && u < (a.R >> 3), split = turned && !a.interleaved;
  const int lo = on ? (split ? 4 * u : 8 * u) : 0, hi = on ? (split ? (a.R >> 1) + 4 * u : 8 * u + 4) : 0;
  const float inv_d = 1.f / float(a.D);
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f), one = make_float4(1.f, 1.f, 1.f, 1.f);
  const float4 gq0 = a.gq ? *reinterpret_cast<const float4*>(a.gq + lo) : one;
  const float4 gq1 = a.gq ? *reinterpret_cast<const float4*>(a.gq + hi) : one;
  const float4 gk0 = a.gk ? *reinterpret_cast<const float4*>(a.gk + lo) : one;
  const float4 gk1 = a.gk ? *reinterpret_cast<const float4*>(a.gk + hi) : one;
  float4 sq0 = zero, sq1 = zero, sk0 = zero, sk1 = zero;
  bool bad = false, range = false;
  int64_t m_next = 0, c_next = 0, p_next = 0;        // asked for an item ahead: the table's row follows the position
  auto ask = [&](int64_t i) {
    if (i >= items) return;
    split_index(i, chunks, items < (int64_t(1) << 31), m_next, c_next);
    p_next = a.R ? a.pos[m_next] : 0;
  };
  ask(int64_t(blockIdx.x) * per_block + grp);
  for (int64_t base = int64_t(blockIdx.x) * per_block; base < items; base += step) {
    const int64_t i = base + grp;
    const bool live = i < items;
    const int64_t m = m_next, p = p_next;
    const int h0 = int(c_next) * kHeads;
    const bool ok = p >= 0 && (a.R == 0 || p < a.P);
    if (live && !ok) range = true;
    const bool work = live && on && ok;
    float4 x[kHeads], y[kHeads], e[kHeads], f[kHeads];
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const int h = h0 + j;
      const bool value = h >= a.Hq + a.Hkv, query = h < a.Hq;
      x[j] = y[j] = e[j] = f[j] = zero;
      if (!work || h >= heads) continue;
      const T* d = query ? static_cast<const T*>(a.dq) + (m * a.Hq + h) * a.D
                         : static_cast<const T*>(value ? a.dv : a.dk) + (m * a.Hkv + (value ? h - a.Hq - a.Hkv : h - a.Hq)) * a.D;
      e[j] = ld4(d + (value ? 8 * u : lo));
      f[j] = ld4(d + (value ? 8 * u + 4 : hi));
      if (value) continue;
      const float* row = query ? a.q + m * a.ldq + int64_t(h) * a.D : a.k + m * a.ldk + int64_t(h - a.Hq) * a.D;
      x[j] = ld_stream_f4(reinterpret_cast<const float4*>(row + lo));
      y[j] = ld_stream_f4(reinterpret_cast<const float4*>(row + hi));
    }
    float4 cs = one, sn = zero;
    if (work && turned) {
      cs = *reinterpret_cast<const float4*>(a.table + p * a.R + 4 * u);
      sn = *reinterpret_cast<const float4*>(a.table + p * a.R + (a.R >> 1) + 4 * u);
      sn = make_float4(-sn.x, -sn.y, -sn.z, -sn.w);
    }
    ask(i + step);
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const int h = h0 + j;
      const bool value = h >= a.Hq + a.Hkv, query = h < a.Hq;
      if (turned && !value) rotate(e[j], f[j], cs, sn, a.interleaved != 0);
      const float ss = head_sum(dot4(x[j], x[j], dot4(y[j], y[j], 0.f)), lanes);
      const float r = 1.f / sqrtf(fmaf(ss, inv_d, a.eps));
      x[j] = scale4(x[j], r);
      y[j] = scale4(y[j], r);
      const float4 px = mul4(e[j], x[j]), py = mul4(f[j], y[j]);          // dg terms
      const float4 ge = mul4(e[j], query ? gq0 : gk0), gf = mul4(f[j], query ? gq1 : gk1);
      const float t = head_sum(dot4(ge, x[j], dot4(gf, y[j], 0.f)), lanes) * inv_d;
      if (!work || h >= heads) continue;
      if (value) {
        float* out = a.dxv + m * a.lddv + int64_t(h - a.Hq - a.Hkv) * a.D;
        *reinterpret_cast<float4*>(out + 8 * u) = e[j];
        *reinterpret_cast<float4*>(out + 8 * u + 4) = f[j];
        continue;
      }
      if (!(ss <= 3.4028235e38f) || !(fabsf(t) <= 3.4028235e38f)) bad = true;
      float* out = query ? a.dxq + m * a.lddq + int64_t(h) * a.D : a.dxk + m * a.lddk + int64_t(h - a.Hq) * a.D;
      *reinterpret_cast<float4*>(out + lo) = make_float4(r * fmaf(-x[j].x, t, ge.x), r * fmaf(-x[j].y, t, ge.y),
                                                         r * fmaf(-x[j].z, t, ge.z), r * fmaf(-x[j].w, t, ge.w));
      *reinterpret_cast<float4*>(out + hi) = make_float4(r * fmaf(-y[j].x, t, gf.x), r * fmaf(-y[j].y, t, gf.y),
                                                         r * fmaf(-y[j].z, t, gf.z), r * fmaf(-y[j].w, t, gf.w));
      if (query) {
        sq0 = make_float4(sq0.x + px.x, sq0.y + px.y, sq0.z + px.z, sq0.w + px.w);
        sq1 = make_float4(sq1.x + py.x, sq1.y + py.y, sq1.z + py.z, sq1.w + py.w);
      } else {
        sk0 = make_float4(sk0.x + px.x, sk0.y + px.y, sk0.z + px.z, sk0.w + px.w);
        sk1 = make_float4(sk1.x + py.x, sk1.y + py.y, sk1.z + py.z, sk1.w + py.w);
      }
    }
  }
  if (bad) raise_status(kDevNonFinite);
  if (range) raise_status(kDevRange);
  if (!a.part) return;
  if (on) {
    float* s = sums + int64_t(grp) * 2 * a.D;
    *reinterpret_cast<float4*>(s + lo) = sq0;
    *reinterpret_cast<float4*>(s + hi) = sq1;
    *reinterpret_cast<float4*>(s + a.D + lo) = sk0;
    *reinterpret_cast<float4*>(s + a.D + hi) = sk1;
  }
  __syncthreads();
  for (int d = threadIdx.x; d < 2 * a.D; d += kQrThreads) {
    float s = 0.f;
    for (int j = 0; j < per_block; ++j) s += sums[j * 2 * a.D + d];
    a.part[int64_t(blockIdx.x) * 2 * a.D + d] = s;
  }
}

// dg[d] = sum over the CTAs' partial rows, 32 columns a CTA, 8 slices of rows.
__global__ void __launch_bounds__(256)
gain_sum_kernel(const float* __restrict__ part, int rows, int D, float* __restrict__ dgq, float* __restrict__ dgk) {
  __shared__ float s[8][32];
  const int c = threadIdx.x & 31, sl = threadIdx.x >> 5, d = blockIdx.x * 32 + c;
  float v = 0.f;
  if (d < 2 * D) {
    int r = sl;
    for (; r + 56 < rows; r += 64) {                   // eight loads in flight
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = part[int64_t(r + 8 * e) * 2 * D + d];
#pragma unroll
      for (int e = 0; e < 8; ++e) v += x[e];
    }
    for (; r < rows; r += 8) v += part[int64_t(r) * 2 * D + d];
  }
  s[sl][c] = v;
  __syncthreads();
  if (sl == 0 && d < 2 * D) {
    for (int j = 1; j < 8; ++j) v += s[j][c];
    float* out = d < D ? dgq : dgk;
    if (out) out[d < D ? d : d - D] = v;
  }
}

}  // namespace bl
