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
// shuffles.  Registers cannot hold enough loads in flight beside that (60 us for 8192
// tokens of 48 heads of 128), so many rows come by bulk copies into a ring per warp; then
// the instructions per item count: stepping without divisions 60 -> 51 us, 6.0 TB/s (92%
// of the card's copy rate), 4-head items instead of 8 86 us.  Its gradient, 4096 tokens:
// 45 us, 5.3 TB/s with the gains' sum.  Float32 outputs reach 5.2 TB/s.  At heads that do
// not fill their lanes instructions bind sooner: 48 heads of 80, 52 us, 3.6 TB/s.
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

// Sum over the kLanes lanes that share a head.
template <int kLanes> __device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = kLanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// A head's columns in a lane.
struct QrLane {
  bool on, turned;                  // holds elements; ... of rotated pairs
  int u, lo, hi;                    // lane in the head; its two groups of four columns
};
__device__ __forceinline__ QrLane qr_lane(const QrArgs& a, int u) {
  QrLane l;
  l.u = u;
  l.on = u < (a.D >> 3);
  l.turned = l.on && u < (a.R >> 3);
  const bool split = l.turned && !a.interleaved;
  l.lo = l.on ? (split ? 4 * u : 8 * u) : 0;
  l.hi = l.on ? (split ? (a.R >> 1) + 4 * u : 8 * u + 4) : 0;
  return l;
}
// The gains at four columns; ones where there are none.
__device__ __forceinline__ float4 gain4(const float* g, int col) {
  return g ? *reinterpret_cast<const float4*>(g + col) : make_float4(1.f, 1.f, 1.f, 1.f);
}
// Both gains in shared memory (a CTA's threads; a barrier follows).
__device__ __forceinline__ void share_gains(const QrArgs& a, float* to) {
  for (int d = threadIdx.x; d < 2 * a.D; d += blockDim.x) {
    const float* g = d < a.D ? a.gq : a.gk;
    to[d] = g ? g[d < a.D ? d : d - a.D] : 1.f;
  }
}
__device__ __forceinline__ float2 lo2(float4 a) { return make_float2(a.x, a.y); }
__device__ __forceinline__ float2 hi2(float4 a) { return make_float2(a.z, a.w); }
__device__ __forceinline__ float4 join4(float2 a, float2 b) { return make_float4(a.x, a.y, b.x, b.y); }
// The eight products' sum, packed: a0 b0 + a1 b1.
__device__ __forceinline__ float dot8(float4 a0, float4 b0, float4 a1, float4 b1) {
  float2 t = mul2(lo2(a0), lo2(b0));
  t = fma2(hi2(a0), hi2(b0), t);
  t = fma2(lo2(a1), lo2(b1), t);
  t = fma2(hi2(a1), hi2(b1), t);
  return t.x + t.y;
}
__device__ __forceinline__ float4 mul4(float4 a, float4 b) { return join4(mul2(lo2(a), lo2(b)), mul2(hi2(a), hi2(b))); }
__device__ __forceinline__ float4 scale4(float4 a, float s) { return mul4(a, make_float4(s, s, s, s)); }
__device__ __forceinline__ float4 fma4(float4 a, float4 b, float4 c) {
  return join4(fma2(lo2(a), lo2(b), lo2(c)), fma2(hi2(a), hi2(b), hi2(c)));
}
constexpr float kMaxF32 = 3.4028235e38f;
__device__ __forceinline__ float4 neg4(float4 a) { return make_float4(-a.x, -a.y, -a.z, -a.w); }

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
  const float4 x = fma4(a, c, neg4(mul4(b, s))), y = fma4(a, s, mul4(b, c));
  if (interleaved) {
    lo = make_float4(x.x, y.x, x.y, y.y);
    hi = make_float4(x.z, y.z, x.w, y.w);
  } else {
    lo = x;
    hi = y;
  }
}

// Few rows, where latency counts.  Item i of the work is a token and one of its Hq + 2 Hkv
// heads (queries, keys, values).
template <typename T, bool kAppend, int kLanes>
__global__ void __launch_bounds__(kQrThreads)
qk_norm_rope_kernel(const QrArgs a) {
  constexpr int kPerBlock = kQrThreads / kLanes;
  const QrLane l = qr_lane(a, threadIdx.x & (kLanes - 1));
  const int u = l.u, nk = a.Hq + a.Hkv, heads = nk + a.Hkv;
  const int64_t items = a.M * heads, step = int64_t(gridDim.x) * kPerBlock;
  const float inv_d = 1.f / float(a.D);
  bool bad = false, range = false;
  float top = 0.f;                                     // of what is stored, before its rounding
  // whole warps take every turn together: the shuffles need all lanes
  for (int64_t base = int64_t(blockIdx.x) * kPerBlock; base < items; base += step) {
    const int64_t i = base + threadIdx.x / kLanes;
    const bool live = i < items;
    int64_t m = 0, hh = 0;
    split_index(live ? i : 0, heads, items < (int64_t(1) << 31), m, hh);
    const int h = int(hh);
    const bool value = h >= nk, query = h < a.Hq;
    const int c0 = value ? 8 * u : l.lo, c1 = value ? 8 * u + 4 : l.hi;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    if (live && l.on) {
      const float* row = query ? a.q + m * a.ldq + h * a.D
                               : (value ? a.v + m * a.ldv - int64_t(nk) * a.D : a.k + m * a.ldk - int64_t(a.Hq) * a.D) + h * a.D;
      x = ld_stream_f4(reinterpret_cast<const float4*>(row + c0));
      y = ld_stream_f4(reinterpret_cast<const float4*>(row + c1));
    }
    const int64_t at = kAppend && live ? a.slots[m] : 0;
    const int64_t p = live && a.R ? a.pos[m] : 0;
    const bool ok = p >= 0 && (a.R == 0 || p < a.P);
    if (!ok || at >= (kAppend ? a.nslots : 1)) range = true;
    const float ss = head_sum<kLanes>(dot8(x, x, y, y));
    if (!live || !ok || !l.on) continue;
    if (!value) {
      if (!(ss <= kMaxF32)) bad = true;
      const float r = rsqrtf(fmaf(ss, inv_d, a.eps));
      const float* g = query ? a.gq : a.gk;
      x = mul4(scale4(x, r), gain4(g, l.lo));
      y = mul4(scale4(y, r), gain4(g, l.hi));
      if (l.turned)
        rotate(x, y, *reinterpret_cast<const float4*>(a.table + p * a.R + 4 * u),
               *reinterpret_cast<const float4*>(a.table + p * a.R + (a.R >> 1) + 4 * u), a.interleaved != 0);
    }
    top = top4(top4(top, x), y);
    T* out;
    if (query) {
      out = static_cast<T*>(a.oq) + (m * a.Hq + h) * a.D;
    } else {
      const int hk = value ? h - nk : h - a.Hq;
      out = static_cast<T*>(value ? a.ov : a.ok);
      if (kAppend) {
        if (at < 0 || at >= a.nslots) continue;
        int64_t page, in;
        split_index(at, a.page, a.nslots < (int64_t(1) << 31), page, in);
        out += ((page * a.Hkv + hk) * a.page + in) * a.D;
      } else {
        out += (m * a.Hkv + hk) * a.D;
      }
    }
    st4(out + c0, x);
    st4(out + c1, y);
  }
  if (bad || !reached<T>(top)) raise_status(kDevNonFinite);
  if (range) raise_status(kDevRange);
}

// The same for many rows, fed by the copy engine: each warp keeps three items of up to
// 128 / kLanes heads of a token (4 KB) in shared memory (bulk copies of whole runs of heads,
// two ahead of its work), so that 128 KB an SM are on their way whatever the registers allow.
constexpr int kQrRing = 3, kQrRingWarps = 8;
template <int kLanes> struct QrRing {
  static constexpr int kHeads = 128 / kLanes, kBackHeads = 64 / kLanes;   // of an item; of the gradient's
};

// An item of a warp: chunk c of token m; stepping from one to the next takes no division.
struct QrItem {
  int m, c, dm, dc;
  __device__ __forceinline__ QrItem(int64_t first, int64_t step, int chunks)
      : m(int(first / chunks)), c(int(first % chunks)), dm(int(step / chunks)), dc(int(step % chunks)) {}
  __device__ __forceinline__ void next(int chunks) {
    m += dm;
    c += dc;
    if (c >= chunks) {
      c -= chunks;
      ++m;
    }
  }
};
// What an item needs besides its rows.
template <bool kAppend>
struct QrAhead {
  int m, c, p;
  int64_t at;
  float4 cs, sn;
  __device__ __forceinline__ void ask(const QrArgs& a, const QrItem& i, bool live) {
    m = i.m;
    c = i.c;
    p = live && a.R ? a.pos[m] : 0;
    if (kAppend) at = live ? a.slots[m] : -1;
  }
  __device__ __forceinline__ bool fits(const QrArgs& a) const { return p >= 0 && (a.R == 0 || p < a.P); }
  __device__ __forceinline__ void turn(const QrArgs& a, const QrLane& l) {
    if (!l.turned || !fits(a)) return;
    const float* t = a.table + int64_t(p) * a.R + 4 * l.u;
    cs = *reinterpret_cast<const float4*>(t);
    sn = *reinterpret_cast<const float4*>(t + (a.R >> 1));
  }
};

// What one lane copies of each item: the heads lo .. hi - 1, `size` bytes each, of the token's
// row at src + m * row, to the item's place `to` on.
struct QrRun {
  const unsigned char* src;
  int64_t row;
  int lo, hi, size, to;
  __device__ __forceinline__ void copy(unsigned char* stage, int m, int h0, int h1, uint64_t* bar) const {
    const int a = max(lo, h0), b = min(hi, h1);
    if (a < b) bulk_g2s(stage + to + (a - h0) * size, src + int64_t(m) * row + (a - lo) * size, uint32_t((b - a) * size), bar);
  }
};

template <typename T, bool kAppend, int kLanes>
__global__ void __launch_bounds__(32 * kQrRingWarps, 2)
qk_norm_rope_ring_kernel(const QrArgs a) {
  extern __shared__ __align__(128) unsigned char qr_smem[];
  __shared__ uint64_t full[kQrRingWarps][kQrRing];
  __shared__ __align__(16) float gains[2 * 256];
  constexpr int kRingHeads = QrRing<kLanes>::kHeads;
  constexpr int kAtOnce = 32 / kLanes, kPasses = kRingHeads / kAtOnce;   // heads that the warp works on at a time
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const QrLane l = qr_lane(a, lane & (kLanes - 1));
  const int u = l.u, nk = a.Hq + a.Hkv, heads = nk + a.Hkv, chunks = (heads + kRingHeads - 1) / kRingHeads;
  const int64_t items = a.M * chunks, step = int64_t(gridDim.x) * kQrRingWarps;
  const int64_t first = int64_t(blockIdx.x) * kQrRingWarps + warp;
  const float inv_d = 1.f / float(a.D);
  float* ring = reinterpret_cast<float*>(qr_smem) + warp * kQrRing * kRingHeads * a.D;
  if (lane == 0) {
    for (int i = 0; i < kQrRing; ++i) mbar_init(&full[warp][i], 1);
    fence_mbar_init();
  }
  share_gains(a, gains);
  __syncthreads();
  // lanes 0..2 each copy the run of an item's heads that lies in q, k or v
  QrRun run;
  run.src = reinterpret_cast<const unsigned char*>(lane == 0 ? a.q : lane == 1 ? a.k : a.v);
  run.row = (lane == 0 ? a.ldq : lane == 1 ? a.ldk : a.ldv) * 4;
  run.lo = lane == 0 ? 0 : lane == 1 ? a.Hq : nk;
  run.hi = lane == 0 ? a.Hq : lane == 1 ? nk : lane == 2 ? heads : 0;
  run.size = a.D * 4;
  run.to = 0;
  auto issue = [&](const QrItem& i, int st) {
    const int h0 = i.c * kRingHeads, h1 = min(h0 + kRingHeads, heads);
    if (lane == 0) mbar_arrive_expect_tx(&full[warp][st], uint32_t((h1 - h0) * a.D * 4));
    __syncwarp();
    run.copy(reinterpret_cast<unsigned char*>(ring + st * kRingHeads * a.D), i.m, h0, h1, &full[warp][st]);
  };
  bool bad = false, range = false;
  float top = 0.f;                                     // of what is stored, before its rounding
  // Ahead of the work: an item's token, position and slot two items, its table row (which
  // follows the position) one.
  static_assert(kQrRing == 3, "copies and questions run two items ahead");
  QrItem item(first, step, chunks);
  QrAhead<kAppend> one, two;
  one.ask(a, item, first < items);
  if (first < items) issue(item, 0);
  one.turn(a, l);
  item.next(chunks);
  two.ask(a, item, first + step < items);
  if (first + step < items) issue(item, 1);
  int n = 0;
  for (int64_t i = first; i < items; i += step, ++n) {
    const int st = n % kQrRing;
    const QrAhead<kAppend> now = one;
    const bool more = i + 2 * step < items;
    item.next(chunks);
    one = two;
    one.turn(a, l);
    two.ask(a, item, more);
    const int m = now.m;
    const int64_t at = now.at;
    const int h0 = now.c * kRingHeads;
    __syncwarp();                                      // the item before has been read: its place takes the next copy
    if (more) issue(item, (n + 2) % kQrRing);
    const bool ok = now.fits(a);
    if (!ok) range = true;
    T* oq = static_cast<T*>(a.oq) + int64_t(m) * (a.Hq * a.D);
    T *ok_, *ov;
    bool store = true;
    int stride = a.D;
    if (kAppend) {
      store = at >= 0 && at < a.nslots;
      if (at >= a.nslots) range = true;
      int64_t page = 0, in = 0;
      split_index(store ? at : 0, a.page, a.nslots < (int64_t(1) << 31), page, in);
      stride = a.page * a.D;
      const int64_t to = page * a.Hkv * stride + in * a.D;
      ok_ = static_cast<T*>(a.ok) + to - int64_t(a.Hq) * stride;
      ov = static_cast<T*>(a.ov) + to - int64_t(nk) * stride;
    } else {
      const int64_t to = int64_t(m) * (a.Hkv * a.D);
      ok_ = static_cast<T*>(a.ok) + to - a.Hq * a.D;
      ov = static_cast<T*>(a.ov) + to - nk * a.D;
    }
    if (__any_sync(0xffffffffu, !mbar_wait_near(&full[warp][st], uint32_t(n / kQrRing) & 1u))) {
      if (lane == 0) raise_status(kDevTimeout);        // and no copy left in flight
      for (int k = 1; k < kQrRing; ++k)
        if (i + k * step < items) mbar_wait(&full[warp][(n + k) % kQrRing], uint32_t((n + k) / kQrRing) & 1u);
      break;
    }
    const float* rows = ring + st * kRingHeads * a.D;
    // all passes' sums first, so that their exchanges overlap
    float4 x[kPasses], y[kPasses];
    float ss[kPasses];
#pragma unroll
    for (int j = 0; j < kPasses; ++j) {
      const int slot = j * kAtOnce + lane / kLanes, h = h0 + slot;
      x[j] = y[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (h < heads && l.on) {
        x[j] = *reinterpret_cast<const float4*>(rows + slot * a.D + (h < nk ? l.lo : 8 * u));
        y[j] = *reinterpret_cast<const float4*>(rows + slot * a.D + (h < nk ? l.hi : 8 * u + 4));
      }
      ss[j] = head_sum<kLanes>(dot8(x[j], x[j], y[j], y[j]));
    }
#pragma unroll
    for (int j = 0; j < kPasses; ++j) {
      const int h = h0 + j * kAtOnce + lane / kLanes;
      if (h >= heads || !l.on || !ok) continue;
      int c0 = 8 * u, c1 = 8 * u + 4;
      if (h < nk) {
        if (!(ss[j] <= kMaxF32)) bad = true;
        const float r = rsqrtf(fmaf(ss[j], inv_d, a.eps));
        const float* g = gains + (h < a.Hq ? 0 : a.D);
        x[j] = mul4(scale4(x[j], r), *reinterpret_cast<const float4*>(g + l.lo));
        y[j] = mul4(scale4(y[j], r), *reinterpret_cast<const float4*>(g + l.hi));
        if (l.turned) rotate(x[j], y[j], now.cs, now.sn, a.interleaved != 0);
        c0 = l.lo;
        c1 = l.hi;
      }
      top = top4(top4(top, x[j]), y[j]);
      if (kAppend && h >= a.Hq && !store) continue;
      T* out = h < a.Hq ? oq + h * a.D : (h < nk ? ok_ : ov) + int64_t(h) * stride;
      st4(out + c0, x[j]);
      st4(out + c1, y[j]);
    }
  }
  if (bad || !reached<T>(top)) raise_status(kDevNonFinite);
  if (range) raise_status(kDevRange);
}

// A head's gradient from its row, its rotated-back gradient (e, f) and both sums.
__device__ __forceinline__ void head_back(const QrArgs& a, const QrLane& l, int h, int nk, float4 x, float4 y, float4 e,
                                          float4 f, float4 g0, float4 g1, float ss, float tt, float inv_d, float* oq,
                                          float* ok, float* ov, float4& sq0, float4& sq1, float4& sk0, float4& sk1, bool& bad,
                                          float& top) {
  if (h >= nk) {
    top = top4(top4(top, e), f);
    float* out = ov + h * a.D + 8 * l.u;
    *reinterpret_cast<float4*>(out) = e;
    *reinterpret_cast<float4*>(out + 4) = f;
    return;
  }
  const bool query = h < a.Hq;
  const float r = rsqrtf(fmaf(ss, inv_d, a.eps));
  const float t = tt * inv_d * r;
  if (!(ss <= kMaxF32)) bad = true;
  x = scale4(x, r);
  y = scale4(y, r);
  const float4 nt = make_float4(-t, -t, -t, -t);
  float* out = (query ? oq : ok) + h * a.D;
  const float4 dx = scale4(fma4(x, nt, mul4(e, g0)), r), dy = scale4(fma4(y, nt, mul4(f, g1)), r);
  *reinterpret_cast<float4*>(out + l.lo) = dx;
  *reinterpret_cast<float4*>(out + l.hi) = dy;
  top = top4(top4(top, dx), dy);
  if (query) {
    sq0 = fma4(e, x, sq0);
    sq1 = fma4(f, y, sq1);
  } else {
    sk0 = fma4(e, x, sk0);
    sk1 = fma4(f, y, sk1);
  }
}

// The CTA's part of the gains' gradients: its groups' sums, added in order.
template <int kGroups>
__device__ __forceinline__ void gain_part(const QrArgs& a, const QrLane& l, int grp, float* sums, float4 sq0, float4 sq1,
                                          float4 sk0, float4 sk1) {
  if (l.on) {
    float* s = sums + grp * 2 * a.D;
    *reinterpret_cast<float4*>(s + l.lo) = sq0;
    *reinterpret_cast<float4*>(s + l.hi) = sq1;
    *reinterpret_cast<float4*>(s + a.D + l.lo) = sk0;
    *reinterpret_cast<float4*>(s + a.D + l.hi) = sk1;
  }
  __syncthreads();
  for (int d = threadIdx.x; d < 2 * a.D; d += blockDim.x) {
    float s = 0.f;
    for (int j = 0; j < kGroups; ++j) s += sums[j * 2 * a.D + d];
    a.part[int64_t(blockIdx.x) * 2 * a.D + d] = s;
  }
}

// The gradient.  A group of lanes keeps the same columns throughout, so the gains'
// gradients stay in its registers until the end; then the CTA adds its groups in
// order and writes one partial row, and gain_sum_kernel adds those in order.
template <typename T, int kLanes>
__global__ void __launch_bounds__(kQrThreads, 2)
qk_norm_rope_backward_kernel(const QrArgs a) {
  extern __shared__ __align__(16) float sums[];      // [kPerBlock, 2, D]
  constexpr int kPerBlock = kQrThreads / kLanes;
  const QrLane l = qr_lane(a, threadIdx.x & (kLanes - 1));
  const int u = l.u, grp = threadIdx.x / kLanes;
  const int nk = a.Hq + a.Hkv, heads = nk + a.Hkv;
  const int64_t items = a.M * heads, step = int64_t(gridDim.x) * kPerBlock;
  const float inv_d = 1.f / float(a.D);
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 sq0 = zero, sq1 = zero, sk0 = zero, sk1 = zero;
  bool bad = false, range = false;
  float top = 0.f;                                     // of the gradients that are stored
  int64_t m_next = 0, h_next = 0, p_next = 0;        // asked for an item ahead: the table's row follows the position
  auto ask = [&](int64_t i) {
    if (i >= items) return;
    split_index(i, heads, items < (int64_t(1) << 31), m_next, h_next);
    p_next = a.R ? a.pos[m_next] : 0;
  };
  ask(int64_t(blockIdx.x) * kPerBlock + grp);
  for (int64_t base = int64_t(blockIdx.x) * kPerBlock; base < items; base += step) {
    const int64_t i = base + grp;
    const bool live = i < items;
    const int64_t m = m_next, p = p_next;
    const int h = int(h_next);
    const bool ok = p >= 0 && (a.R == 0 || p < a.P);
    if (live && !ok) range = true;
    const bool work = live && l.on && ok;
    float4 x = zero, y = zero, e = zero, f = zero;
    if (work) {
      const T* d = (h < a.Hq ? static_cast<const T*>(a.dq) + m * a.Hq * a.D
                             : static_cast<const T*>(h < nk ? a.dk : a.dv) + (m * a.Hkv - (h < nk ? a.Hq : nk)) * a.D) + h * a.D;
      e = ld4(d + (h < nk ? l.lo : 8 * u));
      f = ld4(d + (h < nk ? l.hi : 8 * u + 4));
      if (h < nk) {
        const float* row = (h < a.Hq ? a.q + m * a.ldq : a.k + m * a.ldk - int64_t(a.Hq) * a.D) + h * a.D;
        x = ld_stream_f4(reinterpret_cast<const float4*>(row + l.lo));
        y = ld_stream_f4(reinterpret_cast<const float4*>(row + l.hi));
      }
    }
    ask(i + step);
    if (work && l.turned && h < nk) {
      const float4 cs = *reinterpret_cast<const float4*>(a.table + p * a.R + 4 * u);
      const float4 sn = *reinterpret_cast<const float4*>(a.table + p * a.R + (a.R >> 1) + 4 * u);
      rotate(e, f, cs, make_float4(-sn.x, -sn.y, -sn.z, -sn.w), a.interleaved != 0);
    }
    // both sums at once: sum x^2, and sum x g dy, of which mean(x g dy r) is r / D times
    const float* g = h < a.Hq ? a.gq : a.gk;
    const float4 g0 = gain4(g, l.lo), g1 = gain4(g, l.hi);
    const float ss = head_sum<kLanes>(dot8(x, x, y, y));
    const float tt = head_sum<kLanes>(dot8(mul4(e, g0), x, mul4(f, g1), y));
    if (work)
      head_back(a, l, h, nk, x, y, e, f, g0, g1, ss, tt, inv_d, a.dxq + m * a.lddq, a.dxk + m * a.lddk - int64_t(a.Hq) * a.D,
                a.dxv + m * a.lddv - int64_t(nk) * a.D, sq0, sq1, sk0, sk1, bad, top);
  }
  if (bad || !reached<float>(top)) raise_status(kDevNonFinite);
  if (range) raise_status(kDevRange);
  if (a.part) gain_part<kPerBlock>(a, l, grp, sums, sq0, sq1, sk0, sk1);
}

// The gradient of many rows, fed like qk_norm_rope_ring_kernel: an item is up to 64 / kLanes
// heads of a token, their float32 rows and their gradients.

template <typename T, int kLanes>
__global__ void __launch_bounds__(32 * kQrRingWarps, 2)
qk_norm_rope_backward_ring_kernel(const QrArgs a) {
  extern __shared__ __align__(128) unsigned char qr_smem[];
  __shared__ uint64_t full[kQrRingWarps][kQrRing];
  __shared__ __align__(16) float gains[2 * 256];
  constexpr int kAtOnce = 32 / kLanes, kGroups = kQrRingWarps * kAtOnce;
  constexpr int kBackHeads = QrRing<kLanes>::kBackHeads, kPasses = kBackHeads / kAtOnce;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const QrLane l = qr_lane(a, lane & (kLanes - 1));
  const int u = l.u, nk = a.Hq + a.Hkv, heads = nk + a.Hkv, chunks = (heads + kBackHeads - 1) / kBackHeads;
  const int64_t items = a.M * chunks, step = int64_t(gridDim.x) * kQrRingWarps;
  const int64_t first = int64_t(blockIdx.x) * kQrRingWarps + warp;
  const float inv_d = 1.f / float(a.D);
  const int x_bytes = kBackHeads * a.D * 4, stage = x_bytes + kBackHeads * a.D * int(sizeof(T));
  unsigned char* ring = qr_smem + warp * kQrRing * stage;
  if (lane == 0) {
    for (int i = 0; i < kQrRing; ++i) mbar_init(&full[warp][i], 1);
    fence_mbar_init();
  }
  share_gains(a, gains);
  __syncthreads();
  // lanes 0..4 each copy a run of an item's heads: the rows of q and k, the gradients of all three
  const int size = int(sizeof(T));
  QrRun run;
  run.src = static_cast<const unsigned char*>(lane == 0 ? static_cast<const void*>(a.q) : lane == 1 ? a.k : lane == 2 ? a.dq
                                              : lane == 3 ? a.dk : a.dv);
  run.row = lane == 0 ? a.ldq * 4 : lane == 1 ? a.ldk * 4 : int64_t(lane == 2 ? a.Hq : a.Hkv) * a.D * size;
  run.lo = lane == 0 || lane == 2 ? 0 : lane == 4 ? nk : a.Hq;
  run.hi = lane == 0 || lane == 2 ? a.Hq : lane == 4 ? heads : lane < 4 ? nk : 0;
  run.size = a.D * (lane < 2 ? 4 : size);
  run.to = lane < 2 ? 0 : x_bytes;
  auto issue = [&](const QrItem& i, int st) {
    const int h0 = i.c * kBackHeads, h1 = min(h0 + kBackHeads, heads);
    if (lane == 0)
      mbar_arrive_expect_tx(&full[warp][st], uint32_t(max(0, min(h1, nk) - h0) * a.D * 4 + (h1 - h0) * a.D * size));
    __syncwarp();
    run.copy(ring + st * stage, i.m, h0, h1, &full[warp][st]);
  };
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  float4 sq0 = zero, sq1 = zero, sk0 = zero, sk1 = zero;
  bool bad = false, range = false;
  float top = 0.f;                                     // of the gradients that are stored
  static_assert(kQrRing == 3, "copies and questions run two items ahead");
  QrItem item(first, step, chunks);
  QrAhead<false> one, two;
  one.ask(a, item, first < items);
  if (first < items) issue(item, 0);
  one.turn(a, l);
  item.next(chunks);
  two.ask(a, item, first + step < items);
  if (first + step < items) issue(item, 1);
  int n = 0;
  for (int64_t i = first; i < items; i += step, ++n) {
    const int st = n % kQrRing;
    const QrAhead<false> now = one;
    const bool more = i + 2 * step < items;
    item.next(chunks);
    one = two;
    one.turn(a, l);
    two.ask(a, item, more);
    const int m = now.m;
    const int h0 = now.c * kBackHeads;
    __syncwarp();                                      // the item before has been read: its place takes the next copy
    if (more) issue(item, (n + 2) % kQrRing);
    const bool ok = now.fits(a);
    if (!ok) range = true;
    float* oq = a.dxq + m * a.lddq;
    float* okk = a.dxk + m * a.lddk - int64_t(a.Hq) * a.D;
    float* ov = a.dxv + m * a.lddv - int64_t(nk) * a.D;
    if (__any_sync(0xffffffffu, !mbar_wait_near(&full[warp][st], uint32_t(n / kQrRing) & 1u))) {
      if (lane == 0) raise_status(kDevTimeout);        // and no copy left in flight
      for (int k = 1; k < kQrRing; ++k)
        if (i + k * step < items) mbar_wait(&full[warp][(n + k) % kQrRing], uint32_t((n + k) / kQrRing) & 1u);
      break;
    }
    const float* rows = reinterpret_cast<const float*>(ring + st * stage);
    const T* grads = reinterpret_cast<const T*>(ring + st * stage + x_bytes);
    float4 x[kPasses], y[kPasses], e[kPasses], f[kPasses];
    float ss[kPasses], tt[kPasses];
#pragma unroll
    for (int j = 0; j < kPasses; ++j) {
      const int slot = j * kAtOnce + lane / kLanes, h = h0 + slot;
      const bool live = h < heads && l.on, value = h >= nk;
      x[j] = y[j] = e[j] = f[j] = zero;
      if (live) {
        e[j] = ld4(grads + slot * a.D + (value ? 8 * u : l.lo));
        f[j] = ld4(grads + slot * a.D + (value ? 8 * u + 4 : l.hi));
        if (!value) {
          x[j] = *reinterpret_cast<const float4*>(rows + slot * a.D + l.lo);
          y[j] = *reinterpret_cast<const float4*>(rows + slot * a.D + l.hi);
          if (l.turned) rotate(e[j], f[j], now.cs, neg4(now.sn), a.interleaved != 0);
        }
      }
      const float* g = gains + (h < a.Hq ? 0 : a.D);
      ss[j] = head_sum<kLanes>(dot8(x[j], x[j], y[j], y[j]));
      tt[j] = head_sum<kLanes>(dot8(mul4(e[j], *reinterpret_cast<const float4*>(g + l.lo)), x[j],
                                    mul4(f[j], *reinterpret_cast<const float4*>(g + l.hi)), y[j]));
    }
#pragma unroll
    for (int j = 0; j < kPasses; ++j) {
      const int slot = j * kAtOnce + lane / kLanes, h = h0 + slot;
      const float* g = gains + (h < a.Hq ? 0 : a.D);
      if (h < heads && l.on && ok)
        head_back(a, l, h, nk, x[j], y[j], e[j], f[j], *reinterpret_cast<const float4*>(g + l.lo),
                  *reinterpret_cast<const float4*>(g + l.hi), ss[j], tt[j], inv_d, oq, okk, ov, sq0, sq1, sk0, sk1, bad, top);
    }
  }
  if (bad || !reached<float>(top)) raise_status(kDevNonFinite);
  if (range) raise_status(kDevRange);
  if (!a.part) return;
  __syncthreads();                                     // the rings are read: their place takes the sums
  gain_part<kGroups>(a, l, threadIdx.x / kLanes, reinterpret_cast<float*>(qr_smem), sq0, sq1, sk0, sk1);
}

// dg[d] = sum over the CTAs' partial rows, 32 columns a CTA, 8 slices of rows.
__global__ void __launch_bounds__(256)
gain_sum_kernel(const float* __restrict__ part, int rows, int D, float* __restrict__ dgq, float* __restrict__ dgk) {
  __shared__ float s[8][32];
  griddep_wait();                                      // launched early: the parts are the kernel before's
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
