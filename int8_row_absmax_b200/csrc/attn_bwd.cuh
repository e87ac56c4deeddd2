// Gradients of attention over packed sequences on the tensor cores.
//
// With the scores' log-sum-exp from the forward, per pair of a query and a key it sees
//   P = 2^(c S - lse'),  dP = dO V^T,  dS = P (dP - delta),  delta = rowsum(dO O),
//   dV = P^T dO,  dK = scale dS^T Q,  dQ = scale dS K.
// Two kernels, so that every sum has a fixed order and no atomics:
//   attn_dkv_kernel   one CTA per 128 keys of a key head; walks the query blocks that see
//     them, for each head of the group, with the transposed products (keys are the rows):
//     S^T = K Q^T and dP^T = V dO^T into tensor memory, P^T and dS^T written back over
//     them in the inputs' type, dV += P^T dO and dK += dS^T Q with the accumulators in
//     tensor memory throughout: 4 matrix products a block.  Where that leaves SMs idle, a
//     group's heads are shared out over several CTAs, whose float32 parts
//     attn_dkv_join_kernel adds in order;
//   attn_dq_kernel    one CTA per 128 queries of a head; S, dP, dQ += dS K: 3 products.
// Seven products for the formula's five: recomputing S and dP costs 40% more matrix work
// than one kernel would, whose dQ would have to be summed across CTAs (atomics in float32,
// whose order changes the result, or a turn-taking between CTAs).
//
// Eight softmax warps share a block, a thread half a row (64 columns): while they form P
// the tensor core runs dK of the block before and dP of this one, while they form dS it
// runs dV and the next S.  Bound: 512 cycles per product and block at D = 128 against 1024
// of exponentials, and shared memory: the two products with both operands there read 128
// bytes a cycle, all it has, besides the 64 KB that arrive per block (about 2300 cycles a
// block for dK/dV, 1800 for dQ; measured about 3000 and 2600).  What feeding them early
// brought, dK/dV of 2 x 4096 tokens, 20/5 heads of 128: dO's place freed after dV and
// lse asked for a block ahead 529 -> 317 us, a third stage of Q and P in two parts 307.
//
// Measured there, bfloat16: 0.55 ms in all in bursts (780 TFLOP/s of the formula's five
// products, 1.09 PFLOP/s of the seven done): dQ 0.25, dK/dV 0.31, part of it in dQ's tail, row
// sums 0.016. Back to back 0.63 ms, under the card's power limit (1.39 PFLOP/s sustained).
//
// float16: P is stored 2^14 times larger and dS 2^k times, k from the largest norms of the
// rows of dO and V (|dP - delta| <= 2 |dO| |V|): neither overflows, and a dS down to 2^-28 of
// that bound is a normal number. k is one for each sequence and key head, the pairs that a CTA
// of dK/dV adds up: a sequence's gradients do not depend on what it is packed with. bfloat16
// needs neither.
#pragma once

#include "attn_fwd.cuh"

namespace bl {

constexpr int kAbThreads = 320;                        // 8 softmax warps, MMA warp, TMA warp
constexpr float kNoRow = 1e30f;                        // a log-sum-exp that makes every P zero

struct alignas(64) AttnBwdMaps {
  CUtensorMap q, k, v, dout;
};

template <int DP>
struct AbCfg {
  static constexpr int kTile = 128 * DP * 2;
  // K, V, three stages of Q with the rows' lse, two of dO with delta, barriers: all but a few
  // hundred bytes of an SM at D = 128, so nothing static and no room to align the base in
  static constexpr int kDkvRows = 7 * kTile, kDkvBars = kDkvRows + 5 * 512, kDkvSmem = kDkvBars + 256;
  static constexpr int kDqSmem = 7 * kTile + 1024;           // Q, dO, three K, two V
};

template <typename T> __device__ __forceinline__ constexpr float p_scale_log2() { return std::is_same<T, __half>::value ? 14.f : 0.f; }

// 2^k for dS (float16), from the largest squared row norms of dO and V that the CTAs of the row
// sums found of sequence b and key head hk; for whole warps.
template <typename T> __device__ __forceinline__ float ds_scale(const AttnArgs& a, const float* norms, int b, int hk, int lane) {
  if (!std::is_same<T, __half>::value) return 1.f;
  const float2* part = reinterpret_cast<const float2*>(norms) + (int64_t(b) * a.Hkv + hk) * a.parts;
  float o = 0.f, v = 0.f;
#pragma unroll 4
  for (int i = lane; i < a.parts; i += 32) {
    o = fmaxf(o, part[i].x);
    v = fmaxf(v, part[i].y);
  }
  const float most = 2.02f * sqrtf(warp_max(o)) * sqrtf(warp_max(v));
  if (!(most > 0.f && most < INFINITY)) return 1.f;
  return exp2f(fminf(fmaxf(floorf(log2f(32768.f / most)), -100.f), 100.f));
}

// delta[h, row] = sum dO O, one group of DP / 8 lanes a row; for float16 also the largest
// squared norms of the rows of dO and V (order does not matter to a maximum).  bfloat16 takes
// all rows alike.  For float16 a CTA takes the heads of one key head over some tokens of one
// sequence, about two rows a group, and as many of the sequence's keys, and leaves its two norms
// in a place of its own: no atomics, and nothing to clear before (a clearing takes 3 us).  (Four
// rows: 9.9 against 8.0 us for 5 sequences of up to 777 tokens, 6/2 heads; 23.6 against 27.6 for
// 2 x 4096, 20/5 heads.)  Rows dealt out over all sequences there, too, with atomics, took 10 us more for 64 sequences of 128 tokens, 8 heads of 64 (55 us in all): atomics
// wherever a group's row passes into another sequence; in bfloat16 looking up the sequence costs
// 13.5 -> 18.6 us (4096 tokens, 32 heads of 128).
template <typename T, int DP> struct AdCfg {
  static constexpr bool kNorms = std::is_same<T, __half>::value;
  static constexpr int kLanes = DP / 8, kRows = 256 / kLanes, kMost = 2 * kRows;   // rows at a time; keys of a CTA
  __host__ __device__ static int tokens(int group) { return group < kMost ? kMost / group : 1; }   // of a CTA
};
// The sum of a head's products x y, in all lanes of its group, and where asked for that of y's squares.
template <typename T, int kLanes>
__device__ __forceinline__ float2 row_sums(uint4 x, uint4 y, bool squares) {
  const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
  float d = 0.f, n = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 p = unpack2<T>(xs[e]), g = unpack2<T>(ys[e]);
    d = fmaf(p.x, g.x, fmaf(p.y, g.y, d));
    n = fmaf(g.x, g.x, fmaf(g.y, g.y, n));
  }
  for (int o = kLanes / 2; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  for (int o = kLanes / 2; squares && o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return make_float2(d, n);
}
template <typename T, int DP>
__global__ void __launch_bounds__(256, AdCfg<T, DP>::kNorms ? 6 : 8)  // bfloat16, 6: 17.7 us for 14.2 (4096 tokens, 32 heads of 128)
attn_delta_kernel(const AttnArgs a, float* norms) {
  using C = AdCfg<T, DP>;
  if (blockIdx.x >= unsigned(a.work)) return clear_rest(a, 256);
  const int u = threadIdx.x % C::kLanes, in = threadIdx.x / C::kLanes;
  const bool on = 8 * u < a.D;
  auto ask = [&](const void* p, int64_t at, bool live) {
    return live && on ? *reinterpret_cast<const uint4*>(static_cast<const T*>(p) + at + 8 * u) : make_uint4(0, 0, 0, 0);
  };
  if constexpr (!C::kNorms) {
    const int64_t rows = a.Tq * a.Hq;
    for (int64_t r0 = int64_t(blockIdx.x) * C::kRows; r0 < rows; r0 += int64_t(a.work) * C::kRows) {
      const int64_t r = r0 + in;
      const float d = row_sums<T, C::kLanes>(ask(a.o, r * a.D, r < rows), ask(a.dout, r * a.D, r < rows), false).x;
      int64_t token, h;
      split_index(r, a.Hq, rows < (int64_t(1) << 31), token, h);
      if (u == 0 && r < rows) a.delta[h * a.Tq + token] = d;
    }
  } else {
    const int hk = int(blockIdx.x % unsigned(a.Hkv)), rest = int(blockIdx.x / unsigned(a.Hkv)), b = rest % a.B;
    const int group = a.Hq / a.Hkv, tokens = C::tokens(group);
    Seq s;
    if (!load_seq(a, b, s, true)) return;
    float top_o = 0.f, top_v = 0.f;
    const int steps = max((s.nq + tokens - 1) / tokens, (s.nk + C::kMost - 1) / C::kMost);
    for (int c = rest / a.B; c < steps; c += a.parts) {
      const int i0 = min(c * tokens, s.nq), rows = min(tokens, s.nq - i0) * group;
      for (int r0 = 0; r0 < rows; r0 += C::kRows) {
        const int r = r0 + in, i = i0 + r / group, h = hk * group + r % group;
        const int64_t at = (int64_t(s.q0 + i) * a.Hq + h) * a.D;
        const float2 t = row_sums<T, C::kLanes>(ask(a.o, at, r < rows), ask(a.dout, at, r < rows), true);
        if (i + s.nk - s.nq >= 0 && t.y < INFINITY) top_o = fmaxf(top_o, t.y);          // rows that see a key
        if (u == 0 && r < rows) a.delta[int64_t(h) * a.Tq + s.q0 + i] = t.x;
      }
      const int j0 = int(min(int64_t(c) * C::kMost, int64_t(s.nk))), keys = min(C::kMost, s.nk - j0);   // c may count queries
      for (int r0 = 0; r0 < keys; r0 += C::kRows) {
        const int j = j0 + r0 + in;
        const uint4 x = ask(a.v, int64_t(s.k0 + j) * a.ldv + hk * a.D, r0 + in < keys);
        const float n = row_sums<T, C::kLanes>(x, x, false).x;
        const bool seen = a.window == 0 || j < a.sinks || j > s.nk - s.nq - a.window;   // by some query
        if (seen && n < INFINITY) top_v = fmaxf(top_v, n);
      }
    }
    __shared__ float tops[2][8];
    top_o = warp_max(top_o);
    top_v = warp_max(top_v);
    if ((threadIdx.x & 31) == 0) {
      tops[0][threadIdx.x >> 5] = top_o;
      tops[1][threadIdx.x >> 5] = top_v;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
      float t = 0.f;
      for (int w = 0; w < 8; ++w) t = fmaxf(t, tops[threadIdx.x][w]);
      norms[2 * ((int64_t(b) * a.Hkv + hk) * a.parts + rest / a.B) + threadIdx.x] = t;
    }
  }
}

// D (128 x DP) += P B over 128 rows of B, with P's columns of rows 64.. at +64 (each half
// of the softmax warps writes over the columns that it has read itself).
template <typename T, int DP>
__device__ __forceinline__ void mma_pv_halves(uint32_t d, uint32_t p, uint32_t b, bool acc) {
  mma_pv_part<T, DP, 64>(d, p, b, acc);
  mma_pv_part<T, DP, 64>(d, p + 64, b + 8192, true);
}

// A row of an accumulator, times f, to float32 memory.
template <int DP>
__device__ __forceinline__ void store_row_f32(uint32_t taddr, float* out, int D, float f, bool store, bool zero) {
#pragma unroll 1
  for (int u = 0; u < DP / 32; ++u) {
    uint32_t o[32];
    __syncwarp();
    tmem_ld32(taddr + u * 32, o);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      if (!store || u * 32 + e >= D) break;
      const float4 y = make_float4(__uint_as_float(o[e]) * f, __uint_as_float(o[e + 1]) * f, __uint_as_float(o[e + 2]) * f,
                                   __uint_as_float(o[e + 3]) * f);
      *reinterpret_cast<float4*>(out + u * 32 + e) = zero ? make_float4(0.f, 0.f, 0.f, 0.f) : y;
    }
  }
}

// dK and dV from the parts of the CTAs that shared a key block's query heads, in their order.
template <typename T>
__global__ void __launch_bounds__(256)
attn_dkv_join_kernel(const AttnArgs a) {
  griddep_wait();                                      // launched early: the parts are the kernel before's
  const int hk = int(blockIdx.x % unsigned(a.Hkv)), rest = int(blockIdx.x / unsigned(a.Hkv));
  const int j0 = rest / a.B * 128, b = rest % a.B;
  Seq s;
  if (!load_seq(a, b, s, true) || j0 >= s.nk) return;
  const int64_t step = 2 * int64_t(a.B) * a.max_k * a.Hkv * a.D;         // from one CTA's part to the next one's
  // 16 rows a CTA: 32 lanes a row (one quad each at D = 128), 8 rows at a time
  const int c = threadIdx.x & 31;
  uint32_t bad = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int which = i & 1, r = j0 + int(blockIdx.y) * 16 + (i >> 1) * 8 + (threadIdx.x >> 5);
    if (r >= s.nk || 4 * c >= a.D) continue;
    const int64_t at = (int64_t(s.k0 + r) * a.Hkv + hk) * a.D + 4 * c;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* part = part_row(a, 0, which, b, r, hk) + 4 * c;
#pragma unroll 4
    for (int z = 0; z < a.splits; ++z) {
      const float4 x = *reinterpret_cast<const float4*>(part + z * step);
      y = make_float4(y.x + x.x, y.y + x.y, y.z + x.z, y.w + x.w);
    }
    const uint2 w = make_uint2(pack2<T>(y.x, y.y), pack2<T>(y.z, y.w));
    bad |= not_finite2<T>(w.x) | not_finite2<T>(w.y);
    *reinterpret_cast<uint2*>(static_cast<T*>(which ? a.dv : a.dk) + at) = w;
  }
  if (bad) raise_status(kDevNonFinite);
}

// A row of an accumulator, times f, to 16-bit memory (D elements); false if any is stored as not finite.
template <typename T, int DP>
__device__ __forceinline__ bool store_row(uint32_t taddr, T* out, int D, float f, bool store, bool zero) {
  uint32_t bad = 0;
#pragma unroll 1
  for (int u = 0; u < DP / 32; ++u) {
    uint32_t o[32];
    __syncwarp();
    tmem_ld32(taddr + u * 32, o);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 32; e += 8) {
      if (!store || u * 32 + e >= D) break;
      uint32_t y[4];
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const float f0 = zero ? 0.f : __uint_as_float(o[e + 2 * z]) * f, f1 = zero ? 0.f : __uint_as_float(o[e + 2 * z + 1]) * f;
        y[z] = pack2<T>(f0, f1);
        bad |= not_finite2<T>(y[z]);
      }
      *reinterpret_cast<uint4*>(out + u * 32 + e) = make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
  return bad == 0;
}

template <typename T, int DP>
__global__ void __launch_bounds__(kAbThreads, 1)
attn_dkv_kernel(const __grid_constant__ AttnBwdMaps maps, const AttnArgs a, const float* norms) {
  using C = AbCfg<DP>;
  extern __shared__ __align__(1024) unsigned char dkv_smem[];
  unsigned char* smem = dkv_smem;
  const uint32_t base = smem_u32(smem);
  float* lse_rows = reinterpret_cast<float*>(smem + C::kDkvRows);       // [3][128]
  float* delta_rows = lse_rows + 3 * 128;                               // [2][128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kDkvBars);
  uint64_t &kv_full = bars[0], &s_full = bars[1], &dp_full = bars[2], &ds_ready = bars[3], &drain = bars[4];
  uint64_t *q_full = bars + 5, *q_empty = bars + 8, *g_full = bars + 11, *g_empty = bars + 13, *p_ready = bars + 15;
  uint64_t* d_full = bars + 17;
  uint32_t& s_tmem = *reinterpret_cast<uint32_t*>(bars + 19);
  volatile int* err = reinterpret_cast<volatile int*>(bars + 20);
  constexpr int kBoxes = DP / 64;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;

  if (base & 1023u) {                                                   // never, with nothing static before it
    raise_status(kDevBadWorkspace);
    griddep_wait();
    return;
  }
  // the work: parts of a group's heads and key heads fastest, early key blocks (which most queries see) first
  const int unit = int(blockIdx.x % unsigned(a.Hkv * a.splits)), rest = int(blockIdx.x / unsigned(a.Hkv * a.splits));
  const int hk = unit / a.splits, z = unit - hk * a.splits, group = a.Hq / a.Hkv;
  const int j0 = rest / a.B * 128, h0 = hk * group + z * a.split_heads, heads = min(a.split_heads, group - z * a.split_heads);
  const int b = rest % a.B;
  Seq s;
  // Launched while dQ's CTAs still run, and reads nothing of theirs (delta is from the kernel before
  // them); but it ends after they have ended, so that what follows it on the stream follows both.
  if (!load_seq(a, b, s, true) || j0 >= s.nk) {
    griddep_wait();
    return;
  }
  s.q0 = uniform(s.q0);
  s.nq = uniform(s.nq);
  s.k0 = uniform(s.k0);
  s.nk = uniform(s.nk);
  const int off = s.nk - s.nq;
  // query blocks that see these keys: rows from `first` (any row, not a multiple of 128) to `last`
  const int first = max(0, j0 - off);
  const int last = a.window == 0 || j0 < a.sinks ? s.nq - 1 : min(s.nq - 1, j0 + 126 + a.window - off);
  const int per = last < first ? 0 : (last - first) / 128 + 1;          // blocks of one head
  const int n = per * heads;

  // tiles: K, V, three of Q, two of dO
  auto q_tile = [&](int it) { return (2 + it % 3) * C::kTile; };
  auto g_tile = [&](int it) { return (5 + (it & 1)) * C::kTile; };
  if (tid == 0) {
    *err = 0;
    mbar_init(&kv_full, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&g_full[i], 1);
      mbar_init(&g_empty[i], 1);
      mbar_init(&p_ready[i], 8);
      mbar_init(&d_full[i], 1);
    }
    mbar_init(&s_full, 1);
    mbar_init(&dp_full, 1);
    mbar_init(&ds_ready, 8);
    mbar_init(&drain, 1);
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uint32_t(uniform(int(s_tmem)));                 // S, dP, dV, dK: 128 columns each
  float mult = 1.f;                                                     // dS's scale, in the softmax warps

  if (warp == 9) {
    if (lane == 0 && n > 0) {
      mbar_arrive_expect_tx(&kv_full, 2 * C::kTile);
      tma_rows(smem, &maps.k, kBoxes, hk, s.k0 + j0, &kv_full);
      tma_rows(smem + C::kTile, &maps.v, kBoxes, hk, s.k0 + j0, &kv_full);
    }
    // a block's lse and delta are asked for while the block before waits for its places
    float l[4], e[4];
    auto ask = [&](int it) {
      const int h = h0 + it / per, i0 = first + it % per * 128;
      const int64_t at = int64_t(h) * a.Tq + s.q0 + i0 + lane;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool in = i0 + lane + 32 * u < s.nq;
        l[u] = in ? a.lse[at + 32 * u] : -INFINITY;
        e[u] = in ? a.delta[at + 32 * u] : 0.f;
      }
    };
    if (n > 0) ask(0);
    int it = 0;
    for (; it < n; ++it) {
      const int qs = it % 3, gs = it & 1, h = h0 + it / per, i0 = first + it % per * 128;
      // places come free in this order: Q's (and lse's) after dK of three blocks ago, dO's after dV of two
      // blocks ago, delta's, which is read after that, after dK of two blocks ago
      if (it >= 3 && !mbar_wait_near(&q_empty[qs], uint32_t(it / 3 - 1) & 1u)) *err = 1;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        lse_rows[qs * 128 + lane + 32 * u] = l[u] == -INFINITY ? kNoRow : fmaf(l[u], kLog2e, -p_scale_log2<T>());
      __syncwarp();
      if (__any_sync(0xffffffffu, *err)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&q_full[qs], C::kTile);
        tma_rows(smem + q_tile(it), &maps.q, kBoxes, h, s.q0 + i0, &q_full[qs]);
      }
      if (it >= 2 && !mbar_wait_near(&g_empty[gs], uint32_t(it / 2 - 1) & 1u)) *err = 1;
      if (__any_sync(0xffffffffu, *err)) {
        ++it;
        break;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(&g_full[gs], C::kTile);
        tma_rows(smem + g_tile(it), &maps.dout, kBoxes, h, s.q0 + i0, &g_full[gs]);
      }
      if (it >= 2 && !mbar_wait_near(&q_empty[(it - 2) % 3], uint32_t((it - 2) / 3) & 1u)) *err = 1;
#pragma unroll
      for (int u = 0; u < 4; ++u) delta_rows[gs * 128 + lane + 32 * u] = e[u];
      __syncwarp();
      if (lane == 0) mbar_arrive(&d_full[gs]);
      if (it + 1 < n) ask(it + 1);
    }
    if (*err && n > 0) {                                                // leave no copy in flight behind
      mbar_wait_near(&kv_full, 0u);
      for (int i = max(0, it - 3); i < it; ++i) mbar_wait_near(&q_full[i % 3], uint32_t(i / 3) & 1u);
      for (int i = max(0, it - 2); i < it; ++i) mbar_wait_near(&g_full[i & 1], uint32_t(i / 2) & 1u);
    }
  } else if (warp == 8) {
    bool good = true;                                                   // the same in every lane
    auto wait = [&](uint64_t* bar, int parity) {
      if (good && __any_sync(0xffffffffu, !mbar_wait_near(bar, uint32_t(parity) & 1u))) {
        good = false;
        *err = 1;
      }
      tc_fence_after();
    };
    const uint32_t S = tmem, dP = tmem + 128, dV = tmem + 256, dK = tmem + 384;
    // rows of no query of the sequence must not meet P's and dS's zeros
    auto trim = [&](unsigned char* tile, int it) {
      const int i0 = first + it % per * 128;
      if (i0 + 128 > s.nq && s.q0 + s.nq < a.Tq) zero_rows(tile, kBoxes, s.nq - i0, 128, lane);
    };
    auto wait_q = [&](int it) {
      wait(&q_full[it % 3], it / 3);
      trim(smem + q_tile(it), it);
    };
    auto wait_g = [&](int it) {
      wait(&g_full[it & 1], it / 2);
      trim(smem + g_tile(it), it);
    };
    if (n > 0) {
      wait(&kv_full, 0);
      wait_q(0);
      if (good) {
        mma_qk<T, DP>(S, base, base + q_tile(0));
        umma_commit_warp(&s_full);
      }
      wait_g(0);
      if (good) {
        mma_qk<T, DP>(dP, base + C::kTile, base + g_tile(0));
        umma_commit_warp(&dp_full);
      }
    }
    for (int it = 0; it < n && good; ++it) {
      const bool more = it + 1 < n;
      // P comes in two parts: columns 0..31 of each half, then 32..63
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        wait(&p_ready[part], it);
        if (good) {
          mma_pv_part<T, DP, 32>(dV, S + part * 16, base + g_tile(it) + part * 4096, it > 0 || part > 0);
          mma_pv_part<T, DP, 32>(dV, S + 64 + part * 16, base + g_tile(it) + 8192 + part * 4096, true);
        }
      }
      if (good) umma_commit_warp(&g_empty[it & 1]);
      if (more) {
        wait_q(it + 1);
        if (good) {
          mma_qk<T, DP>(S, base, base + q_tile(it + 1));                  // in order behind the product that reads P
          umma_commit_warp(&s_full);
        }
      }
      wait(&ds_ready, it);
      if (good) {
        mma_pv_halves<T, DP>(dK, dP, base + q_tile(it), it > 0);
        umma_commit_warp(&q_empty[it % 3]);
      }
      if (more) {
        wait_g(it + 1);
        if (good) {
          mma_qk<T, DP>(dP, base + C::kTile, base + g_tile(it + 1));
          umma_commit_warp(&dp_full);
        }
      }
    }
    umma_commit_warp(&drain);
  } else {
    const int half = warp >> 2, row = (warp & 3) * 32 + lane, j = j0 + row;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t S = tmem + lanes + half * 64, dP = S + 128;
    const float c = a.scale * kLog2e;
    mult = ds_scale<T>(a, norms, b, hk, lane);
    const float f = mult * exp2f(-p_scale_log2<T>());
    bool fine = true;
    for (int it = 0; it < n; ++it) {
      const int i0 = first + it % per * 128;
      const float4* lse = reinterpret_cast<const float4*>(lse_rows + it % 3 * 128 + half * 64);
      const float4* del = reinterpret_cast<const float4*>(delta_rows + (it & 1) * 128 + half * 64);
      fine = mbar_wait_near(&q_full[it % 3], uint32_t(it / 3) & 1u) && mbar_wait_near(&s_full, uint32_t(it) & 1u) && !*err;
      if (__any_sync(0xffffffffu, !fine)) {
        *err = 1;
        break;
      }
      tc_fence_after();
      float p[64];
      uint32_t w[32];
      tmem_ld32(S, reinterpret_cast<uint32_t*>(p));
      tmem_ld32(S + 32, reinterpret_cast<uint32_t*>(p) + 32);
      tmem_ld_wait();
      // some key of the block is not seen by some query of the block
      const bool masked = i0 + off < j0 + 127 || (a.window != 0 && i0 + 127 + off >= j0 + a.window && j0 + 128 > a.sinks);
      const int bot = j - off - i0 - half * 64;
      const int top = a.window == 0 || j < a.sinks ? 128 : j + a.window - off - i0 - half * 64;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        float* pp = p + part * 32;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float4 l = lse[part * 8 + u];
          pp[4 * u] = exp2_approx(fmaf(pp[4 * u], c, -l.x));
          pp[4 * u + 1] = exp2_approx(fmaf(pp[4 * u + 1], c, -l.y));
          pp[4 * u + 2] = exp2_approx(fmaf(pp[4 * u + 2], c, -l.z));
          pp[4 * u + 3] = exp2_approx(fmaf(pp[4 * u + 3], c, -l.w));
        }
        if (masked) {
          const uint32_t seen = low_bits(top - part * 32) & ~low_bits(bot - part * 32);
#pragma unroll
          for (int u = 0; u < 32; ++u)
            if (!(seen & (1u << u))) pp[u] = 0.f;
        }
#pragma unroll
        for (int u = 0; u < 16; ++u) w[part * 16 + u] = pack2<T>(pp[2 * u], pp[2 * u + 1]);
        tmem_st16(S + part * 16, w + part * 16);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[part]);
      }

      fine = mbar_wait_near(&d_full[it & 1], uint32_t(it / 2) & 1u) && mbar_wait_near(&dp_full, uint32_t(it) & 1u) && !*err;
      if (__any_sync(0xffffffffu, !fine)) {
        *err = 1;
        break;
      }
      tc_fence_after();
      float d[64];
      tmem_ld32(dP, reinterpret_cast<uint32_t*>(d));
      tmem_ld32(dP + 32, reinterpret_cast<uint32_t*>(d) + 32);
      tmem_ld_wait();
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const float4 e = del[u];
        d[4 * u] = p[4 * u] * (d[4 * u] - e.x);
        d[4 * u + 1] = p[4 * u + 1] * (d[4 * u + 1] - e.y);
        d[4 * u + 2] = p[4 * u + 2] * (d[4 * u + 2] - e.z);
        d[4 * u + 3] = p[4 * u + 3] * (d[4 * u + 3] - e.w);
      }
      if (masked) {                                                     // zero whatever V holds there
#pragma unroll
        for (int u = 0; u < 64; ++u)
          if (p[u] == 0.f) d[u] = 0.f;
      }
#pragma unroll
      for (int u = 0; u < 32; ++u)
        w[u] = std::is_same<T, __half>::value ? pack2<T>(d[2 * u] * f, d[2 * u + 1] * f) : pack2<T>(d[2 * u], d[2 * u + 1]);
      tmem_st32(dP, w);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ds_ready);                            // (lse and delta of the stage have been read, too)
    }
  }

  // every product done: warps 0..3 store dV, warps 4..7 dK
  __syncthreads();
  if (warp == 8) {
    if (!mbar_wait_near(&drain, 0u)) *err = 1;
    __syncwarp();
    if (*err && lane == 0) raise_status(kDevTimeout);
  }
  __syncthreads();
  tc_fence_after();
  if (warp < 8 && !*err) {
    const int row = (warp & 3) * 32 + lane, j = j0 + row;
    const bool keys = warp >= 4;
    const uint32_t acc = tmem + (uint32_t((warp & 3) * 32) << 16) + (keys ? 384 : 256);
    const float f = keys ? a.scale / mult : exp2f(-p_scale_log2<T>());
    const int64_t at = (int64_t(s.k0 + j) * a.Hkv + hk) * a.D;
    T* out = static_cast<T*>(keys ? a.dk : a.dv) + at;
    if (a.splits > 1)
      store_row_f32<DP>(acc, part_row(a, z, keys ? 0 : 1, b, j, hk), a.D, f, j < s.nk, n == 0);
    else if (!store_row<T, DP>(acc, out, a.D, f, j < s.nk, n == 0) && j < s.nk) raise_status(kDevNonFinite);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  griddep_wait();
}

template <typename T, int DP>
__global__ void __launch_bounds__(kAbThreads, 1)
attn_dq_kernel(const __grid_constant__ AttnBwdMaps maps, const AttnArgs a, const float* norms) {
  using C = AbCfg<DP>;
  extern __shared__ unsigned char ab_smem[];
  __shared__ uint64_t q_full, k_full[3], k_empty[3], v_full[2], v_empty[2], s_full[2], dp_full, ds_ready, drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_err;
  constexpr int kBoxes = DP / 64;
  volatile int* err = &s_err;
  griddep_launch_dependents();                                          // dK/dV may take SMs as soon as they are free
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;

  const int nblk = (a.max_q + 127) / 128;
  const int h = int(blockIdx.x % unsigned(a.Hq)), rest = int(blockIdx.x / unsigned(a.Hq));
  const int i0 = (nblk - 1 - rest / a.B) * 128, hk = h / (a.Hq / a.Hkv), b = rest % a.B;
  Seq s;
  if (!load_seq(a, b, s, true) || i0 >= s.nq) return;
  s.q0 = uniform(s.q0);
  s.nq = uniform(s.nq);
  s.k0 = uniform(s.k0);
  s.nk = uniform(s.nk);
  const int off = s.nk - s.nq;
  const Blocks blocks = key_blocks(i0 + off, min(i0 + 128, s.nq) - 1 + off, a.window, a.sinks);
  const int n = blocks.n;

  const uint32_t base = (smem_u32(ab_smem) + 1023u) & ~1023u;
  unsigned char* smem = ab_smem + (base - smem_u32(ab_smem));
  if (tid == 0) {
    s_err = 0;
    mbar_init(&q_full, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
    }
    mbar_init(&dp_full, 1);
    mbar_init(&ds_ready, 8);
    mbar_init(&drain, 1);
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uint32_t(uniform(int(s_tmem)));                 // S0, S1, dP, dQ: 128 columns each
  float mult = 1.f;                                                     // dS's scale, in the softmax warps

  if (warp == 9) {
    if (lane == 0 && n > 0) {
      mbar_arrive_expect_tx(&q_full, 2 * C::kTile);
      tma_rows(smem, &maps.q, kBoxes, h, s.q0 + i0, &q_full);
      tma_rows(smem + C::kTile, &maps.dout, kBoxes, h, s.q0 + i0, &q_full);
      int it = 0;
      for (; it < n; ++it) {
        const int ks = it % 3, vs = it & 1, j0 = blocks.at(it);
        if (it >= 3 && !mbar_wait_near(&k_empty[ks], uint32_t(it / 3 - 1) & 1u)) *err = 1;
        if (it >= 2 && !mbar_wait_near(&v_empty[vs], uint32_t(it / 2 - 1) & 1u)) *err = 1;
        if (*err) break;
        mbar_arrive_expect_tx(&k_full[ks], C::kTile);
        tma_rows(smem + (2 + ks) * C::kTile, &maps.k, kBoxes, hk, s.k0 + j0, &k_full[ks]);
        mbar_arrive_expect_tx(&v_full[vs], C::kTile);
        tma_rows(smem + (5 + vs) * C::kTile, &maps.v, kBoxes, hk, s.k0 + j0, &v_full[vs]);
      }
      if (*err) {                                                       // leave no copy in flight behind
        mbar_wait_near(&q_full, 0u);
        for (int i = max(0, it - 3); i < it; ++i) mbar_wait_near(&k_full[i % 3], uint32_t(i / 3) & 1u);
        for (int i = max(0, it - 2); i < it; ++i) mbar_wait_near(&v_full[i & 1], uint32_t(i / 2) & 1u);
      }
    }
  } else if (warp == 8) {
    bool good = true;                                                   // the same in every lane
    auto wait = [&](uint64_t* bar, int parity) {
      if (good && __any_sync(0xffffffffu, !mbar_wait_near(bar, uint32_t(parity) & 1u))) {
        good = false;
        *err = 1;
      }
      tc_fence_after();
    };
    const uint32_t dP = tmem + 256, dQ = tmem + 384;
    auto k_at = [&](int it) { return base + uint32_t((2 + it % 3) * C::kTile); };
    auto wait_k = [&](int it) {
      wait(&k_full[it % 3], it / 3);
      zero_dead_keys(smem + (2 + it % 3) * C::kTile, kBoxes, blocks.at(it), s, a.window, a.sinks, a.Tk, lane);
    };
    auto issue_s = [&](int it) {
      if (!good) return;
      mma_qk<T, DP>(tmem + (it & 1) * 128, base, k_at(it));
      umma_commit_warp(&s_full[it & 1]);
    };
    auto issue_dp = [&](int it) {
      if (!good) return;
      mma_qk<T, DP>(dP, base + C::kTile, base + uint32_t((5 + (it & 1)) * C::kTile));
      umma_commit_warp(&dp_full);
      umma_commit_warp(&v_empty[it & 1]);
    };
    if (n > 0) {
      wait(&q_full, 0);
      wait_k(0);
      issue_s(0);
      wait(&v_full[0], 0);
      issue_dp(0);
      if (n > 1) {
        wait_k(1);
        issue_s(1);
      }
    }
    for (int it = 0; it < n && good; ++it) {
      if (it + 1 < n) wait(&v_full[(it + 1) & 1], (it + 1) / 2);        // loaded long since
      wait(&ds_ready, it);
      if (it + 1 < n) issue_dp(it + 1);                                 // dP of this block has been read
      if (good) {
        mma_pv_halves<T, DP>(dQ, tmem + (it & 1) * 128, k_at(it), it > 0);
        umma_commit_warp(&k_empty[it % 3]);
      }
      if (it + 2 < n) {
        wait_k(it + 2);
        issue_s(it + 2);                                                // in order behind the product that reads dS
      }
    }
    umma_commit_warp(&drain);
  } else {
    const int half = warp >> 2, row = (warp & 3) * 32 + lane, i = i0 + row;
    const int pos = i < s.nq ? i + off : -1, lo = a.window ? pos - a.window + 1 : 0;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t dP = tmem + lanes + 256 + half * 64;
    const float c = a.scale * kLog2e;
    float lse = kNoRow, delta = 0.f;
    if (i < s.nq) {
      const float l = a.lse[int64_t(h) * a.Tq + s.q0 + i];
      lse = l == -INFINITY ? kNoRow : l * kLog2e;
      delta = a.delta[int64_t(h) * a.Tq + s.q0 + i];
    }
    mult = ds_scale<T>(a, norms, b, hk, lane);
    bool fine = true;
    for (int it = 0; it < n; ++it) {
      const int j0 = blocks.at(it);
      const uint32_t S = tmem + lanes + (it & 1) * 128 + half * 64;
      fine = mbar_wait_near(&s_full[it & 1], uint32_t(it / 2) & 1u) && !*err;
      if (__any_sync(0xffffffffu, !fine)) {
        *err = 1;
        break;
      }
      tc_fence_after();
      float p[64];
      tmem_ld32(S, reinterpret_cast<uint32_t*>(p));
      tmem_ld32(S + 32, reinterpret_cast<uint32_t*>(p) + 32);
      tmem_ld_wait();
#pragma unroll
      for (int u = 0; u < 64; ++u) p[u] = exp2_approx(fmaf(p[u], c, -lse));
      // a key of the block is not seen by some row of the tile
      const bool masked = j0 + 127 > i0 + off ||
                          (a.window != 0 && j0 <= min(i0 + 128, s.nq) - 1 + off - a.window && j0 + 128 > a.sinks);
      if (masked) {
        const int top = pos - j0 - half * 64, bot = lo - j0 - half * 64, lead = a.window ? a.sinks - j0 - half * 64 : 0;
#pragma unroll
        for (int f = 0; f < 64; f += 32) {
          const uint32_t seen = seen_bits(f, top, bot, lead);
#pragma unroll
          for (int u = 0; u < 32; ++u)
            if (!(seen & (1u << u))) p[f + u] = 0.f;
        }
      }
      fine = mbar_wait_near(&dp_full, uint32_t(it) & 1u) && !*err;
      if (__any_sync(0xffffffffu, !fine)) {
        *err = 1;
        break;
      }
      tc_fence_after();
      float d[64];
      uint32_t w[32];
      tmem_ld32(dP, reinterpret_cast<uint32_t*>(d));
      tmem_ld32(dP + 32, reinterpret_cast<uint32_t*>(d) + 32);
      tmem_ld_wait();
#pragma unroll
      for (int u = 0; u < 64; ++u) d[u] = p[u] * (d[u] - delta);
      if (masked) {                                                     // zero whatever V holds there
#pragma unroll
        for (int u = 0; u < 64; ++u)
          if (p[u] == 0.f) d[u] = 0.f;
      }
#pragma unroll
      for (int u = 0; u < 32; ++u)
        w[u] = std::is_same<T, __half>::value ? pack2<T>(d[2 * u] * mult, d[2 * u + 1] * mult) : pack2<T>(d[2 * u], d[2 * u + 1]);
      tmem_st32(S, w);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ds_ready);
    }
  }

  __syncthreads();
  if (warp == 8) {
    if (!mbar_wait_near(&drain, 0u)) *err = 1;
    __syncwarp();
    if (*err && lane == 0) raise_status(kDevTimeout);
  }
  __syncthreads();
  tc_fence_after();
  if (warp < 4 && !*err) {
    const int row = warp * 32 + lane, i = i0 + row;
    T* out = static_cast<T*>(a.dq) + (int64_t(s.q0 + i) * a.Hq + h) * a.D;
    const uint32_t acc = tmem + (uint32_t(warp * 32) << 16) + 384;
    if (!store_row<T, DP>(acc, out, a.D, a.scale / mult, i < s.nq, n == 0) && i < s.nq) raise_status(kDevNonFinite);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace bl
