// Attention over packed sequences on the tensor cores (forward).
//
// One CTA takes two tiles of 128 query rows that read the same keys (two heads of a
// group, or two neighbouring row blocks where the group is odd) and walks the
// 128-key blocks that they see.  Per block and tile, on tcgen05 kind::f16:
//   S = Q K^T   (128 x 128, float32 in tensor memory; Q, K from shared memory),
//   P = 2^(c S - m) by the tile's four softmax warps, one thread a row: the row never
//       leaves its thread, so maximum and sum need no exchange; P goes back to tensor
//       memory over S in the inputs' type,
//   O += P V    (P from tensor memory, V from shared memory as it lies, MN-major).
// The two tiles take turns: the tensor core works on one while the other's softmax
// runs.  m is only raised when a row's maximum grows by more than 2^kLazy, since P up
// to that size loses nothing; then the warp scales its rows of O in tensor memory.
// For float16 P is kept 2^7 higher, out of the subnormals (at most 2^15 in all).
//
// Bound: 2 x 512 cycles of matrix work per block and tile at D = 128 and, of the same
// size, 128 x 128 exponentials at 16 a cycle (1024 cycles); at D = 64 the exponentials
// alone.  A tile's own round is not overlapped with itself: about 1850 cycles of softmax
// (440 of them the loads and the maximum), then 1200 until its next S is there, 3070 in
// all for both tiles against 2048 at the bound.  Measured (clock stamps): P handed over
// in two parts takes 256 cycles off it, four parts cost more in waits than they gain.
// Two threads a row (16 softmax warps) and a polynomial 2^y on the multiply-add pipe for
// part of the row were both slower: 480 and 474 against 443 us.
//
// Measured, bfloat16, 32/8 heads, one sequence of 8192 tokens: 0.444 ms at D = 128 (1.24
// PFLOP/s, 75% of the card's measured matrix rate; 0.51 ms, 1.07 of 1.39, in long runs
// under the power limit), 0.384 ms at D = 64, 0.176 ms with a window of 1024.
//
// Rows of V that no row of the sequence sees are set to zero in shared memory before
// they meet P's zeros; keys need none of that, their scores are replaced.
#pragma once

#include "attn.cuh"

namespace bl {

constexpr int kAfThreads = 320;                        // 2 x 4 softmax warps, MMA warp, TMA warp
constexpr int kAfRing = 4;                             // K and V tiles in flight
constexpr int kAfParts = 2;                            // parts in which a row of P is handed over
constexpr float kAfLazy = 8.f;                         // log2 of the growth that is let pass
// A row maximum m = round(c x) beyond which the exact product c x less m, what the exponentials
// take, may pass P's room: m's last place is a half there. A maximum of kLow needs nothing.
constexpr float kAfFar = 4194304.f;
constexpr float kLow = -3.4028235e38f;                 // a row maximum before anything is seen: the lowest finite number

struct alignas(64) AttnMaps {
  CUtensorMap q, k, v;                                 // [rows, heads, D], boxes of 128 rows x 64 elements
};

// An average of values of type T is within T's range. P is rounded and the row's sum is not, so
// that the quotient may pass the largest number by 2^-11 of it, which float16 stores as Inf
// already (in bfloat16 sums of such values pass float32 first): it is held at the largest number.
// Infinities and NaN stay.
template <typename T> __device__ __forceinline__ float within_type(float x) {
  if (!std::is_same<T, __half>::value) return x;
  return fabsf(x) < 66000.f ? fminf(fmaxf(x, -65504.f), 65504.f) : x;
}

template <int DP>
struct AfCfg {
  static constexpr int kTile = 128 * DP * 2;           // a 128-row operand tile: DP / 64 boxes of 128 x 128 bytes
  static constexpr int kSmem = (2 + kAfRing) * kTile + 1024;
};

__device__ __forceinline__ void tma_rows(void* dst, const CUtensorMap* map, int boxes, int head, int row, uint64_t* bar) {
  for (int i = 0; i < boxes; ++i)
    tma_load_3d(static_cast<unsigned char*>(dst) + i * 16384, map, i * 64, head, row, bar);
}

// kind::f16 instruction descriptor: float32 accumulator, A K-major, B K-major or (mn) MN-major.
template <typename T> __host__ __device__ constexpr uint32_t umma_idesc_16(int m, int n, bool mn) {
  const uint32_t fmt = std::is_same<T, __half>::value ? 0u : 1u;
  return (1u << 4) | (fmt << 7) | (fmt << 10) | (mn ? 1u << 16 : 0u) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}
// The issuing warp stays whole: every lane computes the (uniform) operands and one elected
// lane issues.  Behind a branch on the lane, the operands' way into the uniform registers
// that the instruction reads took about 90 cycles per product.
__device__ __forceinline__ void umma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void umma_commit_warp(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// A value that every lane of the warp holds, known to be uniform.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
// MN-major operand: rows (contraction index) of 128 bytes with 128-byte swizzle, 8-row
// groups 1024 bytes apart; the next 64 columns a box of 128 rows further.
__device__ __forceinline__ uint64_t umma_desc_mn_sw128(uint32_t addr) {
  return uint64_t((addr & 0x3FFFFu) >> 4) | (uint64_t(16384 >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// D (128 x 128) = A B^T over DP elements, both tiles K-major in shared memory.
template <typename T, int DP>
__device__ __forceinline__ void mma_qk(uint32_t d, uint32_t a, uint32_t b) {
  constexpr uint32_t idesc = umma_idesc_16<T>(128, 128, false);
#pragma unroll
  for (int k = 0; k < DP / 16; ++k) {
    const uint32_t off = uint32_t(k / 4) * 16384u + uint32_t(k % 4) * 32u;
    umma_f16(d, umma_desc_k_sw128(a + off), umma_desc_k_sw128(b + off), idesc, k > 0 ? 1u : 0u);
  }
}
// D (128 x DP) += P B over kRows rows of B: P in tensor memory, B MN-major in shared memory.
template <typename T, int DP, int kRows>
__device__ __forceinline__ void mma_pv_part(uint32_t d, uint32_t p, uint32_t b, bool acc) {
  constexpr uint32_t idesc = umma_idesc_16<T>(128, DP, true);
#pragma unroll
  for (int k = 0; k < kRows / 16; ++k)
    umma_f16_ts(d, p + uint32_t(k) * 8u, umma_desc_mn_sw128(b + uint32_t(k) * 2048u), idesc, acc || k > 0 ? 1u : 0u);
}

// Zeros rows [r0, r1) of a 128-row tile (one warp), visible to the tensor core after it.
__device__ __forceinline__ void zero_rows(unsigned char* tile, int boxes, int r0, int r1, int lane) {
  r0 = max(r0, 0);
  r1 = min(r1, 128);
  for (int i = 0; i < boxes; ++i)
    for (int e = r0 * 8 + lane; e < r1 * 8; e += 32) *reinterpret_cast<uint4*>(tile + i * 16384 + e * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}
// Rows of the key block at j0 that no query of the sequence sees, and that lie in the
// buffer: behind the sequence's end, or between the first tokens and the first window.
__device__ __forceinline__ void zero_dead_keys(unsigned char* tile, int boxes, int j0, const Seq& s, int window, int sinks,
                                               int64_t tk, int lane) {
  if (j0 + 128 > s.nk && s.k0 + s.nk < tk) zero_rows(tile, boxes, s.nk - j0, 128, lane);
  const int first = s.nk - s.nq - window + 1;         // of the first query's window
  if (window != 0 && first > sinks && j0 < first && j0 + 128 > sinks) zero_rows(tile, boxes, sinks - j0, first - j0, lane);
}

// The 128-key blocks that the rows at positions lo .. hi see: `lead` from key 0, the others
// from key `from` on, which is the first window's first key itself and not the multiple of
// 128 below it (a copy may start at any row): a block less for most windows.
struct Blocks {
  int lead, from, n;
  __device__ __forceinline__ int at(int i) const { return i < lead ? i * 128 : from + (i - lead) * 128; }
};
__device__ __forceinline__ Blocks key_blocks(int lo, int hi, int window, int sinks) {
  Blocks b;
  b.lead = b.from = 0;
  if (window != 0 && lo >= window) {
    const int ws = lo - window + 1;
    b.lead = (min(sinks, ws) + 127) / 128;
    b.from = max(b.lead * 128, ws);
  }
  b.n = hi < 0 ? 0 : b.lead + (max(0, hi + 1 - b.from) + 127) / 128;
  return b;
}

template <typename T, int DP>
__global__ void __launch_bounds__(kAfThreads, 1)
attn_fwd_kernel(const __grid_constant__ AttnMaps maps, const AttnArgs a) {
  using C = AfCfg<DP>;
  extern __shared__ unsigned char af_smem[];
  __shared__ uint64_t q_full, kv_full[kAfRing], kv_empty[kAfRing], s_full[2], p_full[2][kAfParts], o_full[2], drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_err;
  constexpr int kBoxes = DP / 64;
  constexpr float kShift = std::is_same<T, __half>::value ? 7.f : 0.f;
  volatile int* err = &s_err;
  if (blockIdx.x >= unsigned(a.work)) return clear_rest(a, kAfThreads);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;

  // the work: heads (or a pair of them) fastest, long row blocks first
  const int group = a.Hq / a.Hkv;
  const bool two = (group & 1) == 0;                   // two heads of a group, else two row blocks
  const int units = two ? a.Hq / 2 : a.Hq, rows = two ? 128 : 256;
  const int nblk = (a.max_q + rows - 1) / rows;
  const int unit = int(blockIdx.x % unsigned(units)), rest = int(blockIdx.x / unsigned(units));
  const int i0 = (nblk - 1 - rest / a.B) * rows;
  Seq s;
  if (!load_seq(a, rest % a.B, s, false) || i0 >= s.nq) return;
  s.q0 = uniform(s.q0);
  s.nq = uniform(s.nq);
  s.k0 = uniform(s.k0);
  s.nk = uniform(s.nk);
  const int off = s.nk - s.nq;
  const int h0 = two ? 2 * unit : unit, hk = h0 / group;
  const int r1 = two ? i0 : i0 + 128;                  // first row of tile 1
  const Blocks blocks = key_blocks(i0 + off, min(i0 + rows, s.nq) - 1 + off, a.window, a.sinks);
  // whether tile t (first row r) sees any key of the block at j0
  auto active = [&](int r, int j0) {
    return r < s.nq && j0 <= min(r + 128, s.nq) - 1 + off && (a.window == 0 || j0 + 127 > r + off - a.window || j0 < a.sinks);
  };

  const uint32_t base = (smem_u32(af_smem) + 1023u) & ~1023u;
  unsigned char* smem = af_smem + (base - smem_u32(af_smem));
  if (tid == 0) {
    s_err = 0;
    mbar_init(&q_full, 1);
    mbar_init(&drain, 1);
    for (int i = 0; i < kAfRing; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      for (int i = 0; i < kAfParts; ++i) mbar_init(&p_full[t][i], 4);
      mbar_init(&o_full[t], 1);
    }
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uint32_t(uniform(int(s_tmem)));                        // S0, S1, O0, O1: 128 columns each
  unsigned char* ring = smem + 2 * C::kTile;

  if (warp == 9) {
    if (lane == 0 && blocks.n > 0) {
      mbar_arrive_expect_tx(&q_full, (r1 < s.nq ? 2 : 1) * C::kTile);
      tma_rows(smem, &maps.q, kBoxes, h0, s.q0 + i0, &q_full);
      if (r1 < s.nq) tma_rows(smem + C::kTile, &maps.q, kBoxes, two ? h0 + 1 : h0, s.q0 + r1, &q_full);
      int n = 0;
      for (; n < 2 * blocks.n; ++n) {                  // K of block 0, V of block 0, K of block 1, ...
        const int st = n % kAfRing;
        if (n >= kAfRing && !mbar_wait_near(&kv_empty[st], uint32_t(n / kAfRing - 1) & 1u)) *err = 1;
        if (*err) break;
        mbar_arrive_expect_tx(&kv_full[st], C::kTile);
        tma_rows(ring + st * C::kTile, (n & 1) ? &maps.v : &maps.k, kBoxes, hk, s.k0 + blocks.at(n >> 1), &kv_full[st]);
      }
      if (*err) {                                      // leave no copy in flight behind
        mbar_wait_near(&q_full, 0u);
        for (int i = max(0, n - kAfRing); i < n; ++i) mbar_wait_near(&kv_full[i % kAfRing], uint32_t(i / kAfRing) & 1u);
      }
    }
  } else if (warp == 8) {
    bool good = true;                                    // the same in every lane
    auto wait = [&](uint64_t* bar, int parity) {
      if (good && __any_sync(0xffffffffu, !mbar_wait_near(bar, uint32_t(parity) & 1u))) {
        good = false;
        *err = 1;
      }
      tc_fence_after();
    };
    auto wait_kv = [&](int n) {
      wait(&kv_full[n % kAfRing], n / kAfRing);
      return base + uint32_t((2 + n % kAfRing) * C::kTile);
    };
    int cnt[2] = {0, 0};
    if (blocks.n > 0) {
      wait(&q_full, 0);
      const uint32_t k = wait_kv(0);
      if (good) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (active(t ? r1 : i0, blocks.at(0))) {
            mma_qk<T, DP>(tmem + t * 128, base + t * C::kTile, k);
            umma_commit_warp(&s_full[t]);
          }
        umma_commit_warp(&kv_empty[0]);
      }
    }
    for (int j = 0; j < blocks.n && good; ++j) {
      const int j0 = blocks.at(j), nv = 2 * j + 1, nk = 2 * j + 2;
      const uint32_t v = wait_kv(nv);
      zero_dead_keys(ring + (nv % kAfRing) * C::kTile, kBoxes, j0, s, a.window, a.sinks, a.Tk, lane);
      const bool more = j + 1 < blocks.n;
      const int j1 = more ? blocks.at(j + 1) : 0;
      const uint32_t k = more ? wait_kv(nk) : 0;         // loaded long since: not on the way from P to the next S
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int r = t ? r1 : i0;
        if (active(r, j0)) {
#pragma unroll
          for (int part = 0; part < kAfParts; ++part) {
            wait(&p_full[t][part], cnt[t]);
            if (good)
              mma_pv_part<T, DP, 128 / kAfParts>(tmem + 256 + t * 128, tmem + t * 128 + part * (64 / kAfParts),
                                                 v + part * (16384 / kAfParts), cnt[t] > 0 || part > 0);
          }
          umma_commit_warp(&o_full[t]);
          ++cnt[t];
        }
        if (more && good && active(r, j1)) {
          mma_qk<T, DP>(tmem + t * 128, base + t * C::kTile, k);   // in order behind the product that reads P
          umma_commit_warp(&s_full[t]);
        }
      }
      umma_commit_warp(&kv_empty[nv % kAfRing]);
      if (more) umma_commit_warp(&kv_empty[nk % kAfRing]);
    }
    umma_commit_warp(&drain);
  } else {
    const int t = warp >> 2, row = (warp & 3) * 32 + lane, r = t ? r1 : i0, i = r + row;
    const int h = two ? h0 + t : h0;
    const int p = i < s.nq ? i + off : -1;             // this row's position
    const int lo = a.window ? p - a.window + 1 : 0;
    const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
    const uint32_t st = tmem + lanes + t * 128, ot = tmem + lanes + 256 + t * 128;
    const float c = a.scale * kLog2e;
    float m = kLow, l = 0.f, lim = INFINITY;           // maximum, sum, what a block's maximum has to pass to raise m
    int cnt = 0;
    bool fine = true;
    for (int j = 0; j < blocks.n && r < s.nq; ++j) {
      const int j0 = blocks.at(j);
      if (!active(r, j0)) continue;
      fine = mbar_wait_near(&s_full[t], uint32_t(cnt) & 1u) && !*err;
      if (__any_sync(0xffffffffu, !fine)) {
        *err = 1;
        break;
      }
      tc_fence_after();
      float x[128];
      uint32_t* w = reinterpret_cast<uint32_t*>(x);
#pragma unroll
      for (int u = 0; u < 4; ++u) tmem_ld32(st + u * 32, w + u * 32);
      tmem_ld_wait();
      // the block is masked for some row of the tile
      if (j0 + 127 > r + off || (a.window != 0 && j0 <= min(r + 128, s.nq) - 1 + off - a.window && j0 + 128 > a.sinks)) {
        const int top = p - j0, bot = lo - j0, lead = a.window ? a.sinks - j0 : 0;
#pragma unroll
        for (int f = 0; f < 128; f += 32) {
          const uint32_t seen = seen_bits(f, top, bot, lead);
#pragma unroll
          for (int u = 0; u < 32; ++u)
            if (!(seen & (1u << u))) x[f + u] = -INFINITY;
        }
      }
      float top4[4] = {x[0], x[1], x[2], x[3]};          // four chains: one would be 64 dependent steps
#pragma unroll
      for (int u = 4; u < 124; u += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) top4[e] = fmaxf(fmaxf(x[u + 2 * e], x[u + 2 * e + 1]), top4[e]);
#pragma unroll
      for (int e = 0; e < 4; ++e) top4[e] = fmaxf(x[124 + e], top4[e]);
      const float mx = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * c;
      float less = m;                                    // what the exponents take off
      if (cnt == 0 || __any_sync(0xffffffffu, mx > lim)) {
        const float up = fmaxf(mx, m), f = exp2_approx(m - up);
        m = less = up;
        const bool far = p >= 0 && fabsf(m) > kAfFar && m > kLow;
        lim = p < 0 ? INFINITY : far ? -INFINITY : m + kAfLazy;   // (a row behind the sequence's end is another's)
        if (cnt > 0) {
          l *= f;
          fine = mbar_wait_near(&o_full[t], uint32_t(cnt - 1) & 1u);
          if (__any_sync(0xffffffffu, !fine)) {
            *err = 1;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int u = 0; u < DP / 32; ++u) {
            uint32_t o[32];
            tmem_ld32(ot + u * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(ot + u * 32, o);
          }
        }
        if (__any_sync(0xffffffffu, far)) {              // the difference first
          const float by = far ? c : 1.f, off = far ? m : 0.f, back = far ? 1.f / c : 1.f;
#pragma unroll
          for (int u = 0; u < 128; ++u) x[u] = (x[u] * by - off) * back;
          less = m - off;
        }
      }
      const float sub = kShift - less;
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int part = 0; part < kAfParts; ++part) {      // the tensor core starts on the first keys meanwhile
        constexpr int kKeys = 128 / kAfParts;
#pragma unroll
        for (int u = part * kKeys; u < (part + 1) * kKeys; u += 2) {
          const float2 y = fma2(make_float2(x[u], x[u + 1]), make_float2(c, c), make_float2(sub, sub));
          const float2 e = make_float2(exp2_approx(y.x), exp2_approx(y.y));
          sum[(u >> 1) & 1] = add2(sum[(u >> 1) & 1], e);
          w[u >> 1] = pack2<T>(e.x, e.y);
        }
        tmem_st32(st + part * 32, w + part * 32);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t][part]);
      }
      sum[0] = add2(sum[0], sum[1]);
      l += sum[0].x + sum[0].y;
      ++cnt;
    }
    if (fine && cnt > 0) {
      fine = mbar_wait_near(&o_full[t], uint32_t(cnt - 1) & 1u) && !*err;
      if (!fine) *err = 1;
      tc_fence_after();
    }
    fine = !__any_sync(0xffffffffu, !fine);
    if (fine && r < s.nq) {
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);     // NaN stays
      // a row that sees a key (its own position's, at least) has a sum, unless its scores passed float32
      uint32_t bad = l < INFINITY && (l > 0.f || p < 0) ? 0u : 1u;
      T* out = static_cast<T*>(a.out) + (int64_t(s.q0 + i) * a.Hq + h) * a.D;
#pragma unroll 1
      for (int u = 0; u < DP / 32; ++u) {
        uint32_t o[32];
        if (cnt > 0) {
          tmem_ld32(ot + u * 32, o);
          tmem_ld_wait();
        }
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          if (i >= s.nq || u * 32 + e >= a.D) break;
          uint32_t y[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const float f0 = l == 0.f ? 0.f : __uint_as_float(o[e + 2 * z]) * inv;
            const float f1 = l == 0.f ? 0.f : __uint_as_float(o[e + 2 * z + 1]) * inv;
            y[z] = pack2<T>(within_type<T>(f0), within_type<T>(f1));
            bad |= not_finite2<T>(y[z]);
          }
          *reinterpret_cast<uint4*>(out + u * 32 + e) = make_uint4(y[0], y[1], y[2], y[3]);
        }
        __syncwarp();
      }
      if (i < s.nq) {
        if (a.lse) a.lse[int64_t(h) * a.Tq + s.q0 + i] = l == 0.f ? -INFINITY : (m - kShift + log2f(l)) * kLn2;
        if (bad) raise_status(kDevNonFinite);
      }
    }
    tc_fence_before();
  }

  __syncthreads();
  if (warp == 8) {
    const bool drained = mbar_wait_near(&drain, 0u);
    if ((!drained || *err) && lane == 0) raise_status(kDevTimeout);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace bl
