// Attention of one new token per sequence over a paged key-value cache.
//
// "ultragraph-1bit 0.12.0" (PyPI): a cached step gives what the full forward
// gives.  Row b: softmax(scale q_b K^T) V over the visible tokens of sequence b.
//
// Bound by memory: every visible key and value is read once, 4 D bytes per token
// and key head, for 4 D operations per query head.  So
//   - the visible 64-token tiles of all sequences and key heads form one line that
//     is cut into equal parts, one per CTA (three or four CTAs an SM: a tile's chain of
//     products, exchanges and exponentials is long, other warps fill it): ragged batches
//     and a single long sequence load every SM alike;
//   - tiles arrive by 16-byte asynchronous copies, kStages in flight, the page of
//     each row looked up two tiles ahead; rows that are not visible are filled with
//     zeros instead of being read;
//   - the scores are taken transposed, S^T = K q^T (keys are the 16-row side of the
//     m16n8k16 matrix instruction, the group's query heads its 8 columns), and so is
//     O^T = V^T P^T: a group of up to 8 heads shares each tile's one trip through
//     shared memory.  The tensor pipe is far from its limit at 8 columns, and
//     tcgen05's tiles (at least 64 rows of one operand, 8 columns of the other, but
//     staged through tensor memory with its own waits) would add latency and no rate;
//   - P keeps float32's precision: it is split into terms of the cache's type (three
//     bfloat16 terms of 8 bits, two float16 terms of 11), each its own product;
//   - each warp keeps the running maximum and sum of its own 16 keys per tile, so the
//     loop has one barrier; warps are joined when a head ends, CTAs by the last one
//     to finish (a counter per head part, reset by it), in the order of the line.
//
// Measured: 64 ragged sequences of up to 8192 tokens (32/8 heads of 128, bfloat16, pages of
// 16) 171 us, 6.3 TB/s, 96% of the card's copy rate; two of 131071 tokens (20/5 heads of
// 64, float16) 64 us, 5.2 TB/s: 59 parts a head are joined at its end; one of 301 tokens
// 8.1 us: a chain of dependent reads (lengths, pages, rows, parts), nothing to overlap it.
// Two CTAs an SM took 195 and 89 us: a tile's chain of products, exchanges and
// exponentials is then the bound, not memory.
#pragma once

#include <type_traits>

#include "attn_common.cuh"

namespace bl {

constexpr int kPaThreads = 128, kPaTile = 64;
constexpr int kPaMaxCtas = 148 * 4;                  // planned for B200's 148 SMs
constexpr int kPaMaxLen = INT32_MAX - (kPaTile - 1);  // the last tile's key numbers still fit 32 bits
constexpr float kPaLow = -3.4028235e38f;             // a maximum before anything is seen: the lowest finite number

struct PaArgs {
  const void *q, *k, *v;
  const int32_t *table, *lens;
  int64_t ldt, pages, B;
  int Hq, Hkv, D, page, window, sinks;
  int most;                 // longest length: the table's ldt * page tokens, and kPaMaxLen at most
  float scale_log2;
  void* out;
  unsigned int* count;      // [kPaMaxCtas]
  float* part;              // [2 kPaMaxCtas][8 NT DP of O, then 8 NT pairs of maximum and sum]
  int group, chunks;        // query heads per key head; ceil(group / (8 NT))
  uint32_t page_magic, page_shift;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <typename T> __device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1);
template <> __device__ __forceinline__ void mma16816<__half>(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk c of row r in a tile with rows of DP elements; the
// xor spreads the 8 rows that one ldmatrix phase reads over all banks.
template <int DP> __device__ __forceinline__ uint32_t pa_off(int r, int c) {
  const int x = DP >= 64 ? (r & 7) : ((r >> 1) & 3);
  return uint32_t(r * DP * 2 + ((c ^ x) << 4));
}

// a / b of values that are not negative; 32 bits where they do (64-bit division is a long
// software routine).
__device__ __forceinline__ int64_t div_near(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
}

// The visible tiles of a sequence of `len` tokens: `lead` of them from tile 0, the
// others from tile `from` on.
struct PaTiles {
  int lead, from, n;
};
__device__ __forceinline__ PaTiles pa_tiles(int len, int window, int sinks) {
  PaTiles t;
  const int all = (len + kPaTile - 1) / kPaTile;
  t.lead = 0;
  t.from = 0;
  if (window != 0 && len > window) {
    const int ws = len - window;
    t.lead = (min(sinks, ws) + kPaTile - 1) / kPaTile;
    t.from = max(t.lead, ws / kPaTile);
  }
  t.n = t.lead + all - t.from;
  return t;
}
__device__ __forceinline__ int pa_len(const PaArgs& a, int64_t b, bool& range) {
  const int n = a.lens[b];
  if (n < 0 || n > a.most) range = true;
  return min(max(n, 0), a.most);
}

template <typename T, int DP, int NT>
struct PaCfg {
  static constexpr int kTileBytes = kPaTile * DP * 2;
  static constexpr int kStage = 2 * kTileBytes;
  static constexpr int kHeads = 8 * NT;
  static constexpr int kPerSm = DP == 128 ? 3 : 4;     // CTAs an SM
  static constexpr int kStages = DP == 128 ? 2 : 3;
  static constexpr int kCtas = 148 * kPerSm;
  static constexpr int kJoinRow = DP + 4;              // a row of O in shared memory: the lanes' heads in banks of their own
  static constexpr int kJoin = kHeads * kJoinRow * 4 > kPaThreads * 16 ? kHeads * kJoinRow * 4 : kPaThreads * 16;   // O, or a float4 a thread
  static constexpr int kSmem = kStages * kStage + kJoin;
};

// Position in the line of tiles: sequence b, key head and chunk (item), tile t of it.
struct PaAt {
  int64_t flat;             // line index of the item's first tile
  int b, item, t, len;      // item = hk * chunks + chunk
  PaTiles tiles;
};

template <typename T, int DP, int NT, typename OutT>
__global__ void __launch_bounds__(kPaThreads, NT == 1 ? PaCfg<T, DP, NT>::kPerSm : 2)
paged_attn_kernel(const PaArgs a) {
  using C = PaCfg<T, DP, NT>;
  extern __shared__ __align__(128) unsigned char pa_smem[];
  unsigned char* smem = pa_smem;
  __shared__ int64_t s_row[C::kStages][kPaTile]; // element offset of each row's head data, -1: not visible
  __shared__ float s_m[4][C::kHeads], s_l[4][C::kHeads];
  __shared__ int64_t s_scan[4];
  __shared__ int64_t s_find[3];                  // sequence of this CTA's first tile, line index of its first tile, its length
  __shared__ int s_empty, s_longest;             // whether a sequence has no tokens; tiles of the longest
  __shared__ int64_t s_line[2];                  // the line's tiles and CTAs, for the joins
  __shared__ float2 s_join[kPaThreads];
  __shared__ unsigned int s_last;
  constexpr int kTerms = std::is_same<T, __half>::value ? 2 : 3;
  constexpr float kShift = std::is_same<T, __half>::value ? 14.f : 0.f;   // keeps float16 terms of small probabilities normal
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = smem_u32(smem);
  float* join = reinterpret_cast<float*>(smem + C::kStages * C::kStage);
  const int items = a.Hkv * a.chunks;
  bool range = false, bad = false;

  // The line: total tiles, this CTA's part, and the sequence where it begins.  Cutting it finer
  // shortens each part by a tile's time (about 1 us) but adds parts to the join of the longest
  // item (about 0.1 us each per 128 columns of four): a part has at least the square root of
  // that item's tiles times the ratio.  One sequence of 12816 tokens, 15/3 heads of 80: 444 CTAs
  // 49 us, 118 CTAs 23 us.  What the rule costs: at D = 64 with up to 8 heads a key head its values
  // no longer fit the registers of four CTAs an SM (36 bytes spilled); two sequences of 131071
  // tokens, whose parts it leaves as they are, went from 62.6 to 64.6 us.
  int64_t total = 0, ctas = 0, lo = 0, hi = 0;
  {
    const int64_t rounds = ceil_div(a.B, kPaThreads);
    int64_t n = 0, x = 0, before = 0;                // of sequence b: line tiles, and up to it within the round
    int len = 0, longest = 0;
    if (tid == 0) s_empty = s_longest = 0;
    auto scan = [&](int64_t b) {                     // returns the round's tiles
      len = b < a.B ? pa_len(a, b, range) : 0;
      n = int64_t(pa_tiles(len, a.window, a.sinks).n) * items;
      x = n;
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();
      if (lane == 31) s_scan[warp] = x;
      if (b < a.B && n == 0) s_empty = 1;
      __syncthreads();
      for (int w = 0; w < warp; ++w) x += s_scan[w];
      return s_scan[0] + s_scan[1] + s_scan[2] + s_scan[3];
    };
    for (int64_t r = 0; r < rounds; ++r) {
      total += scan(r * kPaThreads + tid);
      longest = max(longest, pa_tiles(len, a.window, a.sinks).n);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) atomicMax(&s_longest, longest);
    __syncthreads();
    const float least = sqrtf(float(s_longest) * float(min(a.group, C::kHeads) * (DP / 4)) * (0.1f / 128.f));
    ctas = min(int64_t(gridDim.x), total);
    if (least > 1.f) ctas = min(ctas, max(int64_t(1), int64_t(float(total) / least)));
    if (tid == 0) {
      s_line[0] = total;
      s_line[1] = ctas;
    }
    if (int64_t(blockIdx.x) < ctas) {
      lo = div_near(int64_t(blockIdx.x) * total, ctas);
      hi = div_near((int64_t(blockIdx.x) + 1) * total, ctas);
      for (int64_t r = 0; r < rounds; ++r) {
        const int64_t sum = rounds == 1 ? total : scan(r * kPaThreads + tid);
        const int64_t first = before + x - n;
        if (n > 0 && first <= lo && lo < first + n) {
          s_find[0] = r * kPaThreads + tid;
          s_find[1] = first;
          s_find[2] = len;
        }
        before += sum;
        if (before > lo) break;
      }
      __syncthreads();
    }
  }
  // rows without tokens are nobody's tiles: zeros, from the CTAs in turn
  auto empty_rows = [&]() {
    for (int64_t b = blockIdx.x; s_empty && b < a.B; b += gridDim.x)
      if (pa_len(a, b, range) == 0)
        for (int i = tid; i < a.Hq * a.D; i += kPaThreads)
          static_cast<OutT*>(a.out)[b * a.Hq * a.D + i] = from_f32<OutT>(0.f);
    if (range) raise_status(kDevRange);
  };
  if (int64_t(blockIdx.x) >= ctas) {
    empty_rows();
    return;
  }

  auto enter = [&](PaAt& p, int b, int64_t first, int len, int64_t x) {   // line index x, in sequence b whose tiles begin at first
    p.b = b;
    p.len = len;
    p.tiles = pa_tiles(p.len, a.window, a.sinks);
    p.item = int(div_near(x - first, p.tiles.n));
    p.flat = first + int64_t(p.item) * p.tiles.n;
    p.t = int(x - p.flat);
  };
  auto advance = [&](PaAt& p) {                                      // to the next tile of the line
    if (++p.t < p.tiles.n) return;
    p.t = 0;
    p.flat += p.tiles.n;
    if (++p.item < items) return;
    p.item = 0;
    do {
      if (++p.b >= a.B) return;
      p.len = pa_len(a, p.b, range);
      p.tiles = pa_tiles(p.len, a.window, a.sinks);
    } while (p.tiles.n == 0);
  };
  // Thread tid looks up where row tid % 64 of a tile is, in two steps so that the page
  // number's way from memory overlaps a tile's work
  struct Pending {
    int in, page;                                    // the row's place within its page's head, -1: not visible; the page
  };
  auto look_up = [&](const PaAt& p) {
    Pending d;
    d.in = -1;
    d.page = 0;
    const int t = p.t < p.tiles.lead ? p.t : p.t - p.tiles.lead + p.tiles.from;
    const int j = t * kPaTile + (tid & (kPaTile - 1));
    if (j < p.len && sees(p.len - 1, j, a.window, a.sinks)) {
      const uint32_t n = a.page == 1 ? uint32_t(j) : __umulhi(uint32_t(j), a.page_magic) >> a.page_shift;
      d.in = j - int(n) * a.page;
      d.page = a.table[int64_t(p.b) * a.ldt + n];
    }
    return d;
  };
  auto place = [&](const Pending& d, int head, int tile) {
    int64_t off = -1;
    if (d.in >= 0) {
      if (d.page < 0 || d.page >= a.pages) range = true;
      else off = ((int64_t(d.page) * a.Hkv + head) * a.page + d.in) * a.D;
    }
    s_row[tile % C::kStages][tid & (kPaTile - 1)] = off;
  };
  constexpr int kRowChunks = DP / 8, kRowStep = kPaThreads / kRowChunks;
  const int my_chunk = tid % kRowChunks, my_row = tid / kRowChunks;
  auto issue = [&](int stage) {
    if (8 * my_chunk >= a.D) return;
    const uint32_t kd = base + stage * C::kStage, vd = kd + C::kTileBytes;
#pragma unroll
    for (int i = 0; i < kPaTile / kRowStep; ++i) {
      const int r = my_row + i * kRowStep;
      const int64_t off = s_row[stage][r];
      const int n = off < 0 ? 0 : 16;
      const int64_t e = off < 0 ? 0 : off + 8 * my_chunk;
      const uint32_t d = pa_off<DP>(r, my_chunk);
      cp_async16(kd + d, static_cast<const T*>(a.k) + e, n);
      cp_async16(vd + d, static_cast<const T*>(a.v) + e, n);
    }
  };

  if (a.D < DP) {                                    // columns past D: zeros, never written again
    const int pad = (DP - a.D) / 8;
    for (int i = tid; i < C::kStages * 2 * kPaTile * pad; i += kPaThreads) {
      const int r = i / pad, c = a.D / 8 + i - r * pad;            // row of all stages' tiles, K and V
      *reinterpret_cast<uint4*>(smem + (r / kPaTile) * C::kTileBytes + pa_off<DP>(r % kPaTile, c)) = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
  }

  PaAt cur, load;
  enter(cur, int(s_find[0]), s_find[1], int(s_find[2]), lo);
  load = cur;
  const int n = int(hi - lo);                        // tiles of this CTA
  // the first tiles' rows all at once (threads 0..63 the even ones, 64..127 the odd ones)
  {
    Pending d[(C::kStages + 1) / 2];
    int head[C::kStages];
#pragma unroll
    for (int t = 0; t < C::kStages; ++t) {
      head[t] = load.item / a.chunks;
      if (t < n && (tid / kPaTile) == (t & 1)) d[t / 2] = look_up(load);
      if (t < n) advance(load);
    }
#pragma unroll
    for (int t = 0; t < C::kStages; ++t)
      if (t < n && (tid / kPaTile) == (t & 1)) place(d[t / 2], head[t], t);
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < C::kStages - 1; ++t) {
    if (t < n) issue(t);
    cp_async_commit();
  }
  Pending next;                                      // of tile kStages, then of those after it
  next.in = -1;
  if (tid < kPaTile && C::kStages < n) next = look_up(load);

  // per-lane state: heads 2 (lane % 4) + {0, 1} of each 8
  float m[NT][2], l[NT][2], o[DP / 16][NT][4];
  uint32_t qf[DP / 16][NT][2];
  const int hpair = (lane & 3) * 2;
  auto begin_item = [&]() {
    const int hk = cur.item / a.chunks, ch = cur.item - hk * a.chunks;
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      const int hg = ch * C::kHeads + u * 8 + (lane >> 2);      // head in the group: the B operand's column
      const T* q = static_cast<const T*>(a.q) + (int64_t(cur.b) * a.Hq + hk * a.group + hg) * a.D;
#pragma unroll
      for (int ks = 0; ks < DP / 16; ++ks)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int d = ks * 16 + half * 8 + hpair;
          qf[ks][u][half] = hg < a.group && d < a.D ? *reinterpret_cast<const uint32_t*>(q + d) : 0u;
        }
      m[u][0] = m[u][1] = kPaLow;
      l[u][0] = l[u][1] = 0.f;
#pragma unroll
      for (int i = 0; i < DP / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][u][e] = 0.f;
    }
  };
  begin_item();
  int seg_first = cur.t;                             // first tile of this segment within the item

  for (int it = 0; it < n; ++it) {
    cp_async_wait<C::kStages - 2>();
    __syncthreads();
    if (it + C::kStages - 1 < n) issue((it + C::kStages - 1) % C::kStages);
    cp_async_commit();
    // the rows of tile it + kStages, asked for a tile ago, into the place of tile it's
    if (it + C::kStages < n) {
      if (tid < kPaTile) place(next, load.item / a.chunks, it + C::kStages);
      advance(load);
      if (tid < kPaTile && it + C::kStages + 1 < n) next = look_up(load);
    }

    const uint32_t ks_base = base + (it % C::kStages) * C::kStage, vs_base = ks_base + C::kTileBytes;
    const int r0 = warp * 16;
    float s[NT][4];
#pragma unroll
    for (int u = 0; u < NT; ++u) s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < DP / 16; ++ks) {
      uint32_t f[4];
      ldsm4(f, ks_base + pa_off<DP>(r0 + (lane & 15), 2 * ks + (lane >> 4)));
#pragma unroll
      for (int u = 0; u < NT; ++u) mma16816<T>(s[u], f, qf[ks][u][0], qf[ks][u][1]);
    }
    const int tile = cur.t < cur.tiles.lead ? cur.t : cur.t - cur.tiles.lead + cur.tiles.from;
    const int j = tile * kPaTile + r0 + (lane >> 2);
    const bool v0 = j < cur.len && sees(cur.len - 1, j, a.window, a.sinks);
    const bool v1 = j + 8 < cur.len && sees(cur.len - 1, j + 8, a.window, a.sinks);
    uint32_t pf[NT][kTerms][2];
#pragma unroll
    for (int u = 0; u < NT; ++u) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x0 = v0 ? s[u][e] * a.scale_log2 : -INFINITY, x1 = v1 ? s[u][2 + e] * a.scale_log2 : -INFINITY;
        float t = fmaxf(x0, x1);
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
        if (t > m[u][e]) {                           // the same for the eight lanes of a column
          const float f = exp2_approx(m[u][e] - t);
          m[u][e] = t;
          l[u][e] *= f;
#pragma unroll
          for (int i = 0; i < DP / 16; ++i) {
            o[i][u][e] *= f;
            o[i][u][2 + e] *= f;
          }
        }
        s[u][e] = exp2_approx(x0 - m[u][e] + kShift);
        s[u][2 + e] = exp2_approx(x1 - m[u][e] + kShift);
        l[u][e] += s[u][e] + s[u][2 + e];
      }
#pragma unroll
      for (int k = 0; k < kTerms; ++k) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t w = pack2<T>(s[u][2 * half], s[u][2 * half + 1]);
          const float2 back = unpack2<T>(w);
          s[u][2 * half] -= back.x;
          s[u][2 * half + 1] -= back.y;
          pf[u][k][half] = movm_t(w);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {
      uint32_t f[4];
      ldsm4_t(f, vs_base + pa_off<DP>(r0 + (lane & 7) + ((lane >> 4) << 3), 2 * i + ((lane >> 3) & 1)));
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        // a fresh accumulator: the matrix unit truncates its sums, which would add up over the tiles
        float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = kTerms - 1; k >= 0; --k) mma16816<T>(y, f, pf[u][k][0], pf[u][k][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][u][e] += y[e];
      }
    }

    const bool item_ends = cur.t + 1 == cur.tiles.n;
    if (item_ends || it + 1 == n) {
      // join the warps: statistics first, then O in the order of the warps
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = l[u][e];
          x += __shfl_xor_sync(0xffffffffu, x, 4);
          x += __shfl_xor_sync(0xffffffffu, x, 8);
          x += __shfl_xor_sync(0xffffffffu, x, 16);
          if (lane < 4) {
            s_m[warp][u * 8 + hpair + e] = m[u][e];
            s_l[warp][u * 8 + hpair + e] = x;
          }
        }
      __syncthreads();
      float f[NT][2];
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int h = u * 8 + hpair + e;
          const float top = fmaxf(fmaxf(s_m[0][h], s_m[1][h]), fmaxf(s_m[2][h], s_m[3][h]));
          f[u][e] = exp2_approx(m[u][e] - top);
        }
      for (int w = 0; w < 4; ++w) {
        if (w == warp) {
#pragma unroll
          for (int u = 0; u < NT; ++u)
#pragma unroll
            for (int i = 0; i < DP / 16; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float* d = join + (u * 8 + hpair + (e & 1)) * C::kJoinRow + i * 16 + (lane >> 2) + 8 * (e >> 1);
                const float x = o[i][u][e] * f[u][e & 1];
                *d = w == 0 ? x : *d + x;
              }
        }
        __syncthreads();
      }
      const int hk = cur.item / a.chunks, ch = cur.item - hk * a.chunks;
      const int nh = min(C::kHeads, a.group - ch * C::kHeads);       // live heads
      OutT* out = static_cast<OutT*>(a.out) + (int64_t(cur.b) * a.Hq + hk * a.group + ch * C::kHeads) * a.D;
      if (item_ends && seg_first == 0) {                             // the whole item is this CTA's
        for (int i = tid; i < nh * a.D; i += kPaThreads) {
          const int h = i / a.D, d = i - h * a.D;
          const float top = fmaxf(fmaxf(s_m[0][h], s_m[1][h]), fmaxf(s_m[2][h], s_m[3][h]));
          float sum = 0.f;
          for (int w = 0; w < 4; ++w) sum = fmaf(s_l[w][h], exp2_approx(s_m[w][h] - top), sum);
          const float r = join[h * C::kJoinRow + d] / sum;
          if (!(fabsf(r) < INFINITY)) bad = true;
          out[i] = from_f32<OutT>(r);
        }
      } else {
        // its part to the workspace: slot 0 of the CTA if the item began before it, slot 1 if it goes on
        float* part = a.part + (2 * int64_t(blockIdx.x) + (seg_first == 0 ? 1 : 0)) * C::kHeads * (DP + 2);
        for (int i = tid; i < nh * DP / 4; i += kPaThreads)
          __stcg(reinterpret_cast<float4*>(part) + i,
                 *reinterpret_cast<const float4*>(join + i / (DP / 4) * C::kJoinRow + i % (DP / 4) * 4));
        for (int h = tid; h < nh; h += kPaThreads) {
          const float top = fmaxf(fmaxf(s_m[0][h], s_m[1][h]), fmaxf(s_m[2][h], s_m[3][h]));
          float sum = 0.f;
          for (int w = 0; w < 4; ++w) sum = fmaf(s_l[w][h], exp2_approx(s_m[w][h] - top), sum);
          __stcg(reinterpret_cast<float2*>(part + C::kHeads * DP) + h, make_float2(top, sum));
        }
        // CTAs of the item: those that hold its first and its last tile, and all between
        const int64_t tiles = s_line[0], share = s_line[1];
        const int64_t c0 = div_near((cur.flat + 1) * share + tiles - 1, tiles) - 1;
        const int64_t c1 = div_near((cur.flat + cur.tiles.n) * share + tiles - 1, tiles) - 1;
        __syncthreads();
        if (tid == 0) {
          // releases what the CTA has written before the barrier, and acquires what the other CTAs have
          unsigned int before;
          asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(a.count + c0) : "memory");
          s_last = before == unsigned(c1 - c0);
          if (s_last) a.count[c0] = 0u;
          if (before > unsigned(c1 - c0)) raise_status(kDevBadWorkspace);
        }
        __syncthreads();
        if (s_last) {
          // a thread takes four columns of every `groups`-th part, eight parts' loads in flight; then
          // the groups are joined through shared memory
          constexpr int kStride = C::kHeads * (DP + 2);
          const int cols = nh * DP / 4, parts = int(c1 - c0) + 1;
          const int groups = min(kPaThreads / min(cols, kPaThreads), parts);
          for (int col0 = 0; col0 < cols; col0 += kPaThreads) {
            const int col = col0 + (groups > 1 ? tid % cols : tid), g = groups > 1 ? tid / cols : 0;
            const bool on = col < cols && g < groups;
            const int h = col * 4 / DP;
            float top = kPaLow, sum = 0.f;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = g; on && k < parts; k += 8 * groups) {
              float2 ps[8];
              float4 px[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int64_t at = c0 + min(k + e * groups, parts - 1);
                const float* p = a.part + (2 * at + (at == c0 ? 1 : 0)) * kStride;
                ps[e] = __ldcg(reinterpret_cast<const float2*>(p + C::kHeads * DP) + h);
                px[e] = __ldcg(reinterpret_cast<const float4*>(p) + col);
              }
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (k + e * groups < parts) {
                  const float t = fmaxf(top, ps[e].x), f0 = exp2_approx(top - t), f1 = exp2_approx(ps[e].x - t);
                  sum = fmaf(sum, f0, ps[e].y * f1);
                  x = make_float4(fmaf(x.x, f0, px[e].x * f1), fmaf(x.y, f0, px[e].y * f1), fmaf(x.z, f0, px[e].z * f1),
                                  fmaf(x.w, f0, px[e].w * f1));
                  top = t;
                }
            }
            __syncthreads();
            if (on && g > 0) {
              reinterpret_cast<float4*>(join)[tid] = x;
              s_join[tid] = make_float2(top, sum);
            }
            __syncthreads();
            if (on && g == 0) {
              for (int o = 1; o < groups; ++o) {
                const float4 y = reinterpret_cast<const float4*>(join)[o * cols + col];
                const float2 ys = s_join[o * cols + col];
                const float t = fmaxf(top, ys.x), f0 = exp2_approx(top - t), f1 = exp2_approx(ys.x - t);
                sum = fmaf(sum, f0, ys.y * f1);
                x = make_float4(fmaf(x.x, f0, y.x * f1), fmaf(x.y, f0, y.y * f1), fmaf(x.z, f0, y.z * f1),
                                fmaf(x.w, f0, y.w * f1));
                top = t;
              }
              const int d = col * 4 - h * DP;
              if (d < a.D) {
                const float inv = 1.f / sum, r[4] = {x.x * inv, x.y * inv, x.z * inv, x.w * inv};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if (!(fabsf(r[e]) < INFINITY)) bad = true;
                  out[h * a.D + d + e] = from_f32<OutT>(r[e]);
                }
              }
            }
          }
        }
      }
      __syncthreads();                                               // join, s_m free again
      if (it + 1 < n) {
        advance(cur);
        begin_item();
        seg_first = 0;
      }
    } else {
      advance(cur);
    }
  }
  if (bad) raise_status(kDevNonFinite);
  empty_rows();
}

}  // namespace bl
