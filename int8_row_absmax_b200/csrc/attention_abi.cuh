// C ABI of the attention operators (declared in include/bitlinear.h): argument
// checks, workspace sizes and launches.  Included by bitlinear_lib.cu, whose
// helpers it uses.
#pragma once

#include <atomic>

#include "attn.cuh"
#include "attn_bwd.cuh"
#include "attn_fwd.cuh"
#include "paged_attn.cuh"
#include "qk_rope.cuh"

namespace bl {
namespace {

constexpr int kAttnMaxD = 128, kRopeMaxD = 256;
constexpr int64_t kAttnMaxRows = int64_t(1) << 29;      // sums of three positions stay within 31 bits

bool half_type(bl_dtype t) { return t == BL_T_F16 || t == BL_T_BF16; }
bool any_type(bl_dtype t) { return t == BL_T_F32 || half_type(t); }
bool int32_max(int64_t v) { return v < (int64_t(1) << 31); }

// Allows a kernel `bytes` of dynamic shared memory, once per device and kernel (the call
// costs about a microsecond, as much as the rest of a small call's host work).
template <typename K>
bool allow_smem(K kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  done.fetch_or(bit, std::memory_order_release);
  return true;
}

// A launch that may begin while the kernel before it on the stream still runs (programmatic
// dependent launch); the kernel itself waits where it has to.
template <typename... P, typename... A>
bool launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...) == cudaSuccess;
}

// ---- norms and rotation ----------------------------------------------------------
bl_status check_rows(const bl_qkv_rows* r, bool values) {
  if (!r) return BL_ERR_INVALID_ARG;
  if (r->M < 0 || r->M >= kAttnMaxRows || r->Hq < 1 || r->Hkv < 1 || r->Hq > 65535 || r->Hkv > 65535 ||
      r->Hq % r->Hkv != 0)
    return BL_ERR_INVALID_ARG;
  if (r->D < 8 || r->D % 8 != 0 || r->D > kRopeMaxD) return BL_ERR_INVALID_ARG;
  if (r->R < 0 || r->R % 8 != 0 || r->R > r->D || (r->interleaved != 0 && r->interleaved != 1)) return BL_ERR_INVALID_ARG;
  if (!eps_ok(r->eps)) return BL_ERR_INVALID_ARG;
  if (r->R > 0 && r->P < 1) return BL_ERR_INVALID_ARG;
  if (r->M == 0) return BL_OK;
  if (!r->q || !r->k || (values && !r->v) || (r->R > 0 && (!r->pos || !r->table))) return BL_ERR_INVALID_ARG;
  const int64_t wq = int64_t(r->Hq) * r->D, wk = int64_t(r->Hkv) * r->D;
  if (r->ldq < wq || r->ldk < wk || (values && r->ldv < wk)) return BL_ERR_INVALID_ARG;
  if (r->ldq % 4 != 0 || r->ldk % 4 != 0 || (values && r->ldv % 4 != 0)) return BL_ERR_ALIGNMENT;
  if (!is_aligned(r->q, 16) || !is_aligned(r->k, 16) || (values && !is_aligned(r->v, 16))) return BL_ERR_ALIGNMENT;
  if (!is_aligned(r->gq, 16) || !is_aligned(r->gk, 16)) return BL_ERR_ALIGNMENT;
  if (r->R > 0 && (!is_aligned(r->table, 16) || !is_aligned(r->pos, 4))) return BL_ERR_ALIGNMENT;
  return BL_OK;
}

QrArgs rows_args(const bl_qkv_rows* r) {
  QrArgs a;
  memset(&a, 0, sizeof(a));
  a.M = r->M;
  a.Hq = r->Hq;
  a.Hkv = r->Hkv;
  a.D = r->D;
  a.q = r->q;
  a.k = r->k;
  a.v = r->v;
  a.ldq = r->ldq;
  a.ldk = r->ldk;
  a.ldv = r->ldv;
  a.pos = r->pos;
  a.table = r->table;
  a.P = r->P;
  a.R = r->R;
  a.interleaved = r->interleaved;
  a.gq = r->gq;
  a.gk = r->gk;
  a.eps = r->eps;
  a.page = 1;
  return a;
}

// Lanes that share a head: the power of two from 4 to 32 that covers D / 8.
int rows_lanes(int D) { return D <= 32 ? 4 : D <= 64 ? 8 : D <= 128 ? 16 : 32; }

// Whether rows go through a ring kernel, whose items are up to `per` heads of a token: once
// the items fill the warps that an SM holds of it twice, and are themselves half full.  Both
// sides measured, ring kernel against the one of single heads, us: 48 heads of 128, 512
// tokens 6.6 / 6.0, 768 tokens 7.4 / 7.9, 4096 tokens 29.6 / 30.3; their gradients 256 tokens
// 9.2 / 8.9, 512 tokens 11.5 / 12.7, 4096 tokens 44 / 76; 30 heads of 64, 2048 tokens 7.2 /
// 7.1, 26041 tokens 56 / 65; 12 heads of 32 (items 3/8 full), 130208 tokens 86 / 72.
bool rows_by_ring(int64_t M, int heads, int per, int64_t warps) {
  const int64_t chunks = ceil_div(heads, per);
  return M * chunks >= 2 * warps && 2 * int64_t(heads) >= chunks * per;
}

// The kernel and CTAs of a call.  A ring kernel's CTAs share the items out evenly, so they are no
// more than run at once: two an SM, by registers (120 of 256 threads) at every head size, though
// the rings of small heads would leave room for more. Two against as many as the rings' room
// allows (three here), us: 8192 tokens, 48 heads of 80: 51.9 / 58.7; of 96: 52.3 / 59.2; 16384
// tokens, 48 heads of 40: 49.4 / 56.7.
struct RowsPlan {
  bool ring;
  unsigned grid;
};
RowsPlan rows_plan(int64_t M, int heads, int D) {
  const int lanes = rows_lanes(D), per = 128 / lanes;
  const int64_t ctas = int64_t(num_sms()) * 2;
  if (!rows_by_ring(M, heads, per, ctas * kQrRingWarps)) return {false, grid_for(M * heads, kQrThreads / lanes, 16)};
  const int64_t grid = ceil_div(M * ceil_div(heads, per), kQrRingWarps);
  return {true, unsigned(grid < ctas ? grid : ctas)};
}

template <typename T, bool kAppend, int kLanes>
bl_status launch_rows(const QrArgs& a, cudaStream_t st) {
  static_assert(QrRing<kLanes>::kHeads == 128 / kLanes, "as the plan counts items");
  const RowsPlan p = rows_plan(a.M, a.Hq + 2 * a.Hkv, a.D);
  if (p.ring) {
    static std::atomic<uint64_t> done{0};
    constexpr int kPerD = kQrRingWarps * kQrRing * QrRing<kLanes>::kHeads * 4;   // bytes per element of a head: 96 KB at most
    if (!allow_smem(qk_norm_rope_ring_kernel<T, kAppend, kLanes>, kPerD * 8 * kLanes, done)) return BL_ERR_CUDA;
    qk_norm_rope_ring_kernel<T, kAppend, kLanes><<<p.grid, 32 * kQrRingWarps, kPerD * a.D, st>>>(a);
  } else {
    qk_norm_rope_kernel<T, kAppend, kLanes><<<p.grid, kQrThreads, 0, st>>>(a);
  }
  return launch_status();
}
template <typename T, bool kAppend>
bl_status launch_norm_rope(const QrArgs& a, cudaStream_t st) {
  switch (rows_lanes(a.D)) {
    case 4: return launch_rows<T, kAppend, 4>(a, st);
    case 8: return launch_rows<T, kAppend, 8>(a, st);
    case 16: return launch_rows<T, kAppend, 16>(a, st);
    default: return launch_rows<T, kAppend, 32>(a, st);
  }
}

// CTAs of the backward (and rows of its partial sums): planned for 148 SMs.
constexpr int kQrBackCtas = 148 * 2;
int rows_back_grid(int64_t M, int heads, int D) {
  const int64_t g = ceil_div(M * heads, int64_t(kQrThreads / rows_lanes(D)));
  return int(g < 1 ? 1 : g < kQrBackCtas ? g : kQrBackCtas);
}
RowsPlan rows_back_plan(int64_t M, int heads, int D) {
  const int grid = rows_back_grid(M, heads, D);
  return {rows_by_ring(M, heads, 64 / rows_lanes(D), int64_t(grid) * kQrRingWarps), unsigned(grid)};
}

template <typename T, int kLanes>
bl_status launch_rows_back(const QrArgs& a, cudaStream_t st) {
  static_assert(QrRing<kLanes>::kBackHeads == 64 / kLanes, "as the plan counts items");
  const RowsPlan p = rows_back_plan(a.M, a.Hq + 2 * a.Hkv, a.D);
  if (p.ring) {
    static std::atomic<uint64_t> done{0};
    constexpr int kPerD = kQrRingWarps * kQrRing * QrRing<kLanes>::kBackHeads * (4 + int(sizeof(T)));   // bytes per element of a head
    if (!allow_smem(qk_norm_rope_backward_ring_kernel<T, kLanes>, kPerD * 8 * kLanes, done)) return BL_ERR_CUDA;
    qk_norm_rope_backward_ring_kernel<T, kLanes><<<p.grid, 32 * kQrRingWarps, size_t(kPerD) * a.D, st>>>(a);
  } else {
    qk_norm_rope_backward_kernel<T, kLanes><<<p.grid, kQrThreads, size_t(kQrThreads / kLanes) * 2 * a.D * 4, st>>>(a);
  }
  return launch_status();
}
template <typename T>
bl_status launch_norm_rope_back(const QrArgs& a, cudaStream_t st) {
  switch (rows_lanes(a.D)) {
    case 4: return launch_rows_back<T, 4>(a, st);
    case 8: return launch_rows_back<T, 8>(a, st);
    case 16: return launch_rows_back<T, 16>(a, st);
    default: return launch_rows_back<T, 32>(a, st);
  }
}

bl_status check_cache(const bl_kv_pages* c) {
  if (!c || !c->k || !c->v || !half_type(c->t)) return BL_ERR_INVALID_ARG;
  if (c->pages < 1 || !int32_max(c->pages) || c->page < 1 || c->Hkv < 1 || c->Hkv > 65535) return BL_ERR_INVALID_ARG;
  if (c->D < 8 || c->D % 8 != 0 || !int32_max(int64_t(c->page) * c->D)) return BL_ERR_INVALID_ARG;
  if (!is_aligned(c->k, 16) || !is_aligned(c->v, 16)) return BL_ERR_ALIGNMENT;
  return BL_OK;
}

// ---- attention over packed sequences ----------------------------------------------
bl_status check_attn(const bl_attn_call* c) {
  if (!c || !half_type(c->t)) return BL_ERR_INVALID_ARG;
  if (c->Hq < 1 || c->Hkv < 1 || c->Hq > 65535 || c->Hq % c->Hkv != 0) return BL_ERR_INVALID_ARG;
  if (c->D < 8 || c->D % 8 != 0 || c->D > kAttnMaxD) return BL_ERR_INVALID_ARG;
  if (c->Tq < 0 || c->Tk < 0 || c->Tq >= kAttnMaxRows || c->Tk >= kAttnMaxRows) return BL_ERR_INVALID_ARG;
  if (c->B < 0 || c->B > 65535 || c->max_q < 0 || c->max_k < 0 || c->window < 0 || c->sinks < 0) return BL_ERR_INVALID_ARG;
  if (!std::isfinite(c->scale) || !(c->scale > 0.f)) return BL_ERR_INVALID_ARG;
  if (c->B == 0 || (c->Tq == 0 && c->Tk == 0)) return BL_OK;
  if ((c->Tq > 0 && !c->q) || !c->cu_q || !c->cu_k || (c->Tk > 0 && (!c->k || !c->v))) return BL_ERR_INVALID_ARG;
  const int64_t wq = int64_t(c->Hq) * c->D, wk = int64_t(c->Hkv) * c->D;
  if ((c->Tq > 0 && c->ldq < wq) || (c->Tk > 0 && (c->ldk < wk || c->ldv < wk))) return BL_ERR_INVALID_ARG;
  if (c->ldq % 8 != 0 || c->ldk % 8 != 0 || c->ldv % 8 != 0) return BL_ERR_ALIGNMENT;
  if (!is_aligned(c->q, 16) || !is_aligned(c->k, 16) || !is_aligned(c->v, 16) || !is_aligned(c->cu_q, 4) ||
      !is_aligned(c->cu_k, 4))
    return BL_ERR_ALIGNMENT;
  return BL_OK;
}

// A longest length as the kernels take it: at least one block, to find sequences that are
// longer, and no more than the buffer's rows, which no sequence exceeds (row blocks are counted
// in 32 bits on the device: a length near 2^31 would wrap, and its blocks begin at negative rows).
int longest(int32_t most, int64_t rows) { return int(most < 1 || rows < 1 ? 1 : most < rows ? most : rows); }

AttnArgs attn_args(const bl_attn_call* c) {
  AttnArgs a;
  memset(&a, 0, sizeof(a));
  a.q = c->q;
  a.k = c->k;
  a.v = c->v;
  a.ldq = c->ldq;
  a.ldk = c->ldk;
  a.ldv = c->ldv;
  a.Tq = c->Tq;
  a.Tk = c->Tk;
  a.cu_q = c->cu_q;
  a.cu_k = c->cu_k;
  a.Hq = c->Hq;
  a.Hkv = c->Hkv;
  a.D = c->D;
  a.B = c->B;
  a.max_q = longest(c->max_q, c->Tq);
  a.max_k = longest(c->max_k, c->Tk);
  a.window = c->window >= c->Tk ? 0 : c->window;         // no window at all, then
  a.sinks = c->sinks;
  a.scale = c->scale;
  return a;
}

// 16-bit rows [tokens, heads, D] as boxes of 128 tokens x 64 elements of one head,
// 128-byte swizzle; elements past D and tokens past the buffer read as zero.
bool make_map_rows(CUtensorMap* map, bool f16, const void* base, int64_t ld, int heads, int D, int64_t tokens) {
  EncodeTiledFn fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(heads), cuuint64_t(tokens)};
  const cuuint64_t strides[2] = {cuuint64_t(D) * 2, cuuint64_t(ld) * 2};
  const cuuint32_t box[3] = {64u, 1u, 128u};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
            dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int DP>
bl_status launch_attn_fwd(AttnArgs a, cudaStream_t st) {
  constexpr bool f16 = std::is_same<T, __half>::value;
  AttnMaps maps;
  if (!make_map_rows(&maps.q, f16, a.q, a.ldq, a.Hq, a.D, a.Tq)) return BL_ERR_CUDA;
  if (a.Tk > 0) {
    if (!make_map_rows(&maps.k, f16, a.k, a.ldk, a.Hkv, a.D, a.Tk) ||
        !make_map_rows(&maps.v, f16, a.v, a.ldv, a.Hkv, a.D, a.Tk))
      return BL_ERR_CUDA;
  } else {
    maps.k = maps.v = maps.q;                            // no keys: never loaded from
  }
  constexpr int smem = AfCfg<DP>::kSmem;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(attn_fwd_kernel<T, DP>, smem, done)) return BL_ERR_CUDA;
  const bool two = (a.Hq / a.Hkv) % 2 == 0;
  const int64_t grid = int64_t(two ? a.Hq / 2 : a.Hq) * a.B * ceil_div(a.max_q, two ? 128 : 256);
  if (!int32_max(grid + kClearCtas)) return BL_ERR_UNSUPPORTED;
  a.work = int(grid);
  attn_fwd_kernel<T, DP><<<unsigned(a.work + (a.clear ? kClearCtas : 0)), kAfThreads, smem, st>>>(maps, a);
  return launch_status();
}
template <typename T>
bl_status run_attn(const AttnArgs& a, cudaStream_t st) {
  return a.D <= 64 ? launch_attn_fwd<T, 64>(a, st) : launch_attn_fwd<T, 128>(a, st);
}

// Clears the rows of no sequence by itself.
bl_status clear_alone(AttnArgs a, cudaStream_t st) {
  a.work = 0;
  attn_clear_kernel<<<kClearCtas, 256, 0, st>>>(a);
  return launch_status();
}

// CTAs of the float16 row sums by sequence and key head: no more than run at once (6 an SM),
// whatever the longest lengths say (they may be loose). 4096 tokens, 32/8 heads of 128, 18.6 us,
// one CTA a piece 22.6.
template <int DP> int norm_parts(const bl_attn_call* c) {
  using Ad = AdCfg<__half, DP>;
  const int64_t queries = ceil_div(longest(c->max_q, c->Tq), Ad::tokens(c->Hq / c->Hkv));
  const int64_t keys = ceil_div(longest(c->max_k, c->Tk), Ad::kMost), pairs = int64_t(c->Hkv) * c->B;
  const int64_t parts = queries > keys ? queries : keys, most = 148 * 6 / pairs > 1 ? 148 * 6 / pairs : 1;
  return int(parts < most ? parts : most);
}
int norm_parts(const bl_attn_call* c) { return c->t != BL_T_F16 ? 0 : c->D <= 64 ? norm_parts<64>(c) : norm_parts<128>(c); }
// The backward's workspace: the row sums' norms of each sequence and key head (float16), delta
// [Hq, Tq], the parts of dK and dV.
size_t norm_bytes(const bl_attn_call* c) {
  const size_t bytes = size_t(c->B) * size_t(c->Hkv) * size_t(norm_parts(c)) * 8;
  return align_up(bytes ? bytes : 1);
}
size_t delta_bytes(const bl_attn_call* c) { return align_up(size_t(c->Tq) * size_t(c->Hq) * 4); }

// CTAs that share the query heads of one key block: one as soon as the key blocks fill
// B200's 148 SMs, else as many as fill them twice.  Both sides measured, whole backward: 5
// sequences of up to 777 tokens, 6/2 heads of 80 (70 key blocks), one CTA 74 us (dQ's tail
// not yet overlapped), two 53, three 41; 2 x 4096 tokens, 20/5 heads of
// 128 (320 key blocks), one 549 us, two 604: the parts cost more than the evener load gives.
int dkv_splits(const bl_attn_call* c) {
  const int group = c->Hq / c->Hkv;
  const int64_t ctas = int64_t(c->Hkv) * c->B * ceil_div(longest(c->max_k, c->Tk), 128);
  if (ctas < 1 || ctas >= 148) return 1;
  const int64_t want = 296 / ctas < group ? 296 / ctas : group;
  const int64_t heads = ceil_div(group, want);
  return int(ceil_div(group, heads));
}
// Parts by sequence and key, not by the buffer's row: fewer than 148 key blocks are shared out, so
// that they never pass 39 MB, whatever the buffers hold besides.
size_t dkv_part_bytes(const bl_attn_call* c) {
  const int splits = dkv_splits(c);
  return splits > 1 ? align_up(size_t(splits) * 2 * size_t(c->B) * size_t(longest(c->max_k, c->Tk)) * size_t(c->Hkv) * size_t(c->D) * 4) : 0;
}

template <typename T, int DP>
bl_status launch_attn_bwd(AttnArgs a, float* norms, cudaStream_t st) {
  constexpr bool f16 = std::is_same<T, __half>::value;
  AttnBwdMaps maps;
  const bool queries = a.Tq > 0, keys = a.Tk > 0;
  if (queries && (!make_map_rows(&maps.q, f16, a.q, a.ldq, a.Hq, a.D, a.Tq) ||
                  !make_map_rows(&maps.dout, f16, a.dout, int64_t(a.Hq) * a.D, a.Hq, a.D, a.Tq)))
    return BL_ERR_CUDA;
  if (keys && (!make_map_rows(&maps.k, f16, a.k, a.ldk, a.Hkv, a.D, a.Tk) ||
               !make_map_rows(&maps.v, f16, a.v, a.ldv, a.Hkv, a.D, a.Tk)))
    return BL_ERR_CUDA;
  if (!queries) maps.q = maps.dout = maps.k;             // never loaded from
  if (!keys) maps.k = maps.v = maps.q;
  static std::atomic<uint64_t> done_kv{0}, done_q{0};
  if (!allow_smem(attn_dkv_kernel<T, DP>, AbCfg<DP>::kDkvSmem, done_kv) ||
      !allow_smem(attn_dq_kernel<T, DP>, AbCfg<DP>::kDqSmem, done_q))
    return BL_ERR_CUDA;
  const int64_t gq = int64_t(a.Hq) * a.B * ceil_div(a.max_q, 128), gk = int64_t(a.Hkv) * a.B * ceil_div(a.max_k, 128);
  using Ad = AdCfg<T, DP>;
  const int64_t gd = Ad::kNorms ? int64_t(a.Hkv) * a.B * a.parts : int64_t(grid_for(a.Tq * a.Hq, Ad::kRows, 8));
  if (!int32_max(gq) || !int32_max(gk * a.splits) || !int32_max(gd + kClearCtas)) return BL_ERR_UNSUPPORTED;
  a.work = int(gd);
  if (queries) attn_delta_kernel<T, DP><<<unsigned(a.work + (a.clear ? kClearCtas : 0)), 256, 0, st>>>(a, norms);
  else if (a.clear && clear_alone(a, st) != BL_OK) return BL_ERR_CUDA;
  if (queries && gq > 0) attn_dq_kernel<T, DP><<<unsigned(gq), kAbThreads, AbCfg<DP>::kDqSmem, st>>>(maps, a, norms);
  if (keys && gk > 0) {
    // dK/dV needs nothing of dQ's: its CTAs take the SMs as those of dQ leave them
    const bool early = queries && gq > 0;
    if (early && !launch_early(attn_dkv_kernel<T, DP>, dim3(unsigned(gk * a.splits)), kAbThreads, AbCfg<DP>::kDkvSmem, st,
                               maps, a, norms))
      return BL_ERR_CUDA;
    if (!early) attn_dkv_kernel<T, DP><<<unsigned(gk * a.splits), kAbThreads, AbCfg<DP>::kDkvSmem, st>>>(maps, a, norms);
    if (a.splits > 1 && !launch_early(attn_dkv_join_kernel<T>, dim3(unsigned(gk), 8), 256, 0, st, a)) return BL_ERR_CUDA;
  }
  return launch_status();
}
template <typename T>
bl_status run_attn_backward(const AttnArgs& a, float* norms, cudaStream_t st) {
  return a.D <= 64 ? launch_attn_bwd<T, 64>(a, norms, st) : launch_attn_bwd<T, 128>(a, norms, st);
}

// ---- paged attention ----------------------------------------------------------------
int paged_pad(int D) { return D <= 32 ? 32 : D <= 64 ? 64 : 128; }
int paged_nt(int Hq, int Hkv) { return Hq / Hkv <= 8 ? 1 : 2; }
constexpr size_t kPaCountBytes = 4096;
static_assert(kPaMaxCtas * 4 <= kPaCountBytes, "counters fit");

template <typename T, int DP, int NT, typename OutT>
bl_status launch_paged(const PaArgs& a, cudaStream_t st) {
  constexpr int smem = PaCfg<T, DP, NT>::kSmem;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(paged_attn_kernel<T, DP, NT, OutT>, smem, done)) return BL_ERR_CUDA;
  // no more CTAs than tiles (counted in a double: the product may pass 64 bits)
  const double tiles = double(a.B) * a.Hkv * a.chunks * double(ceil_div(a.most, kPaTile));
  const int grid = tiles < PaCfg<T, DP, NT>::kCtas ? int(tiles) : PaCfg<T, DP, NT>::kCtas;
  paged_attn_kernel<T, DP, NT, OutT><<<unsigned(grid), kPaThreads, smem, st>>>(a);
  return launch_status();
}
template <typename T, int DP, int NT>
bl_status launch_paged_out(const PaArgs& a, bool f32, cudaStream_t st) {
  return f32 ? launch_paged<T, DP, NT, float>(a, st) : launch_paged<T, DP, NT, T>(a, st);
}
template <typename T>
bl_status launch_paged_t(const PaArgs& a, bool f32, cudaStream_t st) {
  const int dp = paged_pad(a.D), nt = paged_nt(a.Hq, a.Hkv);
  if (nt == 1)
    return dp == 32 ? launch_paged_out<T, 32, 1>(a, f32, st)
                    : dp == 64 ? launch_paged_out<T, 64, 1>(a, f32, st) : launch_paged_out<T, 128, 1>(a, f32, st);
  return dp == 32 ? launch_paged_out<T, 32, 2>(a, f32, st)
                  : dp == 64 ? launch_paged_out<T, 64, 2>(a, f32, st) : launch_paged_out<T, 128, 2>(a, f32, st);
}

}  // namespace
}  // namespace bl

extern "C" {

bl_status bl_rope_table(float* table, int64_t P, int R, double base, cudaStream_t stream) {
  if (!table || P < 1 || R < 2 || R % 2 != 0 || !std::isfinite(base) || !(base > 0.0)) return BL_ERR_INVALID_ARG;
  if (P > (int64_t(1) << 40) / R) return BL_ERR_INVALID_ARG;
  if (!is_aligned(table, 4)) return BL_ERR_ALIGNMENT;
  rope_table_kernel<<<grid_for(P * (R / 2), 256), 256, 0, stream>>>(table, P, R / 2, base);
  return launch_status();
}

bl_status bl_qk_norm_rope(const bl_qkv_rows* rows, bl_dtype t, void* q, void* k, void* v, cudaStream_t stream) {
  const bl_status st = check_rows(rows, true);
  if (st != BL_OK) return st;
  if (!any_type(t)) return BL_ERR_INVALID_ARG;
  if (rows->M == 0) return BL_OK;
  if (!q || !k || !v) return BL_ERR_INVALID_ARG;
  if (!is_aligned(q, 16) || !is_aligned(k, 16) || !is_aligned(v, 16)) return BL_ERR_ALIGNMENT;
  QrArgs a = rows_args(rows);
  a.oq = q;
  a.ok = k;
  a.ov = v;
  if (t == BL_T_F32) return launch_norm_rope<float, false>(a, stream);
  return t == BL_T_F16 ? launch_norm_rope<__half, false>(a, stream) : launch_norm_rope<__nv_bfloat16, false>(a, stream);
}

bl_status bl_qk_norm_rope_append(const bl_qkv_rows* rows, void* q, const bl_kv_pages* cache, const int64_t* slots,
                                 cudaStream_t stream) {
  bl_status st = check_rows(rows, true);
  if (st != BL_OK) return st;
  st = check_cache(cache);
  if (st != BL_OK) return st;
  if (cache->Hkv != rows->Hkv || cache->D != rows->D) return BL_ERR_INVALID_ARG;
  if (rows->M == 0) return BL_OK;
  if (!q || !slots) return BL_ERR_INVALID_ARG;
  if (!is_aligned(q, 16) || !is_aligned(slots, 8)) return BL_ERR_ALIGNMENT;
  QrArgs a = rows_args(rows);
  a.oq = q;
  a.ok = cache->k;
  a.ov = cache->v;
  a.slots = slots;
  a.nslots = cache->pages * cache->page;
  a.page = cache->page;
  return cache->t == BL_T_F16 ? launch_norm_rope<__half, true>(a, stream)
                              : launch_norm_rope<__nv_bfloat16, true>(a, stream);
}

int bl_qk_norm_rope_plan(const bl_qkv_rows* rows, int backward, int* ctas) {
  if (check_rows(rows, false) != BL_OK || rows->M == 0) return -1;
  const int heads = rows->Hq + 2 * rows->Hkv;
  const RowsPlan p = backward ? rows_back_plan(rows->M, heads, rows->D) : rows_plan(rows->M, heads, rows->D);
  if (ctas) *ctas = int(p.grid);
  return p.ring ? 1 : 0;
}

size_t bl_qk_norm_rope_backward_workspace_size(const bl_qkv_rows* rows) {
  if (check_rows(rows, false) != BL_OK || rows->M == 0) return 0;
  return align_up(size_t(rows_back_grid(rows->M, rows->Hq + 2 * rows->Hkv, rows->D)) * 2 * size_t(rows->D) * 4);
}

bl_status bl_qk_norm_rope_backward(const bl_qkv_rows* rows, bl_dtype t, const void* dq, const void* dk, const void* dv,
                                   float* dxq, int64_t lddq, float* dxk, int64_t lddk, float* dxv, int64_t lddv,
                                   float* dgq, float* dgk, void* ws, size_t ws_bytes, cudaStream_t stream) {
  bl_status st = check_rows(rows, false);
  if (st != BL_OK) return st;
  if (!any_type(t)) return BL_ERR_INVALID_ARG;
  if (!is_aligned(dgq, 4) || !is_aligned(dgk, 4)) return BL_ERR_ALIGNMENT;
  if (rows->M == 0) {                                  // no rows: the gains' gradients are zero
    if (dgq && cudaMemsetAsync(dgq, 0, size_t(rows->D) * 4, stream) != cudaSuccess) return BL_ERR_CUDA;
    if (dgk && cudaMemsetAsync(dgk, 0, size_t(rows->D) * 4, stream) != cudaSuccess) return BL_ERR_CUDA;
    return BL_OK;
  }
  if (!dq || !dk || !dv || !dxq || !dxk || !dxv) return BL_ERR_INVALID_ARG;
  const int64_t wq = int64_t(rows->Hq) * rows->D, wk = int64_t(rows->Hkv) * rows->D;
  if (lddq < wq || lddk < wk || lddv < wk) return BL_ERR_INVALID_ARG;
  if (lddq % 4 != 0 || lddk % 4 != 0 || lddv % 4 != 0) return BL_ERR_ALIGNMENT;
  if (!is_aligned(dq, 16) || !is_aligned(dk, 16) || !is_aligned(dv, 16) || !is_aligned(dxq, 16) ||
      !is_aligned(dxk, 16) || !is_aligned(dxv, 16))
    return BL_ERR_ALIGNMENT;
  QrArgs a = rows_args(rows);
  const int grid = rows_back_grid(a.M, a.Hq + 2 * a.Hkv, a.D);
  if (dgq || dgk) {
    st = check_ws(ws, ws_bytes, bl_qk_norm_rope_backward_workspace_size(rows));
    if (st != BL_OK) return st;
    a.part = static_cast<float*>(ws);
  }
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.dxq = dxq;
  a.dxk = dxk;
  a.dxv = dxv;
  a.lddq = lddq;
  a.lddk = lddk;
  a.lddv = lddv;
  st = t == BL_T_F32   ? launch_norm_rope_back<float>(a, stream)
       : t == BL_T_F16 ? launch_norm_rope_back<__half>(a, stream)
                       : launch_norm_rope_back<__nv_bfloat16>(a, stream);
  if (st != BL_OK) return st;
  if (a.part && !launch_early(gain_sum_kernel, dim3(unsigned(ceil_div(2 * a.D, 32))), 256, 0, stream, a.part, grid, a.D,
                              dgq, dgk))
    return BL_ERR_CUDA;
  return launch_status();
}

bl_status bl_attention(const bl_attn_call* call, void* out, float* lse, cudaStream_t stream) {
  return bl_attention_ex(call, out, lse, 0, stream);
}

bl_status bl_attention_ex(const bl_attn_call* call, void* out, float* lse, int clear, cudaStream_t stream) {
  const bl_status st = check_attn(call);
  if (st != BL_OK) return st;
  if ((clear & ~(BL_CLEAR_OUT | BL_CLEAR_LSE)) != 0) return BL_ERR_INVALID_ARG;
  if (call->Tq == 0 || (call->B == 0 && clear == 0)) return BL_OK;
  if (!out || ((clear & BL_CLEAR_LSE) && !lse)) return BL_ERR_INVALID_ARG;
  if (!is_aligned(out, 16) || !is_aligned(lse, 4)) return BL_ERR_ALIGNMENT;
  AttnArgs a = attn_args(call);
  a.out = out;
  a.lse = lse;
  a.clear = clear;
  if (call->B == 0) return clear_alone(a, stream);
  return call->t == BL_T_F16 ? run_attn<__half>(a, stream) : run_attn<__nv_bfloat16>(a, stream);
}

size_t bl_attention_backward_workspace_size(const bl_attn_call* call) {
  if (check_attn(call) != BL_OK || call->B == 0) return 0;
  return norm_bytes(call) + delta_bytes(call) + dkv_part_bytes(call);
}

bl_status bl_attention_backward(const bl_attn_call* call, const void* out, const float* lse, const void* dout,
                                void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, cudaStream_t stream) {
  return bl_attention_backward_ex(call, out, lse, dout, dq, dk, dv, ws, ws_bytes, 0, stream);
}

bl_status bl_attention_backward_ex(const bl_attn_call* call, const void* out, const float* lse, const void* dout,
                                   void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, int clear, cudaStream_t stream) {
  bl_status st = check_attn(call);
  if (st != BL_OK) return st;
  if ((clear & ~(BL_CLEAR_DQ | BL_CLEAR_DK | BL_CLEAR_DV)) != 0) return BL_ERR_INVALID_ARG;
  if ((call->B == 0 && clear == 0) || (call->Tq == 0 && call->Tk == 0)) return BL_OK;
  if (call->B == 0) {                                    // nothing is read, and no workspace needed
    if ((call->Tq > 0 && (clear & BL_CLEAR_DQ) && !dq) ||
        (call->Tk > 0 && (((clear & BL_CLEAR_DK) && !dk) || ((clear & BL_CLEAR_DV) && !dv))))
      return BL_ERR_INVALID_ARG;
    if (!is_aligned(dq, 16) || !is_aligned(dk, 16) || !is_aligned(dv, 16)) return BL_ERR_ALIGNMENT;
    AttnArgs a = attn_args(call);
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.clear = clear;
    return clear_alone(a, stream);
  }
  if ((call->Tq > 0 && (!out || !lse || !dout || !dq)) || (call->Tk > 0 && (!dk || !dv))) return BL_ERR_INVALID_ARG;
  if (!is_aligned(out, 16) || !is_aligned(lse, 4) || !is_aligned(dout, 16) || !is_aligned(dq, 16) ||
      !is_aligned(dk, 16) || !is_aligned(dv, 16))
    return BL_ERR_ALIGNMENT;
  st = check_ws(ws, ws_bytes, bl_attention_backward_workspace_size(call));
  if (st != BL_OK) return st;
  AttnArgs a = attn_args(call);
  a.o = out;
  a.lse = const_cast<float*>(lse);
  a.dout = dout;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.clear = clear;
  float* norms = static_cast<float*>(ws);
  a.delta = reinterpret_cast<float*>(static_cast<char*>(ws) + norm_bytes(call));
  a.parts = norm_parts(call);
  a.splits = dkv_splits(call);
  a.split_heads = int(ceil_div(call->Hq / call->Hkv, a.splits));
  a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + norm_bytes(call) + delta_bytes(call));
  return call->t == BL_T_F16 ? run_attn_backward<__half>(a, norms, stream)
                             : run_attn_backward<__nv_bfloat16>(a, norms, stream);
}

size_t bl_paged_attention_workspace_size(int64_t B, int Hq, const bl_kv_pages* cache) {
  if (!cache || B < 1 || Hq < 1 || cache->Hkv < 1 || Hq % cache->Hkv != 0 || cache->D < 8 || cache->D > kAttnMaxD) return 0;
  const int heads = 8 * paged_nt(Hq, cache->Hkv);
  return kPaCountBytes + align_up(size_t(2 * kPaMaxCtas) * size_t(heads) * size_t(paged_pad(cache->D) + 2) * 4);
}

bl_status bl_paged_attention(const void* q, int64_t B, int Hq, const bl_kv_pages* cache, const int32_t* table,
                             int64_t ldt, const int32_t* lens, int32_t window, int32_t sinks, float scale,
                             bl_dtype out_t, void* out, void* ws, size_t ws_bytes, cudaStream_t stream) {
  bl_status st = check_cache(cache);
  if (st != BL_OK) return st;
  if (B < 0 || !int32_max(B) || Hq < 1 || Hq > 65535 || Hq % cache->Hkv != 0 || cache->D > kAttnMaxD) return BL_ERR_INVALID_ARG;
  if (ldt < 1 || !int32_max(ldt) || window < 0 || sinks < 0 || !std::isfinite(scale) || !(scale > 0.f))
    return BL_ERR_INVALID_ARG;
  if (out_t != BL_T_F32 && out_t != cache->t) return BL_ERR_INVALID_ARG;
  if (B == 0) return BL_OK;
  if (!q || !table || !lens || !out) return BL_ERR_INVALID_ARG;
  if (!is_aligned(q, 16) || !is_aligned(table, 4) || !is_aligned(lens, 4) || !is_aligned(out, 16)) return BL_ERR_ALIGNMENT;
  st = check_ws(ws, ws_bytes, bl_paged_attention_workspace_size(B, Hq, cache));
  if (st != BL_OK) return st;
  PaArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q;
  a.k = cache->k;
  a.v = cache->v;
  a.table = table;
  a.lens = lens;
  a.ldt = ldt;
  a.pages = cache->pages;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = cache->Hkv;
  a.D = cache->D;
  a.page = cache->page;
  a.most = int(ldt * cache->page < kPaMaxLen ? ldt * cache->page : kPaMaxLen);
  a.window = window;
  a.sinks = sinks;
  a.scale_log2 = scale * kLog2e;
  a.out = out;
  a.count = static_cast<unsigned int*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + kPaCountBytes);
  a.group = Hq / cache->Hkv;
  a.chunks = int(ceil_div(a.group, 8 * paged_nt(Hq, cache->Hkv)));
  // j / page for j < 2^31 as umulhi(j, magic) >> shift, shift = ceil(log2 page) - 1
  if (a.page > 1) {
    while ((uint64_t(2) << a.page_shift) < uint64_t(a.page)) ++a.page_shift;
    a.page_magic = uint32_t((uint64_t(1) << (32 + a.page_shift)) / uint64_t(a.page) + 1);
  }
  const bool f32 = out_t == BL_T_F32;
  return cache->t == BL_T_F16 ? launch_paged_t<__half>(a, f32, stream) : launch_paged_t<__nv_bfloat16>(a, f32, stream);
}

}  // extern "C"
