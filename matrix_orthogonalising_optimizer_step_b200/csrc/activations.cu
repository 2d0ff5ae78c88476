// Host side and C ABI of the activation operators (see include/muonclip.h):
// activations in 8 bits, the root-mean-square norm, weight gradients and tokens
// by expert.  Kernels: act8.cuh, norm.cuh, weight_grad.cuh, experts.cuh.
#include <algorithm>
#include <climits>
#include <cstring>

#include "host.h"
#include "act8.cuh"
#include "experts.cuh"
#include "norm.cuh"
#include "weight_grad.cuh"

namespace {

using namespace mc;

// Rows and columns of one operand: indices of rows and pairs are 32-bit.
constexpr int64_t kMaxRows = INT32_MAX;
constexpr int64_t kMaxCols = int64_t(1) << 24;

bool is_dtype(int d) { return d == MC_F32 || d == MC_BF16; }
int64_t dtype_bytes(int d) { return d == MC_F32 ? 4 : 2; }

// Whether [p, p + n) and [q, q + m) share bytes without being the same start.
bool crosses(const void* p, int64_t n, const void* q, int64_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && n > 0 && m > 0 && a != b && a < b + static_cast<uintptr_t>(m) && b < a + static_cast<uintptr_t>(n);
}
bool meets(const void* p, int64_t n, const void* q, int64_t m) {
  return crosses(p, n, q, m) || (p && p == q && n > 0 && m > 0);
}

int check_shape(int64_t rows, int64_t cols) {
  if (rows < 0 || rows > kMaxRows) return fail(MC_ERR_INVAL, "rows must be in [0, 2^31 - 1]");
  if (cols < 1 || cols > kMaxCols) return fail(MC_ERR_INVAL, "columns must be in [1, 2^24]");
  return MC_OK;
}

int check_act8(const mc_act8* a) {
  if (!a) return fail(MC_ERR_INVAL, "NULL mc_act8");
  if (a->fmt != MC_ACT_E4M3 && a->fmt != MC_ACT_INT8) return fail(MC_ERR_INVAL, "mc_act8: fmt must be MC_ACT_E4M3 or MC_ACT_INT8");
  const int rc = check_shape(a->rows, a->cols);
  if (rc != MC_OK) return rc;
  if (a->q_ld < a->cols || a->q_ld % 16 != 0) return fail(MC_ERR_INVAL, "mc_act8: q_ld must be a multiple of 16, at least cols");
  if (a->s_ld < (a->cols + ACT_BLOCK - 1) / ACT_BLOCK || a->s_ld % 16 != 0)
    return fail(MC_ERR_INVAL, "mc_act8: s_ld must be a multiple of 16, at least one byte per 32 columns");
  if (a->q_ld > (int64_t(1) << 30) || a->s_ld > (int64_t(1) << 30)) return fail(MC_ERR_INVAL, "mc_act8: row strides too large");
  if (a->rows > 0 && (!a->q || !a->scale)) return fail(MC_ERR_INVAL, "mc_act8: NULL q or scale");
  if (!aligned16(a->q) || !aligned16(a->scale)) return fail(MC_ERR_ALIGN, "mc_act8: q and scale must be 16-byte aligned");
  return MC_OK;
}
int64_t q_bytes(const mc_act8* a) { return a->rows * a->q_ld; }
int64_t s_bytes(const mc_act8* a) { return a->rows * a->s_ld; }

int take_workspace(DeviceState* st, size_t need, void** ws, size_t bytes) {
  if (*ws) {
    if (!aligned16(*ws)) return fail(MC_ERR_ALIGN, "workspace must be 16-byte aligned");
    if (bytes < need)
      return fail(MC_ERR_NOSPC, "workspace has " + std::to_string(bytes) + " bytes, needs " + std::to_string(need));
    return MC_OK;
  }
  return own_workspace(*st, need, ws);
}

// A launch that may begin while the stream's previous kernel runs out; the
// kernel waits for that one before it touches memory.
template <typename... P, typename... A>
void early_launch(void (*kernel)(P...), unsigned blocks, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  set_pdl(attr[0], true);
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// ----------------------------------------------- run-time choices to constants
template <typename F>
void with_nv(int nv, F&& f) {
  if (nv == 1) f(std::integral_constant<int, 1>{});
  else if (nv == 2) f(std::integral_constant<int, 2>{});
  else f(std::integral_constant<int, 4>{});
}
// Columns that one access moves: 8, 2 or 1, as the rows of `cols` columns begin.
template <typename F>
void with_group(int64_t cols, F&& f) {
  if (cols % 8 == 0) f(std::integral_constant<int, 8>{});
  else if (cols % 2 == 0) f(std::integral_constant<int, 2>{});
  else f(std::integral_constant<int, 1>{});
}
// Bytes of an access that every row of `cols` elements begins on a boundary of.
template <typename T, typename F>
void with_width(int64_t cols, F&& f) {
  if (cols * int64_t(sizeof(T)) % 16 == 0) f(std::integral_constant<int, 16>{});
  else if (sizeof(T) == 4 || cols % 2 == 0) f(std::integral_constant<int, 4>{});
  else f(std::integral_constant<int, int(sizeof(T))>{});
}
template <typename F>
void with_fmt(int fmt, F&& f) {
  if (fmt == MC_ACT_E4M3) f(std::integral_constant<int, ACT_E4M3>{});
  else if (fmt == MC_ACT_INT8) f(std::integral_constant<int, ACT_INT8>{});
  else f(std::integral_constant<int, ACT_NONE>{});
}
template <typename F>
void with_dtype(int dtype, F&& f) {
  if (dtype == MC_F32) f(float{});
  else f(__nv_bfloat16{});
}

// ------------------------------------------------------------ pack, unpack
// Blocks for `items` warp items, `per` of them per warp and step: at most 32 a
// SM, and every block as many steps.  More blocks than an SM holds at once (4 or
// 5) even out the SMs' speeds: 16384 x 14336 unpacked by items of one run with 8
// a SM 126 us, with 32 116 us, with one block per step 120 us.
unsigned item_blocks(long long items, int per, int warps, int sms) {
  const long long step = (long long)per * warps;
  const long long want = (items + step - 1) / step, most = 32LL * sms;
  const long long steps = std::max<long long>(1, (want + most - 1) / most);
  return static_cast<unsigned>(std::max<long long>(1, (want + steps - 1) / steps));
}

// Items of 4, 2 or 1 runs of 256 columns (see the kernels): f(runs, chunks a row, blocks).
template <typename F>
void with_runs(int64_t rows, int64_t cols, int sms, F&& f) {
  const int n = static_cast<int>((cols + WARP_COLS - 1) / WARP_COLS);
  auto take = [&](auto r) {
    constexpr int R = decltype(r)::value;
    const int chunks = (n + R - 1) / R;
    f(r, chunks, item_blocks(rows * chunks, PACK_FRAGS / R, ACT_THREADS / 32, sms));
  };
  auto fits = [&](int r) { return 4 * n >= 3 * r * ((n + r - 1) / r); };
  if (fits(4)) take(std::integral_constant<int, 4>{});
  else if (fits(2)) take(std::integral_constant<int, 2>{});
  else take(std::integral_constant<int, 1>{});
}

template <typename T, int FMT, int G>
void pack_launch(const void* x, const mc_act8* a, int sms, cudaStream_t s) {
  with_runs(a->rows, a->cols, sms, [&](auto r, int chunks, unsigned blocks) {
    act8_pack_kernel<T, FMT, G, decltype(r)::value><<<blocks, ACT_THREADS, 0, s>>>(
      static_cast<const T*>(x), static_cast<uint8_t*>(a->q), static_cast<uint8_t*>(a->scale), a->rows,
      static_cast<int>(a->cols), a->q_ld, a->s_ld, chunks);
  });
}
template <typename T, int FMT, int G>
void unpack_launch(const mc_act8* a, void* out, int64_t out_ld, int sms, cudaStream_t s) {
  with_runs(a->rows, a->cols, sms, [&](auto r, int chunks, unsigned blocks) {
    early_launch(act8_unpack_kernel<T, FMT, G, decltype(r)::value>, blocks, ACT_THREADS, s, static_cast<const uint8_t*>(a->q),
                 static_cast<const uint8_t*>(a->scale), static_cast<T*>(out), a->rows, static_cast<int>(a->cols), a->q_ld,
                 a->s_ld, out_ld, chunks);
  });
}

// The rows of `a` to `out`, rows of out_ld elements.
int unpack(const DeviceState& st, const mc_act8* a, void* out, int dtype, int64_t out_ld, int kind, cudaStream_t s) {
  const int64_t rows = a->rows;
  if (rows == 0) return MC_OK;
  const bool e4 = a->fmt == MC_ACT_E4M3;
  ProfScope prof(kind, s, 0, 0, double(rows) * a->cols * (dtype_bytes(dtype) + 1 + 1.0 / ACT_BLOCK));
  with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    // rows of `out` may be padded to whole words, which are then written whole
    with_group(out_ld % 8 == 0 ? 8 : a->cols, [&](auto g) {
      constexpr int G = decltype(g)::value;
      if (e4) unpack_launch<T, ACT_E4M3, G>(a, out, out_ld, st.sms, s);
      else unpack_launch<T, ACT_INT8, G>(a, out, out_ld, st.sms, s);
    });
  });
  MC_CUDA(cudaGetLastError());
  return MC_OK;
}

// -------------------------------------------------------------------- norm
struct NormShape {
  int nv, wpr, groups, threads;
};
// Fragments per thread, warps per row and rows per block.  Many rows: four
// fragments a thread (their loads are in flight together) and blocks of about
// eight warps.  Few rows (less than two blocks per SM that way): one fragment
// a thread, so that a row's latency is spread over the most warps.
NormShape norm_shape(int64_t rows, int64_t cols, int sms) {
  const int frags = static_cast<int>((cols + WARP_COLS - 1) / WARP_COLS);
  NormShape n;
  n.nv = frags >= 4 ? 4 : (frags >= 2 ? 2 : 1);
  if (frags <= 32) {
    const int wpr4 = (frags + n.nv - 1) / n.nv;
    const int per_block = std::max(1, 8 / wpr4);
    if ((rows + per_block - 1) / per_block < 2LL * sms) n.nv = 1;
  }
  n.wpr = (frags + n.nv - 1) / n.nv;
  n.groups = std::max(1, 8 / n.wpr);
  n.threads = 32 * n.wpr * n.groups;
  return n;
}
// The gradient: as few fragments as a block of 8 warps (32 for the widest
// rows) can hold; dw stays in registers over the whole walk.
NormShape norm_bwd_shape(int64_t cols) {
  const int frags = static_cast<int>((cols + WARP_COLS - 1) / WARP_COLS);
  NormShape n;
  n.nv = frags <= 8 ? 1 : (frags <= 16 ? 2 : 4);
  n.wpr = (frags + n.nv - 1) / n.nv;
  n.groups = std::max(1, 8 / n.wpr);
  n.threads = 32 * n.wpr * n.groups;
  return n;
}
constexpr int kNormBwdBlocks = 640;  // most blocks of the gradient's walk

// The gradient through the shared-memory ring.  wpr = 0: the row does not fit.
constexpr int kNormRingBytes = 100 * 1024;      // of a block that shares an SM with another
constexpr int kNormRingBytesWide = 200 * 1024;  // of a block that has an SM to itself
NormShape norm_ring_shape(int64_t cols, int64_t row_bytes, int64_t q_row, int64_t s_row, bool dh, NormRing* R) {
  const int frags = static_cast<int>((cols + WARP_COLS - 1) / WARP_COLS);
  NormShape n;
  n.nv = frags <= 8 ? 1 : (frags <= 16 ? 2 : 4);
  n.wpr = (frags + n.nv - 1) / n.nv;
  n.groups = std::max(1, 8 / n.wpr);
  n.threads = 32 * n.wpr * n.groups;
  auto at = [](int64_t b) { return (b + 127) / 128 * 128; };
  const int64_t rows_b = at(n.groups * row_bytes);
  const int64_t h_b = q_row ? at(n.groups * q_row) + at(n.groups * s_row) : rows_b;
  const int64_t stage = rows_b * (dh ? 2 : 1) + h_b;
  // two blocks an SM where two stages of either fit, else one
  const int64_t room = n.wpr <= 8 && 2 * stage <= kNormRingBytes ? kNormRingBytes : kNormRingBytesWide;
  const int64_t stages = std::min<int64_t>(NORM_RING_STAGES, room / stage);
  if (n.wpr > 16 || stages < 2) {
    n.wpr = 0;
    return n;
  }
  R->stages = static_cast<int>(stages);
  R->stage_bytes = static_cast<int>(stage);
  R->off_dh = static_cast<int>(rows_b);
  R->off_h = static_cast<int>(rows_b * (dh ? 2 : 1));
  R->off_s = static_cast<int>(R->off_h + at(n.groups * q_row));
  R->row_bytes = static_cast<int>(row_bytes);
  R->q_row = static_cast<int>(q_row);
  R->s_row = static_cast<int>(s_row);
  return n;
}

int check_norm(const void* w, int dtype, int w_dtype, int64_t rows, int64_t cols) {
  if (!is_dtype(dtype) || !is_dtype(w_dtype)) return fail(MC_ERR_INVAL, "dtype must be MC_F32 or MC_BF16");
  const int rc = check_shape(rows, cols);
  if (rc != MC_OK) return rc;
  if (cols > NORM_MAX_COLS) return fail(MC_ERR_INVAL, "a normed row has at most " + std::to_string(NORM_MAX_COLS) + " columns");
  if (!w) return fail(MC_ERR_INVAL, "NULL weight");
  if (!aligned16(w)) return fail(MC_ERR_ALIGN, "weight must be 16-byte aligned");
  return MC_OK;
}

// ------------------------------------------------------------ weight gradient
// Longest contraction one accumulator takes, in k-blocks, for an fp32 and for a
// bf16 output.  14336 x 4096 from 16384 rows to bf16: 1461 us with one accumulator,
// 1474 with chunks of 32 k-blocks, 1487 with 16; entries that are not the rounded
// formula's: 0.34 %, 0.044 %, 0.023 % (a fp32 matrix product: 0.033 %).
constexpr int kWgradChunkKb = 16;
constexpr int kWgradChunkKbBf16 = 32;

struct WgradPlan {
  int64_t ldx, ldy;          // rows of the bf16 X and of dY
  int64_t tiles, split;      // one weight: tiles in all, those of them whose contraction is split
  int ranges, kb_range;      // into so many ranges of so many k-blocks
  bool copy_dy;
  size_t off_x, off_dy, off_part, off_maps, off_ranges, off_reached, total;
};

// CTA pairs that the plan counts on; the launch takes what the device has.
constexpr int kPlanPairs = 74;

// The split of one weight's contraction: the tiles beyond the whole waves of
// all pairs, each into r ranges, where that is estimated to take less time than
// a partial wave does.  The estimate: a k-block of a tile takes about 0.32 us,
// the joining launch 4 us, and a partial product of 256 KB is written and read
// at 5 TB/s.
void wgrad_split(int64_t rows, int64_t M, int64_t N, WgradPlan& p) {
  p.tiles = ((M + BM - 1) / BM) * ((N + MMA_N - 1) / MMA_N);
  const int64_t kb = (rows + BK - 1) / BK, rem = p.tiles % kPlanPairs;
  p.split = 0;
  p.ranges = 1;
  p.kb_range = static_cast<int>(kb);
  double best = double(kb) * 0.32;  // the partial wave
  for (int64_t r = 2; rem > 0 && r <= 32 && r * 4 <= kb; ++r) {
    const int64_t per = (kb + r - 1) / r, used = (kb + per - 1) / per;  // none of the ranges empty
    const int64_t waves = (rem * used + kPlanPairs - 1) / kPlanPairs;
    const double us = double(waves) * per * 0.32 + 4.0 + double(rem * used) * (2.0 * BM * MMA_N * 4) / 5e6;
    if (us < best) {
      best = us;
      p.split = rem;
      p.ranges = static_cast<int>(used);
      p.kb_range = static_cast<int>(per);
    }
  }
}

WgradPlan wgrad_plan(int64_t rows, int64_t M, int64_t N, int experts) {
  WgradPlan p;
  p.ldx = round8(N);
  p.copy_dy = M % 8 != 0;
  p.ldy = round8(M);
  wgrad_split(rows, M, N, p);
  if (experts > 0) p.split = 0;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += align_up(bytes, 256);
    return o;
  };
  p.off_x = take(size_t(rows) * p.ldx * 2);
  // experts: room for dY without the rows that no pair has, too
  p.off_dy = take(p.copy_dy || experts > 0 ? size_t(rows) * p.ldy * 2 : 0);
  p.off_part = take(size_t(p.split) * p.ranges * BM * MMA_N * 4);
  p.off_maps = take(size_t(experts) * 2 * sizeof(CUtensorMap));
  p.off_ranges = take(size_t(experts) * sizeof(int4));
  p.off_reached = take(experts > 0 ? size_t(rows) : 0);
  p.total = at + 256;  // the parts start at the first 256-byte boundary (tensor maps need 128)
  return p;
}

int act_device_state(DeviceState** out) {
  const int rc = device_state(out);
  if (rc != MC_OK) return rc;
  if (!(*out)->act_init) {
    const int gemm_smem = static_cast<int>(WGRAD_SMEM_BYTES);
    MC_CUDA(cudaFuncSetAttribute(weight_grad_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, gemm_smem));
    MC_CUDA(cudaFuncSetAttribute(weight_grad_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, gemm_smem));
    const int sort_smem = sort_place_smem<SORT_CLUSTER_THREADS>(MAX_EXPERTS);
    MC_CUDA(cudaFuncSetAttribute(expert_place_kernel<int, SORT_CLUSTER_THREADS, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, sort_smem));
    MC_CUDA(cudaFuncSetAttribute(expert_place_kernel<long long, SORT_CLUSTER_THREADS, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, sort_smem));
    (*out)->act_init = true;
  }
  return MC_OK;
}

int map_rows(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t ld) {
  const uint64_t dims[2] = {uint64_t(cols), uint64_t(rows)};
  const uint64_t strides[1] = {uint64_t(ld) * 2};
  const uint32_t box[2] = {64, BK};
  return make_map(map, base, 2, dims, strides, box);
}

int check_wgrad(const void* dy, const mc_act8* x, int64_t rows, int64_t M, const void* g, int g_dtype, int accumulate) {
  int rc = check_act8(x);
  if (rc != MC_OK) return rc;
  if ((rc = check_shape(rows, M)) != MC_OK) return rc;
  if (!is_dtype(g_dtype)) return fail(MC_ERR_INVAL, "g_dtype must be MC_F32 or MC_BF16");
  if (accumulate && g_dtype != MC_F32)
    return fail(MC_ERR_INVAL, "gradients accumulate in fp32 only: adding to a bf16 sum would lose small contributions");
  if (!g || (rows > 0 && !dy)) return fail(MC_ERR_INVAL, "NULL dy or g");
  if (!aligned16(dy) || !aligned16(g)) return fail(MC_ERR_ALIGN, "pointers must be 16-byte aligned");
  return MC_OK;
}

// G (one weight: offsets NULL) or every expert's G.  Caller holds g_mu.
int weight_grad(const void* dy, int64_t rows, const mc_act8* x, const int* offsets, const int* position, int top_k,
                int experts, int64_t M, void* g, int g_dtype, int accumulate, void* workspace, size_t workspace_bytes,
                cudaStream_t s) {
  DeviceState* st = nullptr;
  int rc = act_device_state(&st);
  if (rc != MC_OK) return rc;
  const int64_t N = x->cols;
  const int count = std::max(experts, 1);
  if (rows == 0) {
    if (!accumulate) MC_CUDA(cudaMemsetAsync(g, 0, size_t(count) * M * N * dtype_bytes(g_dtype), s));
    return MC_OK;
  }
  const WgradPlan p = wgrad_plan(rows, M, N, experts);
  if ((rc = take_workspace(st, p.total, &workspace, workspace_bytes)) != MC_OK) return rc;
  uint8_t* ws = reinterpret_cast<uint8_t*>(align_up(reinterpret_cast<uintptr_t>(workspace), 256));
  const void* a = dy;
  if (p.copy_dy) {
    ProfScope prof(K_WGRAD_PREP, s, 0, 0, 4.0 * double(rows) * M);
    wgrad_copy_kernel<<<static_cast<unsigned>(std::min<int64_t>(rows, 32LL * st->sms)), 256, 0, s>>>(
        static_cast<const uint16_t*>(dy), reinterpret_cast<uint32_t*>(ws + p.off_dy), rows, static_cast<int>(M), static_cast<int>(p.ldy));
    MC_CUDA(cudaGetLastError());
    a = ws + p.off_dy;
  }
  WgradParams P;
  std::memset(&P, 0, sizeof(P));
  if ((rc = map_rows(&P.map_a, a, rows, M, p.ldy)) != MC_OK) return rc;
  if ((rc = map_rows(&P.map_b, ws + p.off_x, rows, N, p.ldx)) != MC_OK) return rc;
  // rows of the workspace are padded to whole 16 bytes, so the 8-bit rows always take the wide path
  if (position) {
    const int segments = static_cast<int>((N + 4 * WARP_COLS - 1) / (4 * WARP_COLS));
    const unsigned blocks = item_blocks(x->rows * segments, 1, ACT_THREADS / 32, st->sms);
    MC_CUDA(cudaMemsetAsync(ws + p.off_reached, 0, size_t(rows), s));
    ProfScope prof(K_WGRAD_PREP, s, 0, 0, double(x->rows) * N * (1 + 1.0 / ACT_BLOCK) + 2.0 * double(rows) * N);
    auto go = [&](auto kernel) {
      kernel<<<blocks, ACT_THREADS, 0, s>>>(static_cast<const uint8_t*>(x->q), static_cast<const uint8_t*>(x->scale),
                                            reinterpret_cast<__nv_bfloat16*>(ws + p.off_x), ws + p.off_reached, position, top_k, x->rows,
                                            static_cast<int>(N), x->q_ld, x->s_ld, p.ldx, segments);
    };
    if (x->fmt == MC_ACT_E4M3) go(act8_scatter_kernel<ACT_E4M3>);
    else go(act8_scatter_kernel<ACT_INT8>);
    MC_CUDA(cudaGetLastError());
  }
  if (offsets) {
    WgradMapsParams mp;
    std::memset(&mp, 0, sizeof(mp));
    mp.map_a = P.map_a;
    mp.map_b = P.map_b;
    mp.offsets = offsets;
    mp.a = static_cast<const uint8_t*>(a);
    mp.a_patched = ws + p.off_dy;
    mp.b = ws + p.off_x;
    mp.a_row_bytes = p.ldy * 2;
    mp.b_row_bytes = p.ldx * 2;
    mp.reached = position ? ws + p.off_reached : nullptr;
    mp.maps = reinterpret_cast<CUtensorMap*>(ws + p.off_maps);
    mp.ranges = reinterpret_cast<int4*>(ws + p.off_ranges);
    mp.rows = static_cast<int>(rows);
    {
      ProfScope prof(K_WGRAD_PREP, s);
      early_launch(wgrad_maps_kernel, static_cast<unsigned>(experts), MAPS_THREADS, s, mp);
      MC_CUDA(cudaGetLastError());
    }
    if (position) {
      ProfScope prof(K_WGRAD_PREP, s);
      early_launch(wgrad_patch_kernel, static_cast<unsigned>(2 * st->sms), MAPS_THREADS, s, mp, experts);
      MC_CUDA(cudaGetLastError());
    }
    P.maps = mp.maps;
    P.ranges_of = mp.ranges;
  }
  if (!position && (rc = unpack(*st, x, ws + p.off_x, MC_BF16, p.ldx, K_WGRAD_PREP, s)) != MC_OK) return rc;

  P.M = static_cast<int>(M);
  P.N = static_cast<int>(N);
  P.rows = static_cast<int>(rows);
  P.kb_total = static_cast<int>((rows + BK - 1) / BK);
  P.out = g;
  P.out_f32 = g_dtype == MC_F32 ? 1 : 0;
  P.add = accumulate ? 1 : 0;
  P.chunk_kb = P.out_f32 ? kWgradChunkKb : kWgradChunkKbBf16;
  P.tiles_m = static_cast<int>((M + BM - 1) / BM);
  P.tiles_n = static_cast<int>((N + MMA_N - 1) / MMA_N);
  P.band = 8;
  const int64_t items = count * p.tiles - p.split + p.split * p.ranges;
  if (items > INT32_MAX / 2) return fail(MC_ERR_INVAL, "the gradients have too many tiles of 256 x 256");
  P.full_items = static_cast<int>(count * p.tiles - p.split);
  P.items = static_cast<int>(items);
  P.ranges = p.ranges;
  P.kb_range = p.kb_range;
  const int64_t es = dtype_bytes(g_dtype);
  P.out_bs = M * N;
  P.err = st->err_ptr;
  P.tma_out = (N * es) % 16 == 0 ? 1 : 0;
  if (P.tma_out) {
    const uint64_t dims[3] = {uint64_t(N), uint64_t(M), uint64_t(count)};
    const uint64_t strides[2] = {uint64_t(N * es), uint64_t(N * es) * uint64_t(M)};
    const uint32_t box[3] = {P.out_f32 ? 32u : 64u, 32, 1};
    if ((rc = make_map(&P.map_o, g, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                       P.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16)) != MC_OK)
      return rc;
  }
  if (p.split) {
    const uint64_t dims[3] = {uint64_t(MMA_N), uint64_t(BM), uint64_t(p.split) * p.ranges};
    const uint64_t strides[2] = {uint64_t(MMA_N) * 4, uint64_t(MMA_N) * BM * 4};
    const uint32_t box[3] = {32, 32, 1};
    if ((rc = make_map(&P.map_p, ws + p.off_part, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_DATA_TYPE_FLOAT32)) != MC_OK)
      return rc;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  set_pdl(attr[0], true);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.stream = s;
  cfg.attrs = attr;
  {
    const double flops = 2.0 * double(rows) * M * N;
    ProfScope prof(K_WGRAD, s, flops, flops);
    cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min(st->pair_clusters, P.items)));
    cfg.blockDim = dim3(GEMM_THREADS);
    cfg.dynamicSmemBytes = WGRAD_SMEM_BYTES;
    cfg.numAttrs = 2;
    if (P.out_f32) {
      MC_CUDA(cudaLaunchKernelEx(&cfg, weight_grad_kernel<true>, P));
    } else {
      MC_CUDA(cudaLaunchKernelEx(&cfg, weight_grad_kernel<false>, P));
    }
  }
  if (p.split) {
    ProfScope prof(K_WGRAD_JOIN, s, 0, 0, double(p.split) * BM * MMA_N * (4.0 * p.ranges + es));
    cfg.gridDim = dim3(static_cast<unsigned>(p.split * (BM / JOIN_ROWS)));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    const float* part = reinterpret_cast<const float*>(ws + p.off_part);
    const int first = P.full_items;
    if (P.out_f32) {
      MC_CUDA(cudaLaunchKernelEx(&cfg, wgrad_join_kernel<float>, part, static_cast<float*>(g), P.M, P.N, P.tiles_m, P.tiles_n, P.band,
                                 first, P.ranges, accumulate));
    } else {
      MC_CUDA(cudaLaunchKernelEx(&cfg, wgrad_join_kernel<__nv_bfloat16>, part, static_cast<__nv_bfloat16*>(g), P.M, P.N, P.tiles_m,
                                 P.tiles_n, P.band, first, P.ranges, 0));
    }
  }
  return MC_OK;
}

// -------------------------------------------------------------------- experts
int check_pairs(int64_t tokens, int top_k) {
  if (tokens < 0) return fail(MC_ERR_INVAL, "tokens must not be negative");
  if (top_k < 1 || top_k > MAX_EXPERTS) return fail(MC_ERR_INVAL, "top_k must be in [1, 1024]");
  if (tokens > kMaxRows / top_k) return fail(MC_ERR_INVAL, "tokens * top_k must be at most 2^31 - 1");
  return MC_OK;
}
int check_move(int dtype, int64_t tokens, int top_k, int64_t cols) {
  if (!is_dtype(dtype)) return fail(MC_ERR_INVAL, "dtype must be MC_F32 or MC_BF16");
  const int rc = check_pairs(tokens, top_k);
  return rc != MC_OK ? rc : check_shape(tokens, cols);
}
int64_t sort_tiles(int64_t pairs) { return (pairs + SORT_TILE - 1) / SORT_TILE; }

// Blocks of the one-launch sort's cluster (a power of two), or 0 where it is not used.
int sort_cluster(int64_t pairs) {
  if (pairs <= SORT_TILE || pairs > SORT_CLUSTER_PAIRS) return 0;
  int c = 1;
  while (int64_t(c) * SORT_CLUSTER_TILE < pairs) c *= 2;
  return c;
}

template <typename I>
int sort_launch(const I* idx, int64_t pairs, int E, int* offsets, int* source, int* position, int* counts, cudaStream_t s) {
  if (const int c = sort_cluster(pairs)) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(c);
    cfg.blockDim = dim3(SORT_CLUSTER_THREADS);
    cfg.dynamicSmemBytes = sort_place_smem<SORT_CLUSTER_THREADS>(E);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int* none = nullptr;
    MC_CUDA(cudaLaunchKernelEx(&cfg, expert_place_kernel<I, SORT_CLUSTER_THREADS, true>, idx, none, none, offsets, source, position,
                               static_cast<long long>(pairs), E));
    return MC_OK;
  }
  const unsigned tiles = static_cast<unsigned>(sort_tiles(pairs));
  int* totals = tiles > SORT_SCAN_TILES ? counts + size_t(tiles) * (E + 1) : nullptr;
  if (tiles > 1) {
    expert_count_kernel<I><<<tiles, SORT_THREADS, (E + 1) * sizeof(int), s>>>(idx, counts, pairs, E);
    MC_CUDA(cudaGetLastError());
  }
  if (totals) {
    expert_scan_kernel<<<E + 1, SORT_THREADS, 0, s>>>(counts, totals, static_cast<int>(tiles), E + 1);
    MC_CUDA(cudaGetLastError());
  }
  expert_place_kernel<I, SORT_THREADS, false><<<tiles, SORT_THREADS, sort_place_smem<SORT_THREADS>(E), s>>>(
      idx, tiles > 1 ? counts : nullptr, totals, offsets, source, position, pairs, E);
  MC_CUDA(cudaGetLastError());
  return MC_OK;
}

}  // namespace

// ============================================================ activations in 8 bits
MC_API int mc_act8_pack(const void* x, int x_dtype, const mc_act8* a, void* stream) {
  int rc = check_act8(a);
  if (rc != MC_OK) return rc;
  if (!is_dtype(x_dtype)) return fail(MC_ERR_INVAL, "x_dtype must be MC_F32 or MC_BF16");
  if (a->rows == 0) return MC_OK;
  if (!x) return fail(MC_ERR_INVAL, "NULL x");
  if (!aligned16(x)) return fail(MC_ERR_ALIGN, "x must be 16-byte aligned");
  const int64_t xb = a->rows * a->cols * dtype_bytes(x_dtype);
  if (meets(x, xb, a->q, q_bytes(a)) || meets(x, xb, a->scale, s_bytes(a)) || meets(a->q, q_bytes(a), a->scale, s_bytes(a)))
    return fail(MC_ERR_INVAL, "x, q and scale must not overlap");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState* st = nullptr;
  if ((rc = act_device_state(&st)) != MC_OK) return rc;
  ProfScope prof(K_ACT_PACK, s, 0, 0, double(a->rows) * a->cols * (dtype_bytes(x_dtype) + 1 + 1.0 / ACT_BLOCK));
  with_dtype(x_dtype, [&](auto t) {
    using T = decltype(t);
    with_group(a->cols, [&](auto g) {
      constexpr int G = decltype(g)::value;
      if (a->fmt == MC_ACT_E4M3) pack_launch<T, ACT_E4M3, G>(x, a, st->sms, s);
      else pack_launch<T, ACT_INT8, G>(x, a, st->sms, s);
    });
  });
  MC_CUDA(cudaGetLastError());
  return MC_OK;
}

MC_API int mc_act8_unpack(const mc_act8* a, void* out, int out_dtype, void* stream) {
  int rc = check_act8(a);
  if (rc != MC_OK) return rc;
  if (!is_dtype(out_dtype)) return fail(MC_ERR_INVAL, "out_dtype must be MC_F32 or MC_BF16");
  if (a->rows == 0) return MC_OK;
  if (!out) return fail(MC_ERR_INVAL, "NULL out");
  if (!aligned16(out)) return fail(MC_ERR_ALIGN, "out must be 16-byte aligned");
  const int64_t ob = a->rows * a->cols * dtype_bytes(out_dtype);
  if (meets(out, ob, a->q, q_bytes(a)) || meets(out, ob, a->scale, s_bytes(a)))
    return fail(MC_ERR_INVAL, "out must not overlap q or scale");
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState* st = nullptr;
  if ((rc = act_device_state(&st)) != MC_OK) return rc;
  return unpack(*st, a, out, out_dtype, a->cols, K_ACT_UNPACK,
                static_cast<cudaStream_t>(stream));
}

// ==================================================================== norm
MC_API int mc_rms_norm(const void* x, const void* residual, const void* w, int dtype, int w_dtype, int64_t rows,
                       int64_t cols, float eps, void* h_out, void* y_out, const mc_act8* y8, float* rstd_out, void* stream) {
  int rc = check_norm(w, dtype, w_dtype, rows, cols);
  if (rc != MC_OK) return rc;
  if (!(eps >= 0.f) || eps > 1e30f) return fail(MC_ERR_INVAL, "eps must be finite and not negative");
  if (rows == 0) return MC_OK;
  if ((y_out != nullptr) == (y8 != nullptr)) return fail(MC_ERR_INVAL, "exactly one of y_out and y8 must be given");
  if (y8) {
    if ((rc = check_act8(y8)) != MC_OK) return rc;
    if (y8->rows != rows || y8->cols != cols) return fail(MC_ERR_INVAL, "y8 must have the shape of x");
  }
  if ((residual != nullptr) != (h_out != nullptr)) return fail(MC_ERR_INVAL, "h_out goes with residual, and residual with h_out");
  if (!x || !rstd_out) return fail(MC_ERR_INVAL, "NULL x or rstd_out");
  if (!aligned16(x) || !aligned16(residual) || !aligned16(h_out) || !aligned16(y_out) || !aligned16(rstd_out))
    return fail(MC_ERR_ALIGN, "pointers must be 16-byte aligned");
  const int64_t n = rows * cols, xb = n * dtype_bytes(dtype), wb = cols * dtype_bytes(w_dtype);
  const void* in[2] = {x, residual};
  const void* y = y8 ? y8->q : y_out;
  const int64_t yb = y8 ? q_bytes(y8) : 2 * n;
  for (const void* i : in)
    if (crosses(i, xb, h_out, xb) || meets(i, xb, y, yb) || (y8 && meets(i, xb, y8->scale, s_bytes(y8))) ||
        meets(i, xb, rstd_out, 4 * rows))
      return fail(MC_ERR_INVAL, "outputs must not overlap the inputs (h_out may be x or residual itself)");
  if (meets(h_out, xb, y, yb) || (y8 && meets(h_out, xb, y8->scale, s_bytes(y8))) || meets(h_out, xb, rstd_out, 4 * rows) ||
      meets(y, yb, rstd_out, 4 * rows) || (y8 && (meets(y, yb, y8->scale, s_bytes(y8)) || meets(y8->scale, s_bytes(y8), rstd_out, 4 * rows))))
    return fail(MC_ERR_INVAL, "outputs must not overlap each other");
  if (meets(w, wb, h_out, xb) || meets(w, wb, y, yb) || (y8 && meets(w, wb, y8->scale, s_bytes(y8))) || meets(w, wb, rstd_out, 4 * rows))
    return fail(MC_ERR_INVAL, "outputs must not overlap the weight");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState* st = nullptr;
  if ((rc = act_device_state(&st)) != MC_OK) return rc;
  const NormShape sh = norm_shape(rows, cols, st->sms);
  const unsigned blocks = static_cast<unsigned>((rows + sh.groups - 1) / sh.groups);
  const dim3 dim(32 * sh.wpr, sh.groups);
  ProfScope prof(K_RMS_NORM, s, 0, 0, double(xb) * (residual ? 3 : 1) + double(n) * (y8 ? 1 + 1.0 / ACT_BLOCK : 2));
  with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    NormFwdArgs<T> a;
    a.x = static_cast<const T*>(x);
    a.r = static_cast<const T*>(residual);
    a.w = w;
    a.h = static_cast<T*>(h_out);
    a.y = static_cast<__nv_bfloat16*>(y_out);
    a.q = y8 ? static_cast<uint8_t*>(y8->q) : nullptr;
    a.s = y8 ? static_cast<uint8_t*>(y8->scale) : nullptr;
    a.rstd = rstd_out;
    a.rows = rows;
    a.q_ld = y8 ? y8->q_ld : 0;
    a.s_ld = y8 ? y8->s_ld : 0;
    a.D = static_cast<int>(cols);
    a.w_f32 = w_dtype == MC_F32 ? 1 : 0;
    a.eps = eps;
    a.d = static_cast<double>(cols);
    a.inv_d = 1.0 / a.d;
    with_fmt(y8 ? y8->fmt : -1, [&](auto f) {
      with_group(cols, [&](auto g) {
        constexpr int F = decltype(f)::value;
        constexpr int G = decltype(g)::value;
        if (sh.threads <= 256) {
          with_nv(sh.nv, [&](auto nv) { rms_norm_kernel<T, F, G, decltype(nv)::value, 256><<<blocks, dim, 0, s>>>(a); });
        } else if (sh.nv == 1) {
          rms_norm_kernel<T, F, G, 1, NORM_MAX_THREADS><<<blocks, dim, 0, s>>>(a);
        } else {
          rms_norm_kernel<T, F, G, 4, NORM_MAX_THREADS><<<blocks, dim, 0, s>>>(a);
        }
      });
    });
  });
  MC_CUDA(cudaGetLastError());
  return MC_OK;
}

MC_API size_t mc_rms_norm_backward_workspace_size(int64_t rows, int64_t cols) {
  if (rows < 0 || rows > kMaxRows || cols < 1 || cols > NORM_MAX_COLS) return 0;
  // a part is the sum of one group of warps; either form of the kernel has at
  // most 8 / ceil(fragments / 4) groups a block
  const int64_t frags = (cols + WARP_COLS - 1) / WARP_COLS;
  const int64_t groups = std::max<int64_t>(1, 8 / ((frags + 3) / 4));
  const int64_t parts = std::min<int64_t>(std::max<int64_t>(rows, 1) + groups - 1, kNormBwdBlocks * groups);
  return align_up(size_t(parts) * cols * sizeof(float), 256);
}

MC_API int mc_rms_norm_backward(const void* dy, const void* dh, const void* h, const mc_act8* h8, const void* w,
                                const float* rstd, int dtype, int w_dtype, int64_t rows, int64_t cols, void* dx, float* dw,
                                void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_norm(w, dtype, w_dtype, rows, cols);
  if (rc != MC_OK) return rc;
  if (!dw) return fail(MC_ERR_INVAL, "NULL dw");
  if (!aligned16(dw)) return fail(MC_ERR_ALIGN, "dw must be 16-byte aligned");
  if (h && h8) return fail(MC_ERR_INVAL, "one of h and h8 must be given");
  if (h8) {
    if ((rc = check_act8(h8)) != MC_OK) return rc;
    if (h8->rows != rows || h8->cols != cols) return fail(MC_ERR_INVAL, "h8 must have the shape of dy");
  }
  if (rows > 0 && (!dy || !(h || h8) || !rstd || !dx)) return fail(MC_ERR_INVAL, "NULL dy, h, rstd or dx");
  if (!aligned16(dy) || !aligned16(dh) || !aligned16(h) || !aligned16(rstd) || !aligned16(dx))
    return fail(MC_ERR_ALIGN, "pointers must be 16-byte aligned");
  const int64_t n = rows * cols, nb = n * dtype_bytes(dtype), wb = cols * dtype_bytes(w_dtype);
  if (crosses(dx, nb, dy, nb) || crosses(dx, nb, dh, nb) || meets(dx, nb, h, nb) || meets(dx, nb, w, wb) ||
      meets(dx, nb, rstd, 4 * rows) || (h8 && (meets(dx, nb, h8->q, q_bytes(h8)) || meets(dx, nb, h8->scale, s_bytes(h8)))) ||
      meets(dx, nb, dw, 4 * cols))
    return fail(MC_ERR_INVAL, "dx must not overlap the other operands (it may be dy or dh itself)");
  if (meets(dw, 4 * cols, dy, nb) || meets(dw, 4 * cols, dh, nb) || meets(dw, 4 * cols, h, nb) || meets(dw, 4 * cols, w, wb) ||
      meets(dw, 4 * cols, rstd, 4 * rows) ||
      (h8 && (meets(dw, 4 * cols, h8->q, q_bytes(h8)) || meets(dw, 4 * cols, h8->scale, s_bytes(h8)))))
    return fail(MC_ERR_INVAL, "dw must not overlap the other operands");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState* st = nullptr;
  if ((rc = act_device_state(&st)) != MC_OK) return rc;
  if (rows == 0) {
    MC_CUDA(cudaMemsetAsync(dw, 0, cols * sizeof(float), s));
    return MC_OK;
  }
  if ((rc = take_workspace(st, mc_rms_norm_backward_workspace_size(rows, cols), &workspace, workspace_bytes)) != MC_OK) return rc;
  const int64_t q_row = h8 ? (cols + 15) / 16 * 16 : 0, s_row = h8 ? ((cols + ACT_BLOCK - 1) / ACT_BLOCK + 15) / 16 * 16 : 0;
  NormRing ring = {};
  const NormShape rs = cols % 8 == 0 ? norm_ring_shape(cols, cols * dtype_bytes(dtype), q_row, s_row, dh != nullptr, &ring) : NormShape{};
  const NormShape sh = norm_bwd_shape(cols);
  int parts = 0;
  cudaError_t err = cudaSuccess;
  {
    ProfScope prof(K_RMS_NORM_BWD, s, 0, 0, double(nb) * (dh ? 3 : 2) + double(n) * (h8 ? 1 + 1.0 / ACT_BLOCK : dtype_bytes(dtype)));
    with_dtype(dtype, [&](auto t) {
      using T = decltype(t);
      NormBwdArgs<T> a;
      a.dy = static_cast<const T*>(dy);
      a.dh = static_cast<const T*>(dh);
      a.h = static_cast<const T*>(h);
      a.q = h8 ? static_cast<const uint8_t*>(h8->q) : nullptr;
      a.s = h8 ? static_cast<const uint8_t*>(h8->scale) : nullptr;
      a.w = w;
      a.rstd = rstd;
      a.dx = static_cast<T*>(dx);
      a.partial = static_cast<float*>(workspace);
      a.rows = rows;
      a.q_ld = h8 ? h8->q_ld : 0;
      a.s_ld = h8 ? h8->s_ld : 0;
      a.D = static_cast<int>(cols);
      a.wpr = rs.wpr ? rs.wpr : sh.wpr;
      a.w_f32 = w_dtype == MC_F32 ? 1 : 0;
      with_fmt(h8 ? h8->fmt : -1, [&](auto f) {
        if (rs.wpr) {
          auto launch = [&](auto kernel, int per_sm) {
            const int smem = ring.stages * ring.stage_bytes;
            if (st->wide_smem.insert(reinterpret_cast<const void*>(kernel)).second)
              err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormRingBytesWide);
            if (err != cudaSuccess) {
              st->wide_smem.erase(reinterpret_cast<const void*>(kernel));
              return;
            }
            const unsigned blocks = static_cast<unsigned>(
                std::min<int64_t>((rows + rs.groups - 1) / rs.groups, std::min<int64_t>(kNormBwdBlocks, int64_t(per_sm) * st->sms)));
            parts = static_cast<int>(blocks) * rs.groups;
            kernel<<<blocks, rs.threads + 32, smem, s>>>(a, ring, st->err_ptr);
          };
          constexpr int F = decltype(f)::value;
          if (rs.threads > 256) {
            launch(rms_norm_bwd_ring_kernel<T, F, 4, 512>, 1);
          } else {
            with_nv(rs.nv, [&](auto nv) { launch(rms_norm_bwd_ring_kernel<T, F, decltype(nv)::value, 256>, 2); });
          }
          return;
        }
        auto launch = [&](auto kernel) {
          int per_sm = 0;
          err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, sh.threads, 0);
          if (err != cudaSuccess) return;
          const int64_t most = std::min<int64_t>(kNormBwdBlocks, int64_t(std::max(per_sm, 1)) * st->sms);
          const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((rows + sh.groups - 1) / sh.groups, most));
          parts = static_cast<int>(blocks) * sh.groups;
          kernel<<<blocks, sh.threads, 0, s>>>(a);
        };
        constexpr int F = decltype(f)::value;
        if (cols % 8 == 0) {  // rows too wide for the ring
          launch(rms_norm_bwd_kernel<T, F, 8, 4, NORM_MAX_THREADS>);
        } else {
          auto odd = [&](auto g) {
            constexpr int G = decltype(g)::value;
            if (sh.threads > 256) launch(rms_norm_bwd_kernel<T, F, G, 4, NORM_MAX_THREADS>);
            else with_nv(sh.nv, [&](auto nv) { launch(rms_norm_bwd_kernel<T, F, G, decltype(nv)::value, 256>); });
          };
          if (cols % 2 == 0) odd(std::integral_constant<int, 2>{});
          else odd(std::integral_constant<int, 1>{});
        }
      });
    });
  }
  MC_CUDA(err);
  MC_CUDA(cudaGetLastError());
  ProfScope prof(K_RMS_NORM_DW, s, 0, 0, 4.0 * parts * double(cols));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  set_pdl(attr[0], true);
  cfg.gridDim = dim3(static_cast<unsigned>((cols + 31) / 32));
  cfg.blockDim = dim3(NORM_DW_WARPS * 32);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  MC_CUDA(cudaLaunchKernelEx(&cfg, rms_norm_dw_kernel, static_cast<const float*>(workspace), dw, parts, static_cast<int>(cols)));
  return MC_OK;
}

// ========================================================= weight gradients
MC_API size_t mc_weight_grad_workspace_size(int64_t rows, int64_t out_features, int64_t in_features) {
  if (rows < 0 || rows > kMaxRows || out_features < 1 || out_features > kMaxCols || in_features < 1 || in_features > kMaxCols) return 0;
  return wgrad_plan(rows, out_features, in_features, 0).total;
}

MC_API int mc_weight_grad(const void* dy, const mc_act8* x, int64_t out_features, void* g, int g_dtype, int accumulate,
                          void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_act8(x);
  if (rc != MC_OK) return rc;
  if ((rc = check_wgrad(dy, x, x->rows, out_features, g, g_dtype, accumulate)) != MC_OK) return rc;
  const int64_t gb = out_features * x->cols * dtype_bytes(g_dtype);
  if (meets(g, gb, dy, 2 * x->rows * out_features) || meets(g, gb, x->q, q_bytes(x)) || meets(g, gb, x->scale, s_bytes(x)))
    return fail(MC_ERR_INVAL, "g must not overlap dy or x");
  std::lock_guard<std::mutex> lock(g_mu);
  return weight_grad(dy, x->rows, x, nullptr, nullptr, 1, 0, out_features, g, g_dtype, accumulate, workspace, workspace_bytes,
                     static_cast<cudaStream_t>(stream));
}

MC_API size_t mc_expert_weight_grad_workspace_size(int64_t rows, int experts, int64_t out_features, int64_t in_features) {
  if (rows < 0 || rows > kMaxRows || out_features < 1 || out_features > kMaxCols || in_features < 1 || in_features > kMaxCols ||
      experts < 1 || experts > MAX_EXPERTS)
    return 0;
  return wgrad_plan(rows, out_features, in_features, experts).total;
}

MC_API int mc_expert_weight_grad(const void* dy, int64_t rows, const mc_act8* x, const int32_t* offsets, const int32_t* position,
                                 int top_k, int experts, int64_t out_features, void* g, int g_dtype, int accumulate,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_act8(x);
  if (rc != MC_OK) return rc;
  if ((rc = check_wgrad(dy, x, rows, out_features, g, g_dtype, accumulate)) != MC_OK) return rc;
  if (experts < 1 || experts > MAX_EXPERTS) return fail(MC_ERR_INVAL, "experts must be in [1, 1024]");
  if (!offsets) return fail(MC_ERR_INVAL, "NULL offsets");
  if (position) {
    if (top_k < 1 || top_k > MAX_EXPERTS) return fail(MC_ERR_INVAL, "top_k must be in [1, 1024]");
    if (x->rows > kMaxRows / top_k || x->rows * top_k != rows)
      return fail(MC_ERR_INVAL, "with position, rows must be top_k times the rows of x");
  } else if (x->rows != rows) {
    return fail(MC_ERR_INVAL, "without position, x must have the rows of dy");
  }
  if (!aligned16(offsets) || !aligned16(position)) return fail(MC_ERR_ALIGN, "pointers must be 16-byte aligned");
  const int64_t gb = int64_t(experts) * out_features * x->cols * dtype_bytes(g_dtype);
  if (meets(g, gb, dy, 2 * rows * out_features) || meets(g, gb, x->q, q_bytes(x)) || meets(g, gb, x->scale, s_bytes(x)) ||
      meets(g, gb, offsets, 4 * (experts + 1)) || meets(g, gb, position, 4 * rows))
    return fail(MC_ERR_INVAL, "g must not overlap the inputs");
  std::lock_guard<std::mutex> lock(g_mu);
  return weight_grad(dy, rows, x, offsets, position, position ? top_k : 1, experts, out_features, g, g_dtype, accumulate, workspace,
                     workspace_bytes, static_cast<cudaStream_t>(stream));
}

// ================================================================== experts
MC_API size_t mc_expert_sort_workspace_size(int64_t tokens, int top_k, int experts) {
  if (tokens < 0 || top_k < 1 || top_k > MAX_EXPERTS || tokens > kMaxRows / top_k || experts < 1 || experts > MAX_EXPERTS) return 0;
  const int64_t tiles = sort_tiles(tokens * top_k);
  return align_up(tiles > 1 && !sort_cluster(tokens * top_k) ? size_t(tiles + 1) * (experts + 1) * sizeof(int) : 16, 256);
}

MC_API int mc_expert_sort(const void* idx, int idx_bits, int64_t tokens, int top_k, int experts, int32_t* offsets,
                          int32_t* source, int32_t* position, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_pairs(tokens, top_k);
  if (rc != MC_OK) return rc;
  if (experts < 1 || experts > MAX_EXPERTS) return fail(MC_ERR_INVAL, "experts must be in [1, 1024]");
  if (idx_bits != 32 && idx_bits != 64) return fail(MC_ERR_INVAL, "idx_bits must be 32 or 64");
  const int64_t pairs = tokens * top_k;
  if (!offsets || (pairs > 0 && (!idx || !source || !position))) return fail(MC_ERR_INVAL, "NULL idx, offsets, source or position");
  if (!aligned16(idx) || !aligned16(offsets) || !aligned16(source) || !aligned16(position))
    return fail(MC_ERR_ALIGN, "pointers must be 16-byte aligned");
  const int64_t ib = pairs * (idx_bits / 8), ob = 4 * (experts + 1);
  if (meets(idx, ib, offsets, ob) || meets(idx, ib, source, 4 * pairs) || meets(idx, ib, position, 4 * pairs) ||
      meets(offsets, ob, source, 4 * pairs) || meets(offsets, ob, position, 4 * pairs) || meets(source, 4 * pairs, position, 4 * pairs))
    return fail(MC_ERR_INVAL, "idx, offsets, source and position must not overlap");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState* st = nullptr;
  if ((rc = act_device_state(&st)) != MC_OK) return rc;
  if (pairs == 0) {
    MC_CUDA(cudaMemsetAsync(offsets, 0, ob, s));
    return MC_OK;
  }
  if ((rc = take_workspace(st, mc_expert_sort_workspace_size(tokens, top_k, experts), &workspace, workspace_bytes)) != MC_OK) return rc;
  ProfScope prof(K_EXPERT_SORT, s, 0, 0, double(ib) + 8.0 * pairs);
  int* counts = static_cast<int*>(workspace);
  return idx_bits == 32 ? sort_launch(static_cast<const int*>(idx), pairs, experts, offsets, source, position, counts, s)
                        : sort_launch(static_cast<const long long*>(idx), pairs, experts, offsets, source, position, counts, s);
}

MC_API int mc_expert_gather(const void* x, int dtype, int64_t tokens, int top_k, int64_t cols, const int32_t* position,
                            void* rows_out, void* stream) {
  int rc = check_move(dtype, tokens, top_k, cols);
  if (rc != MC_OK) return rc;
  if (tokens == 0) return MC_OK;
  if (!x || !position || !rows_out) return fail(MC_ERR_INVAL, "NULL x, position or rows_out");
  if (!aligned16(x) || !aligned16(position) || !aligned16(rows_out)) return fail(MC_ERR_ALIGN, "pointers must be 16-byte aligned");
  const int64_t es = dtype_bytes(dtype), xb = tokens * cols * es, pairs = tokens * top_k;
  if (meets(rows_out, xb * top_k, x, xb) || meets(rows_out, xb * top_k, position, 4 * pairs))
    return fail(MC_ERR_INVAL, "rows_out must not overlap the inputs");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState* st = nullptr;
  if ((rc = act_device_state(&st)) != MC_OK) return rc;
  ProfScope prof(K_EXPERT_GATHER, s, 0, 0, double(xb) * (1 + top_k));
  with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const int seg_cols = GATHER_RUNS * run_cols<T>();
    const int segments = static_cast<int>((cols + seg_cols - 1) / seg_cols);
    const unsigned blocks = item_blocks(tokens * segments, 1, MOVE_THREADS / 32, st->sms);
    with_width<T>(cols, [&](auto v) {
      early_launch(expert_gather_kernel<T, decltype(v)::value>, blocks, MOVE_THREADS, s, static_cast<const T*>(x), position,
                   static_cast<T*>(rows_out), tokens, top_k, static_cast<int>(cols), segments);
    });
  });
  MC_CUDA(cudaGetLastError());
  return MC_OK;
}

MC_API int mc_expert_combine(const void* y, int dtype, int64_t tokens, int top_k, int64_t cols, const int32_t* position,
                             const float* weights, void* out, void* stream) {
  int rc = check_move(dtype, tokens, top_k, cols);
  if (rc != MC_OK) return rc;
  if (tokens == 0) return MC_OK;
  if (!y || !position || !out) return fail(MC_ERR_INVAL, "NULL y, position or out");
  if (!aligned16(y) || !aligned16(position) || !aligned16(weights) || !aligned16(out))
    return fail(MC_ERR_ALIGN, "pointers must be 16-byte aligned");
  const int64_t es = dtype_bytes(dtype), ob = tokens * cols * es, pairs = tokens * top_k;
  if (meets(out, ob, y, ob * top_k) || meets(out, ob, position, 4 * pairs) || meets(out, ob, weights, 4 * pairs))
    return fail(MC_ERR_INVAL, "out must not overlap the inputs");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState* st = nullptr;
  if ((rc = act_device_state(&st)) != MC_OK) return rc;
  ProfScope prof(K_EXPERT_COMBINE, s, 0, 0, double(ob) * (1 + top_k));
  with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const int seg_cols = COMBINE_RUNS * run_cols<T>();
    const int segments = static_cast<int>((cols + seg_cols - 1) / seg_cols);
    const unsigned blocks = item_blocks(tokens * segments, 1, MOVE_THREADS / 32, st->sms);
    with_width<T>(cols, [&](auto v) {
      expert_combine_kernel<T, decltype(v)::value><<<blocks, MOVE_THREADS, 0, s>>>(
          static_cast<const T*>(y), position, weights, static_cast<T*>(out), tokens, top_k, static_cast<int>(cols), segments);
    });
  });
  MC_CUDA(cudaGetLastError());
  return MC_OK;
}

MC_API int mc_expert_combine_backward(const void* dout, const void* y, int dtype, int64_t tokens, int top_k, int64_t cols,
                                      const int32_t* position, const float* weights, void* dy, float* dweights, void* stream) {
  int rc = check_move(dtype, tokens, top_k, cols);
  if (rc != MC_OK) return rc;
  if (tokens == 0) return MC_OK;
  if (!dout || !y || !position || !weights || !dy || !dweights)
    return fail(MC_ERR_INVAL, "NULL dout, y, position, weights, dy or dweights");
  if (!aligned16(dout) || !aligned16(y) || !aligned16(position) || !aligned16(weights) || !aligned16(dy) || !aligned16(dweights))
    return fail(MC_ERR_ALIGN, "pointers must be 16-byte aligned");
  const int64_t es = dtype_bytes(dtype), tb = tokens * cols * es, rb = tb * top_k, pb = 4 * tokens * top_k;
  if (meets(dy, rb, dout, tb) || crosses(dy, rb, y, rb) || meets(dy, rb, position, pb) || meets(dy, rb, weights, pb) ||
      meets(dy, rb, dweights, pb) || meets(dweights, pb, dout, tb) || meets(dweights, pb, y, rb) || meets(dweights, pb, position, pb) ||
      meets(dweights, pb, weights, pb))
    return fail(MC_ERR_INVAL, "dy and dweights must not overlap the other operands (dy may be y itself)");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> lock(g_mu);
  DeviceState* st = nullptr;
  if ((rc = act_device_state(&st)) != MC_OK) return rc;
  ProfScope prof(K_EXPERT_COMBINE_BWD, s, 0, 0, double(tb) * (1 + 2 * top_k));
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(tokens, INT32_MAX));
  with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const int runs = static_cast<int>((cols + run_cols<T>() - 1) / run_cols<T>());
    int warps = 1, idle = INT_MAX;
    for (int w = std::min(runs, MOVE_THREADS / 32); w >= 1 && w >= std::min(runs, 4); --w) {
      const int left = (runs + w - 1) / w * w - runs;
      if (left < idle) {
        idle = left;
        warps = w;
      }
    }
    with_width<T>(cols, [&](auto v) {
      expert_combine_bwd_kernel<T, decltype(v)::value><<<blocks, 32 * warps, 0, s>>>(
          static_cast<const T*>(dout), static_cast<const T*>(y), position, weights, static_cast<T*>(dy), dweights, tokens, top_k,
          static_cast<int>(cols));
    });
  });
  MC_CUDA(cudaGetLastError());
  return MC_OK;
}
