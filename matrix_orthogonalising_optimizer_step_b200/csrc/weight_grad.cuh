// Weight gradients on the tensor cores: G[m, n] = sum over tokens t of
// dY[t, m] X[t, n], for one weight or for every expert's weight, each over its
// own rows of dY and X.
//
// The contraction runs over rows, so both operands are MN-major: a stage
// holds 64 tokens as boxes of {64 columns, 64 tokens}, straight from the row-
// major matrices by TMA, nothing is transposed in memory.  X comes as bf16,
// exactly the values that the 8-bit form stands for (act8_unpack_kernel writes
// them just before; they are multiples of a power of two with at most 8
// significant bits, so this pass loses nothing).
//
// Execution, as in the GEMMs of umma_gemm.cuh: CTA pairs run 2-SM MMAs on
// 256 x 256 tiles with two accumulators in TMEM, so that a tile's epilogue runs
// under the next tile's MMAs; warp 0 issues the TMA loads, warp 1 the MMAs,
// warps 2.. drain.  Rows behind an expert's last one must not enter its
// gradient, not even as 0 x NaN: every expert has tensor maps of its own, made
// on the device from the offsets, whose row extent ends with the expert, so
// that the loads themselves fill the rest of the last 64 tokens with zeros.
//
// X in token order (the input of the experts' first products) is copied to
// sorted bf16 rows first, each token read once.  Measured on 32768 rows of 7168
// columns for 64 experts, 2048 wide, the product alone takes 0.82 ms from that
// copy; fetching the rows by index inside it took 3.4 ms by TMA's four-row
// gather (about 110 cycles per copy of 512 bytes) and 1.6 ms by 16-byte
// asynchronous copies of four more warps.
//
// Tiles are dealt to the pairs in whole waves; the tiles of a last, partial
// wave have their contraction split into `ranges`, whose fp32 partial products
// go to scratch and are joined by one more launch, in order (4096 x 4096 from 8192
// rows is 256 tiles for 74 pairs, 3.46 waves: see wgrad_plan for the figures).
//
// The tensor cores' own fp32 additions lose up to a unit in the last place per
// step, always toward zero, so an accumulator takes at most `chunk_kb` k-blocks; the
// epilogue threads add the chunks in registers, rounding to nearest, and round
// once more for a bf16 output.  (One accumulator for the whole contraction of a
// bf16 output, as if its rounding hid the rest: from 16384 rows 0.34 % of the
// rounded entries were not those of the formula; an fp32 product: 0.03 %.)
#pragma once

#include "umma_gemm.cuh"

namespace mc {

struct WgradParams {
  CUtensorMap map_a, map_b;   // one weight: dY [K][M] and X [K][N], boxes {64, 64}
  CUtensorMap map_o;          // output [count][M][N]: boxes of 32 rows x 128 bytes
  CUtensorMap map_p;          // partial products [split items][256][256] fp32: boxes of 32 x 32
  const CUtensorMap* maps;    // experts: [2 * count] maps of dY's and X's rows of each, else null
  const int4* ranges_of;      // experts: {first row, rows, ..} of each
  void* out;
  long long out_bs;           // elements from one problem's output to the next
  int items;                  // work items: whole tiles, then the ranges of the split ones
  int full_items;             // count * tiles_m * tiles_n less the split tiles
  int ranges;                 // one weight: ranges of each split tile
  int kb_range;               // and their k-blocks
  int M, N;
  int rows, kb_total;         // one weight: rows and k-blocks of the whole contraction
  int chunk_kb;
  int tiles_m, tiles_n, band;
  int out_f32, add, tma_out;
  int* err;
};

__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* m, uint32_t bar_cluster, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar_cluster), "r"(c0), "r"(c1)
      : "memory");
}
// Adds this CTA's fp32 box to the tensor.
__device__ __forceinline__ void tma_add_3d(const CUtensorMap* m, uint32_t src, int c0, int c1, int c2) {
  asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(src), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
// Makes a tensor map that an earlier kernel wrote to global memory usable by this thread's copies.
__device__ __forceinline__ void tmap_acquire(const CUtensorMap* m) {
  asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// ------------------------------------------------------------ experts' maps
// One block per expert: its row range from the offsets (clamped, so that no
// offsets can reach outside the `rows` rows of the operands), whether a pair has
// each of these rows, and the two tensor maps of the rows, copies of the whole
// operands' maps with another base address and row extent.
//
// A row inside the range that no pair has (its pair was dropped after the sort)
// must add nothing, whatever dY holds there and scratch was before.  Where an
// expert has such rows its dY map points to the copy `a_patched`, in which
// wgrad_patch_kernel makes them zeros, as it does in X.
constexpr int MAPS_THREADS = 256;
struct WgradMapsParams {
  CUtensorMap map_a, map_b;
  const int* offsets;
  const uint8_t* a;
  uint8_t* a_patched;      // may be a itself
  uint8_t* b;
  long long a_row_bytes, b_row_bytes;
  const uint8_t* reached;  // [rows] 1: a pair has the row; null: all of them count
  CUtensorMap* maps;
  int4* ranges;            // {first row, rows, some of them without a pair, 0} of each expert
  int rows;
};
__global__ void __launch_bounds__(MAPS_THREADS) wgrad_maps_kernel(const __grid_constant__ WgradMapsParams P) {
  __shared__ alignas(128) CUtensorMap sm[2];
  const int e = blockIdx.x, lane = threadIdx.x;
  griddep_launch_dependents();
  griddep_wait();  // the rows' pairs are being marked
  const int lo = min(max(P.offsets[e], 0), P.rows);
  const int n = max(min(P.offsets[e + 1], P.rows) - lo, 0);
  bool hole = false;
  if (P.reached && n > 0) {
    // four rows' marks a word; those of rows outside the range count as set
    const uint32_t* marks = reinterpret_cast<const uint32_t*>(P.reached);
    const long long end = static_cast<long long>(lo) + n;
    for (long long w = lo / 4 + static_cast<int>(threadIdx.x); 4 * w < end; w += MAPS_THREADS) {
      uint32_t m = marks[w];
      if (4 * w < lo) m |= (1u << (8 * (lo - static_cast<int>(4 * w)))) - 1u;
      if (4 * w + 4 > end) m |= 0xFFFFFFFFu << (8 * static_cast<int>(end - 4 * w));
      hole |= (m & 0x01010101u) != 0x01010101u;
    }
  }
  hole = __syncthreads_or(hole) != 0;
  if (threadIdx.x >= 32) return;
  const uint32_t* src_a = reinterpret_cast<const uint32_t*>(&P.map_a);
  const uint32_t* src_b = reinterpret_cast<const uint32_t*>(&P.map_b);
  reinterpret_cast<uint32_t*>(&sm[0])[lane] = src_a[lane];
  reinterpret_cast<uint32_t*>(&sm[1])[lane] = src_b[lane];
  __syncwarp();
  if (lane == 0) {
    P.ranges[e] = make_int4(lo, n, hole ? 1 : 0, 0);
    const uint64_t base[2] = {reinterpret_cast<uint64_t>(hole ? P.a_patched : P.a) + static_cast<uint64_t>(lo) * P.a_row_bytes,
                              reinterpret_cast<uint64_t>(P.b) + static_cast<uint64_t>(lo) * P.b_row_bytes};
    if (n > 0) {  // an expert without rows is never loaded; its maps stay whole (a zero extent is no map)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t m = smem_u32(&sm[i]);
        asm volatile("tensormap.replace.tile.global_address.shared::cta.b1024.b64 [%0], %1;" ::"r"(m), "l"(base[i]) : "memory");
        asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"r"(m), "r"(n) : "memory");
      }
    }
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 2; ++i)
    asm volatile("tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned [%0], [%1], 128;" ::"l"(
                     reinterpret_cast<uint64_t>(P.maps + 2 * e + i)),
                 "r"(smem_u32(&sm[i]))
                 : "memory");
}
// The rows of experts that have some without a pair: dY's to a_patched, and those
// without a pair as zeros there and in X.  A warp takes a row.  (No expert has any
// when the plan is as the sort made it; then this is an empty launch.)
__global__ void __launch_bounds__(MAPS_THREADS) wgrad_patch_kernel(const WgradMapsParams P, int experts) {
  __shared__ int4 range[MAPS_THREADS];
  griddep_launch_dependents();  // the product may set itself up
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (MAPS_THREADS / 32);
  const long long first = (long long)blockIdx.x * (MAPS_THREADS / 32) + (threadIdx.x >> 5);
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (int e0 = 0; e0 < experts; e0 += MAPS_THREADS) {
    const int e = e0 + static_cast<int>(threadIdx.x);
    const int4 mine = e < experts ? P.ranges[e] : make_int4(0, 0, 0, 0);
    range[threadIdx.x] = mine;
    const bool some = __syncthreads_or(mine.z) != 0;
    for (int i = 0; some && i < min(MAPS_THREADS, experts - e0); ++i) {
      if (!range[i].z) continue;
      for (long long k = first; k < range[i].y; k += warps) {
        const long long row = range[i].x + k;
        const bool kept = P.reached[row] != 0;
        const uint4* src = reinterpret_cast<const uint4*>(P.a + row * P.a_row_bytes);
        uint4* dst = reinterpret_cast<uint4*>(P.a_patched + row * P.a_row_bytes);
        uint4* x = reinterpret_cast<uint4*>(P.b + row * P.b_row_bytes);
        if (!kept || src != dst)
          for (long long c = lane; c < P.a_row_bytes / 16; c += 32) dst[c] = kept ? src[c] : zero;
        if (!kept)
          for (long long c = lane; c < P.b_row_bytes / 16; c += 32) x[c] = zero;
      }
    }
    __syncthreads();  // before the next experts' ranges
  }
}

// ------------------------------------------------------------------- tiles
struct WgradItem {
  int prob, tm, tn;
  int kb_first, num_kb;
  int rows;  // of the contraction, from kb_first on
  int part;  // index of the partial product, -1: the tile's whole contraction
};
// Row and column of tile `tl` of one output, in bands of `band` tile columns.
__host__ __device__ inline void wgrad_tile(int tl, int tiles_m, int tiles_n, int band, int& tm, int& tn) {
  const int per_band = tiles_m * band;
  const int b = tl / per_band, x = tl - b * per_band;
  const int rem = tiles_n - b * band;
  const int w = rem < band ? rem : band;
  tm = x / w;
  tn = b * band + x % w;
}
__device__ __forceinline__ WgradItem wgrad_item(const WgradParams& P, int t) {
  WgradItem it;
  it.prob = 0;
  it.kb_first = 0;
  it.num_kb = P.kb_total;
  it.rows = P.rows;
  it.part = -1;
  if (t >= P.items) return it;
  int tl = t;
  if (t >= P.full_items) {
    it.part = t - P.full_items;
    const int i = it.part / P.ranges;
    tl = P.full_items + i;
    it.kb_first = (it.part - i * P.ranges) * P.kb_range;
    it.num_kb = min(P.kb_range, P.kb_total - it.kb_first);
    it.rows = P.rows - it.kb_first * BK;
  } else if (P.maps) {
    const int tiles = P.tiles_m * P.tiles_n;
    it.prob = t / tiles;
    tl = t - it.prob * tiles;
    it.rows = P.ranges_of[it.prob].y;
    it.num_kb = (it.rows + BK - 1) / BK;
  }
  wgrad_tile(tl, P.tiles_m, P.tiles_n, P.band, it.tm, it.tn);
  return it;
}

constexpr size_t WGRAD_SMEM_BYTES = TileCfg<0>::SMEM_BYTES + size_t(NUM_EPI_WARPS) * EPI_BUF_BYTES;

// One warp's 32 rows x 128 bytes (fp32 or bf16 columns, `v`: those of this lane's
// row) through its buffer to a tensor; `adding`: to what is there.
template <bool F32>
__device__ __forceinline__ void wgrad_tma_out(const CUtensorMap* map, int c0, int r0, int c2, int lane, uint8_t* buf, const float* v,
                                              bool adding) {
  if (lane == 0) bulk_wait_read_all();  // the previous store has read the buffer
  __syncwarp();
  uint32_t w[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) w[i] = F32 ? __float_as_uint(v[i]) : pack_bf16x2(v[2 * i], v[2 * i + 1]);
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint4*>(buf + epi_swz(lane, c)) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (adding) {
      tma_add_3d(map, smem_u32(buf), c0, r0, c2);
    } else {
      tma_store_3d(map, smem_u32(buf), c0, r0, c2);
    }
    bulk_commit_group();
  }
}
// The same to the output.  Rows that are not whole 16-byte words go element by
// element, a row of the block at a time: neighbouring lanes write neighbouring
// addresses, and each element is written (and added to) by one lane, the same
// in every call.
template <bool F32>
__device__ __forceinline__ void wgrad_store(const WgradParams& P, int prob, int r0, int c0, int lane, uint8_t* buf,
                                            const float* v, bool adding) {
  constexpr int COLS = F32 ? 32 : 64;
  if (P.tma_out) {
    wgrad_tma_out<F32>(&P.map_o, c0, r0, prob, lane, buf, v, adding);
    return;
  }
  // (the buffer may still be read by a tensor store of a partial product)
  if (lane == 0) bulk_wait_read_all();
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = F32 ? __float_as_uint(v[4 * c + i]) : pack_bf16x2(v[8 * c + 2 * i], v[8 * c + 2 * i + 1]);
    *reinterpret_cast<uint4*>(buf + epi_swz(lane, c)) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __syncwarp();
  const long long base = prob * P.out_bs + (long long)r0 * P.N + c0;
  const int rows = min(32, P.M - r0), cols = min(COLS, P.N - c0);
  constexpr int AHEAD = 4;  // rows read from the buffer before the first is stored (8 and 16: slower)
#pragma unroll 1
  for (int rb = 0; rb < rows; rb += AHEAD) {
#pragma unroll
    for (int h = 0; h < COLS / 32; ++h) {
      const int j = 32 * h + lane;
      if constexpr (F32) {
        float* o = static_cast<float*>(P.out) + base + (long long)rb * P.N + j;
        float x[AHEAD], old[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) x[i] = *reinterpret_cast<const float*>(buf + epi_swz(rb + i, j >> 2) + (j & 3) * 4);
        if (adding) {
#pragma unroll
          for (int i = 0; i < AHEAD; ++i) old[i] = (rb + i < rows && j < cols) ? o[(long long)i * P.N] : 0.f;
#pragma unroll
          for (int i = 0; i < AHEAD; ++i) x[i] += old[i];
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
          if (rb + i < rows && j < cols) o[(long long)i * P.N] = x[i];
      } else {
        uint16_t* o = static_cast<uint16_t*>(P.out) + base + (long long)rb * P.N + j;
        uint16_t x[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) x[i] = *reinterpret_cast<const uint16_t*>(buf + epi_swz(rb + i, j >> 3) + (j & 7) * 2);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
          if (rb + i < rows && j < cols) o[(long long)i * P.N] = x[i];
      }
    }
  }
  __syncwarp();
}

template <bool F32>
__global__ void __launch_bounds__(GEMM_THREADS, 1) weight_grad_kernel(const __grid_constant__ WgradParams P) {
  using T = TileCfg<0>;
  constexpr int STAGES = T::STAGES;
  constexpr int NACC = T::NACC;
  constexpr uint32_t STAGE_BYTES = T::STAGE_BYTES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES + size_t(NUM_EPI_WARPS) * EPI_BUF_BYTES);
  uint64_t* full_bar = bars;                           // [STAGES]  used in the leader only
  uint64_t* empty_bar = bars + STAGES;                 // [STAGES]  every CTA
  uint64_t* tfull_bar = bars + 2 * STAGES;             // [NACC]    every CTA
  uint64_t* tempty_bar = bars + 2 * STAGES + NACC;     // [NACC]    used in the leader only
  uint64_t* drain_bar = bars + 2 * STAGES + 2 * NACC;  // [1]       leader
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((2 * STAGES + 2 * NACC + 1) * 8 + 8 <= GEMM_BARRIER_BYTES, "barrier block");

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0 = leader (issues the MMAs)
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    for (int b = 0; b < NACC; ++b) {
      mbar_init(smem_u32(&tfull_bar[b]), 1);
      mbar_init(smem_u32(&tempty_bar[b]), 2 * NUM_EPI_WARPS);
    }
    mbar_init(smem_u32(drain_bar), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    if (!P.maps) {
      prefetch_tmap(&P.map_a);
      prefetch_tmap(&P.map_b);
    }
    if (P.tma_out) prefetch_tmap(&P.map_o);
    if (P.items > P.full_items) prefetch_tmap(&P.map_p);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // barriers initialised and TMEM allocated in both CTAs
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_launch_dependents();
  griddep_wait();
  const int first_item = blockIdx.x >> 1;
  const int item_step = gridDim.x >> 1;

  if (warp == 0) {
    // ------------------------------------------------------- TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t filled = 0, fill_parity = 0;
      bool ok = true;
      int mapped = -1;
      for (int t = first_item; ok && t < P.items; t += item_step) {
        const WgradItem it = wgrad_item(P, t);
        const CUtensorMap* ma = P.maps ? P.maps + 2 * it.prob : &P.map_a;
        const CUtensorMap* mb = P.maps ? P.maps + 2 * it.prob + 1 : &P.map_b;
        if (P.maps && mapped != it.prob) {
          tmap_acquire(ma);
          tmap_acquire(mb);
          mapped = it.prob;
        }
        const int m0 = it.tm * BM + HALF * static_cast<int>(rank);
        const int n0 = it.tn * T::N + HALF * static_cast<int>(rank);
        // stages do not straddle chunks: the other sides count them the same way
        for (int c0 = 0; ok && c0 < it.num_kb; c0 += P.chunk_kb) {
          const int c1 = min(c0 + P.chunk_kb, it.num_kb);
          for (int kb0 = c0; kb0 < c1; kb0 += T::KPS) {
            const int nk = min(c1 - kb0, T::KPS);
            if (!wait_bounded(smem_u32(&empty_bar[stage]), phase ^ 1, abort_flag, P.err)) {
              ok = false;
              break;
            }
            const uint32_t fb_local = smem_u32(&full_bar[stage]);
            if (leader) {
              mbar_arrive_expect_tx(fb_local, uint32_t(nk) * T::PAIR_KB_BYTES);
              filled |= 1u << stage;
              fill_parity = (fill_parity & ~(1u << stage)) | (phase << stage);
            }
            const uint32_t fb = mapa_shared(fb_local, 0);
            for (int j = 0; j < nk; ++j) {
              const uint32_t sa = smem_u32(smem + stage * STAGE_BYTES + j * T::KB_BYTES);
              const uint32_t sb = sa + A_STAGE_BYTES;
              const int k0 = (it.kb_first + kb0 + j) * BK;
              tma_load_2d_pair(sa, ma, fb, m0, k0);
              tma_load_2d_pair(sa + MN_BOX_BYTES, ma, fb, m0 + 64, k0);
              tma_load_2d_pair(sb, mb, fb, n0, k0);
              tma_load_2d_pair(sb + MN_BOX_BYTES, mb, fb, n0 + 64, k0);
            }
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
      }
      // every copy of the pair lands before anyone leaves
      if (leader)
        for (int s = 0; s < STAGES; ++s)
          if (filled & (1u << s)) {
            volatile int no_abort = 0;
            wait_bounded(smem_u32(&full_bar[s]), (fill_parity >> s) & 1u, &no_abort, nullptr, kDrainLimitCycles);
          }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------- MMA issuer (leader)
    if (leader && lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      const uint32_t s0 = smem_u32(smem);
      const uint32_t idesc = idesc_bf16_f32(BM, MMA_N, 1, 1);
      const uint64_t ad0 = smem_desc_sw128(s0, MN_BOX_BYTES, 1024);
      const uint64_t bd0 = smem_desc_sw128(s0 + A_STAGE_BYTES, MN_BOX_BYTES, 1024);
      for (int t = first_item; ok && t < P.items; t += item_step) {
        const WgradItem it = wgrad_item(P, t);
        for (int c0 = 0; ok && c0 < it.num_kb; c0 += P.chunk_kb) {
          const int c1 = min(c0 + P.chunk_kb, it.num_kb);
          if (!wait_bounded(smem_u32(&tempty_bar[acc]), acc_phase ^ 1, abort_flag, P.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + acc * T::N;
          for (int kb0 = c0; kb0 < c1; kb0 += T::KPS) {
            const int nk = min(c1 - kb0, T::KPS);
            if (!wait_bounded(smem_u32(&full_bar[stage]), phase, abort_flag, P.err)) {
              ok = false;
              break;
            }
#pragma unroll
            for (int j = 0; j < T::KPS; ++j) {
              if (j >= nk) break;
              const uint64_t soff = static_cast<uint64_t>((stage * STAGE_BYTES + j * T::KB_BYTES) >> 4);
              const int left = it.rows - (kb0 + j) * BK;  // the last k-block: no products of its zeros
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk) {
                if (kk * 16 >= left) break;
                const uint64_t koff = soff + ((kk * 16u * 128u) >> 4);
                umma_bf16_pair(d_tmem, ad0 + koff, bd0 + koff, idesc, ((kb0 - c0 + j) | kk) != 0);
              }
            }
            umma_commit_pair_mc(smem_u32(&empty_bar[stage]), 0x3);
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (!ok) break;
          umma_commit_pair_mc(smem_u32(&tfull_bar[acc]), 0x3);
          if (++acc == NACC) {
            acc = 0;
            acc_phase ^= 1;
          }
        }
      }
      // every MMA of the pair completes before TMEM is released
      umma_commit_pair(smem_u32(drain_bar));
      volatile int no_abort = 0;
      wait_bounded(smem_u32(drain_bar), 0, &no_abort, nullptr, kDrainLimitCycles);
    }
  } else {
    // ------------------------------------------------------- epilogue
    constexpr int WCOLS = T::N / EPI_COL_GROUPS;  // columns per epilogue warp
    constexpr int COLS = F32 ? 32 : 64;           // columns per store
    const int q = warp & 3;                       // TMEM lane quarter this warp may read
    const int half = (warp - 2) >> 2;             // which column group of the tile
    uint8_t* buf = smem + STAGES * STAGE_BYTES + (warp - 2) * EPI_BUF_BYTES;
    uint32_t tempty_leader[NACC];
#pragma unroll
    for (int b = 0; b < NACC; ++b) tempty_leader[b] = mapa_shared(smem_u32(&tempty_bar[b]), 0);
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int t = first_item; ok && t < P.items; t += item_step) {
      const WgradItem it = wgrad_item(P, t);
      const int r0 = it.tm * BM + HALF * static_cast<int>(rank) + q * 32;
      const int cbase = it.tn * T::N + half * WCOLS;
      if (it.num_kb == 0) {  // no rows: the gradient is zero
        if (!P.add && r0 < P.M) {
          float v[COLS];
#pragma unroll
          for (int j = 0; j < COLS; ++j) v[j] = 0.f;
          for (int cb = 0; cb < WCOLS && cbase + cb < P.N; cb += COLS)
            wgrad_store<F32>(P, it.prob, r0, cbase + cb, lane, buf, v, false);
        }
        continue;
      }
      if (!F32 && it.num_kb <= P.chunk_kb && it.part < 0) {
        // one chunk has no sums to hold: half of the columns is stored before the other
        // half is read (64 experts' 2048 x 7168 from 32768 rows: 1076 us with this path,
        // 1088 through the sums)
        const bool got = wait_bounded(smem_u32(&tfull_bar[acc]), acc_phase, abort_flag, P.err);
        if (!__all_sync(0xffffffffu, got)) break;
        tc_fence_after();
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * T::N + half * WCOLS;
#pragma unroll
        for (int cb = 0; cb < WCOLS; cb += 64) {
          float v[64];
          tmem_ld64(t_row + cb, v);
          if (cb + 64 == WCOLS) {  // the accumulator is in registers: the next tile may have it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty_leader[acc]);
          }
          if (r0 < P.M && cbase + cb < P.N) wgrad_store<F32>(P, it.prob, r0, cbase + cb, lane, buf, v, false);
        }
        if (++acc == NACC) {
          acc = 0;
          acc_phase ^= 1;
        }
        continue;
      }
      // every chunk's columns into this thread's sums (its row's WCOLS columns)
      float sum[WCOLS];
#pragma unroll
      for (int j = 0; j < WCOLS; ++j) sum[j] = 0.f;
      for (int c0 = 0; c0 < it.num_kb; c0 += P.chunk_kb) {
        // every lane waits; the warp goes on only if all of them saw the phase complete
        const bool got = wait_bounded(smem_u32(&tfull_bar[acc]), acc_phase, abort_flag, P.err);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + acc * T::N + half * WCOLS;
#pragma unroll
        for (int cb = 0; cb < WCOLS; cb += 16) {
          float v[16];
          tmem_ld16(t_row + cb, v);
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[cb + j] += v[j];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty_leader[acc]);
        if (++acc == NACC) {
          acc = 0;
          acc_phase ^= 1;
        }
      }
      if (ok && r0 < P.M) {
#pragma unroll
        for (int cb = 0; cb < WCOLS; cb += COLS) {
          if (cbase + cb >= P.N) continue;
          if (it.part >= 0) {
#pragma unroll
            for (int h = 0; h < COLS; h += 32)
              wgrad_tma_out<true>(&P.map_p, half * WCOLS + cb + h, HALF * static_cast<int>(rank) + q * 32, it.part, lane, buf, sum + cb + h,
                                  false);
          } else {
            wgrad_store<F32>(P, it.prob, r0, cbase + cb, lane, buf, sum + cb, F32 && P.add != 0);
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();  // stores complete before the CTA's shared memory is released
    __syncwarp();
  }

  // Nobody leaves (or frees TMEM) while the peer may still signal this CTA's
  // barriers or read its shared memory.
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

// ---------------------------------------------------------- split contraction
// The split tiles of G: (G +) the sum of their ranges' partial products, in
// order.  A block takes JOIN_ROWS rows of one tile, four columns a thread.
constexpr int JOIN_ROWS = 16;
template <typename T>
__global__ void __launch_bounds__(256) wgrad_join_kernel(const float* part, T* out, int M, int N, int tiles_m, int tiles_n,
                                                         int band, int first_tile, int ranges, int add) {
  const int split = blockIdx.x / (BM / JOIN_ROWS), strip = blockIdx.x % (BM / JOIN_ROWS);
  int tm, tn;
  wgrad_tile(first_tile + split, tiles_m, tiles_n, band, tm, tn);
  const int cc = (threadIdx.x & 63) * 4, c = tn * MMA_N + cc;
  const float* p = part + (long long)split * ranges * (BM * MMA_N) + cc;
  griddep_wait();  // the product may still run: no __restrict__, so no read-only loads
  constexpr int ROWS = JOIN_ROWS / 4;  // of a thread; all their sums before the first store, which no load may pass
  const int r0 = strip * JOIN_ROWS + (threadIdx.x >> 6);
  float4 sum[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) sum[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < ranges; ++k) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int rr = r0 + 4 * i;
      if (tm * BM + rr >= M || c >= N) continue;
      const float4 v = *reinterpret_cast<const float4*>(p + (long long)k * (BM * MMA_N) + rr * MMA_N);
      sum[i].x += v.x; sum[i].y += v.y; sum[i].z += v.z; sum[i].w += v.w;
    }
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int r = tm * BM + r0 + 4 * i;
    if (r >= M || c >= N) continue;
    const float4 s = sum[i];
    const float t[4] = {s.x, s.y, s.z, s.w};
    T* o = out + (long long)r * N + c;
    if (N % 4 == 0 && !add) {  // whole aligned words
      if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(o) = s;
      } else {
        *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
      }
      continue;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (c + j < N) {
        if constexpr (sizeof(T) == 4) {
          o[j] = add ? o[j] + t[j] : t[j];
        } else {
          o[j] = __float2bfloat16_rn(t[j]);
        }
      }
    }
  }
}

// dY with rows that TMA cannot step over (not whole 16-byte words), to rows of
// `ld` elements (even): two columns a thread, so that the stores are whole words.
__global__ void __launch_bounds__(256) wgrad_copy_kernel(const uint16_t* __restrict__ src, uint32_t* __restrict__ dst, long long rows,
                                                         int cols, int ld) {
  for (long long r = blockIdx.x; r < rows; r += gridDim.x) {
    const uint16_t* s = src + r * cols;
    uint32_t* d = dst + r * (ld / 2);
#pragma unroll 4
    for (int c = threadIdx.x; c < (cols + 1) / 2; c += 256) {
      const uint32_t lo = s[2 * c], hi = 2 * c + 1 < cols ? s[2 * c + 1] : 0u;
      d[c] = lo | (hi << 16);
    }
  }
}

}  // namespace mc
