// Tokens sorted by expert and back.
//
//   sort      T tokens with K experts each (T*K pairs, pair p = t*K + k): a stable
//             counting sort by expert.  offsets[e] = first sorted row of expert e,
//             source[r] = pair of row r (-1 behind the last), position[p] = row of
//             pair p (-1 if dropped: its expert index is outside [0, E))
//   gather    rows[position[p]] = x[p / K]
//   combine   out[t] = sum over k of w[t, k] y[position[t, k]]   (k ascending, fp32)
//   combine's gradient
//             dy[position[t, k]] = w[t, k] dout[t],  dw[t, k] = <dout[t], y[position[t, k]]>
//   gather's gradient is combine without weights.
//
// All of it is copying: bound by memory, each token's row is read once and each
// expert row read or written once, so the kernels go token by token through
// `position` (reading x once for its K copies) and never through `source`.
// Nothing is added atomically: every sum has one owner and a fixed order.
// Measured on 4096 tokens of 8 pairs, 64 experts, 7168 bf16 columns: sort 12 us
// (with about 4 us of the timing's own), gather 87 us (529 MB, 6.1 TB/s),
// combine's gradient 167 us (998 MB, 6.0 TB/s).
#pragma once

#include "act8.cuh"

namespace mc {

constexpr int SORT_THREADS = 256;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_STEPS = 8;                                   // pairs per thread
constexpr int SORT_TILE = SORT_THREADS * SORT_STEPS;            // pairs per block
constexpr int SORT_SCAN_TILES = 64;
constexpr int MAX_EXPERTS = 1024;

template <typename I>
__device__ __forceinline__ int sort_key(const I* idx, long long p, long long pairs, int E) {
  if (p >= pairs) return -1;
  const I e = idx[p];
  return (e >= 0 && e < static_cast<I>(E)) ? static_cast<int>(e) : E;  // E: dropped
}

// counts[tile][E + 1] of each tile's pairs (integer sums, whatever their order).
template <typename I>
__global__ void __launch_bounds__(SORT_THREADS) expert_count_kernel(const I* __restrict__ idx, int* __restrict__ counts,
                                                                    long long pairs, int E) {
  extern __shared__ int sort_smem[];
  for (int e = threadIdx.x; e <= E; e += SORT_THREADS) sort_smem[e] = 0;
  __syncthreads();
  const long long base = (long long)blockIdx.x * SORT_TILE;
#pragma unroll
  for (int i = 0; i < SORT_STEPS; ++i) {
    const int key = sort_key(idx, base + i * SORT_THREADS + threadIdx.x, pairs, E);
    if (key >= 0) atomicAdd(&sort_smem[key], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += SORT_THREADS) counts[(long long)blockIdx.x * (E + 1) + e] = sort_smem[e];
}

// Many tiles: each column e of counts to its exclusive sums over the tiles, and
// the column's total.  One block per expert.
__global__ void __launch_bounds__(SORT_THREADS) expert_scan_kernel(int* __restrict__ counts, int* __restrict__ totals, int tiles,
                                                                   int n) {
  __shared__ int warp_sum[SORT_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int carry = 0;
  for (int t0 = 0; t0 < tiles; t0 += SORT_THREADS) {
    const int t = t0 + threadIdx.x;
    const long long at = (long long)t * n + blockIdx.x;
    const int c = t < tiles ? counts[at] : 0;
    int s = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    if (lane == 31) warp_sum[warp] = s;
    __syncthreads();
    int add = carry;
#pragma unroll
    for (int w = 0; w < SORT_WARPS; ++w) {
      if (w < warp) add += warp_sum[w];
      carry += warp_sum[w];
    }
    if (t < tiles) counts[at] = add + s - c;
    __syncthreads();
  }
  if (threadIdx.x == 0) totals[blockIdx.x] = carry;
}

// Places one tile's pairs.  A warp ranks 32 pairs at a time among equal
// experts (match), over its own run of the tile; the warps' counts and the
// other tiles' counts then give each (warp, expert) its first row.  The other
// tiles' counts come from
//   CLUSTER  the blocks of this cluster, one tile each, through distributed
//            shared memory: the whole sort is one launch (up to
//            SORT_CLUSTER_PAIRS pairs; 32768 pairs for 64 experts took 18 us
//            as a counting and a placing launch);
//   counts   the counting launch.  `totals` given: counts hold the sums over the
//            tiles before, else every block adds them up itself (up to
//            SORT_SCAN_TILES tiles, where that costs less than a launch);
//   neither  there is one tile.
constexpr int SORT_CLUSTER_THREADS = 512;
constexpr int SORT_CLUSTER_TILE = SORT_CLUSTER_THREADS * SORT_STEPS;
constexpr int SORT_CLUSTER_PAIRS = 8 * SORT_CLUSTER_TILE;

__device__ __forceinline__ int ld_cluster(const int* p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
  return v;
}

template <int THREADS>
__host__ __device__ constexpr int sort_place_smem(int E) { return (THREADS / 32 + 3) * (E + 1) * 4; }

template <typename I, int THREADS, bool CLUSTER>
__global__ void __launch_bounds__(THREADS) expert_place_kernel(const I* __restrict__ idx, const int* __restrict__ counts,
                                                               const int* __restrict__ totals, int* __restrict__ offsets,
                                                               int* __restrict__ source, int* __restrict__ position,
                                                               long long pairs, int E) {
  griddep_launch_dependents();
  extern __shared__ int sort_smem[];
  constexpr int WARPS = THREADS / 32;
  const int n = E + 1;
  int* hist = sort_smem;              // [WARPS][n], then first rows
  int* total = hist + WARPS * n;      // [n] pairs of each expert, in all
  int* before = total + n;            // [n] of them in earlier tiles
  int* local = before + n;            // [n] of them in this tile (CLUSTER)
  __shared__ int warp_sum[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < WARPS * n; i += THREADS) hist[i] = 0;
  __syncthreads();
  const long long base = (long long)blockIdx.x * (THREADS * SORT_STEPS) + warp * (32 * SORT_STEPS);
  int key[SORT_STEPS], rank[SORT_STEPS];
#pragma unroll
  for (int i = 0; i < SORT_STEPS; ++i) key[i] = sort_key(idx, base + 32 * i + lane, pairs, E);
#pragma unroll
  for (int i = 0; i < SORT_STEPS; ++i) {
    const unsigned same = __match_any_sync(0xffffffffu, key[i]);
    const int below = __popc(same & ((1u << lane) - 1u));
    int had = 0;
    if (key[i] >= 0) had = hist[warp * n + key[i]];
    __syncwarp();
    if (key[i] >= 0 && below == 0) hist[warp * n + key[i]] = had + __popc(same);
    __syncwarp();
    rank[i] = had + below;
  }
  __syncthreads();
  if constexpr (CLUSTER) {
    for (int e = threadIdx.x; e < n; e += THREADS) {
      int c = 0;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) c += hist[w * n + e];
      local[e] = c;
    }
    cluster_sync();
  }
  // pairs per expert: of every tile, and of those before this one
  for (int e = threadIdx.x; e < n; e += THREADS) {
    int all = 0, mine = 0;
    if constexpr (CLUSTER) {
      for (unsigned t = 0; t < gridDim.x; ++t) {
        if (t == blockIdx.x) mine = all;
        all += ld_cluster(local + e, t);
      }
    } else if (totals) {
      all = totals[e];
      mine = counts[(long long)blockIdx.x * n + e];
    } else if (counts) {
      for (int t = 0; t < static_cast<int>(gridDim.x); ++t) {
        if (t == static_cast<int>(blockIdx.x)) mine = all;
        all += counts[(long long)t * n + e];
      }
    } else {
#pragma unroll
      for (int w = 0; w < WARPS; ++w) all += hist[w * n + e];
    }
    total[e] = all;
    before[e] = mine;
  }
  if constexpr (CLUSTER) {
    cluster_sync();  // every block has read this one's counts
  } else {
    __syncthreads();
  }
  // exclusive sums over the experts, THREADS at a time
  int carry = 0;
  for (int e0 = 0; e0 < n; e0 += THREADS) {
    const int e = e0 + threadIdx.x;
    const int c = e < n ? total[e] : 0;
    int s = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    if (lane == 31) warp_sum[warp] = s;
    __syncthreads();
    int add = carry, chunk = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) add += warp_sum[w];
      chunk += warp_sum[w];
    }
    if (e < n) {
      const int first = add + s - c;
      if (blockIdx.x == 0) offsets[e] = first;  // offsets[E] = rows in all (the dropped ones come behind)
      int row = first + before[e];
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const int h = hist[w * n + e];
        hist[w * n + e] = row;
        row += h;
      }
    }
    carry += chunk;
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < SORT_STEPS; ++i) {
    if (key[i] < 0) continue;
    const long long p = base + 32 * i + lane;
    const int row = hist[warp * n + key[i]] + rank[i];
    const bool kept = key[i] < E;
    position[p] = kept ? row : -1;
    source[row] = kept ? static_cast<int>(p) : -1;
  }
}

// ----------------------------------------------------------- moving the rows
// Items are (token, segment of columns), one per warp and step.
constexpr int MOVE_THREADS = 256;

// One lane's share of a run of 512 bytes: 16 of them at once (W = 16: rows of
// whole 16-byte words), or 4-byte words (W = 4: rows of whole words) or single
// bf16 elements (W = 2) that neighbouring lanes have neighbours of.
template <typename T>
__host__ __device__ constexpr int move_elems() { return 16 / int(sizeof(T)); }

template <typename T, int W>
__device__ __forceinline__ uint4 move_load(const T* row, int c0, int lane, int D) {
  constexpr int PER = W / int(sizeof(T));  // elements of an access
  static_assert(W == 16 || W == 4 || (W == 2 && sizeof(T) == 2), "whole elements");
  if constexpr (W == 16) {
    const int c = c0 + PER * lane;
    return c < D ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0u, 0u, 0u, 0u);
  } else {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 16 / W; ++i) {
      const int c = c0 + PER * (32 * i + lane);
      if (c < D) {
        if constexpr (W == 4) w[i] = *reinterpret_cast<const uint32_t*>(row + c);
        else w[i >> 1] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(row + c)) << (16 * (i & 1));
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}
template <typename T, int W>
__device__ __forceinline__ void move_store(T* row, int c0, int lane, int D, uint4 q) {
  constexpr int PER = W / int(sizeof(T));
  if constexpr (W == 16) {
    const int c = c0 + PER * lane;
    if (c < D) *reinterpret_cast<uint4*>(row + c) = q;
  } else {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 16 / W; ++i) {
      const int c = c0 + PER * (32 * i + lane);
      if (c < D) {
        if constexpr (W == 4) *reinterpret_cast<uint32_t*>(row + c) = w[i];
        else *reinterpret_cast<uint16_t*>(row + c) = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
      }
    }
  }
}
template <typename T>
__device__ __forceinline__ void move_floats(uint4 q, float (&v)[move_elems<T>()]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
template <typename T>
__device__ __forceinline__ uint4 move_words(const float (&v)[move_elems<T>()]) {
  if constexpr (sizeof(T) == 4) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  } else {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}
template <typename T>
__host__ __device__ constexpr int run_cols() { return 32 * move_elems<T>(); }  // columns of one 512-byte run

constexpr int GATHER_RUNS = 4;
template <typename T, int W>
__global__ void __launch_bounds__(MOVE_THREADS) expert_gather_kernel(const T* x, const int* position, T* out, long long tokens, int K, int D,
                                                                     int segments) {
  griddep_wait();  // the sort, or what wrote x, may still run: no __restrict__, so no read-only loads
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (MOVE_THREADS / 32);
  const long long first = (long long)blockIdx.x * (MOVE_THREADS / 32) + (threadIdx.x >> 5);
  const long long step_rows = warps / segments;
  const int step_seg = static_cast<int>(warps % segments);
  const long long rows = tokens * K;
  RowWalk w{first / segments, static_cast<int>(first % segments)};
  for (; w.row < tokens; walk_next(w, step_rows, step_seg, segments)) {
    const int c0 = w.chunk * GATHER_RUNS * run_cols<T>();
    uint4 q[GATHER_RUNS];
#pragma unroll
    for (int u = 0; u < GATHER_RUNS; ++u) q[u] = move_load<T, W>(x + w.row * D, c0 + u * run_cols<T>(), lane, D);
    for (int k0 = 0; k0 < K; k0 += 32) {
      const int mine = k0 + lane < K ? position[w.row * K + k0 + lane] : -1;
      const int kn = min(32, K - k0);
      for (int k = 0; k < kn; ++k) {
        const int r = __shfl_sync(0xffffffffu, mine, k);
        if (r < 0 || r >= rows) continue;
#pragma unroll
        for (int u = 0; u < GATHER_RUNS; ++u)
          move_store<T, W>(out + (long long)r * D, c0 + u * run_cols<T>(), lane, D, q[u]);
      }
    }
  }
}

constexpr int COMBINE_RUNS = 2;
template <typename T, int W>
__global__ void __launch_bounds__(MOVE_THREADS) expert_combine_kernel(const T* __restrict__ y, const int* __restrict__ position,
                                                                      const float* __restrict__ weights, T* __restrict__ out,
                                                                      long long tokens, int K, int D, int segments) {
  constexpr int N = move_elems<T>();
  constexpr int AHEAD = 4;  // rows in flight
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (MOVE_THREADS / 32);
  const long long first = (long long)blockIdx.x * (MOVE_THREADS / 32) + (threadIdx.x >> 5);
  const long long step_rows = warps / segments;
  const int step_seg = static_cast<int>(warps % segments);
  const long long rows = tokens * K;
  RowWalk w{first / segments, static_cast<int>(first % segments)};
  for (; w.row < tokens; walk_next(w, step_rows, step_seg, segments)) {
    const int c0 = w.chunk * COMBINE_RUNS * run_cols<T>();
    float sum[COMBINE_RUNS][N];
#pragma unroll
    for (int u = 0; u < COMBINE_RUNS; ++u)
#pragma unroll
      for (int i = 0; i < N; ++i) sum[u][i] = 0.f;
    for (int k0 = 0; k0 < K; k0 += 32) {
      const int mine = k0 + lane < K ? position[w.row * K + k0 + lane] : -1;
      const float wmine = (weights && k0 + lane < K) ? weights[w.row * K + k0 + lane] : 1.f;
      const int kn = min(32, K - k0);
      for (int k = 0; k < kn; k += AHEAD) {
        uint4 q[AHEAD][COMBINE_RUNS];
        bool live[AHEAD];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
          const int r = k + a < 32 ? __shfl_sync(0xffffffffu, mine, (k + a) & 31) : -1;
          live[a] = k + a < kn && r >= 0 && r < rows;
          if (live[a]) {
#pragma unroll
            for (int u = 0; u < COMBINE_RUNS; ++u)
              q[a][u] = move_load<T, W>(y + (long long)r * D, c0 + u * run_cols<T>(), lane, D);
          }
        }
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) {
          const float wk = __shfl_sync(0xffffffffu, wmine, (k + a) & 31);
          if (!live[a]) continue;
#pragma unroll
          for (int u = 0; u < COMBINE_RUNS; ++u) {
            float v[N];
            move_floats<T>(q[a][u], v);
#pragma unroll
            for (int i = 0; i < N; ++i) sum[u][i] = fmaf(wk, v[i], sum[u][i]);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < COMBINE_RUNS; ++u)
      move_store<T, W>(out + w.row * D, c0 + u * run_cols<T>(), lane, D, move_words<T>(sum[u]));
  }
}

// One block per token: its warps (as many, up to 8, as leave the fewest idle in
// the last of their turns over the row's 512-byte runs) share the row, every
// pair's dot product is kept by thread over the whole row and joined at the end
// (lanes by a tree, then warps in order).  dy may be y itself: a thread reads what it overwrites.
// Four pairs' loads are in flight at a time: all eight (145 registers) left one
// block an SM and took 273 us for the case above; eight or two at 3 or 4 blocks
// an SM 199 and 193 us.
constexpr int BACK_PAIRS = 8;  // pairs whose sums a pass over the row keeps
constexpr int BACK_AHEAD = 4;  // pairs loaded together
template <typename T, int W>
__global__ void __launch_bounds__(MOVE_THREADS, 3) expert_combine_bwd_kernel(const T* __restrict__ dout, const T* y,
                                                                             const int* __restrict__ position,
                                                                             const float* __restrict__ weights, T* dy,
                                                                             float* __restrict__ dweights, long long tokens, int K,
                                                                             int D) {
  constexpr int N = move_elems<T>();
  __shared__ float part[MOVE_THREADS / 32][BACK_PAIRS];
  const int warps = blockDim.x >> 5;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long rows = tokens * K;
  for (long long t = blockIdx.x; t < tokens; t += gridDim.x) {
    for (int k0 = 0; k0 < K; k0 += BACK_PAIRS) {
      // lane a < BACK_PAIRS holds pair k0 + a's row and weight
      int mine = -1;
      float wmine = 0.f;
      if (lane < BACK_PAIRS && k0 + lane < K) {
        mine = position[t * K + k0 + lane];
        if (mine >= rows) mine = -1;
        wmine = weights[t * K + k0 + lane];
      }
      float dot[BACK_PAIRS];
#pragma unroll
      for (int a = 0; a < BACK_PAIRS; ++a) dot[a] = 0.f;
      for (int c0 = warp * run_cols<T>(); c0 < D; c0 += warps * run_cols<T>()) {
        float g[N];
        move_floats<T>(move_load<T, W>(dout + t * D, c0, lane, D), g);
#pragma unroll
        for (int a0 = 0; a0 < BACK_PAIRS; a0 += BACK_AHEAD) {
          uint4 q[BACK_AHEAD];
          int pos[BACK_AHEAD];
#pragma unroll
          for (int a = 0; a < BACK_AHEAD; ++a) {
            pos[a] = __shfl_sync(0xffffffffu, mine, a0 + a);
            if (pos[a] >= 0) q[a] = move_load<T, W>(y + (long long)pos[a] * D, c0, lane, D);
          }
#pragma unroll
          for (int a = 0; a < BACK_AHEAD; ++a) {
            const float wk = __shfl_sync(0xffffffffu, wmine, a0 + a);
            if (pos[a] < 0) continue;
            float v[N];
            move_floats<T>(q[a], v);
#pragma unroll
            for (int i = 0; i < N; ++i) {
              dot[a0 + a] = fmaf(g[i], v[i], dot[a0 + a]);
              v[i] = wk * g[i];
            }
            move_store<T, W>(dy + (long long)pos[a] * D, c0, lane, D, move_words<T>(v));
          }
        }
      }
#pragma unroll
      for (int a = 0; a < BACK_PAIRS; ++a) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot[a] += __shfl_xor_sync(0xffffffffu, dot[a], o);
        if (lane == 0) part[warp][a] = dot[a];
      }
      __syncthreads();
      if (threadIdx.x < BACK_PAIRS && k0 + static_cast<int>(threadIdx.x) < K) {
        float s = 0.f;
        for (int w = 0; w < warps; ++w) s += part[w][threadIdx.x];
        dweights[t * K + k0 + threadIdx.x] = s;  // 0 for a dropped pair
      }
      __syncthreads();
    }
  }
}

}  // namespace mc
