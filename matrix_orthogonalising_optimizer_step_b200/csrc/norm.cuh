// Root-mean-square norm with the residual's addition, and its gradient.
//
//   forward   h = x + r (stored in the inputs' type; x itself without r)
//             rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd w
//             y goes out as bf16 or in the 8-bit form of act8.cuh
//   backward  xhat = h rstd, g = dy w
//             dx = rstd (g - xhat mean(g xhat)) + dh,   dw = sum over rows of dy xhat
//             (dh: gradient reaching h past the norm; h as stored, in 8 bits if it was kept so)
//
// Both are bound by memory: a row is read once, kept in registers between its
// sum and its output, and written once.  `wpr` warps share a row (a warp holds
// 256 columns per fragment, NV fragments), so a block of 8 warps takes 8 / wpr
// rows; sums are fp32 trees of a fixed order.
#pragma once

#include "act8.cuh"

namespace mc {

constexpr int NORM_MAX_THREADS = 1024;
constexpr int NORM_MAX_COLS = 32768;  // 1024 threads x 4 fragments x 8 columns

// Sum over the `wpr` warps that share a row; every thread of the block calls it.
__device__ __forceinline__ float row_sum(float v, int wpr, float* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (wpr == 1) return v;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) buf[warp] = v;
  __syncthreads();
  const int w0 = warp / wpr * wpr;
  float t = 0.f;
  for (int i = 0; i < wpr; ++i) t += buf[w0 + i];
  return t;
}

// The norm's weight of one fragment (bf16 or fp32), 0 past D.
template <bool VEC>
__device__ __forceinline__ void load_weight(const void* w, int w_f32, int c0, int lane, int D, float (&v)[8]) {
  if (w_f32) {
    RawFrag<float> f;
    load_frag<VEC>(f, static_cast<const float*>(w), c0, lane, D);
    frag_floats(f, v);
  } else {
    RawFrag<__nv_bfloat16> f;
    load_frag<VEC>(f, static_cast<const __nv_bfloat16*>(w), c0, lane, D);
    frag_floats(f, v);
  }
}

template <typename T>
struct NormFwdArgs {
  const T* x;
  const T* r;          // residual or null
  const void* w;
  T* h;                // written when r is given
  __nv_bfloat16* y;    // ACT_NONE
  uint8_t* q;          // 8-bit output
  uint8_t* s;
  float* rstd;
  long long rows, q_ld, s_ld;
  int D, wpr, w_f32;
  float eps;
};

template <typename T, int FMT, bool VEC, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) rms_norm_kernel(const NormFwdArgs<T> a) {
  __shared__ float buf[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = (blockDim.x >> 5) / a.wpr;
  const long long row = (long long)blockIdx.x * groups + warp / a.wpr;
  const int wr = warp % a.wpr;
  const bool live = row < a.rows;
  const long long base = row * a.D;
  float v[NV][8];
  float sum = 0.f;
  if (live) {
    RawFrag<T> fx[NV], fr[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) load_frag<VEC>(fx[j], a.x + base, (j * a.wpr + wr) * WARP_COLS, lane, a.D);
    if (a.r) {
#pragma unroll
      for (int j = 0; j < NV; ++j) load_frag<VEC>(fr[j], a.r + base, (j * a.wpr + wr) * WARP_COLS, lane, a.D);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      frag_floats(fx[j], v[j]);
      if (a.r) {
        float t[8];
        frag_floats(fr[j], t);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[j][i] += t[i];
          // the norm sees h as the next layers will: rounded to the stored type
          if constexpr (sizeof(T) == 2) v[j][i] = __bfloat162float(__float2bfloat16_rn(v[j][i]));
        }
        store_frag<VEC>(a.h + base, (j * a.wpr + wr) * WARP_COLS, lane, a.D, v[j]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(v[j][i], v[j][i], sum);
    }
  }
  sum = row_sum(sum, a.wpr, buf);
  if (!live) return;
  const float rstd = 1.f / sqrtf(sum / static_cast<float>(a.D) + a.eps);
  if (wr == 0 && lane == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c0 = (j * a.wpr + wr) * WARP_COLS;
    if (c0 >= a.D) break;
    float w[8];
    load_weight<VEC>(a.w, a.w_f32, c0, lane, a.D, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] = frag_col<VEC>(c0, lane, i) < a.D ? v[j][i] * rstd * w[i] : 0.f;
    if constexpr (FMT == ACT_NONE) {
      store_frag<VEC>(a.y + base, c0, lane, a.D, v[j]);
    } else {
      store_frag8<FMT, VEC>(a.q + row * a.q_ld, a.s + row * a.s_ld, c0, lane, a.D, v[j]);
    }
  }
}

template <typename T>
struct NormBwdArgs {
  const T* dy;
  const T* dh;         // or null
  const T* h;          // ACT_NONE
  const uint8_t* q;    // h in 8 bits
  const uint8_t* s;
  const void* w;
  const float* rstd;
  T* dx;
  float* partial;      // [gridDim * groups][D] sums of dy xhat
  long long rows, q_ld, s_ld;
  int D, wpr, w_f32;
};

template <typename T, int FMT>
struct NormBwdRaw {
  RawFrag<T> dy, dh, h;
};
template <typename T>
struct NormBwdRaw<T, ACT_E4M3> {
  RawFrag<T> dy, dh;
  Raw8 h;
};
template <typename T>
struct NormBwdRaw<T, ACT_INT8> {
  RawFrag<T> dy, dh;
  Raw8 h;
};

// A block walks rows with a fixed step and keeps dw of its columns in
// registers; the next row's loads are issued before this row's sum, so that
// the memory stays busy across the block-wide reduction.
template <typename T, int FMT, bool VEC, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) rms_norm_bwd_kernel(const NormBwdArgs<T> a) {
  __shared__ float buf[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = (blockDim.x >> 5) / a.wpr;
  const int group = warp / a.wpr, wr = warp % a.wpr;
  const long long step = (long long)gridDim.x * groups;
  const float inv_d = 1.f / static_cast<float>(a.D);
  float dw[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;

  auto load = [&](long long row, NormBwdRaw<T, FMT>(&f)[NV], float& rstd) {
    if (row >= a.rows) return;
    rstd = a.rstd[row];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c0 = (j * a.wpr + wr) * WARP_COLS;
      if (c0 >= a.D) break;
      load_frag<VEC>(f[j].dy, a.dy + row * a.D, c0, lane, a.D);
      if constexpr (FMT == ACT_NONE) {
        load_frag<VEC>(f[j].h, a.h + row * a.D, c0, lane, a.D);
      } else {
        load_frag8<VEC>(f[j].h, a.q + row * a.q_ld, a.s + row * a.s_ld, c0, lane, a.D);
      }
      if (a.dh) load_frag<VEC>(f[j].dh, a.dh + row * a.D, c0, lane, a.D);
    }
  };
  auto values = [&](const NormBwdRaw<T, FMT>& f, int c0, float rstd, float (&dy)[8], float (&xhat)[8]) {
    frag_floats(f.dy, dy);
    if constexpr (FMT == ACT_NONE) {
      frag_floats(f.h, xhat);
    } else {
      frag8_floats<FMT, VEC>(f.h, c0, lane, a.D, xhat);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) xhat[i] *= rstd;
  };

  NormBwdRaw<T, FMT> cur[NV], next[NV];
  float rstd = 0.f, rstd_next = 0.f;
  long long row = (long long)blockIdx.x * groups + group;
  long long first = (long long)blockIdx.x * groups;  // the loop is uniform over the block
  load(row, cur, rstd);
  int flip = 0;
  for (; first < a.rows; first += step, row += step) {
    load(row + step, next, rstd_next);
    const bool live = row < a.rows;
    float dot = 0.f;
    if (live) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c0 = (j * a.wpr + wr) * WARP_COLS;
        if (c0 >= a.D) break;
        float dy[8], xhat[8], w[8];
        values(cur[j], c0, rstd, dy, xhat);
        load_weight<VEC>(a.w, a.w_f32, c0, lane, a.D, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool in = frag_col<VEC>(c0, lane, i) < a.D;
          const float p = in ? dy[i] * xhat[i] : 0.f;
          dw[j][i] += p;
          dot = fmaf(p, w[i], dot);
        }
      }
    }
    // two buffers in turn: a warp still reading one row's sums never meets the next row's writes
    const float c = row_sum(dot, a.wpr, buf[flip]) * inv_d;
    flip ^= 1;
    if (live) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c0 = (j * a.wpr + wr) * WARP_COLS;
        if (c0 >= a.D) break;
        float dy[8], xhat[8], w[8], o[8];
        values(cur[j], c0, rstd, dy, xhat);
        load_weight<VEC>(a.w, a.w_f32, c0, lane, a.D, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = rstd * (dy[i] * w[i] - xhat[i] * c);
        if (a.dh) {
          float t[8];
          frag_floats(cur[j].dh, t);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] += t[i];
        }
        store_frag<VEC>(a.dx + row * a.D, c0, lane, a.D, o);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) cur[j] = next[j];
    rstd = rstd_next;
  }
  float* out = a.partial + ((long long)blockIdx.x * groups + group) * a.D;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c0 = (j * a.wpr + wr) * WARP_COLS;
    if (c0 >= a.D) break;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = frag_col<VEC>(c0, lane, i);
      if (c < a.D) out[c] = dw[j][i];
    }
  }
}

// dw[c] = sum of the partial rows, each column's in a fixed order: warp w of a
// block takes rows w, w + 16, ..., then the 16 sums are added in turn.
constexpr int NORM_DW_WARPS = 16;
__global__ void __launch_bounds__(NORM_DW_WARPS * 32) rms_norm_dw_kernel(const float* __restrict__ partial, float* __restrict__ dw,
                                                                         int parts, int D) {
  __shared__ float buf[NORM_DW_WARPS][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float t[4] = {0.f, 0.f, 0.f, 0.f};
  if (c < D) {
    int p = warp;
    for (; p + 3 * NORM_DW_WARPS < parts; p += 4 * NORM_DW_WARPS) {
#pragma unroll
      for (int u = 0; u < 4; ++u) t[u] += partial[(long long)(p + u * NORM_DW_WARPS) * D + c];
    }
    for (; p < parts; p += NORM_DW_WARPS) t[0] += partial[(long long)p * D + c];
  }
  buf[warp][lane] = (t[0] + t[1]) + (t[2] + t[3]);
  __syncthreads();
  if (warp == 0 && c < D) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < NORM_DW_WARPS; ++w) v += buf[w][lane];
    dw[c] = v;
  }
}

}  // namespace mc
