// Root-mean-square norm with the residual's addition, and its gradient.
//
//   forward   h = x + r (stored in the inputs' type; x itself without r)
//             rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd w
//             y goes out as bf16 or in the 8-bit form of act8.cuh
//   backward  xhat = h rstd, g = dy w
//             dx = rstd (g - xhat mean(g xhat)) + dh,   dw = sum over rows of dy xhat
//             (dh: gradient reaching h past the norm; h as stored, in 8 bits if it was kept so)
//
// Both are bound by memory: a row is read once, kept in registers (forward) or
// shared memory (backward) between its sum and its output, and written once.
// `wpr` warps share a row (a warp holds 256 columns per fragment, NV fragments),
// so a block of 8 warps takes 8 / wpr rows; sums are trees of a fixed order.
// Measured on 16384 x 4096 bf16 rows: forward with residual and e4m3 output 79 us
// (472 MB, 6.0 TB/s of the 6.55 a copy reaches here), to bf16 84 us (537 MB, 6.4 TB/s),
// backward 94 us (537 MB, 5.7 TB/s) with under 8 us for the sum of dw's parts in it.
#pragma once

#include "act8.cuh"

namespace mc {

constexpr int NORM_MAX_THREADS = 1024;
constexpr int NORM_MAX_COLS = 32768;  // 1024 threads x 4 fragments x 8 columns

// Sum over the `wpr` warps that share a row, warps w0.. of the block, of which
// this is the wr-th; every thread of the block calls it.
template <typename F>
__device__ __forceinline__ F row_sum(F v, int wpr, int w0, int wr, F* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (wpr == 1) return v;
  if ((threadIdx.x & 31) == 0) buf[w0 + wr] = v;
  __syncthreads();
  F t = 0;
  for (int i = 0; i < wpr; ++i) t += buf[w0 + i];
  return t;
}

// 1 / sqrt(m) to about 2^-43: the fp32 estimate and one Newton step; outside
// its range (and for m = 0, infinities and NaN) the library's square root.
__device__ __forceinline__ double rsqrt64(double m) {
  if (m > 1e-37 && m < 1e38) {
    const double r = rsqrtf(static_cast<float>(m));
    return r * (1.5 - 0.5 * m * r * r);
  }
  return 1.0 / sqrt(m);
}

// v * r * w of eight values for an 8-bit output, r given as r_hi + r_lo: fp32 numbers
// that round to 8 bits as the products themselves do.  The products are known to
// about 2^-43 and rounded to the nearest fp32 number, which lies on the same side
// as the product of everything that decides a code or a scale, the middle of two
// codes and the largest value of a scale: those have at most 8 significant bits.  Only
// a result that has as few may have been rounded to such a border; it goes
// back to the side that the product is on, one step off, unless the product
// is within 2^-40 of it: that is the border (a tie, to even; the largest value, in its scale).
// BF16: v and w are bf16 numbers, whose product is exact in fp32.
template <bool BF16>
__device__ __forceinline__ void scaled_for_codes(float (&v)[8], const float (&w)[8], float r_hi, float r_lo) {
  auto factors = [&](int i, float& x, float& t_hi, float& t_lo) {
    if constexpr (BF16) {
      x = v[i] * w[i];
      t_hi = r_hi;
      t_lo = r_lo;
    } else {
      x = v[i];
      t_hi = r_hi * w[i];
      t_lo = fmaf(r_lo, w[i], fmaf(r_hi, w[i], -t_hi));
    }
  };
  float p[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float x, t_hi, t_lo;
    factors(i, x, t_hi, t_lo);
    p[i] = fmaf(x, t_hi, x * t_lo);
  }
  // the least lower half of the eight words
  auto word = [&](int i) { return __float_as_uint(p[i]); };
  const uint32_t least = __vminu2(__vimin3_u16x2(__vimin3_u16x2(word(0), word(1), word(2)), word(3), word(4)),
                                  __vimin3_u16x2(word(5), word(6), word(7)));
  if ((least & 0xFFFFu) == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (__float_as_uint(p[i]) & 0xFFFFu) continue;
      float x, t_hi, t_lo;
      factors(i, x, t_hi, t_lo);
      const float rest = fmaf(x, t_hi, -p[i]) + x * t_lo;
      if (fabsf(rest) > 0x1p-40f * fabsf(p[i]))
        p[i] = __int_as_float(__float_as_int(p[i]) + ((rest > 0.f) == (p[i] > 0.f) ? 1 : -1));
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = p[i];
}

// The norm's weight of one fragment (bf16 or fp32), 0 past D.
template <int G>
__device__ __forceinline__ void load_weight(const void* w, int w_f32, int c0, int lane, int D, float (&v)[8]) {
  if (w_f32) {
    RawFrag<float> f;
    load_frag<G>(f, static_cast<const float*>(w), c0, lane, D);
    frag_floats(f, v);
  } else {
    RawFrag<__nv_bfloat16> f;
    load_frag<G>(f, static_cast<const __nv_bfloat16*>(w), c0, lane, D);
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
  int D, w_f32;
  float eps;
  double d, inv_d;     // D and 1 / D
};

// The sum of squares is kept in 64 bits beyond each fragment's eight terms: its
// error would move every value of the row the same way.  (Every square in 64
// bits: 115 us for 16384 x 4096 bf16 rows, bound by the conversions.)
// Four blocks an SM for bf16 rows: left to itself the compiler takes a few registers
// more than that allows (16384 x 4096: 88 us, 8192 x 4095: 111 us; so 79 and 85).
template <typename T, int FMT, int G, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS <= 256 && sizeof(T) == 2 ? 4 : 1) rms_norm_kernel(const NormFwdArgs<T> a) {
  __shared__ double buf[32];
  griddep_launch_dependents();
  // blockDim: {32 * warps of a row, rows}
  const int lane = threadIdx.x & 31, wr = threadIdx.x >> 5, wpr = blockDim.x >> 5;
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = row < a.rows;
  const long long base = row * a.D;
  RawFrag<T> f[NV];
  double sum = 0.0;
  if (live) {
#pragma unroll
    for (int j = 0; j < NV; ++j) load_frag<G>(f[j], a.x + base, (j * wpr + wr) * WARP_COLS, lane, a.D);
    if (a.r) {
      RawFrag<T> fr[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) load_frag<G>(fr[j], a.r + base, (j * wpr + wr) * WARP_COLS, lane, a.D);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        frag_add(f[j], fr[j]);  // the norm sees h as the next layers will: in the stored type
        store_raw<G>(a.h + base, (j * wpr + wr) * WARP_COLS, lane, a.D, f[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float v[8];
      frag_floats(f[j], v);
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) t = fmaf(v[i], v[i], t);
      sum += static_cast<double>(t);
    }
  }
  sum = row_sum(sum, wpr, threadIdx.y * wpr, wr, buf);
  if (!live) return;
  // sum / D: exact where it is a number of 53 bits (an infinite sum stays so)
  const double near = sum * a.inv_d;
  const double mean = fma(fma(-near, a.d, sum), a.inv_d, near);
  const double r64 = rsqrt64((mean == mean ? mean : near) + static_cast<double>(a.eps));
  const float rstd = static_cast<float>(r64);
  const float r_lo = static_cast<float>(r64 - static_cast<double>(rstd));
  if (wr == 0 && lane == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c0 = (j * wpr + wr) * WARP_COLS;
    if (c0 >= a.D) break;
    float v[8], w[8];
    frag_floats(f[j], v);
    load_weight<G>(a.w, a.w_f32, c0, lane, a.D, w);
    // columns past D hold x = w = 0
    if constexpr (FMT == ACT_NONE) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] * rstd * w[i];
      store_frag<G>(a.y + base, c0, lane, a.D, v);
    } else {
      if (sizeof(T) == 2 && !a.w_f32) {
        scaled_for_codes<true>(v, w, rstd, r_lo);
      } else {
        scaled_for_codes<false>(v, w, rstd, r_lo);
      }
      store_frag8<FMT, G>(a.q + row * a.q_ld, a.s + row * a.s_ld, c0, lane, a.D, v);
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
template <typename T, int FMT, int G, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS <= 256 ? 2 : 1) rms_norm_bwd_kernel(const NormBwdArgs<T> a) {
  __shared__ float buf[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = (blockDim.x >> 5) / a.wpr;
  const int group = warp / a.wpr, wr = warp % a.wpr;
  const long long step = (long long)gridDim.x * groups;
  const float inv_d = 1.f / static_cast<float>(a.D);
  griddep_launch_dependents();  // the sum over the parts may get ready
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
      load_frag<G>(f[j].dy, a.dy + row * a.D, c0, lane, a.D);
      if constexpr (FMT == ACT_NONE) {
        load_frag<G>(f[j].h, a.h + row * a.D, c0, lane, a.D);
      } else {
        load_frag8<G>(f[j].h, a.q + row * a.q_ld, a.s + row * a.s_ld, c0, lane, a.D);
      }
      if (a.dh) load_frag<G>(f[j].dh, a.dh + row * a.D, c0, lane, a.D);
    }
  };
  auto values = [&](const NormBwdRaw<T, FMT>& f, int c0, float rstd, float (&dy)[8], float (&xhat)[8]) {
    frag_floats(f.dy, dy);
    if constexpr (FMT == ACT_NONE) {
      frag_floats(f.h, xhat);
    } else {
      frag8_floats<FMT, G>(f.h, c0, lane, a.D, xhat);
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
        load_weight<G>(a.w, a.w_f32, c0, lane, a.D, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool in = frag_col<G>(c0, lane, i) < a.D;
          const float p = in ? dy[i] * xhat[i] : 0.f;
          dw[j][i] += p;
          dot = fmaf(p, w[i], dot);
        }
      }
    }
    // two buffers in turn: a warp still reading one row's sums never meets the next row's writes
    const float c = row_sum(dot, a.wpr, group * a.wpr, wr, buf[flip]) * inv_d;
    flip ^= 1;
    if (live) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c0 = (j * a.wpr + wr) * WARP_COLS;
        if (c0 >= a.D) break;
        float dy[8], xhat[8], w[8], o[8];
        values(cur[j], c0, rstd, dy, xhat);
        load_weight<G>(a.w, a.w_f32, c0, lane, a.D, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = rstd * (dy[i] * w[i] - xhat[i] * c);
        if (a.dh) {
          float t[8];
          frag_floats(cur[j].dh, t);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] += t[i];
        }
        store_frag<G>(a.dx + row * a.D, c0, lane, a.D, o);
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
      const int c = frag_col<G>(c0, lane, i);
      if (c < a.D) out[c] = dw[j][i];
    }
  }
}

// The same for rows of whole 16-byte words that fit in shared memory: a
// producer warp copies rows (bulk asynchronous copies) into a ring of stages, as
// many as the shared memory of half an SM holds, and the other warps read them
// twice from there, for the row's sum and for its output, so that what is in
// flight does not depend on registers.  dw and the weight stay in registers.
// A stage holds one row for each of the block's groups of `wpr` warps.
// (The next row's loads in registers instead, as above: 137 us for the 95 us
// case; 122 registers left two blocks an SM and half the bytes in flight.)
struct NormRing {
  int stages, stage_bytes;
  int off_dh, off_h, off_s;             // of a stage's dh rows, h rows (or codes) and scale bytes (dy at 0)
  int row_bytes, q_row, s_row;          // bytes of a row of dy, of codes, of scale bytes
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}
// Barrier of one group of warps; returns whether any of its threads brought `p`,
// the same answer to all of them (so that they leave a loop together).
__device__ __forceinline__ bool group_any(int id, int threads, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\t"
      "setp.ne.u32 a, %3, 0;\n\t"
      "barrier.cta.red.or.pred b, %1, %2, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(p ? 1u : 0u)
      : "memory");
  return r != 0;
}

constexpr int NORM_RING_STAGES = 8;
template <typename T, int FMT, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS + 32, THREADS <= 256 ? 2 : 1) rms_norm_bwd_ring_kernel(const NormBwdArgs<T> a, const NormRing R,
                                                                                             int* err) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full_bar[NORM_RING_STAGES], empty_bar[NORM_RING_STAGES];
  __shared__ float buf[2][32];
  __shared__ int abort_flag;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int workers = (blockDim.x >> 5) - 1;
  const int groups = workers / a.wpr;
  if (threadIdx.x == 0) {
    for (int i = 0; i < R.stages; ++i) {
      mbar_init(smem_u32(&full_bar[i]), 1);
      mbar_init(smem_u32(&empty_bar[i]), workers);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  griddep_launch_dependents();  // the sum over the parts may get ready
  const long long step = (long long)gridDim.x * groups;
  if (warp == workers) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, filled = 0, parity = 0;
      for (long long row = (long long)blockIdx.x * groups; row < a.rows; row += step) {
        if (!wait_bounded(smem_u32(&empty_bar[stage]), phase ^ 1, &abort_flag, err)) break;
        const int n = static_cast<int>(min(static_cast<long long>(groups), a.rows - row));
        const uint32_t dst = smem_u32(ring) + stage * R.stage_bytes, bar = smem_u32(&full_bar[stage]);
        const uint32_t rows_bytes = static_cast<uint32_t>(n) * R.row_bytes;
        mbar_arrive_expect_tx(bar, rows_bytes * (a.dh ? 2u : 1u) +
                                       (FMT == ACT_NONE ? rows_bytes : static_cast<uint32_t>(n) * (R.q_row + R.s_row)));
        bulk_load(dst, a.dy + row * a.D, rows_bytes, bar);
        if (a.dh) bulk_load(dst + R.off_dh, a.dh + row * a.D, rows_bytes, bar);
        if constexpr (FMT == ACT_NONE) {
          bulk_load(dst + R.off_h, a.h + row * a.D, rows_bytes, bar);
        } else {
          for (int g = 0; g < n; ++g) {
            bulk_load(dst + R.off_h + g * R.q_row, a.q + (row + g) * a.q_ld, R.q_row, bar);
            bulk_load(dst + R.off_s + g * R.s_row, a.s + (row + g) * a.s_ld, R.s_row, bar);
          }
        }
        filled |= 1u << stage;
        parity = (parity & ~(1u << stage)) | (phase << stage);
        if (++stage == R.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      // every copy lands before the block leaves
      for (int i = 0; i < R.stages; ++i)
        if (filled & (1u << i)) {
          volatile int no_abort = 0;
          wait_bounded(smem_u32(&full_bar[i]), (parity >> i) & 1u, &no_abort, nullptr, kDrainLimitCycles);
        }
    }
    return;
  }
  // --------------------------------------------------------------- workers
  const int group = warp / a.wpr, wr = warp % a.wpr;
  const float inv_d = 1.f / static_cast<float>(a.D);
  float dw[NV][8], w[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    load_weight<8>(a.w, a.w_f32, (j * a.wpr + wr) * WARP_COLS, lane, a.D, w[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.f;
  }
  int stage = 0, flip = 0;
  uint32_t phase = 0;
  for (long long first = (long long)blockIdx.x * groups; first < a.rows; first += step) {
    const long long row = first + group;
    bool live = row < a.rows;
    const uint8_t* st = ring + stage * R.stage_bytes;
    const T* s_dy = reinterpret_cast<const T*>(st + group * R.row_bytes);
    const T* s_dh = reinterpret_cast<const T*>(st + R.off_dh + group * R.row_bytes);
    const T* s_h = reinterpret_cast<const T*>(st + R.off_h + group * R.row_bytes);
    const uint8_t* s_q = st + R.off_h + group * R.q_row;
    const uint8_t* s_s = st + R.off_s + group * R.s_row;
    const float rstd = live ? a.rstd[row] : 0.f;
    const bool got = __all_sync(0xffffffffu, wait_bounded(smem_u32(&full_bar[stage]), phase, &abort_flag, err));
    live = live && got;
    auto values = [&](int c0, float (&dy)[8], float (&xhat)[8]) {
      RawFrag<T> f;
      load_frag<8>(f, s_dy, c0, lane, a.D);
      frag_floats(f, dy);
      if constexpr (FMT == ACT_NONE) {
        load_frag<8>(f, s_h, c0, lane, a.D);
        frag_floats(f, xhat);
      } else {
        Raw8 q;
        load_frag8<8>(q, s_q, s_s, c0, lane, a.D);
        frag8_floats<FMT, 8>(q, c0, lane, a.D, xhat);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) xhat[i] *= rstd;
    };
    float dot = 0.f;
    if (live) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c0 = (j * a.wpr + wr) * WARP_COLS;
        if (c0 >= a.D) break;
        float dy[8], xhat[8];
        values(c0, dy, xhat);  // zeros past D
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = dy[i] * xhat[i];
          dw[j][i] += p;
          dot = fmaf(p, w[j][i], dot);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (a.wpr > 1) {
      // two buffers in turn, as above; the groups go their own pace
      if (lane == 0) buf[flip][warp] = dot;
      if (group_any(1 + group, 32 * a.wpr, !got)) break;
      dot = 0.f;
      for (int i = 0; i < a.wpr; ++i) dot += buf[flip][group * a.wpr + i];
      flip ^= 1;
    } else if (!got) {
      break;
    }
    const float c = dot * inv_d;
    if (live) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c0 = (j * a.wpr + wr) * WARP_COLS;
        if (c0 >= a.D) break;
        float dy[8], xhat[8], o[8];
        values(c0, dy, xhat);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = rstd * fmaf(-xhat[i], c, dy[i] * w[j][i]);
        if (a.dh) {
          RawFrag<T> f;
          float t[8];
          load_frag<8>(f, s_dh, c0, lane, a.D);
          frag_floats(f, t);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] += t[i];
        }
        store_frag<8>(a.dx + row * a.D, c0, lane, a.D, o);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&empty_bar[stage]));
    if (++stage == R.stages) {
      stage = 0;
      phase ^= 1;
    }
  }
  float* out = a.partial + ((long long)blockIdx.x * groups + group) * a.D;
#pragma unroll
  for (int j = 0; j < NV; ++j) store_frag<8>(out, (j * a.wpr + wr) * WARP_COLS, lane, a.D, dw[j]);
}

// dw[c] = sum of the partial rows, each column's in a fixed order: warp w of a
// block takes rows w, w + 16, ..., then the 16 sums are added in turn.
constexpr int NORM_DW_WARPS = 16;
__global__ void __launch_bounds__(NORM_DW_WARPS * 32) rms_norm_dw_kernel(const float* partial, float* dw, int parts, int D) {
  __shared__ float buf[NORM_DW_WARPS][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  griddep_wait();  // launched while the walk still runs: no __restrict__, so no read-only loads
  constexpr int AHEAD = 8;
  float t[AHEAD];
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) t[u] = 0.f;
  if (c < D) {
    for (int p = warp; p < parts; p += AHEAD * NORM_DW_WARPS) {
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int r = p + u * NORM_DW_WARPS;
        if (r < parts) t[u] += partial[(long long)r * D + c];
      }
    }
  }
  buf[warp][lane] = ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
  __syncthreads();
  if (warp == 0 && c < D) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < NORM_DW_WARPS; ++w) v += buf[w][lane];
    dw[c] = v;
  }
}

}  // namespace mc
