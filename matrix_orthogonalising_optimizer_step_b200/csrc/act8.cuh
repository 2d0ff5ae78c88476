// Activations in 8 bits: blocks of 32 consecutive columns of a row, one scale
// byte s each (standing for 2^(s - 127); 255: the block is NaN) and one code per
// value, an e4m3 number or an int8.
//
//   pack    k = least integer >= -120 with max|x| <= TOP 2^k (TOP = 448 or 127),
//           s = k + 127, code = x 2^-k to the nearest, ties to even
//   unpack  x' = code 2^(s - 127)
//
// A power of two as the scale costs int8 up to one bit of its eight, and
// makes every x' exact in bf16 (at most 8 significant bits; k >= -120 keeps
// the least code above bf16's subnormal step), so that products of x' on the
// tensor cores see exactly the stored values, and whoever quantises the same
// bf16 numbers gets the same bytes.
//
// All kernels here and the norm kernels share one mapping of columns to
// threads: a warp holds 256 consecutive columns of a row, eight values a
// lane.  VEC (rows of whole 16-byte words): lane l holds columns 8l..8l+7, a
// block is four neighbouring lanes.  Otherwise: value i of lane l is column
// 32i + l, a block is one value of all 32 lanes; single elements are loaded,
// but neighbouring lanes still touch neighbouring addresses.
#pragma once

#include "ptx.cuh"

namespace mc {

enum ActFmt : int { ACT_NONE = 0, ACT_E4M3 = 1, ACT_INT8 = 2 };
constexpr int ACT_BLOCK = 32;
constexpr int WARP_COLS = 256;

// ---------------------------------------------------------------- fragments
template <bool VEC>
__device__ __forceinline__ int frag_col(int c0, int lane, int i) {
  return VEC ? c0 + 8 * lane + i : c0 + 32 * i + lane;
}

// Raw words of one fragment: loaded early, turned into floats when needed.
template <typename T>
struct RawFrag;
template <>
struct RawFrag<__nv_bfloat16> {
  uint4 q;
};
template <>
struct RawFrag<float> {
  float4 a, b;
};

template <bool VEC>
__device__ __forceinline__ void load_frag(RawFrag<__nv_bfloat16>& f, const __nv_bfloat16* row, int c0, int lane, int D) {
  if constexpr (VEC) {
    const int c = c0 + 8 * lane;
    f.q = c < D ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0u, 0u, 0u, 0u);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ca = c0 + 64 * i + lane, cb = ca + 32;
      const uint32_t lo = ca < D ? *reinterpret_cast<const uint16_t*>(row + ca) : 0u;
      const uint32_t hi = cb < D ? *reinterpret_cast<const uint16_t*>(row + cb) : 0u;
      w[i] = lo | (hi << 16);
    }
    f.q = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
template <bool VEC>
__device__ __forceinline__ void load_frag(RawFrag<float>& f, const float* row, int c0, int lane, int D) {
  if constexpr (VEC) {
    const int c = c0 + 8 * lane;
    const float4* p = reinterpret_cast<const float4*>(row + c);
    f.a = c < D ? p[0] : make_float4(0.f, 0.f, 0.f, 0.f);
    f.b = c < D ? p[1] : make_float4(0.f, 0.f, 0.f, 0.f);
  } else {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = c0 + 32 * i + lane;
      w[i] = c < D ? row[c] : 0.f;
    }
    f.a = make_float4(w[0], w[1], w[2], w[3]);
    f.b = make_float4(w[4], w[5], w[6], w[7]);
  }
}
__device__ __forceinline__ void frag_floats(const RawFrag<__nv_bfloat16>& f, float (&v)[8]) {
  const uint32_t w[4] = {f.q.x, f.q.y, f.q.z, f.q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void frag_floats(const RawFrag<float>& f, float (&v)[8]) {
  v[0] = f.a.x; v[1] = f.a.y; v[2] = f.a.z; v[3] = f.a.w;
  v[4] = f.b.x; v[5] = f.b.y; v[6] = f.b.z; v[7] = f.b.w;
}

template <bool VEC>
__device__ __forceinline__ void store_frag(__nv_bfloat16* row, int c0, int lane, int D, const float (&v)[8]) {
  if constexpr (VEC) {
    const int c = c0 + 8 * lane;
    if (c < D)
      *reinterpret_cast<uint4*>(row + c) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                      pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = c0 + 32 * i + lane;
      if (c < D) row[c] = __float2bfloat16_rn(v[i]);
    }
  }
}
template <bool VEC>
__device__ __forceinline__ void store_frag(float* row, int c0, int lane, int D, const float (&v)[8]) {
  if constexpr (VEC) {
    const int c = c0 + 8 * lane;
    if (c < D) {
      float4* p = reinterpret_cast<float4*>(row + c);
      p[0] = make_float4(v[0], v[1], v[2], v[3]);
      p[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = c0 + 32 * i + lane;
      if (c < D) row[c] = v[i];
    }
  }
}

// f + g, rounded to the type.  Two bf16 numbers: their sum is exact in fp32
// unless they are so far apart (over 2^16) that it rounds to the larger one, so
// one rounding and the detour over fp32 give the same.
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 s = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&s);
}
__device__ __forceinline__ void frag_add(RawFrag<__nv_bfloat16>& f, const RawFrag<__nv_bfloat16>& g) {
  f.q = make_uint4(add_bf16x2(f.q.x, g.q.x), add_bf16x2(f.q.y, g.q.y), add_bf16x2(f.q.z, g.q.z), add_bf16x2(f.q.w, g.q.w));
}
__device__ __forceinline__ void frag_add(RawFrag<float>& f, const RawFrag<float>& g) {
  f.a = make_float4(f.a.x + g.a.x, f.a.y + g.a.y, f.a.z + g.a.z, f.a.w + g.a.w);
  f.b = make_float4(f.b.x + g.b.x, f.b.y + g.b.y, f.b.z + g.b.z, f.b.w + g.b.w);
}
// The fragment as it is to memory.
template <bool VEC, typename T>
__device__ __forceinline__ void store_raw(T* row, int c0, int lane, int D, const RawFrag<T>& f) {
  if constexpr (VEC && sizeof(T) == 2) {
    const int c = c0 + 8 * lane;
    if (c < D) *reinterpret_cast<uint4*>(row + c) = f.q;
  } else {
    float v[8];
    frag_floats(f, v);
    store_frag<VEC>(row, c0, lane, D, v);
  }
}

// max(|a|, |b|), NaN if either is
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// ------------------------------------------------------------------- codes
// k of a block whose largest |x| has these bits; any finite value.
template <int FMT>
__device__ __forceinline__ int act_exponent(uint32_t amax_bits) {
  // TOP 2^k >= amax  <=>  the significand of amax is at most TOP's, at TOP's binade
  constexpr uint32_t TOP_FRACTION = FMT == ACT_E4M3 ? 0x600000u : 0x7E0000u;  // 448 = 1.75 2^8, 127 = 1.984375 2^6
  constexpr int TOP_EXP = FMT == ACT_E4M3 ? 8 : 6;
  const int k = static_cast<int>(amax_bits >> 23) - 127 - TOP_EXP + ((amax_bits & 0x7FFFFFu) > TOP_FRACTION ? 1 : 0);
  return k < -120 ? -120 : k;
}
// 2^e for -126 <= e <= 127
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }
// The value of a scale byte.
__device__ __forceinline__ float act_scale_value(uint32_t s) {
  return __uint_as_float(s == 255u ? 0x7FC00000u : (s == 0u ? 0x00400000u : s << 23));
}

template <int FMT>
__device__ __forceinline__ uint32_t act_encode2(float lo, float hi) {
  if constexpr (FMT == ACT_E4M3) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
  } else {
    return (static_cast<uint32_t>(__float2int_rn(lo)) & 0xFFu) | ((static_cast<uint32_t>(__float2int_rn(hi)) & 0xFFu) << 8);
  }
}
template <int FMT>
__device__ __forceinline__ float2 act_decode2(uint32_t two) {
  if constexpr (FMT == ACT_E4M3) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
    return __half22float2(*reinterpret_cast<__half2*>(&h));
  } else {
    return make_float2(static_cast<float>(static_cast<int8_t>(two & 0xFFu)),
                       static_cast<float>(static_cast<int8_t>((two >> 8) & 0xFFu)));
  }
}

// One fragment to 8 bits.  All 32 lanes take part; columns at or past D hold 0.
template <int FMT, bool VEC>
__device__ __forceinline__ void store_frag8(uint8_t* qrow, uint8_t* srow, int c0, int lane, int D, const float (&v)[8]) {
  if constexpr (VEC) {
    float big = max_abs(max_abs(max_abs(v[0], v[1]), max_abs(v[2], v[3])), max_abs(max_abs(v[4], v[5]), max_abs(v[6], v[7])));
    big = max_abs(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = max_abs(big, __shfl_xor_sync(0xffffffffu, big, 2));
    const uint32_t m = __float_as_uint(big);
    const bool fine = m < 0x7F800000u;
    const int k = act_exponent<FMT>(m);
    const float r = exp2_int(-k);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = act_encode2<FMT>(v[4 * i] * r, v[4 * i + 1] * r) | (act_encode2<FMT>(v[4 * i + 2] * r, v[4 * i + 3] * r) << 16);
    const int c = c0 + 8 * lane;
    if (c < D) {
      *reinterpret_cast<uint2*>(qrow + c) = fine ? make_uint2(w[0], w[1]) : make_uint2(0u, 0u);
      if ((lane & 3) == 0) srow[c / ACT_BLOCK] = fine ? static_cast<uint8_t>(k + 127) : 255;
    }
  } else {
    // lane i (mod 8) works out block i's scale, for all lanes
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t mi = __reduce_max_sync(0xffffffffu, __float_as_uint(v[i]) & 0x7FFFFFFFu);
      if ((lane & 7) == i) m = mi;
    }
    const bool fine = m < 0x7F800000u;
    const int k = act_exponent<FMT>(m);
    const float r = fine ? exp2_int(-k) : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float ri = __shfl_sync(0xffffffffu, r, i);
      const uint32_t code = act_encode2<FMT>(v[i] * ri, 0.f);
      const int c = c0 + 32 * i + lane;
      if (c < D) qrow[c] = ri > 0.f ? static_cast<uint8_t>(code) : 0;
    }
    if (lane < 8 && c0 + 32 * lane < D) srow[c0 / ACT_BLOCK + lane] = fine ? static_cast<uint8_t>(k + 127) : 255;
  }
}

// Raw codes and scale bytes of one fragment.
struct Raw8 {
  uint2 q;
  uint2 s;
};
template <bool VEC>
__device__ __forceinline__ void load_frag8(Raw8& f, const uint8_t* qrow, const uint8_t* srow, int c0, int lane, int D) {
  if constexpr (VEC) {
    const int c = c0 + 8 * lane;
    f.q = c < D ? *reinterpret_cast<const uint2*>(qrow + c) : make_uint2(0u, 0u);
    f.s.x = c < D ? srow[c / ACT_BLOCK] : 0u;
  } else {
    // the eight scale bytes of these columns (srow rows are 16-byte aligned and padded to 16 bytes)
    f.s = *reinterpret_cast<const uint2*>(srow + c0 / ACT_BLOCK);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = c0 + 32 * i + lane;
      const uint32_t b = c < D ? qrow[c] : 0u;
      w[i >> 2] |= b << (8 * (i & 3));
    }
    f.q = make_uint2(w[0], w[1]);
  }
}
template <int FMT, bool VEC>
__device__ __forceinline__ void frag8_floats(const Raw8& f, int c0, int lane, int D, float (&v)[8]) {
  const uint32_t w[2] = {f.q.x, f.q.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = act_decode2<FMT>(w[i] & 0xFFFFu), b = act_decode2<FMT>(w[i] >> 16);
    v[4 * i] = a.x;
    v[4 * i + 1] = a.y;
    v[4 * i + 2] = b.x;
    v[4 * i + 3] = b.y;
  }
  if constexpr (VEC) {
    const float s = act_scale_value(f.s.x);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= s;
  } else {
    // a column past D multiplies by no scale: the bytes behind the last block are not read as one
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t s = ((i < 4 ? f.s.x : f.s.y) >> (8 * (i & 3))) & 0xFFu;
      v[i] = c0 + 32 * i + lane < D ? v[i] * act_scale_value(s) : 0.f;
    }
  }
}

// -------------------------------------------------------------- pack, unpack
// Work items are (row, 256-column chunk) pairs, one per warp and step; a warp
// takes UNROLL items at once so that their loads are in flight together.
struct RowWalk {
  long long row;
  int chunk;
};
__device__ __forceinline__ void walk_next(RowWalk& w, long long step_rows, int step_chunks, int chunks) {
  w.row += step_rows;
  w.chunk += step_chunks;
  if (w.chunk >= chunks) {
    w.chunk -= chunks;
    ++w.row;
  }
}

constexpr int ACT_THREADS = 256;

template <typename T, int FMT, bool VEC>
__global__ void __launch_bounds__(ACT_THREADS) act8_pack_kernel(const T* __restrict__ x, uint8_t* __restrict__ q,
                                                                uint8_t* __restrict__ s, long long rows, int D,
                                                                long long q_ld, long long s_ld, int chunks) {
  constexpr int UNROLL = 4;
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (ACT_THREADS / 32);
  const long long first = (long long)blockIdx.x * (ACT_THREADS / 32) + (threadIdx.x >> 5);
  const long long step_rows = warps / chunks;
  const int step_chunks = static_cast<int>(warps % chunks);
  RowWalk w{first / chunks, static_cast<int>(first % chunks)};
  while (w.row < rows) {
    RowWalk at[UNROLL];
    RawFrag<T> f[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      at[u] = w;
      if (w.row < rows) load_frag<VEC>(f[u], x + w.row * D, w.chunk * WARP_COLS, lane, D);
      walk_next(w, step_rows, step_chunks, chunks);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (at[u].row >= rows) break;
      float v[8];
      frag_floats(f[u], v);
      store_frag8<FMT, VEC>(q + at[u].row * q_ld, s + at[u].row * s_ld, at[u].chunk * WARP_COLS, lane, D, v);
    }
  }
}

// The rows of an 8-bit activation to bf16 or fp32.
template <typename T, int FMT, bool VEC>
__global__ void __launch_bounds__(ACT_THREADS) act8_unpack_kernel(const uint8_t* __restrict__ q,
                                                                  const uint8_t* __restrict__ s, T* __restrict__ out,
                                                                  long long rows, int D, long long q_ld,
                                                                  long long s_ld, long long out_ld, int chunks) {
  constexpr int UNROLL = 4;
  griddep_launch_dependents();  // a weight gradient's product may set itself up
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (ACT_THREADS / 32);
  const long long first = (long long)blockIdx.x * (ACT_THREADS / 32) + (threadIdx.x >> 5);
  const long long step_rows = warps / chunks;
  const int step_chunks = static_cast<int>(warps % chunks);
  RowWalk w{first / chunks, static_cast<int>(first % chunks)};
  while (w.row < rows) {
    RowWalk at[UNROLL];
    Raw8 f[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      at[u] = w;
      if (w.row < rows) load_frag8<VEC>(f[u], q + w.row * q_ld, s + w.row * s_ld, w.chunk * WARP_COLS, lane, D);
      walk_next(w, step_rows, step_chunks, chunks);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (at[u].row >= rows) break;
      float v[8];
      frag8_floats<FMT, VEC>(f[u], at[u].chunk * WARP_COLS, lane, D, v);
      store_frag<VEC>(out + at[u].row * out_ld, at[u].chunk * WARP_COLS, lane, D, v);
    }
  }
}

// Rows in token order to their pairs' sorted rows in bf16: output row
// position[t * top_k + k] is row t, for every pair that is not dropped.  A token's
// codes are read and converted once for all its rows.  out_ld is a multiple of
// 8 and the bytes up to it may be written, whatever D.
template <int FMT>
__global__ void __launch_bounds__(ACT_THREADS) act8_scatter_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s,
                                                                   __nv_bfloat16* __restrict__ out,
                                                                   const int* __restrict__ position, int top_k, long long tokens,
                                                                   int D, long long q_ld, long long s_ld, long long out_ld,
                                                                   int segments) {
  constexpr int RUNS = 4;  // 256-column runs of an item
  griddep_launch_dependents();  // the product may set itself up
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (ACT_THREADS / 32);
  const long long first = (long long)blockIdx.x * (ACT_THREADS / 32) + (threadIdx.x >> 5);
  const long long step_rows = warps / segments;
  const int step_seg = static_cast<int>(warps % segments);
  const long long rows = tokens * top_k;
  RowWalk w{first / segments, static_cast<int>(first % segments)};
  for (; w.row < tokens; walk_next(w, step_rows, step_seg, segments)) {
    const int c0 = w.chunk * RUNS * WARP_COLS;
    Raw8 f[RUNS];
#pragma unroll
    for (int u = 0; u < RUNS; ++u)
      load_frag8<true>(f[u], q + w.row * q_ld, s + w.row * s_ld, c0 + u * WARP_COLS, lane, D);
    uint4 v[RUNS];
#pragma unroll
    for (int u = 0; u < RUNS; ++u) {
      float x[8];
      frag8_floats<FMT, true>(f[u], c0 + u * WARP_COLS, lane, D, x);
      v[u] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
    for (int k0 = 0; k0 < top_k; k0 += 32) {
      const int mine = k0 + lane < top_k ? position[w.row * top_k + k0 + lane] : -1;
      const int kn = min(32, top_k - k0);
      for (int k = 0; k < kn; ++k) {
        const int r = __shfl_sync(0xffffffffu, mine, k);
        if (r < 0 || r >= rows) continue;
#pragma unroll
        for (int u = 0; u < RUNS; ++u) {
          const int c = c0 + u * WARP_COLS + 8 * lane;
          if (c < D) *reinterpret_cast<uint4*>(out + r * out_ld + c) = v[u];
        }
      }
    }
  }
}

}  // namespace mc
