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
// threads: a warp holds 256 consecutive columns of a row, eight values a lane,
// in groups of G neighbours that one access moves:
//   G = 8  rows of whole 16-byte words: lane l holds columns 8l..8l+7, a block is
//          four neighbouring lanes
//   G = 2  even widths: value 2p, 2p + 1 of lane l are columns 64p + 2l, + 1, a
//          block is one pair of half a warp
//   G = 1  odd widths: value i of lane l is column 32i + l, a block is one value
//          of all lanes
// Neighbouring lanes always touch neighbouring addresses.
#pragma once

#include "ptx.cuh"

namespace mc {

enum ActFmt : int { ACT_NONE = 0, ACT_E4M3 = 1, ACT_INT8 = 2 };
constexpr int ACT_BLOCK = 32;
constexpr int WARP_COLS = 256;

// ---------------------------------------------------------------- fragments
template <int G>
__device__ __forceinline__ int frag_col(int c0, int lane, int i) { return c0 + (i / G) * 32 * G + lane * G + i % G; }

// Raw words of one fragment: loaded early, turned into floats when needed.
template <typename T>
struct RawFrag {
  uint32_t w[2 * sizeof(T)];
};

// The fragment's columns of a row of D; those at or past D as zeros.  Rows begin
// on a boundary of G elements (16 bytes at most).
template <int G, typename T>
__device__ __forceinline__ void load_frag(RawFrag<T>& f, const T* row, int c0, int lane, int D) {
  constexpr int BYTES = G * int(sizeof(T));
#pragma unroll
  for (int i = 0; i < 8; i += G) {
    const int c = frag_col<G>(c0, lane, i);
    const bool in = c < D;
    uint32_t* w = f.w + i * int(sizeof(T)) / 4;
    if constexpr (BYTES >= 16) {
#pragma unroll
      for (int k = 0; k < BYTES / 16; ++k) {
        const uint4 q = in ? reinterpret_cast<const uint4*>(row + c)[k] : make_uint4(0u, 0u, 0u, 0u);
        w[4 * k] = q.x;
        w[4 * k + 1] = q.y;
        w[4 * k + 2] = q.z;
        w[4 * k + 3] = q.w;
      }
    } else if constexpr (BYTES == 8) {
      const uint2 q = in ? *reinterpret_cast<const uint2*>(row + c) : make_uint2(0u, 0u);
      w[0] = q.x;
      w[1] = q.y;
    } else if constexpr (BYTES == 4) {
      w[0] = in ? *reinterpret_cast<const uint32_t*>(row + c) : 0u;
    } else {
      const uint32_t h = in ? *reinterpret_cast<const uint16_t*>(row + c) : 0u;
      w[0] = (i & 1) ? w[0] | (h << 16) : h;
    }
  }
}
// The fragment as it is to memory, none of it at or past D.
template <int G, typename T>
__device__ __forceinline__ void store_raw(T* row, int c0, int lane, int D, const RawFrag<T>& f) {
  constexpr int BYTES = G * int(sizeof(T));
#pragma unroll
  for (int i = 0; i < 8; i += G) {
    const int c = frag_col<G>(c0, lane, i);
    if (c >= D) continue;
    const uint32_t* w = f.w + i * int(sizeof(T)) / 4;
    if constexpr (BYTES >= 16) {
#pragma unroll
      for (int k = 0; k < BYTES / 16; ++k)
        reinterpret_cast<uint4*>(row + c)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    } else if constexpr (BYTES == 8) {
      *reinterpret_cast<uint2*>(row + c) = make_uint2(w[0], w[1]);
    } else if constexpr (BYTES == 4) {
      *reinterpret_cast<uint32_t*>(row + c) = w[0];
    } else {
      *reinterpret_cast<uint16_t*>(row + c) = static_cast<uint16_t>((i & 1) ? w[0] >> 16 : w[0]);
    }
  }
}

__device__ __forceinline__ void frag_floats(const RawFrag<__nv_bfloat16>& f, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(f.w[i] << 16);
    v[2 * i + 1] = __uint_as_float(f.w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void frag_floats(const RawFrag<float>& f, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(f.w[i]);
}
// Values rounded to the fragment's type.
__device__ __forceinline__ void frag_round(RawFrag<__nv_bfloat16>& f, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f.w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ void frag_round(RawFrag<float>& f, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f.w[i] = __float_as_uint(v[i]);
}
// f + g, rounded to the type.  Two bf16 numbers: their sum is exact in fp32
// unless they are so far apart (over 2^16) that it rounds to the larger one, so
// one rounding and the detour over fp32 give the same.
__device__ __forceinline__ void frag_add(RawFrag<__nv_bfloat16>& f, const RawFrag<__nv_bfloat16>& g) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 s = __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&f.w[i]), *reinterpret_cast<const __nv_bfloat162*>(&g.w[i]));
    f.w[i] = *reinterpret_cast<const uint32_t*>(&s);
  }
}
__device__ __forceinline__ void frag_add(RawFrag<float>& f, const RawFrag<float>& g) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f.w[i] = __float_as_uint(__uint_as_float(f.w[i]) + __uint_as_float(g.w[i]));
}
template <int G, typename T>
__device__ __forceinline__ void store_frag(T* row, int c0, int lane, int D, const float (&v)[8]) {
  RawFrag<T> f;
  frag_round(f, v);
  store_raw<G>(row, c0, lane, D, f);
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
template <int FMT, int G>
__device__ __forceinline__ void store_frag8(uint8_t* qrow, uint8_t* srow, int c0, int lane, int D, const float (&v)[8]) {
  if constexpr (G == 8) {
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
    // `PER` blocks share the lanes at a time (halves of the warp, or all of it);
    // the lane that is to a block what `duty` is to it works its scale out for all
    constexpr int PER = G, TURNS = 8 / G;
    const int part = PER == 2 ? lane >> 4 : 0, duty = lane & (TURNS - 1);
    const unsigned mask = PER == 2 ? 0x0000FFFFu << (16 * part) : 0xFFFFFFFFu;
    uint32_t m = 0;
#pragma unroll
    for (int t = 0; t < TURNS; ++t) {
      const float big = PER == 2 ? max_abs(v[2 * t], v[2 * t + 1]) : fabsf(v[t]);
      const uint32_t mt = __reduce_max_sync(mask, __float_as_uint(big));
      if (duty == t) m = mt;
    }
    const bool fine = m < 0x7F800000u;
    const int k = act_exponent<FMT>(m);
    const float r = fine ? exp2_int(-k) : 0.f;
#pragma unroll
    for (int t = 0; t < TURNS; ++t) {
      const float rt = __shfl_sync(0xffffffffu, r, 16 * part + t);
      const int c = frag_col<G>(c0, lane, t * G);
      if constexpr (PER == 2) {
        const uint32_t two = act_encode2<FMT>(v[2 * t] * rt, v[2 * t + 1] * rt);
        if (c < D) *reinterpret_cast<uint16_t*>(qrow + c) = rt > 0.f ? static_cast<uint16_t>(two) : 0;
      } else {
        const uint32_t one = act_encode2<FMT>(v[t] * rt, 0.f);
        if (c < D) qrow[c] = rt > 0.f ? static_cast<uint8_t>(one) : 0;
      }
    }
    const int b = PER * duty + part;  // this lane's block of the 256 columns
    if ((lane & (PER == 2 ? 15 : 31)) < TURNS && c0 + ACT_BLOCK * b < D)
      srow[c0 / ACT_BLOCK + b] = fine ? static_cast<uint8_t>(k + 127) : 255;
  }
}

// Raw codes and scale bytes of one fragment.
struct Raw8 {
  uint2 q;
  uint2 s;
};
template <int G>
__device__ __forceinline__ void load_frag8(Raw8& f, const uint8_t* qrow, const uint8_t* srow, int c0, int lane, int D) {
  if constexpr (G == 8) {
    const int c = c0 + 8 * lane;
    f.q = c < D ? *reinterpret_cast<const uint2*>(qrow + c) : make_uint2(0u, 0u);
    f.s.x = c < D ? srow[c / ACT_BLOCK] : 0u;
  } else {
    // the eight scale bytes of these columns (srow rows are 16-byte aligned and padded to 16 bytes)
    f.s = c0 < D ? *reinterpret_cast<const uint2*>(srow + c0 / ACT_BLOCK) : make_uint2(0u, 0u);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; i += G) {
      const int c = frag_col<G>(c0, lane, i);
      uint32_t b = 0u;
      if (c < D) b = G == 2 ? *reinterpret_cast<const uint16_t*>(qrow + c) : qrow[c];
      w[i >> 2] |= b << (8 * (i & 3));
    }
    f.q = make_uint2(w[0], w[1]);
  }
}
template <int FMT, int G>
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
  if constexpr (G == 8) {
    const float s = act_scale_value(f.s.x);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= s;
  } else {
    // a column past D multiplies by no scale: the bytes behind the last block are not read as one
#pragma unroll
    for (int i = 0; i < 8; i += G) {
      const int b = G == 2 ? i + (lane >> 4) : i;  // block of the 256 columns
      const uint32_t s = ((b < 4 ? f.s.x : f.s.y) >> (8 * (b & 3))) & 0xFFu;
      const float x = act_scale_value(s);
#pragma unroll
      for (int j = i; j < i + G; ++j) v[j] = frag_col<G>(c0, lane, j) < D ? v[j] * x : 0.f;
    }
  }
}

// -------------------------------------------------------------- pack, unpack
// Bound by memory: 16384 x 14336 bf16 packed to e4m3 in 114 us and unpacked in 112 us
// (712 MB: 6.24 and 6.37 TB/s of the 6.55 a copy reaches here).
// Work items are (row, chunk of RUNS 256-column runs) pairs, one per warp and step; a
// warp takes PACK_FRAGS / RUNS items at once, so that PACK_FRAGS runs' loads are in
// flight together.  An item's runs share its addresses: with one run an item the
// pack spent its issue slots on them (2^27 bf16 to e4m3: 82 us with one run, 74
// with two, 70 with four; 16384 x 14336: 133 with one).  Runs past the row's end are idle (1280 columns: 82 us
// with items of one or two runs, 88 with four), so RUNS is the largest of 4, 2, 1 that
// leaves at most a quarter idle.
constexpr int PACK_FRAGS = 4;
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

template <typename T, int FMT, int G, int RUNS>
__global__ void __launch_bounds__(ACT_THREADS) act8_pack_kernel(const T* __restrict__ x, uint8_t* __restrict__ q,
                                                                uint8_t* __restrict__ s, long long rows, int D,
                                                                long long q_ld, long long s_ld, int chunks) {
  griddep_launch_dependents();
  constexpr int UNROLL = PACK_FRAGS / RUNS;
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (ACT_THREADS / 32);
  const long long first = (long long)blockIdx.x * (ACT_THREADS / 32) + (threadIdx.x >> 5);
  const long long step_rows = warps / chunks;
  const int step_chunks = static_cast<int>(warps % chunks);
  RowWalk w{first / chunks, static_cast<int>(first % chunks)};
  while (w.row < rows) {
    RowWalk at[UNROLL];
    RawFrag<T> f[UNROLL][RUNS];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      at[u] = w;
      if (w.row < rows) {
        const T* xr = x + w.row * D;
        const int c0 = w.chunk * (RUNS * WARP_COLS);
#pragma unroll
        for (int j = 0; j < RUNS; ++j) load_frag<G>(f[u][j], xr, c0 + j * WARP_COLS, lane, D);
      }
      walk_next(w, step_rows, step_chunks, chunks);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (at[u].row >= rows) break;
      uint8_t* qr = q + at[u].row * q_ld;
      uint8_t* sr = s + at[u].row * s_ld;
      const int c0 = at[u].chunk * (RUNS * WARP_COLS);
#pragma unroll
      for (int j = 0; j < RUNS; ++j) {
        float v[8];
        frag_floats(f[u][j], v);
        store_frag8<FMT, G>(qr, sr, c0 + j * WARP_COLS, lane, D, v);
      }
    }
  }
}

// The rows of an 8-bit activation to bf16 or fp32.  Kernels that start while
// the stream's previous one runs read memory that it may still be writing, so
// none of their pointers is __restrict__: read-only loads are defined only for
// data that does not change while the kernel lives.
template <typename T, int FMT, int G, int RUNS>
__global__ void __launch_bounds__(ACT_THREADS) act8_unpack_kernel(const uint8_t* q, const uint8_t* s, T* out, long long rows,
                                                                  int D, long long q_ld, long long s_ld, long long out_ld,
                                                                  int chunks) {
  constexpr int UNROLL = PACK_FRAGS / RUNS;
  griddep_launch_dependents();  // a weight gradient's product may set itself up
  griddep_wait();               // what wrote the codes may still run
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (ACT_THREADS / 32);
  const long long first = (long long)blockIdx.x * (ACT_THREADS / 32) + (threadIdx.x >> 5);
  const long long step_rows = warps / chunks;
  const int step_chunks = static_cast<int>(warps % chunks);
  RowWalk w{first / chunks, static_cast<int>(first % chunks)};
  while (w.row < rows) {
    RowWalk at[UNROLL];
    Raw8 f[UNROLL][RUNS];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      at[u] = w;
      if (w.row < rows) {
        const uint8_t* qr = q + w.row * q_ld;
        const uint8_t* sr = s + w.row * s_ld;
        const int c0 = w.chunk * (RUNS * WARP_COLS);
#pragma unroll
        for (int j = 0; j < RUNS; ++j) load_frag8<G>(f[u][j], qr, sr, c0 + j * WARP_COLS, lane, D);
      }
      walk_next(w, step_rows, step_chunks, chunks);
    }
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      if (at[u].row >= rows) break;
      T* o = out + at[u].row * out_ld;
      const int c0 = at[u].chunk * (RUNS * WARP_COLS);
#pragma unroll
      for (int j = 0; j < RUNS; ++j) {
        float v[8];
        frag8_floats<FMT, G>(f[u][j], c0 + j * WARP_COLS, lane, D, v);
        store_frag<G>(o, c0 + j * WARP_COLS, lane, D, v);
      }
    }
  }
}

// Rows in token order to their pairs' sorted rows in bf16: output row
// position[t * top_k + k] is row t, for every pair that is not dropped.  A token's
// codes are read and converted once for all its rows.  out_ld is a multiple of
// 8 and the bytes up to it may be written, whatever D.  `reached`, zeros before,
// gets a 1 for each row that a pair has.
template <int FMT>
__global__ void __launch_bounds__(ACT_THREADS) act8_scatter_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s,
                                                                   __nv_bfloat16* __restrict__ out, uint8_t* __restrict__ reached,
                                                                   const int* __restrict__ position, int top_k, long long tokens,
                                                                   int D, long long q_ld, long long s_ld, long long out_ld,
                                                                   int segments) {
  constexpr int RUNS = 4;  // 256-column runs of an item
  griddep_launch_dependents();  // the maps' kernel may set itself up
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
      load_frag8<8>(f[u], q + w.row * q_ld, s + w.row * s_ld, c0 + u * WARP_COLS, lane, D);
    uint4 v[RUNS];
#pragma unroll
    for (int u = 0; u < RUNS; ++u) {
      float x[8];
      frag8_floats<FMT, 8>(f[u], c0 + u * WARP_COLS, lane, D, x);
      v[u] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
    for (int k0 = 0; k0 < top_k; k0 += 32) {
      const int mine = k0 + lane < top_k ? position[w.row * top_k + k0 + lane] : -1;
      const int kn = min(32, top_k - k0);
      for (int k = 0; k < kn; ++k) {
        const int r = __shfl_sync(0xffffffffu, mine, k);
        if (r < 0 || r >= rows) continue;
        if (w.chunk == 0 && lane == 0) reached[r] = 1;
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
