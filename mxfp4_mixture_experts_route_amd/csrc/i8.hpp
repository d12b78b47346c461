// Device-side helpers of the 8-bit integer projections: the row format, the packed weight layout,
// the row quantization and the typed loads and stores.
#pragma once

#include <hip/hip_fp16.h>

#include "common.hpp"

namespace moe {

typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t i32x16_t __attribute__((ext_vector_type(16)));

constexpr int kI8Chunk = 64;        // K values of a weight tile (one 16x16x64 MFMA step)
constexpr int kI8TileRows = 16;     // weight rows of a tile
constexpr int kI8TileBytes = kI8Chunk * kI8TileRows;

// Row pitch of quantized rows: K padded (with zeros) to whole chunks.
__host__ __device__ __forceinline__ int i8_pitch(int K) {
  return (K + kI8Chunk - 1) & ~(kI8Chunk - 1);
}

// Weight tiles of an expert: N rows in tiles of 16, or, packed for SwiGLU, each half (gate rows,
// up rows) in tiles of its own, so that a gate tile and its up tile always match row for row.
__host__ __device__ __forceinline__ int i8_half_tiles(int N, int glu) {
  return ((glu ? N / 2 : N) + kI8TileRows - 1) / kI8TileRows;
}
__host__ __device__ __forceinline__ int i8_tiles(int N, int glu) {
  return i8_half_tiles(N, glu) * (glu ? 2 : 1);
}

// Channel of row r of tile t, or -1 in the padding of a tile.
__device__ __forceinline__ int i8_channel(int t, int r, int N, int glu) {
  if (!glu) {
    const int n = t * kI8TileRows + r;
    return n < N ? n : -1;
  }
  const int F = N >> 1, FT = i8_half_tiles(N, 1);
  const int half = t >= FT;
  const int n = (t - half * FT) * kI8TileRows + r;
  return n < F ? half * F + n : -1;
}

// Typed element access (MOE_BF16 / MOE_F16 / MOE_F32).
template <int DT>
__device__ __forceinline__ float load_elem(const void* p, int64_t i) {
  if constexpr (DT == MOE_F32) return ((const float*)p)[i];
  if constexpr (DT == MOE_F16) return __half2float(((const __half*)p)[i]);
  return bf16_bits_to_f32(((const uint16_t*)p)[i]);
}
__device__ __forceinline__ void store_elem(void* p, int64_t i, float v, int dt) {
  if (dt == MOE_F32)
    ((float*)p)[i] = v;
  else if (dt == MOE_F16)
    ((__half*)p)[i] = __float2half_rn(v);
  else
    ((uint16_t*)p)[i] = (uint16_t)f32_to_bf16_bits(v);
}

// Row quantization: with m the row's largest magnitude, the scale is m / 127 (rounded to f32) and
// the codes are 127 x / m, the exact quotient, rounded half to even. A zero row takes scale 0 and
// codes 0; a row that holds a NaN or an infinity has no scale: NaN, and codes 0, so that every
// value the row stands for is NaN.
struct I8Quant {
  float s;      // the row's scale
  float pre;    // exact power of two that lifts a tiny row (127 / m would overflow)
  float m;      // m * pre
  float inv;    // 127 / (m * pre), 0 for a row of zeros and for a row without a scale

  // mbits: largest |x| of the row as an f32 pattern (NaN and infinity are the largest of all)
  __device__ __forceinline__ explicit I8Quant(uint32_t mbits) {
    const bool none = mbits >= 0x7F800000u;
    const float top = none ? 0.0f : __uint_as_float(mbits);
    s = none ? __uint_as_float(0x7FC00000u) : top / 127.0f;
    pre = top < 0x1p-100f ? 0x1p100f : 1.0f;
    m = top * pre;
    inv = m > 0.0f ? 127.0f / m : 0.0f;
  }

  // The code of x, in the low byte of the result (the rest is not cleared).
  //
  // 16-bit inputs: p = x * inv carries a relative error of at most 2^-23, that is less than 2
  // units in its last place. Where 127 x / m is a tie (j + 1/2, at most 8 significant bits) p has
  // to become it exactly; anywhere else the quotient of two 11-bit significands is at least
  // 2^-20 (relative) away from a tie. So p rounded to a grid of 8 units (a spacing of at most
  // 2^-20, ties of the code on the grid, the error under half of the spacing) is the tie where
  // there is one and stays on its own side elsewhere: the code is that of the exact quotient for
  // six plain operations, where a division takes about ten.
  // f32 inputs come nearer to a tie than any f32 quotient shows: there the code is checked
  // against the exact remainder in 64 bits (31 significant bits) when it is near one.
  template <int DT>
  __device__ __forceinline__ uint32_t code(float x) const {
    constexpr float kRound = 12582912.0f;   // 1.5 * 2^23: adding it rounds to a whole number
    if constexpr (DT != MOE_F32) {
      const float p = (x * pre) * inv;
      const uint32_t b = (__float_as_uint(p) + 4u) & ~7u;
      return __float_as_uint(__uint_as_float(b) + kRound);
    } else {
      const float xs = inv > 0.0f ? x * pre : 0.0f;   // a row without a scale: x may be a NaN
      const float p = xs * inv;
      float r = rintf(p);
      if (fabsf(p - r) > 0.4999f) {
        const double rem = 127.0 * (double)xs - (double)r * (double)m;   // exact
        const double two = 2.0 * fabs(rem);
        const bool odd = ((int)r & 1) != 0;
        if (two > (double)m || (two == (double)m && odd)) r += rem > 0.0 ? 1.0f : -1.0f;
      }
      return (uint32_t)(int)r;
    }
  }
};

// A row without a scale may hold NaN or infinity: p would be NaN and the code's bits arbitrary.
// inv = 0 makes p 0 for every finite x; NaN and infinity are taken to 0 here.
template <int DT>
__device__ __forceinline__ float i8_finite(float x) {
  return (__float_as_uint(x) & 0x7F800000u) == 0x7F800000u ? 0.0f : x;
}

// 8 values of a row at p (element index i0), zeros past n. VEC: the row is 16-byte aligned.
template <int DT, bool VEC>
__device__ __forceinline__ void load8(const void* p, int64_t i0, int n, float (&v)[8]) {
  if (VEC && n >= 8) {
    if constexpr (DT == MOE_F32) {
      const float4 a = *reinterpret_cast<const float4*>((const float*)p + i0);
      const float4 b = *reinterpret_cast<const float4*>((const float*)p + i0 + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>((const uint16_t*)p + i0);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (DT == MOE_BF16) {
          v[2 * i] = __uint_as_float(w[i] << 16);
          v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
          v[2 * i] = __half2float(__ushort_as_half((unsigned short)(w[i] & 0xFFFFu)));
          v[2 * i + 1] = __half2float(__ushort_as_half((unsigned short)(w[i] >> 16)));
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? load_elem<DT>(p, i0 + i) : 0.0f;
  }
}

__device__ __forceinline__ uint32_t max_abs8(const float (&v)[8], uint32_t m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

template <int DT>
__device__ __forceinline__ uint2 codes8(const I8Quant& z, const float (&v)[8]) {
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = z.code<DT>(i8_finite<DT>(v[i]));
  uint2 o;
  // v_perm: byte 0 of each pair, then of the pairs
  const uint32_t a = __builtin_amdgcn_perm(c[1], c[0], 0x0c0c0400u);
  const uint32_t b = __builtin_amdgcn_perm(c[3], c[2], 0x0c0c0400u);
  o.x = __builtin_amdgcn_perm(b, a, 0x05040100u);
  const uint32_t d = __builtin_amdgcn_perm(c[5], c[4], 0x0c0c0400u);
  const uint32_t e = __builtin_amdgcn_perm(c[7], c[6], 0x0c0c0400u);
  o.y = __builtin_amdgcn_perm(e, d, 0x05040100u);
  return o;
}

// The clamped SwiGLU of a pair, NaN where either is NaN (the clamps alone would take a NaN to the
// limit, and a row without a scale has to stay without a value).
__device__ __forceinline__ float i8_swiglu(float gate, float up, float alpha, float limit) {
  const float h = swiglu_oai(gate, up, alpha, limit);
  return __builtin_isunordered(gate, up) ? __uint_as_float(0x7FC00000u) : h;
}

__device__ __forceinline__ uint32_t wave_umax(uint32_t m) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
  return m;
}

}  // namespace moe
