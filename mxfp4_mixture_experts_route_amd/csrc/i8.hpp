// Device-side helpers of the 8-bit integer projections: the row format, the packed weight layout,
// the row quantization and the typed loads and stores.
#pragma once

#include <hip/hip_fp16.h>

#include <type_traits>

#include "common.hpp"

namespace moe {

typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t i32x16_t __attribute__((ext_vector_type(16)));

constexpr int kI8Chunk = 64;        // K values of a weight tile (one 16x16x64 MFMA step)
constexpr int kI8TileRows = 16;     // weight rows of a tile
constexpr int kI8TileBytes = kI8Chunk * kI8TileRows;

// Row pitch of quantized rows: K padded (with zeros) to whole cache lines of 128 bytes. A row is
// read in pieces: of 64 bytes they would take twice as long (every load moves whole lines: reads
// of 64-byte pieces reach 17 TB/s from L2 and 3.6 from memory, of 128 bytes 36 and 7).
__host__ __device__ __forceinline__ int i8_pitch(int K) { return (K + 127) & ~127; }

// Chunks of 64 K values of the packed weights.
__host__ __device__ __forceinline__ int i8_chunks(int K) { return (K + kI8Chunk - 1) / kI8Chunk; }

// Weight tiles of an expert: N rows in tiles of 16, or, packed for SwiGLU, each half (gate rows,
// up rows) in tiles of its own, so that a gate tile and its up tile always match row for row. Up to
// N = 2^31 - 1 (N >= 1, >= 2 for SwiGLU) nothing here leaves 32 bits.
__host__ __device__ __forceinline__ int i8_half_tiles(int N, int glu) {
  return ((glu ? N / 2 : N) - 1) / kI8TileRows + 1;
}
__host__ __device__ __forceinline__ int i8_tiles(int N, int glu) {
  return i8_half_tiles(N, glu) * (glu ? 2 : 1);
}

// Rows that a product quantizes before it starts: values of type dt, ld from one row to the next.
struct I8Plain {
  const void* x;
  int dt;
  int64_t ld;
};

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

// float -> bf16 bits by the hardware conversion (round to nearest even, subnormals kept; checked
// against the integer rounding of f32_to_bf16_bits over every exponent), a pair at a time or one.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const bf16x2_t p = {(__bf16)lo, (__bf16)hi};
  uint32_t u;
  __builtin_memcpy(&u, &p, sizeof(u));
  return u;
}
__device__ __forceinline__ uint16_t bf16_one(float v) {
  const __bf16 b = (__bf16)v;
  uint16_t u;
  __builtin_memcpy(&u, &b, sizeof(u));
  return u;
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
    ((uint16_t*)p)[i] = bf16_one(v);
}

// Row quantization: with m the row's largest magnitude, the scale is m / 127 (rounded to f32) and
// the codes are 127 x / m, the exact quotient, rounded half to even. A zero row takes scale 0 and
// codes 0; a row that holds a NaN or an infinity has no scale: NaN, and codes 0, so that every
// value the row stands for is NaN.
struct I8Quant {
  float s;      // the row's scale
  float m;      // the largest magnitude (lifted)
  float inv;    // 127 / m, 0 for a row of zeros and for a row without a scale
  bool lift;    // a tiny row is lifted by 2^100, exactly: 127 / m would overflow

  // mbits: largest |x| of the row as an f32 pattern (NaN and infinity are the largest of all),
  // the same on every lane of the wavefront
  __device__ __forceinline__ explicit I8Quant(uint32_t mbits) {
    const bool none = mbits >= 0x7F800000u;
    const float top = none ? 0.0f : __uint_as_float(mbits);
    s = none ? __uint_as_float(0x7FC00000u) : top / 127.0f;
    lift = (uint32_t)__builtin_amdgcn_readfirstlane((int)mbits) < 0x0D800000u;   // 2^-100
    m = lift ? top * 0x1p100f : top;
    inv = m > 0.0f ? 127.0f / m : 0.0f;
  }

  // The code of x (lifted), in the low byte of the result (the rest is not cleared); of no meaning
  // in a row without a scale.
  //
  // 16-bit inputs: p = x * inv carries a relative error of at most 2^-23, that is less than 2
  // units in its last place. Where 127 x / m is a tie (j + 1/2, at most 8 significant bits) p has
  // to become it exactly; anywhere else the quotient of two 11-bit significands is at least
  // 2^-20 (relative) away from a tie. So p rounded to a grid of 8 units (a spacing of at most
  // 2^-20, ties of the code on the grid, the error under half of the spacing) is the tie where
  // there is one and stays on its own side elsewhere: the code is that of the exact quotient for
  // four plain operations, where a division takes about ten.
  // f32 inputs come nearer to a tie than any f32 quotient shows: there the code is checked
  // against the exact remainder in 64 bits (31 significant bits) when it is near one.
  template <int DT>
  __device__ __forceinline__ uint32_t code(float x) const {
    constexpr float kRound = 12582912.0f;   // 1.5 * 2^23: adding it rounds to a whole number
    const float p = x * inv;
    if constexpr (DT != MOE_F32) {
      const uint32_t b = (__float_as_uint(p) + 4u) & ~7u;
      return __float_as_uint(__uint_as_float(b) + kRound);
    } else {
      float r = rintf(p);
      if (fabsf(p - r) > 0.4999f) {
        const double rem = 127.0 * (double)x - (double)r * (double)m;   // exact
        const double two = 2.0 * fabs(rem);
        const bool odd = ((int)r & 1) != 0;
        if (two > (double)m || (two == (double)m && odd)) r += rem > 0.0 ? 1.0f : -1.0f;
      }
      return (uint32_t)(int)r;
    }
  }
};

// 16 bytes at any alignment of the element type, by one load (the memory system takes loads of any
// alignment: 4346 rows of 5951 f16 values are quantized in 25 us, by elements in 38).
struct I8Bytes16 {
  uint8_t b[16];
};
__device__ __forceinline__ uint4 load16_any(const void* p) {
  uint4 a;
  __builtin_memcpy(&a, p, sizeof(a));
  return a;
}

// 8 values of a row at p (element index i0), zeros past n.
template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t i0, int n, float (&v)[8]) {
  if (n >= 8) {
    if constexpr (DT == MOE_F32) {
      const uint4 a = load16_any((const float*)p + i0), b = load16_any((const float*)p + i0 + 4);
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    } else {
      const uint4 a = load16_any((const uint16_t*)p + i0);
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

// The codes of 8 values, zeros in a row without a scale (whose values may be NaN or infinite).
template <int DT>
__device__ __forceinline__ uint2 codes8(const I8Quant& z, float (&v)[8]) {
  uint32_t c[8];
  if (z.lift)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= 0x1p100f;
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = z.code<DT>(v[i]);
  // v_perm: the low bytes of two registers, then of two pairs
  const uint32_t a = __builtin_amdgcn_perm(c[1], c[0], 0x0c0c0400u);
  const uint32_t b = __builtin_amdgcn_perm(c[3], c[2], 0x0c0c0400u);
  const uint32_t d = __builtin_amdgcn_perm(c[5], c[4], 0x0c0c0400u);
  const uint32_t e = __builtin_amdgcn_perm(c[7], c[6], 0x0c0c0400u);
  uint2 o;
  o.x = z.inv > 0.0f ? __builtin_amdgcn_perm(b, a, 0x05040100u) : 0u;
  o.y = z.inv > 0.0f ? __builtin_amdgcn_perm(e, d, 0x05040100u) : 0u;
  return o;
}

// Values of sums of products: sum * (sr * sc) + bias, with the scales of a row and of a channel, as
// one f32 product and one fused multiply-add. Where the product of the scales is no normal f32 (zero,
// subnormal: few or no bits left; infinite: a sum of zero would give NaN) the value may be an
// ordinary number all the same: it is then computed in 64 bits, which hold the product of two f32
// exactly, and rounded to f32. One branch covers the N values: such scales are rare.
template <int N>
__device__ __forceinline__ void i8_scaled(const int (&sum)[N], const float (&sr)[N], const float (&sc)[N],
                                          const float (&bias)[N], float (&v)[N]) {
  constexpr int kNormalOrNaN = 0x10B;   // v_cmp_class: NaN (1, 2), normal numbers (8, 0x100)
  bool odd[N], any = false;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float p = sr[i] * sc[i];
    odd[i] = !__builtin_amdgcn_classf(p, kNormalOrNaN);
    any |= odd[i];
    v[i] = fmaf((float)sum[i], p, bias[i]);
  }
  if (__builtin_expect(any, 0)) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (odd[i]) v[i] = (float)fma((double)sum[i], (double)sr[i] * (double)sc[i], (double)bias[i]);
  }
}
__device__ __forceinline__ float i8_scaled(int sum, float sr, float sc, float bias) {
  float v[1];
  i8_scaled<1>({sum}, {sr}, {sc}, {bias}, v);
  return v[0];
}

// The clamped SwiGLU of a pair, NaN where either is NaN (the clamps alone would take a NaN to the
// limit, and a row without a scale has to stay without a value).
__device__ __forceinline__ float i8_swiglu(float gate, float up, float alpha, float limit) {
  const float h = swiglu_oai(gate, up, alpha, limit);
  return __builtin_isunordered(gate, up) ? __uint_as_float(0x7FC00000u) : h;
}

// The largest value of the wavefront's lanes, by moves between lanes inside the vector ALU (rows of
// 16, then their last lanes into the rows behind): six dependent steps of LDS shuffles cost several
// times as much (a kernel that quantizes one row and multiplies it: 6.7 -> 6.5 us).
__device__ __forceinline__ uint32_t wave_umax(uint32_t m) {
  auto step = [&](auto ctrl, auto rows) {
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, decltype(ctrl)::value,
                                                     decltype(rows)::value, 0xf, false));
  };
  step(std::integral_constant<int, 0x111>(), std::integral_constant<int, 0xf>());   // row_shr:1
  step(std::integral_constant<int, 0x112>(), std::integral_constant<int, 0xf>());   // row_shr:2
  step(std::integral_constant<int, 0x114>(), std::integral_constant<int, 0xf>());   // row_shr:4
  step(std::integral_constant<int, 0x118>(), std::integral_constant<int, 0xf>());   // row_shr:8
  step(std::integral_constant<int, 0x142>(), std::integral_constant<int, 0xa>());   // row_bcast:15
  step(std::integral_constant<int, 0x143>(), std::integral_constant<int, 0xc>());   // row_bcast:31
  return (uint32_t)__builtin_amdgcn_readlane((int)m, kWave - 1);
}

// LDS pitch of a quantized row: an odd multiple of 128 bytes, so that with the 16-byte pieces of
// each 128 permuted by i8_swizzle the 16 rows of a B operand are read without bank conflicts.
__host__ __device__ __forceinline__ int i8_lds_pitch(int KP) {
  return (((KP + 127) >> 7) | 1) << 7;
}
__device__ __forceinline__ int i8_swizzle(int m, int off) { return off ^ (((m >> 1) & 7) << 4); }

// A row spread over a wavefront: NV vectors of 8 values per lane, vector i of lane l holding values
// 8 (64 i + l) .. + 7, zeros past the row. TAIL: rows of any length, else of K % 8 == 0 values.
template <int NV, int DT = MOE_BF16>
struct I8Row {
  static constexpr int kWords = DT == MOE_F32 ? 8 : 4;   // 32-bit words of a vector
  uint32_t v[NV][kWords];
  template <bool TAIL>
  __device__ __forceinline__ void load(const void* __restrict__ row, int K) {
    const int lane = (int)(threadIdx.x & 63);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int u = i * kWave + lane;
#pragma unroll
      for (int j = 0; j < kWords; ++j) v[i][j] = 0u;
      if constexpr (TAIL) {
        if (u * 8 < K && u * 8 + 8 > K) {   // the vector at the end of the row
#pragma unroll
          for (int j = 0; j < 7; ++j)
            if (u * 8 + j < K) {
              if constexpr (DT == MOE_F32)
                v[i][j] = ((const uint32_t*)row)[u * 8 + j];
              else
                v[i][j >> 1] |= (uint32_t)((const uint16_t*)row)[u * 8 + j] << (16 * (j & 1));
            }
          continue;
        }
      }
      if (u * 8 < K) {
#pragma unroll
        for (int j = 0; j < kWords / 4; ++j) {
          const uint4 t = load16_any((const I8Bytes16*)row + u * (kWords / 4) + j);
          v[i][4 * j] = t.x;
          v[i][4 * j + 1] = t.y;
          v[i][4 * j + 2] = t.z;
          v[i][4 * j + 3] = t.w;
        }
      }
    }
  }
  // Largest magnitude as an f32 pattern, the same in every lane. Patterns without their sign
  // order as the values do, NaN above infinity: 16-bit ones go two a step as unsigned halves.
  __device__ __forceinline__ uint32_t largest() const {
    if constexpr (DT == MOE_F32) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < kWords; ++j) m = max(m, v[i][j] & 0x7FFFFFFFu);
      return wave_umax(m);
    } else {
      typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));
      u16x2_t m = {0, 0};
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          const uint32_t w = v[i][j] & 0x7FFF7FFFu;
          u16x2_t t;
          __builtin_memcpy(&t, &w, sizeof(t));
          m = __builtin_elementwise_max(m, t);
        }
      const uint32_t top = wave_umax(max((uint32_t)m[0], (uint32_t)m[1]));
      if constexpr (DT == MOE_BF16) return top << 16;
      return __float_as_uint(__half2float(__ushort_as_half((unsigned short)top)));
    }
  }
  __device__ __forceinline__ uint2 codes(const I8Quant& z, int i) const {
    float f[8];
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      if constexpr (DT == MOE_F32) {
        f[j] = __uint_as_float(v[i][j]);
      } else if constexpr (DT == MOE_F16) {
        f[2 * j] = __half2float(__ushort_as_half((unsigned short)(v[i][j] & 0xFFFFu)));
        f[2 * j + 1] = __half2float(__ushort_as_half((unsigned short)(v[i][j] >> 16)));
      } else {
        f[2 * j] = __uint_as_float(v[i][j] << 16);
        f[2 * j + 1] = __uint_as_float(v[i][j] & 0xFFFF0000u);
      }
    }
    return codes8<DT>(z, f);
  }
  // Codes of the vectors i with i % parts == part (parts a power of two) into row m of an LDS
  // image (pitch LP)
  __device__ __forceinline__ void store_codes(const I8Quant& z, uint8_t* lds, int m, int LP, int KP,
                                              int part, int parts) const {
    const int lane = (int)(threadIdx.x & 63);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if ((i & (parts - 1)) != part) continue;
      const int off = (i * kWave + lane) * 8;
      if (off < KP)
        *reinterpret_cast<uint2*>(lds + m * LP + i8_swizzle(m, off & ~15) + (off & 8)) = codes(z, i);
      __builtin_amdgcn_sched_barrier(0);   // one vector's values at a time in registers
    }
  }
  // Codes of the vectors [u0, u1) of the row, one after another
  __device__ __forceinline__ void store_part(const I8Quant& z, uint8_t* lds, int u0, int u1) const {
    const int lane = (int)(threadIdx.x & 63);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i * kWave >= u1 || (i + 1) * kWave <= u0) continue;   // the same for the whole wavefront
      const int u = i * kWave + lane;
      if (u >= u0 && u < u1) *reinterpret_cast<uint2*>(lds + (u - u0) * 8) = codes(z, i);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
};

// The same for any row from element r0 of x on, read twice: its scale, and its codes into row m of
// an LDS image.
template <int DT>
__device__ __forceinline__ float i8_row_to_lds(const void* __restrict__ x, int64_t r0, int K,
                                               uint8_t* lds, int m, int LP, int KP) {
  const int lane = (int)(threadIdx.x & 63);
  uint32_t top = 0;
  for (int u = lane; u * 8 < K; u += kWave) {
    float t[8];
    load8<DT>(x, r0 + u * 8, K - u * 8, t);
    top = max_abs8(t, top);
  }
  const I8Quant z(wave_umax(top));
  for (int u = lane; u * 8 < KP; u += kWave) {
    float t[8];
    load8<DT>(x, r0 + u * 8, K - u * 8, t);
    *reinterpret_cast<uint2*>(lds + m * LP + i8_swizzle(m, (u * 8) & ~15) + ((u * 8) & 8)) =
        codes8<DT>(z, t);
  }
  return z.s;
}

// A barrier for what was written to LDS: loads from memory stay in flight (__syncthreads() would
// wait for all of them).
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// A run of n <= NR chunks of one weight tile: where its first chunk starts in an expert's stack.
// A run of no chunks reads nothing (its loads are out of range and give zeros).
struct I8Run {
  __amdgpu_buffer_rsrc_t r;
  uint32_t off, step;
  int n;
};

// NR chunks of a run in registers, refilled one by one from the run after it as they are used, so
// that a wavefront has NR KB in flight from its first run to its last. Buffer loads: the
// resource is one expert's stack and the chunk a scalar offset, so that a load takes no address
// registers. Chunks past the end of a run are zeros, and so are their products.
template <int NR>
struct I8Ring {
  u32x4_t v[NR];
  __device__ __forceinline__ void load(int i, const I8Run& run) {
    const uint32_t lane16 = (threadIdx.x & 63) * 16;
    v[i] = buf_load16_nt(run.r, i < run.n ? lane16 : kOOB, i < run.n ? run.off + (uint32_t)i * run.step : 0u);
  }
  __device__ __forceinline__ void fill(const I8Run& run) {
#pragma unroll
    for (int i = 0; i < NR; ++i) load(i, run);
  }
  // acc += the products of the run held with the B operands from LDS row bp (its m-th row), the
  // run's first chunk being c0; the ring is refilled from `next`
  __device__ __forceinline__ void take(const uint8_t* bp, int m, int c0, int clast, const I8Run& next,
                                       i32x4_t& acc, i32x4_t& acc1) {
    const int g16 = ((int)(threadIdx.x & 63) >> 4) * 16;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const i32x4_t b = *reinterpret_cast<const i32x4_t*>(
          bp + i8_swizzle(m, min(c0 + i, clast) * kI8Chunk + g16));
      i32x4_t a;
      __builtin_memcpy(&a, &v[i], sizeof(a));
      if (i & 1)
        acc1 = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, acc1, 0, 0, 0);
      else
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, acc, 0, 0, 0);
      load(i, next);
      if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);   // few B operands at a time
    }
  }
};

}  // namespace moe
