// i8_quantize: rows of bf16, f16 or f32 values -> rows of 8-bit whole numbers with one scale each,
// the activations of the 8-bit integer projections. i8_pack_experts: the one-time weight repack.
//
// The row's largest magnitude m gives the scale m / 127; the codes are 127 x / m rounded half to
// even, exactly (i8.hpp). The format and the operators on it are not on the pages, which keep
// activations in 16 bits on the GPU and quantize them to 8-bit blocks on the CPU only.
//
// Bound by memory: K * size bytes in, K out, a row read once (it stays in registers between the
// maximum and the rounding). 4096 rows of 8192 bf16 values take 20 us (5.0 TB/s); up to some
// hundred rows it is the launch, 4 us.
#include "i8.hpp"
#include "launch.hpp"

namespace moe {

constexpr int kI8QuantThreads = 256;
constexpr int64_t kI8MaxGrid = 1 << 23;   // workgroups of a launch: 2^32 threads are too many

// TPR threads per row (a wavefront or the whole workgroup), NV vectors of 8 values per thread in
// registers; what a longer row has past TPR * NV * 8 values is read a second time.
template <int DT, int TPR, int NV>
__global__ void __launch_bounds__(kI8QuantThreads)
i8_quantize_kernel(const void* __restrict__ x, int64_t ld, const int32_t* __restrict__ live,
                   int64_t rows, int K, int8_t* __restrict__ q, float* __restrict__ s) {
  const int KP = i8_pitch(K), V = KP >> 3;
  const int lane = (int)threadIdx.x % TPR;
  const int64_t r = (int64_t)blockIdx.x * (kI8QuantThreads / TPR) + threadIdx.x / TPR;
  if (r >= rows || (live && live[r] < 0)) return;   // TPR lanes leave together
  const int64_t base = r * ld;
  float v[NV][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int u = lane + i * TPR;
    if (u < V) {
      load8<DT>(x, base + (int64_t)u * 8, K - u * 8, v[i]);
      m = max_abs8(v[i], m);
    }
  }
  for (int u = lane + NV * TPR; u < V; u += TPR) {
    float t[8];
    load8<DT>(x, base + (int64_t)u * 8, K - u * 8, t);
    m = max_abs8(t, m);
  }
  m = wave_umax(m);
  if constexpr (TPR > kWave) {
    __shared__ uint32_t part[TPR / kWave];
    if ((lane & 63) == 0) part[lane >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TPR / kWave; ++w) m = max(m, part[w]);
  }
  const I8Quant z(m);
  int8_t* dst = q + r * KP;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int u = lane + i * TPR;
    if (u < V) *reinterpret_cast<uint2*>(dst + u * 8) = codes8<DT>(z, v[i]);
  }
  for (int u = lane + NV * TPR; u < V; u += TPR) {
    float t[8];
    load8<DT>(x, base + (int64_t)u * 8, K - u * 8, t);
    *reinterpret_cast<uint2*>(dst + u * 8) = codes8<DT>(z, t);
  }
  if (lane == 0) s[r] = z.s;
}

// A wavefront per tile of the packed stack, a lane per 16 bytes: tile t of chunk c holds rows 16 t ..
// 16 t + 15 and K values 64 c .. 64 c + 63 in the lane order of the MFMA operand (lane l: row l % 16,
// values 16 (l / 16) ..), zeros past N and K. A workgroup takes four chunks of a tile, so that it
// reads whole cache lines of the rows (32 experts of 5760 x 2880: 176 us, 6.0 TB/s).
__global__ void __launch_bounds__(256)
i8_pack_kernel(const int8_t* __restrict__ src, int64_t first, int N, int K, int glu,
               int8_t* __restrict__ dst) {
  const int NT = i8_tiles(N, glu), C = i8_chunks(K), quads = (C + 3) / 4;
  const int64_t item = first + blockIdx.x, eq = item / NT, e = eq / quads;
  const int t = (int)(item - eq * NT), c = (int)(eq - e * quads) * 4 + (int)(threadIdx.x >> 6);
  if (c >= C) return;
  const int l = (int)(threadIdx.x & 63);
  const int n = i8_channel(t, l & 15, N, glu);
  const int k0 = c * kI8Chunk + (l >> 4) * 16;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (n >= 0) {
    const int8_t* row = src + (e * N + n) * (int64_t)K;
    if (k0 + 16 <= K) {
      v = load16_any(row + k0);
    } else {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (k0 + i < K) w[i >> 2] |= (uint32_t)(uint8_t)row[k0 + i] << (8 * (i & 3));
      v = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  *reinterpret_cast<uint4*>(dst + (((e * C + c) * NT + t) * kWave + l) * 16) = v;
}

template <int DT>
int launch_quantize(const void* x, int64_t ld, const int32_t* live, int64_t rows, int K,
                    int8_t* q, float* s, hipStream_t st) {
  constexpr int kSize = DT == MOE_F32 ? 4 : 2;
  // many rows: a wavefront each (4 a workgroup); few rows, or rows that a wavefront does not
  // hold in registers: a workgroup each (rows of 2880: 1024 of them 4.3 us, by wavefronts 5.5; 8672
  // of them 23 and 19)
  const bool wave = K <= kWave * 8 * 8 && rows > 2048;
  const int64_t per = wave ? 4 : 1;
  for (int64_t r0 = 0; r0 < rows; r0 += kI8MaxGrid * per) {
    const int64_t n = rows - r0 < kI8MaxGrid * per ? rows - r0 : kI8MaxGrid * per;
    const dim3 grid((unsigned)((n + per - 1) / per));
    auto go = [&](auto kernel) {
      launch(kernel, grid, dim3(kI8QuantThreads), 0, st, (const void*)((const uint8_t*)x + r0 * ld * kSize),
             ld, live ? live + r0 : nullptr, n, K, q + r0 * i8_pitch(K), s + r0);
    };
    if (wave)
      go(i8_quantize_kernel<DT, 64, 8>);
    else
      go(i8_quantize_kernel<DT, 256, 4>);
    if (hipGetLastError() != hipSuccess) return MOE_ELAUNCH;
  }
  return MOE_OK;
}

}  // namespace moe

extern "C" int64_t i8_packed_bytes(int E, int N, int K, int glu) {
  if (E < 1 || N < 1 || K < 1 || K > MOE_I8_MAX_K || (glu != 0 && (N & 1))) return -1;
  const int64_t each = (int64_t)moe::i8_tiles(N, glu != 0) * moe::i8_chunks(K) * moe::kI8TileBytes;
  return E <= INT64_MAX / each ? E * each : -1;
}

extern "C" int i8_pack_experts(const int8_t* q_src, int E, int N, int K, int glu, int8_t* q_dst,
                               void* stream) {
  if (!q_src || !q_dst || E < 1 || N < 1 || K < 1) return MOE_EINVAL;
  const int64_t bytes = i8_packed_bytes(E, N, K, glu);
  if (bytes < 0 || E > MOE_MAX_E) return MOE_ESHAPE;
  if (((uintptr_t)q_dst) & 15) return MOE_EALIGN;
  const int64_t items = (int64_t)E * ((moe::i8_chunks(K) + 3) / 4) * moe::i8_tiles(N, glu != 0);
  for (int64_t first = 0; first < items; first += moe::kI8MaxGrid) {
    const int64_t n = items - first < moe::kI8MaxGrid ? items - first : moe::kI8MaxGrid;
    moe::launch(moe::i8_pack_kernel, dim3((unsigned)n), dim3(256), 0, (hipStream_t)stream, q_src,
                first, N, K, glu != 0, q_dst);
    if (hipGetLastError() != hipSuccess) return MOE_ELAUNCH;
  }
  return MOE_OK;
}

extern "C" int i8_quantize(const void* x, int x_dtype, int64_t ld, const int32_t* live,
                           int64_t rows, int K, int8_t* q, float* s, void* stream) {
  if (!x || !q || !s || rows < 1 || K < 1) return MOE_EINVAL;
  if (x_dtype != MOE_BF16 && x_dtype != MOE_F16 && x_dtype != MOE_F32) return MOE_EINVAL;
  if (K > MOE_I8_MAX_K || ld < K || rows > 0x7FFFFFFFLL) return MOE_ESHAPE;
  if ((((uintptr_t)q) & 15) || (((uintptr_t)s) & 3) || (((uintptr_t)live) & 3) ||
      (((uintptr_t)x) & (x_dtype == MOE_F32 ? 3 : 1)))
    return MOE_EALIGN;
  const hipStream_t st = (hipStream_t)stream;
  if (x_dtype == MOE_BF16) return moe::launch_quantize<MOE_BF16>(x, ld, live, rows, K, q, s, st);
  if (x_dtype == MOE_F16) return moe::launch_quantize<MOE_F16>(x, ld, live, rows, K, q, s, st);
  return moe::launch_quantize<MOE_F32>(x, ld, live, rows, K, q, s, st);
}
