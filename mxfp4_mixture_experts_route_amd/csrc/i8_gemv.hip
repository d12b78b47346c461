// 8-bit integer projections of few rows: out = (sum_k aq wq) * s_row * s_channel + bias, dense or
// over the routed rows of every expert, with the clamped SwiGLU as an optional epilogue.
//
// Products run on v_mfma_i32_16x16x64_i8: a weight tile of 16 rows is the A operand, up to 16
// rows of activations are the columns of B, and the sums are exact 32-bit integers (K <= 65536
// keeps 127 * 128 * K below 2^31), so the split of K over wavefronts changes no result.
#include "i8.hpp"
#include "launch.hpp"

namespace moe {

constexpr int kI8GemvThreads = 256;
constexpr int kI8GemvSeg = 8;       // chunks loaded ahead of their products

// grid (units, experts); a unit is one tile of 16 channels (SwiGLU: a gate tile and its up tile).
// The four wavefronts split K (SwiGLU: two a tile), rows go in groups of 16 * NB.
template <int NB, bool GLU>
__global__ void __launch_bounds__(kI8GemvThreads)
i8_gemv_kernel(const int8_t* __restrict__ a, const float* __restrict__ as,
               const int32_t* __restrict__ a_row, int64_t a_rows, const int8_t* __restrict__ wq,
               const float* __restrict__ wsc, const float* __restrict__ bias, int N, int K,
               int glu, const int32_t* __restrict__ counts, const int32_t* __restrict__ basep,
               int64_t rows, int64_t mpad, float alpha, float limit, void* __restrict__ out,
               int out_dt, int64_t ld_out) {
  constexpr int KS = GLU ? 2 : 4;
  __shared__ i32x4_t red[4][NB][kWave];
  const int e = (int)blockIdx.y;
  int64_t count = counts ? counts[e] : rows;
  const int64_t base = counts ? basep[e] : 0;
  count = min(count, mpad - base);   // never past the output, whatever the CSR holds
  if (count <= 0 || base < 0) return;
  const int tid = (int)threadIdx.x, lane = tid & 63, col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int part = wave % KS;
  const int unit = (int)blockIdx.x;
  const int NT = i8_tiles(N, glu), HT = i8_half_tiles(N, glu);
  const int tile = GLU && wave / KS ? HT + unit : unit;
  const int KP = i8_pitch(K), C = KP / kI8Chunk;
  const int cb = C * part / KS, ce = C * (part + 1) / KS;
  const int64_t step = (int64_t)NT * kI8TileBytes;
  const int8_t* wp = wq + ((int64_t)e * C * NT + tile) * kI8TileBytes + lane * 16;

  for (int64_t r0 = 0; r0 < count; r0 += 16 * NB) {
    const int8_t* ap[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      // rows past the count and rows whose index is out of range read row 0 and are not stored
      const int64_t r = r0 + b * 16 + col;
      int64_t src = r < count ? (a_row ? (int64_t)a_row[base + r] : base + r) : 0;
      if ((uint64_t)src >= (uint64_t)a_rows) src = 0;
      ap[b] = a + src * KP + g * 16;
    }
    i32x4_t acc[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[b] = i32x4_t{0, 0, 0, 0};
    for (int c0 = cb; c0 < ce; c0 += kI8GemvSeg) {
      i32x4_t wv[kI8GemvSeg], av[kI8GemvSeg][NB];
#pragma unroll
      for (int i = 0; i < kI8GemvSeg; ++i) {
        const int c = min(c0 + i, ce - 1);
        wv[i] = *reinterpret_cast<const i32x4_t*>(wp + (int64_t)c * step);
#pragma unroll
        for (int b = 0; b < NB; ++b)
          av[i][b] = *reinterpret_cast<const i32x4_t*>(ap[b] + c * kI8Chunk);
      }
#pragma unroll
      for (int i = 0; i < kI8GemvSeg; ++i)
        if (c0 + i < ce)
#pragma unroll
          for (int b = 0; b < NB; ++b)
            acc[b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[i], av[i][b], acc[b], 0, 0, 0);
    }
    __syncthreads();   // the last group's sums are read
#pragma unroll
    for (int b = 0; b < NB; ++b) red[wave][b][lane] = acc[b];
    __syncthreads();
    // one thread per output of the unit: 16 channels of a row on 16 consecutive threads
    const int j = tid & 15;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int m = tid >> 4;
      const int64_t r = r0 + b * 16 + m;
      if (r >= count) continue;
      const int64_t src = a_row ? (int64_t)a_row[base + r] : base + r;
      if ((uint64_t)src >= (uint64_t)a_rows) continue;
      const int from = (j >> 2) * 16 + m;
      const float sa = as[src];
      int sum[GLU ? 2 : 1];
#pragma unroll
      for (int h = 0; h < (GLU ? 2 : 1); ++h) {
        sum[h] = 0;
#pragma unroll
        for (int p = 0; p < KS; ++p) sum[h] += red[h * KS + p][b][from][j & 3];
      }
      if constexpr (GLU) {
        const int F = N >> 1, n = unit * 16 + j;
        if (n >= F) continue;
        const int64_t cg = (int64_t)e * N + n;
        const float gate = fmaf((float)sum[0], sa * wsc[cg], bias ? bias[cg] : 0.0f);
        const float up = fmaf((float)sum[1], sa * wsc[cg + F], bias ? bias[cg + F] : 0.0f);
        store_elem(out, (base + r) * ld_out + n, i8_swiglu(gate, up, alpha, limit), out_dt);
      } else {
        const int n = i8_channel(unit, j, N, glu);
        if (n < 0) continue;
        const int64_t cg = (int64_t)e * N + n;
        const float v = fmaf((float)sum[0], sa * wsc[cg], bias ? bias[cg] : 0.0f);
        store_elem(out, (base + r) * ld_out + n, v, out_dt);
      }
    }
  }
}

}  // namespace moe

int moe_launch_i8_gemv(const int8_t* a, const float* as, const int32_t* a_row, int64_t a_rows,
                       const i8_experts* w, const int32_t* counts, const int32_t* basep,
                       int64_t rows, int64_t mpad, int act, float alpha, float limit, void* out,
                       int out_dt, int64_t ld_out, hipStream_t st) {
  const bool glu = act == MOE_ACT_SWIGLU_OAI;
  const int units = glu ? moe::i8_half_tiles(w->N, 1) : moe::i8_tiles(w->N, w->glu);
  const dim3 grid((unsigned)units, (unsigned)(counts ? w->E : 1));
  auto go = [&](auto kernel) {
    moe::launch(kernel, grid, dim3(moe::kI8GemvThreads), 0, st, a, as, a_row, a_rows, w->q, w->s,
                w->bias, w->N, w->K, w->glu, counts, basep, rows, mpad, alpha, limit, out,
                out_dt, ld_out);
  };
  if (glu)
    go(moe::i8_gemv_kernel<1, true>);
  else
    go(moe::i8_gemv_kernel<1, false>);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ELAUNCH;
}
