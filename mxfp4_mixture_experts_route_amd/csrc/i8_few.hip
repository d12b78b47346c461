// i8_linear of a few rows in one launch: every workgroup quantizes the rows into LDS and runs one
// tile of 16 channels over them, its wavefronts splitting K.
//
// Bound by the stream of weights (N K bytes), and for small matrices by latency: the row is read,
// its largest magnitude found and its codes formed while the first weights are on their way
// (2880 -> 5760 channels, 16.6 MB: 6.6 us for one row, 7.3 for four; the least there is to do, one
// tile of 64 values, 3.3; a launch that does next to nothing 1.6. Calls captured into one graph.)
// Products run on v_mfma_i32_16x16x64_i8 (a weight tile is A, the rows are columns of B); the sums
// are exact 32-bit integers (K <= 65536 keeps 128 * 128 * K below 2^31), so the split of K changes
// no result.
#include "i8.hpp"
#include "launch.hpp"

namespace moe {

constexpr int kI8FewThreads = 256;
constexpr int kI8FewRing = 12;                // weight chunks of a wavefront in flight
constexpr int kI8FewVec = 8;                  // row vectors per lane in registers (K <= 4096)
constexpr int64_t kI8FewMaxRows = 8, kI8FewMaxValues = 24 * 1024;

template <int DT, bool TAIL>
__global__ void __launch_bounds__(kI8FewThreads)
i8_few_kernel(const void* __restrict__ x, int64_t ld, int rows, const int8_t* __restrict__ wq,
              const float* __restrict__ wsc, const float* __restrict__ bias, int N, int K, int glu,
              int held, void* __restrict__ out, int out_dt, int64_t ld_out) {
  extern __shared__ __attribute__((aligned(16))) uint8_t rowsq[];   // the quantized rows
  constexpr int kWaves = kI8FewThreads / kWave;
  constexpr int kSize = DT == MOE_F32 ? 4 : 2;
  __shared__ float sx[kI8TileRows];
  __shared__ i32x4_t red[kWaves][kWave];
  const int tid = (int)threadIdx.x, lane = tid & 63, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int unit = (int)blockIdx.x, NT = i8_tiles(N, glu);
  const int KP = i8_pitch(K), LP = i8_lds_pitch(KP), C = i8_chunks(K);
  const int cb = C * wave / kWaves, len = C * (wave + 1) / kWaves - cb;
  const uint32_t step = (uint32_t)NT * kI8TileBytes;
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(wq, (uint32_t)C * step);
  auto run = [&](int c0) {
    return I8Run{rw, ((uint32_t)(cb + c0) * NT + unit) * kI8TileBytes, step, len - c0};
  };
  I8Ring<kI8FewRing> ring;
  const int jj = tid & 15, m = tid >> 4, n = i8_channel(unit, jj, N, glu);
  float sc = 0.0f, bi = 0.0f;
  if (!held) {
    ring.fill(run(0));
    for (int r = wave; r < rows; r += kWaves) {
      const float s = i8_row_to_lds<DT>(x, r * ld, K, rowsq, r, LP, KP);
      if (lane == 0) sx[r] = s;
    }
  } else {
    // a row per wavefront; of a single row every wavefront takes a share of the codes. Loads
    // return in the order of their issue: the weights go out behind the last row
    I8Row<kI8FewVec, DT> xr;
    const int parts = rows == 1 ? kWaves : 1, share = rows == 1 ? wave : 0;
    for (int r = rows == 1 ? 0 : wave;; r += kWaves) {
      if (r < rows) xr.template load<TAIL>((const uint8_t*)x + r * ld * kSize, K);
      __builtin_amdgcn_sched_barrier(0);
      if (r + kWaves >= rows) ring.fill(run(0));
      if (r < rows) {
        const I8Quant z(xr.largest());
        xr.store_codes(z, rowsq, r, LP, KP, share, parts);
        if (lane == 0) sx[r] = z.s;
      }
      if (r + kWaves >= rows) break;
    }
  }
  if (n >= 0) {
    sc = wsc[n];
    if (bias) bi = bias[n];
  }
  lds_barrier();
  const int mb = min(col, rows - 1);   // columns past the rows repeat the last row
  const uint8_t* bp = rowsq + mb * LP;
  i32x4_t acc = {0, 0, 0, 0}, acc1 = {0, 0, 0, 0};
  for (int c0 = 0; c0 < len; c0 += kI8FewRing)
    ring.take(bp, mb, cb + c0, C - 1, run(c0 + kI8FewRing), acc, acc1);
  red[wave][lane] = acc + acc1;
  lds_barrier();
  if (m < rows && n >= 0) {
    const int from = (jj >> 2) * 16 + m, i = jj & 3;
    int sum = 0;
#pragma unroll
    for (int p = 0; p < kWaves; ++p) sum += red[p][from][i];
    store_elem(out, m * ld_out + n, i8_scaled(sum, sx[m], sc, bi), out_dt);
  }
}

}  // namespace moe

// Whether a product of `rows` rows is taken by moe_launch_i8_few. Every workgroup quantizes all the
// rows, four at a time, against a launch of its own for that (calls in a loop, us, here and there):
// 2880 -> 5760 channels 4 rows 7.3 / 9.1, 8 rows 8.4 / 9.8, 16 rows 11.0 / 9.7; 4096 -> 8192 6 rows
// 10.2 / 11.0, 8 rows 11.8 / 11.0; 8000 -> 128 2 rows 11.8 / 11.7, 4 rows 12.5 / 11.8.
bool moe_i8_few(int64_t rows, const i8_experts* w) {
  return rows <= moe::kI8FewMaxRows && rows * w->K <= moe::kI8FewMaxValues;
}

int moe_launch_i8_few(const void* x, int x_dt, int64_t ld, int rows, const i8_experts* w, void* out,
                      int out_dt, int64_t ld_out, hipStream_t st) {
  const int held = w->K <= moe::kI8FewVec * 8 * moe::kWave;   // rows that fit in registers
  const size_t lds = (size_t)rows * moe::i8_lds_pitch(moe::i8_pitch(w->K));
  auto go = [&](auto kernel) {
    moe::launch(kernel, dim3((unsigned)moe::i8_tiles(w->N, w->glu)), dim3(moe::kI8FewThreads), lds,
                st, x, ld, rows, w->q, w->s, w->bias, w->N, w->K, w->glu, held, out, out_dt, ld_out);
  };
  const bool tail = w->K % 8 != 0;
  if (x_dt == MOE_BF16)
    tail ? go(moe::i8_few_kernel<MOE_BF16, true>) : go(moe::i8_few_kernel<MOE_BF16, false>);
  else if (x_dt == MOE_F16)
    tail ? go(moe::i8_few_kernel<MOE_F16, true>) : go(moe::i8_few_kernel<MOE_F16, false>);
  else
    tail ? go(moe::i8_few_kernel<MOE_F32, true>) : go(moe::i8_few_kernel<MOE_F32, false>);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ELAUNCH;
}
