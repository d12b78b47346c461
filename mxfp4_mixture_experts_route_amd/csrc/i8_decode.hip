// i8_moe_decode: the whole 8-bit mixture-of-experts layer of a few tokens in two launches.
//
// The chain is the one of mx4_moe_decode (PR #3579 "dasLLAMA gpt-oss arc", section "Fused MoE
// expert chain": stage 1 gate and up rows + bias + activation, stage 2 every routed expert's down
// row + bias and the routing-weighted sum in slot order) with 8-bit weights and with activations
// quantized per row in both stages:
//  * Launch 1: every workgroup routes all tokens (a wavefront per token, the picks meet in LDS),
//    takes the j-th picked expert with the tokens that picked it, quantizes their rows of x into
//    LDS and runs one gate tile and its up tile over them; h is written in routed-row order, in
//    bf16. One extra workgroup writes ids and w.
//  * Launch 2: a workgroup owns 16 channels of every token. It finds the scale of every h row,
//    runs the tile of each picked expert once over the rows of the tokens that picked it (h is
//    quantized on the way into the MFMA), and sums the slots of each token in slot order.
// An expert is read once however many of the tokens picked it. Sums are exact integers, so the
// results are those of i8_quantize, i8_moe_gemm and moe_combine bit for bit.
#include "i8.hpp"
#include "launch.hpp"
#include "route_core.hpp"

namespace moe {

constexpr int kI8DecMaxR = MOE_DECODE_MAX_T * MOE_DECODE_MAX_K;   // routed rows of a call
constexpr int kI8DecThreads = 256;
constexpr int kI8DownThreads = 512;
constexpr int kI8DecSeg = 8;
constexpr size_t kI8DecMaxLds = 144 * 1024;   // the quantized tokens of launch 1

// LDS pitch of a quantized row: an odd multiple of 128 bytes, so that with the pieces of 16 bytes
// of each 128 permuted by i8_swizzle the 16 rows of a B operand are read without bank conflicts.
__host__ __device__ __forceinline__ int i8_lds_pitch(int KP) {
  return (((KP + 127) >> 7) | 1) << 7;
}
__device__ __forceinline__ int i8_swizzle(int m, int off) { return off ^ (((m >> 1) & 7) << 4); }

// The j-th expert (ascending) of those set in a bitmap of E <= 1024 bits, or -1; every lane of
// the calling wavefront gets it.
__device__ __forceinline__ int nth_expert(const uint32_t* bits, int j) {
  const int lane = (int)(threadIdx.x & 63);
  uint32_t w = lane < MOE_MAX_E / 32 ? bits[lane] : 0u;
  const int c = __popc(w);
  int before = c;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int u = __shfl_up(before, o);
    if (lane >= o) before += u;
  }
  before -= c;
  const bool mine = j >= before && j < before + c;
  int id = 0;
  if (mine) {
    for (int i = before; i < j; ++i) w &= w - 1;
    id = lane * 32 + __ffs((int)w) - 1;
  }
  const uint64_t who = __ballot(mine);
  return who ? __shfl(id, __ffsll((unsigned long long)who) - 1) : -1;
}

// The routed rows (ascending) whose pick is expert e into list, their number returned to every
// lane of the calling wavefront; at most one per token.
__device__ __forceinline__ int rows_of_expert(const int* sid, int R, int e, int* list) {
  const int lane = (int)(threadIdx.x & 63);
  int n = 0;
  for (int r0 = 0; r0 < R; r0 += 64) {
    const bool hit = r0 + lane < R && sid[r0 + lane] == e;
    const uint64_t b = __ballot(hit);
    if (hit) list[n + __popcll(b & ((1ull << lane) - 1))] = r0 + lane;
    n += __popcll(b);
  }
  return n;
}

__global__ void __launch_bounds__(kI8DecThreads)
i8_decode_gate_up_kernel(const float* __restrict__ logits, const uint16_t* __restrict__ x, int T,
                         int E, int k, const int8_t* __restrict__ wq,
                         const float* __restrict__ wsc, const float* __restrict__ bias, int N,
                         int K, float alpha, float limit, int units, int32_t* __restrict__ ids,
                         float* __restrict__ w, uint16_t* __restrict__ h) {
  extern __shared__ __attribute__((aligned(16))) uint8_t rowsq[];   // 16 quantized rows
  __shared__ int sid[kI8DecMaxR], list[MOE_DECODE_MAX_T];
  __shared__ float sx[MOE_DECODE_MAX_T];
  __shared__ uint32_t bits[MOE_MAX_E / 32];
  __shared__ int sel[2];
  __shared__ i32x4_t red[4][kWave];
  const int tid = (int)threadIdx.x, lane = tid & 63, col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int R = T * k;

  if (blockIdx.x == 0) {   // the routing, for the caller and for launch 2
    for (int t = wave; t < T; t += kI8DecThreads / kWave) {
      int my_id;
      float my_v;
      wave_topk(logits + (size_t)t * E, E, k, my_id, my_v);
      write_topk(my_id, my_v, k, ids + t * k, w + t * k);
    }
    return;
  }
  const int item = (int)blockIdx.x - 1;
  const int j = item / units, unit = item - j * units;

  if (tid < MOE_MAX_E / 32) bits[tid] = 0u;
  __syncthreads();
  for (int t = wave; t < T; t += kI8DecThreads / kWave) {
    int my_id;
    float my_v;
    wave_topk(logits + (size_t)t * E, E, k, my_id, my_v);
    if (lane < k) {
      my_id = min(max(my_id, 0), E - 1);
      sid[t * k + lane] = my_id;
      atomicOr(&bits[my_id >> 5], 1u << (my_id & 31));
    }
  }
  __syncthreads();
  if (wave == 0) {
    const int e0 = nth_expert(bits, j);
    const int n0 = e0 >= 0 ? rows_of_expert(sid, R, e0, list) : 0;
    if (lane == 0) {
      sel[0] = e0;
      sel[1] = n0;
    }
  }
  __syncthreads();
  const int e = __builtin_amdgcn_readfirstlane(sel[0]);
  const int cnt = __builtin_amdgcn_readfirstlane(sel[1]);
  if (e < 0) return;   // fewer experts were picked than there could have been

  const int KP = i8_pitch(K), LP = i8_lds_pitch(KP), V = KP >> 3;
  for (int m = wave; m < cnt; m += kI8DecThreads / kWave) {
    const int64_t base = (int64_t)(list[m] / k) * K;
    uint32_t top = 0;
    for (int u = lane; u < V; u += kWave) {
      float t[8];
      load8<MOE_BF16, false>(x, base + u * 8, K - u * 8, t);
      top = max_abs8(t, top);
    }
    const I8Quant z(wave_umax(top));
    for (int u = lane; u < V; u += kWave) {
      float t[8];
      load8<MOE_BF16, false>(x, base + u * 8, K - u * 8, t);
      const int off = u * 8;
      *reinterpret_cast<uint2*>(rowsq + m * LP + i8_swizzle(m, off & ~15) + (off & 15)) =
          codes8<MOE_BF16>(z, t);
    }
    if (lane == 0) sx[m] = z.s;
  }
  __syncthreads();

  const int NT = i8_tiles(N, 1), HT = i8_half_tiles(N, 1), C = KP / kI8Chunk;
  const int part = wave & 1, tile = (wave >> 1) ? HT + unit : unit;
  const int cb = C * part / 2, ce = C * (part + 1) / 2;
  const int64_t step = (int64_t)NT * kI8TileBytes;
  const int8_t* wp = wq + ((int64_t)e * C * NT + tile) * kI8TileBytes + lane * 16;
  const int mb = min(col, cnt - 1);   // columns past the rows repeat the last row
  const uint8_t* bp = rowsq + mb * LP;
  i32x4_t acc = {0, 0, 0, 0};
  for (int c0 = cb; c0 < ce; c0 += kI8DecSeg) {
    i32x4_t wv[kI8DecSeg];
#pragma unroll
    for (int i = 0; i < kI8DecSeg; ++i)
      wv[i] = *reinterpret_cast<const i32x4_t*>(wp + (int64_t)min(c0 + i, ce - 1) * step);
#pragma unroll
    for (int i = 0; i < kI8DecSeg; ++i)
      if (c0 + i < ce) {
        const i32x4_t b = *reinterpret_cast<const i32x4_t*>(
            bp + i8_swizzle(mb, (c0 + i) * kI8Chunk + g * 16));
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[i], b, acc, 0, 0, 0);
      }
  }
  red[wave][lane] = acc;
  __syncthreads();
  const int F = N >> 1, jj = tid & 15, m = tid >> 4, n = unit * 16 + jj;
  if (m < cnt && n < F) {
    const int from = (jj >> 2) * 16 + m, i = jj & 3;
    const int64_t cg = (int64_t)e * N + n;
    const float sa = sx[m];
    const float gate = fmaf((float)(red[0][from][i] + red[1][from][i]), sa * wsc[cg],
                            bias ? bias[cg] : 0.0f);
    const float up = fmaf((float)(red[2][from][i] + red[3][from][i]), sa * wsc[cg + F],
                          bias ? bias[cg + F] : 0.0f);
    h[(int64_t)list[m] * F + n] = (uint16_t)f32_to_bf16_bits(i8_swiglu(gate, up, alpha, limit));
  }
}

__global__ void __launch_bounds__(kI8DownThreads)
i8_decode_down_kernel(const uint16_t* __restrict__ h, int T, int E, int k,
                      const int32_t* __restrict__ ids, const float* __restrict__ w,
                      const int8_t* __restrict__ wq, const float* __restrict__ wsc,
                      const float* __restrict__ bias, int D, int F, float* __restrict__ d,
                      void* __restrict__ y, int y_dt) {
  constexpr int kWaves = kI8DownThreads / kWave;
  __shared__ int sid[kI8DecMaxR];
  __shared__ float sh[kI8DecMaxR];                   // scale of each h row
  __shared__ uint32_t top[kI8DecMaxR];               // its largest magnitude
  __shared__ int acc_s[kI8DecMaxR][kI8TileRows];     // sums of each routed row
  __shared__ uint32_t bits[MOE_MAX_E / 32];
  __shared__ int lists[kWaves][MOE_DECODE_MAX_T];
  const int tid = (int)threadIdx.x, lane = tid & 63, col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int R = T * k, unit = (int)blockIdx.x;
  const int FP = i8_pitch(F), C = FP / kI8Chunk, NT = i8_tiles(D, 0);
  if (tid < MOE_MAX_E / 32) bits[tid] = 0u;
  for (int i = tid; i < R * kI8TileRows; i += kI8DownThreads) (&acc_s[0][0])[i] = 0;
  __syncthreads();
  for (int r = tid; r < R; r += kI8DownThreads) {
    const int e = min(max(ids[r], 0), E - 1);
    sid[r] = e;
    atomicOr(&bits[e >> 5], 1u << (e & 31));
  }
  for (int r = wave; r < R; r += kWaves) {
    uint32_t m = 0;
    for (int i = lane; i < F; i += kWave) m = max(m, ((uint32_t)h[(int64_t)r * F + i] << 16) & 0x7FFFFFFFu);
    m = wave_umax(m);
    if (lane == 0) {
      top[r] = m;
      sh[r] = I8Quant(m).s;
    }
  }
  __syncthreads();
  int picked = 0;
  for (int i = 0; i < MOE_MAX_E / 32; ++i) picked += __popc(bits[i]);
  constexpr int KS = 4;
  for (int it = wave; it < picked * KS; it += kWaves) {
    const int part = it % KS;
    const int e = nth_expert(bits, it / KS);
    const int cnt = rows_of_expert(sid, R, e, lists[wave]);
    // the list is written and read by the lanes of one wavefront, whose LDS operations complete
    // in order: only the compiler has to keep them so
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int rho = lists[wave][min(col, cnt - 1)];
    const uint16_t* hp = h + (int64_t)rho * F;
    const I8Quant z(top[rho]);
    const int cb = C * part / KS, ce = C * (part + 1) / KS;
    const int8_t* wp = wq + ((int64_t)e * C * NT + unit) * kI8TileBytes + lane * 16;
    const int64_t step = (int64_t)NT * kI8TileBytes;
    i32x4_t acc = {0, 0, 0, 0};
    for (int c = cb; c < ce; ++c) {
      const i32x4_t wv = *reinterpret_cast<const i32x4_t*>(wp + (int64_t)c * step);
      const int k0 = c * kI8Chunk + g * 16;
      float t0[8], t1[8];
      load8<MOE_BF16, false>(hp, k0, F - k0, t0);
      load8<MOE_BF16, false>(hp, k0 + 8, F - k0 - 8, t1);
      const uint2 lo = codes8<MOE_BF16>(z, t0), hi = codes8<MOE_BF16>(z, t1);
      const i32x4_t b = {(int)lo.x, (int)lo.y, (int)hi.x, (int)hi.y};
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv, b, acc, 0, 0, 0);
    }
    if (col < cnt)
#pragma unroll
      for (int i = 0; i < 4; ++i) atomicAdd(&acc_s[rho][4 * g + i], acc[i]);   // exact integers
  }
  __syncthreads();
  for (int i = tid; i < T * kI8TileRows; i += kI8DownThreads) {
    const int t = i >> 4, jj = i & 15, n = unit * 16 + jj;
    if (n >= D) continue;
    float yv = 0.0f;
    for (int s = 0; s < k; ++s) {
      const int r = t * k + s;
      const int64_t cg = (int64_t)sid[r] * D + n;
      const float dv = fmaf((float)acc_s[r][jj], sh[r] * wsc[cg], bias ? bias[cg] : 0.0f);
      if (d) d[(int64_t)r * D + n] = dv;
      yv = fmaf(w[r], dv, yv);
    }
    store_elem(y, (int64_t)t * D + n, yv, y_dt);
  }
}

}  // namespace moe

extern "C" int i8_moe_decode(const float* logits, const uint16_t* x, int64_t T, int E, int k,
                             const i8_experts* w_gu, const i8_experts* w_dn, float alpha,
                             float limit, int32_t* ids, float* w, uint16_t* h, float* d, void* y,
                             int y_dtype, void* stream) {
  if (!logits || !x || !w_gu || !w_dn || !ids || !w || !h || !y || !w_gu->q || !w_gu->s ||
      !w_dn->q || !w_dn->s || T < 1 || E < 1 || k < 1 || k > E)
    return MOE_EINVAL;
  if (y_dtype != MOE_BF16 && y_dtype != MOE_F16 && y_dtype != MOE_F32) return MOE_EINVAL;
  if (T > MOE_DECODE_MAX_T || E > MOE_MAX_E || k > MOE_DECODE_MAX_K) return MOE_ESHAPE;
  const int D = w_gu->K, N = w_gu->N, F = N / 2;
  if (w_gu->E != E || w_dn->E != E || w_gu->glu != 1 || w_dn->glu != 0 || N < 2 || (N & 1) ||
      D < 1 || w_dn->N != D || w_dn->K != F || D > MOE_I8_MAX_K || F > MOE_I8_MAX_K)
    return MOE_ESHAPE;
  if ((((uintptr_t)x) & 15) || (((uintptr_t)h) & 15) || (((uintptr_t)w_gu->q) & 15) ||
      (((uintptr_t)w_dn->q) & 15) || (((uintptr_t)w_gu->s) & 3) || (((uintptr_t)w_dn->s) & 3) ||
      (((uintptr_t)logits) & 3) || (d && (((uintptr_t)d) & 3)) ||
      (((uintptr_t)y) & (y_dtype == MOE_F32 ? 3 : 1)))
    return MOE_EALIGN;
  const int units = moe::i8_half_tiles(N, 1);
  const size_t lds = (size_t)T * moe::i8_lds_pitch(moe::i8_pitch(D));
  if (lds > moe::kI8DecMaxLds || (int64_t)units * 32 * moe::i8_pitch(D) >= (int64_t)1 << 31 ||
      (int64_t)moe::i8_tiles(D, 0) * 16 * moe::i8_pitch(F) >= (int64_t)1 << 31)
    return MOE_ESHAPE;
  static bool lds_attr_set[moe::kMaxDevices] = {};   // > 64 KB of LDS: opt in once per device
  const int dslot = moe::device_slot();
  if (lds > 65536 && (dslot < 0 || !lds_attr_set[dslot])) {
    if (hipFuncSetAttribute(reinterpret_cast<const void*>(&moe::i8_decode_gate_up_kernel),
                            hipFuncAttributeMaxDynamicSharedMemorySize,
                            (int)moe::kI8DecMaxLds) != hipSuccess)
      return MOE_ELAUNCH;
    if (dslot >= 0) lds_attr_set[dslot] = true;
  }
  const hipStream_t st = (hipStream_t)stream;
  const int64_t picks = T * k < E ? T * k : E;
  moe::launch(moe::i8_decode_gate_up_kernel, dim3((unsigned)(1 + picks * units)),
              dim3(moe::kI8DecThreads), lds, st, logits, x, (int)T, E, k, w_gu->q, w_gu->s,
              w_gu->bias, N, D, alpha, limit, units, ids, w, h);
  if (hipGetLastError() != hipSuccess) return MOE_ELAUNCH;
  moe::launch(moe::i8_decode_down_kernel, dim3((unsigned)moe::i8_tiles(D, 0)),
              dim3(moe::kI8DownThreads), 0, st, h, (int)T, E, k, ids, w, w_dn->q, w_dn->s,
              w_dn->bias, D, F, d, y, y_dtype);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ELAUNCH;
}
