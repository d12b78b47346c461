// 8-bit integer projections of many rows, dense or over the routed rows of every expert, with the
// clamped SwiGLU as an optional epilogue; the function of i8_gemv.hip, bit for bit (the sums are
// exact 32-bit integers).
//
// A workgroup computes BM rows of activations by BN channels. K goes in chunks of 64: the chunk's
// weight tiles and activation rows are copied by LDS-DMA into a ring of NST buffers, NST - 1
// chunks ahead, so that one barrier per chunk is all the synchronization there is, and the
// products run on v_mfma_i32_32x32x32_i8 (weights = A, activations = B).
//  * Weights lie in tiles of 16 rows in the MFMA's lane order, so copies and reads of them are
//    contiguous.
//  * Activations lie as rows of 64 bytes, their four 16-byte pieces permuted by the row
//    (piece p of row m at p ^ ((m >> 2) & 3)): the 64 lanes of a B read then meet every bank once
//    per quarter (16-byte LDS reads serve lanes 0-3, 12-15, 20-27 of each half together).
//  * SwiGLU: gate tiles and up tiles alternate, so a lane's 16 sums of a 32x32 block are 8 gate
//    values and the 8 up values of the same channels.
#include "i8.hpp"
#include "launch.hpp"

namespace moe {

typedef __attribute__((address_space(1))) const void* gptr_t;
typedef __attribute__((address_space(3))) void* lptr_t;

template <int BM_, int BN_, int WM_, int WN_, int NST_>
struct I8Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NST = NST_;
  static constexpr int kWaves = WM * WN, kThreads = kWaves * kWave;
  static constexpr int FM = BM / WM / 32, FN = BN / WN / 32;      // 32x32 blocks per wavefront
  static constexpr int kOps = (BM + BN) / 16;                     // 1 KB copies per chunk
  static constexpr int kOpsW = (kOps + kWaves - 1) / kWaves;      // of a wavefront
  static constexpr int kStage = (BM + BN) * kI8Chunk;
  static constexpr int kLds = NST * kStage + (BM + BN) * 8;       // + what the epilogue needs per row and channel
  static_assert(BM % (32 * WM) == 0 && BN % (32 * WN) == 0, "whole blocks");
  static_assert((NST - 1) * kOpsW <= 63, "vmcnt range");
  static_assert(kLds <= 160 * 1024, "LDS");
};

// The work item of a routed launch: (expert, block of rows) number `blk` of those that hold live
// rows, in expert order; every wavefront computes it for itself. Returns the number of all such
// blocks; e < 0 where blk is past them.
template <int BM>
__device__ __forceinline__ int routed_block(const int32_t* __restrict__ counts, int E, int blk,
                                            int& e, int& m) {
  const int lane = (int)(threadIdx.x & 63);
  const int per = (E + kWave - 1) / kWave;
  const int e0 = lane * per;
  int mine = 0;
  for (int i = 0; i < per; ++i)
    if (e0 + i < E) mine += (max(counts[e0 + i], 0) + BM - 1) / BM;
  int upto = mine;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int u = __shfl_up(upto, o);
    if (lane >= o) upto += u;
  }
  const int total = __shfl(upto, kWave - 1);
  const bool here = blk >= upto - mine && blk < upto;
  int fe = -1, fm = 0;
  if (here) {
    int left = blk - (upto - mine);
    for (int i = 0; i < per; ++i) {
      const int b = e0 + i < E ? (max(counts[e0 + i], 0) + BM - 1) / BM : 0;
      if (left < b) {
        fe = e0 + i;
        fm = left;
        break;
      }
      left -= b;
    }
  }
  const uint64_t who = __ballot(here);
  const int src = who ? __ffsll((unsigned long long)who) - 1 : 0;
  e = __shfl(fe, src);
  m = __shfl(fm, src);
  return total;
}

template <class TL, bool GLU, bool ROUTED, int OUT>
__global__ void __launch_bounds__(TL::kThreads)
i8_gemm_kernel(const int8_t* __restrict__ a, const float* __restrict__ as,
               const int32_t* __restrict__ a_row, int64_t a_rows, const int8_t* __restrict__ wq,
               const float* __restrict__ wsc, const float* __restrict__ bias, int E, int N, int K,
               int glu, const int32_t* __restrict__ counts, const int32_t* __restrict__ basep,
               int64_t rows, int64_t mpad, int nblocks, float alpha, float limit,
               void* __restrict__ out, int64_t ld_out, int vec) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  constexpr int BM = TL::BM, BN = TL::BN, NST = TL::NST, FM = TL::FM, FN = TL::FN;
  constexpr int kUnits = GLU ? BN / 32 : BN / 16;   // 16-channel units of the workgroup
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // 1. the item: workgroups are dealt to the 8 XCDs round robin, so item numbers are dealt in 8
  // contiguous shares, and an XCD's L2 sees neighbouring items
  int e = 0, mb, nb;
  {
    const int x = (int)blockIdx.x & 7, i = (int)blockIdx.x >> 3;
    if constexpr (ROUTED) {
      int m0;
      const int blocks = routed_block<BM>(counts, E, 0, e, m0);
      const int total = blocks * nblocks, per = (total + 7) >> 3;
      const int item = x * per + i;
      if (i >= per || item >= total) return;
      // items of an expert are neighbours, its row blocks the nearest (they share the weights)
      const int blk0 = item / nblocks;
      routed_block<BM>(counts, E, blk0, e, m0);
      const int first = blk0 - m0;                              // the expert's first block
      const int eb = ((int)counts[e] + BM - 1) / BM;            // its number of blocks
      const int in = item - first * nblocks;
      nb = in / eb;
      mb = in - nb * eb;
    } else {
      const int mblocks = (int)((rows + BM - 1) / BM);
      const int total = mblocks * nblocks, per = (total + 7) >> 3;
      const int item = x * per + i;
      if (i >= per || item >= total) return;
      // groups of 8 row blocks, channels ascending inside a group: a share is a near-square
      constexpr int G = 8;
      const int g = item / (G * nblocks), in = item - g * G * nblocks;
      const int gm = min(G, mblocks - g * G);
      nb = in / gm;
      mb = g * G + (in - nb * gm);
    }
  }
  e = __builtin_amdgcn_readfirstlane(e);
  mb = __builtin_amdgcn_readfirstlane(mb);
  nb = __builtin_amdgcn_readfirstlane(nb);
  int64_t count = ROUTED ? (int64_t)counts[e] : rows;
  const int64_t base = ROUTED ? (int64_t)basep[e] : 0;
  count = min(count, mpad - base);   // never past the output, whatever the CSR holds
  if (base < 0) return;
  const int64_t r0 = (int64_t)mb * BM;
  const int live = (int)min((int64_t)BM, count - r0);
  if (live <= 0) return;

  // 2. source row and scale of every row of the block, scale and bias of every channel
  const int NT = i8_tiles(N, glu), HT = i8_half_tiles(N, glu);
  const int u0 = nb * kUnits;
  int* const src_s = reinterpret_cast<int*>(lds + NST * TL::kStage);
  float* const scale_s = reinterpret_cast<float*>(src_s + BM);
  float* const wsc_s = scale_s + BM;
  float* const bias_s = wsc_s + BN;
  for (int m = tid; m < BM; m += TL::kThreads) {
    int64_t src = -1;
    if (m < live) {
      src = a_row ? (int64_t)a_row[base + r0 + m] : base + r0 + m;
      if ((uint64_t)src >= (uint64_t)a_rows) src = -1;   // such a row is not stored
    }
    src_s[m] = (int)src;
    scale_s[m] = src >= 0 ? as[src] : 0.0f;
  }
  for (int j = tid; j < BN; j += TL::kThreads) {
    const int u = j >> 4;   // the unit, or of SwiGLU the gate or up tile of it
    const int t = GLU ? ((u & 1) ? HT : 0) + min(u0 + (u >> 1), HT - 1) : min(u0 + u, NT - 1);
    const int n = i8_channel(t, j & 15, N, glu);
    wsc_s[j] = n >= 0 ? wsc[(int64_t)e * N + n] : 0.0f;
    bias_s[j] = n >= 0 && bias ? bias[(int64_t)e * N + n] : 0.0f;
  }
  __syncthreads();

  // 3. copies of a chunk: operation j < BN / 16 is weight tile j, the others 16 rows each
  const int KP = i8_pitch(K), C = KP / kI8Chunk;
  const int8_t* src[TL::kOpsW];
  int64_t step[TL::kOpsW];
  int dst[TL::kOpsW];
#pragma unroll
  for (int i = 0; i < TL::kOpsW; ++i) {
    // a surplus operation repeats the last one (the same bytes to the same place)
    const int j = min(wave + i * TL::kWaves, TL::kOps - 1);
    dst[i] = j * 1024;
    if (j < BN / 16) {
      // tiles past the last one repeat it; their channels are not stored
      const int t = GLU ? (j & 1) * HT + min(u0 + (j >> 1), HT - 1) : min(u0 + j, NT - 1);
      src[i] = wq + ((int64_t)e * C * NT + t) * kI8TileBytes + lane * 16;
      step[i] = (int64_t)NT * kI8TileBytes;
    } else {
      const int m = (j - BN / 16) * 16 + (lane >> 2);
      const int piece = (lane & 3) ^ ((m >> 2) & 3);
      src[i] = a + (int64_t)max(src_s[m], 0) * KP + piece * 16;
      step[i] = kI8Chunk;
    }
  }
  auto issue = [&](int slot) {
#pragma unroll
    for (int i = 0; i < TL::kOpsW; ++i) {
      __builtin_amdgcn_global_load_lds((gptr_t)src[i],
                                       (lptr_t)(lds + slot * TL::kStage + dst[i]), 16, 0, 0);
      src[i] += step[i];
    }
  };

  // 4. the K loop
  const int wm = wave % TL::WM, wn = wave / TL::WM;
  const int l31 = lane & 31, hi = lane >> 5;
  // weight block f: tiles 2 f and 2 f + 1 of the wavefront's; piece 2 ks + hi of a row
  const int wo = (wn * FN * 2 + (l31 >> 4)) * 1024 + (l31 & 15) * 16 + hi * 256;
  const int ml = wm * FM * 32 + l31;
  const int ao = BN * kI8Chunk + ml * kI8Chunk;
  const int p0 = (hi ^ ((ml >> 2) & 3)) * 16;          // ks = 0; ks = 1 is piece ^ 2
  i32x16_t acc[FN][FM];
#pragma unroll
  for (int f = 0; f < FN; ++f)
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[f][m][i] = 0;

#pragma unroll
  for (int s = 0; s < NST - 1; ++s)
    if (s < C) issue(s);
  int slot = 0, fill = NST - 1;
  for (int c = 0; c < C; ++c) {
    // this wavefront's copies of chunk c have landed (those of the chunks after it may be in
    // flight); the barrier says so for every wavefront, and that chunk c - 1 has been read
    __builtin_amdgcn_sched_barrier(0);
    if (c + NST - 1 <= C)
      __builtin_amdgcn_s_waitcnt(waitcnt_vm((NST - 2) * TL::kOpsW));
    else
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if (c + NST - 1 < C) issue(fill);
    fill = fill == NST - 1 ? 0 : fill + 1;
    const uint8_t* st = lds + slot * TL::kStage;
    slot = slot == NST - 1 ? 0 : slot + 1;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      i32x4_t wv[FN], av[FM];
#pragma unroll
      for (int f = 0; f < FN; ++f)
        wv[f] = *reinterpret_cast<const i32x4_t*>(st + wo + f * 2048 + ks * 512);
#pragma unroll
      for (int m = 0; m < FM; ++m)
        av[m] = *reinterpret_cast<const i32x4_t*>(st + ao + m * 32 * kI8Chunk + (p0 ^ (ks * 32)));
#pragma unroll
      for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int m = 0; m < FM; ++m)
          acc[f][m] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wv[f], av[m], acc[f][m], 0, 0, 0);
    }
  }

  // 5. scales, bias, activation: a lane holds, for row m of the block, channels 8 q + 4 hi + i
  // (q, i < 4) of each 32-channel block (SwiGLU: q = 0, 1 gate values, q + 2 the up values)
  const int F = N >> 1;
#pragma unroll
  for (int m = 0; m < FM; ++m) {
    const int mr = ml + m * 32;
    if (src_s[mr] < 0) continue;
    const float sa = scale_s[mr];
    const int64_t at = (base + r0 + mr) * ld_out;
#pragma unroll
    for (int f = 0; f < FN; ++f) {
#pragma unroll
      for (int q = 0; q < (GLU ? 2 : 4); ++q) {
        const int j = (wn * FN + f) * 32 + 8 * q + 4 * hi;   // place in the workgroup's channels
        const float4 sw = *reinterpret_cast<const float4*>(wsc_s + j);
        const float4 sb = *reinterpret_cast<const float4*>(bias_s + j);
        float v[4] = {fmaf((float)acc[f][m][4 * q], sa * sw.x, sb.x),
                      fmaf((float)acc[f][m][4 * q + 1], sa * sw.y, sb.y),
                      fmaf((float)acc[f][m][4 * q + 2], sa * sw.z, sb.z),
                      fmaf((float)acc[f][m][4 * q + 3], sa * sw.w, sb.w)};
        int ch, some;   // first channel of the four, how many of them there are
        if constexpr (GLU) {
          const float4 uw = *reinterpret_cast<const float4*>(wsc_s + j + 16);
          const float4 ub = *reinterpret_cast<const float4*>(bias_s + j + 16);
          v[0] = i8_swiglu(v[0], fmaf((float)acc[f][m][8 + 4 * q], sa * uw.x, ub.x), alpha, limit);
          v[1] = i8_swiglu(v[1], fmaf((float)acc[f][m][9 + 4 * q], sa * uw.y, ub.y), alpha, limit);
          v[2] = i8_swiglu(v[2], fmaf((float)acc[f][m][10 + 4 * q], sa * uw.z, ub.z), alpha, limit);
          v[3] = i8_swiglu(v[3], fmaf((float)acc[f][m][11 + 4 * q], sa * uw.w, ub.w), alpha, limit);
          ch = (u0 + wn * FN + f) * 16 + 8 * q + 4 * hi;
          some = F - ch;
        } else {
          const int tl = u0 + (wn * FN + f) * 2 + (q >> 1), half = glu && tl >= HT;
          ch = (tl - half * HT) * 16 + 8 * (q & 1) + 4 * hi;
          some = tl < NT ? (glu ? F : N) - ch : 0;
          ch += half * F;
        }
        if (vec && some >= 4) {
          if constexpr (OUT == MOE_F32) {
            *reinterpret_cast<float4*>((float*)out + at + ch) = make_float4(v[0], v[1], v[2], v[3]);
          } else {
            uint32_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              b[i] = OUT == MOE_F16 ? (uint32_t)__half_as_ushort(__float2half_rn(v[i]))
                                    : f32_to_bf16_bits(v[i]);
            *reinterpret_cast<uint2*>((uint16_t*)out + at + ch) =
                make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < some) store_elem(out, at + ch + i, v[i], OUT);
        }
      }
    }
  }
}

struct I8GemmArgs {
  const int8_t* a;
  const float* as;
  const int32_t* a_row;
  int64_t a_rows;
  const i8_experts* w;
  const int32_t *counts, *basep;
  int64_t rows, mpad;
  float alpha, limit;
  void* out;
  int out_dt;
  int64_t ld_out;
};

template <class TL, bool GLU, bool ROUTED, int OUT>
int launch_tile(const I8GemmArgs& g, hipStream_t st) {
  static bool lds_attr_set[kMaxDevices] = {};   // > 64 KB of LDS: opt in once per device
  const int dslot = device_slot();
  if (TL::kLds > 65536 && (dslot < 0 || !lds_attr_set[dslot])) {
    if (hipFuncSetAttribute(reinterpret_cast<const void*>(&i8_gemm_kernel<TL, GLU, ROUTED, OUT>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, TL::kLds) != hipSuccess)
      return MOE_ELAUNCH;
    if (dslot >= 0) lds_attr_set[dslot] = true;
  }
  const i8_experts* w = g.w;
  const int units = GLU ? i8_half_tiles(w->N, 1) : i8_tiles(w->N, w->glu);
  const int per = GLU ? TL::BN / 32 : TL::BN / 16;
  const int64_t nblocks = (units + per - 1) / per;
  // routed: at most one partly filled block per expert beside the full ones
  const int64_t mblocks = ROUTED ? g.mpad / TL::BM + (w->E < g.mpad ? w->E : g.mpad)
                                 : (g.rows + TL::BM - 1) / TL::BM;
  const int64_t grid = (mblocks * nblocks + 7) / 8 * 8;
  if (grid > 0x7FFFFFFFLL) return MOE_ESHAPE;
  constexpr int size = OUT == MOE_F32 ? 4 : 2;
  const int vec = !((uintptr_t)g.out & (4 * size - 1)) && (g.ld_out & 3) == 0 &&
                  (!w->glu || (w->N / 2) % 4 == 0);
  launch(i8_gemm_kernel<TL, GLU, ROUTED, OUT>, dim3((unsigned)grid), dim3(TL::kThreads), TL::kLds, st,
         g.a, g.as, g.a_row, g.a_rows, w->q, w->s, w->bias, w->E, w->N, w->K, w->glu, g.counts,
         g.basep, g.rows, g.mpad, (int)nblocks, g.alpha, g.limit, g.out, g.ld_out, vec);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ELAUNCH;
}

template <class TL>
int launch_form(const I8GemmArgs& g, bool glu, hipStream_t st) {
  if (g.counts)
    return glu ? launch_tile<TL, true, true, MOE_BF16>(g, st)
               : launch_tile<TL, false, true, MOE_F32>(g, st);
  return g.out_dt == MOE_F32   ? launch_tile<TL, false, false, MOE_F32>(g, st)
         : g.out_dt == MOE_F16 ? launch_tile<TL, false, false, MOE_F16>(g, st)
                               : launch_tile<TL, false, false, MOE_BF16>(g, st);
}

}  // namespace moe

int moe_launch_i8_gemv(const int8_t* a, const float* as, const int32_t* a_row, int64_t a_rows,
                       const i8_experts* w, const int32_t* counts, const int32_t* basep,
                       int64_t rows, int64_t mpad, int act, float alpha, float limit, void* out,
                       int out_dt, int64_t ld_out, hipStream_t st);

int moe_launch_i8_gemm(const int8_t* a, const float* as, const int32_t* a_row, int64_t a_rows,
                       const i8_experts* w, const int32_t* counts, const int32_t* basep,
                       int64_t rows, int64_t mpad, int act, float alpha, float limit, void* out,
                       int out_dt, int64_t ld_out, hipStream_t st) {
  const bool glu = act == MOE_ACT_SWIGLU_OAI;
  const moe::I8GemmArgs g{a, as, a_row, a_rows, w, counts, basep, rows, mpad, alpha, limit,
                          out, out_dt, ld_out};
  // rows per product (routed: the mean over the experts, padding included)
  const int64_t per = counts ? mpad / w->E : rows;
  int form = per <= 24 ? 0 : per <= 96 ? 1 : 2;
  if (form == 2 && ((rows + 255) / 256) * ((w->N + 255) / 256) >= 256) form = 3;
  if (form == 0)
    return moe_launch_i8_gemv(a, as, a_row, a_rows, w, counts, basep, rows, mpad, act, alpha, limit,
                              out, out_dt, ld_out, st);
  if (form == 1) return moe::launch_form<moe::I8Tile<64, 128, 1, 4, 6>>(g, glu, st);
  if (form == 2) return moe::launch_form<moe::I8Tile<128, 128, 2, 2, 4>>(g, glu, st);
  return moe::launch_form<moe::I8Tile<256, 256, 2, 4, 4>>(g, glu, st);
}
