// 8-bit integer projections, dense or over the routed rows of every expert, with the clamped
// SwiGLU as an optional epilogue: out = (sum_k aq wq) * (s_row * s_channel) + bias. The sums are
// exact 32-bit integers (K <= 65536 keeps 128 * 128 * K below 2^31), so every tile and every split
// of K gives the same bits.
//
// A workgroup computes BM rows of activations by BN channels on v_mfma_i32_32x32x32_i8 (weights =
// A, activations = B). K goes in steps of 128, a whole cache line of an activation row (see
// i8_pitch), that is two chunks of the packed weights. Two forms:
//  * I8Tile: weights and activations of a step are copied by LDS-DMA into a ring of NST buffers.
//  * I8Direct: every wavefront has 32 channels of its own and streams their weights into a ring of
//    registers; LDS holds only activations. More bytes are in flight on a CU.
// Either way one barrier per step is all the synchronization there is, and the operands of each
// half chunk (32 of K) are read from LDS while the products of the half before run.
//  * Weights lie in tiles of 16 rows in the MFMA's lane order, so copies and reads of them are
//    contiguous.
//  * Activations lie in LDS as rows of 128 bytes, their eight 16-byte pieces permuted by the row
//    (piece p of row m at p ^ ((m >> 1) & 7)): the 64 lanes of a B read then meet every bank once
//    per quarter (16-byte LDS reads serve lanes 0-3, 12-15, 20-27 of each half together).
//  * SwiGLU: gate tiles and up tiles alternate, so a lane's 16 sums of a 32x32 block are 8 gate
//    values and the 8 up values of the same channels.
//
// What bounds it: with few rows an expert the stream of weights (32 experts of 5760 x 2880, 64
// tokens: 79 us, 6.8 TB/s); with more of them what a CU takes in, weights and activations, from L2
// and beyond (512 tokens: 101 us, matrix cores busy 28 % of the time); in large dense products the
// matrix cores (4096 rows, 8192 -> 8192: 248 to 256 us, 2.2 POPS, matrix cores busy 52 %).
#include "i8.hpp"
#include "launch.hpp"

namespace moe {

typedef __attribute__((address_space(1))) const void* gptr_t;
typedef __attribute__((address_space(3))) void* lptr_t;

// 16 bytes per lane from a buffer into 1 KB of LDS (zeros past the buffer).
__device__ __forceinline__ void buf_copy16(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t voff,
                                           uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lptr_t)lds, 16, voff, soff, 0, 0);
}

constexpr int kI8Step = 2 * kI8Chunk;   // K of a step

// WK > 1: WK wavefronts split K, each with a ring of its own, and their sums meet in LDS at the end;
// there is no barrier in the K loop.
template <int BM_, int BN_, int WM_, int WN_, int NST_, int WK_ = 1>
struct I8Tile {
  static constexpr bool kDirect = false;
  static constexpr int kSimd = 1;   // wavefronts a SIMD has registers for, at least
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NST = NST_, WK = WK_;
  static constexpr int kWaves = WM * WN, kThreads = kWaves * WK * kWave;   // (waves of a group)
  static constexpr int FM = BM / WM / 32, FN = BN / WN / 32;      // 32x32 blocks per wavefront
  // 1 KB copies of a wavefront per step: weight tiles of both chunks, then 8 activation rows each
  static constexpr int kOpsB = BN / 8 / kWaves, kOpsA = BM / 8 / kWaves, kOpsW = kOpsB + kOpsA;
  static constexpr int kStageA = BN * kI8Step;                    // where a step's activations lie
  static constexpr int kStage = (BM + BN) * kI8Step;
  static constexpr int kRing = WK * NST * kStage;
  static constexpr int kRed = WK > 1 ? WK * BM * BN * 4 : 0;   // sums of the groups, where the rings were
  static constexpr int kLds = kRing + (BM + BN) * 8;   // + what the epilogue needs per row and channel
  static_assert(BN / 16 % kWaves == 0 && BM / 8 % kWaves == 0, "the same number of copies each");
  static_assert(BM % (32 * WM) == 0 && BN % (32 * WN) == 0, "whole blocks");
  static_assert(NST * kOpsW <= 63, "vmcnt range");
  static_assert(WK == 1 || kWaves == 1, "groups of one wavefront");
  static_assert(kLds <= 160 * 1024, "LDS");
};

// NST: steps in flight, of activations in LDS and of weights in registers. WK > 1: WK such groups of
// wavefronts split K, so that one group's products cover the other's waits.
template <int BM_, int BN_, int NST_, int WK_ = 1>
struct I8Direct {
  static constexpr bool kDirect = true;
  // (with registers for two instead of three, 512 tokens: gate_up 103 -> 112 us, down 69 -> 76)
  static constexpr int kSimd = WK_ > 1 ? 2 : 3;
  static constexpr int BM = BM_, BN = BN_, WM = 1, WN = BN / 32, NST = NST_, WK = WK_;
  static constexpr int kWaves = WN, kThreads = kWaves * WK * kWave;
  static constexpr int FM = BM / 32, FN = 1;
  static constexpr int kChunks = 2 * NST;                         // weight chunks in registers
  static constexpr int kOpsB = 1, kOpsA = BM / 8 / kWaves;        // (kOpsB: unused)
  static constexpr int kStageA = 0, kStage = BM * kI8Step;
  static constexpr int kRed = WK > 1 ? WK * BM * BN * 4 : 0;
  static constexpr int kOut = kRed + (WK > 1 ? BM : 32) * (BN * 4 + 16);   // (for the epilogue)
  static constexpr int kRing = WK * NST * kStage > kOut ? WK * NST * kStage : kOut;
  static constexpr int kLds = kRing + (BM + BN) * 8;
  static_assert(BM / 8 % kWaves == 0, "the same number of copies each");
  static_assert(4 * NST - 4 + (NST - 2) * kOpsA <= 63 && NST >= 2, "vmcnt range");
  static_assert(kLds <= 160 * 1024, "LDS");
};

// The row blocks of a routed launch: the experts' blocks of BM rows, numbered in expert order.
// Lane l of every wavefront holds the experts l * per .. of the list.
template <int BM>
struct I8Blocks {
  int per, upto, mine, total;   // experts a lane, blocks up to and of this lane's, all blocks

  __device__ __forceinline__ int of(const int32_t* __restrict__ counts, int e, int E) const {
    return e < E ? (max(counts[e], 0) + BM - 1) / BM : 0;
  }
  __device__ __forceinline__ I8Blocks(const int32_t* __restrict__ counts, int E) {
    const int lane = (int)(threadIdx.x & 63);
    per = (E + kWave - 1) / kWave;
    mine = 0;
    for (int i = 0; i < per; ++i) mine += of(counts, lane * per + i, E);
    upto = mine;
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
      const int u = __shfl_up(upto, o);
      if (lane >= o) upto += u;
    }
    total = __builtin_amdgcn_readlane(upto, kWave - 1);
  }
  // Expert of block number blk (< total), its block there, the number of its blocks.
  __device__ __forceinline__ void find(const int32_t* __restrict__ counts, int E, int blk, int& e,
                                       int& m, int& n) const {
    const int lane = (int)(threadIdx.x & 63);
    const bool here = blk >= upto - mine && blk < upto;
    int left = blk - (upto - mine), fe = lane, fn = mine;
    if (per > 1 && here)
      for (int i = 0; i < per; ++i) {
        fe = lane * per + i;
        fn = of(counts, fe, E);
        if (left < fn) break;
        left -= fn;
      }
    const int src = __ffsll((unsigned long long)__ballot(here)) - 1;
    e = __builtin_amdgcn_readlane(fe, src);
    m = __builtin_amdgcn_readlane(left, src);
    n = __builtin_amdgcn_readlane(fn, src);
  }
};

template <class TL, bool GLU, bool ROUTED, int OUT>
__global__ void __launch_bounds__(TL::kThreads, TL::kSimd)
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
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wave = TL::WK > 1 ? wid % TL::kWaves : wid;   // in its group
  const int part = TL::WK > 1 ? wid / TL::kWaves : 0;     // the group

  // 1. the item: workgroups are dealt to the 8 XCDs round robin, so item numbers are dealt in 8
  // contiguous shares, and an XCD's L2 sees neighbouring items
  int e = 0, mb, nb;
  bool once;   // the only block of rows that reads these weights
  {
    const int x = (int)blockIdx.x & 7, i = (int)blockIdx.x >> 3;
    if constexpr (ROUTED) {
      const I8Blocks<BM> blocks(counts, E);
      const int total = blocks.total * nblocks, per = (total + 7) >> 3;
      const int item = x * per + i;
      if (i >= per || item >= total) return;
      // items of an expert are neighbours, its row blocks the nearest (they share the weights)
      const int blk0 = item / nblocks;
      int m0, eb;
      blocks.find(counts, E, blk0, e, m0, eb);
      const int in = item - (blk0 - m0) * nblocks;
      nb = in / eb;
      mb = in - nb * eb;
      once = eb == 1;
    } else {
      const int mblocks = (int)((rows + BM - 1) / BM);
      const int total = mblocks * nblocks, per = (total + 7) >> 3;
      once = mblocks == 1;
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
  count = min(count, mpad - base);   // never past the output
  if (base < 0) return;
  const int64_t r0 = (int64_t)mb * BM;
  const int live = (int)min((int64_t)BM, count - r0);
  if (live <= 0) return;

  // 2. the source rows of the block are on their way while the first weights go out
  const int NT = i8_tiles(N, glu), HT = i8_half_tiles(N, glu);
  const int u0 = nb * kUnits;
  int* const src_s = reinterpret_cast<int*>(lds + TL::kRing);
  float* const scale_s = reinterpret_cast<float*>(src_s + BM);
  float* const wsc_s = scale_s + BM;
  float* const bias_s = wsc_s + BN;
  constexpr int kRowsT = (BM + TL::kThreads - 1) / TL::kThreads;
  int src_r[kRowsT];
#pragma unroll
  for (int i = 0; i < kRowsT; ++i) {
    const int m = tid + i * TL::kThreads;
    int64_t src = -1;
    if (m < live) src = ROUTED && a_row ? (int64_t)a_row[base + r0 + m] : base + r0 + m;
    src_r[i] = (int)src;
  }
  __builtin_amdgcn_sched_barrier(0);
  const int wm = wave % TL::WM, wn = wave / TL::WM;
  const int l31 = lane & 31, hi = lane >> 5;

  // 3. copies. Steps [db, db + S) of K are this group's; the last step may have one chunk (the
  // rows' padding is zero: it is multiplied with the weights of the chunk before)
  const int KP = i8_pitch(K), CK = i8_chunks(K), DK = (CK + 1) / 2;
  const int db = DK * part / TL::WK, S = DK * (part + 1) / TL::WK - db;
  uint8_t* const ring = lds + part * NST * TL::kStage;
  const int64_t wstep = (int64_t)NT * kI8TileBytes;
  const int first = ROUTED ? 0 : (int)r0;   // (the rows of a routed product lie within 4 GB)
  const int8_t* const a0 = a + (int64_t)first * KP;
  auto tile_of = [&](int i) { return wave + i * TL::kWaves; };   // weight tile of copy i
  auto rows_of = [&](int i) { return wave + i * TL::kWaves; };   // group of 8 rows of copy i
  // I8Tile: 64-bit scalar addresses that step through K and a 32-bit offset per lane
  const int8_t* wbase = wq + ((int64_t)e * CK + 2 * db) * wstep;
  const int8_t* abase = a0 + db * kI8Step;
  int wnext = 2 * db;   // chunk at wbase
  uint32_t wvoff[TL::kOpsB], avoff[TL::kOpsA];
#pragma unroll
  for (int i = 0; i < (TL::kDirect ? 0 : TL::kOpsB / 2); ++i) {
    // tiles past the last one repeat it; their channels are not stored
    const int j = tile_of(i);
    const int t = GLU ? (j & 1) * HT + min(u0 + (j >> 1), HT - 1) : min(u0 + j, NT - 1);
    wvoff[i] = (uint32_t)t * kI8TileBytes + lane * 16;
  }
  // Weights that no other workgroup reads carry the nontemporal hint, so that they do not push
  // the activations out of L2 (gate_up of 64 tokens: 92 -> 80 us); with more row blocks an expert
  // the others find them there (256 tokens with the hint everywhere: 89 -> 98 us)
  auto issue_w = [&](int slot) {
    const int64_t second = wnext + 1 < CK ? wstep : 0;
#pragma unroll
    for (int i = 0; i < TL::kOpsB; ++i) {
      const int half = i / ((TL::kOpsB + 1) / 2), ti = i % ((TL::kOpsB + 1) / 2);
      const int8_t* const p = (half ? wbase + second : wbase) + wvoff[ti];
      uint8_t* const to = ring + slot * TL::kStage + half * BN * kI8Chunk + tile_of(ti) * 1024;
      if (once)
        __builtin_amdgcn_global_load_lds((gptr_t)p, (lptr_t)to, 16, 0, 2);
      else
        __builtin_amdgcn_global_load_lds((gptr_t)p, (lptr_t)to, 16, 0, 0);
    }
    wbase += 2 * wstep;
    wnext += 2;
  };
  auto issue_a = [&](int slot) {
#pragma unroll
    for (int i = 0; i < TL::kOpsA; ++i)
      __builtin_amdgcn_global_load_lds((gptr_t)(abase + avoff[i]),
                                       (lptr_t)(ring + slot * TL::kStage + TL::kStageA + rows_of(i) * 1024), 16, 0, 0);
    abase += kI8Step;
  };
  // I8Direct: buffer loads; what lies past the end is out of range (zeros, nothing read), so that
  // every trip has the same loads in flight. The wavefront's two tiles are the halves of a 32-row
  // operand.
  constexpr int kChunks = TL::kDirect ? 2 * NST : 1;
  // every group makes the same number of trips (they meet in the barriers)
  const int cb = TL::WK > 1 ? 2 * db : 0, ce = TL::WK > 1 ? min(CK, 2 * (db + S)) : CK;
  const int trips = TL::WK == 1 ? CK : 2 * ((DK + TL::WK - 1) / TL::WK);
  const int dt = GLU ? ((l31 >> 4) ? HT : 0) + min(u0 + wave, HT - 1) : min(u0 + 2 * wave + (l31 >> 4), NT - 1);
  const uint32_t dvoff = (uint32_t)dt * kI8TileBytes + hi * 256 + (l31 & 15) * 16;
  u32x4_t dw[kChunks][2];
  auto load_w = [&](int i, int c) {
    const __amdgpu_buffer_rsrc_t r =
        make_rsrc(wq + (int64_t)e * CK * wstep, cb + c < ce ? (uint32_t)(CK * wstep) : 0u);
    const uint32_t soff = cb + c < ce ? (uint32_t)((cb + c) * wstep) : 0u;
    dw[i][0] = once ? buf_load16_nt(r, dvoff, soff) : buf_load16(r, dvoff, soff);
    dw[i][1] = once ? buf_load16_nt(r, dvoff + 512, soff) : buf_load16(r, dvoff + 512, soff);
  };
  const uint32_t abytes = (uint32_t)((ROUTED ? a_rows : (int64_t)live) * KP);
  auto load_a = [&](int slot, int d) {
    const __amdgpu_buffer_rsrc_t r = make_rsrc(a0, d < S ? abytes : 0u);
#pragma unroll
    for (int i = 0; i < TL::kOpsA; ++i)
      buf_copy16(r, ring + slot * TL::kStage + rows_of(i) * 1024, avoff[i], (db + d) * kI8Step);
  };

  if constexpr (TL::kDirect) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) load_w(i, i);
  } else {
#pragma unroll
    for (int s = 0; s < NST; ++s)
      if (s < S) issue_w(s);
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < kRowsT; ++i) {
    const int m = tid + i * TL::kThreads;
    // a source row out of range: the row is not stored
    if (m < BM) src_s[m] = (uint64_t)(int64_t)src_r[i] < (uint64_t)a_rows ? src_r[i] : -1;
  }
  lds_barrier();
#pragma unroll
  for (int i = 0; i < TL::kOpsA; ++i) {
    const int m = rows_of(i) * 8 + (lane >> 3);
    const int piece = (lane & 7) ^ ((m >> 1) & 7);
    avoff[i] = (uint32_t)max(src_s[m] - first, 0) * (uint32_t)KP + piece * 16;
    // no row: past any buffer, so that nothing is read
    if (TL::kDirect && src_s[m] < 0) avoff[i] = 0xFFFFFFF0u;
  }
#pragma unroll
  for (int s = 0; s < NST; ++s) {
    if constexpr (TL::kDirect)
      load_a(s, s);
    else if (s < S)
      issue_a(s);
  }
  __builtin_amdgcn_sched_barrier(0);

  // what the epilogue needs goes out behind the first copies: the scale of a row, scale and bias
  // of a channel
  constexpr int kChT = (BN + TL::kThreads - 1) / TL::kThreads;
  float row_scale[kRowsT], ch_scale[kChT], ch_bias[kChT];
#pragma unroll
  for (int i = 0; i < kRowsT; ++i) {
    const int m = tid + i * TL::kThreads;
    row_scale[i] = 1.0f;   // (of what is not stored)
    if (m < BM && src_s[m] >= 0) row_scale[i] = as[src_s[m]];
  }
#pragma unroll
  for (int i = 0; i < kChT; ++i) {
    const int j = tid + i * TL::kThreads, u = j >> 4;   // SwiGLU: even tiles are gate, odd ones up
    const int t = GLU ? ((u & 1) ? HT : 0) + min(u0 + (u >> 1), HT - 1) : min(u0 + u, NT - 1);
    const int n = j < BN ? i8_channel(t, j & 15, N, glu) : -1;
    ch_scale[i] = 1.0f;
    ch_bias[i] = 0.0f;
    if (n >= 0) {
      ch_scale[i] = wsc[(int64_t)e * N + n];
      if (bias) ch_bias[i] = bias[(int64_t)e * N + n];
    }
  }
  __builtin_amdgcn_sched_barrier(0);

  // 4. the K loop: half chunk h (0..3) of a step multiplies pieces 2 h + hi of the rows with the
  // same pieces of the weights
  const int wo = (wn * FN * 2 + (l31 >> 4)) * 1024 + (l31 & 15) * 16 + hi * 256;
  const int ml = wm * FM * 32 + l31, sw = (ml >> 1) & 7;
  i32x16_t acc[FN][FM];
#pragma unroll
  for (int f = 0; f < FN; ++f)
#pragma unroll
    for (int m = 0; m < FM; ++m)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[f][m][i] = 0;
  i32x4_t wv[2][FN], av[2][FM];   // operands of the half in hand and of the next
  auto read = [&](int h, const uint8_t* st) {
    if constexpr (!TL::kDirect)
#pragma unroll
      for (int f = 0; f < FN; ++f)
        wv[h & 1][f] = *reinterpret_cast<const i32x4_t*>(st + (h >> 1) * BN * kI8Chunk + wo + f * 2048 + (h & 1) * 512);
    const uint8_t* const p = st + TL::kStageA + ml * kI8Step + (((2 * h + hi) ^ sw) << 4);
#pragma unroll
    for (int m = 0; m < FM; ++m)
      av[h & 1][m] = *reinterpret_cast<const i32x4_t*>(p + m * 32 * kI8Step);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&](int h) {
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
      for (int m = 0; m < FM; ++m)
        acc[f][m] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wv[h & 1][f], av[h & 1][m], acc[f][m], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  };
  // the activations' copies of the first steps lie behind all their weights'
  if (TL::kDirect || S >= NST)
    __builtin_amdgcn_s_waitcnt(waitcnt_vm((NST - 1) * TL::kOpsA));
  else
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
  if constexpr (TL::WK == 1 || TL::kDirect) __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  if (S > 0 || TL::kDirect) read(0, ring);
  if constexpr (TL::kDirect) {
    for (int c0 = 0; c0 < trips; c0 += kChunks) {
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c = c0 + i, h = (i & 1) * 2;
        if (c >= trips) break;
        const uint8_t* const st = ring + (i >> 1) * TL::kStage;
        read(h + 1, st);
        __builtin_memcpy(&wv[0][0], &dw[i][0], 16);
        multiply(h);
        if (i & 1) {
          // this wavefront has read the step, and its activations of the next have landed (behind
          // them: the weights of their own trip and of 2 NST - 3 more, the activations of NST - 2
          // steps; at first the activations of NST - 2 steps at least); the barrier says so for
          // every wavefront
          if (c < 2 * NST - 2)
            __builtin_amdgcn_s_waitcnt(waitcnt_vm((NST - 2) * TL::kOpsA) & ~(15 << 8));
          else
            __builtin_amdgcn_s_waitcnt(waitcnt_vm(4 * NST - 4 + (NST - 2) * TL::kOpsA) & ~(15 << 8));
          __builtin_amdgcn_s_barrier();
          __builtin_amdgcn_sched_barrier(0);
          load_a(i >> 1, (c >> 1) + NST);
          read(0, ring + ((i >> 1) + 1) % NST * TL::kStage);
        } else {
          read(2, st);
        }
        __builtin_memcpy(&wv[1][0], &dw[i][1], 16);
        multiply(h + 1);
        load_w(i, c + kChunks);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));   // no copy into LDS outlives the loop
  } else {
    int slot = 0;
    for (int s = 0; s < S; ++s) {
      const int next = slot == NST - 1 ? 0 : slot + 1;
      const uint8_t* const st = ring + slot * TL::kStage;
#pragma unroll
      for (int h = 0; h < 3; ++h) {
        read(h + 1, st);
        multiply(h);
      }
      if (s + 1 < S) {
        // this wavefront has read the step, and its copies of the next have landed (those of the
        // steps after it may be in flight); the barrier says so for every wavefront
        if (s + NST > S)
          __builtin_amdgcn_s_waitcnt(waitcnt_vm(0) & ~(15 << 8));
        else if (s < NST - 1)   // behind it: the activations' copies of NST - 2 - s steps at least
          __builtin_amdgcn_s_waitcnt(waitcnt_vm((NST - 2) * TL::kOpsA) & ~(15 << 8));
        else
          __builtin_amdgcn_s_waitcnt(waitcnt_vm((NST - 2) * TL::kOpsW) & ~(15 << 8));
        if constexpr (TL::WK == 1) __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        if (s + NST < S) {
          issue_w(slot);
          issue_a(slot);
        }
        read(0, ring + next * TL::kStage);
      }
      multiply(3);
      slot = next;
    }
  }

#pragma unroll
  for (int i = 0; i < kRowsT; ++i)
    if (tid + i * TL::kThreads < BM) scale_s[tid + i * TL::kThreads] = row_scale[i];
#pragma unroll
  for (int i = 0; i < kChT; ++i)
    if (tid + i * TL::kThreads < BN) {
      wsc_s[tid + i * TL::kThreads] = ch_scale[i];
      bias_s[tid + i * TL::kThreads] = ch_bias[i];
    }
  lds_barrier();   // (and every group is done with its ring)

  // 5. the groups' sums meet: a block's 16 sums of a lane lie as four quads of 256 x 4 bytes
  i32x4_t* const red = reinterpret_cast<i32x4_t*>(lds);
  if constexpr (TL::WK > 1) {
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
      for (int m = 0; m < FM; ++m)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          red[((((part * TL::kWaves + wave) * FN + f) * FM + m) * 4 + q) * kWave + lane] =
              i32x4_t{acc[f][m][4 * q], acc[f][m][4 * q + 1], acc[f][m][4 * q + 2], acc[f][m][4 * q + 3]};
    lds_barrier();
  }
  auto quad = [&](int f, int m, int q) {
    if constexpr (TL::WK > 1) {
      i32x4_t s = {0, 0, 0, 0};
#pragma unroll
      for (int p = 0; p < TL::WK; ++p) s += red[((((p * TL::kWaves + wave) * FN + f) * FM + m) * 4 + q) * kWave + lane];
      return s;
    } else {
      return i32x4_t{acc[f][m][4 * q], acc[f][m][4 * q + 1], acc[f][m][4 * q + 2], acc[f][m][4 * q + 3]};
    }
  };

  // 6. scales, bias, activation: a lane holds, for row m of the block, channels 8 q + 4 hi + i
  // (q, i < 4) of each 32-channel block (SwiGLU: q = 0, 1 gate values, q + 2 the up values). The
  // values go through LDS, where the rings were, and out as whole row pieces: stored from the
  // lanes, 8 to 16 bytes of 32 rows at a time, they cost 15 % of a 512-token gate_up projection
  constexpr int kSize = OUT == MOE_F32 ? 4 : 2;
  constexpr int kCh = GLU ? BN / 2 : BN;                 // output channels of the workgroup
  constexpr int kPitch = kCh * kSize + 16;
  // all rows at once where they fit, else one 32-row block of every wavefront after the other
  constexpr bool kAll = BM * kPitch + TL::kRed <= TL::kRing;
  static_assert(TL::WK == 1 || kAll, "LDS");
  constexpr int kPassRows = kAll ? BM : TL::WM * 32;
  static_assert(kPassRows * kPitch + TL::kRed <= TL::kRing, "LDS");
  uint8_t* const stage = lds + TL::kRed;
  auto emit = [&](int f, int m, int q, int lr) {         // lr: row of the pass
    const float sa = scale_s[ml + m * 32];
    const int j = (wn * FN + f) * 32 + 8 * q + 4 * hi;   // place in the workgroup's channels
    const float4 sw = *reinterpret_cast<const float4*>(wsc_s + j);
    const float4 sb = *reinterpret_cast<const float4*>(bias_s + j);
    const i32x4_t t = quad(f, m, q);
    float v[4];
    int ch = j;
    if constexpr (GLU) {
      const float4 uw = *reinterpret_cast<const float4*>(wsc_s + j + 16);
      const float4 ub = *reinterpret_cast<const float4*>(bias_s + j + 16);
      const i32x4_t u = quad(f, m, q + 2);
      float gu[8];
      i8_scaled<8>({t[0], t[1], t[2], t[3], u[0], u[1], u[2], u[3]}, {sa, sa, sa, sa, sa, sa, sa, sa},
                   {sw.x, sw.y, sw.z, sw.w, uw.x, uw.y, uw.z, uw.w},
                   {sb.x, sb.y, sb.z, sb.w, ub.x, ub.y, ub.z, ub.w}, gu);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = i8_swiglu(gu[i], gu[i + 4], alpha, limit);
      ch = (wn * FN + f) * 16 + 8 * q + 4 * hi;
    } else {
      i8_scaled<4>({t[0], t[1], t[2], t[3]}, {sa, sa, sa, sa}, {sw.x, sw.y, sw.z, sw.w},
                   {sb.x, sb.y, sb.z, sb.w}, v);
    }
    uint8_t* const dst = stage + lr * kPitch + ch * kSize;
    if constexpr (OUT == MOE_F32) {
      *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      if constexpr (OUT == MOE_F16) {
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = (uint32_t)__half_as_ushort(__float2half_rn(v[i]));
        *reinterpret_cast<uint2*>(dst) = make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
      } else {
        *reinterpret_cast<uint2*>(dst) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
      }
    }
  };
  // channel of place ch of the workgroup's output, or -1
  auto channel = [&](int ch) {
    if constexpr (GLU) {
      const int n = u0 * 16 + ch;
      return n < (N >> 1) ? n : -1;
    }
    const int t = u0 + (ch >> 4);
    return t < NT ? i8_channel(t, ch & 15, N, glu) : -1;
  };
  auto store = [&](int m) {                               // the rows of pass m
    auto row_of = [&](int lr) { return kAll ? lr : (lr >> 5) * FM * 32 + m * 32 + (lr & 31); };
    if (vec) {
      constexpr int kPer = 16 / kSize, kPieces = kCh / kPer;   // 16-byte pieces of a row
      for (int i = tid; i < kPassRows * kPieces; i += TL::kThreads) {
        const int lr = i / kPieces, ch = i % kPieces * kPer, mr = row_of(lr);
        if (src_s[mr] < 0) continue;
        const int n = channel(ch);
        const uint8_t* from = stage + lr * kPitch + ch * kSize;
        uint8_t* to = (uint8_t*)out + ((base + r0 + mr) * ld_out + n) * kSize;
        if (n >= 0 && channel(ch + kPer - 1) >= 0) {
          *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
        } else {
          for (int c = 0; c < kPer; ++c)
            if (channel(ch + c) >= 0) {
              if constexpr (kSize == 4)
                ((uint32_t*)to)[c] = ((const uint32_t*)from)[c];
              else
                ((uint16_t*)to)[c] = ((const uint16_t*)from)[c];
            }
        }
      }
    } else {
      for (int i = tid; i < kPassRows * kCh; i += TL::kThreads) {
        const int lr = i / kCh, ch = i % kCh, mr = row_of(lr), n = channel(ch);
        if (src_s[mr] < 0 || n < 0) continue;
        const uint8_t* from = stage + lr * kPitch + ch * kSize;
        uint8_t* to = (uint8_t*)out + ((base + r0 + mr) * ld_out + n) * kSize;
        if constexpr (kSize == 4)
          *(uint32_t*)to = *(const uint32_t*)from;
        else
          *(uint16_t*)to = *(const uint16_t*)from;
      }
    }
  };
  constexpr int QN = GLU ? 2 : 4;
  if constexpr (TL::WK > 1) {   // the quads of the blocks are dealt to the wavefronts
    for (int i = part; i < FM * FN * QN; i += TL::WK)
      emit(i / (FM * QN), i / QN % FM, i % QN, i / QN % FM * 32 + l31);
    lds_barrier();
    store(0);
  } else {
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      if (!kAll && m) lds_barrier();   // the rows of the pass before are out
      if ((wm * FM + m) * 32 < live)   // (blocks of 32 rows past the last are not formed)
#pragma unroll
      for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int q = 0; q < QN; ++q) emit(f, m, q, kAll ? ml + m * 32 : wm * 32 + l31);
      if (!kAll || m == FM - 1) {
        lds_barrier();
        store(m);
      }
    }
  }
}

struct I8GemmArgs {
  const I8Plain* plain;   // the rows before quantization, or NULL: a and as hold them quantized
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
  if (grid * TL::kThreads > 0xFFFFFFFFLL) return MOE_ESHAPE;   // threads of a launch
  constexpr int size = OUT == MOE_F32 ? 4 : 2;
  const int vec = !((uintptr_t)g.out & 15) && g.ld_out * size % 16 == 0 &&
                  (GLU || !w->glu || (w->N / 2) * size % 16 == 0);
  if (!ROUTED && g.plain) {   // behind every check, so that a refused call has enqueued nothing
    const int qs = i8_quantize(g.plain->x, g.plain->dt, g.plain->ld, nullptr, g.rows, w->K,
                               const_cast<int8_t*>(g.a), const_cast<float*>(g.as), st);
    if (qs != MOE_OK) return qs;
  }
  launch(i8_gemm_kernel<TL, GLU, ROUTED, OUT>, dim3((unsigned)grid), dim3(TL::kThreads), TL::kLds, st,
         g.a, g.as, g.a_row, g.a_rows, w->q, w->s, w->bias, w->E, w->N, w->K, w->glu, g.counts,
         g.basep, g.rows, g.mpad, (int)nblocks, g.alpha, g.limit, g.out, g.ld_out, vec);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ELAUNCH;
}

using I8Few = I8Tile<32, 32, 1, 1, 4, 4>;     // few rows: K split over four wavefronts
using I8Low = I8Tile<32, 64, 1, 1, 3, 4>;
using I8Half = I8Tile<64, 64, 1, 1, 2, 4>;
using I8Pair = I8Direct<64, 128, 4, 2>;       // K split over two groups
using I8Mid = I8Direct<64, 128, 3>;
using I8Wide = I8Direct<128, 128, 3>;
using I8Big = I8Tile<256, 256, 2, 4, 2>;

template <class TL>
int launch_dense(const I8GemmArgs& g, hipStream_t st) {
  return g.out_dt == MOE_F32   ? launch_tile<TL, false, false, MOE_F32>(g, st)
         : g.out_dt == MOE_F16 ? launch_tile<TL, false, false, MOE_F16>(g, st)
                               : launch_tile<TL, false, false, MOE_BF16>(g, st);
}

template <class TL>
int launch_routed(const I8GemmArgs& g, bool glu, hipStream_t st) {
  return glu ? launch_tile<TL, true, true, MOE_BF16>(g, st)
             : launch_tile<TL, false, true, MOE_F32>(g, st);
}

// Time of a dense product per chunk of K, in ns: a CU goes through ceil(tiles / 256) tiles, `one`
// ns a chunk where that is one and `each` ns for each of several, as measured at 2880 -> 5760
// channels and (I8Big) 8192 -> 8192 on 256 CUs. The least of them names the tile: at 64 rows
// I8Low takes 7.0 us, I8Few 10.0, I8Half 10.8, I8Pair 15; at 128 rows I8Half 9.6, I8Pair 11.8, I8Low
// 12.9; at 256 rows I8Pair 12.2, I8Mid 13.5; at 512 rows I8Mid 17.0, I8Wide 18.6, I8Pair 22, I8Half
// 25; at 2048 rows I8Wide 38.8, I8Mid 43.6, I8Big 46.2; 4096 rows of 8192: I8Big 267, I8Wide 302;
// 256 rows of 8192: I8Pair 25.4, I8Mid 30.8.
template <class TL>
double chunk_ns(int64_t rows, int64_t E, int units, double one, double each) {
  const int64_t tiles = E * ((rows + TL::BM - 1) / TL::BM) * ((units + TL::BN / 16 - 1) / (TL::BN / 16));
  const int64_t rounds = (tiles + 255) / 256;
  return rounds == 1 ? one : (double)rounds * each;
}

}  // namespace moe

int moe_launch_i8_gemm(const moe::I8Plain* plain, const int8_t* a, const float* as,
                       const int32_t* a_row, int64_t a_rows, const i8_experts* w,
                       const int32_t* counts, const int32_t* basep, int64_t rows, int64_t mpad,
                       int act, float alpha, float limit, void* out, int out_dt, int64_t ld_out,
                       hipStream_t st) {
  using namespace moe;
  const I8GemmArgs g{plain, a, as, a_row, a_rows, w, counts, basep, rows, mpad, alpha, limit,
                     out, out_dt, ld_out};
  // rows of a product and products: of the experts' rows only their sum is known here, so each is
  // taken to have the mean, padding included: with much padding the tile is too tall (64 tokens of
  // 32 experts: tile_m 16 87 us by I8Mid, tile_m 64 and 256 92 by I8Wide). The many rounds of I8Mid
  // over many experts take 172 ns each. gate_up of 32 experts, 64 tokens: I8Mid 79 us, I8Wide 88;
  // 256 tokens: 89 and 96; 512 tokens: 115 and 107; 2048 tokens: 228 and 195. 10 experts of 87
  // rows, 2338 -> 69 channels: I8Few 6.2 us, I8Wide 22.9; 6 of 3 rows, 1331 -> 1105: I8Few 5.4,
  // I8Mid 12.3; 20 of 134 rows, 1982 -> 2 x 98: I8Half 10.8, I8Wide 19.8; 59 of 130 rows, 573 ->
  // 326: I8Mid 14.2, I8Wide 19.7
  const bool glu = act == MOE_ACT_SWIGLU_OAI;
  const int64_t n = counts ? (mpad + w->E - 1) / w->E : rows, E = counts ? w->E : 1;
  const int units = i8_tiles(w->N, w->glu);
  const double ns[] = {chunk_ns<I8Few>(n, E, units, 45, 68),    chunk_ns<I8Low>(n, E, units, 70, 100),
                       chunk_ns<I8Half>(n, E, units, 120, 150), chunk_ns<I8Pair>(n, E, units, 185, 205),
                       chunk_ns<I8Mid>(n, E, units, 215, counts ? 172 : 147),
                       chunk_ns<I8Wide>(n, E, units, 310, 270), chunk_ns<I8Big>(n, E, units, 930, 1025)};
  int best = 0;
  for (int i = 1; i < (counts ? 6 : 7); ++i)
    if (ns[i] < ns[best]) best = i;
  if (counts) {
    switch (best) {
      case 0: return launch_routed<I8Few>(g, glu, st);
      case 1: return launch_routed<I8Low>(g, glu, st);
      case 2: return launch_routed<I8Half>(g, glu, st);
      case 3: return launch_routed<I8Pair>(g, glu, st);
      case 4: return launch_routed<I8Mid>(g, glu, st);
      default: return launch_routed<I8Wide>(g, glu, st);
    }
  }
  switch (best) {
    case 0: return launch_dense<I8Few>(g, st);
    case 1: return launch_dense<I8Low>(g, st);
    case 2: return launch_dense<I8Half>(g, st);
    case 3: return launch_dense<I8Pair>(g, st);
    case 4: return launch_dense<I8Mid>(g, st);
    case 5: return launch_dense<I8Wide>(g, st);
    default: return launch_dense<I8Big>(g, st);
  }
}
