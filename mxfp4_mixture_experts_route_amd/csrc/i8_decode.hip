// i8_moe_decode: the whole 8-bit mixture-of-experts layer of a few tokens in two launches (three for
// more than 16 routed rows).
//
// The chain is the one of mx4_moe_decode (PR #3579 "dasLLAMA gpt-oss arc", section "Fused MoE
// expert chain": stage 1 gate and up rows + bias + activation, stage 2 every routed expert's down
// row + bias and the routing-weighted sum in slot order) with 8-bit weights and with activations
// quantized per row in both stages:
//  * Launch 1: every workgroup routes all tokens (a wavefront per token, the picks meet in LDS),
//    takes the j-th picked expert with the tokens that picked it, quantizes their rows of x into
//    LDS and runs one gate tile and its up tile over them; h is written in routed-row order, in
//    bf16. One extra workgroup writes ids and w.
//  * Launch 2: a workgroup owns 16 channels of every token. It quantizes the h rows into LDS (more
//    than 16 are quantized by a launch between), runs the tile of each picked expert once over the
//    rows of the tokens that picked it, and sums the slots of each token in slot order.
// An expert is read once however many of the tokens picked it. Sums are exact integers, so the
// results are those of i8_quantize, i8_moe_gemm and moe_combine bit for bit.
//
// Bound by the stream of weights: 3 D F bytes of every picked expert. At D = F = 2880, k = 4: one
// token 11.7 + 9.6 us (99.5 MB, 4.7 TB/s); 16 tokens of 32 experts 71 + 5 + 38 us (620 MB, 5.4 TB/s);
// 5 tokens of 128 experts 50 + 5 + 29 us (470 MB, 5.6 TB/s).
// Rows of more than 4096 values do not fit the registers: they are read twice and the weights go out
// behind them, and one token goes the way of several (32 experts, k = 4, D = F = 4096 and 4160, by the
// rate of the weights: one token 5.1 and 3.3 TB/s, 5 tokens 5.6 and 4.8, 16 tokens 5.9 and 5.1).
// More than 128 experts are routed by the slower wave_topk (5 tokens: 128 experts 86 us, 129 90).
#include "i8.hpp"
#include "launch.hpp"
#include "route_core.hpp"

namespace moe {

constexpr int kI8DecMaxR = MOE_DECODE_MAX_T * MOE_DECODE_MAX_K;   // routed rows of a call
constexpr int kI8DecThreads = 256;
constexpr int kI8DownThreads = 512;
constexpr int kI8UpRing = 12;       // weight chunks of a wavefront in flight, launch 1
constexpr int kI8DownRing = 16;     // and launch 2
constexpr int kI8RowsRing = 12;     // launch 2 over quantized rows (as many of the rows')
constexpr int kI8OneRing = 12;      // launch 2 of one token
constexpr int kI8LdsRows = 16;      // h rows that launch 2 quantizes itself
constexpr int kI8DecVec = 8;        // row vectors per lane held in registers (K <= 4096)
constexpr size_t kI8DecMaxLds = 140 * 1024;   // quantized rows in LDS

// The experts set in a bitmap of E <= 1024 bits, in ascending order, spread over a wavefront.
struct I8Picked {
  uint32_t w;           // the lane's 32 bits
  int before, upto;     // experts in the lanes before it, and with its own
  int total;

  __device__ __forceinline__ explicit I8Picked(const uint32_t* bits) {
    const int lane = (int)(threadIdx.x & 63);
    w = lane < MOE_MAX_E / 32 ? bits[lane] : 0u;
    upto = __popc(w);
    before = -upto;
#pragma unroll
    for (int o = 1; o < MOE_MAX_E / 32; o <<= 1) {
      const int u = __shfl_up(upto, o);
      if (lane >= o) upto += u;
    }
    before += upto;
    total = __builtin_amdgcn_readlane(upto, MOE_MAX_E / 32 - 1);
  }
  // The j-th of them (j < total).
  __device__ __forceinline__ int nth(int j) const {
    const bool mine = j >= before && j < upto;   // (one lane: those past the bitmap are empty)
    int id = 0;
    if (mine) {
      uint32_t left = w;
      for (int i = before; i < j; ++i) left &= left - 1;
      id = (int)(threadIdx.x & 63) * 32 + __ffs((int)left) - 1;
    }
    return __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)__ballot(mine)) - 1);
  }
};

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

// ---- one token -------------------------------------------------------------------------------
// The picks of one token are k different experts with one row each, which is the same row (launch
// 1) or the slot's (launch 2). Every wavefront holds the whole row for its largest magnitude and
// quantizes the part of K it multiplies into LDS of its own, so that no wavefront waits for
// another before the sums meet; and there is little code (it is fetched anew in each launch, as
// the two launches and what runs between them share the instruction cache).

// Codes of the vectors of chunks [cb, ce) into the wavefront's LDS.
__device__ __forceinline__ void codes_of_part(const I8Row<kI8DecVec>& row, int cb, int ce, uint8_t* lds) {
  const I8Quant z(row.largest());
  row.store_part(z, lds, cb * 8, ce * 8);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // read by the same wavefront
}

// The first k <= E <= 64 N experts of a token in the order of rank_key, lane r holding the r-th; v[j]
// of a lane is the logit of expert 64 j + lane. Each round takes the largest key's high word over
// the wavefront and the lowest id that has it.
template <int N>
__device__ __forceinline__ int wave_pick(const float (&v)[N], int E, int k) {
  const int lane = (int)(threadIdx.x & 63);
  uint32_t key[N];   // NaN: 1 (below the word of -inf), taken or absent: 0
#pragma unroll
  for (int j = 0; j < N; ++j)
    key[j] = j * kWave + lane < E ? max((uint32_t)(rank_key(v[j], 0) >> 32), 1u) : 0u;
  int mine = 0;
  for (int r = 0; r < k; ++r) {
    uint32_t top = key[0];
#pragma unroll
    for (int j = 1; j < N; ++j) top = max(top, key[j]);
    top = wave_umax(top);
    int id = 0;
#pragma unroll
    for (int j = N - 1; j >= 0; --j) {
      const uint64_t who = __ballot(key[j] == top);
      if (who) id = j * kWave + __ffsll((unsigned long long)who) - 1;
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (id == j * kWave + lane) key[j] = 0u;
    if (lane == r) mine = id;
  }
  return mine;
}

// Logits of one token for wave_pick.
template <int N>
__device__ __forceinline__ void load_logits(const float* __restrict__ row, int E, float (&v)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int e = j * kWave + (int)(threadIdx.x & 63);
    v[j] = e < E ? row[e] : 0.0f;
  }
}

// Experts of all routed rows into sid and the bitmap, a token per wavefront; the logits of all of a
// wavefront's tokens are loaded together.
template <int N>
__device__ __forceinline__ void route_tokens(const float* __restrict__ logits, int T, int E, int k,
                                             int* sid, uint32_t* bits) {
  constexpr int kWaves = kI8DecThreads / kWave, kEach = (MOE_DECODE_MAX_T + kWaves - 1) / kWaves;
  const int lane = (int)(threadIdx.x & 63);
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  float v[kEach][N];
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    load_logits(logits + (size_t)min(wave + i * kWaves, T - 1) * E, E, v[i]);
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int t = wave + i * kWaves;
    if (t >= T) continue;
    const int id = wave_pick(v[i], E, k);
    if (lane < k) {
      sid[t * k + lane] = id;
      atomicOr(&bits[id >> 5], 1u << (id & 31));
    }
  }
}

// The expert of pick j of the token, the same on every lane.
__device__ __forceinline__ int route_one(const float* __restrict__ logits, float lv, int E, int k,
                                         int j, uint64_t* keys) {
  const int lane = (int)(threadIdx.x & 63);
  if (E <= kWave) return rank_pick(wave_rank_keys(rank_key(lv, lane), keys, E), j);
  if (E <= 2 * kWave) {
    float v[2];
    load_logits(logits, E, v);
    return __builtin_amdgcn_readlane(wave_pick(v, E, j + 1), j);
  }
  int my_id;
  float my_v;
  wave_topk(logits, E, k, my_id, my_v);
  return min(max(__builtin_amdgcn_readlane(my_id, j), 0), E - 1);
}

// Launch 1: workgroup 0 writes the routing, the others one unit (16 gate and 16 up rows) of a pick
// each: wavefronts {gate, up} x {halves of K}.
template <bool TAIL>
__global__ void __launch_bounds__(kI8DecThreads)
i8_one_gate_up_kernel(const float* __restrict__ logits, const uint16_t* __restrict__ x, int E, int k,
                      const int8_t* __restrict__ wq, const float* __restrict__ wsc,
                      const float* __restrict__ bias, int N, int K, float alpha, float limit,
                      int units, int32_t* __restrict__ ids, float* __restrict__ w,
                      uint16_t* __restrict__ h) {
  extern __shared__ __attribute__((aligned(16))) uint8_t rowsq[];   // part of the row per wavefront
  constexpr int kWaves = kI8DecThreads / kWave;
  __shared__ __attribute__((aligned(16))) uint64_t keys[kWaves][kWave];
  static_assert(__alignof__(keys) >= 16, "wave_rank_keys reads the keys in pairs");
  __shared__ int red[kWaves][kI8TileRows];
  const int tid = (int)threadIdx.x, lane = tid & 63, col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (blockIdx.x == 0) {
    if (wave == 0) {
      int my_id;
      float my_v;
      wave_topk(logits, E, k, my_id, my_v);
      write_topk(my_id, my_v, k, ids, w);
    }
    return;
  }
  const int item = (int)blockIdx.x - 1, j = item / units, unit = item - j * units;
  float lv = 0.0f;
  if (lane < E) lv = logits[lane];
  __builtin_amdgcn_sched_barrier(0);   // the logits come first
  I8Row<kI8DecVec> row;
  if (E <= kWave) row.load<TAIL>(x, K);
  __builtin_amdgcn_sched_barrier(0);
  const int e = __builtin_amdgcn_readfirstlane(route_one(logits, lv, E, k, j, keys[wave]));
  if (E > kWave) row.load<TAIL>(x, K);       // (the routing of more experts needs the registers)

  const int C = i8_chunks(K), NT = i8_tiles(N, 1), HT = i8_half_tiles(N, 1);
  const int part = wave & 1, tile = (wave >> 1) ? HT + unit : unit;
  const int cb = C * part / 2, len = C * (part + 1) / 2 - cb;
  const uint32_t step = (uint32_t)NT * kI8TileBytes;
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(wq + (int64_t)e * C * step, (uint32_t)C * step);
  auto run = [&](int c0) {
    return I8Run{rw, ((uint32_t)(cb + c0) * NT + tile) * kI8TileBytes, step, len - c0};
  };
  I8Ring<kI8UpRing> ring;
  ring.fill(run(0));
  const int F = N >> 1, n = unit * 16 + col;
  const int64_t cg = (int64_t)e * N + min(n, F - 1);
  float sg = 0.0f, su = 0.0f, bg = 0.0f, bu = 0.0f;
  if (wave == 0) {
    sg = wsc[cg];
    su = wsc[cg + F];
    if (bias) {
      bg = bias[cg];
      bu = bias[cg + F];
    }
  }
  uint8_t* const mine = rowsq + wave * ((C + 1) / 2) * kI8Chunk;
  codes_of_part(row, cb, cb + len, mine);
  const I8Quant z(row.largest());
  i32x4_t acc = {0, 0, 0, 0}, acc1 = {0, 0, 0, 0};
  for (int c0 = 0; c0 < len; c0 += kI8UpRing)
    ring.take(mine, 0, c0, max(len - 1, 0), run(c0 + kI8UpRing), acc, acc1);
  acc += acc1;
  if (col == 0)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][4 * g + i] = acc[i];
  lds_barrier();
  if (tid < kI8TileRows && n < F) {
    const float gate = i8_scaled(red[0][tid] + red[1][tid], z.s, sg, bg);
    const float up = i8_scaled(red[2][tid] + red[3][tid], z.s, su, bu);
    h[(int64_t)j * F + n] = bf16_one(i8_swiglu(gate, up, alpha, limit));
  }
}

// Launch 2: a workgroup owns 16 channels; wavefronts {slots} x {parts of K}.
template <bool TAIL>
__global__ void __launch_bounds__(1024)
i8_one_down_kernel(const uint16_t* __restrict__ h, int E, int k, int parts,
                   const int32_t* __restrict__ ids, const float* __restrict__ w,
                   const int8_t* __restrict__ wq, const float* __restrict__ wsc,
                   const float* __restrict__ bias, int D, int F, float* __restrict__ d,
                   void* __restrict__ y, int y_dt) {
  extern __shared__ __attribute__((aligned(16))) uint8_t rowsq[];   // part of a row per wavefront
  __shared__ int red[16][kI8TileRows];
  __shared__ float dv_s[MOE_DECODE_MAX_K][kI8TileRows];
  const int tid = (int)threadIdx.x, lane = tid & 63, col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int unit = (int)blockIdx.x, slot = wave / parts, part = wave - slot * parts;
  int e = ids[slot];
  const float wt = w[slot];
  __builtin_amdgcn_sched_barrier(0);   // the id comes first
  I8Row<kI8DecVec> row;
  row.load<TAIL>(h + (int64_t)slot * F, F);
  __builtin_amdgcn_sched_barrier(0);
  e = __builtin_amdgcn_readfirstlane(min(max(e, 0), E - 1));
  const int C = i8_chunks(F), NT = i8_tiles(D, 0);
  const int cb = C * part / parts, len = C * (part + 1) / parts - cb;
  const uint32_t step = (uint32_t)NT * kI8TileBytes;
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(wq + (int64_t)e * C * step, (uint32_t)C * step);
  auto run = [&](int c0) {
    return I8Run{rw, ((uint32_t)(cb + c0) * NT + unit) * kI8TileBytes, step, len - c0};
  };
  I8Ring<kI8OneRing> ring;
  ring.fill(run(0));
  const int n = unit * 16 + col;
  const int64_t cg = (int64_t)e * D + min(n, D - 1);
  float sc = 0.0f, bi = 0.0f;
  if (part == 0) {
    sc = wsc[cg];
    if (bias) bi = bias[cg];
  }
  uint8_t* const mine = rowsq + wave * ((C + parts - 1) / parts) * kI8Chunk;
  codes_of_part(row, cb, cb + len, mine);
  const I8Quant z(row.largest());
  i32x4_t acc = {0, 0, 0, 0}, acc1 = {0, 0, 0, 0};
  for (int c0 = 0; c0 < len; c0 += kI8OneRing)
    ring.take(mine, 0, c0, max(len - 1, 0), run(c0 + kI8OneRing), acc, acc1);
  acc += acc1;
  if (col == 0)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[wave][4 * g + i] = acc[i];
  lds_barrier();
  if (part == 0 && lane < kI8TileRows) {
    int sum = 0;
    for (int p = 0; p < parts; ++p) sum += red[wave + p][lane];
    const float dv = i8_scaled(sum, z.s, sc, bi);
    if (d && n < D) d[(int64_t)slot * D + n] = dv;
    dv_s[slot][lane] = wt;
    red[wave][lane] = __float_as_int(dv);
  }
  lds_barrier();
  if (tid < kI8TileRows && n < D) {
    float yv = 0.0f;
    for (int s = 0; s < k; ++s) yv = fmaf(dv_s[s][tid], __int_as_float(red[s * parts][tid]), yv);
    store_elem(y, n, yv, y_dt);
  }
}

// ---- several tokens --------------------------------------------------------------------------

template <bool TAIL>
__global__ void __launch_bounds__(kI8DecThreads, TAIL ? 3 : 4)   // (TAIL spills at four)
i8_decode_gate_up_kernel(const float* __restrict__ logits, const uint16_t* __restrict__ x, int T,
                         int E, int k, const int8_t* __restrict__ wq,
                         const float* __restrict__ wsc, const float* __restrict__ bias, int N,
                         int K, float alpha, float limit, int units, int upw, int held,
                         int32_t* __restrict__ ids, float* __restrict__ w,
                         uint16_t* __restrict__ h) {
  extern __shared__ __attribute__((aligned(16))) uint8_t rowsq[];   // quantized rows
  constexpr int kWaves = kI8DecThreads / kWave;
  __shared__ int sid[kI8DecMaxR], lists[kWaves][MOE_DECODE_MAX_T];
  __shared__ float sx[MOE_DECODE_MAX_T];
  __shared__ uint32_t bits[MOE_MAX_E / 32];
  __shared__ i32x4_t red[2][kWaves][kWave];
  const int tid = (int)threadIdx.x, lane = tid & 63, col = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int R = T * k;

  if (blockIdx.x == 0) {   // the routing, for the caller and for launch 2
    for (int t = wave; t < T; t += kWaves) {
      int my_id;
      float my_v;
      wave_topk(logits + (size_t)t * E, E, k, my_id, my_v);
      write_topk(my_id, my_v, k, ids + t * k, w + t * k);
    }
    return;
  }
  const int item = (int)blockIdx.x - 1;
  const int groups = (units + upw - 1) / upw, j = item / groups;
  const int ubase = (item - j * groups) * upw, uend = min(ubase + upw, units);
  const int KP = i8_pitch(K), LP = i8_lds_pitch(KP), C = i8_chunks(K);

  // 1. routing
  if (tid < MOE_MAX_E / 32) bits[tid] = 0u;
  lds_barrier();
  if (E <= kWave) {
    route_tokens<1>(logits, T, E, k, sid, bits);
  } else if (E <= 2 * kWave) {
    route_tokens<2>(logits, T, E, k, sid, bits);
  } else {
    for (int t = wave; t < T; t += kWaves) {
      int my_id;
      float my_v;
      wave_topk(logits + (size_t)t * E, E, k, my_id, my_v);
      if (lane < k) {
        my_id = min(max(my_id, 0), E - 1);
        sid[t * k + lane] = my_id;
        atomicOr(&bits[my_id >> 5], 1u << (my_id & 31));
      }
    }
  }
  lds_barrier();
  int* const list = lists[wave];   // a copy per wavefront: no barrier
  const I8Picked picked(bits);
  if (j >= picked.total) return;   // fewer experts were picked than there could have been
  const int e = picked.nth(j);
  int cnt = rows_of_expert(sid, R, e, list);
  // the list is written and read by the lanes of one wavefront, whose LDS operations complete in
  // order: only the compiler has to keep them so
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  cnt = __builtin_amdgcn_readfirstlane(cnt);

  // 2. rows of x quantized into LDS. Loads return in the order of their issue: the weights go out
  // behind the last row, before its codes are formed
  const int NT = i8_tiles(N, 1), HT = i8_half_tiles(N, 1);
  const int part = wave & 1, half = (wave >> 1) ? HT : 0;
  const int cb = C * part / 2, len = C * (part + 1) / 2 - cb;
  const uint32_t step = (uint32_t)NT * kI8TileBytes;
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(wq + (int64_t)e * C * step, (uint32_t)C * step);
  auto run = [&](int unit, int c0) {   // the chunks of a unit's tile from c0 on
    return I8Run{rw, ((uint32_t)(cb + c0) * NT + half + unit) * kI8TileBytes, step,
                 unit < uend ? len - c0 : 0};
  };
  I8Ring<kI8UpRing> ring;
  I8Row<kI8DecVec> xr;
  if (!held) {
    for (int m = wave; m < cnt; m += kWaves) {
      const float s = i8_row_to_lds<MOE_BF16>(x, (int64_t)(list[m] / k) * K, K, rowsq, m, LP, KP);
      if (lane == 0) sx[m] = s;
    }
    ring.fill(run(ubase, 0));
  } else {
    // a row per wavefront; of a single row every wavefront takes a share of the codes
    const int parts = cnt == 1 ? kWaves : 1, share = cnt == 1 ? wave : 0;
    for (int m = cnt == 1 ? 0 : wave;; m += kWaves) {
      if (m < cnt) xr.load<TAIL>(x + (int64_t)(list[m] / k) * K, K);
      if (m + kWaves >= cnt) ring.fill(run(ubase, 0));
      if (m < cnt) {
        const I8Quant z(xr.largest());
        xr.store_codes(z, rowsq, m, LP, KP, share, parts);
        if (lane == 0) sx[m] = z.s;
      }
      if (m + kWaves >= cnt) break;
    }
  }
  lds_barrier();

  // 3. products of the workgroup's units, one after another
  const int F = N >> 1, jj = tid & 15, m = tid >> 4;
  const int mb = min(col, cnt - 1);   // columns past the rows repeat the last row
  const uint8_t* bp = rowsq + mb * LP;
  for (int unit = ubase; unit < uend; ++unit) {
    const int n = unit * 16 + jj;
    const int64_t cg = (int64_t)e * N + min(n, F - 1);
    const float sg = wsc[cg], su = wsc[cg + F];
    const float bg = bias ? bias[cg] : 0.0f, bu = bias ? bias[cg + F] : 0.0f;
    i32x4_t acc = {0, 0, 0, 0}, acc1 = {0, 0, 0, 0};
    int c0 = 0;
    do {
      const int cn = c0 + kI8UpRing;
      ring.take(bp, mb, cb + c0, C - 1, cn < len ? run(unit, cn) : run(unit + 1, 0), acc, acc1);
      c0 = cn;
    } while (c0 < len);
    i32x4_t (*const rd)[kWave] = red[(unit - ubase) & 1];   // two in turn: one barrier per unit
    rd[wave][lane] = acc + acc1;
    lds_barrier();
    if (m < cnt && n < F) {
      const int from = (jj >> 2) * 16 + m, i = jj & 3;
      const float sa = sx[m];
      const float gate = i8_scaled(rd[0][from][i] + rd[1][from][i], sa, sg, bg);
      const float up = i8_scaled(rd[2][from][i] + rd[3][from][i], sa, su, bu);
      h[(int64_t)list[m] * F + n] = bf16_one(i8_swiglu(gate, up, alpha, limit));
    }
  }
}

// Launch 2 of several tokens. ROWS: the h rows come quantized (hq, hs) and go to the MFMA straight
// from memory; otherwise (few rows) every workgroup quantizes all of them into LDS first.
template <bool ROWS, bool TAIL>
__global__ void __launch_bounds__(kI8DownThreads)
i8_decode_down_kernel(const uint16_t* __restrict__ h, const int8_t* __restrict__ hq,
                      const float* __restrict__ hs, int T, int E, int k,
                      const int32_t* __restrict__ ids, const float* __restrict__ w,
                      const int8_t* __restrict__ wq, const float* __restrict__ wsc,
                      const float* __restrict__ bias, int D, int F, int held,
                      float* __restrict__ d, void* __restrict__ y, int y_dt) {
  extern __shared__ __attribute__((aligned(16))) uint8_t rowsq[];   // R quantized rows, or none
  constexpr int kWaves = kI8DownThreads / kWave;
  constexpr int NR = ROWS ? kI8RowsRing : kI8DownRing;
  constexpr int kSums = kI8DecMaxR * kI8TileRows / kI8DownThreads;   // sums of a thread
  __shared__ int sid[kI8DecMaxR], lists[kWaves][MOE_DECODE_MAX_T];
  __shared__ uint32_t bits[MOE_MAX_E / 32];
  __shared__ float sw[kI8DecMaxR], sh[kI8DecMaxR];   // routing weight and scale of each h row
  __shared__ int acc_s[kI8DecMaxR][kI8TileRows];     // sums of each routed row, then its d (f32)
  const int tid = (int)threadIdx.x, lane = tid & 63, col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int R = T * k, unit = (int)blockIdx.x;
  const int FP = i8_pitch(F), LP = i8_lds_pitch(FP), C = i8_chunks(F), NT = i8_tiles(D, 0);

  // the picked experts
  int id = 0;
  if (tid < R) {
    id = min(max(ids[tid], 0), E - 1);
    sw[tid] = w[tid];
    sid[tid] = id;
    if (ROWS) sh[tid] = hs[tid];
  }
  if (tid < MOE_MAX_E / 32) bits[tid] = 0u;
  for (int i = tid; i < R * kI8TileRows; i += kI8DownThreads) (&acc_s[0][0])[i] = 0;
  lds_barrier();
  if (tid < R) atomicOr(&bits[id >> 5], 1u << (id & 31));
  lds_barrier();
  const I8Picked picked(bits);

  // an item is one picked expert's tile over a segment of K: its chunks, the number of its rows
  // and the lane's row (columns past the rows repeat the last one). Past the last item nothing is
  // read
  const int segs = (C + NR - 1) / NR, items = picked.total * segs;
  const uint32_t step = (uint32_t)NT * kI8TileBytes;
  int* const list = lists[wave];
  auto find = [&](int it, int& rho, int& cnt) {
    if (it >= items) {
      rho = cnt = 0;
      return I8Run{make_rsrc(wq, 0u), 0u, step, 0};
    }
    const int jx = it / segs, seg = it - jx * segs;
    const int cb = C * seg / segs, ce = C * (seg + 1) / segs;
    const int e = picked.nth(jx);
    cnt = __builtin_amdgcn_readfirstlane(rows_of_expert(sid, R, e, list));
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // written and read by one wavefront
    rho = list[min(col, cnt - 1)];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    return I8Run{make_rsrc(wq + (int64_t)e * C * step, (uint32_t)C * step),
                 ((uint32_t)cb * NT + unit) * kI8TileBytes, step, ce - cb};
  };
  int rho, cnt;
  const I8Run first = find(wave, rho, cnt);
  I8Ring<NR> ring;
  // ROWS: the lane's pieces of its row over the item's chunks
  u32x4_t bv[ROWS ? NR : 1];
  const __amdgpu_buffer_rsrc_t rh = make_rsrc(hq, ROWS ? (uint32_t)(R * FP) : 0u);
  if constexpr (ROWS) {
    ring.fill(first);
    const int c0 = C * (wave % segs) / segs;
#pragma unroll
    for (int i = 0; i < NR; ++i)
      bv[i] = buf_load16(rh, (uint32_t)(rho * FP + g * 16), (uint32_t)min(c0 + i, C - 1) * kI8Chunk);
  } else {
    if (held) {   // loads return in the order of their issue: the weights go behind the last row
      I8Row<kI8DecVec> hr;
      for (int m = wave;; m += kWaves) {
        const bool last = m + kWaves >= R;
        if (m < R) hr.load<TAIL>(h + (int64_t)m * F, F);
        if (last) ring.fill(first);
        if (m < R) {
          const I8Quant z(hr.largest());
          hr.store_codes(z, rowsq, m, LP, FP, 0, 1);
          if (lane == 0) sh[m] = z.s;
        }
        if (last) break;
      }
    } else {
      for (int m = wave; m < R; m += kWaves) {
        const float s = i8_row_to_lds<MOE_BF16>(h, (int64_t)m * F, F, rowsq, m, LP, FP);
        if (lane == 0) sh[m] = s;
      }
      ring.fill(first);
    }
    lds_barrier();
  }

  // scales and biases of the sums this thread turns into d: channel tid % 16 of rows tid / 16 + 32 i
  const int jj = tid & 15, n = unit * 16 + jj;
  float dsc[kSums], dbi[kSums];
#pragma unroll
  for (int i = 0; i < kSums; ++i) {
    const int r = (tid >> 4) + i * (kI8DownThreads / kI8TileRows);
    dsc[i] = 1.0f;
    dbi[i] = 0.0f;
    if (r < R && n < D) {
      const int64_t cg = (int64_t)sid[r] * D + n;
      dsc[i] = wsc[cg];
      if (bias) dbi[i] = bias[cg];
    }
  }

  for (int it = wave; it < items; it += kWaves) {
    int rho_next, cnt_next;
    const I8Run next = find(it + kWaves, rho_next, cnt_next);
    i32x4_t acc = {0, 0, 0, 0}, acc1 = {0, 0, 0, 0};
    if constexpr (ROWS) {
      const uint32_t bo = (uint32_t)(rho_next * FP + g * 16);
      const int cn = C * ((it + kWaves) % segs) / segs;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        i32x4_t a, b;
        __builtin_memcpy(&a, &ring.v[i], sizeof(a));
        __builtin_memcpy(&b, &bv[i], sizeof(b));
        if (i & 1)
          acc1 = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, acc1, 0, 0, 0);
        else
          acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, acc, 0, 0, 0);
        ring.load(i, next);
        bv[i] = buf_load16(rh, bo, (uint32_t)min(cn + i, C - 1) * kI8Chunk);
      }
    } else {
      ring.take(rowsq + rho * LP, rho, C * (it % segs) / segs, C - 1, next, acc, acc1);
    }
    acc += acc1;
    if (col < cnt) {
#pragma unroll
      for (int i = 0; i < 4; ++i) atomicAdd(&acc_s[rho][4 * g + i], acc[i]);   // exact integers
    }
    rho = rho_next;
    cnt = cnt_next;
  }
  lds_barrier();

  // d of every routed row, summed in slot order
#pragma unroll
  for (int i = 0; i < kSums; ++i) {
    const int r = (tid >> 4) + i * (kI8DownThreads / kI8TileRows);
    if (r >= R) break;
    const float dv = i8_scaled(acc_s[r][jj], sh[r], dsc[i], dbi[i]);
    if (d && n < D) d[(int64_t)r * D + n] = dv;
    acc_s[r][jj] = __float_as_int(dv);
  }
  lds_barrier();
  if (tid < T * kI8TileRows && n < D) {
    const int t = tid >> 4;
    float yv = 0.0f;
    for (int s = 0; s < k; ++s) yv = fmaf(sw[t * k + s], __int_as_float(acc_s[t * k + s][jj]), yv);
    store_elem(y, (int64_t)t * D + n, yv, y_dt);
  }
}

}  // namespace moe

extern "C" int i8_moe_decode(const float* logits, const uint16_t* x, int64_t T, int E, int k,
                             const i8_experts* w_gu, const i8_experts* w_dn, float alpha,
                             float limit, int32_t* ids, float* w, uint16_t* h, int8_t* q_ws,
                             float* s_ws, float* d, void* y, int y_dtype, void* stream) {
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
      (((uintptr_t)w_gu->bias) & 3) || (((uintptr_t)w_dn->bias) & 3) || (((uintptr_t)ids) & 3) ||
      (((uintptr_t)w) & 3) || (((uintptr_t)logits) & 3) || (((uintptr_t)d) & 3) ||
      (((uintptr_t)y) & (y_dtype == MOE_F32 ? 3 : 1)))
    return MOE_EALIGN;
  // launch 1 holds up to T quantized rows of x in LDS, launch 2 those of h where they are few
  const int R = (int)T * k, units = moe::i8_half_tiles(N, 1);
  const int64_t xrow = moe::i8_lds_pitch(moe::i8_pitch(D)), hrow = moe::i8_lds_pitch(moe::i8_pitch(F));
  if (T * xrow > (int64_t)moe::kI8DecMaxLds ||
      (int64_t)units * 2 * moe::i8_chunks(D) * moe::kI8TileBytes >= (int64_t)1 << 31 ||
      (int64_t)moe::i8_tiles(D, 0) * moe::i8_chunks(F) * moe::kI8TileBytes >= (int64_t)1 << 31)
    return MOE_ESHAPE;
  const bool own_rows = R <= moe::kI8LdsRows && R * hrow <= (int64_t)moe::kI8DecMaxLds;
  if (!own_rows) {
    if (!q_ws || !s_ws) return MOE_EINVAL;
    if ((((uintptr_t)q_ws) & 15) || (((uintptr_t)s_ws) & 3)) return MOE_EALIGN;
  }
  const size_t lds1 = (size_t)(T * xrow), lds2 = own_rows ? (size_t)(R * hrow) : 0;
  // rows that fit in registers, and rows that end inside a vector of 8
  const int held1 = D <= moe::kI8DecVec * 8 * moe::kWave;
  const int held2 = F <= moe::kI8DecVec * 8 * moe::kWave;
  const bool tail1 = D % 8 != 0, tail2 = F % 8 != 0;
  auto gate_up = tail1 ? moe::i8_decode_gate_up_kernel<true> : moe::i8_decode_gate_up_kernel<false>;
  auto down = !own_rows ? moe::i8_decode_down_kernel<true, false>
              : tail2   ? moe::i8_decode_down_kernel<false, true>
                        : moe::i8_decode_down_kernel<false, false>;
  static bool lds_attr_set[moe::kMaxDevices] = {};   // > 64 KB of LDS: opt in once per device
  const int dslot = moe::device_slot();
  if (dslot < 0 || !lds_attr_set[dslot]) {
    for (const void* f : {reinterpret_cast<const void*>(&moe::i8_decode_gate_up_kernel<true>),
                          reinterpret_cast<const void*>(&moe::i8_decode_gate_up_kernel<false>),
                          reinterpret_cast<const void*>(&moe::i8_decode_down_kernel<false, true>),
                          reinterpret_cast<const void*>(&moe::i8_decode_down_kernel<false, false>)})
      if (hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize,
                              (int)moe::kI8DecMaxLds) != hipSuccess)
        return MOE_ELAUNCH;
    if (dslot >= 0) lds_attr_set[dslot] = true;
  }
  const hipStream_t st = (hipStream_t)stream;
  if (T == 1 && held1 && held2) {
    const int Cd = moe::i8_chunks(D), Cf = moe::i8_chunks(F);
    // launch 2: 16 wavefronts, or as many as there are slots and chunks for
    int parts = 16 / k;
    while (parts > 1 && Cf < 4 * parts) --parts;
    moe::launch(tail1 ? moe::i8_one_gate_up_kernel<true> : moe::i8_one_gate_up_kernel<false>,
                dim3((unsigned)(1 + k * units)), dim3(moe::kI8DecThreads),
                (size_t)(4 * ((Cd + 1) / 2) * moe::kI8Chunk), st, logits, x, E, k, w_gu->q, w_gu->s,
                w_gu->bias, N, D, alpha, limit, units, ids, w, h);
    if (hipGetLastError() != hipSuccess) return MOE_ELAUNCH;
    moe::launch(tail2 ? moe::i8_one_down_kernel<true> : moe::i8_one_down_kernel<false>,
                dim3((unsigned)moe::i8_tiles(D, 0)), dim3((unsigned)(64 * k * parts)),
                (size_t)(k * parts * ((Cf + parts - 1) / parts) * moe::kI8Chunk), st, h, E, k, parts, ids,
                w, w_dn->q, w_dn->s, w_dn->bias, D, F, d, y, y_dtype);
    return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ELAUNCH;
  }
  const int picks = R < E ? R : E;
  // launch 1: units per workgroup. Routing and the rows' quantization are paid once per workgroup,
  // so it takes as many units as it needs for the expected number of picked experts to fill the
  // resident workgroups once (3 a CU, fewer where LDS holds fewer), and an odd number: with 4 or 8
  // the workgroups start on strides of a power of two and meet on the same memory channels (16
  // tokens, 32 experts: 5 units 70 us, 4 83 us, 8 93 us, 1 106 us; 8 tokens: 51, 60, 57, 55 us)
  double none = 1.0;   // an expert's chance to be picked by no token
  for (int t = 0; t < T; ++t) none *= 1.0 - (double)k / E;
  const double live = E * (1.0 - none);
  const int fit = (int)((160 * 1024) / (lds1 + 12 * 1024));
  const double slots = 256.0 * (fit < 3 ? fit : 3);
  int upw = 1;
  while (upw < units && live * ((units + upw - 1) / upw) > slots) upw += 2;
  const int groups = (units + upw - 1) / upw;
  moe::launch(gate_up, dim3((unsigned)(1 + picks * groups)),
              dim3(moe::kI8DecThreads), lds1, st, logits, x, (int)T, E, k, w_gu->q, w_gu->s,
              w_gu->bias, N, D, alpha, limit, units, upw, held1, ids, w, h);
  if (hipGetLastError() != hipSuccess) return MOE_ELAUNCH;
  const dim3 grid2((unsigned)moe::i8_tiles(D, 0));
  if (own_rows) {
    moe::launch(down, grid2, dim3(moe::kI8DownThreads), lds2, st, h,
                (const int8_t*)nullptr, (const float*)nullptr, (int)T, E, k, ids, w, w_dn->q, w_dn->s,
                w_dn->bias, D, F, held2, d, y, y_dtype);
  } else {
    // every workgroup of launch 2 would quantize every row, some 2 us for 8 of them: more than 16
    // rows are quantized once, by a launch of its own
    const int qs = i8_quantize(h, MOE_BF16, F, nullptr, R, F, q_ws, s_ws, stream);
    if (qs != MOE_OK) return qs;
    moe::launch(down, grid2, dim3(moe::kI8DownThreads), 0, st, h,
                (const int8_t*)q_ws, (const float*)s_ws, (int)T, E, k, ids, w, w_dn->q, w_dn->s,
                w_dn->bias, D, F, held2, d, y, y_dtype);
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ELAUNCH;
}
