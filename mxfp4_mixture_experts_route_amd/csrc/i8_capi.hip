// C ABI entry points of the 8-bit integer projections: host-side argument checks, then the
// launch. Every check runs before anything is enqueued, the product's own limits included (i8_linear
// quantizes behind them); a call that is refused has enqueued nothing.
#include "i8.hpp"

int moe_launch_i8_gemm(const moe::I8Plain* plain, const int8_t* a, const float* as,
                       const int32_t* a_row, int64_t a_rows, const i8_experts* w,
                       const int32_t* counts, const int32_t* basep, int64_t rows, int64_t mpad,
                       int act, float alpha, float limit, void* out, int out_dt, int64_t ld_out,
                       hipStream_t stream);

bool moe_i8_few(int64_t rows, const i8_experts* w);
int moe_launch_i8_few(const void* x, int x_dt, int64_t ld, int rows, const i8_experts* w, void* out,
                      int out_dt, int64_t ld_out, hipStream_t stream);

namespace {

bool known_dtype(int dt) { return dt == MOE_BF16 || dt == MOE_F16 || dt == MOE_F32; }
int elem_size(int dt) { return dt == MOE_F32 ? 4 : 2; }

int check_stack(const i8_experts* w) {
  if (!w || !w->q || !w->s || w->E < 1 || w->N < 1 || w->K < 1) return MOE_EINVAL;
  if (w->glu != 0 && w->glu != 1) return MOE_EINVAL;
  if (w->E > MOE_MAX_E || w->K > MOE_I8_MAX_K || (w->glu && (w->N & 1))) return MOE_ESHAPE;
  // one expert's packed weights are addressed with 31 bits
  if ((int64_t)moe::i8_tiles(w->N, w->glu) * moe::i8_chunks(w->K) * moe::kI8TileBytes >= (int64_t)1 << 31)
    return MOE_ESHAPE;
  return MOE_OK;
}

int check_align(const void* aq, const float* as, const i8_experts* w, const void* out, int dt) {
  if ((((uintptr_t)aq) & 15) || (((uintptr_t)w->q) & 15) || (((uintptr_t)as) & 3) ||
      (((uintptr_t)w->s) & 3) || (((uintptr_t)w->bias) & 3) ||
      (((uintptr_t)out) & (elem_size(dt) - 1)))
    return MOE_EALIGN;
  return MOE_OK;
}

}  // namespace

extern "C" int i8_gemm(const int8_t* aq, const float* as, int64_t rows, const i8_experts* w,
                       void* out, int out_dtype, int64_t ld_out, void* stream) {
  if (!aq || !as || !out || rows < 1 || !known_dtype(out_dtype)) return MOE_EINVAL;
  int st = check_stack(w);
  if (st != MOE_OK) return st;
  if (w->E != 1 || ld_out < w->N || rows > 0x7FFFFFFFLL) return MOE_ESHAPE;
  st = check_align(aq, as, w, out, out_dtype);
  if (st != MOE_OK) return st;
  return moe_launch_i8_gemm(nullptr, aq, as, nullptr, rows, w, nullptr, nullptr, rows, rows,
                            MOE_ACT_NONE, 0.0f, 0.0f, out, out_dtype, ld_out, (hipStream_t)stream);
}

extern "C" int i8_moe_gemm(const int8_t* aq, const float* as, const int32_t* a_row,
                           int64_t a_rows, const i8_experts* w, const int32_t* counts,
                           const int32_t* basep, int tile_m, int64_t mpad_max, int act,
                           float alpha, float limit, void* out, void* stream) {
  if (!aq || !as || !counts || !basep || !out || a_rows < 1 || mpad_max < 1) return MOE_EINVAL;
  if (act != MOE_ACT_NONE && act != MOE_ACT_SWIGLU_OAI) return MOE_EINVAL;
  int st = check_stack(w);
  if (st != MOE_OK) return st;
  if (act == MOE_ACT_SWIGLU_OAI && !w->glu) return MOE_ESHAPE;
  if (tile_m < 1 || tile_m > MOE_MAX_TILE_M || mpad_max > 0x7FFFFFFFLL || a_rows > 0x7FFFFFFFLL)
    return MOE_ESHAPE;
  if (!a_row && a_rows < mpad_max) return MOE_ESHAPE;
  if (a_rows * moe::i8_pitch(w->K) >= (int64_t)1 << 32) return MOE_ESHAPE;   // rows within 4 GB
  const bool glu = act == MOE_ACT_SWIGLU_OAI;
  const int out_dt = glu ? MOE_BF16 : MOE_F32;
  st = check_align(aq, as, w, out, out_dt);
  if (st != MOE_OK) return st;
  if ((((uintptr_t)a_row) & 3) || (((uintptr_t)counts) & 3) || (((uintptr_t)basep) & 3)) return MOE_EALIGN;
  return moe_launch_i8_gemm(nullptr, aq, as, a_row, a_rows, w, counts, basep, 0, mpad_max, act,
                            alpha, limit, out, out_dt, glu ? w->N / 2 : w->N, (hipStream_t)stream);
}

extern "C" int i8_linear(const void* x, int x_dtype, int64_t ld, int64_t rows,
                         const i8_experts* w, int8_t* q_ws, float* s_ws, void* out, int out_dtype,
                         int64_t ld_out, void* stream) {
  if (!x || !q_ws || !s_ws || !out || rows < 1 || !known_dtype(x_dtype) ||
      !known_dtype(out_dtype))
    return MOE_EINVAL;
  int st = check_stack(w);
  if (st != MOE_OK) return st;
  if (w->E != 1 || ld_out < w->N || ld < w->K || rows > 0x7FFFFFFFLL) return MOE_ESHAPE;
  st = check_align(q_ws, s_ws, w, out, out_dtype);
  if (st != MOE_OK) return st;
  if (((uintptr_t)x) & (elem_size(x_dtype) - 1)) return MOE_EALIGN;
  if (moe_i8_few(rows, w))
    return moe_launch_i8_few(x, x_dtype, ld, (int)rows, w, out, out_dtype, ld_out,
                             (hipStream_t)stream);
  const moe::I8Plain plain{x, x_dtype, ld};
  return moe_launch_i8_gemm(&plain, q_ws, s_ws, nullptr, rows, w, nullptr, nullptr, rows, rows,
                            MOE_ACT_NONE, 0.0f, 0.0f, out, out_dtype, ld_out,
                            (hipStream_t)stream);
}
