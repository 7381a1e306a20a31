// train_api.cu - C ABI entry points of the training pass and of the dense product with a fused
// epilogue (declared in include/moe.h): argument checks and the order of the launches.
#include <initializer_list>

#include "api_checks.h"
#include "kernels.h"

using namespace moe;

namespace {

bool all_aligned16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned16(p)) return false;
  return true;
}

moe_status check_grad_flags(int32_t flags) {
  if (flags & ~(MOE_GRAD_F32 | MOE_GRAD_ACCUMULATE)) return MOE_ERR_INVALID_ARG;
  if ((flags & MOE_GRAD_ACCUMULATE) && !(flags & MOE_GRAD_F32)) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// Row and feature numbers are rounded up to whole tiles in 32 bits.
constexpr long long kMaxExtent = 0x7fffffffLL - 1024;

moe_status train_checks(const moe_dims* d) {
  MOE_TRY(check_dims(d));
  if (d->T * static_cast<long long>(d->K) > kMaxExtent || d->H > kMaxExtent || d->F > kMaxExtent)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  return device_ok() ? MOE_OK : MOE_ERR_NO_DEVICE;
}

moe_status check_dense_shape(int64_t M, int32_t N, int32_t Kd) {
  if (M < 0 || N < 8 || Kd < 8) return MOE_ERR_INVALID_ARG;
  if (N % 8 != 0 || Kd % 8 != 0 || M > kMaxExtent || N > kMaxExtent || Kd > kMaxExtent) return MOE_ERR_UNSUPPORTED_SHAPE;
  return MOE_OK;
}

moe_status clear(void* p, size_t bytes, void* stream) {
  return p ? cuda_status(cudaMemsetAsync(p, 0, bytes, as_stream(stream))) : MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_grouped_gate_up_train(const void* xp, const int32_t* offsets, const void* w_gate, const void* w_up,
                                     const moe_dims* d, float* g, float* u, void* h, void* ws, size_t ws_bytes,
                                     void* stream) {
  MOE_TRY(train_checks(d));
  MOE_TRY(check_ws_header(ws, ws_bytes));
  if (d->T == 0) return MOE_OK;
  if (!xp || !offsets || !w_gate || !w_up || !g || !u || !h) return MOE_ERR_INVALID_ARG;
  if (!all_aligned16({xp, w_gate, w_up, g, u, h})) return MOE_ERR_INVALID_ARG;
  const long long TK = d->T * static_cast<long long>(d->K);
  if (grouped_small_fits(TK, d->E, d->F, 256))
    return cuda_status(small_gate_up_train(xp, offsets, w_gate, w_up, d->E, TK, d->H, d->F, g, u, h, ws_status(ws),
                                           as_stream(stream)));
  return cuda_status(gemm_gate_up_train(xp, offsets, w_gate, w_up, d->E, TK, d->H, d->F, g, u, h, ws_status(ws),
                                        ws_sched(ws, kSchedGateUp), as_stream(stream)));
}

moe_status moe_grouped_ffn_backward(const void* xp, const float* g, const float* u, const void* h, const void* dy,
                                    const int32_t* offsets, const void* w_gate, const void* w_up, const void* w_down,
                                    const moe_dims* d, void* dg, void* du, void* dxp, void* dw_gate, void* dw_up,
                                    void* dw_down, int32_t grad_flags, void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(train_checks(d));
  MOE_TRY(check_ws_header(ws, ws_bytes));
  MOE_TRY(check_grad_flags(grad_flags));
  if (!dw_gate != !dw_up) return MOE_ERR_INVALID_ARG;
  const int f32 = (grad_flags & MOE_GRAD_F32) != 0, acc = (grad_flags & MOE_GRAD_ACCUMULATE) != 0;
  if (d->T == 0) {  // no rows: the weight gradients are zero
    if (acc) return MOE_OK;
    const size_t bytes = static_cast<size_t>(d->E) * d->F * d->H * (f32 ? 4 : 2);
    MOE_TRY(clear(dw_gate, bytes, stream));
    MOE_TRY(clear(dw_up, bytes, stream));
    return clear(dw_down, bytes, stream);
  }
  const bool need_g = dxp || dw_gate;  // dg and du are wanted
  if (!offsets || !dy) return MOE_ERR_INVALID_ARG;
  if (need_g && (!g || !u || !dg || !du || !w_down)) return MOE_ERR_INVALID_ARG;
  if ((dxp && (!w_gate || !w_up)) || (dw_gate && !xp) || (dw_down && !h)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned16({xp, g, u, h, dy, w_gate, w_up, w_down, dg, du, dxp, dw_gate, dw_up, dw_down}))
    return MOE_ERR_INVALID_ARG;
  const long long TK = d->T * static_cast<long long>(d->K);
  int* status = ws_status(ws);
  cudaStream_t s = as_stream(stream);
  // dWd does not read dg and du, and dWg and dWu only what was complete before the kernel before them:
  // their many small tiles start while the large tiles of dg and du, and of dxp, run out (late_wait),
  // on tile schedules of their own.
  // Beside a large product the small tiles of a weight gradient only take SMs from it (2 x 2048 rows, 1024
  // x 1024: 72 us a call, 84 with them), so they follow a small one.
  const bool small_g = grouped_small_fits(TK, d->E, d->F, 512), small_x = grouped_small_fits(TK, d->E, d->H, 512);
  if (need_g && small_g)
    MOE_CUDA(small_down_bwd(dy, g, u, offsets, w_down, d->E, TK, d->H, d->F, dg, du, status, s));
  else if (need_g)
    MOE_CUDA(gemm_down_bwd(dy, g, u, offsets, w_down, d->E, TK, d->H, d->F, dg, du, status,
                           ws_sched(ws, kSchedDown), s));
  if (dw_down && (!need_g || small_g) && grad_small_fits(d->E, d->H, d->F, 512))
    MOE_CUDA(small_grad(dy, nullptr, h, offsets, d->E, TK, d->H, d->F, dw_down, nullptr, f32, acc, need_g, status, s));
  else if (dw_down)
    MOE_CUDA(gemm_grad_down(dy, h, offsets, d->E, TK, d->H, d->F, dw_down, f32, acc, need_g, status,
                            ws_sched(ws, kSchedDense), s));
  if (dxp && small_x)
    MOE_CUDA(small_rows_bwd(dg, du, offsets, w_gate, w_up, d->E, TK, d->H, d->F, dxp, status, s));
  else if (dxp)
    MOE_CUDA(gemm_rows_bwd(dg, du, offsets, w_gate, w_up, d->E, TK, d->H, d->F, dxp, status,
                           ws_sched(ws, kSchedGateUp), s));
  if (dw_gate && (!dxp || small_x) && grad_small_fits(d->E, d->F, d->H, 256))
    MOE_CUDA(small_grad(dg, du, xp, offsets, d->E, TK, d->F, d->H, dw_gate, dw_up, f32, acc, dxp != nullptr, status, s));
  else if (dw_gate)
    MOE_CUDA(gemm_grad_gate_up(dg, du, xp, offsets, d->E, TK, d->H, d->F, dw_gate, dw_up, f32, acc, dxp != nullptr,
                               status, ws_sched(ws, kSchedGating), s));
  return MOE_OK;
}

moe_status moe_combine_backward(const void* dout, const void* y, const int32_t* row_of_assign, const float* topk_w,
                                const moe_dims* d, void* dy, float* dw, void* stream) {
  MOE_TRY(common_checks(d));
  if (d->T == 0) return MOE_OK;
  if (!dout || !row_of_assign || !topk_w || (dw && !y)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned16({dout, y, dy})) return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_combine_bwd(dout, y, row_of_assign, topk_w, d->T, d->H, d->K, dy, dw, as_stream(stream)));
}

size_t moe_dense_workspace_bytes(int64_t M, int32_t N, int32_t Kd) {
  return check_dense_shape(M, N, Kd) == MOE_OK ? kWsHeader : 0;
}

moe_status moe_dense_epilogue(const void* a, const void* w, const float* bias, const void* residual, int32_t act,
                              int64_t M, int32_t N, int32_t Kd, void* out, float* pre, void* ws, size_t ws_bytes,
                              void* stream) {
  MOE_TRY(check_dense_shape(M, N, Kd));
  if (act < MOE_ACT_NONE || act > MOE_ACT_GELU_TANH) return MOE_ERR_INVALID_ARG;
  if (!device_ok()) return MOE_ERR_NO_DEVICE;
  MOE_TRY(check_ws_header(ws, ws_bytes));
  if (M == 0) return MOE_OK;
  if (!a || !w || !out || !all_aligned16({a, w, residual, out, pre})) return MOE_ERR_INVALID_ARG;
  if (dense_small_fits(M, N))
    return cuda_status(dense_small(a, w, 0, bias, residual, act, M, N, Kd, out, pre, ws_status(ws), as_stream(stream)));
  return cuda_status(gemm_dense_epilogue(a, w, bias, residual, act, M, N, Kd, out, pre, ws_status(ws),
                                         ws_sched(ws, kSchedDense), as_stream(stream)));
}

moe_status moe_dense_backward(const void* dout, const void* a, const void* w, const float* pre, int32_t act, int64_t M,
                              int32_t N, int32_t Kd, void* dpre, void* da, void* dw, float* dbias, int32_t grad_flags,
                              void* ws, size_t ws_bytes, void* stream) {
  MOE_TRY(check_dense_shape(M, N, Kd));
  if (act < MOE_ACT_NONE || act > MOE_ACT_GELU_TANH) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_grad_flags(grad_flags));
  if (!device_ok()) return MOE_ERR_NO_DEVICE;
  MOE_TRY(check_ws_header(ws, ws_bytes));
  const int f32 = (grad_flags & MOE_GRAD_F32) != 0, acc = (grad_flags & MOE_GRAD_ACCUMULATE) != 0;
  if (M == 0) {
    if (acc) return MOE_OK;
    MOE_TRY(clear(dw, static_cast<size_t>(N) * Kd * (f32 ? 4 : 2), stream));
    return clear(dbias, static_cast<size_t>(N) * 4, stream);
  }
  const bool plain = act == MOE_ACT_NONE;  // dpre is dout
  if (!dout || (!plain && (!pre || ((da || dw) && !dpre))) || (da && !w) || (dw && !a)) return MOE_ERR_INVALID_ARG;
  if (!all_aligned16({dout, a, w, pre, dpre, da, dw})) return MOE_ERR_INVALID_ARG;
  cudaStream_t s = as_stream(stream);
  int* status = ws_status(ws);
  void* rounded = !plain && (da || dw) ? dpre : nullptr;
  MOE_CUDA(launch_act_bwd(dout, pre, act, M, N, rounded, dbias, acc, s));
  const void* dp = plain ? dout : dpre;
  // dw does not read da: after a small da, which leaves room on the SMs, it starts at once (late_wait: 333 x
  // 776 x 520 with GELU 14.8 -> 11.3 us, 300 x 4104 x 2056 42.3 -> 40.8); beside a large one it would take
  // SMs from it (4096 x 2048 x 7168: 210 -> 261 us).
  const bool small_da = da && dense_small_fits(M, Kd);
  if (small_da)
    MOE_CUDA(dense_small(dp, w, 1, nullptr, nullptr, MOE_ACT_NONE, M, Kd, N, da, nullptr, status, s));
  else if (da)
    MOE_CUDA(gemm_rows_bwd(dp, nullptr, nullptr, w, nullptr, 1, M, Kd, N, da, status, ws_sched(ws, kSchedDense), s));
  if (dw && grad_small_fits(1, N, Kd, 512))
    MOE_CUDA(small_grad(dp, nullptr, a, nullptr, 1, M, N, Kd, dw, nullptr, f32, acc, small_da, status, s));
  else if (dw)
    MOE_CUDA(gemm_grad_down(dp, a, nullptr, 1, M, N, Kd, dw, f32, acc, small_da, status, ws_sched(ws, kSchedDense), s));
  return MOE_OK;
}

}  // extern "C"
