// ttt_block_api.cpp -- C ABI entry points of the RMS norm, the 8-bit input
// projection, the short convolution and the selective state space scan
// (include/ttt.h): host checks (ttt_block_validate.cpp), then the gfx950
// kernels on the caller's stream.
#include "ttt.h"

#include <hip/hip_runtime.h>

#include "ttt_block.hpp"
#include "ttt_block_validate.hpp"

namespace {

ttt_status status_of(hipError_t e) { return e == hipSuccess ? TTT_OK : TTT_ERR_DEVICE; }
hipStream_t stream_of(void* s) { return static_cast<hipStream_t>(s); }
bool bf16_of(const ttt_params* p) { return p->io_dtype == TTT_BF16; }

}  // namespace

extern "C" {

ttt_status ttt_rms_norm_forward(int64_t rows, int32_t width, int32_t io_dtype, float eps,
                                const void* x, const void* residual, const float* weight,
                                void* y, void* res_out, void* hip_stream) {
  tttk::NormArgs a;
  const ttt_status st = tttv::rms_norm(rows, width, io_dtype, eps, x, residual, weight, y, false,
                                       nullptr, res_out, &a);
  if (st != TTT_OK) return st;
  return status_of(tttk::launch_norm(a, io_dtype == TTT_BF16, stream_of(hip_stream)));
}

ttt_status ttt_rms_norm_forward_f8(int64_t rows, int32_t width, int32_t io_dtype, float eps,
                                   const void* x, const void* residual, const float* weight,
                                   void* y8, float* scale, void* res_out, void* hip_stream) {
  tttk::NormArgs a;
  const ttt_status st = tttv::rms_norm(rows, width, io_dtype, eps, x, residual, weight, y8, true,
                                       scale, res_out, &a);
  if (st != TTT_OK) return st;
  return status_of(tttk::launch_norm(a, io_dtype == TTT_BF16, stream_of(hip_stream)));
}

uint64_t ttt_rms_norm_backward_workspace_bytes(int64_t rows, int32_t width) {
  return tttv::rms_norm_backward_workspace_bytes(rows, width);
}

ttt_status ttt_rms_norm_backward(int64_t rows, int32_t width, int32_t io_dtype, float eps,
                                 const void* r, const float* weight, const void* dy,
                                 const void* dr, void* dx, float* dweight, void* workspace,
                                 uint64_t workspace_bytes, void* hip_stream) {
  tttk::NormBackwardArgs a;
  const ttt_status st = tttv::rms_norm_backward(rows, width, io_dtype, eps, r, weight, dy, dr,
                                                dx, dweight, workspace, workspace_bytes, &a);
  if (st != TTT_OK) return st;
  return status_of(tttk::launch_norm_backward(a, io_dtype == TTT_BF16, stream_of(hip_stream)));
}

ttt_status ttt_input_projection_f8(const ttt_params* p, int32_t d_model, const void* x,
                                   const float* x_scale, const void* w_in,
                                   const float* w_scale, const float* b_eta, float eta_base,
                                   void* q, void* k, void* v, float* eta, void* hip_stream) {
  tttk::InputF8Args a;
  const ttt_status st = tttv::input_projection_f8(p, d_model, x, x_scale, w_in, w_scale, b_eta,
                                                  eta_base, q, k, v, eta, &a);
  if (st != TTT_OK) return st;
  return status_of(tttk::launch_input_f8(a, stream_of(hip_stream)));
}

ttt_status ttt_conv_forward(const ttt_params* p, int32_t taps, uint32_t flags, const void* x,
                            const float* w, const float* bias, const void* state0, void* y,
                            void* state_out, void* hip_stream) {
  tttk::ConvArgs a;
  const ttt_status st = tttv::conv_forward(p, taps, flags, x, w, bias, state0, y, state_out, &a);
  if (st != TTT_OK) return st;
  return status_of(tttk::launch_conv(a, bf16_of(p), stream_of(hip_stream)));
}

ttt_status ttt_conv_decode_step(const ttt_params* p, int32_t taps, uint32_t flags,
                                const void* x, const float* w, const float* bias, void* state,
                                void* y, void* hip_stream) {
  tttk::ConvArgs a;
  const ttt_status st = tttv::conv_decode(p, taps, flags, x, w, bias, state, y, &a);
  if (st != TTT_OK) return st;
  return status_of(tttk::launch_conv_decode(a, bf16_of(p), stream_of(hip_stream)));
}

uint64_t ttt_conv_backward_workspace_bytes(const ttt_params* p, int32_t taps) {
  return tttv::conv_backward_workspace_bytes(p, taps);
}

ttt_status ttt_conv_backward(const ttt_params* p, int32_t taps, uint32_t flags, const void* x,
                             const float* w, const float* bias, const void* state0,
                             const void* dy, const void* dstate, void* dx, float* dw,
                             float* dbias, void* dstate0, void* workspace,
                             uint64_t workspace_bytes, void* hip_stream) {
  tttk::ConvBackwardArgs a;
  const ttt_status st =
      tttv::conv_backward(p, taps, flags, x, w, bias, state0, dy, dstate, dx, dw, dbias, dstate0,
                          workspace, workspace_bytes, &a);
  if (st != TTT_OK) return st;
  return status_of(tttk::launch_conv_backward(a, bf16_of(p), stream_of(hip_stream)));
}

uint64_t ttt_ssm_forward_workspace_bytes(const ttt_params* p, int32_t groups, int32_t n) {
  return tttv::ssm_forward_workspace_bytes(p, groups, n);
}

ttt_status ttt_ssm_forward(const ttt_params* p, int32_t groups, int32_t n, const void* x,
                           const float* dt, const float* a, const void* b, const void* c,
                           const float* d_skip, const float* state0, void* y,
                           float* state_out, void* workspace, uint64_t workspace_bytes,
                           void* hip_stream) {
  tttk::SsmArgs s;
  const ttt_status st = tttv::ssm_forward(p, groups, n, x, dt, a, b, c, d_skip, state0, y,
                                          state_out, workspace, workspace_bytes, &s);
  if (st != TTT_OK) return st;
  return status_of(tttk::launch_ssm(s, bf16_of(p), stream_of(hip_stream)));
}

ttt_status ttt_ssm_decode_step(const ttt_params* p, int32_t groups, int32_t n, const void* x,
                               const float* dt, const float* a, const void* b, const void* c,
                               const float* d_skip, float* state, void* y, void* hip_stream) {
  tttk::SsmArgs s;
  const ttt_status st = tttv::ssm_decode(p, groups, n, x, dt, a, b, c, d_skip, state, y, &s);
  if (st != TTT_OK) return st;
  return status_of(tttk::launch_ssm_decode(s, bf16_of(p), stream_of(hip_stream)));
}

uint64_t ttt_ssm_backward_workspace_bytes(const ttt_params* p, int32_t groups, int32_t n) {
  return tttv::ssm_backward_workspace_bytes(p, groups, n);
}

ttt_status ttt_ssm_backward(const ttt_params* p, int32_t groups, int32_t n, const void* x,
                            const float* dt, const float* a, const void* b, const void* c,
                            const float* d_skip, const float* state0, const void* dy,
                            const float* dstate, void* dx, float* ddt, float* da, void* db,
                            void* dc, float* dd, float* dstate0, void* workspace,
                            uint64_t workspace_bytes, void* hip_stream) {
  tttk::SsmBackwardArgs s;
  const ttt_status st =
      tttv::ssm_backward(p, groups, n, x, dt, a, b, c, d_skip, state0, dy, dstate, dx, ddt, da,
                         db, dc, dd, dstate0, workspace, workspace_bytes, &s);
  if (st != TTT_OK) return st;
  return status_of(tttk::launch_ssm_backward(s, bf16_of(p), stream_of(hip_stream)));
}

}  // extern "C"
