// ttt_block_validate.hpp -- host-side argument checks of the RMS norm, the
// 8-bit input projection, the short convolution and the selective state
// space scan, and the fill of their launch arguments.  As ttt_validate.hpp:
// no HIP dependency, TTT_OK with *a filled or the status of the first failed
// check with *a unspecified.
#pragma once

#include <stdint.h>

#include "ttt.h"
#include "ttt_block_args.hpp"

namespace tttv {

ttt_status rms_norm(int64_t rows, int32_t width, int32_t io_dtype, float eps, const void* x,
                    const void* residual, const float* weight, void* y, bool f8, float* scale,
                    void* res_out, tttk::NormArgs* a);

// Row groups of the norm's backward: one partial weight gradient each.
int32_t norm_groups(int64_t rows);
uint64_t rms_norm_backward_workspace_bytes(int64_t rows, int32_t width);
ttt_status rms_norm_backward(int64_t rows, int32_t width, int32_t io_dtype, float eps,
                             const void* r, const float* weight, const void* dy, const void* dr,
                             void* dx, float* dweight, void* workspace, uint64_t workspace_bytes,
                             tttk::NormBackwardArgs* a);

ttt_status input_projection_f8(const ttt_params* p, int32_t d_model, const void* x,
                               const float* x_scale, const void* w_in, const float* w_scale,
                               const float* b_eta, float eta_base, void* q, void* k, void* v,
                               float* eta, tttk::InputF8Args* a);

ttt_status conv_forward(const ttt_params* p, int32_t taps, uint32_t flags, const void* x,
                        const float* w, const float* bias, const void* state0, void* y,
                        void* state_out, tttk::ConvArgs* a);
ttt_status conv_decode(const ttt_params* p, int32_t taps, uint32_t flags, const void* x,
                       const float* w, const float* bias, void* state, void* y,
                       tttk::ConvArgs* a);
uint64_t conv_backward_workspace_bytes(const ttt_params* p, int32_t taps);
ttt_status conv_backward(const ttt_params* p, int32_t taps, uint32_t flags, const void* x,
                         const float* w, const float* bias, const void* state0, const void* dy,
                         const void* dstate, void* dx, float* dw, float* dbias, void* dstate0,
                         void* workspace, uint64_t workspace_bytes, tttk::ConvBackwardArgs* a);

uint64_t ssm_forward_workspace_bytes(const ttt_params* p, int32_t groups, int32_t n);
ttt_status ssm_forward(const ttt_params* p, int32_t groups, int32_t n, const void* x,
                       const float* dt, const float* a, const void* b, const void* c,
                       const float* d_skip, const float* state0, void* y, float* state_out,
                       void* workspace, uint64_t workspace_bytes, tttk::SsmArgs* out);
ttt_status ssm_decode(const ttt_params* p, int32_t groups, int32_t n, const void* x,
                      const float* dt, const float* a, const void* b, const void* c,
                      const float* d_skip, float* state, void* y, tttk::SsmArgs* out);
uint64_t ssm_backward_workspace_bytes(const ttt_params* p, int32_t groups, int32_t n);
ttt_status ssm_backward(const ttt_params* p, int32_t groups, int32_t n, const void* x,
                        const float* dt, const float* a, const void* b, const void* c,
                        const float* d_skip, const float* state0, const void* dy,
                        const float* dstate, void* dx, float* ddt, float* da, void* db, void* dc,
                        float* dd, float* dstate0, void* workspace, uint64_t workspace_bytes,
                        tttk::SsmBackwardArgs* out);

}  // namespace tttv
