// ttt_block.hpp -- launch interfaces of the RMS norm (ttt_norm.hip), the
// 8-bit input projection (ttt_input_f8.hip), the short convolution
// (ttt_conv.hip) and the selective state space scan (ttt_ssm.hip,
// ttt_ssm_backward.hip).  Argument structs in ttt_block_args.hpp; the host
// API has validated every field before a launcher is called.  Each returns
// the hipError_t of its launches.
#pragma once

#include <hip/hip_runtime.h>

#include "ttt_block_args.hpp"

namespace tttk {

hipError_t launch_norm(const NormArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_norm_backward(const NormBackwardArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_input_f8(const InputF8Args& a, hipStream_t stream);
hipError_t launch_conv(const ConvArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_conv_decode(const ConvArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_conv_backward(const ConvBackwardArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_ssm(const SsmArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_ssm_decode(const SsmArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_ssm_backward(const SsmBackwardArgs& a, bool bf16, hipStream_t stream);

}  // namespace tttk
