// ttt_block_args.hpp -- launch arguments of the kernels around and beside the
// TTT scans: the RMS norm, the 8-bit input projection, the short causal
// convolution and the selective state space scan.  Plain structs with no HIP
// dependency, filled by ttt_block_validate.cpp.
#pragma once

#include <stdint.h>

namespace tttk {

struct NormArgs {
  const void* x;          // [rows, width] io
  const void* residual;   // [rows, width] io or nullptr
  const float* weight;    // [width]
  void* y;                // [rows, width] io, or e4m3 bytes
  float* scale;           // [rows]: e4m3 form only
  void* res_out;          // [rows, width] io or nullptr
  int64_t rows;
  int32_t width;
  float eps;
};

struct NormBackwardArgs {
  const void* r;          // [rows, width] io
  const float* weight;
  const void* dy;
  const void* dr;         // cotangent of r itself, or nullptr
  void* dx;
  float* dweight;         // [width]
  float* partial;         // [groups, width]
  int64_t rows;
  int32_t width, groups;
  float eps;
};

struct InputF8Args {
  const void* x;          // [B,T,D] e4m3
  const float* x_scale;   // [B,T]
  const void* w;          // [3 H 64 + H, D] e4m3
  const float* w_scale;   // [3 H 64 + H]
  const float* b_eta;     // [H]
  void* q;                // [B,H,T,64] bf16
  void* k;
  void* v;
  float* eta;             // [B,H,T]
  int32_t B, T, D, H;
  float eta_base;
};

struct ConvArgs {
  const void* x;          // [B,H,T,d] io
  const float* w;         // [H,K,d]
  const float* bias;      // [H,d] or nullptr
  const void* state0;     // [B,H,K-1,d] io or nullptr
  void* y;                // [B,H,T,d] io
  void* state_out;        // [B,H,K-1,d] io or nullptr (the step: the state itself)
  int32_t B, H, T, d, taps, silu;
};

// Tokens of one partial filter gradient, a workgroup's: 16 for each of the rows
// of d / 4 threads that 256 threads make, at least 64.
inline int32_t conv_chunk(int32_t d) {
  const int32_t tokens = 256 / (d / 4) * 16;
  return tokens < 64 ? 64 : tokens;
}

struct ConvBackwardArgs {
  const void* x;
  const float* w;
  const float* bias;
  const void* state0;
  const void* dy;         // [B,H,T,d] io
  const void* dstate;     // cotangent of the final state, or nullptr
  void* dx;
  float* dw;              // [H,K,d]
  float* dbias;           // [H,d]
  void* dstate0;          // [B,H,K-1,d] io or nullptr
  float* partial;         // [B][chunks][H][K+1][d]
  int32_t B, H, T, d, taps, silu, chunk, chunks;
};

struct SsmArgs {
  const void* x;          // [B,H,T,64] io
  const float* dt;        // [B,H,T]
  const float* a;         // [H]
  const void* b;          // [B,G,T,N] io
  const void* c;          // [B,G,T,N] io
  const float* d_skip;    // [H] or nullptr
  const float* state0;    // [B,H,N,64] or nullptr
  void* y;                // [B,H,T,64] io
  float* state_out;       // [B,H,N,64] or nullptr (the step: the state itself)
  int32_t B, H, G, T, N;
  // time segments of seg_tiles tiles of tile tokens (scan only)
  int32_t tile, segs, seg_tiles;
  float* ws_state;        // [units][segs][N][64]
  double* ws_fade;        // [units][segs]: log2 of a segment's whole decay
};

struct SsmBackwardArgs {
  SsmArgs f;              // the forward's inputs; y, state_out and f.ws_state as described below
  const void* dy;
  const float* dstate;    // cotangent of the final state, or nullptr
  void* dx;
  float* ddt;             // [B,H,T]
  float* da;              // [H]
  void* db;               // [B,G,T,N] io
  void* dc;
  float* dd;              // [H] or nullptr
  float* dstate0;         // [B,H,N,64] or nullptr
  float* ws_tile;         // [units][tiles][N][64]: state before a tile, from zero at its segment
  float* ws_adj;          // [units][segs][N][64]: adjoint behind each segment
  float* ws_sums;         // [units][segs][2]: da and dd of a segment
  float* ws_db;           // [B,H,T,N] per-head gradients where heads share b and c, else nullptr
  float* ws_dc;
};

}  // namespace tttk
