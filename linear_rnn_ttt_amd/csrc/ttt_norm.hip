// ttt_norm.hip -- RMS norm with the residual's addition for gfx950, its form
// with an 8-bit output, and its backward.
//
// Forward, one pass over each row:
//     r = x + residual,  y = r rsqrt(mean(r^2) + eps) w
// A row lives in registers from its load to its stores, so each input is read
// and each output written once; fp32 throughout, each output rounded once.
// Backward, the same way, with xh = r rstd and u = dy w:
//     dx = rstd (u - xh mean(u xh)) + dr,   dw = sum over rows of dy xh
// where each workgroup sums dw over its rows in registers and leaves one
// partial row; a second launch adds the partial rows in order.
//
// Bound by HBM: forward with residual, bf16, 32768 rows of 2048: 99 us, 5.4 TB/s
// (a copy on this card reaches 5.4); backward, 16384 rows of 768: 20.7 us with
// its second launch, 4.9 TB/s.  All of a row's loads go out before the first of
// them is waited for: reading, widening and adding step by step took 26.7 us
// for that backward, 530 instead of 432 us for a forward of 16384 rows of 16384.
// Loading the next row as well, ahead of the sums, gained nothing (21.4 us): there are
// enough waves.  Backward workgroups: 512, each with a row of partial sums;
// 256 take 23.2 us, 1024 22.4.
#include "ttt_block.hpp"
#include "ttt_block_io.hpp"

namespace tttk {
namespace {

constexpr int NT = 256;          // threads of a workgroup
constexpr float F8_MAX = 448.f;  // largest e4m3
// below this a row's scale would leave fp32's normal range: it is stored with scale 1
constexpr float F8_LEAST = 448.f * 1.17549435e-38f;

// Threads of one row (LANES) share it in V steps of 8 values each.
template <int LANES>
struct RowSum {
  __device__ static float sum(float x, float*) { return wave_sum(x); }
  __device__ static float max(float x, float*) { return wave_max(x); }
  __device__ static void sum2(float* x, float* y, float*, float*) {
    *x = wave_sum(*x);
    *y = wave_sum(*y);
  }
};
template <>
struct RowSum<NT> {
  __device__ static void sum2(float* x, float* y, float* lds, float* lds2) {
    *x = wave_sum(*x);
    *y = wave_sum(*y);
    if ((threadIdx.x & 63) == 0) {
      lds[threadIdx.x >> 6] = *x;
      lds2[threadIdx.x >> 6] = *y;
    }
    lds_barrier();
    *x = (lds[0] + lds[1]) + (lds[2] + lds[3]);
    *y = (lds2[0] + lds2[1]) + (lds2[2] + lds2[3]);
  }
  // every thread gets the four waves' total; `lds` has 4 floats, and a second
  // call has to bring another 4
  __device__ static float sum(float x, float* lds) {
    x = wave_sum(x);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    lds_barrier();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
  }
  __device__ static float max(float x, float* lds) {
    x = wave_max(x);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    lds_barrier();
    return fmaxf(fmaxf(lds[0], lds[1]), fmaxf(lds[2], lds[3]));
  }
};

// OUT: 0 y of the I/O type, 1 e4m3 with a scale per row.
template <bool BF16, int LANES, int V, int OUT, bool RES>
__global__ __launch_bounds__(NT) void ttt_norm_k(NormArgs a) {
  constexpr int ROWS = NT / LANES;
  __shared__ float red[2][2][4];
  const int lane = threadIdx.x % LANES;
  const int W = a.width;
  F8 w[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int f = 8 * (lane + LANES * j);
    if (f < W) w[j] = load8_f32(a.weight + f);
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
  int turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / LANES; row < a.rows;
       row += step, turn ^= 1) {
    const size_t at = static_cast<size_t>(row) * W;
    Raw8<BF16> rx[V], rq[RES ? V : 1];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int f = 8 * (lane + LANES * j);
      if (f < W) {
        rx[j] = load8_raw<BF16>(a.x, at + f);
        if constexpr (RES) rq[j] = load8_raw<BF16>(a.residual, at + f);
      }
    }
    F8 r[V];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int f = 8 * (lane + LANES * j);
      if (f < W) {
        r[j] = widen8(rx[j]);
        if constexpr (RES) {
          const F8 q = widen8(rq[j]);
#pragma unroll
          for (int i = 0; i < 8; ++i) r[j].v[i] += q.v[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += r[j].v[i] * r[j].v[i];
      }
    }
    ss = RowSum<LANES>::sum(ss, red[turn][0]);
    const float rstd = 1.0f / sqrtf(ss / static_cast<float>(W) + a.eps);
    if constexpr (RES) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int f = 8 * (lane + LANES * j);
        if (f < W) store8<BF16>(a.res_out, at + f, r[j]);
      }
    }
    float top = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int f = 8 * (lane + LANES * j);
      if (f < W) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          r[j].v[i] = r[j].v[i] * rstd * w[j].v[i];
          if constexpr (OUT == 1) top = fmaxf(top, fabsf(r[j].v[i]));
        }
        if constexpr (OUT == 0) store8<BF16>(a.y, at + f, r[j]);
      }
    }
    if constexpr (OUT == 1) {
      top = RowSum<LANES>::max(top, red[turn][1]);
      const bool some = top >= F8_LEAST;
      const float inv = some ? F8_MAX / top : 1.0f;
      if (lane == 0) a.scale[row] = some ? top / F8_MAX : 1.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int f = 8 * (lane + LANES * j);
        if (f < W) {
          uint32_t b[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            int t = __builtin_amdgcn_cvt_pk_fp8_f32(r[j].v[4 * h] * inv, r[j].v[4 * h + 1] * inv,
                                                    0, false);
            t = __builtin_amdgcn_cvt_pk_fp8_f32(r[j].v[4 * h + 2] * inv, r[j].v[4 * h + 3] * inv,
                                                t, true);
            b[h] = static_cast<uint32_t>(t);
          }
          *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(a.y) + at + f) = u32x2{b[0], b[1]};
        }
      }
    }
  }
}

template <bool BF16, int LANES, int V>
__global__ __launch_bounds__(NT) void ttt_norm_bwd_k(NormBackwardArgs a) {
  constexpr int ROWS = NT / LANES;
  __shared__ float red[2][2][4];
  __shared__ float part[LANES == NT ? 1 : 3 * 8 * LANES];
  const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES;
  const int W = a.width;
  F8 w[V], dw[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int f = 8 * (lane + LANES * j);
    if (f < W) w[j] = load8_f32(a.weight + f);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j].v[i] = 0.f;
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
  int turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + slot; row < a.rows;
       row += step, turn ^= 1) {
    const size_t at = static_cast<size_t>(row) * W;
    Raw8<BF16> rr[V], rg[V], ro[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int f = 8 * (lane + LANES * j);
      if (f < W) {
        rr[j] = load8_raw<BF16>(a.r, at + f);
        rg[j] = load8_raw<BF16>(a.dy, at + f);
        ro[j] = a.dr ? load8_raw<BF16>(a.dr, at + f) : zero8_raw<BF16>();
      }
    }
    float ss = 0.f, su = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int f = 8 * (lane + LANES * j);
      if (f < W) {
        const F8 r = widen8(rr[j]), g = widen8(rg[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss += r.v[i] * r.v[i];
          su += g.v[i] * w[j].v[i] * r.v[i];
        }
      }
    }
    RowSum<LANES>::sum2(&ss, &su, red[turn][0], red[turn][1]);
    const float rstd = 1.0f / sqrtf(ss / static_cast<float>(W) + a.eps);
    // xh mean(u xh) rstd = r (rstd^3 sum(u r) / W)
    const float back = rstd * rstd * rstd * (su / static_cast<float>(W));
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int f = 8 * (lane + LANES * j);
      if (f < W) {
        const F8 r = widen8(rr[j]), g = widen8(rg[j]);
        F8 o = widen8(ro[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o.v[i] += rstd * g.v[i] * w[j].v[i] - r.v[i] * back;
          dw[j].v[i] += g.v[i] * (r.v[i] * rstd);
        }
        store8<BF16>(a.dx, at + f, o);
      }
    }
  }
  // the workgroup's weight gradient: its waves' in order (one row per wave), or already whole
  float* out = a.partial + static_cast<size_t>(blockIdx.x) * W;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int f = 8 * (lane + LANES * j);
    if constexpr (LANES != NT) {
      __syncthreads();
      if (slot > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) part[((slot - 1) * 8 + i) * LANES + lane] = dw[j].v[i];
      }
      __syncthreads();
      if (slot == 0) {
#pragma unroll
        for (int s = 0; s < 3; ++s)
#pragma unroll
          for (int i = 0; i < 8; ++i) dw[j].v[i] += part[(s * 8 + i) * LANES + lane];
      }
    }
    if (slot == 0 && f < W) store8<false>(out, f, dw[j]);
  }
}

// dweight[f]: the groups' partial rows in order.
__global__ __launch_bounds__(NT) void ttt_norm_bwd_sum_k(NormBackwardArgs a) {
  column_sums(a.partial, a.width, a.groups, [&](size_t f, float s) { a.dweight[f] = s; });
}

// A row is one wave's (no barrier) or, where that leaves each lane with too many
// loads, a workgroup's; V steps of 8 values for each lane.  Measured, bf16, us,
// a wave / a workgroup a row:
//   forward     512 rows: width 512 2.1 / 2.2, 768 2.5 / 2.3, 1024 2.6 / 2.4, 2048 3.7 / 2.9
//             2048 rows:        512 2.7 / 2.9, 768 3.3 / 3.3, 1024 3.7 / 3.6, 2048 6.4 / 6.0
//             8192 rows:        512 6.0 / 6.1, 768 8.3 / 9.2, 1024 11.1 / 11.5, 2048 20.7 / 20.4
//   backward    512 rows:       512 4.6 / 6.9, 1024 5.7 / 7.5, 2048 7.6 / 8.0
//            32768 rows:        512 26.9 / 86, 1024 48.7 / 98, 2048 116 / 155
constexpr int64_t kMaxGrid = 2048;      // 8 workgroups per compute unit, then rows in turn
constexpr int64_t kWaveRows = 2048;     // forward, widths of 520 to 1024: fewer take workgroups

template <bool BF16, int LANES, int V>
hipError_t norm_launch(const NormArgs& a, hipStream_t stream) {
  const int64_t rows = NT / LANES, need = (a.rows + rows - 1) / rows;
  const dim3 grid(static_cast<uint32_t>(need < kMaxGrid ? need : kMaxGrid)), block(NT);
  if (a.scale) {
    if (a.residual) hipLaunchKernelGGL((ttt_norm_k<BF16, LANES, V, 1, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((ttt_norm_k<BF16, LANES, V, 1, false>), grid, block, 0, stream, a);
  } else {
    if (a.residual) hipLaunchKernelGGL((ttt_norm_k<BF16, LANES, V, 0, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((ttt_norm_k<BF16, LANES, V, 0, false>), grid, block, 0, stream, a);
  }
  return hipGetLastError();
}

template <bool BF16>
hipError_t norm_pick(const NormArgs& a, hipStream_t stream) {
  const int w = a.width;
  if (w <= 512) return norm_launch<BF16, 64, 1>(a, stream);
  if (w <= 1024 && a.rows >= kWaveRows) return norm_launch<BF16, 64, 2>(a, stream);
  if (w <= 2048) return norm_launch<BF16, NT, 1>(a, stream);
  if (w <= 4096) return norm_launch<BF16, NT, 2>(a, stream);
  if (w <= 8192) return norm_launch<BF16, NT, 4>(a, stream);
  return norm_launch<BF16, NT, 8>(a, stream);
}

template <bool BF16, int LANES, int V>
hipError_t norm_bwd_launch(const NormBackwardArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((ttt_norm_bwd_k<BF16, LANES, V>), dim3(a.groups), dim3(NT), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(ttt_norm_bwd_sum_k, dim3((a.width + 15) / 16), dim3(NT), 0, stream, a);
  return hipGetLastError();
}

template <bool BF16>
hipError_t norm_bwd_pick(const NormBackwardArgs& a, hipStream_t stream) {
  const int w = a.width;
  if (w <= 512) return norm_bwd_launch<BF16, 64, 1>(a, stream);
  if (w <= 1024) return norm_bwd_launch<BF16, 64, 2>(a, stream);
  if (w <= 2048) return norm_bwd_launch<BF16, 64, 4>(a, stream);
  if (w <= 4096) return norm_bwd_launch<BF16, NT, 2>(a, stream);
  if (w <= 8192) return norm_bwd_launch<BF16, NT, 4>(a, stream);
  return norm_bwd_launch<BF16, NT, 8>(a, stream);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? norm_pick<true>(a, stream) : norm_pick<false>(a, stream);
}

hipError_t launch_norm_backward(const NormBackwardArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? norm_bwd_pick<true>(a, stream) : norm_bwd_pick<false>(a, stream);
}

}  // namespace tttk
