// ttt_conv.hip -- the short causal convolution for gfx950: one filter of K = 2
// to 4 taps per head and feature along the tokens of a [T, d] unit, with bias
// and an optional SiLU; its one-token step and its backward.
//
//     u_t = bias + sum_{j<K} w_j x_{t-K+1+j},   y_t = u_t or u_t / (1 + exp(-u_t))
// Backward, with du_t = dy_t act'(u_t) (u made again from x):
//     dx_t = sum_j w_j du_{t+K-1-j},   dw_j = sum_t du_t x_{t-K+1+j},   dbias = sum_t du_t
// The final state is the last K-1 inputs, so its cotangent adds to their dx.
//
// Bound by HBM: 2 K + 6 operations a value against 4 bytes.  A thread owns 8
// features (16 bytes) over a strip of tokens and keeps the window of K inputs
// in registers, so x comes from HBM once; the K - 1 inputs in front of a strip
// are the neighbouring strip's lines, in cache.  The loads of a strip are
// issued together before any of them is used.
#include "ttt_block.hpp"
#include "ttt_block_io.hpp"

namespace tttk {
namespace {

constexpr int NT = 256;
constexpr int S = 8;              // tokens of a strip
constexpr uint32_t MAX_GRID = 1u << 20;

__device__ __forceinline__ float sigmoid(float u) { return 1.0f / (1.0f + __expf(-u)); }

template <int K>
struct Filter {
  F8 w[K], bias;
};

template <int K>
__device__ __forceinline__ Filter<K> load_filter(const float* w, const float* bias, int h, int d,
                                                 int f) {
  Filter<K> r;
#pragma unroll
  for (int j = 0; j < K; ++j) r.w[j] = load8_f32(w + (static_cast<size_t>(h) * K + j) * d + f);
  if (bias) {
    r.bias = load8_f32(bias + static_cast<size_t>(h) * d + f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.bias.v[i] = 0.f;
  }
  return r;
}

// Input t of a unit (t >= 1-K; before 0 from state0 or zero; from T on zero).
template <bool BF16, int K>
__device__ __forceinline__ Raw8<BF16> input_at(const void* x, const void* state0, size_t unit,
                                               int t, int T, int d, int f) {
  if (t >= 0)
    return t < T ? load8_raw<BF16>(x, (unit * T + t) * d + f) : zero8_raw<BF16>();
  return state0 ? load8_raw<BF16>(state0, (unit * (K - 1) + (t + K - 1)) * d + f)
                : zero8_raw<BF16>();
}

template <bool BF16, int K>
__global__ __launch_bounds__(NT) void ttt_conv_k(ConvArgs a) {
  const int T = a.T, d = a.d;
  const uint32_t lanes = d / 8, strips = (T + S - 1) / S;
  const uint64_t per_unit = static_cast<uint64_t>(lanes) * strips;
  const uint64_t total = per_unit * a.B * a.H;
  for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * NT + threadIdx.x; i < total;
       i += static_cast<uint64_t>(gridDim.x) * NT) {
    size_t unit;
    uint32_t in;
    if (total <= 0xffffffffull) {
      unit = static_cast<uint32_t>(i) / static_cast<uint32_t>(per_unit);
      in = static_cast<uint32_t>(i) - static_cast<uint32_t>(unit) * static_cast<uint32_t>(per_unit);
    } else {
      unit = i / per_unit;
      in = static_cast<uint32_t>(i - unit * per_unit);
    }
    const uint32_t strip = in / lanes;
    const int f = 8 * (in - strip * lanes), t0 = strip * S;
    Raw8<BF16> in8[S + K - 1];
#pragma unroll
    for (int s = 0; s < S + K - 1; ++s)
      in8[s] = input_at<BF16, K>(a.x, a.state0, unit, t0 + s - (K - 1), T, d, f);
    const Filter<K> flt = load_filter<K>(a.w, a.bias, static_cast<int>(unit % a.H), d, f);
    F8 win[K];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) win[j + 1] = widen8(in8[j]);
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j) win[j] = win[j + 1];
      win[K - 1] = widen8(in8[s + K - 1]);
      F8 y = flt.bias;
#pragma unroll
      for (int j = 0; j < K; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) y.v[e] += flt.w[j].v[e] * win[j].v[e];
      if (a.silu) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y.v[e] *= sigmoid(y.v[e]);
      }
      if (t0 + s < T) store8<BF16>(a.y, (unit * T + t0 + s) * d + f, y);
    }
    if (a.state_out && strip == strips - 1) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
        store8<BF16>(a.state_out, (unit * (K - 1) + j) * d + f,
                     widen8(input_at<BF16, K>(a.x, a.state0, unit, T - (K - 1) + j, T, d, f)));
    }
  }
}

// One token: state0 = state_out, moved on by the thread that read it.
template <bool BF16, int K>
__global__ __launch_bounds__(NT) void ttt_conv_step_k(ConvArgs a) {
  const int d = a.d;
  const uint32_t lanes = d / 8;
  const uint64_t total = static_cast<uint64_t>(lanes) * a.B * a.H;
  const uint64_t i = static_cast<uint64_t>(blockIdx.x) * NT + threadIdx.x;
  if (i >= total) return;
  const size_t unit = i / lanes;
  const int f = 8 * static_cast<int>(i - unit * lanes);
  Raw8<BF16> win[K];
#pragma unroll
  for (int j = 0; j < K - 1; ++j)
    win[j] = load8_raw<BF16>(a.state_out, (unit * (K - 1) + j) * d + f);
  win[K - 1] = load8_raw<BF16>(a.x, unit * d + f);
  const Filter<K> flt = load_filter<K>(a.w, a.bias, static_cast<int>(unit % a.H), d, f);
  F8 y = flt.bias;
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const F8 x = widen8(win[j]);
#pragma unroll
    for (int e = 0; e < 8; ++e) y.v[e] += flt.w[j].v[e] * x.v[e];
  }
  if (a.silu) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y.v[e] *= sigmoid(y.v[e]);
  }
  store8<BF16>(a.y, unit * d + f, y);
#pragma unroll
  for (int j = 0; j < K - 1; ++j)
    store8<BF16>(a.state_out, (unit * (K - 1) + j) * d + f, widen8(win[j + 1]));
}

// Backward: a workgroup takes one unit's chunk of CHUNK tokens.  Threads are
// (strip of S tokens) x (8 features); where a chunk's strips do not fit at
// once (d > 64) they take turns.  The filter gradients are summed over a
// thread's strips in registers, over the workgroup's strips through LDS and
// left as one partial [K+1][d] per chunk.
constexpr int CHUNK = 256;

template <bool BF16, int K>
__global__ __launch_bounds__(NT) void ttt_conv_bwd_k(ConvBackwardArgs a) {
  __shared__ float red[NT][9];
  const int T = a.T, d = a.d;
  const int lanes = d / 8, rows = NT / lanes;       // d <= 1024: lanes <= 128
  const size_t unit = blockIdx.x / a.chunks;
  const int chunk = blockIdx.x - static_cast<uint32_t>(unit) * a.chunks;
  const int h = static_cast<int>(unit % a.H), b = static_cast<int>(unit / a.H);
  const int row = threadIdx.x / lanes, f = 8 * (threadIdx.x - row * lanes);
  F8 acc[K + 1];
#pragma unroll
  for (int j = 0; j <= K; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[j].v[e] = 0.f;
  if (row < rows) {
    const Filter<K> flt = load_filter<K>(a.w, a.bias, h, d, f);
    for (int strip = row; strip < CHUNK / S; strip += rows) {
      const int t0 = chunk * CHUNK + strip * S;
      if (t0 >= T) break;
      // inputs t0-K+1 .. t0+S+K-2 and cotangents t0 .. t0+S+K-2
      Raw8<BF16> in8[S + 2 * (K - 1)], g8[S + K - 1];
#pragma unroll
      for (int s = 0; s < S + 2 * (K - 1); ++s)
        in8[s] = input_at<BF16, K>(a.x, a.state0, unit, t0 + s - (K - 1), T, d, f);
#pragma unroll
      for (int s = 0; s < S + K - 1; ++s)
        g8[s] = t0 + s < T ? load8_raw<BF16>(a.dy, (unit * T + t0 + s) * d + f)
                           : zero8_raw<BF16>();
      F8 win[K], dus[K];   // dus[j] = du of token (current - (K-1) + j)
#pragma unroll
      for (int j = 0; j < K - 1; ++j) win[j + 1] = widen8(in8[j]);
#pragma unroll
      for (int j = 0; j < K; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) dus[j].v[e] = 0.f;
      const bool first = t0 == 0 && a.dstate0;
#pragma unroll
      for (int s = 0; s < S + K - 1; ++s) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
          win[j] = win[j + 1];
          dus[j] = dus[j + 1];
        }
        win[K - 1] = widen8(in8[s + K - 1]);
        F8 du = widen8(g8[s]);
        if (a.silu) {
          F8 u = flt.bias;
#pragma unroll
          for (int j = 0; j < K; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) u.v[e] += flt.w[j].v[e] * win[j].v[e];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float sg = sigmoid(u.v[e]);
            du.v[e] *= sg * (1.0f + u.v[e] * (1.0f - sg));
          }
        }
        dus[K - 1] = du;
        if (s < S && t0 + s < T) {
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[K].v[e] += du.v[e];
#pragma unroll
          for (int j = 0; j < K; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[j].v[e] += du.v[e] * win[j].v[e];
        }
        // dx of token t0 + s - (K-1): its du's are dus[0..K-1]
        const int t = t0 + s - (K - 1);
        if ((s >= K - 1 && t < T) || (first && s < K - 1)) {
          F8 dx;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            dx.v[e] = 0.f;
#pragma unroll
            for (int j = 0; j < K; ++j) dx.v[e] += flt.w[K - 1 - j].v[e] * dus[j].v[e];
          }
          if (a.dstate && t >= T - (K - 1)) {   // also an input of the final state
            const F8 g = load8<BF16>(a.dstate, (unit * (K - 1) + (t - (T - (K - 1)))) * d + f);
#pragma unroll
            for (int e = 0; e < 8; ++e) dx.v[e] += g.v[e];
          }
          if (t >= 0) store8<BF16>(a.dx, (unit * T + t) * d + f, dx);
          else store8<BF16>(a.dstate0, (unit * (K - 1) + (t + K - 1)) * d + f, dx);
        }
      }
    }
  }
  float* out = a.partial +
               ((static_cast<size_t>(b) * a.chunks + chunk) * a.H + h) * (K + 1) * d;
#pragma unroll
  for (int j = 0; j <= K; ++j) {
    __syncthreads();
    if (row < rows) {
#pragma unroll
      for (int e = 0; e < 8; ++e) red[threadIdx.x][e] = acc[j].v[e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < d; i += NT) {
      float s = 0.f;
      for (int r = 0; r < rows; ++r) s += red[r * lanes + i / 8][i % 8];
      out[static_cast<size_t>(j) * d + i] = s;
    }
  }
}

// dw, dbias: the partials of every (batch, chunk) in order; 16 columns per
// workgroup, 16 threads a column.
template <int K>
__global__ __launch_bounds__(NT) void ttt_conv_bwd_sum_k(ConvBackwardArgs a) {
  __shared__ float part[16][17];
  const int col = threadIdx.x & 15, slot = threadIdx.x >> 4;
  const size_t n = static_cast<size_t>(a.H) * (K + 1) * a.d;
  const size_t i = 16 * static_cast<size_t>(blockIdx.x) + col;
  const int64_t parts = static_cast<int64_t>(a.B) * a.chunks;
  float s = 0.f;
  if (i < n)
    for (int64_t p = slot; p < parts; p += 16) s += a.partial[p * n + i];
  part[slot][col] = s;
  __syncthreads();
  if (slot == 0 && i < n) {
#pragma unroll
    for (int k = 1; k < 16; ++k) s += part[k][col];
    const size_t h = i / (static_cast<size_t>(K + 1) * a.d);
    const int in = static_cast<int>(i - h * (K + 1) * a.d);
    if (in < K * a.d) a.dw[h * K * a.d + in] = s;
    else a.dbias[h * a.d + (in - K * a.d)] = s;
  }
}

template <bool BF16, int K>
hipError_t conv_launch(const ConvArgs& a, hipStream_t stream) {
  const uint64_t total = static_cast<uint64_t>(a.d / 8) * ((a.T + S - 1) / S) * a.B * a.H;
  const uint64_t need = (total + NT - 1) / NT;
  hipLaunchKernelGGL((ttt_conv_k<BF16, K>), dim3(need < MAX_GRID ? need : MAX_GRID), dim3(NT), 0,
                     stream, a);
  return hipGetLastError();
}

template <bool BF16, int K>
hipError_t conv_step_launch(const ConvArgs& a, hipStream_t stream) {
  const uint64_t total = static_cast<uint64_t>(a.d / 8) * a.B * a.H;
  hipLaunchKernelGGL((ttt_conv_step_k<BF16, K>), dim3((total + NT - 1) / NT), dim3(NT), 0, stream,
                     a);
  return hipGetLastError();
}

template <bool BF16, int K>
hipError_t conv_bwd_launch(const ConvBackwardArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((ttt_conv_bwd_k<BF16, K>),
                     dim3(static_cast<uint32_t>(a.B) * a.H * a.chunks), dim3(NT), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const uint64_t n = static_cast<uint64_t>(a.H) * (K + 1) * a.d;
  hipLaunchKernelGGL((ttt_conv_bwd_sum_k<K>), dim3((n + 15) / 16), dim3(NT), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_conv(const ConvArgs& a, bool bf16, hipStream_t stream) {
  if (a.taps == 2) return bf16 ? conv_launch<true, 2>(a, stream) : conv_launch<false, 2>(a, stream);
  if (a.taps == 3) return bf16 ? conv_launch<true, 3>(a, stream) : conv_launch<false, 3>(a, stream);
  return bf16 ? conv_launch<true, 4>(a, stream) : conv_launch<false, 4>(a, stream);
}

hipError_t launch_conv_decode(const ConvArgs& a, bool bf16, hipStream_t stream) {
  if (a.taps == 2)
    return bf16 ? conv_step_launch<true, 2>(a, stream) : conv_step_launch<false, 2>(a, stream);
  if (a.taps == 3)
    return bf16 ? conv_step_launch<true, 3>(a, stream) : conv_step_launch<false, 3>(a, stream);
  return bf16 ? conv_step_launch<true, 4>(a, stream) : conv_step_launch<false, 4>(a, stream);
}

hipError_t launch_conv_backward(const ConvBackwardArgs& a, bool bf16, hipStream_t stream) {
  if (a.taps == 2)
    return bf16 ? conv_bwd_launch<true, 2>(a, stream) : conv_bwd_launch<false, 2>(a, stream);
  if (a.taps == 3)
    return bf16 ? conv_bwd_launch<true, 3>(a, stream) : conv_bwd_launch<false, 3>(a, stream);
  return bf16 ? conv_bwd_launch<true, 4>(a, stream) : conv_bwd_launch<false, 4>(a, stream);
}

}  // namespace tttk
