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
// issued together before any of them is used.  bf16, 4 taps, SiLU, B4 H32 T8192
// d64: 51 us, 5.3 TB/s (a copy on this card reaches 5.4).
#include <type_traits>

#include "ttt_block.hpp"
#include "ttt_block_io.hpp"

namespace tttk {
namespace {

constexpr int NT = 256;
constexpr int S = 8;   // tokens loaded together (4, 8, 16: forward 55, 54, 59 us, backward 27, 24, 40 us)
constexpr uint32_t MAX_GRID = 1u << 20;

// v_exp_f32 and v_rcp_f32, one unit each: far below what the tests' fp32 bound
// allows, and a third of the instructions of a full division.
__device__ __forceinline__ float sigmoid(float u) {
  return __builtin_amdgcn_rcpf(1.0f + __expf(-u));
}

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

// Backward: a workgroup takes one unit's chunk of tokens.  Threads are (run of
// tokens) x (4 features: with 8 the windows of x, dy and du took over 256
// registers and left one wave per SIMD, 38.6 us at B8 H12 T2048).  A thread
// walks its run (16 tokens, more where d / 4 threads hardly fit) keeping the
// windows, so the K - 1 cotangents behind a run, of which dx needs du again,
// cost 3 in 19 steps (strips of 8 on their own: 25.1 instead of 23.3 us with
// the sum's launch).  The filter gradients are summed over a run in registers,
// over the workgroup's runs through LDS and left as one partial [K+1][d] per
// chunk.  Bound by the vector unit (u, its sigmoid and slope again), 84 % busy.
template <bool BF16>
using Raw4 = std::conditional_t<BF16, u32x2, f32x4>;

template <bool BF16>
__device__ __forceinline__ Raw4<BF16> load4_raw(const void* p, size_t i) {
  return *reinterpret_cast<const Raw4<BF16>*>(static_cast<const char*>(p) + i * kIoBytes<BF16>);
}
template <bool BF16>
__device__ __forceinline__ f32x4 to_f32(const Raw4<BF16>& r) {
  if constexpr (BF16)
    return f32x4{bf16_lo_to_f32(r.x), bf16_hi_to_f32(r.x), bf16_lo_to_f32(r.y),
                 bf16_hi_to_f32(r.y)};
  else
    return r;
}
template <bool BF16>
__device__ __forceinline__ void store4(void* p, size_t i, f32x4 v) {
  if constexpr (BF16)
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p) + i) =
        u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
  else
    *reinterpret_cast<f32x4*>(static_cast<float*>(p) + i) = v;
}

template <bool BF16, int K>
__global__ __launch_bounds__(NT) void ttt_conv_bwd_k(ConvBackwardArgs a) {
  __shared__ float red[K + 1][4][NT + 1];
  const int T = a.T, d = a.d;
  const int lanes = d / 4, rows = NT / lanes;       // d <= 1024: lanes <= 256
  const size_t unit = blockIdx.x / a.chunks;
  const int chunk = blockIdx.x - static_cast<uint32_t>(unit) * a.chunks;
  const int h = static_cast<int>(unit % a.H), b = static_cast<int>(unit / a.H);
  const int row = threadIdx.x / lanes, f = 4 * (threadIdx.x - row * lanes);
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  auto input = [&](int t) {   // as input_at
    if (t >= 0) return t < T ? load4_raw<BF16>(a.x, (unit * T + t) * d + f) : Raw4<BF16>{};
    return a.state0 ? load4_raw<BF16>(a.state0, (unit * (K - 1) + (t + K - 1)) * d + f)
                    : Raw4<BF16>{};
  };
  f32x4 acc[K + 1];
#pragma unroll
  for (int j = 0; j <= K; ++j) acc[j] = zero;
  if (row < rows) {
    f32x4 w[K], bias = zero;
#pragma unroll
    for (int j = 0; j < K; ++j)
      w[j] = *reinterpret_cast<const f32x4*>(a.w + (static_cast<size_t>(h) * K + j) * d + f);
    if (a.bias) bias = *reinterpret_cast<const f32x4*>(a.bias + static_cast<size_t>(h) * d + f);
    const int share = (a.chunk / S + rows - 1) / rows * S;   // tokens of a thread, one after another
    const int t0 = chunk * a.chunk + row * share;
    const int stop = min(min(t0 + share, (chunk + 1) * a.chunk), T);
    if (t0 < stop) {
      auto cotangent = [&](int t) {
        return t < T ? load4_raw<BF16>(a.dy, (unit * T + t) * d + f) : Raw4<BF16>{};
      };
      f32x4 win[K], dus[K];   // dus[j] = du of token (current - (K-1) + j)
#pragma unroll
      for (int j = 0; j < K - 1; ++j) win[j + 1] = to_f32<BF16>(input(t0 + j - (K - 1)));
#pragma unroll
      for (int j = 0; j < K; ++j) dus[j] = zero;
      const bool first = t0 == 0 && a.dstate0;
      // token t, and dx of token t - (K-1), whose du's are then dus[0..K-1]
      auto step = [&](int t, Raw4<BF16> in, Raw4<BF16> g) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
          win[j] = win[j + 1];
          dus[j] = dus[j + 1];
        }
        win[K - 1] = to_f32<BF16>(in);
        f32x4 du = to_f32<BF16>(g);
        if (a.silu) {
          f32x4 u = bias;
#pragma unroll
          for (int j = 0; j < K; ++j) u += w[j] * win[j];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float sg = sigmoid(u[e]);
            du[e] *= sg * (1.0f + u[e] * (1.0f - sg));
          }
        }
        dus[K - 1] = du;
        if (t < stop) {
          acc[K] += du;
#pragma unroll
          for (int j = 0; j < K; ++j) acc[j] += du * win[j];
        }
        const int to = t - (K - 1);
        if ((to >= t0 && to < stop) || (first && to < 0)) {
          f32x4 dx = zero;
#pragma unroll
          for (int j = 0; j < K; ++j) dx += w[K - 1 - j] * dus[j];
          if (a.dstate && to >= T - (K - 1))   // also an input of the final state
            dx += to_f32<BF16>(
                load4_raw<BF16>(a.dstate, (unit * (K - 1) + (to - (T - (K - 1)))) * d + f));
          if (to >= 0) store4<BF16>(a.dx, (unit * T + to) * d + f, dx);
          else store4<BF16>(a.dstate0, (unit * (K - 1) + (to + K - 1)) * d + f, dx);
        }
      };
      for (int t = t0; t < stop; t += S) {
        Raw4<BF16> in[S], g[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
          in[s] = input(t + s);
          g[s] = cotangent(t + s);
        }
#pragma unroll
        for (int s = 0; s < S; ++s) step(t + s, in[s], g[s]);
      }
      // the cotangents behind that reach back into the share
      const int last = (stop - t0 + S - 1) / S * S + t0;
      Raw4<BF16> in[K - 1], g[K - 1];
#pragma unroll
      for (int s = 0; s < K - 1; ++s) {
        in[s] = input(last + s);
        g[s] = cotangent(last + s);
      }
#pragma unroll
      for (int s = 0; s < K - 1; ++s) step(last + s, in[s], g[s]);
    }
#pragma unroll
    for (int j = 0; j <= K; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[j][e][threadIdx.x] = acc[j][e];
  }
  __syncthreads();
  float* out = a.partial +
               ((static_cast<size_t>(b) * a.chunks + chunk) * a.H + h) * (K + 1) * d;
  for (int i = threadIdx.x; i < (K + 1) * d; i += NT) {
    const int j = i / d, in = i - j * d;
    const float* p = &red[j][in & 3][in >> 2];
    float s = 0.f;
    for (int r = 0; r < rows; ++r) s += p[r * lanes];
    out[i] = s;
  }
}

// dw, dbias: the partials of every (batch, chunk) in order.
template <int K>
__global__ __launch_bounds__(NT) void ttt_conv_bwd_sum_k(ConvBackwardArgs a) {
  const size_t n = static_cast<size_t>(a.H) * (K + 1) * a.d;
  column_sums(a.partial, n, static_cast<int64_t>(a.B) * a.chunks, [&](size_t i, float s) {
    const size_t h = i / (static_cast<size_t>(K + 1) * a.d);
    const int in = static_cast<int>(i - h * (K + 1) * a.d);
    if (in < K * a.d) a.dw[h * K * a.d + in] = s;
    else a.dbias[h * a.d + (in - K * a.d)] = s;
  });
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
