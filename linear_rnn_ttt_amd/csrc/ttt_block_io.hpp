// ttt_block_io.hpp -- 8-value vectors of the I/O types, and sums over a wave,
// for the memory-bound kernels (ttt_norm.hip, ttt_conv.hip, ttt_ssm_step).
#pragma once

#include "ttt_device.hpp"

namespace tttk {

template <bool BF16>
constexpr int kIoBytes = BF16 ? 2 : 4;

// Eight consecutive values in fp32, and back rounded once (16-byte accesses).
struct F8 {
  float v[8];
};

template <bool BF16>
struct Raw8;
template <>
struct Raw8<true> {
  u32x4 a;
};
template <>
struct Raw8<false> {
  f32x4 a, b;
};

template <bool BF16>
__device__ __forceinline__ Raw8<BF16> load8_raw(const void* p, size_t i) {
  Raw8<BF16> r;
  if constexpr (BF16) {
    r.a = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i);
  } else {
    r.a = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i);
    r.b = *reinterpret_cast<const f32x4*>(static_cast<const float*>(p) + i + 4);
  }
  return r;
}

template <bool BF16>
__device__ __forceinline__ Raw8<BF16> zero8_raw() {
  Raw8<BF16> r;
  if constexpr (BF16) {
    r.a = u32x4{0, 0, 0, 0};
  } else {
    r.a = r.b = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  return r;
}

__device__ __forceinline__ F8 widen8(const Raw8<true>& r) {
  F8 f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f.v[2 * j] = bf16_lo_to_f32(r.a[j]);
    f.v[2 * j + 1] = bf16_hi_to_f32(r.a[j]);
  }
  return f;
}
__device__ __forceinline__ F8 widen8(const Raw8<false>& r) {
  F8 f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f.v[j] = r.a[j];
    f.v[4 + j] = r.b[j];
  }
  return f;
}

template <bool BF16>
__device__ __forceinline__ F8 load8(const void* p, size_t i) {
  return widen8(load8_raw<BF16>(p, i));
}

__device__ __forceinline__ F8 load8_f32(const float* p) { return load8<false>(p, 0); }

template <bool BF16>
__device__ __forceinline__ void store8(void* p, size_t i, const F8& f) {
  if constexpr (BF16) {
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack_bf16(f.v[2 * j], f.v[2 * j + 1]);
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) = w;
  } else {
    float* o = static_cast<float*>(p) + i;
    *reinterpret_cast<f32x4*>(o) = f32x4{f.v[0], f.v[1], f.v[2], f.v[3]};
    *reinterpret_cast<f32x4*>(o + 4) = f32x4{f.v[4], f.v[5], f.v[6], f.v[7]};
  }
}

// x plus its value in another lane of the same 16-lane row.
template <int CTRL>
__device__ __forceinline__ float row_peer(float x) {
  return bitsf(static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(fbits(x)), CTRL, 0xf, 0xf, false)));
}

// Sum over the 16 lanes of a row, in every lane: neighbour swaps, then half-row
// and row mirrors.
__device__ __forceinline__ float row_sum16(float x) {
  x += row_peer<0xb1>(x);    // quad_perm 1,0,3,2
  x += row_peer<0x4e>(x);    // quad_perm 2,3,0,1
  x += row_peer<0x141>(x);   // row_half_mirror
  x += row_peer<0x140>(x);   // row_mirror
  return x;
}

// The sums of four values over the 16 lanes of a row, lane c holding that of
// x[c % 4]: neighbours exchange what the other is to sum, then lanes 4 and 8
// apart are added (half the instructions of four whole sums).
__device__ __forceinline__ float row_sums4(f32x4 x, int c) {
  const bool odd = c & 1, high = c & 2;
  const float a = (odd ? x[1] : x[0]) + row_peer<0xb1>(odd ? x[0] : x[1]);
  const float b = (odd ? x[3] : x[2]) + row_peer<0xb1>(odd ? x[2] : x[3]);
  float s = (high ? b : a) + row_peer<0x4e>(high ? a : b);
  s += row_peer<0x124>(s);   // row_ror 4
  s += row_peer<0x128>(s);   // row_ror 8
  return s;
}

// Sum over the 64 lanes, in every lane.
__device__ __forceinline__ float wave_sum(float x) { return group_sum(row_sum16(x)); }

__device__ __forceinline__ float wave_max(float x) {
  x = fmaxf(x, row_peer<0xb1>(x));
  x = fmaxf(x, row_peer<0x4e>(x));
  x = fmaxf(x, row_peer<0x141>(x));
  x = fmaxf(x, row_peer<0x140>(x));
  const auto r = __builtin_amdgcn_permlane16_swap(fbits(x), fbits(x), false, false);
  const float y = fmaxf(bitsf(r[0]), bitsf(r[1]));
  const auto q = __builtin_amdgcn_permlane32_swap(fbits(y), fbits(y), false, false);
  return fmaxf(bitsf(q[0]), bitsf(q[1]));
}

// put(i, sum over `rows` of partial[row][i]) for the columns i < n of a
// workgroup of 256 threads: 16 columns (16 blockIdx.x ..), 16 threads each,
// every thread's rows in four interleaved sums so that their loads overlap.
// The order is fixed, so the sums are the same from run to run.
template <class Put>
__device__ __forceinline__ void column_sums(const float* partial, size_t n, int64_t rows,
                                            Put put) {
  __shared__ float part[16][17];
  const int col = threadIdx.x & 15, slot = threadIdx.x >> 4;
  const size_t i = 16 * static_cast<size_t>(blockIdx.x) + col;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (i < n) {
    int64_t r = slot;
    for (; r + 112 < rows; r += 128) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = partial[(r + 16 * k) * n + i];
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k & 3] += v[k];
    }
    for (; r < rows; r += 16) s[0] += partial[r * n + i];
  }
  part[slot][col] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  if (slot == 0 && i < n) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) t += part[k][col];
    put(i, t);
  }
}

}  // namespace tttk
