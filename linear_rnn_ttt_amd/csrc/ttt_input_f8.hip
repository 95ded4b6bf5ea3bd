// ttt_input_f8.hip -- the input side of a TTT layer from 8-bit operands for
// gfx950: x and the stacked weights W_in as e4m3 bytes with one scale per row,
//     Y[m, n] = sx[m] sw[n] sum_j x[m, j] w[n, j]
// with the columns of ttt_input.hip (q, k, v of every head, then the gates)
// and its outputs: q, k, v bf16 in [B, H, T, 64] and eta = eta_base /
// (1 + exp(-(y + b_eta))) fp32.
//
// Tiling: 256 x 128 outputs per workgroup, 8 waves of 64 x 64.  D is walked in
// steps of 128 bytes through three LDS buffers that global_load_lds fills two
// steps ahead; the 16-byte chunk q of row r sits at chunk q ^ (r % 8).  One
// 16x16x128 product takes chunks g and g + 4 of its rows (the same for both
// operands, so the contraction's order does not matter).  D is a multiple of
// 64: an odd last half step fetches its first half twice and multiplies the
// second copy by zero.
//
// Precision.  The 8-bit matrix product adds its 128 exact products with fewer
// bits than fp32 (measured: 2e-5 of a sum's typical size), far below the bf16
// rounding of q, k, v but not below that of an fp32 gate: the waves of the
// gate columns widen their operands to bf16 (exact) and use the 16x16x32 bf16
// product, which sums in fp32.  They are 1 column block in 49 at H = 32.
//
// Tile order over the 8 XCDs as in ttt_input.hip.
#include "ttt_block.hpp"
#include "ttt_device.hpp"

#define TTT_LDS __attribute__((address_space(3)))

namespace tttk {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int BM = 256, BN = 128, BK = 128, NT = 512, HD = 64, XCDS = 8, GM = 4;

struct F8Lds {
  uint8_t a[3][BM][BK];
  uint8_t b[3][BN][BK];
};

__device__ __forceinline__ float sigmoid(float y) { return 1.0f / (1.0f + expf(-y)); }

__device__ __forceinline__ u32x4 chunk(const uint8_t* row, int q, int r) {
  return *reinterpret_cast<const u32x4*>(row + ((q ^ (r & 7)) << 4));
}

__device__ __forceinline__ f32x4 mfma_f8(u32x4 a0, u32x4 a1, u32x4 b0, u32x4 b1, f32x4 c) {
  const i32x8 a = {static_cast<int>(a0.x), static_cast<int>(a0.y), static_cast<int>(a0.z),
                   static_cast<int>(a0.w), static_cast<int>(a1.x), static_cast<int>(a1.y),
                   static_cast<int>(a1.z), static_cast<int>(a1.w)};
  const i32x8 b = {static_cast<int>(b0.x), static_cast<int>(b0.y), static_cast<int>(b0.z),
                   static_cast<int>(b0.w), static_cast<int>(b1.x), static_cast<int>(b1.y),
                   static_cast<int>(b1.z), static_cast<int>(b1.w)};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// Eight e4m3 (two words) as bf16: exact.
__device__ __forceinline__ u32x4 widen(uint32_t lo, uint32_t hi) {
  u32x4 r;
  f32x2 v = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(lo), false);
  r.x = pack_bf16(v.x, v.y);
  v = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(lo), true);
  r.y = pack_bf16(v.x, v.y);
  v = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(hi), false);
  r.z = pack_bf16(v.x, v.y);
  v = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(hi), true);
  r.w = pack_bf16(v.x, v.y);
  return r;
}

__global__ __launch_bounds__(NT) void ttt_input_f8_k(InputF8Args a) {
  __shared__ F8Lds L;
  const int M = a.B * a.T, N = 3 * a.H * HD + a.H, D = a.D;
  const int ntm = (M + BM - 1) / BM, ntn = (N + BN - 1) / BN, nt = ntm * ntn;
  const int per = (nt + XCDS - 1) / XCDS;
  const int tile = (blockIdx.x % XCDS) * per + blockIdx.x / XCDS;
  if (tile >= nt) return;
  const int grp = tile / (GM * ntn), within = tile % (GM * ntn);
  const int gsize = min(GM, ntm - grp * GM);
  const int m0 = (grp * GM + within % gsize) * BM, n0 = (within / gsize) * BN;

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int g = lane >> 4, c = lane & 15;
  const int wm = wave >> 1, wn = wave & 1;

  // copies: as in ttt_input.hip, 8 rows of 128 bytes per wave instruction;
  // rows past M and N are clamped (valid memory, results unused)
  const int cr = lane >> 3, cq = lane & 7;
  const uint8_t* xg = static_cast<const uint8_t*>(a.x);
  const uint8_t* wg = static_cast<const uint8_t*>(a.w);
  const uint8_t* pa[4];
  const uint8_t* pb[2];
  // chunk fetched by this lane (rows of a block: r % 8 = cr), and the one
  // that takes its place in a half step (chunks 4-7 lie past the row's end)
  const int full = 16 * (cq ^ cr), half = 16 * ((cq ^ cr) & 3);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    pa[j] = xg + static_cast<size_t>(min(m0 + 8 * (wave + 8 * j) + cr, M - 1)) * D;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    pb[j] = wg + static_cast<size_t>(min(n0 + 8 * (wave + 8 * j) + cr, N - 1)) * D;
  const int steps = (D + BK - 1) / BK;
  const bool odd = D % BK != 0;
  auto issue = [&](int buf, int step) {
    const int s = min(step, steps - 1);   // past the end: the last step again
    const int at = s * BK + (odd && s == steps - 1 ? half : full);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      __builtin_amdgcn_global_load_lds(pa[j] + at, (TTT_LDS void*)&L.a[buf][8 * (wave + 8 * j)][0],
                                       16, 0, 0);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      __builtin_amdgcn_global_load_lds(pb[j] + at, (TTT_LDS void*)&L.b[buf][8 * (wave + 8 * j)][0],
                                       16, 0, 0);
  };

  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int QKV = 3 * a.H * HD;
  const int nb0 = n0 + 64 * wn;
  const bool gate = nb0 >= QKV;             // of the wave; its 64 columns are one kind
  const u32x4 zero = {0, 0, 0, 0};
  auto compute = [&](int buf, bool whole) {
    u32x4 a0[4], a1[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* row = L.a[buf][64 * wm + 16 * i + c];
      a0[i] = chunk(row, g, c);
      a1[i] = whole ? chunk(row, g + 4, c) : zero;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint8_t* row = L.b[buf][64 * wn + 16 * j + c];
      const u32x4 b0 = chunk(row, g, c);
      const u32x4 b1 = whole ? chunk(row, g + 4, c) : zero;
      if (!gate) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i][j] = mfma_f8(a0[i], a1[i], b0, b1, acc[i][j]);
      } else if (nb0 + 16 * j < N) {
        const u32x4 w0 = widen(b0.x, b0.y), w1 = widen(b0.z, b0.w);
        const u32x4 w2 = widen(b1.x, b1.y), w3 = widen(b1.z, b1.w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[i][j] = mfma32(widen(a0[i].x, a0[i].y), w0, acc[i][j]);
          acc[i][j] = mfma32(widen(a0[i].z, a0[i].w), w1, acc[i][j]);
          acc[i][j] = mfma32(widen(a1[i].x, a1[i].y), w2, acc[i][j]);
          acc[i][j] = mfma32(widen(a1[i].z, a1[i].w), w3, acc[i][j]);
        }
      }
    }
  };

  issue(0, 0);
  issue(1, 1);
  asm volatile("s_waitcnt vmcnt(6)" ::: "memory");
  lds_barrier_copies_in_flight();
  int cur = 0;
  for (int s = 0; s < steps; ++s) {
    compute(cur, !(odd && s == steps - 1));
    issue(cur == 0 ? 2 : cur - 1, s + 2);   // buffer (s + 2) % 3
    asm volatile("s_waitcnt vmcnt(6)" ::: "memory");
    lds_barrier_copies_in_flight();
    cur = cur == 2 ? 0 : cur + 1;
  }
  // the last copies (repeats of the last step) land before the LDS is reused
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  lds_barrier_copies_in_flight();

  // epilogue: accumulator (i, j) holds row m0 + 64 wm + 16 i + 4 g + r, column nb0 + 16 j + c
  const int T = a.T, H = a.H;
  float sw[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) sw[j] = a.w_scale[min(nb0 + 16 * j + c, N - 1)];
  float sx[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      sx[i][r] = a.x_scale[min(m0 + 64 * wm + 16 * i + 4 * g + r, M - 1)];
  if (!gate) {
    // 64 output rows of 128 bytes, staged through the wave's own 8 KB of LDS
    uint16_t (*W)[64] = reinterpret_cast<uint16_t (*)[64]>(&L.a[0][0][0]) + 64 * wave;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          W[16 * i + 4 * g + r][(16 * j + c) ^ (((4 * g + r) & 7) << 3)] = static_cast<uint16_t>(
              pack_bf16(acc[i][j][r] * (sx[i][r] * sw[j]), 0.f) & 0xffffu);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the wave's own rows, in order
    const int which = nb0 / (H * HD), h = (nb0 / HD) % H;
    uint16_t* out = which == 0 ? static_cast<uint16_t*>(a.q)
                               : which == 1 ? static_cast<uint16_t*>(a.k)
                                            : static_cast<uint16_t*>(a.v);
    const int col = 8 * (lane & 7);
#pragma unroll
    for (int pass = 0; pass < 8; ++pass) {
      const int row = (lane >> 3) + 8 * pass;
      const int m = m0 + 64 * wm + row;
      const u32x4 val = *reinterpret_cast<const u32x4*>(&W[row][col ^ ((row & 7) << 3)]);
      if (m < M) {
        const int b = m / T, t = m - b * T;
        *reinterpret_cast<u32x4*>(out + ((static_cast<size_t>(b) * H + h) * T + t) * HD + col) =
            val;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int m = m0 + 64 * wm + 16 * i + 4 * g + r;
        if (m >= M) continue;
        const int b = m / T, t = m - b * T;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int h = nb0 + 16 * j + c - QKV;
          if (h < H)
            a.eta[(static_cast<size_t>(b) * H + h) * T + t] =
                a.eta_base * sigmoid(acc[i][j][r] * (sx[i][r] * sw[j]) + a.b_eta[h]);
        }
      }
  }
}

}  // namespace

hipError_t launch_input_f8(const InputF8Args& a, hipStream_t stream) {
  const int64_t M = static_cast<int64_t>(a.B) * a.T, N = 3 * static_cast<int64_t>(a.H) * HD + a.H;
  const int64_t nt = ((M + BM - 1) / BM) * ((N + BN - 1) / BN);
  hipLaunchKernelGGL(ttt_input_f8_k, dim3(static_cast<uint32_t>((nt + XCDS - 1) / XCDS * XCDS)),
                     dim3(NT), 0, stream, a);
  return hipGetLastError();
}

}  // namespace tttk
