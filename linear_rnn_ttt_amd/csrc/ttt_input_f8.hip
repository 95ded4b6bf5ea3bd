// ttt_input_f8.hip -- the input side of a TTT layer from 8-bit operands for
// gfx950: x and the stacked weights W_in as e4m3 bytes with one scale per row,
//     Y[m, n] = sx[m] sw[n] sum_j x[m, j] w[n, j]
// with the columns of ttt_input.hip (q, k, v of every head, then the gates)
// and its outputs: q, k, v bf16 in [B, H, T, 64] and eta = eta_base /
// (1 + exp(-(y + b_eta))) fp32.
//
// Tiling: D is walked in steps of 128 bytes through two LDS buffers, the next
// step's copies (global_load_lds) on their way while one is worked on.  The
// 16-byte chunks of a row are swizzled so that a fragment's rows spread over the
// banks.  One 16x16x128 product takes chunks g and g + 4 of its rows (the same
// for both operands, so the contraction's order does not matter).  D is a
// multiple of 64: an odd last half step fetches its first half twice and
// multiplies the second copy by zero.  With tiles for most compute units a
// workgroup takes 256 x 256 outputs at a time (f8_stream), else 128 x 128
// (f8_tile).
//
// What bounds it (B4 T8192 D2048 H32, 396 us, 2.1 PFLOP/s; a library product of
// this size reaches 3.0): the products alone take 288 us of every 2048 of D,
// where reads, products and barriers of the two groups of waves alternate, and
// the 403 MB of outputs some 70 us beside them.
//
// The same columns come a second way, f8_block: 64 x 32 outputs per workgroup,
// each wave a share of D read from memory straight into fragments, the waves'
// sums joined through LDS.  It makes the gates (below), and all columns where
// few rows (a token per stream) would leave most compute units without a tile
// and make every one wait for D / 128 round trips.
//
// Precision.  The 8-bit matrix product adds its exact products with fewer bits
// than fp32 (measured: 1.4e-5 of a sum's typical size, in the 128- and the
// 32-deep form alike), far below the bf16 rounding of q, k, v but not below
// that of an fp32 gate: gates are summed by 16x16x32 bf16 products (widening
// e4m3 to bf16 is exact), whose sums are fp32.  They have workgroups of their
// own, the launch's first: 1 column in 193, and a branch for them inside the
// tile's loop spoils its schedule (594 -> 432 us at B4 T8192 D2048 H32 with
// 256 x 256 tiles).  They take no measurable time there.
//
// Tile order: each of the 8 XCDs (consecutive workgroups land on them in turn)
// takes a contiguous run of tiles.
#include <type_traits>

#include "ttt_block.hpp"
#include "ttt_device.hpp"

#define TTT_LDS __attribute__((address_space(3)))

namespace tttk {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int BK = 128, HD = 64, XCDS = 8, CUS = 256, GM = 4;

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

// The product of two steps of 128 bytes in bf16.
__device__ __forceinline__ f32x4 mfma_widened(u32x4 a0, u32x4 a1, u32x4 b0, u32x4 b1, f32x4 c) {
  c = mfma32(widen(a0.x, a0.y), widen(b0.x, b0.y), c);
  c = mfma32(widen(a0.z, a0.w), widen(b0.z, b0.w), c);
  c = mfma32(widen(a1.x, a1.y), widen(b1.x, b1.y), c);
  return mfma32(widen(a1.z, a1.w), widen(b1.z, b1.w), c);
}

__device__ __forceinline__ uint16_t* head_out(const InputF8Args& a, int col, int* h) {
  const int which = col / (a.H * HD);
  *h = (col / HD) % a.H;
  return which == 0 ? static_cast<uint16_t*>(a.q)
                    : which == 1 ? static_cast<uint16_t*>(a.k) : static_cast<uint16_t*>(a.v);
}

// WM x WN waves of 16 MI rows x 64 columns.
template <int WM, int WN, int MI>
struct F8Tile {
  static constexpr int BM = WM * MI * 16, BN = WN * 64, NT = WM * WN * 64;
  static constexpr int COPIES_A = BM / 8 / (WM * WN), COPIES_B = BN / 8 / (WM * WN);
  uint8_t a[2][BM][BK];
  uint8_t b[2][BN][BK];
};

template <int WM, int WN, int MI>
__device__ __forceinline__ void f8_tile(const InputF8Args& a, F8Tile<WM, WN, MI>& L, int id) {
  using Tile = F8Tile<WM, WN, MI>;
  constexpr int BM = Tile::BM, BN = Tile::BN, CA = Tile::COPIES_A, CB = Tile::COPIES_B;
  const int M = a.B * a.T, N = 3 * a.H * HD, D = a.D;   // without the gates
  const int ntm = (M + BM - 1) / BM, ntn = (N + BN - 1) / BN, nt = ntm * ntn;
  const int per = (nt + XCDS - 1) / XCDS;
  const int tile = (id % XCDS) * per + id / XCDS;
  if (tile >= nt) return;
  const int grp = tile / (GM * ntn), within = tile % (GM * ntn);
  const int gsize = min(GM, ntm - grp * GM);
  const int m0 = (grp * GM + within % gsize) * BM, n0 = (within / gsize) * BN;

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int g = lane >> 4, c = lane & 15;
  const int wm = wave / WN, wn = wave % WN;

  // copies: 8 rows of 128 bytes per wave instruction, lane l landing at byte
  // 16 l; rows past M and N are clamped (valid memory, results unused)
  const int cr = lane >> 3, cq = lane & 7;
  const uint8_t* xg = static_cast<const uint8_t*>(a.x) + static_cast<size_t>(m0) * D;
  const uint8_t* wg = static_cast<const uint8_t*>(a.w) + static_cast<size_t>(n0) * D;
  uint32_t oa[CA], ob[CB];   // within the tile's rows
#pragma unroll
  for (int j = 0; j < CA; ++j)
    oa[j] = static_cast<uint32_t>(min(8 * (wave + WM * WN * j) + cr, M - 1 - m0)) * D;
#pragma unroll
  for (int j = 0; j < CB; ++j)
    ob[j] = static_cast<uint32_t>(min(8 * (wave + WM * WN * j) + cr, N - 1 - n0)) * D;
  // the chunk that belongs in this lane's slot (rows of a block: r % 8 = cr),
  // and the one fetched in its place in a half step (chunks 4-7 lie past the row's end)
  const int full = 16 * (cq ^ cr), half = 16 * ((cq ^ cr) & 3);
  const int steps = (D + BK - 1) / BK;
  const bool odd = D % BK != 0;
  auto issue = [&](int s) {
    const int buf = s & 1;
    const uint32_t at = s * BK + (odd && s == steps - 1 ? half : full);
#pragma unroll
    for (int j = 0; j < CA; ++j)
      __builtin_amdgcn_global_load_lds(
          xg + (oa[j] + at), (TTT_LDS void*)&L.a[buf][8 * (wave + WM * WN * j)][0], 16, 0, 0);
#pragma unroll
    for (int j = 0; j < CB; ++j)
      __builtin_amdgcn_global_load_lds(
          wg + (ob[j] + at), (TTT_LDS void*)&L.b[buf][8 * (wave + WM * WN * j)][0], 16, 0, 0);
  };

  f32x4 acc[MI][4];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int nb0 = n0 + 64 * wn;
  const u32x4 zero = {0, 0, 0, 0};
  u32x4 a0[MI], a1[MI], b0[4], b1[4];
  auto read = [&](int buf, auto whole) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint8_t* row = L.b[buf][64 * wn + 16 * j + c];
      b0[j] = chunk(row, g, c);
      b1[j] = whole ? chunk(row, g + 4, c) : zero;
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const uint8_t* row = L.a[buf][16 * MI * wm + 16 * i + c];
      a0[i] = chunk(row, g, c);
      a1[i] = whole ? chunk(row, g + 4, c) : zero;
    }
  };
  auto multiply = [&] {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = mfma_f8(a0[i], a1[i], b0[j], b1[j], acc[i][j]);
  };
  auto landed = [] { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); };
  // One wave per SIMD and two workgroups per compute unit: the other
  // workgroup's products run beside this one's reads.
  auto step = [&](int s, auto whole) {
    if (s + 1 < steps) issue(s + 1);
    read(s & 1, whole);
    multiply();
    landed();
    lds_barrier_copies_in_flight();
  };
  issue(0);
  landed();
  lds_barrier_copies_in_flight();
  const int whole = odd ? steps - 1 : steps;
  for (int s = 0; s < whole; ++s) step(s, std::true_type{});
  if (odd) step(whole, std::false_type{});

  // epilogue: accumulator (i, j) holds row m0 + 16 (MI wm + i) + 4 g + r, column nb0 + 16 j + c
  const int T = a.T, H = a.H;
  float sw[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) sw[j] = a.w_scale[min(nb0 + 16 * j + c, N - 1)];
  if (nb0 >= N) return;
  // 64 output rows of 128 bytes at a time, staged through the wave's own 8 KB of LDS
  static_assert(sizeof(Tile) >= static_cast<size_t>(WM) * WN * 8192, "staging fits");
  uint16_t (*W)[64] = reinterpret_cast<uint16_t (*)[64]>(&L.a[0][0][0]) + 64 * wave;
  int h;
  uint16_t* out = head_out(a, nb0, &h);
#pragma unroll
  for (int part = 0; part < MI / 4; ++part) {
    const int mp = m0 + 16 * (MI * wm + 4 * part);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * i + 4 * g + r;
        const float sx = a.x_scale[min(mp + row, M - 1)];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          W[row][(16 * j + c) ^ ((row & 7) << 3)] = static_cast<uint16_t>(
              pack_bf16(acc[4 * part + i][j][r] * (sx * sw[j]), 0.f) & 0xffffu);
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the wave's own rows, in order
    const int col = 8 * (lane & 7);
#pragma unroll
    for (int pass = 0; pass < 8; ++pass) {
      const int row = (lane >> 3) + 8 * pass;
      const int m = mp + row;
      const u32x4 val = *reinterpret_cast<const u32x4*>(&W[row][col ^ ((row & 7) << 3)]);
      if (m < M) {
        const int b = m / T, t = m - b * T;
        *reinterpret_cast<u32x4*>(out + ((static_cast<size_t>(b) * H + h) * T + t) * HD + col) =
            val;
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read before the next part's writes
  }
}

// Many rows: a workgroup per compute unit takes 256 x 256 tiles one after
// another, eight waves of 128 rows x 64 columns (one head), and its stream of
// steps runs on across tiles, so that a tile's first steps land while the last
// one's products and stores are under way.
//
// The products are W_in x^T: with rows 32 (i / 2) + 8 (c / 4) + 4 (i % 2) + c % 4
// of the head in block i, a lane holds features 8 g .. 8 g + 7 and 32 + 8 g .. of
// one token, and its two stores of 16 bytes fill half a 128-byte row each with
// those of three other lanes.
struct F8Stream {
  static constexpr int BM = 256, BN = 256, NT = 512, GRID = CUS;
  uint8_t a[2][BM][BK];
  uint8_t b[2][BN][BK];
  // scales of the workgroup's last tiles: with one step a tile, the second
  // tile behind one is fetched while the first is being stored
  float sx[4][BM], sw[4][BN];
};

__device__ __forceinline__ void f8_stream(const InputF8Args& a, F8Stream& L, int id) {
  constexpr int BM = F8Stream::BM, BN = F8Stream::BN, MI = 8;
  const int M = a.B * a.T, N = 3 * a.H * HD, D = a.D;   // without the gates
  const int ntm = (M + BM - 1) / BM, ntn = (N + BN - 1) / BN, nt = ntm * ntn;
  // groups of as many columns of tiles as have 3 MB of weights, which stay in an
  // XCD's L2 while the rows of x pass by
  const int cols = max(1, (3 << 20) / (BN * D));
  // each XCD a contiguous run of tiles, its 32 workgroups taking them in turn
  const int per = (nt + XCDS - 1) / XCDS, run = (id % XCDS) * per;
  const int run_end = min(run + per, nt), stride = F8Stream::GRID / XCDS;
  const int first = run + id / XCDS;
  if (first >= run_end) return;
  const int steps = (D + BK - 1) / BK;
  const bool odd = D % BK != 0;
  const int total = ((run_end - first - 1) / stride + 1) * steps;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, c = lane & 15, wm = wave >> 2, wn = wave & 3;
  const bool second = wm == 1;
  auto rows_at = [&](int tile, int* m0, int* n0) {
    const int grp = tile / (cols * ntm), within = tile - grp * (cols * ntm);
    const int gsize = min(cols, ntn - grp * cols);
    const int row = within / gsize;
    *m0 = __builtin_amdgcn_readfirstlane(row * BM);
    *n0 = __builtin_amdgcn_readfirstlane((grp * cols + within - row * gsize) * BN);
  };

  // copies: 8 rows of 128 bytes per wave instruction, lane l landing at byte
  // 16 l, i.e. in slot cq of row cr, which holds chunk cq ^ (the row's swizzle):
  // r % 8 for x, and for W_in r % 4 + 4 (r / 8 % 2), as its fragments' rows run
  const int cr = lane >> 3, cq = lane & 7;
  const int qa = cq ^ cr, qb = cq ^ ((cr & 3) | (wave & 1) << 2);
  const uint8_t *xg = nullptr, *wg = nullptr;
  int last_x = 0, last_w = 0;   // rows of the tile that exist, less one
  int next_tile = first, next_step = 0, issued = 0;
  auto row_of = [&](int j, int last) {
    return static_cast<uint32_t>(min(8 * (wave + 8 * j) + cr, last)) * static_cast<uint32_t>(D);
  };
  auto issue = [&] {
    if (next_step == 0) {   // a new tile: its rows (clamped at the ends) and scales
      int m0, n0;
      rows_at(next_tile, &m0, &n0);
      xg = static_cast<const uint8_t*>(a.x) + static_cast<size_t>(m0) * D;
      wg = static_cast<const uint8_t*>(a.w) + static_cast<size_t>(n0) * D;
      last_x = M - 1 - m0;
      last_w = N - 1 - n0;
      const int buf = ((next_tile - first) / stride) & 3;
      const float* from = wm == 0 ? a.x_scale + min(m0 + 64 * wn + lane, M - 1)
                                  : a.w_scale + min(n0 + 64 * wn + lane, N - 1);
      float* to = wm == 0 ? &L.sx[buf][64 * wn] : &L.sw[buf][64 * wn];
      __builtin_amdgcn_global_load_lds(from, (TTT_LDS void*)to, 4, 0, 0);
    }
    const bool short_step = odd && next_step == steps - 1;   // chunks 4-7 lie past the row's end
    const uint32_t at = next_step * BK;
    const uint32_t ka = at + 16 * (short_step ? qa & 3 : qa);
    const uint32_t kb = at + 16 * (short_step ? qb & 3 : qb);
    const int buf = issued & 1;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      __builtin_amdgcn_global_load_lds(xg + (row_of(j, last_x) + ka),
                                       (TTT_LDS void*)&L.a[buf][8 * (wave + 8 * j)][0], 16, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      __builtin_amdgcn_global_load_lds(wg + (row_of(j, last_w) + kb),
                                       (TTT_LDS void*)&L.b[buf][8 * (wave + 8 * j)][0], 16, 0, 0);
    ++issued;
    if (++next_step == steps) {
      next_step = 0;
      next_tile += stride;
    }
  };

  f32x4 acc[4][MI];
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < MI; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  u32x4 x0[MI], x1[MI], w0[4], w1[4];
  auto read = [&](int buf) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 64 * wn + 32 * (i >> 1) + 8 * (c >> 2) + 4 * (i & 1) + (c & 3);
      const int sw = (c & 3) | (((c >> 2) & 1) << 2);
      w0[i] = *reinterpret_cast<const u32x4*>(&L.b[buf][r][(g ^ sw) << 4]);
      w1[i] = *reinterpret_cast<const u32x4*>(&L.b[buf][r][((g + 4) ^ sw) << 4]);
    }
#pragma unroll
    for (int j = 0; j < MI; ++j) {
      const uint8_t* row = L.a[buf][128 * wm + 16 * j + c];
      x0[j] = chunk(row, g, c);
      x1[j] = chunk(row, g + 4, c);
    }
  };
  auto drop_second_half = [&] {
    const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) w1[i] = zero;
#pragma unroll
    for (int j = 0; j < MI; ++j) x1[j] = zero;
  };
  auto store_tile = [&](int tile) {   // whether it made exactly 2 MI stores
    int m0, n0;
    rows_at(tile, &m0, &n0);
    const int buf = ((tile - first) / stride) & 3, nb0 = n0 + 64 * wn;
    if (nb0 >= N) return false;
    f32x4 sw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sw[i] = *reinterpret_cast<const f32x4*>(
          &L.sw[buf][64 * wn + 32 * (i >> 1) + 8 * g + 4 * (i & 1)]);
    int h;
    uint16_t* out = head_out(a, nb0, &h);
    const uint32_t T = a.T;
    auto put = [&](int j, auto whole) {
      const uint32_t in = 128 * wm + 16 * j + c, m = m0 + in;
      const float sx = L.sx[buf][in];
      const uint32_t b = m / T, t = m - b * T;
      uint16_t* p = out + ((static_cast<size_t>(b) * a.H + h) * T + t) * HD + 8 * g;
      u32x4 v[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4 y = acc[i][j] * (sw[i] * sx);
        v[i >> 1][2 * (i & 1)] = pack_bf16(y[0], y[1]);
        v[i >> 1][2 * (i & 1) + 1] = pack_bf16(y[2], y[3]);
      }
      if (whole || m < static_cast<uint32_t>(M)) {
        // past the L2, which holds what the products read (411 -> 396 us)
        __builtin_nontemporal_store(v[0], reinterpret_cast<u32x4*>(p));
        __builtin_nontemporal_store(v[1], reinterpret_cast<u32x4*>(p + 32));
      }
    };
    if (m0 + BM <= M) {
#pragma unroll
      for (int j = 0; j < MI; ++j) put(j, std::true_type{});
      return true;
    }
#pragma unroll
    for (int j = 0; j < MI; ++j) put(j, std::false_type{});
    return false;
  };
  // The wave's copies have landed.  Stores are counted with them, in the order
  // of issue: where exactly the 16 of a whole tile follow the copies, they are
  // left under way.
  auto landed = [](bool stores) {
    if (stores) asm volatile("s_waitcnt vmcnt(16)" ::: "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  };
  // a barrier that products do not cross either
  auto meet = [] {
    __builtin_amdgcn_sched_barrier(0);
    lds_barrier_copies_in_flight();
    __builtin_amdgcn_sched_barrier(0);
  };

  // Two waves per SIMD, w and w + 4, half a step apart: while one group reads
  // its fragments, the other's products run.  With phases between barriers,
  // the first group reads step s in phase 2 s and multiplies in 2 s + 1, the
  // second a phase later; step s + 2 may replace s in its buffer from phase
  // 2 s + 2 on, and has to have landed by the end of 2 s + 3.
  clear();
  issue();
  if (total > 1) issue();
  landed(false);
  meet();
  if (second) meet();
  int tile = first, in_tile = 0;
  bool stores = false;   // behind the last copies
  for (int s = 0; s < total; ++s) {
    if (!second) {
      if (s > 0 && s + 1 < total) issue();
      stores = false;
    }
    read(s & 1);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (second) landed(stores);
    meet();
    if (second) {
      if (s + 2 < total) issue();
      stores = false;
    }
    const bool last = ++in_tile == steps;
    if (odd && last) drop_second_half();
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int j = 0; j < MI; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i][j] = mfma_f8(w0[i], w1[i], x0[j], x1[j], acc[i][j]);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    if (last) {
      stores = store_tile(tile);
      clear();
      in_tile = 0;
      tile += stride;
    }
    if (!second) landed(stores);
    meet();
  }
  if (!second) meet();
}

// 64 x 32 outputs, wave w of W taking steps w, w + W, ... of D.  GATE: the
// columns are gates (n0 counts from the first).
constexpr int FM = 64, FN = 32;

template <int W>
using F8Part = f32x4[W][8][64];

template <int W, bool GATE>
__device__ __forceinline__ void f8_block(const InputF8Args& a, F8Part<W>& part, int m0, int n0) {
  const int M = a.B * a.T, QKV = 3 * a.H * HD, N = GATE ? a.H : QKV, D = a.D;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  const int first = GATE ? QKV : 0;
  const uint8_t* pa[4];
  const uint8_t* pb[2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    pa[i] = static_cast<const uint8_t*>(a.x) +
            static_cast<size_t>(min(m0 + 16 * i + c, M - 1)) * D + 16 * g;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    pb[j] = static_cast<const uint8_t*>(a.w) +
            static_cast<size_t>(first + min(n0 + 16 * j + c, N - 1)) * D + 16 * g;
  f32x4 acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const u32x4 zero = {0, 0, 0, 0};
  for (int k = BK * wave; k < D; k += BK * W) {
    const bool whole = k + BK <= D;   // else the last 64 bytes
    u32x4 a0[4], a1[4], b0[2], b1[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a0[i] = *reinterpret_cast<const u32x4*>(pa[i] + k);
      a1[i] = whole ? *reinterpret_cast<const u32x4*>(pa[i] + k + 64) : zero;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      b0[j] = *reinterpret_cast<const u32x4*>(pb[j] + k);
      b1[j] = whole ? *reinterpret_cast<const u32x4*>(pb[j] + k + 64) : zero;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (!GATE) acc[i][j] = mfma_f8(a0[i], a1[i], b0[j], b1[j], acc[i][j]);
        else acc[i][j] = mfma_widened(a0[i], a1[i], b0[j], b1[j], acc[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) part[wave][2 * i + j][lane] = acc[i][j];
  __syncthreads();
  // wave w joins blocks w, w + W, ...: row block i / 2, column block i % 2
  for (int i = wave; i < 8; i += W) {
    f32x4 sum = part[0][i][lane];
#pragma unroll
    for (int k = 1; k < W; ++k) sum += part[k][i][lane];
    const int col = n0 + 16 * (i & 1) + c;
    if (col >= N) continue;
    const float sw = a.w_scale[first + col];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int m = m0 + 16 * (i >> 1) + 4 * g + r;
      if (m >= M) break;
      const int b = m / a.T, t = m - b * a.T;
      const float y = sum[r] * (a.x_scale[m] * sw);
      if constexpr (GATE) {
        a.eta[(static_cast<size_t>(b) * a.H + col) * a.T + t] =
            a.eta_base * sigmoid(y + a.b_eta[col]);
      } else {
        int h;
        uint16_t* out = head_out(a, col, &h);
        out[((static_cast<size_t>(b) * a.H + h) * a.T + t) * HD + col % HD] =
            static_cast<uint16_t>(pack_bf16(y, 0.f) & 0xffffu);
      }
    }
  }
}

// Workgroups of the gates of `rows` rows and H heads.
__host__ __device__ inline int gate_blocks(int rows, int H) {
  return ((rows + FM - 1) / FM) * ((H + FN - 1) / FN);
}

// The bodies are device functions: the host pass leaves a kernel template that
// holds the 16-byte global_load_lds without its launch stub.
template <int W>
__device__ __forceinline__ bool gate_role(const InputF8Args& a, char* smem, int* id) {
  const int blocks = gate_blocks(a.B * a.T, a.H);
  const int gates = (blocks + XCDS - 1) / XCDS * XCDS;
  if (*id >= gates) {
    *id -= gates;
    return false;
  }
  if (*id < blocks) {
    const int cols = (a.H + FN - 1) / FN;
    f8_block<W, true>(a, *reinterpret_cast<F8Part<W>*>(smem), *id / cols * FM, *id % cols * FN);
  }
  return true;
}

__global__ __launch_bounds__(F8Stream::NT) void ttt_input_f8_k(InputF8Args a) {
  static_assert(sizeof(F8Stream) >= sizeof(F8Part<8>), "the gates' sums fit");
  __shared__ alignas(16) char smem[sizeof(F8Stream)];
  int id = blockIdx.x;
  if (!gate_role<8>(a, smem, &id))
    f8_stream(a, *reinterpret_cast<F8Stream*>(smem), id);
}

using F8Mid = F8Tile<2, 2, 4>;

__global__ __launch_bounds__(F8Mid::NT) void ttt_input_f8_mid_k(InputF8Args a) {
  static_assert(sizeof(F8Mid) >= sizeof(F8Part<4>), "the gates' sums fit");
  __shared__ alignas(16) char smem[sizeof(F8Mid)];
  int id = blockIdx.x;
  if (!gate_role<4>(a, smem, &id))
    f8_tile<2, 2, 4>(a, *reinterpret_cast<F8Mid*>(smem), id);
}

__global__ __launch_bounds__(512) void ttt_input_f8_few_k(InputF8Args a) {
  __shared__ F8Part<8> part;
  const int gates = gate_blocks(a.B * a.T, a.H), id = blockIdx.x;
  if (id < gates) {
    const int cols = (a.H + FN - 1) / FN;
    f8_block<8, true>(a, part, id / cols * FM, id % cols * FN);
  } else {
    const int cols = 3 * a.H * HD / FN;
    f8_block<8, false>(a, part, (id - gates) / cols * FM, (id - gates) % cols * FN);
  }
}

}  // namespace

hipError_t launch_input_f8(const InputF8Args& a, hipStream_t stream) {
  const int64_t M = static_cast<int64_t>(a.B) * a.T, N = 3 * static_cast<int64_t>(a.H) * HD;
  auto tiles = [&](int64_t bm, int64_t bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
  const int64_t gates = gate_blocks(static_cast<int>(M), a.H);
  const int64_t padded = (gates + XCDS - 1) / XCDS * XCDS;
  // Measured (us; 64 x 32 blocks, 128 x 128 tiles, 256 x 256 tiles):
  //   D 2048, 32 heads: 64 rows (192 blocks) 9.1 / 13.5, 128 rows (384) 15.8 / 13.7;
  //   D 768, 12 heads: 128 rows (144 blocks) 5.3 / 7.9, 256 rows (288) 8.7 / 8.1:
  //   blocks while one round of the compute units has them all;
  //   D 2048, 32 heads: 1024 rows (96 large tiles) 23.3 / 33.3, 1536 (144) 34.2 / 33.4,
  //   2048 (192) 37.3 / 33.6, 4096 (384) 68 / 62; D 768, 12 heads: 4096 rows (144)
  //   17.8 / 16.4, 7168 (252) 27.2 / 21.5, 16384 (576) 52.6 / 53.0: large tiles from
  //   144 on.
  if (tiles(FM, FN) <= CUS) {
    hipLaunchKernelGGL(ttt_input_f8_few_k, dim3(static_cast<uint32_t>(gates + tiles(FM, FN))),
                       dim3(512), 0, stream, a);
  } else if (tiles(F8Stream::BM, F8Stream::BN) >= 144) {
    hipLaunchKernelGGL(ttt_input_f8_k, dim3(static_cast<uint32_t>(padded + F8Stream::GRID)),
                       dim3(F8Stream::NT), 0, stream, a);
  } else {
    const int64_t nt = (tiles(F8Mid::BM, F8Mid::BN) + XCDS - 1) / XCDS * XCDS;
    hipLaunchKernelGGL(ttt_input_f8_mid_k, dim3(static_cast<uint32_t>(padded + nt)),
                       dim3(F8Mid::NT), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace tttk
