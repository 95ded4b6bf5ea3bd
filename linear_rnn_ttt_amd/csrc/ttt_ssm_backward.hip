// ttt_ssm_backward.hip -- gradients of the selective state space scan for
// gfx950 (ttt_ssm.hip holds the forward and its notation).
//
// With the adjoint A_t of the state (A_T = dstate + c_T^T dy_T,
// A_t = c_t^T dy_t + exp(a dt_{t+1}) A_{t+1}), token by token:
//     dc_t = S_t dy_t,   db_t = dt_t A_t x_t,   dx_t = dt_t b_t A_t + d dy_t
//     ddt_t = b_t A_t x_t + a e_t,   da = sum dt_t e_t,   e_t = exp(a dt_t) <A_t, S_{t-1}>
// For a tile, with S the state before it, A the adjoint behind it and
// F[t, s] = exp(cum_t - cum_s) for s <= t, else 0:
//     W1 = (C B^T) F,   W2 = (dY X^T) F                    (elementwise by F)
//     dX = diag(dt) [W1^T dY + diag(tail) B A] + d dY
//     dB = diag(dt) [W2^T C + diag(tail) X A^T]
//     dC = W2 diag(dt) B + diag(head) dY S^T
//     A before the tile = exp(cum_L) A + C^T diag(head) dY
// e needs no products of its own: a decay exponent at token t scales every
// path that crosses it, so with u_t = head_t c_t S dy_t (paths from the state
// before the tile), v_s = tail_s b_s A x_s (paths to the adjoint behind it) and
// Z[t, s] = W1 W2 / F (elementwise: paths inside it),
//     e_t = exp(cum_L) <S, A> + sum_{t' >= t} u_t' + sum_{s < t} dt_s v_s
//           + sum_{t' >= t} (sum_{s < t'} Z[t', s] dt_s - dt_t' sum_{t'' > t'} Z[t'', t'])
//     ddt_t = v_t + sum_{t' >= t} Z[t', t] + a e_t
// Row and column sums of Z are taken in fp32 from the blocks as they are made,
// the sums over tokens in fp64, anew in every tile, so that no error runs along
// the sequence; u and v come from S and A in three parts, because ddt and da
// are fp32.
//
// Launches: (1) each segment of tiles walks forward from a state of zero,
// leaving the state before every tile and what the segment adds, and the
// segments behind the first walk backward for what they add to the adjoint in
// front of them; (2) the states in front of the segments and the adjoints
// behind them; (3) the gradients, each segment's tiles last to first with A
// in registers; (4) the sums of da and dd over batch and segments in order and,
// where heads share b and c, of their db and dc.
//
// In (3) a workgroup has eight waves: wave w and w + 4 share features 16 w ..
// of x (of dX^T and A; each has one half of A's rows) and rows 16 w .. (and
// 16 (w + 4) ..) of the state (of dB^T and dC^T), and each has half of the
// tile's token blocks, an early and a late one.  A reaches the other waves
// through LDS, where W1 and W2, shared out by blocks, take its place once it
// has been read: with bf16 data and N <= 64 two workgroups then fit a compute
// unit (four waves a SIMD).  W1 and W2 carry dt_s, and W1 d on its diagonal,
// so that dX, dB and dC come whole from their products; they are written by
// rows and read by rows or, transposed, by columns.
//
// At bf16, B8 H12 T2048 N64: walks 32 us (4.7 TB/s with the states of every tile
// that they write), join 7, gradients 87, sums 4.  The gradients are bound
// by the vector unit (56 % busy: splitting into parts, decays and the sums over
// Z) and by waiting between the four barriers of a tile (44 % of the waves' time);
// the matrix unit is 16 % busy, and the 278 MB that they move would take 52 us.
#include "ttt_block.hpp"
#include "ttt_block_io.hpp"
#include "ttt_ssm_tile.hpp"

namespace tttk {
namespace {

constexpr int NT = SSM_NT, P = SSM_P, GT = 512;   // GT: threads of a gradient workgroup

// ---- one walk over a segment: the states before its tiles, or its adjoint ---

template <int NI, int N>
struct WalkLds {
  static constexpr int L = kSsmTile<NI>;
  Plane<NI, L, P> x;
  Plane<NI, L, N> b;
  Tokens<L> tk[2];   // of even and odd tiles
};

// ADJ false: S over x and b, first tile to last.  ADJ true: A over dy and c,
// last to first, for the segments behind the first.
template <int NI, int N, bool ADJ>
__device__ __forceinline__ void walk(const SsmBackwardArgs& a, WalkLds<NI, N>& lds, uint32_t id) {
  constexpr int L = kSsmTile<NI>;
  const SsmArgs& f = a.f;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, c = lane & 15;
  const Place at(f, id, ADJ ? f.segs - 1 : f.segs);
  const int seg = at.seg + (ADJ ? 1 : 0);
  const size_t unit = at.unit, shared = at.shared;
  const int tiles = (f.T + L - 1) / L;
  const int first = seg * f.seg_tiles, end = min(first + f.seg_tiles, tiles), n = end - first;
  const float ah = f.a[at.h];
  const void* rows = ADJ ? a.dy : f.x;
  const void* cols = ADJ ? f.c : f.b;
  f32x4 S[N / 16];
#pragma unroll
  for (int i = 0; i < N / 16; ++i) S[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto save = [&](float* out) {
#pragma unroll
    for (int i = 0; i < N / 16; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) out[(16 * i + 4 * g + r) * P + 16 * wave + c] = S[i][r];
  };
  Fetch<NI, L, P, NT> fx;
  Fetch<NI, L, N, NT> fb;
  auto tile_of = [&](int i) { return ADJ ? end - 1 - i : first + i; };
  auto valid_of = [&](int i) { return i < n ? min(L, f.T - tile_of(i) * L) : 0; };
  auto fetch = [&](int i) {
    const int t0 = tile_of(i) * L, valid = valid_of(i);
    fx.load(row_ptr<NI>(rows, unit * f.T + t0, P), valid, tid);
    fb.load(row_ptr<NI>(cols, shared * f.T + t0, N), valid, tid);
  };
  auto steps_of = [&](int i) {
    return load_steps(f.dt + unit * f.T + tile_of(i) * L, valid_of(i), lane);
  };
  double total = 0.0;
  float step = steps_of(0);
  fetch(0);
  if (wave == 0) total = lds.tk[0].fill(step, ah, lane);
  step = steps_of(1);
  for (int i = 0; i < n; ++i) {
    fx.store(lds.x, tid);
    fb.store(lds.b, tid);
    lds_barrier();
    const Tokens<L>& tk = lds.tk[i & 1];
    fetch(i + 1);
    if (wave == 0 && i + 1 < n) total += lds.tk[(i + 1) & 1].fill(step, ah, lane);
    step = steps_of(i + 2);
    if (!ADJ && i > 0) save(a.ws_tile + (unit * tiles + first + i) * (N * P));
    if constexpr (ADJ) add_tile(S, lds.b, 0, lds.x, wave, tk.fade, tk.head, g, c);
    else add_tile(S, lds.b, 0, lds.x, wave, tk.fade, tk.into, g, c);
    lds_barrier();
  }
  if (ADJ) {
    save(a.ws_adj + (unit * f.segs + seg) * (N * P));
  } else {
    save(f.ws_state + (unit * f.segs + seg) * (N * P));
    if (tid == 0) f.ws_fade[unit * f.segs + seg] = total;
  }
}

template <int NI, int N>
__global__ __launch_bounds__(NT, 2) void ttt_ssm_bwd_walk_k(SsmBackwardArgs a) {
  __shared__ alignas(16) WalkLds<NI, N> lds;
  const uint32_t forward = static_cast<uint32_t>(a.f.B) * a.f.H * a.f.segs;
  if (blockIdx.x < forward) walk<NI, N, false>(a, lds, blockIdx.x);
  else walk<NI, N, true>(a, lds, blockIdx.x - forward);
}

// States in front of the segments (the first half of the workgroups), and
// adjoints behind them.
__global__ __launch_bounds__(NT) void ttt_ssm_bwd_join_k(SsmBackwardArgs a) {
  const SsmArgs& f = a.f;
  const bool adjoint = blockIdx.x >= gridDim.x / 2;
  const uint32_t block = adjoint ? blockIdx.x - gridDim.x / 2 : blockIdx.x;
  const JoinPlace place(f.N, block, threadIdx.x);
  const size_t unit = place.unit, at = place.at, size = static_cast<size_t>(f.N) * P;
  const double* fades = f.ws_fade + unit * f.segs;
  const float* first = adjoint ? a.dstate : f.state0;
  const f32x4 S = first ? *reinterpret_cast<const f32x4*>(first + unit * size + at)
                        : f32x4{0.f, 0.f, 0.f, 0.f};
  if (adjoint)
    join_segments(a.ws_adj + (unit * f.segs + f.segs - 1) * size + at, size, fades + f.segs - 1,
                  f.segs, f.segs - 1, -1, S);
  else
    join_segments(f.ws_state + unit * f.segs * size + at, size, fades, f.segs, f.segs - 1, 1, S);
}

// ---- the gradients ----------------------------------------------------------

template <int NI, int N>
struct GradLds {
  static constexpr int L = kSsmTile<NI>, TB = L / 16, BLOCKS = TB * (TB + 1) / 2;
  static constexpr int NM = NI == 1 ? 2 : 3;   // parts of W1 and W2, and of A for dX
  Plane<NI, L, P> x, dy;
  Plane<NI, L, N> b, c;
  union {
    Plane<3, P, N> adj;         // A behind the tile: row = feature of x, column = state row
    struct {
      Plane<NM, L, L> w1, w2;   // row = t, column = s
    };
  };
  Tokens<L> tk[2];              // of even and odd tiles
  // of even and odd tiles: u and v by the waves' state rows; sums of Z by
  // blocks and its diagonal; <S, A> by the waves' state rows
  float u[2][4][L], v[2][4][L], zrow[2][BLOCKS][16], zcol[2][BLOCKS][16], zdiag[2][L], dot[2][4];
  float before;                 // decay from the segment's start to the tile
  float dd[GT / 64];
};

template <int NI, int N>
__global__ __launch_bounds__(GT, NI == 1 && N <= 64 ? 4 : 2) void ttt_ssm_bwd_k(
    SsmBackwardArgs a) {
  using Lds = GradLds<NI, N>;
  constexpr int L = Lds::L, TB = Lds::TB, NM = Lds::NM, JN = TB / 2, NA = N / 32;
  constexpr int NB = N >= 64 ? N / 64 : 1;   // state row blocks of a wave (N = 32: waves 0, 1, 4, 5)
  __shared__ alignas(16) Lds lds;
  const SsmArgs& f = a.f;
  const int tid = threadIdx.x, lane = tid & 63, g0 = lane >> 4, c0 = lane & 15;
  const int full_wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wave = full_wave & 3, half = full_wave >> 2;
  const Place at(f, blockIdx.x, f.segs);
  const int seg = at.seg;
  const size_t unit = at.unit, shared = at.shared;
  const int tiles = (f.T + L - 1) / L;
  const int first = seg * f.seg_tiles, end = min(first + f.seg_tiles, tiles);
  const float ah = f.a[at.h], skip = f.d_skip ? f.d_skip[at.h] : 0.f;
  const bool has_rows = N >= 64 || wave < N / 16;
  auto block = [&](int jj) { return TB == 4 ? (half ? 1 + jj : 3 * jj) : half; };   // of tokens
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};

  // A behind the segment: rows 16 (half NA + i) .., features 16 wave ..
  f32x4 A[NA];
  {
    const float* from = a.ws_adj + (unit * f.segs + seg) * (N * P);
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        A[i][r] = from[(16 * (half * NA + i) + 4 * g0 + r) * P + 16 * wave + c0];
  }
  // a state by rows: row 16 (wave + 4 nb) + c, features 32 k + 16 hh + 4 g .. of lane (g, c)
  auto row_of = [&](const float* p, int nb, int k, int hh) {
    return *reinterpret_cast<const f32x4*>(p + (16 * (wave + 4 * nb) + c0) * P + 32 * k + 16 * hh +
                                           4 * g0);
  };
  const float* seg_state = f.ws_state + (unit * f.segs + seg) * (N * P);
  double rest = f.ws_fade[unit * f.segs + seg];   // log2 decay from the segment's start
  float dd_sum = 0.f;
  double da_sum = 0.0;

  Fetch<NI, L, P, GT> fx, fy;
  Fetch<NI, L, N, GT> fb, fc;
  auto valid_of = [&](int tile) { return tile >= first ? min(L, f.T - tile * L) : 0; };
  auto fetch = [&](int tile) {
    const int t0 = tile * L, valid = valid_of(tile), id = anew(tid);
    fx.load(row_ptr<NI>(f.x, unit * f.T + t0, P), valid, id);
    fy.load(row_ptr<NI>(a.dy, unit * f.T + t0, P), valid, id);
    fb.load(row_ptr<NI>(f.b, shared * f.T + t0, N), valid, id);
    fc.load(row_ptr<NI>(f.c, shared * f.T + t0, N), valid, id);
  };
  auto steps_of = [&](int tile) {
    return load_steps(f.dt + unit * f.T + tile * L, valid_of(tile), lane);
  };
  // ddt of a tile whose sums stand in LDS, and its share of da; by one wave,
  // which kept the tile's steps and its fade
  auto finish = [&](int tile, float dt, float fade) {
    const int e = tile & 1, valid = valid_of(tile);
    const int lane = anew(tid & 63);
    double after = 0.0, upto = 0.0;   // of the token: u + row - column sums of Z; dt v
    float direct = 0.f;
    if (lane < L) {
      const float us = (lds.u[e][0][lane] + lds.u[e][1][lane]) +
                       (lds.u[e][2][lane] + lds.u[e][3][lane]);
      const float vs = (lds.v[e][0][lane] + lds.v[e][1][lane]) +
                       (lds.v[e][2][lane] + lds.v[e][3][lane]);
      float row = 0.f, col = 0.f;
      const int mine = lane >> 4, in = lane & 15;
#pragma unroll
      for (int k = 0; k < TB; ++k) {
        if (k <= mine) row += lds.zrow[e][mine * (mine + 1) / 2 + k][in];
        if (k >= mine) col += lds.zcol[e][k * (k + 1) / 2 + mine][in];
      }
      after = static_cast<double>(us) + row - static_cast<double>(dt) * col;
      upto = static_cast<double>(dt) * vs;
      direct = vs + (col + lds.zdiag[e][lane]);
    }
    const double after_to = wave_scan(after), upto_to = wave_scan(upto);
    const float d = (lds.dot[e][0] + lds.dot[e][1]) + (lds.dot[e][2] + lds.dot[e][3]);
    const double ex = (last_lane(after_to) - after_to + after) + (upto_to - upto) + fade * d;
    if (lane < valid) {
      a.ddt[unit * f.T + tile * L + lane] = static_cast<float>(direct + ah * ex);
      da_sum += dt * ex;
    }
  };

  // the segment's own part of the state before a tile
  f32x4 own[NB][P / 32][2];
  auto load_own = [&](int tile) {
    const int g0 = anew((tid & 63) >> 4), c0 = anew(tid & 15);
    auto row_of = [&](const float* p, int nb, int k, int hh) {
      return *reinterpret_cast<const f32x4*>(p + (16 * (wave + 4 * nb) + c0) * P + 32 * k +
                                             16 * hh + 4 * g0);
    };
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int k = 0; k < P / 32; ++k)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)
          own[nb][k][hh] = has_rows && tile > first
                               ? row_of(a.ws_tile + (unit * tiles + tile) * (N * P), nb, k, hh)
                               : zero;
  };
  fetch(end - 1);
  load_own(end - 1);
  float step = steps_of(end - 1);
  if (full_wave == 7) {
    rest -= lds.tk[(end - 1) & 1].fill(step, ah, lane);
    if (lane == 0) lds.before = exp2_raw(static_cast<float>(rest));
  }
  step = steps_of(end - 2);
  float done_dt = 0.f, done_fade = 0.f;   // of the tile to finish
  for (int tile = end - 1; tile >= first; --tile) {
    const int t0 = tile * L, valid = valid_of(tile), e = tile & 1;
    const Tokens<L>& tk = lds.tk[e];
    int g = anew(g0), c = anew(c0);
    const int id = anew(tid);
    fx.store(lds.x, id);
    fy.store(lds.dy, id);
    fb.store(lds.b, id);
    fc.store(lds.c, id);
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      u32x2 p[3];
      split_parts<3>(A[i], p);
#pragma unroll
      for (int k = 0; k < 3; ++k)
        lds.adj.put4(k, 16 * wave + c, 16 * (half * NA + i) + 4 * g, p[k]);
    }
    lds_barrier();
    const float before = lds.before;

    // what the adjoint behind the tile and the state before it give
    g = anew(g0), c = anew(c0);
    f32x4 dx[JN], db[NB][JN], dc[NB][JN];
#pragma unroll
    for (int jj = 0; jj < JN; ++jj) {
      dx[jj] = zero;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) db[nb][jj] = dc[nb][jj] = zero;
    }
#pragma unroll
    for (int k = 0; k < N / 32; ++k) {
      const Parts<NM> ap = lds.adj.template rows<NM>(16 * wave, 32 * k, g, c);
#pragma unroll
      for (int jj = 0; jj < JN; ++jj)
        dx[jj] = mfma_parts(ap, lds.b.rows(16 * block(jj), 32 * k, g, c), dx[jj]);
    }
    f32x4 sa = zero;   // S A^T of the wave's rows: <S, A> on its diagonal
    if (has_rows) {
#pragma unroll
      for (int k = 0; k < P / 32; ++k) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          // what came in front of the segment
          f32x4 S[2] = {row_of(seg_state, nb, k, 0), row_of(seg_state, nb, k, 1)};
          const Parts<3> ar = lds.adj.cols(32 * k, 16 * (wave + 4 * nb), g, c);
#pragma unroll
          for (int jj = 0; jj < JN; ++jj)
            db[nb][jj] =
                mfma_parts(ar, lds.x.rows(16 * block(jj), 32 * k, g, c), db[nb][jj]);
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) S[hh] = S[hh] * before + own[nb][k][hh];
          const Parts<3> sp = split_frag<3>(S[0], S[1]);
          if (half == 0) sa = mfma_parts(sp, ar, sa);
#pragma unroll
          for (int jj = 0; jj < JN; ++jj)
            dc[nb][jj] =
                mfma_parts(sp, lds.dy.rows(16 * block(jj), 32 * k, g, c), dc[nb][jj]);
        }
      }
    }
    if (half == 0) {
      float dot = 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) dot += 4 * g + r == c ? sa[r] : 0.f;
      dot = wave_sum(dot);
      if (lane == 0) lds.dot[e][wave] = dot;
    }
#pragma unroll
    for (int jj = 0; jj < JN; ++jj) {
      const int t = 16 * block(jj) + c;
      const float into = tk.into[t], head = tk.head[t];
      float us = 0.f, vs = 0.f;
      if (has_rows) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int n = 16 * (wave + 4 * nb) + 4 * g;
          const f32x4 pv = lds.b.four(t, n) * db[nb][jj], pu = lds.c.four(t, n) * dc[nb][jj];
          vs += (pv[0] + pv[1]) + (pv[2] + pv[3]);
          us += (pu[0] + pu[1]) + (pu[2] + pu[3]);
          db[nb][jj] *= into;
          dc[nb][jj] *= head;
        }
      }
      dx[jj] *= into;
      us = group_sum(us) * head;
      vs = group_sum(vs) * tk.tail[t];
      if (g == 0) {
        lds.u[e][wave][t] = us;
        lds.v[e][wave][t] = vs;
      }
    }
    lds_barrier();
    fetch(tile - 1);
    load_own(tile - 1);

    // W1 and W2 block by block
    g = anew(g0), c = anew(c0);
    for (int i = full_wave; i < Lds::BLOCKS && full_wave < 6; i += 6) {   // 6, 7: see below
      int tb, sb;
      block_of(i, &tb, &sb);
      f32x4 gt = zero, xt = zero;   // rows s, columns t
#pragma unroll
      for (int k = 0; k < N / 32; ++k)
        gt = mfma_parts(lds.b.rows8(16 * sb, 32 * k, g, c), lds.c.rows8(16 * tb, 32 * k, g, c),
                        gt);
#pragma unroll
      for (int k = 0; k < P / 32; ++k)
        xt = mfma_parts(lds.x.rows8(16 * sb, 32 * k, g, c), lds.dy.rows8(16 * tb, 32 * k, g, c),
                        xt);
      const int t = 16 * tb + c, s0 = 16 * sb + 4 * g;
      const f32x4 fade = tk.fades(tb, sb, t, s0), dt = tk.steps(s0);
      const f32x4 z = gt * xt * fade;
      f32x4 w1 = gt * (fade * dt), w2 = xt * (fade * dt);
      f32x4 off = z;
      if (tb == sb) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (4 * g + r == c) {
            lds.zdiag[e][t] = z[r];
            off[r] = 0.f;
            dd_sum += xt[r];
            w1[r] += skip;
          }
      }
      float row = 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) row += off[r] * dt[r];
      const float col = row_sums4(off, c);
      if (c < 4) lds.zcol[e][i][4 * g + c] = col;
      row = group_sum(row);
      if (g == 0) lds.zrow[e][i][c] = row;
      u32x2 p[NM], q[NM];
      split_parts<NM>(w1, p);
      split_parts<NM>(w2, q);
#pragma unroll
      for (int k = 0; k < NM; ++k) {
        lds.w1.put4(k, t, s0, p[k]);
        lds.w2.put4(k, t, s0, q[k]);
      }
    }
    // the blocks above the diagonal that a product of 32 tokens meets
    if (full_wave >= 8 - JN) {
      const int t = 32 * (full_wave - (8 - JN)) + c, s0 = t - c + 16 + 4 * g;
#pragma unroll
      for (int k = 0; k < NM; ++k) {
        lds.w1.put4(k, t, s0, u32x2{0u, 0u});
        lds.w2.put4(k, t, s0, u32x2{0u, 0u});
      }
    }
    // by waves without blocks: the tile behind is finished, the one before prepared
    if (full_wave == 6) {
      if (tile < end - 1) finish(tile + 1, done_dt, done_fade);
      done_dt = lane < L ? tk.dt[lane] : 0.f;
      done_fade = tk.fade;
    }
    if (full_wave == 7 && tile > first) {
      rest -= lds.tk[e ^ 1].fill(step, ah, lane);
      if (lane == 0) lds.before = exp2_raw(static_cast<float>(rest));
    }
    step = steps_of(tile - 2);
    lds_barrier();

    // and the tile's own tokens
    g = anew(g0), c = anew(c0);
#pragma unroll
    for (int k = 0; k < L / 32; ++k) {
      const Parts<NI> yt = lds.dy.cols(32 * k, 16 * wave, g, c);
#pragma unroll
      for (int jj = 0; jj < JN; ++jj)
        if (block(jj) <= 2 * k + 1)
          dx[jj] = mfma_parts(yt, lds.w1.cols(32 * k, 16 * block(jj), g, c), dx[jj]);
      if (has_rows) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const Parts<NI> ct = lds.c.cols(32 * k, 16 * (wave + 4 * nb), g, c);
          const Parts<NI> bt = lds.b.cols(32 * k, 16 * (wave + 4 * nb), g, c);
#pragma unroll
          for (int jj = 0; jj < JN; ++jj) {
            if (block(jj) <= 2 * k + 1)
              db[nb][jj] =
                  mfma_parts(ct, lds.w2.cols(32 * k, 16 * block(jj), g, c), db[nb][jj]);
            if (block(jj) >= 2 * k)
              dc[nb][jj] =
                  mfma_parts(bt, lds.w2.rows(16 * block(jj), 32 * k, g, c), dc[nb][jj]);
          }
        }
      }
    }

    constexpr int ES = NI == 1 ? 2 : 4;
    const __amdgpu_buffer_rsrc_t out =
        rows_of(row_ptr<NI>(a.dx, unit * f.T + t0, P), valid * P * ES);
#pragma unroll
    for (int jj = 0; jj < JN; ++jj)
      store_row4<NI>(out, 16 * block(jj) + c, P, 16 * wave + 4 * g, dx[jj]);
    if (has_rows) {
      if (a.ws_db) {   // of this head alone, in fp32
        const size_t o = (unit * f.T + t0) * N;
        const __amdgpu_buffer_rsrc_t ob = rows_of(a.ws_db + o, valid * N * 4);
        const __amdgpu_buffer_rsrc_t oc = rows_of(a.ws_dc + o, valid * N * 4);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int jj = 0; jj < JN; ++jj) {
            const int t = 16 * block(jj) + c, n = 16 * (wave + 4 * nb) + 4 * g;
            store_row4<3>(ob, t, N, n, db[nb][jj]);
            store_row4<3>(oc, t, N, n, dc[nb][jj]);
          }
      } else {
        const __amdgpu_buffer_rsrc_t ob =
            rows_of(row_ptr<NI>(a.db, shared * f.T + t0, N), valid * N * ES);
        const __amdgpu_buffer_rsrc_t oc =
            rows_of(row_ptr<NI>(a.dc, shared * f.T + t0, N), valid * N * ES);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int jj = 0; jj < JN; ++jj) {
            const int t = 16 * block(jj) + c, n = 16 * (wave + 4 * nb) + 4 * g;
            store_row4<NI>(ob, t, N, n, db[nb][jj]);
            store_row4<NI>(oc, t, N, n, dc[nb][jj]);
          }
      }
    }

    // A before the tile
    g = anew(g0), c = anew(c0);
    add_tile(A, lds.c, half * NA, lds.dy, wave, tk.fade, tk.head, g, c);
    lds_barrier();
  }
  if (full_wave == 6) finish(first, done_dt, done_fade);
  if (a.dstate0 && seg == 0) {
    float* out = a.dstate0 + unit * (N * P);
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        out[(16 * (half * NA + i) + 4 * g0 + r) * P + 16 * wave + c0] = A[i][r];
  }
  // the segment's da and dd
  dd_sum = wave_sum(dd_sum);
  if (lane == 0) lds.dd[full_wave] = dd_sum;
  lds_barrier();
  if (full_wave == 6) {
    const double all = last_lane(wave_scan(da_sum));
    if (lane == 0) {
      float* out = a.ws_sums + (unit * f.segs + seg) * 2;
      float dd = 0.f;
#pragma unroll
      for (int k = 0; k < GT / 64; ++k) dd += lds.dd[k];
      out[0] = static_cast<float>(all);
      out[1] = dd;
    }
  }
}

// da[h], dd[h], by a wave: the sums of (batch, segment).
__device__ __forceinline__ void sum_head(const SsmBackwardArgs& a, int h, int lane) {
  const SsmArgs& f = a.f;
  double da = 0.0, dd = 0.0;
  const uint32_t segs = f.segs, count = static_cast<uint32_t>(f.B) * segs;   // workgroups: < 2^32
  for (uint32_t i = lane; i < count; i += 64) {
    const uint32_t b = i / segs, seg = i - b * segs;
    const f32x2 p = *reinterpret_cast<const f32x2*>(
        a.ws_sums + ((static_cast<size_t>(b) * f.H + h) * segs + seg) * 2);
    da += p[0];
    dd += p[1];
  }
  da = last_lane(wave_scan(da));
  dd = last_lane(wave_scan(dd));
  if (lane == 0) {
    a.da[h] = static_cast<float>(da);
    if (a.dd) a.dd[h] = static_cast<float>(dd);
  }
}

__host__ __device__ inline uint32_t sum_blocks(int H) { return (H + NT / 64 - 1) / (NT / 64); }

__global__ __launch_bounds__(NT) void ttt_ssm_bwd_sum_k(SsmBackwardArgs a) {
  const int h = blockIdx.x * (NT / 64) + wave_of(threadIdx.x);
  if (h < a.f.H) sum_head(a, h, threadIdx.x & 63);
}

// The same by the first workgroups; by the others db, dc of a group: its heads'
// in order, four values a thread.
template <bool BF16>
__global__ __launch_bounds__(NT) void ttt_ssm_bwd_group_k(SsmBackwardArgs a) {
  const SsmArgs& f = a.f;
  const uint32_t sums = sum_blocks(f.H);
  if (blockIdx.x < sums) {
    const int h = blockIdx.x * (NT / 64) + wave_of(threadIdx.x);
    if (h < f.H) sum_head(a, h, threadIdx.x & 63);
    return;
  }
  const int share = f.H / f.G;
  const uint64_t per = static_cast<uint64_t>(f.T) * f.N / 4;   // vectors of one head
  const uint64_t total = per * f.B * f.G;
  for (uint64_t i = static_cast<uint64_t>(blockIdx.x - sums) * NT + threadIdx.x; i < total;
       i += static_cast<uint64_t>(gridDim.x - sums) * NT) {
    const uint64_t group = total <= 0xffffffffull   // batch and group
                               ? static_cast<uint32_t>(i) / static_cast<uint32_t>(per)
                               : i / per;
    const uint64_t at = (group * share * per + (i - group * per)) * 4;   // a group's heads are neighbours
    f32x4 db = {0.f, 0.f, 0.f, 0.f}, dc = db;
#pragma unroll 4
    for (int s = 0; s < share; ++s) {
      db += *reinterpret_cast<const f32x4*>(a.ws_db + at + s * per * 4);
      dc += *reinterpret_cast<const f32x4*>(a.ws_dc + at + s * per * 4);
    }
    if constexpr (BF16) {
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.db) + 4 * i) =
          u32x2{pack_bf16(db[0], db[1]), pack_bf16(db[2], db[3])};
      *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.dc) + 4 * i) =
          u32x2{pack_bf16(dc[0], dc[1]), pack_bf16(dc[2], dc[3])};
    } else {
      *reinterpret_cast<f32x4*>(static_cast<float*>(a.db) + 4 * i) = db;
      *reinterpret_cast<f32x4*>(static_cast<float*>(a.dc) + 4 * i) = dc;
    }
  }
}

template <int NI, int N>
hipError_t bwd_launch(const SsmBackwardArgs& a, hipStream_t stream) {
  const SsmArgs& f = a.f;
  const uint32_t units = static_cast<uint32_t>(f.B) * f.H;
  hipError_t e;
  hipLaunchKernelGGL((ttt_ssm_bwd_walk_k<NI, N>), dim3(units * (2 * f.segs - 1)), dim3(NT), 0,
                     stream, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(ttt_ssm_bwd_join_k, dim3(2 * units * (N * P / 4 / NT)), dim3(NT), 0, stream,
                     a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL((ttt_ssm_bwd_k<NI, N>), dim3(units * f.segs), dim3(GT), 0, stream, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (a.ws_db) {
    const uint64_t total = static_cast<uint64_t>(f.T) * N / 4 * f.B * f.G;
    const uint64_t need = (total + NT - 1) / NT;
    hipLaunchKernelGGL((ttt_ssm_bwd_group_k<NI == 1>),
                       dim3(sum_blocks(f.H) + (need < 8192 ? need : 8192)), dim3(NT), 0, stream, a);
  } else {
    hipLaunchKernelGGL(ttt_ssm_bwd_sum_k, dim3(sum_blocks(f.H)), dim3(NT), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_ssm_backward(const SsmBackwardArgs& a, bool bf16, hipStream_t stream) {
  if (a.f.N == 32) return bf16 ? bwd_launch<1, 32>(a, stream) : bwd_launch<3, 32>(a, stream);
  if (a.f.N == 64) return bf16 ? bwd_launch<1, 64>(a, stream) : bwd_launch<3, 64>(a, stream);
  return bf16 ? bwd_launch<1, 128>(a, stream) : bwd_launch<3, 128>(a, stream);
}

}  // namespace tttk
