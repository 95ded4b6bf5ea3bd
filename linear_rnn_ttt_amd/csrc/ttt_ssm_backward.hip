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
// leaving the state before every tile and what the segment adds; (2) the
// states in front of the segments; (3) with several segments, what each adds
// to the adjoint in front of it; (4) the adjoints behind the segments; (5) the
// gradients, each segment's tiles last to first with A in registers; (6) the
// sums of da and dd over batch and segments in order; (7) where heads share b
// and c, their db and dc added in order.
//
// In (5) wave w owns features 16 w .. of x (A, dX^T) and rows 16 w .. (and
// 16 (w + 4) ..) of the state (dB^T, dC^T); A reaches the other waves through
// LDS.  The matrices W1, W2 and W2^T are shared out by blocks as M in the
// forward; W2 is made in both orientations (its products are two of eight)
// rather than transposed.
#include "ttt_block.hpp"
#include "ttt_block_io.hpp"
#include "ttt_ssm_tile.hpp"

namespace tttk {
namespace {

constexpr int NT = SSM_NT, P = SSM_P;

// ---- one walk over a segment: the states before its tiles, or its adjoint ---

template <int NI, int N>
struct WalkLds {
  static constexpr int L = kSsmTile<NI>;
  Plane<NI, L, P> x;
  Plane<NI, L, N> b;
  Tokens<L> tk;
  float fade;
};

// ADJ false: S over x and b, first tile to last.  ADJ true: A over dy and c,
// last to first, for the segments behind the first.
template <int NI, int N, bool ADJ>
__global__ __launch_bounds__(NT) void ttt_ssm_bwd_walk_k(SsmBackwardArgs a) {
  constexpr int L = kSsmTile<NI>;
  __shared__ alignas(16) WalkLds<NI, N> lds;
  const SsmArgs& f = a.f;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, c = lane & 15;
  const int count = ADJ ? f.segs - 1 : f.segs;
  const int seg = blockIdx.x % count + (ADJ ? 1 : 0);
  const size_t unit = blockIdx.x / count;
  const int h = static_cast<int>(unit % f.H);
  const size_t shared = unit / f.H * f.G + h / (f.H / f.G);
  const int tiles = (f.T + L - 1) / L;
  const int first = seg * f.seg_tiles, end = min(first + f.seg_tiles, tiles);
  const float ah = f.a[h];
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
  float step = 0.f;
  auto fetch = [&](int tile) {
    const int t0 = tile * L, valid = min(L, f.T - t0);
    fx.load(row_ptr<NI>(rows, unit * f.T + t0, P), valid, tid);
    fb.load(row_ptr<NI>(cols, shared * f.T + t0, N), valid, tid);
    step = lane < valid ? f.dt[unit * f.T + t0 + lane] : 0.f;
  };
  double total = 0.0;
  fetch(ADJ ? end - 1 : first);
  for (int i = 0; i < end - first; ++i) {
    const int tile = ADJ ? end - 1 - i : first + i;
    fx.store(lds.x, tid);
    fb.store(lds.b, tid);
    if (wave == 0) {
      const double all = lds.tk.fill(step, ah, lane);
      total += all;
      if (lane == 0) lds.fade = exp2_raw(static_cast<float>(all));
    }
    lds_barrier();
    if (i + 1 < end - first) fetch(ADJ ? tile - 1 : tile + 1);
    if (!ADJ && i > 0) save(a.ws_tile + (unit * tiles + tile) * (N * P));
    add_tile<NI, L, N>(
        S, lds.b, lds.x, lds.fade,
        [&](int t) { return ADJ ? lds.tk.from_state(t) : lds.tk.into_state(t); }, wave, g, c);
    lds_barrier();
  }
  if (ADJ) {
    save(a.ws_adj + (unit * f.segs + seg) * (N * P));
  } else {
    save(f.ws_state + (unit * (f.segs + 1) + seg) * (N * P));
    if (tid == 0) f.ws_fade[unit * f.segs + seg] = total;
  }
}

// States in front of the segments (and behind the last), then adjoints behind them.
__global__ __launch_bounds__(NT) void ttt_ssm_bwd_join_k(SsmBackwardArgs a) {
  const SsmArgs& f = a.f;
  const int per = f.N * P / 4;
  const uint64_t i = static_cast<uint64_t>(blockIdx.x) * NT + threadIdx.x;
  const size_t unit = i / per, at = (i - unit * per) * 4, size = static_cast<size_t>(f.N) * P;
  const double* fades = f.ws_fade + unit * f.segs;
  f32x4 S = {0.f, 0.f, 0.f, 0.f};
  if (f.state0) S = *reinterpret_cast<const f32x4*>(f.state0 + unit * size + at);
  float* p = f.ws_state + unit * (f.segs + 1) * size + at;
  for (int s = 0; s < f.segs; ++s, p += size) {
    const f32x4 added = *reinterpret_cast<const f32x4*>(p);
    *reinterpret_cast<f32x4*>(p) = S;
    S = S * exp2_raw(static_cast<float>(fades[s])) + added;
  }
  *reinterpret_cast<f32x4*>(p) = S;
  f32x4 A = {0.f, 0.f, 0.f, 0.f};
  if (a.dstate) A = *reinterpret_cast<const f32x4*>(a.dstate + unit * size + at);
  p = a.ws_adj + (unit * f.segs + f.segs - 1) * size + at;
  for (int s = f.segs - 1; s > 0; --s, p -= size) {
    const f32x4 added = *reinterpret_cast<const f32x4*>(p);
    *reinterpret_cast<f32x4*>(p) = A;
    A = A * exp2_raw(static_cast<float>(fades[s])) + added;
  }
  *reinterpret_cast<f32x4*>(p) = A;
}

// ---- the gradients ----------------------------------------------------------

template <int NI, int N>
struct GradLds {
  static constexpr int L = kSsmTile<NI>, TB = L / 16, BLOCKS = TB * (TB + 1) / 2;
  static constexpr int NM = NI == 1 ? 2 : 3;   // parts of W1 and W2, and of A for dX
  Plane<NI, L, P> x, dy;
  Plane<NI, L, N> b, c;
  Plane<3, P, N> adj;             // A behind the tile: row = feature of x, column = state row
  Blocks<NM, BLOCKS> w1, w2, w2t; // [t, s], [t, s] and [s, t] with dt_s
  Tokens<L> tk;
  float u[4][L], v[4][L];         // per wave: u and v of its state rows
  float zrow[BLOCKS][16], zcol[BLOCKS][16], zdiag[L];   // sums of Z by blocks; its diagonal
  float dot[4];                   // per wave: <S, A> of its state rows
  float fade, before;             // of the tile; from the segment's start to the tile
};

template <int NI, int N>
__global__ __launch_bounds__(NT) void ttt_ssm_bwd_k(SsmBackwardArgs a) {
  using Lds = GradLds<NI, N>;
  constexpr int L = Lds::L, TB = Lds::TB, NM = Lds::NM;
  constexpr int NB = N >= 64 ? N / 64 : 1;   // state row blocks of a wave (N = 32: waves 0 and 1)
  __shared__ alignas(16) Lds lds;
  const SsmArgs& f = a.f;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, c = lane & 15;
  const int seg = blockIdx.x % f.segs;
  const size_t unit = blockIdx.x / f.segs;
  const int h = static_cast<int>(unit % f.H);
  const size_t shared = unit / f.H * f.G + h / (f.H / f.G);
  const int tiles = (f.T + L - 1) / L;
  const int first = seg * f.seg_tiles, end = min(first + f.seg_tiles, tiles);
  const float ah = f.a[h], skip = f.d_skip ? f.d_skip[h] : 0.f;
  const bool has_rows = N >= 64 || wave < N / 16;

  // A behind the segment
  f32x4 A[N / 16];
  {
    const float* from = a.ws_adj + (unit * f.segs + seg) * (N * P);
#pragma unroll
    for (int i = 0; i < N / 16; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) A[i][r] = from[(16 * i + 4 * g + r) * P + 16 * wave + c];
  }
  // a state by rows: row 16 (wave + 4 nb) + c, features by lane
  struct Rows {
    f32x4 v[NB][P / 32][2];
  };
  auto load_rows = [&](const float* p) {
    Rows r;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int k = 0; k < P / 32; ++k)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)
          r.v[nb][k][hh] = has_rows ? *reinterpret_cast<const f32x4*>(
                                          p + (16 * (wave + 4 * nb) + c) * P + 32 * k + 16 * hh + 4 * g)
                                    : f32x4{0.f, 0.f, 0.f, 0.f};
    return r;
  };
  const float* seg_state = f.ws_state + (unit * (f.segs + 1) + seg) * (N * P);
  double rest = f.ws_fade[unit * f.segs + seg];   // log2 decay from the segment's start
  float dd_sum = 0.f;
  double da_sum = 0.0;

  Fetch<NI, L, P, NT> fx, fy;
  Fetch<NI, L, N, NT> fb, fc;
  float step = 0.f;
  auto fetch = [&](int tile) {
    const int t0 = tile * L, valid = min(L, f.T - t0);
    fx.load(row_ptr<NI>(f.x, unit * f.T + t0, P), valid, tid);
    fy.load(row_ptr<NI>(a.dy, unit * f.T + t0, P), valid, tid);
    fb.load(row_ptr<NI>(f.b, shared * f.T + t0, N), valid, tid);
    fc.load(row_ptr<NI>(f.c, shared * f.T + t0, N), valid, tid);
    step = lane < valid ? f.dt[unit * f.T + t0 + lane] : 0.f;
  };
  fetch(end - 1);
  for (int tile = end - 1; tile >= first; --tile) {
    const int t0 = tile * L, valid = min(L, f.T - t0);
    fx.store(lds.x, tid);
    fy.store(lds.dy, tid);
    fb.store(lds.b, tid);
    fc.store(lds.c, tid);
    if (wave == 0) {
      const double all = lds.tk.fill(step, ah, lane);
      rest -= all;
      if (lane == 0) {
        lds.fade = exp2_raw(static_cast<float>(all));
        lds.before = exp2_raw(static_cast<float>(rest));
      }
    }
#pragma unroll
    for (int i = 0; i < N / 16; ++i) {
      u32x2 p[3];
      split_parts<3>(A[i], p);
#pragma unroll
      for (int k = 0; k < 3; ++k)
        *reinterpret_cast<u32x2*>(&lds.adj.v[k][16 * wave + c][16 * i + 4 * g]) = p[k];
    }
    lds_barrier();
    if (tile > first) fetch(tile - 1);
    // the state before the tile: the segment's own part and what came in front of it
    Rows S = load_rows(seg_state);
    {
      const float w = lds.before;
      if (tile > first) {
        const Rows own = load_rows(a.ws_tile + (unit * tiles + tile) * (N * P));
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int k = 0; k < P / 32; ++k)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
              S.v[nb][k][hh] = S.v[nb][k][hh] * w + own.v[nb][k][hh];
      }
    }

    // W1, W2 and W2^T block by block
    for (int i = wave; i < Lds::BLOCKS; i += 4) {
      int tb, sb;
      block_of(i, &tb, &sb);
      f32x4 w1 = {0.f, 0.f, 0.f, 0.f}, w2 = w1, w2t = w1;
#pragma unroll
      for (int k = 0; k < N / 32; ++k)
        w1 = mfma_parts(lds.c.rows8(16 * tb, 32 * k, g, c), lds.b.rows8(16 * sb, 32 * k, g, c),
                        w1);
#pragma unroll
      for (int k = 0; k < P / 32; ++k) {
        const Parts<NI> yr = lds.dy.rows8(16 * tb, 32 * k, g, c);
        const Parts<NI> xr = lds.x.rows8(16 * sb, 32 * k, g, c);
        w2 = mfma_parts(yr, xr, w2);
        w2t = mfma_parts(xr, yr, w2t);
      }
      float col = 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (tb == sb && 4 * g + r == c) dd_sum += w2[r];
        {
          const int t = 16 * tb + 4 * g + r, s = 16 * sb + c;
          const float fade = lds.tk.fade(t, s);
          w1[r] = s <= t ? w1[r] * fade : 0.f;
          const float z = w1[r] * w2[r];
          w2[r] = s <= t ? w2[r] * fade : 0.f;
          const float row = row_sum16(s < t ? z * lds.tk.dt[s] : 0.f);
          if (c == r) lds.zrow[i][4 * g + r] = row;
          if (s == t) lds.zdiag[t] = z;
          else col += s < t ? z : 0.f;
        }
        {
          const int t = 16 * tb + c, s = 16 * sb + 4 * g + r;
          w2t[r] = s <= t ? w2t[r] * (lds.tk.fade(t, s) * lds.tk.dt[s]) : 0.f;
        }
      }
      col = group_sum(col);
      if (g == 0) lds.zcol[i][c] = col;
      lds.w1.put(i, lane, w1);
      lds.w2.put(i, lane, w2);
      lds.w2t.put(i, lane, w2t);
    }

    // what the adjoint behind the tile and the state before it give
    f32x4 dx[TB], db[NB][TB], dc[NB][TB];
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      dx[j] = zero;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) db[nb][j] = dc[nb][j] = zero;
    }
#pragma unroll
    for (int k = 0; k < N / 32; ++k) {
      const Parts<NM> ap = split_frag<NM>(A[2 * k], A[2 * k + 1]);
#pragma unroll
      for (int j = 0; j < TB; ++j)
        dx[j] = mfma_parts(ap, lds.b.rows(16 * j, 32 * k, g, c), dx[j]);
    }
    float dot = 0.f;
    if (has_rows) {
#pragma unroll
      for (int k = 0; k < P / 32; ++k) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const Parts<3> ar = lds.adj.cols(32 * k, 16 * (wave + 4 * nb), g, c);
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const f32x4 prod = frag_half(ar, hh) * S.v[nb][k][hh];
            dot += (prod[0] + prod[1]) + (prod[2] + prod[3]);
          }
          const Parts<3> sp = split_frag<3>(S.v[nb][k][0], S.v[nb][k][1]);
#pragma unroll
          for (int j = 0; j < TB; ++j) {
            db[nb][j] = mfma_parts(ar, lds.x.rows(16 * j, 32 * k, g, c), db[nb][j]);
            dc[nb][j] = mfma_parts(sp, lds.dy.rows(16 * j, 32 * k, g, c), dc[nb][j]);
          }
        }
      }
    }
    dot = wave_sum(dot);
    if (lane == 0) lds.dot[wave] = dot;
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      const int t = 16 * j + c;
      dx[j] *= lds.tk.tail[t];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        db[nb][j] *= lds.tk.tail[t];
        dc[nb][j] *= lds.tk.head[t];
      }
      float us = 0.f, vs = 0.f;
      if (has_rows) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int n = 16 * (wave + 4 * nb) + 4 * g;
          const f32x4 pv = lds.b.four(t, n) * db[nb][j], pu = lds.c.four(t, n) * dc[nb][j];
          vs += (pv[0] + pv[1]) + (pv[2] + pv[3]);
          us += (pu[0] + pu[1]) + (pu[2] + pu[3]);
        }
      }
      us = group_sum(us);
      vs = group_sum(vs);
      if (g == 0) {
        lds.u[wave][t] = us;
        lds.v[wave][t] = vs;
      }
    }
    lds_barrier();

    // and the tile's own tokens
    auto pair = [&](const Blocks<NM, Lds::BLOCKS>& w, int i0, int i1) {   // -1: zero
      Parts<NM> m;
#pragma unroll
      for (int p = 0; p < NM; ++p)
        m.p[p] = cat(i0 >= 0 ? w.v[i0][p][lane] : u32x2{0u, 0u},
                     i1 >= 0 ? w.v[i1][p][lane] : u32x2{0u, 0u});
      return m;
    };
    auto at = [](int tb, int sb) { return sb <= tb ? tb * (tb + 1) / 2 + sb : -1; };
#pragma unroll
    for (int k = 0; k < L / 32; ++k) {
      const Parts<NI> yt = lds.dy.cols(32 * k, 16 * wave, g, c);
#pragma unroll
      for (int j = 0; j <= 2 * k + 1; ++j)
        dx[j] = mfma_parts(yt, pair(lds.w1, at(2 * k, j), at(2 * k + 1, j)), dx[j]);
      if (has_rows) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const Parts<NI> ct = lds.c.cols(32 * k, 16 * (wave + 4 * nb), g, c);
          const Parts<NI> bt = lds.b.cols(32 * k, 16 * (wave + 4 * nb), g, c);
#pragma unroll
          for (int j = 0; j <= 2 * k + 1; ++j)
            db[nb][j] = mfma_parts(ct, pair(lds.w2, at(2 * k, j), at(2 * k + 1, j)), db[nb][j]);
#pragma unroll
          for (int j = 2 * k; j < TB; ++j)
            dc[nb][j] = mfma_parts(bt, pair(lds.w2t, at(j, 2 * k), at(j, 2 * k + 1)), dc[nb][j]);
        }
      }
    }

    // stores
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      const int t = 16 * j + c;
      const float dt = lds.tk.dt[t];
      {
        f32x4 v = dx[j] * dt;
        if (f.d_skip) v += lds.dy.four(t, 16 * wave + 4 * g) * skip;
        if (t < valid) {
          const size_t o = (unit * f.T + t0 + t) * P + 16 * wave + 4 * g;
          if constexpr (NI == 1)
            *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.dx) + o) =
                u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
          else
            *reinterpret_cast<f32x4*>(static_cast<float*>(a.dx) + o) = v;
        }
      }
      if (has_rows && t < valid) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int n = 16 * (wave + 4 * nb) + 4 * g;
          const f32x4 v = db[nb][j] * dt;
          if (a.ws_db) {
            const size_t o = (unit * f.T + t0 + t) * N + n;
            *reinterpret_cast<f32x4*>(a.ws_db + o) = v;
            *reinterpret_cast<f32x4*>(a.ws_dc + o) = dc[nb][j];
          } else {
            const size_t o = (shared * f.T + t0 + t) * N + n;
            if constexpr (NI == 1) {
              *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.db) + o) =
                  u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
              *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.dc) + o) =
                  u32x2{pack_bf16(dc[nb][j][0], dc[nb][j][1]),
                        pack_bf16(dc[nb][j][2], dc[nb][j][3])};
            } else {
              *reinterpret_cast<f32x4*>(static_cast<float*>(a.db) + o) = v;
              *reinterpret_cast<f32x4*>(static_cast<float*>(a.dc) + o) = dc[nb][j];
            }
          }
        }
      }
    }

    // A before the tile
    add_tile<NI, L, N>(
        A, lds.c, lds.dy, lds.fade, [&](int t) { return lds.tk.from_state(t); }, wave, g, c);
    lds_barrier();

    if (wave == 0) {   // ddt, and the tile's share of da
      double after = 0.0, upto = 0.0;   // of the token: u + row - column sums of Z; dt v
      float dt = 0.f, direct = 0.f;
      if (lane < L) {
        dt = lds.tk.dt[lane];
        const float us = (lds.u[0][lane] + lds.u[1][lane]) + (lds.u[2][lane] + lds.u[3][lane]);
        const float vs = (lds.v[0][lane] + lds.v[1][lane]) + (lds.v[2][lane] + lds.v[3][lane]);
        float row = 0.f, col = 0.f;
        const int mine = lane >> 4, in = lane & 15;
#pragma unroll
        for (int k = 0; k < TB; ++k) {
          if (k <= mine) row += lds.zrow[mine * (mine + 1) / 2 + k][in];
          if (k >= mine) col += lds.zcol[k * (k + 1) / 2 + mine][in];
        }
        after = static_cast<double>(us) + row - static_cast<double>(dt) * col;
        upto = static_cast<double>(dt) * vs;
        direct = vs + (col + lds.zdiag[lane]);
      }
      const double after_to = wave_scan(after), upto_to = wave_scan(upto);
      const float d = (lds.dot[0] + lds.dot[1]) + (lds.dot[2] + lds.dot[3]);
      const double e = (last_lane(after_to) - after_to + after) + (upto_to - upto) + lds.fade * d;
      if (lane < valid) {
        a.ddt[unit * f.T + t0 + lane] = static_cast<float>(direct + ah * e);
        da_sum += dt * e;
      }
    }
  }
  if (a.dstate0 && seg == 0) {
    float* out = a.dstate0 + unit * (N * P);
#pragma unroll
    for (int i = 0; i < N / 16; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) out[(16 * i + 4 * g + r) * P + 16 * wave + c] = A[i][r];
  }
  // the segment's da and dd
  dd_sum = wave_sum(dd_sum);
  lds_barrier();
  if (lane == 0) lds.dot[wave] = dd_sum;
  lds_barrier();
  if (wave == 0) {
    const double all = last_lane(wave_scan(da_sum));
    if (lane == 0) {
      float* out = a.ws_sums + (unit * f.segs + seg) * 2;
      out[0] = static_cast<float>(all);
      out[1] = (lds.dot[0] + lds.dot[1]) + (lds.dot[2] + lds.dot[3]);
    }
  }
}

// da[h], dd[h]: a wave per head over (batch, segment).
__global__ __launch_bounds__(64) void ttt_ssm_bwd_sum_k(SsmBackwardArgs a) {
  const SsmArgs& f = a.f;
  const int h = blockIdx.x, lane = threadIdx.x;
  double da = 0.0, dd = 0.0;
  for (int64_t i = lane; i < static_cast<int64_t>(f.B) * f.segs; i += 64) {
    const size_t b = i / f.segs, seg = i - b * f.segs;
    const float* p = a.ws_sums + ((b * f.H + h) * f.segs + seg) * 2;
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

// db, dc of a group: its heads' in order, four values a thread.
template <bool BF16>
__global__ __launch_bounds__(NT) void ttt_ssm_bwd_group_k(SsmBackwardArgs a) {
  const SsmArgs& f = a.f;
  const int share = f.H / f.G;
  const uint64_t per = static_cast<uint64_t>(f.T) * f.N / 4;   // vectors of one head
  const uint64_t total = per * f.B * f.G;
  for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * NT + threadIdx.x; i < total;
       i += static_cast<uint64_t>(gridDim.x) * NT) {
    const uint64_t group = i / per, in = i - group * per;   // batch and group
    const uint64_t at = (group * share * per + in) * 4;     // heads of a group are neighbours
    f32x4 db = {0.f, 0.f, 0.f, 0.f}, dc = db;
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
  hipLaunchKernelGGL((ttt_ssm_bwd_walk_k<NI, N, false>), dim3(units * f.segs), dim3(NT), 0, stream,
                     a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (f.segs > 1) {
    hipLaunchKernelGGL((ttt_ssm_bwd_walk_k<NI, N, true>), dim3(units * (f.segs - 1)), dim3(NT), 0,
                       stream, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  hipLaunchKernelGGL(ttt_ssm_bwd_join_k, dim3(units * (N * P / 4 / NT)), dim3(NT), 0, stream, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL((ttt_ssm_bwd_k<NI, N>), dim3(units * f.segs), dim3(NT), 0, stream, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(ttt_ssm_bwd_sum_k, dim3(f.H), dim3(64), 0, stream, a);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (a.ws_db) {
    const uint64_t total = static_cast<uint64_t>(f.T) * N / 4 * f.B * f.G;
    const uint64_t need = (total + NT - 1) / NT;
    hipLaunchKernelGGL((ttt_ssm_bwd_group_k<NI == 1>), dim3(need < 8192 ? need : 8192), dim3(NT),
                       0, stream, a);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

hipError_t launch_ssm_backward(const SsmBackwardArgs& a, bool bf16, hipStream_t stream) {
  if (a.f.N == 32) return bf16 ? bwd_launch<1, 32>(a, stream) : bwd_launch<3, 32>(a, stream);
  if (a.f.N == 64) return bf16 ? bwd_launch<1, 64>(a, stream) : bwd_launch<3, 64>(a, stream);
  return bf16 ? bwd_launch<1, 128>(a, stream) : bwd_launch<3, 128>(a, stream);
}

}  // namespace tttk
