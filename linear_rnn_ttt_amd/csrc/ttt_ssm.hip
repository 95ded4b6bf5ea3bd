// ttt_ssm.hip -- the selective state space scan for gfx950: forward over
// prompts, and the one-token step.
//
// Per (batch, head) unit, with the state S [N, 64], b and c of the head's group:
//     S_t = exp(a dt_t) S_{t-1} + dt_t b_t^T x_t,   y_t = c_t S_t + d x_t
// For a tile of L tokens, with cum_t the sum of a dt over the tile up to t and
// S the state before it, the recurrence becomes products for the matrix unit:
//     M[t, s] = (c_t . b_s) exp(cum_t - cum_s) dt_s  for s <= t, else 0
//     Y  = M X + diag(exp(cum_t)) C S (+ d X)
//     S' = exp(cum_L) S + B^T diag(exp(cum_L - cum_s) dt_s) X
// The kernel computes the transposes Y^T = X^T M^T + S^T C^T, so that M^T
// (from B C^T) and S leave one product in the registers as operands of the
// next; X and B are read transposed from LDS by the transposing read.
//
// A workgroup of four waves walks its tiles with S in registers: wave w owns
// features 16 w .. 16 w + 15 of x, y and S.  The blocks of M are shared out
// over the waves and exchanged through LDS.  The next tile is fetched while
// this one is worked on.
//
// Few units leave compute units idle and make a long chain of tiles, so a
// unit's tokens are cut into segments: ttt_ssm_states_k finds what each
// segment adds to a state of zero, ttt_ssm_join_k runs the recurrence over
// the segments (in place), and ttt_ssm_scan_k starts every segment from its
// own state.  With one segment only the last runs.
//
// At bf16, B4 H32 T8192 N64 (8 segments): states 64 us, join 7, scan 113, 181 in
// all.  The scan moves 560 MB, 5.0 TB/s, near the 5.4 that a copy reaches on this
// card; the states, which read x and b once more, 3.9 TB/s (a kernel that only
// reads reached 4.0).  The scan's vector unit is 54 % busy, its matrix unit 25 %.
//
// Precision: bf16 data enter the products exactly; M and S in two bf16 parts
// (16 bits, so that y keeps only its own rounding), what enters the state in
// three (24 bits).  fp32 data are three parts throughout.
#include "ttt_block.hpp"
#include "ttt_block_io.hpp"
#include "ttt_ssm_tile.hpp"

namespace tttk {
namespace {

constexpr int NT = SSM_NT, P = SSM_P;

// ---- what each segment adds to a state of zero ------------------------------

// A segment's state in the workspace, in the order of the registers that hold
// it: vector 64 i is rows 16 i + 4 g .. 4 g + 3 of the lane's feature.
__device__ __forceinline__ f32x4* seg_state(const SsmArgs& a, size_t unit, int seg, int wave,
                                            int lane, int N) {
  return reinterpret_cast<f32x4*>(a.ws_state + (unit * a.segs + seg) * (N * P)) +
         wave * (N / 16) * 64 + lane;
}

template <int NI, int N>
struct StatesLds {
  static constexpr int L = kSsmTile<NI>;
  Plane<NI, L, P> x;
  Plane<NI, L, N> b;
  Tokens<L> tk[2];   // of even and odd tiles
};

template <int NI, int N>
__global__ __launch_bounds__(NT, 2) void ttt_ssm_states_k(SsmArgs a) {
  constexpr int L = kSsmTile<NI>;
  __shared__ alignas(16) StatesLds<NI, N> lds;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_of(tid), g = lane >> 4, c = lane & 15;
  const Place at(a, blockIdx.x, a.segs - 1);   // nothing follows the last segment
  const int seg = at.seg, h = at.h;
  const size_t unit = at.unit, shared = at.shared;
  const int first = seg * a.seg_tiles, end = first + a.seg_tiles;
  const float ah = a.a[h];
  f32x4 S[N / 16];
#pragma unroll
  for (int i = 0; i < N / 16; ++i) S[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  struct Tile {
    Fetch<NI, L, P, NT> x;
    Fetch<NI, L, N, NT> b;
  } next, after;   // on their way: two tiles
  auto valid_of = [&](int tile) { return tile < end ? min(L, a.T - tile * L) : 0; };
  auto fetch = [&](int tile, Tile& to) {
    const int t0 = tile * L, valid = valid_of(tile);
    to.x.load(row_ptr<NI>(a.x, unit * a.T + t0, P), valid, tid);
    to.b.load(row_ptr<NI>(a.b, shared * a.T + t0, N), valid, tid);
  };
  auto steps_of = [&](int tile) {
    return load_steps(a.dt + unit * a.T + tile * L, valid_of(tile), lane);
  };
  // the decays of a tile are made by one wave while the one before is worked on
  double total = 0.0;
  fetch(first, next);
  fetch(first + 1, after);
  float step = steps_of(first);
  if (wave == 0) total = lds.tk[first & 1].fill(step, ah, lane);
  step = steps_of(first + 1);
  auto work = [&](int tile, Tile& now) {
    now.x.store(lds.x, tid);
    now.b.store(lds.b, tid);
    lds_barrier();
    const Tokens<L>& tk = lds.tk[tile & 1];
    fetch(tile + 2, now);
    if (wave == 0 && tile + 1 < end) total += lds.tk[(tile + 1) & 1].fill(step, ah, lane);
    step = steps_of(tile + 2);
    add_tile(S, lds.b, 0, lds.x, wave, tk.fade, tk.into, g, c);
    lds_barrier();
  };
  for (int tile = first; tile < end; tile += 2) {
    work(tile, next);
    if (tile + 1 < end) work(tile + 1, after);
  }
  f32x4* out = seg_state(a, unit, seg, wave, lane, N);
#pragma unroll
  for (int i = 0; i < N / 16; ++i) out[64 * i] = S[i];
  if (tid == 0) a.ws_fade[unit * a.segs + seg] = total;
}

// Up to kScanJoins segments the scan's workgroups work their own start out from
// what the segments add, in place of the join's launch: 124.4 -> 120.5 us for the
// whole call at B4 H32 T4096 N128, 36.9 -> 32.3 at T512 (4 segments); at B4 H32 T8192
// N64 (8 segments) it would cost, 185.8 -> 193.4.  Where the final state takes state0's place, though,
// a segment's workgroup may end before another one has read state0: the join
// reads it first.
constexpr int kScanJoins = 4;
__host__ __device__ inline bool join_launched(const SsmArgs& a) {
  return a.segs > kScanJoins || (a.segs > 1 && a.state0 && a.state0 == a.state_out);
}

// ws_state[seg]: from what the segment adds to the state in front of it.
__global__ __launch_bounds__(NT) void ttt_ssm_join_k(SsmArgs a) {
  const JoinPlace place(a.N, blockIdx.x, threadIdx.x);
  const size_t unit = place.unit, at = place.at, size = static_cast<size_t>(a.N) * P;
  f32x4 S = {0.f, 0.f, 0.f, 0.f};
  if (a.state0) {   // at as in seg_state
    const int lane = at / 4 & 63, block = at / 256, wave = block / (a.N / 16);
    const float* from = a.state0 + unit * size +
                        (16 * (block - wave * (a.N / 16)) + 4 * (lane >> 4)) * P + 16 * wave +
                        (lane & 15);
#pragma unroll
    for (int r = 0; r < 4; ++r) S[r] = from[r * P];
  }
  join_segments(a.ws_state + unit * a.segs * size + at, size, a.ws_fade + unit * a.segs, a.segs,
                a.segs - 1, 1, S);
}

// ---- the scan ---------------------------------------------------------------

template <int NI, int N>
struct ScanLds {
  static constexpr int L = kSsmTile<NI>, TB = L / 16, BLOCKS = TB * (TB + 1) / 2;
  static constexpr int NM = NI == 1 ? 2 : 3;   // parts of M and of S
  Plane<NI, L, P> x;
  Plane<NI, L, N> b, c;
  Tokens<L> tk[2];          // of even and odd tiles
  Blocks<NM, BLOCKS> m;     // M^T: rows s, columns t
};

template <int NI, int N>
__global__ __launch_bounds__(NT, 2) void ttt_ssm_scan_k(SsmArgs a) {
  using Lds = ScanLds<NI, N>;
  constexpr int L = Lds::L, TB = Lds::TB, NM = Lds::NM, BELOW = TB * (TB - 1) / 2;
  __shared__ alignas(16) Lds lds;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_of(tid), g = lane >> 4, c = lane & 15;
  const Place at(a, blockIdx.x, a.segs);
  const int seg = at.seg, h = at.h;
  const size_t unit = at.unit, shared = at.shared;
  const int tiles = (a.T + L - 1) / L;
  const int first = seg * a.seg_tiles, end = min(first + a.seg_tiles, tiles);
  const float ah = a.a[h], skip = a.d_skip ? a.d_skip[h] : 0.f;
  f32x4 S[N / 16];
  if (join_launched(a)) {
    const f32x4* from = seg_state(a, unit, seg, wave, lane, N);
#pragma unroll
    for (int i = 0; i < N / 16; ++i) S[i] = from[64 * i];
  } else {
    const float* from = a.state0 ? a.state0 + unit * (N * P) : nullptr;
#pragma unroll
    for (int i = 0; i < N / 16; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        S[i][r] = from ? from[(16 * i + 4 * g + r) * P + 16 * wave + c] : 0.f;
    constexpr int AT_ONCE = 256 / N;   // segments whose loads are issued together
    for (int s0 = 0; s0 < seg; s0 += AT_ONCE) {
      f32x4 added[AT_ONCE][N / 16];
#pragma unroll
      for (int k = 0; k < AT_ONCE; ++k)
        if (s0 + k < seg) {
          const f32x4* p = seg_state(a, unit, s0 + k, wave, lane, N);
#pragma unroll
          for (int i = 0; i < N / 16; ++i) added[k][i] = p[64 * i];
        }
#pragma unroll
      for (int k = 0; k < AT_ONCE; ++k)
        if (s0 + k < seg) {
          const float fade = exp2_raw(static_cast<float>(a.ws_fade[unit * a.segs + s0 + k]));
#pragma unroll
          for (int i = 0; i < N / 16; ++i) S[i] = S[i] * fade + added[k][i];
        }
    }
  }
  struct Tile {
    Fetch<NI, L, P, NT> x;
    Fetch<NI, L, N, NT> b, c;
  } next;   // on its way
  auto valid_of = [&](int tile) { return tile < end ? min(L, a.T - tile * L) : 0; };
  auto fetch = [&](int tile, Tile& to) {
    const int t0 = tile * L, valid = valid_of(tile);
    to.x.load(row_ptr<NI>(a.x, unit * a.T + t0, P), valid, tid);
    to.b.load(row_ptr<NI>(a.b, shared * a.T + t0, N), valid, tid);
    to.c.load(row_ptr<NI>(a.c, shared * a.T + t0, N), valid, tid);
  };
  auto steps_of = [&](int tile) {
    return load_steps(a.dt + unit * a.T + tile * L, valid_of(tile), lane);
  };
  fetch(first, next);
  float step = steps_of(first);
  if (wave == 0) lds.tk[first & 1].fill(step, ah, lane);
  step = steps_of(first + 1);
  for (int tile = first; tile < end; ++tile) {
    const int t0 = tile * L, valid = valid_of(tile);
    next.x.store(lds.x, tid);
    next.b.store(lds.b, tid);
    next.c.store(lds.c, tid);
    lds_barrier();
    const Tokens<L>& tk = lds.tk[tile & 1];
    fetch(tile + 1, next);
    // the decays of the next tile, by the wave that has fewer blocks below
    if (wave == 3) lds.tk[(tile + 1) & 1].fill(step, ah, lane);
    step = steps_of(tile + 2);

    // M^T block by block: (b_s . c_t), decayed and masked
    auto make = [&](int tb, int sb) {
      f32x4 m = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < N / 32; ++k)
        m = mfma_parts(lds.b.rows8(16 * sb, 32 * k, g, c), lds.c.rows8(16 * tb, 32 * k, g, c), m);
      return m * (tk.fades(tb, sb, 16 * tb + c, 16 * sb + 4 * g) * tk.steps(16 * sb + 4 * g));
    };
    if (TB == 4 || wave < TB) {
      f32x4 m = make(wave, wave);
#pragma unroll
      for (int r = 0; r < 4; ++r) m[r] += 4 * g + r == c ? skip : 0.f;   // d x_t, as a product too
      lds.m.put(wave * (wave + 3) / 2, lane, m);
    }
    if (wave < 3) {   // wave 3 makes decays instead
      for (int o = (wave + 1) % 3; o < BELOW; o += 3) {
        int tb, sb;
        block_of(o, &tb, &sb);
        ++tb;
        lds.m.put(tb * (tb + 1) / 2 + sb, lane, make(tb, sb));
      }
    }

    // Y^T of the wave's features: from the state in front of the tile
    f32x4 y[TB];
#pragma unroll
    for (int j = 0; j < TB; ++j) y[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < N / 32; ++k) {
      const Parts<NM> sp = split_frag<NM>(S[2 * k], S[2 * k + 1]);
#pragma unroll
      for (int j = 0; j < TB; ++j)
        y[j] = mfma_parts(sp, lds.c.rows(16 * j, 32 * k, g, c), y[j]);
    }
#pragma unroll
    for (int j = 0; j < TB; ++j) y[j] *= tk.head[16 * j + c];
    lds_barrier();

    // and from the tile's own tokens
#pragma unroll
    for (int k = 0; k < L / 32; ++k) {
      const Parts<NI> xs = lds.x.cols(32 * k, 16 * wave, g, c);
#pragma unroll
      for (int j = 2 * k; j < TB; ++j) {
        Parts<NM> m;
#pragma unroll
        for (int p = 0; p < NM; ++p) {
          const int i = j * (j + 1) / 2 + 2 * k;
          m.p[p] = cat(lds.m.v[i][p][lane],
                       j > 2 * k ? lds.m.v[i + 1][p][lane] : u32x2{0u, 0u});
        }
        y[j] = mfma_parts(xs, m, y[j]);
      }
    }
    const __amdgpu_buffer_rsrc_t out =
        rows_of(row_ptr<NI>(a.y, unit * a.T + t0, P), valid * P * (NI == 1 ? 2 : 4));
#pragma unroll
    for (int j = 0; j < TB; ++j)
      store_row4<NI>(out, 16 * j + c, P, 16 * wave + 4 * g, y[j]);
    add_tile(S, lds.b, 0, lds.x, wave, tk.fade, tk.into, g, c);
    lds_barrier();
  }
  if (a.state_out && end == tiles) {
    float* out = a.state_out + unit * (N * P);
#pragma unroll
    for (int i = 0; i < N / 16; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) out[(16 * i + 4 * g + r) * P + 16 * wave + c] = S[i][r];
  }
}

// ---- one token --------------------------------------------------------------

// A workgroup per unit: thread (row n mod 16, features 4 j .. 4 j + 3) walks
// the state's rows 16 apart.  Bound by HBM: the state is read and written once;
// 8192 units of N64: 50 us, 5.5 TB/s.
template <bool BF16, int N>
__global__ __launch_bounds__(NT) void ttt_ssm_step_k(SsmArgs a) {
  __shared__ float part[16][P + 4];
  const int tid = threadIdx.x, row = tid >> 4, f = 4 * (tid & 15);
  const size_t unit = blockIdx.x;
  const int h = static_cast<int>(unit % a.H);
  const size_t shared = unit / a.H * a.G + h / (a.H / a.G);
  float* S = a.state_out + unit * (N * P);
  f32x4 s[N / 16];
#pragma unroll
  for (int i = 0; i < N / 16; ++i)
    s[i] = *reinterpret_cast<const f32x4*>(S + (16 * i + row) * P + f);
  auto io = [](const void* p, size_t i) {
    return BF16 ? bf16_lo_to_f32(static_cast<const uint16_t*>(p)[i])
                : static_cast<const float*>(p)[i];
  };
  float b[N / 16], c[N / 16];
#pragma unroll
  for (int i = 0; i < N / 16; ++i) {
    b[i] = io(a.b, shared * N + 16 * i + row);
    c[i] = io(a.c, shared * N + 16 * i + row);
  }
  const float dt = a.dt[unit], fade = expf(a.a[h] * dt);
  f32x4 x, y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int r = 0; r < 4; ++r) x[r] = io(a.x, unit * P + f + r);
#pragma unroll
  for (int i = 0; i < N / 16; ++i) {
    s[i] = s[i] * fade + x * (dt * b[i]);
    y += s[i] * c[i];
    *reinterpret_cast<f32x4*>(S + (16 * i + row) * P + f) = s[i];
  }
  *reinterpret_cast<f32x4*>(&part[row][f]) = y;
  lds_barrier();
  if (tid < P) {
    float t = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) t += part[r][tid];
    if (a.d_skip) t += a.d_skip[h] * io(a.x, unit * P + tid);
    if constexpr (BF16)
      static_cast<uint16_t*>(a.y)[unit * P + tid] =
          static_cast<uint16_t>(pack_bf16(t, 0.f) & 0xffffu);
    else
      static_cast<float*>(a.y)[unit * P + tid] = t;
  }
}

template <int NI, int N>
hipError_t scan_launch(const SsmArgs& a, hipStream_t stream) {
  const uint32_t units = static_cast<uint32_t>(a.B) * a.H;
  hipError_t e;
  if (a.segs > 1) {
    hipLaunchKernelGGL((ttt_ssm_states_k<NI, N>), dim3(units * (a.segs - 1)), dim3(NT), 0, stream,
                       a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (join_launched(a)) {
      hipLaunchKernelGGL(ttt_ssm_join_k, dim3(units * (N * P / 4 / NT)), dim3(NT), 0, stream, a);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  }
  hipLaunchKernelGGL((ttt_ssm_scan_k<NI, N>), dim3(units * a.segs), dim3(NT), 0, stream,
                     a);
  return hipGetLastError();
}

template <int N>
hipError_t step_launch(const SsmArgs& a, bool bf16, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(a.B) * a.H);
  if (bf16) hipLaunchKernelGGL((ttt_ssm_step_k<true, N>), grid, dim3(NT), 0, stream, a);
  else hipLaunchKernelGGL((ttt_ssm_step_k<false, N>), grid, dim3(NT), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_ssm(const SsmArgs& a, bool bf16, hipStream_t stream) {
  if (a.N == 32) return bf16 ? scan_launch<1, 32>(a, stream) : scan_launch<3, 32>(a, stream);
  if (a.N == 64) return bf16 ? scan_launch<1, 64>(a, stream) : scan_launch<3, 64>(a, stream);
  return bf16 ? scan_launch<1, 128>(a, stream) : scan_launch<3, 128>(a, stream);
}

hipError_t launch_ssm_decode(const SsmArgs& a, bool bf16, hipStream_t stream) {
  if (a.N == 32) return step_launch<32>(a, bf16, stream);
  if (a.N == 64) return step_launch<64>(a, bf16, stream);
  return step_launch<128>(a, bf16, stream);
}

}  // namespace tttk
