// ttt_ssm_tile.hpp -- pieces shared by the selective state space scan's
// forward and backward kernels: tiles of tokens in LDS as bf16 parts, the
// matrix-unit fragments read from them, products of operands in parts, and
// the decays of a tile.
//
// Parts.  A value is one bf16 (bf16 data: exact) or the sum of up to three,
// each the rounding of what the ones before leave: two carry 16 bits, three
// 24.  A product of operands in NA and NB parts adds the part products whose
// combined order is below max(NA, NB); what is left out is below the last
// part's own rounding.
//
// Fragments (64-lane wave, g = lane / 16, c = lane % 16) of a 16x16x32
// product are two 4-value halves: half h of lane (g, c) holds contraction
// indices 16 h + 4 g + 0..3 of row (or column) c.  That is the layout of two
// 16x16 accumulators stacked along their rows, so an accumulator of one
// product is an operand of the next without leaving the registers.
#pragma once

#include "ttt_block_args.hpp"
#include "ttt_device.hpp"

namespace tttk {

constexpr int SSM_P = 64;     // features of x per head
constexpr int SSM_NT = 256;   // threads of a workgroup: four waves of 16 features

template <int N>
struct Parts {
  u32x4 p[N];
};

// acc += A B with operands in parts, smallest terms first.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mfma_parts(const Parts<NA>& a, const Parts<NB>& b, f32x4 acc) {
  constexpr int top = NA > NB ? NA : NB;
#pragma unroll
  for (int o = top - 1; o >= 0; --o)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (o - i >= 0 && o - i < NB) acc = mfma32(a.p[i], b.p[o - i], acc);
  return acc;
}

// Four fp32 in NP parts.
template <int NP>
__device__ __forceinline__ void split_parts(f32x4 x, u32x2 out[NP]) {
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    out[p].x = pack_bf16(x[0], x[1]);
    out[p].y = pack_bf16(x[2], x[3]);
    if (p + 1 < NP) {
      x[0] -= bf16_lo_to_f32(out[p].x);
      x[1] -= bf16_hi_to_f32(out[p].x);
      x[2] -= bf16_lo_to_f32(out[p].y);
      x[3] -= bf16_hi_to_f32(out[p].y);
    }
  }
}

template <int NP>
__device__ __forceinline__ Parts<NP> split_frag(f32x4 lo, f32x4 hi) {
  u32x2 l[NP], h[NP];
  split_parts<NP>(lo, l);
  split_parts<NP>(hi, h);
  Parts<NP> r;
#pragma unroll
  for (int p = 0; p < NP; ++p) r.p[p] = cat(l[p], h[p]);
  return r;
}

__device__ __forceinline__ f32x4 widen4(u32x2 w) {
  return f32x4{bf16_lo_to_f32(w.x), bf16_hi_to_f32(w.x), bf16_lo_to_f32(w.y),
               bf16_hi_to_f32(w.y)};
}

// One half (4 values) of a fragment in fp32: exact (the parts are disjoint).
template <int NP>
__device__ __forceinline__ f32x4 frag_half(const Parts<NP>& f, int h) {
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int p = NP - 1; p >= 0; --p)
    x += widen4(h ? u32x2{f.p[p].z, f.p[p].w} : u32x2{f.p[p].x, f.p[p].y});
  return x;
}

// L tokens x W features as NI planes of bf16 parts.  The 16-byte chunk q of row
// t sits at chunk q ^ swizzle(t), so that the 16 rows of a fragment spread over
// the banks without padding (which would cost the scan its fourth workgroup
// per compute unit).
template <int NI, int L, int W>
struct Plane {
  uint16_t v[NI][L][W];

  static __device__ __forceinline__ int swizzle(int t) { return W >= 64 ? t & 7 : (t >> 1) & 3; }
  // where feature f (a multiple of 4) of token t sits in its row
  static __device__ __forceinline__ int place(int t, int f) {
    return (((f >> 3) ^ swizzle(t)) << 3) | (f & 4);
  }
  __device__ __forceinline__ u32x2 get4(int p, int t, int f) const {
    return *reinterpret_cast<const u32x2*>(&v[p][t][place(t, f)]);
  }
  __device__ __forceinline__ void put4(int p, int t, int f, u32x2 x) {
    *reinterpret_cast<u32x2*>(&v[p][t][place(t, f)]) = x;
  }

  // Rows t0 + c, features f0 + {4 g .. 4 g + 3, 16 + 4 g .. 16 + 4 g + 3}.
  template <int NP = NI>
  __device__ __forceinline__ Parts<NP> rows(int t0, int f0, int g, int c) const {
    Parts<NP> r;
#pragma unroll
    for (int p = 0; p < NP; ++p)
      r.p[p] = cat(get4(p, t0 + c, f0 + 4 * g), get4(p, t0 + c, f0 + 16 + 4 * g));
    return r;
  }
  // The same rows with features f0 + 8 g .. 8 g + 7 (one 16-byte read): for
  // products whose two operands are both read this way.
  __device__ __forceinline__ Parts<NI> rows8(int t0, int f0, int g, int c) const {
    Parts<NI> r;
#pragma unroll
    for (int p = 0; p < NI; ++p)
      r.p[p] = *reinterpret_cast<const u32x4*>(&v[p][t0 + c][place(t0 + c, f0 + 8 * g)]);
    return r;
  }
  // Feature f0 + c, tokens t0 + {4 g .. 4 g + 3, 16 + 4 g .. 16 + 4 g + 3}: the
  // transposing LDS read, in which the 16 lanes of a group fetch a 4-token x
  // 16-feature block by rows and receive it by columns.
  __device__ __forceinline__ Parts<NI> cols(int t0, int f0, int g, int c) const {
    typedef short s16x4l __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s16x4l* lp;
    Parts<NI> r;
    const int t = t0 + 4 * g + (c >> 2), f = place(t, f0 + 4 * (c & 3));   // t + 16: same swizzle
#pragma unroll
    for (int p = 0; p < NI; ++p) {
      const u32x2 lo = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)&v[p][t][f]));
      const u32x2 hi = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)&v[p][t + 16][f]));
      r.p[p] = cat(lo, hi);
    }
    return r;
  }
  // Four features of one token in fp32.
  __device__ __forceinline__ f32x4 four(int t, int f) const {
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = NI - 1; p >= 0; --p) x += widen4(get4(p, t, f));
    return x;
  }
};

// A range of memory for buffer loads and stores: reads past `bytes` give zero,
// stores past it do nothing, so a tile's missing rows need no branches.  `bytes`
// is the same in every lane; made a scalar here, as a clamp (a vector instruction)
// would put it, and with it the descriptor, in vector registers and a loop
// around every access.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const void* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), static_cast<short>(0),
                                           __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}

// A tile's rows on their way from memory: 16 bytes per vector, rows from
// `valid` on are zero.
template <int NI, int L, int W, int THREADS>
struct Fetch {
  static constexpr int VE = NI == 1 ? 8 : 4;                 // values of a 16-byte vector
  static constexpr int VECS = L * W / VE, PER = (VECS + THREADS - 1) / THREADS;
  static constexpr int RB = W * (NI == 1 ? 2 : 4);           // bytes of a row
  u32x4 r[PER];

  // src: the tile's first row ([L][W] contiguous); nothing is read for valid <= 0
  __device__ __forceinline__ void load(const void* src, int valid, int tid) {
    const __amdgpu_buffer_rsrc_t m = rows_of(src, max(valid, 0) * RB);
#pragma unroll
    for (int j = 0; j < PER; ++j)
      r[j] = __builtin_bit_cast(
          u32x4, __builtin_amdgcn_raw_buffer_load_b128(m, 16 * (tid + THREADS * j), 0, 0));
  }
  __device__ __forceinline__ void store(Plane<NI, L, W>& to, int tid) const {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = tid + THREADS * j;
      if (VECS % THREADS != 0 && i >= VECS) break;
      const int row = i * VE / W, col = i * VE % W;
      if constexpr (NI == 1) {
        *reinterpret_cast<u32x4*>(&to.v[0][row][to.place(row, col)]) = r[j];
      } else {
        u32x2 p[NI];
        split_parts<NI>(__builtin_bit_cast(f32x4, r[j]), p);
#pragma unroll
        for (int k = 0; k < NI; ++k) to.put4(k, row, col, p[k]);
      }
    }
  }
};

// Four values of row t, feature f of a [.., W] array behind `m`: fp32, or
// rounded once to bf16.
template <int NI>
__device__ __forceinline__ void store_row4(__amdgpu_buffer_rsrc_t m, int t, int W, int f,
                                           f32x4 v) {
  if constexpr (NI == 1) {
    typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));
    __builtin_amdgcn_raw_buffer_store_b64(
        u32x2v{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])}, m, (t * W + f) * 2, 0, 0);
  } else {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), m, (t * W + f) * 4, 0,
                                           0);
  }
}

// Inclusive sum over the wave's lanes (DPP row shifts, then row broadcasts).
__device__ __forceinline__ double wave_scan(double v) {
#define TTT_SCAN_STEP(ctrl, rows)                                                           \
  {                                                                                         \
    const uint64_t b = __builtin_bit_cast(uint64_t, v);                                     \
    const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(                  \
        0, static_cast<int>(b & 0xffffffffu), ctrl, rows, 0xf, false));                     \
    const uint32_t hi = static_cast<uint32_t>(                                              \
        __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), ctrl, rows, 0xf, false)); \
    v += __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);                \
  }
  TTT_SCAN_STEP(0x111, 0xf)   // row_shr 1, 2, 4, 8: within 16 lanes
  TTT_SCAN_STEP(0x112, 0xf)
  TTT_SCAN_STEP(0x114, 0xf)
  TTT_SCAN_STEP(0x118, 0xf)
  TTT_SCAN_STEP(0x142, 0xa)   // row_bcast 15: rows 1 and 3 take their left row's total
  TTT_SCAN_STEP(0x143, 0xc)   // row_bcast 31: rows 2 and 3 take the first half's total
#undef TTT_SCAN_STEP
  return v;
}

__device__ __forceinline__ double lane_of(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b & 0xffffffffu), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), lane);
  return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}

__device__ __forceinline__ double last_lane(double v) { return lane_of(v, 63); }

__device__ __forceinline__ float exp2_raw(float x) { return __builtin_amdgcn_exp2f(x); }

// The steps dt of a tile, lane = token; zero from `valid` on.
__device__ __forceinline__ float load_steps(const float* dt, int valid, int lane) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_raw_buffer_load_b32(rows_of(dt, max(valid, 0) * 4), 4 * lane, 0, 0));
}

// Per-token values of a tile.  cum_t = log2(e) a (dt_0 + ... + dt_t) is summed
// in fp64, and every decay is made from a difference of two of them rounded
// once, so that it keeps fp32's relative precision also behind a large step
// that resets the state.  Decays between tokens of different 16-token blocks
// are products of two factors that meet at the later block's start; those
// within a block are made one by one from cum = hi + lo.
template <int L>
struct alignas(16) Tokens {
  float hi[L], lo[L];        // cum
  float dt[L];
  float head[L];             // exp2(cum_t): from the tile's start through token t
  float tail[L];             // exp2(cum_last - cum_t): from token t to the tile's end
  float into[L];             // tail dt: what the token's input weighs in the state behind the tile
  float row[L];              // exp2(cum_t - cum before t's block)
  float col[L / 16 - 1][L];  // [tb - 1][s], s before block tb: exp2(cum before tb - cum_s)
  float fade;                // exp2(cum_last)

  // By one wave; lane = token, dt = 0 from the tile's valid tokens on.
  // Returns log2 of the whole tile's decay.
  __device__ __forceinline__ double fill(float step, float a, int lane) {
    constexpr double LOG2E = 1.4426950408889634074;
    const double cum = wave_scan(static_cast<double>(step) * (static_cast<double>(a) * LOG2E));
    const double all = lane_of(cum, 63);
    double before = 0.0;     // cum before the lane's block
#pragma unroll
    for (int tb = 1; tb < L / 16; ++tb) {
      const double start = lane_of(cum, 16 * tb - 1);
      if (lane >= 16 * tb) before = start;
      else col[tb - 1][lane] = exp2_raw(static_cast<float>(start - cum));
    }
    if (lane < L) {
      const float h = static_cast<float>(cum);
      hi[lane] = h;
      lo[lane] = static_cast<float>(cum - static_cast<double>(h));
      dt[lane] = step;
      head[lane] = exp2_raw(h);
      const float to_end = exp2_raw(static_cast<float>(all - cum));
      tail[lane] = to_end;
      into[lane] = to_end * step;
      row[lane] = exp2_raw(static_cast<float>(cum - before));
    }
    if (lane == 0) fade = exp2_raw(static_cast<float>(all));
    return all;
  }
  // exp of the decay exponents summed over tokens s+1 .. t for s = s0 .. s0 + 3
  // of block sb and one t of block tb; 0 where s > t
  __device__ __forceinline__ f32x4 fades(int tb, int sb, int t, int s0) const {
    if (sb < tb) return *reinterpret_cast<const f32x4*>(&col[tb - 1][s0]) * row[t];
    const f32x4 h = *reinterpret_cast<const f32x4*>(&hi[s0]);
    const f32x4 l = *reinterpret_cast<const f32x4*>(&lo[s0]);
    f32x4 w;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float e = exp2_raw((hi[t] - h[r]) + (lo[t] - l[r]));
      w[r] = s0 + r <= t ? e : 0.f;
    }
    return w;
  }
  __device__ __forceinline__ f32x4 steps(int s0) const {
    return *reinterpret_cast<const f32x4*>(&dt[s0]);
  }
};

// The tokens x tokens blocks on and below the diagonal, in order of t then s:
// block index of (tb, sb) = tb (tb + 1) / 2 + sb.
__device__ __forceinline__ void block_of(int i, int* tb, int* sb) {
  int t = 0;
  while (i > t) {
    i -= t + 1;
    ++t;
  }
  *tb = t;
  *sb = i;
}

// One wave's 16x16 block of a tokens x tokens matrix as an operand: lane's
// four values (rows 4 g + 0..3) in NP parts, at the lane's own place.
template <int NP, int BLOCKS>
struct Blocks {
  u32x2 v[BLOCKS][NP][64];

  __device__ __forceinline__ void put(int i, int lane, f32x4 x) {
    u32x2 p[NP];
    split_parts<NP>(x, p);
#pragma unroll
    for (int k = 0; k < NP; ++k) v[i][k][lane] = p[k];
  }
};

template <int NI>
constexpr int kSsmTile = NI == 1 ? 64 : 32;

template <int NI>
__device__ __forceinline__ const char* row_ptr(const void* p, size_t row, int width) {
  return static_cast<const char*>(p) + row * width * (NI == 1 ? 2 : 4);
}

// The wave's number as a scalar, so that what depends on it alone is worked out
// once per wave and branches on it are branches.
__device__ __forceinline__ int wave_of(int tid) { return __builtin_amdgcn_readfirstlane(tid >> 6); }

// A lane index that the compiler takes for a new value: LDS addresses made from
// it are made where they are used and not kept in registers around the loop.
__device__ __forceinline__ int anew(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Which unit and segment a workgroup works on (`count` segments per unit), as
// scalars: the divisions run on vector registers.
struct Place {
  int seg, h;
  size_t unit, shared;   // shared: the row of the head's group in b and c
  __device__ __forceinline__ Place(const SsmArgs& a, uint32_t id, int count) {
    const uint32_t u = __builtin_amdgcn_readfirstlane(id / count);
    seg = id - u * count;
    const uint32_t b = __builtin_amdgcn_readfirstlane(u / a.H);
    h = u - b * a.H;
    unit = u;
    shared = static_cast<size_t>(b) * a.G +
             __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(h) / (a.H / a.G));
  }
};

// S = fade S + B^T diag(w) X over a tile, w by token: rows 16 i0 .. of S, COUNT
// blocks of 16, from A = B^T, the features 16 pb .. of x from the weighted X,
// in three parts.
template <int COUNT, int NI, int L, int N>
__device__ __forceinline__ void add_tile(f32x4 (&S)[COUNT], const Plane<NI, L, N>& b, int i0,
                                         const Plane<NI, L, SSM_P>& x, int pb, float fade,
                                         const float (&weight)[L], int g, int c) {
#pragma unroll
  for (int i = 0; i < COUNT; ++i) S[i] *= fade;
#pragma unroll
  for (int k = 0; k < L / 32; ++k) {
    const Parts<NI> xs = x.cols(32 * k, 16 * pb, g, c);
    f32x4 w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      w[h] = frag_half(xs, h) *
             *reinterpret_cast<const f32x4*>(&weight[32 * k + 16 * h + 4 * g]);
    const Parts<3> xw = split_frag<3>(w[0], w[1]);
#pragma unroll
    for (int i = 0; i < COUNT; ++i)
      S[i] = mfma_parts(b.cols(32 * k, 16 * (i0 + i), g, c), xw, S[i]);
  }
}

// Which unit and place in its state (N P / 4 vectors, 256 a workgroup) a thread
// of a joining workgroup takes.
struct JoinPlace {
  size_t unit, at;
  __device__ __forceinline__ JoinPlace(int N, uint32_t block, int tid) {
    const uint32_t each = N * SSM_P / 4 / SSM_NT, u = __builtin_amdgcn_readfirstlane(block / each);
    unit = u;
    at = 4 * ((block - u * each) * SSM_NT + tid);
  }
};

// The states of segments, each slot (`size` floats apart) holding what its
// segment adds, become the states in front of them, starting from S;
// `count` segments' additions are used and `slots` slots written.  dir = 1:
// first segment to last, -1: last to first.  Returns the state behind.  The
// loads of sixteen segments are issued together; the fades, the same in every
// lane and written by an earlier launch, go through scalar loads.
__device__ __forceinline__ f32x4 join_segments(float* p, int64_t size, const double* fades,
                                               int slots, int count, int dir, f32x4 S) {
  constexpr int AT_ONCE = 16;
  typedef __attribute__((address_space(4))) const double* constant;
  const constant scalar = (constant)fades;
  for (int s0 = 0; s0 < slots; s0 += AT_ONCE) {
    f32x4 added[AT_ONCE];
    float fade[AT_ONCE];
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k)
      if (s0 + k < count) {
        added[k] = *reinterpret_cast<const f32x4*>(p + dir * (s0 + k) * size);
        fade[k] = static_cast<float>(scalar[dir * (s0 + k)]);
      }
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      const int s = s0 + k;
      if (s < slots) *reinterpret_cast<f32x4*>(p + dir * s * size) = S;
      if (s < count) S = S * exp2_raw(fade[k]) + added[k];
    }
  }
  return S;
}

}  // namespace tttk
