// ttt_block_validate.cpp -- host-side argument checks of the RMS norm, the
// 8-bit input projection, the short convolution and the selective state
// space scan: shapes, types, null pointers, alignment, aliasing and workspace
// sizes, and the fill of the launch arguments.  Plain C++ (no HIP).
#include "ttt_block_validate.hpp"

#include <cmath>
#include <cstdint>
#include <initializer_list>

namespace tttv {
namespace {

constexpr int32_t kHeadDim = 64;
constexpr int32_t kMaxT = 1 << 22;         // tokens per unit, as in the TTT scans
constexpr uint64_t kMaxTokens = 1ull << 40;
// A launch holds fewer than 2^32 threads, and the kernels count workgroups in
// 32 bits: the most units of the convolution and of the scan, and workgroups
constexpr uint64_t kConvMaxUnits = 1ull << 23, kSsmMaxUnits = 1ull << 20;
constexpr uint64_t kMaxWorkgroups = 1ull << 22;

struct Range {
  uintptr_t lo, hi;  // [lo, hi); lo == 0: not given
};

Range span(const void* p, uint64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Range{a, a + static_cast<uintptr_t>(bytes)};
}

bool overlap(Range a, Range b) {
  if (a.lo == a.hi || b.lo == b.hi || a.lo == 0 || b.lo == 0) return false;
  return a.lo < b.hi && b.lo < a.hi;
}

// Every output against every input and every other output.
bool any_overlap(std::initializer_list<Range> outputs, std::initializer_list<Range> inputs) {
  for (const Range* o = outputs.begin(); o != outputs.end(); ++o) {
    for (const Range& r : inputs)
      if (overlap(*o, r)) return true;
    for (const Range* o2 = o + 1; o2 != outputs.end(); ++o2)
      if (overlap(*o, *o2)) return true;
  }
  return false;
}

// The kernels use 16-byte accesses (a null pointer counts as aligned).
bool misaligned(std::initializer_list<const void*> ptrs, uintptr_t to = 16) {
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) % to != 0) return true;
  return false;
}

bool io_size(int32_t io_dtype, uint64_t* es) {
  if (io_dtype != TTT_F32 && io_dtype != TTT_BF16) return false;
  *es = io_dtype == TTT_BF16 ? 2 : 4;
  return true;
}

uint64_t up256(uint64_t n) { return (n + 255) / 256 * 256; }

// B, H, T and io_dtype of p; *units = B H, *es = bytes of one io value.
ttt_status check_shape(const ttt_params* p, uint64_t* units, uint64_t* es) {
  if (!p) return TTT_ERR_NULL;
  if (!io_size(p->io_dtype, es)) return TTT_ERR_ARG;
  if (p->B < 1 || p->H < 1 || p->T < 1 || p->d < 1 || p->T > kMaxT) return TTT_ERR_SHAPE;
  *units = static_cast<uint64_t>(p->B) * static_cast<uint64_t>(p->H);
  if (*units > 0x7fffffffull || *units * static_cast<uint64_t>(p->T) > kMaxTokens)
    return TTT_ERR_SHAPE;
  return TTT_OK;
}

// ---- norm ----

constexpr int32_t kNormMaxWidth = 16384;   // a row stays in one workgroup's registers
constexpr int32_t kNormGroups = 512;

ttt_status check_norm(int64_t rows, int32_t width, int32_t io_dtype, float eps, uint64_t* es) {
  if (!io_size(io_dtype, es)) return TTT_ERR_ARG;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return TTT_ERR_ARG;
  if (rows < 1 || width < 1 || rows > (1ll << 40)) return TTT_ERR_SHAPE;
  if (width % 8 != 0 || width > kNormMaxWidth) return TTT_ERR_UNSUPPORTED;
  return TTT_OK;
}

// ---- convolution ----

constexpr int32_t kConvMaxDim = 1024;

ttt_status check_conv(const ttt_params* p, int32_t taps, uint32_t flags, uint64_t* units,
                      uint64_t* es) {
  const ttt_status st = check_shape(p, units, es);
  if (st != TTT_OK) return st;
  if (flags & ~static_cast<uint32_t>(TTT_CONV_SILU)) return TTT_ERR_ARG;
  if (taps < 1) return TTT_ERR_SHAPE;
  if (taps < 2 || taps > 4 || p->d % 8 != 0 || p->d > kConvMaxDim) return TTT_ERR_UNSUPPORTED;
  if (*units > kConvMaxUnits) return TTT_ERR_SHAPE;
  return TTT_OK;
}

int32_t conv_chunks(const ttt_params* p) {
  const int32_t chunk = tttk::conv_chunk(p->d);
  return (p->T + chunk - 1) / chunk;
}

// ---- scan ----

// Tokens of a tile: fp32 data keep three 16-bit parts of every value in LDS,
// so their tiles are half as long.
int32_t ssm_tile(const ttt_params* p) { return p->io_dtype == TTT_BF16 ? 64 : 32; }

struct Segments {
  int32_t tiles, segs, seg_tiles;
};

// Time segments of one unit: as many as fill the card once (B4 H32 T8192 N64, four
// workgroups a compute unit: the scan alone with 4, 6, 8 segments 159, 144, 124 us),
// but for few units at most sqrt(40 tiles): the segments are joined one after
// another, the tiles of a segment worked on one after another, and a tile takes the
// time of some 40 joins.  N64 bf16, us, with 20 / 40 / 80 / no limit:
//   forward  B1 H2 T16384 32.2 / 32.8 / 35.3 / 50.5, B1 H1 T131072 73 / 71 / 84 / 159
//   backward              54.0 / 51.2 / 49.5 / 63.1                127 / 118 / 135 / 142
Segments ssm_segments(const ttt_params* p, uint64_t workgroups) {
  const uint64_t units = static_cast<uint64_t>(p->B) * p->H;
  const int32_t tile = ssm_tile(p);
  Segments s;
  s.tiles = (p->T + tile - 1) / tile;
  uint64_t segs = workgroups / units;
  if (segs > static_cast<uint64_t>(s.tiles)) segs = s.tiles;
  const uint64_t most = static_cast<uint64_t>(std::sqrt(40.0 * s.tiles));
  if (segs > most) segs = most;
  if (segs < 1) segs = 1;
  s.seg_tiles = static_cast<int32_t>((s.tiles + segs - 1) / segs);
  s.segs = (s.tiles + s.seg_tiles - 1) / s.seg_tiles;
  return s;
}

// Workgroups that 256 compute units hold at once (by their LDS and registers).
uint64_t scan_workgroups(const ttt_params* p, int32_t n) {
  if (n == 128) return 256 * 2;
  return 256 * (p->io_dtype == TTT_BF16 || n == 32 ? 4 : 3);
}
uint64_t grad_workgroups(const ttt_params* p, int32_t n) {
  return 256 * (n == 32 || (n == 64 && p->io_dtype == TTT_BF16) ? 2 : 1);
}

ttt_status check_ssm(const ttt_params* p, int32_t groups, int32_t n, uint64_t* units,
                     uint64_t* es) {
  const ttt_status st = check_shape(p, units, es);
  if (st != TTT_OK) return st;
  if (groups < 1 || groups > p->H || p->H % groups != 0 || n < 1) return TTT_ERR_SHAPE;
  if (p->d != kHeadDim || (n != 32 && n != 64 && n != 128)) return TTT_ERR_UNSUPPORTED;
  if (*units > kSsmMaxUnits) return TTT_ERR_SHAPE;
  return TTT_OK;
}

uint64_t state_bytes(int32_t n) { return static_cast<uint64_t>(n) * kHeadDim * 4; }

struct ForwardLayout {
  uint64_t fade, total;
};
ForwardLayout ssm_layout(const ttt_params* p, int32_t n) {
  const Segments s = ssm_segments(p, scan_workgroups(p, n));
  const uint64_t units = static_cast<uint64_t>(p->B) * p->H;
  ForwardLayout ly{0, 0};
  if (s.segs > 1) {
    ly.fade = units * s.segs * state_bytes(n);
    ly.total = up256(ly.fade + units * s.segs * 8);
  }
  return ly;
}

struct BackwardLayout {
  uint64_t seg, fade, adj, tile, sums, db, dc, total;
};
BackwardLayout ssm_backward_layout(const ttt_params* p, int32_t groups, int32_t n) {
  const Segments s = ssm_segments(p, grad_workgroups(p, n));
  const uint64_t units = static_cast<uint64_t>(p->B) * p->H;
  const uint64_t sb = state_bytes(n);
  BackwardLayout ly;
  ly.seg = 0;                                                   // [units][segs] states
  ly.adj = ly.seg + units * s.segs * sb;                        // [units][segs] adjoints
  ly.tile = ly.adj + units * s.segs * sb;                       // [units][tiles] states
  ly.fade = ly.tile + units * s.tiles * sb;
  ly.sums = ly.fade + up256(units * s.segs * 8);
  ly.db = ly.sums + up256(units * s.segs * 8);
  ly.dc = ly.db;
  ly.total = ly.db;
  if (groups != p->H) {
    const uint64_t per_head = up256(units * p->T * static_cast<uint64_t>(n) * 4);
    ly.dc = ly.db + per_head;
    ly.total = ly.dc + per_head;
  }
  return ly;
}

void fill_ssm(const ttt_params* p, int32_t groups, int32_t n, const void* x, const float* dt,
              const float* a, const void* b, const void* c, const float* d_skip,
              const float* state0, tttk::SsmArgs* out) {
  *out = tttk::SsmArgs{};
  out->x = x;
  out->dt = dt;
  out->a = a;
  out->b = b;
  out->c = c;
  out->d_skip = d_skip;
  out->state0 = state0;
  out->B = p->B;
  out->H = p->H;
  out->G = groups;
  out->T = p->T;
  out->N = n;
  out->tile = ssm_tile(p);
}

}  // namespace

// ---- RMS norm ---------------------------------------------------------------

ttt_status rms_norm(int64_t rows, int32_t width, int32_t io_dtype, float eps, const void* x,
                    const void* residual, const float* weight, void* y, bool f8, float* scale,
                    void* res_out, tttk::NormArgs* a) {
  uint64_t es = 0;
  const ttt_status st = check_norm(rows, width, io_dtype, eps, &es);
  if (st != TTT_OK) return st;
  if (!x || !weight || !y || (f8 && !scale)) return TTT_ERR_NULL;
  if (!residual != !res_out) return TTT_ERR_NULL;   // both or neither
  if (misaligned({x, residual, weight, y, res_out})) return TTT_ERR_ARG;
  const uint64_t n = static_cast<uint64_t>(rows) * width;
  const Range rx = span(x, n * es), rr = span(residual, n * es), rw = span(weight, width * 4ull);
  const Range ry = span(y, n * (f8 ? 1 : es)), ro = span(res_out, n * es);
  const Range rs = span(f8 ? scale : nullptr, rows * 4ull);
  const bool in_place = res_out && res_out == residual;
  if (any_overlap({ry, rs, ro}, {rx, rw}) || any_overlap({ry, rs}, {rr}) ||
      (!in_place && overlap(ro, rr)))
    return TTT_ERR_ALIAS;
  a->x = x;
  a->residual = residual;
  a->weight = weight;
  a->y = y;
  a->scale = f8 ? scale : nullptr;
  a->res_out = res_out;
  a->rows = rows;
  a->width = width;
  a->eps = eps;
  return TTT_OK;
}

int32_t norm_groups(int64_t rows) {
  const int64_t g = (rows + 3) / 4;   // four rows, one per wave, at least
  return static_cast<int32_t>(g < kNormGroups ? g : kNormGroups);
}

uint64_t rms_norm_backward_workspace_bytes(int64_t rows, int32_t width) {
  uint64_t es = 0;
  if (check_norm(rows, width, TTT_F32, 0.0f, &es) != TTT_OK) return 0;
  return up256(static_cast<uint64_t>(norm_groups(rows)) * width * 4);
}

ttt_status rms_norm_backward(int64_t rows, int32_t width, int32_t io_dtype, float eps,
                             const void* r, const float* weight, const void* dy, const void* dr,
                             void* dx, float* dweight, void* workspace, uint64_t workspace_bytes,
                             tttk::NormBackwardArgs* a) {
  uint64_t es = 0;
  const ttt_status st = check_norm(rows, width, io_dtype, eps, &es);
  if (st != TTT_OK) return st;
  if (!r || !weight || !dy || !dx || !dweight || !workspace) return TTT_ERR_NULL;
  if (workspace_bytes < rms_norm_backward_workspace_bytes(rows, width)) return TTT_ERR_SHAPE;
  if (misaligned({r, weight, dy, dr, dx}) || misaligned({workspace}, 256)) return TTT_ERR_ARG;
  const uint64_t n = static_cast<uint64_t>(rows) * width;
  if (any_overlap({span(dx, n * es), span(dweight, width * 4ull),
                   span(workspace, workspace_bytes)},
                  {span(r, n * es), span(weight, width * 4ull), span(dy, n * es),
                   span(dr, n * es)}))
    return TTT_ERR_ALIAS;
  a->r = r;
  a->weight = weight;
  a->dy = dy;
  a->dr = dr;
  a->dx = dx;
  a->dweight = dweight;
  a->partial = static_cast<float*>(workspace);
  a->rows = rows;
  a->width = width;
  a->groups = norm_groups(rows);
  a->eps = eps;
  return TTT_OK;
}

// ---- 8-bit input projection -------------------------------------------------

ttt_status input_projection_f8(const ttt_params* p, int32_t d_model, const void* x,
                               const float* x_scale, const void* w_in, const float* w_scale,
                               const float* b_eta, float eta_base, void* q, void* k, void* v,
                               float* eta, tttk::InputF8Args* a) {
  uint64_t units = 0, es = 0;
  const ttt_status st = check_shape(p, &units, &es);
  if (st != TTT_OK) return st;
  if (!x || !x_scale || !w_in || !w_scale || !b_eta || !q || !k || !v || !eta)
    return TTT_ERR_NULL;
  if (d_model < 1) return TTT_ERR_SHAPE;
  if (p->d != kHeadDim || p->io_dtype != TTT_BF16 || d_model % 64 != 0 || d_model > (1 << 20))
    return TTT_ERR_UNSUPPORTED;
  if (!(eta_base > 0.0f) || !std::isfinite(eta_base)) return TTT_ERR_ARG;
  if (misaligned({x, w_in, q, k, v})) return TTT_ERR_ARG;
  const uint64_t tokens = static_cast<uint64_t>(p->B) * p->T;
  const uint64_t n_out = 3ull * p->H * kHeadDim + p->H;
  // the kernel indexes rows, columns and tiles (128 x 128 at the smallest for many rows) with int
  if (tokens > (1ull << 30) || n_out > (1ull << 30) ||
      ((tokens + 127) / 128) * ((n_out + 31) / 32) > kMaxWorkgroups * 2)
    return TTT_ERR_SHAPE;
  const uint64_t elems = units * p->T * kHeadDim;
  if (any_overlap({span(q, elems * 2), span(k, elems * 2), span(v, elems * 2),
                   span(eta, tokens * p->H * 4ull)},
                  {span(x, tokens * d_model), span(x_scale, tokens * 4),
                   span(w_in, n_out * d_model), span(w_scale, n_out * 4),
                   span(b_eta, p->H * 4ull)}))
    return TTT_ERR_ALIAS;
  a->x = x;
  a->x_scale = x_scale;
  a->w = w_in;
  a->w_scale = w_scale;
  a->b_eta = b_eta;
  a->q = q;
  a->k = k;
  a->v = v;
  a->eta = eta;
  a->B = p->B;
  a->T = p->T;
  a->D = d_model;
  a->H = p->H;
  a->eta_base = eta_base;
  return TTT_OK;
}

// ---- short causal convolution -----------------------------------------------

ttt_status conv_forward(const ttt_params* p, int32_t taps, uint32_t flags, const void* x,
                        const float* w, const float* bias, const void* state0, void* y,
                        void* state_out, tttk::ConvArgs* a) {
  uint64_t units = 0, es = 0;
  const ttt_status st = check_conv(p, taps, flags, &units, &es);
  if (st != TTT_OK) return st;
  if (!x || !w || !y) return TTT_ERR_NULL;
  if (misaligned({x, w, bias, state0, y, state_out})) return TTT_ERR_ARG;
  const uint64_t row = static_cast<uint64_t>(p->d) * es;
  const uint64_t data = units * p->T * row, tail = units * (taps - 1) * row;
  const uint64_t wb = 4ull * p->H * p->d;
  if (any_overlap({span(y, data), span(state_out, tail)},
                  {span(x, data), span(w, wb * taps), span(bias, wb), span(state0, tail)}))
    return TTT_ERR_ALIAS;
  *a = tttk::ConvArgs{x, w, bias, state0, y, state_out, p->B, p->H, p->T, p->d, taps,
                      (flags & TTT_CONV_SILU) ? 1 : 0};
  return TTT_OK;
}

ttt_status conv_decode(const ttt_params* p, int32_t taps, uint32_t flags, const void* x,
                       const float* w, const float* bias, void* state, void* y,
                       tttk::ConvArgs* a) {
  if (p && p->T != 1) return TTT_ERR_SHAPE;  // one token per unit
  if (p && !state) return TTT_ERR_NULL;
  const ttt_status st = conv_forward(p, taps, flags, x, w, bias, nullptr, y, state, a);
  if (st != TTT_OK) return st;
  a->state0 = state;
  return TTT_OK;
}

uint64_t conv_backward_workspace_bytes(const ttt_params* p, int32_t taps) {
  uint64_t units = 0, es = 0;
  if (check_conv(p, taps, 0, &units, &es) != TTT_OK) return 0;
  return up256(units * conv_chunks(p) * (taps + 1) * static_cast<uint64_t>(p->d) * 4);
}

ttt_status conv_backward(const ttt_params* p, int32_t taps, uint32_t flags, const void* x,
                         const float* w, const float* bias, const void* state0, const void* dy,
                         const void* dstate, void* dx, float* dw, float* dbias, void* dstate0,
                         void* workspace, uint64_t workspace_bytes, tttk::ConvBackwardArgs* a) {
  uint64_t units = 0, es = 0;
  const ttt_status st = check_conv(p, taps, flags, &units, &es);
  if (st != TTT_OK) return st;
  if (units * conv_chunks(p) > kMaxWorkgroups ||
      static_cast<uint64_t>(p->H) * (taps + 1) * p->d / 16 > kMaxWorkgroups)
    return TTT_ERR_SHAPE;
  if (!x || !w || !dy || !dx || !dw || !dbias || !workspace) return TTT_ERR_NULL;
  if (workspace_bytes < conv_backward_workspace_bytes(p, taps)) return TTT_ERR_SHAPE;
  if (misaligned({x, w, bias, state0, dy, dstate, dx, dw, dbias, dstate0}) ||
      misaligned({workspace}, 256))
    return TTT_ERR_ARG;
  const uint64_t row = static_cast<uint64_t>(p->d) * es;
  const uint64_t data = units * p->T * row, tail = units * (taps - 1) * row;
  const uint64_t wb = 4ull * p->H * p->d;
  if (any_overlap({span(dx, data), span(dw, wb * taps), span(dbias, wb), span(dstate0, tail),
                   span(workspace, workspace_bytes)},
                  {span(x, data), span(w, wb * taps), span(bias, wb), span(state0, tail),
                   span(dy, data), span(dstate, tail)}))
    return TTT_ERR_ALIAS;
  *a = tttk::ConvBackwardArgs{x, w, bias, state0, dy, dstate, dx, dw, dbias, dstate0,
                              static_cast<float*>(workspace), p->B, p->H, p->T, p->d, taps,
                              (flags & TTT_CONV_SILU) ? 1 : 0, tttk::conv_chunk(p->d), conv_chunks(p)};
  return TTT_OK;
}

// ---- selective state space scan ---------------------------------------------

uint64_t ssm_forward_workspace_bytes(const ttt_params* p, int32_t groups, int32_t n) {
  uint64_t units = 0, es = 0;
  if (check_ssm(p, groups, n, &units, &es) != TTT_OK) return 0;
  return ssm_layout(p, n).total;
}

ttt_status ssm_forward(const ttt_params* p, int32_t groups, int32_t n, const void* x,
                       const float* dt, const float* a, const void* b, const void* c,
                       const float* d_skip, const float* state0, void* y, float* state_out,
                       void* workspace, uint64_t workspace_bytes, tttk::SsmArgs* out) {
  uint64_t units = 0, es = 0;
  const ttt_status st = check_ssm(p, groups, n, &units, &es);
  if (st != TTT_OK) return st;
  if (!x || !dt || !a || !b || !c || !y) return TTT_ERR_NULL;
  const ForwardLayout ly = ssm_layout(p, n);
  if (ly.total && !workspace) return TTT_ERR_NULL;
  if (workspace && workspace_bytes < ly.total) return TTT_ERR_SHAPE;
  if (misaligned({x, b, c, state0, y, state_out}) || misaligned({workspace}, 256))
    return TTT_ERR_ARG;
  const uint64_t data = units * p->T * kHeadDim * es, sb = units * state_bytes(n);
  const uint64_t shared = static_cast<uint64_t>(p->B) * groups * p->T * n * es;
  if (any_overlap({span(y, data), span(state_out, sb),
                   span(workspace, workspace ? workspace_bytes : 0)},
                  {span(x, data), span(dt, units * p->T * 4), span(a, p->H * 4ull),
                   span(b, shared), span(c, shared), span(d_skip, p->H * 4ull)}) ||
      overlap(span(y, data), span(state0, sb)) ||
      overlap(span(workspace, workspace ? workspace_bytes : 0), span(state0, sb)) ||
      (state_out != state0 && overlap(span(state_out, sb), span(state0, sb))))
    return TTT_ERR_ALIAS;
  fill_ssm(p, groups, n, x, dt, a, b, c, d_skip, state0, out);
  out->y = y;
  out->state_out = state_out;
  const Segments s = ssm_segments(p, scan_workgroups(p, n));
  out->segs = s.segs;
  out->seg_tiles = s.seg_tiles;
  if (s.segs > 1) {
    out->ws_state = static_cast<float*>(workspace);
    out->ws_fade = reinterpret_cast<double*>(static_cast<char*>(workspace) + ly.fade);
  }
  return TTT_OK;
}

ttt_status ssm_decode(const ttt_params* p, int32_t groups, int32_t n, const void* x,
                      const float* dt, const float* a, const void* b, const void* c,
                      const float* d_skip, float* state, void* y, tttk::SsmArgs* out) {
  uint64_t units = 0, es = 0;
  const ttt_status st = check_ssm(p, groups, n, &units, &es);
  if (st != TTT_OK) return st;
  if (p->T != 1) return TTT_ERR_SHAPE;  // one token per unit
  if (!x || !dt || !a || !b || !c || !state || !y) return TTT_ERR_NULL;
  if (misaligned({x, b, c, state, y})) return TTT_ERR_ARG;
  const uint64_t data = units * kHeadDim * es;
  const uint64_t shared = static_cast<uint64_t>(p->B) * groups * n * es;
  if (any_overlap({span(y, data), span(state, units * state_bytes(n))},
                  {span(x, data), span(dt, units * 4), span(a, p->H * 4ull), span(b, shared),
                   span(c, shared), span(d_skip, p->H * 4ull)}))
    return TTT_ERR_ALIAS;
  fill_ssm(p, groups, n, x, dt, a, b, c, d_skip, state, out);
  out->y = y;
  out->state_out = state;
  out->segs = 1;
  out->seg_tiles = 1;
  return TTT_OK;
}

uint64_t ssm_backward_workspace_bytes(const ttt_params* p, int32_t groups, int32_t n) {
  uint64_t units = 0, es = 0;
  if (check_ssm(p, groups, n, &units, &es) != TTT_OK) return 0;
  return ssm_backward_layout(p, groups, n).total;
}

ttt_status ssm_backward(const ttt_params* p, int32_t groups, int32_t n, const void* x,
                        const float* dt, const float* a, const void* b, const void* c,
                        const float* d_skip, const float* state0, const void* dy,
                        const float* dstate, void* dx, float* ddt, float* da, void* db, void* dc,
                        float* dd, float* dstate0, void* workspace, uint64_t workspace_bytes,
                        tttk::SsmBackwardArgs* out) {
  uint64_t units = 0, es = 0;
  const ttt_status st = check_ssm(p, groups, n, &units, &es);
  if (st != TTT_OK) return st;
  if (!x || !dt || !a || !b || !c || !dy || !dx || !ddt || !da || !db || !dc || !workspace)
    return TTT_ERR_NULL;
  if (!d_skip != !dd) return TTT_ERR_NULL;          // both or neither
  const BackwardLayout ly = ssm_backward_layout(p, groups, n);
  if (workspace_bytes < ly.total) return TTT_ERR_SHAPE;
  if (misaligned({x, b, c, state0, dy, dstate, dx, db, dc, dstate0}) ||
      misaligned({workspace}, 256))
    return TTT_ERR_ARG;
  const uint64_t data = units * p->T * kHeadDim * es, sb = units * state_bytes(n);
  const uint64_t shared = static_cast<uint64_t>(p->B) * groups * p->T * n * es;
  const uint64_t steps = units * p->T * 4, heads = p->H * 4ull;
  if (any_overlap({span(dx, data), span(ddt, steps), span(da, heads), span(db, shared),
                   span(dc, shared), span(dd, heads), span(dstate0, sb),
                   span(workspace, workspace_bytes)},
                  {span(x, data), span(dt, steps), span(a, heads), span(b, shared),
                   span(c, shared), span(d_skip, heads), span(state0, sb), span(dy, data),
                   span(dstate, sb)}))
    return TTT_ERR_ALIAS;
  fill_ssm(p, groups, n, x, dt, a, b, c, d_skip, state0, &out->f);
  const Segments s = ssm_segments(p, grad_workgroups(p, n));
  char* base = static_cast<char*>(workspace);
  out->f.segs = s.segs;
  out->f.seg_tiles = s.seg_tiles;
  out->f.ws_state = reinterpret_cast<float*>(base + ly.seg);
  out->f.ws_fade = reinterpret_cast<double*>(base + ly.fade);
  out->dy = dy;
  out->dstate = dstate;
  out->dx = dx;
  out->ddt = ddt;
  out->da = da;
  out->db = db;
  out->dc = dc;
  out->dd = dd;
  out->dstate0 = dstate0;
  out->ws_tile = reinterpret_cast<float*>(base + ly.tile);
  out->ws_adj = reinterpret_cast<float*>(base + ly.adj);
  out->ws_sums = reinterpret_cast<float*>(base + ly.sums);
  out->ws_db = groups != p->H ? reinterpret_cast<float*>(base + ly.db) : nullptr;
  out->ws_dc = groups != p->H ? reinterpret_cast<float*>(base + ly.dc) : nullptr;
  return TTT_OK;
}

}  // namespace tttv
