"""C ABI checks of the norm, the 8-bit projection, the convolution and the state
space scan that need no GPU: bad arguments are refused with the documented
status before anything is launched (the pointers are never dereferenced), the
workspace sizes follow their layouts, and the host checks run clean under the
sanitizers."""
import ctypes
import os
import subprocess

import pytest
import torch

from linear_rnn_ttt_amd import _lib, block_ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE, GAP = 1 << 40, 1 << 36
F32, BF16 = _lib.TTT_F32, _lib.TTT_BF16
NULL, SHAPE, UNSUP = _lib.TTT_ERR_NULL, _lib.TTT_ERR_SHAPE, _lib.TTT_ERR_UNSUPPORTED
ALIAS, ARG = _lib.TTT_ERR_ALIAS, _lib.TTT_ERR_ARG


def _addr(i, off=0):
    return ctypes.c_void_p(BASE + i * GAP + off)


def _p(**kw):
    d = dict(B=2, H=4, T=100, d=64, mini_batch=0, io_dtype=BF16, flags=99, ln_eps=-1.0,
             state0_per_batch=7)          # the fields that are not read hold nonsense
    d.update(kw)
    return _lib.TTTParams(**d)


def _ref(p):
    return ctypes.byref(p) if p is not None else None


def _args(names, ptrs):
    assert set(ptrs) <= set(names), ptrs
    return [ptrs.get(n, _addr(i + 1)) for i, n in enumerate(names)]


# ---- norm ----

def _norm(rows=100, width=512, io=BF16, eps=1e-6, f8=False, **ptrs):
    names = ["x", "res", "w", "y"] + (["scale"] if f8 else []) + ["res_out"]
    fn = _lib.lib().ttt_rms_norm_forward_f8 if f8 else _lib.lib().ttt_rms_norm_forward
    return fn(rows, width, io, ctypes.c_float(eps), *_args(names, ptrs), None)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), SHAPE), (dict(rows=-1), SHAPE), (dict(rows=(1 << 40) + 1), SHAPE),
    (dict(width=0), SHAPE), (dict(width=12), UNSUP), (dict(width=16392), UNSUP),
    (dict(io=5), ARG), (dict(eps=-1.0), ARG), (dict(eps=float("inf")), ARG),
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=None), NULL),
    (dict(res=None), NULL), (dict(res_out=None), NULL),       # both or neither
    (dict(x=_addr(1, 8)), ARG), (dict(y=_addr(4, 4)), ARG), (dict(w=_addr(3, 4)), ARG),
    (dict(y=_addr(1)), ALIAS), (dict(y=_addr(2)), ALIAS), (dict(res_out=_addr(1)), ALIAS),
    (dict(res_out=_addr(2, 16)), ALIAS), (dict(y=_addr(3)), ALIAS),
])
def test_norm_refusals(kw, code, f8):
    assert _norm(f8=f8, **kw) == code
    if f8:
        assert _norm(f8=True, scale=None) == NULL
        assert _norm(f8=True, scale=_addr(4)) == ALIAS


def _norm_bwd(rows=100, width=512, io=BF16, eps=1e-6, ws=_addr(20), nb=None, **ptrs):
    if nb is None:
        nb = _lib.lib().ttt_rms_norm_backward_workspace_bytes(rows, width)
    return _lib.lib().ttt_rms_norm_backward(
        rows, width, io, ctypes.c_float(eps),
        *_args(["r", "w", "dy", "dr", "dx", "dw"], ptrs), ws, nb, None)


def test_norm_backward_refusals():
    size = _lib.lib().ttt_rms_norm_backward_workspace_bytes
    assert size(100, 512) == 25 * 512 * 4 and size(1, 8) == 256
    assert size(100000, 768) == 512 * 768 * 4
    assert size(0, 512) == 0 and size(5, 12) == 0
    for name in ["r", "w", "dy", "dx", "dw"]:
        assert _norm_bwd(**{name: None}) == NULL, name
    assert _norm_bwd(ws=None) == NULL
    assert _norm_bwd(nb=25 * 512 * 4 - 1) == SHAPE
    assert _norm_bwd(ws=_addr(20, 128)) == ARG
    assert _norm_bwd(rows=0, nb=0) == SHAPE and _norm_bwd(width=4, nb=0) == UNSUP
    assert _norm_bwd(dx=_addr(1)) == ALIAS and _norm_bwd(dx=_addr(4)) == ALIAS
    assert _norm_bwd(dw=_addr(2)) == ALIAS and _norm_bwd(ws=_addr(5)) == ALIAS
    assert _norm_bwd(dr=_addr(4, 2)) == ARG


# ---- 8-bit projection ----

def _proj(p=None, D=128, base=0.01, **ptrs):
    a = _args(["x", "xs", "w", "ws", "b", "q", "k", "v", "eta"], ptrs)
    return _lib.lib().ttt_input_projection_f8(_ref(_p() if p is None else p), D, *a[:5],
                                              ctypes.c_float(base), *a[5:], None)


def test_projection_f8_refusals():
    for name in ["x", "xs", "w", "ws", "b", "q", "k", "v", "eta"]:
        assert _proj(**{name: None}) == NULL, name
    assert _proj(D=0) == SHAPE and _proj(D=100) == UNSUP and _proj(D=(1 << 20) + 64) == UNSUP
    assert _proj(_p(io_dtype=F32)) == UNSUP and _proj(_p(d=32)) == UNSUP
    assert _proj(_p(T=0)) == SHAPE and _proj(_p(B=1 << 12, T=1 << 19)) == SHAPE
    assert _proj(_p(B=1 << 8, T=1 << 22, H=64)) == SHAPE             # too many output tiles
    assert _proj(base=0.0) == ARG and _proj(base=float("nan")) == ARG
    assert _proj(x=_addr(1, 8)) == ARG and _proj(v=_addr(8, 2)) == ARG
    assert _proj(q=_addr(1)) == ALIAS and _proj(eta=_addr(4)) == ALIAS
    assert _proj(k=_addr(6)) == ALIAS


# ---- convolution ----

def _conv(p=None, taps=4, flags=1, **ptrs):
    a = _args(["x", "w", "bias", "s0", "y", "s1"], ptrs)
    return _lib.lib().ttt_conv_forward(_ref(_p() if p is None else p), taps, flags, *a, None)


def _conv_step(p=None, taps=4, flags=1, **ptrs):
    a = _args(["x", "w", "bias", "state", "y"], ptrs)
    return _lib.lib().ttt_conv_decode_step(_ref(_p(T=1) if p is None else p), taps, flags, *a,
                                           None)


def _conv_bwd(p=None, taps=4, flags=1, ws=_addr(30), nb=None, **ptrs):
    p = _p() if p is None else p
    if nb is None:
        nb = _lib.lib().ttt_conv_backward_workspace_bytes(_ref(p), taps)
    a = _args(["x", "w", "bias", "s0", "dy", "ds", "dx", "dw", "db", "ds0"], ptrs)
    return _lib.lib().ttt_conv_backward(_ref(p), taps, flags, *a, ws, nb, None)


BAD_CONV = [(dict(taps=0), SHAPE), (dict(taps=1), UNSUP), (dict(taps=5), UNSUP),
            (dict(flags=2), ARG)]


def test_conv_refusals():
    for call, one in ((_conv, 100), (_conv_step, 1), (_conv_bwd, 100)):
        for kw, code in BAD_CONV:
            assert call(**kw) == code, (call, kw)
        for q, code in ((dict(d=12), UNSUP), (dict(d=1032), UNSUP), (dict(d=0), SHAPE),
                        (dict(B=0), SHAPE), (dict(io_dtype=2), ARG),
                        (dict(B=1 << 12, H=(1 << 11) + 1), SHAPE)):
            assert call(_p(**{"T": one, **q})) == code, (call, q)
        assert call(x=None) == NULL and call(w=None) == NULL
        assert call(x=_addr(1, 4)) == ARG and call(bias=_addr(3, 4)) == ARG
    assert _conv(y=None) == NULL
    assert _conv(_p(T=(1 << 22) + 1)) == SHAPE
    assert _conv(y=_addr(1)) == ALIAS and _conv(s1=_addr(4)) == ALIAS and _conv(y=_addr(4)) == ALIAS
    assert _conv_step(_p(T=2)) == SHAPE and _conv_step(state=None) == NULL
    assert _conv_step(state=_addr(1)) == ALIAS and _conv_step(y=_addr(4)) == ALIAS
    assert _lib.lib().ttt_conv_forward(None, 4, 1, *[_addr(i) for i in range(6)], None) == NULL
    assert _lib.lib().ttt_conv_decode_step(None, 4, 1, *[_addr(i) for i in range(5)],
                                           None) == NULL


def test_conv_backward_refusals():
    size = lambda taps=4, **kw: _lib.lib().ttt_conv_backward_workspace_bytes(_ref(_p(**kw)), taps)
    assert size() == 2 * 4 * 5 * 64 * 4 and size(T=257) == 2 * size() and size(taps=9) == 0
    for name in ["dy", "dx", "dw", "db"]:
        assert _conv_bwd(**{name: None}) == NULL, name
    assert _conv_bwd(ws=None) == NULL and _conv_bwd(nb=size() - 1) == SHAPE
    assert _conv_bwd(ws=_addr(30, 64)) == ARG
    assert _conv_bwd(_p(B=1 << 11, H=1 << 11, T=300), nb=1 << 62) == SHAPE  # too many chunks
    assert _conv_bwd(dx=_addr(5)) == ALIAS and _conv_bwd(ds0=_addr(4)) == ALIAS
    assert _conv_bwd(dw=_addr(9)) == ALIAS and _conv_bwd(ws=_addr(7)) == ALIAS


# ---- scan ----

def _ssm(p=None, G=2, N=64, ws=_addr(30), nb=None, **ptrs):
    p = _p() if p is None else p
    if nb is None:
        nb = _lib.lib().ttt_ssm_forward_workspace_bytes(_ref(p), G, N)
    a = _args(["x", "dt", "a", "b", "c", "d", "s0", "y", "s1"], ptrs)
    return _lib.lib().ttt_ssm_forward(_ref(p), G, N, *a, ws, nb, None)


def _ssm_step(p=None, G=2, N=64, **ptrs):
    a = _args(["x", "dt", "a", "b", "c", "d", "state", "y"], ptrs)
    return _lib.lib().ttt_ssm_decode_step(_ref(_p(T=1) if p is None else p), G, N, *a, None)


def _ssm_bwd(p=None, G=2, N=64, ws=_addr(30), nb=None, **ptrs):
    p = _p() if p is None else p
    if nb is None:
        nb = _lib.lib().ttt_ssm_backward_workspace_bytes(_ref(p), G, N)
    a = _args(["x", "dt", "a", "b", "c", "d", "s0", "dy", "ds", "dx", "ddt", "da", "db", "dc",
               "dd", "ds0"], ptrs)
    return _lib.lib().ttt_ssm_backward(_ref(p), G, N, *a, ws, nb, None)


def test_ssm_refusals():
    for call, one in ((_ssm, 100), (_ssm_step, 1), (_ssm_bwd, 100)):
        for kw, code in ((dict(G=0), SHAPE), (dict(G=3), SHAPE), (dict(G=8), SHAPE),
                         (dict(N=0), SHAPE), (dict(N=16), UNSUP), (dict(N=256), UNSUP)):
            assert call(**kw) == code, (call, kw)
        for q, code in ((dict(d=32), UNSUP), (dict(H=0), SHAPE), (dict(io_dtype=9), ARG),
                        (dict(B=1 << 10, H=(1 << 10) + 2), SHAPE)):
            assert call(_p(**{"T": one, **q}), G=1 if "H" in q else 2) == code, (call, q)
        for name in ["x", "dt", "a", "b", "c"]:
            assert call(**{name: None}) == NULL, (call, name)
        assert call(x=_addr(1, 8)) == ARG and call(c=_addr(5, 2)) == ARG
    assert _ssm(y=None) == NULL and _ssm(_p(T=(1 << 22) + 1)) == SHAPE
    assert _ssm(ws=None) == NULL and _ssm(nb=100) == SHAPE and _ssm(ws=_addr(30, 16)) == ARG
    assert _ssm(y=_addr(1)) == ALIAS and _ssm(y=_addr(7)) == ALIAS and _ssm(s1=_addr(4)) == ALIAS
    assert _ssm(s1=_addr(7, 64)) == ALIAS                  # state0, but not the same buffer
    assert _ssm(ws=_addr(5)) == ALIAS and _ssm(ws=_addr(7)) == ALIAS
    assert _ssm_step(_p(T=2)) == SHAPE and _ssm_step(state=None) == NULL
    assert _ssm_step(y=None) == NULL and _ssm_step(state=_addr(4)) == ALIAS
    assert _ssm_step(y=_addr(7)) == ALIAS
    for name in ["dy", "dx", "ddt", "da", "db", "dc"]:
        assert _ssm_bwd(**{name: None}) == NULL, name
    assert _ssm_bwd(dd=None) == NULL and _ssm_bwd(d=None) == NULL       # both or neither
    assert _ssm_bwd(ws=None) == NULL and _ssm_bwd(nb=1000) == SHAPE
    assert _ssm_bwd(ws=_addr(30, 128)) == ARG
    assert _ssm_bwd(dx=_addr(8)) == ALIAS and _ssm_bwd(ds0=_addr(7)) == ALIAS
    assert _ssm_bwd(dc=_addr(13)) == ALIAS and _ssm_bwd(ws=_addr(1)) == ALIAS


def test_ssm_workspace_sizes():
    fwd, bwd = (_lib.lib().ttt_ssm_forward_workspace_bytes,
                _lib.lib().ttt_ssm_backward_workspace_bytes)
    state = 64 * 64 * 4
    # one tile, and as many units as fill the card: one segment, no workspace
    assert fwd(_ref(_p(T=64)), 2, 64) == 0 and fwd(_ref(_p(B=256)), 2, 64) == 0
    # two tiles: two segments of 8 units, and their decays
    assert fwd(_ref(_p()), 2, 64) == 8 * 2 * state + 256
    per_head = 8 * 100 * 64 * 4
    assert bwd(_ref(_p()), 2, 64) == 8 * (2 + 2 + 2) * state + 256 + 256 + 2 * per_head
    assert bwd(_ref(_p()), 4, 64) == 8 * (2 + 2 + 2) * state + 256 + 256
    assert fwd(_ref(_p()), 3, 64) == 0 and bwd(_ref(_p()), 2, 48) == 0 and bwd(None, 2, 64) == 0


def test_python_entry_points_refuse_what_is_no_gpu_tensor():
    x = torch.zeros(2, 4, 8, 64)
    w = torch.zeros(64)
    for call in (lambda: block_ops.ttt_rms_norm_forward(x, w),
                 lambda: block_ops.ttt_rms_norm_forward_f8(x, w),
                 lambda: block_ops.ttt_rms_norm_backward(x, w, x),
                 lambda: block_ops.ttt_input_projection_f8(x, x, x, x, x, heads=1, eta_base=1.0),
                 lambda: block_ops.ttt_conv_forward(x, w),
                 lambda: block_ops.ttt_conv_decode_step(x, w, None, x),
                 lambda: block_ops.ttt_conv_backward(x, w, None, x),
                 lambda: block_ops.ttt_ssm_forward(x, w, w, x, x),
                 lambda: block_ops.ttt_ssm_decode_step(x, w, w, x, x, x),
                 lambda: block_ops.ttt_ssm_backward(x, w, w, x, x, x)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(TypeError):
        block_ops.ttt_rms_norm_forward([1.0], w)


DRIVER = r"""
#include <cstdio>
#include <cstdint>
#include <initializer_list>
#include "ttt_block_validate.hpp"
static int fails = 0;
#define EXPECT(x, want) do { long long s_ = (long long)(x); if (s_ != (long long)(want)) { \
  std::printf("line %d: got %lld want %lld\n", __LINE__, s_, (long long)(want)); ++fails; } } while (0)
static char* A(int i) { return reinterpret_cast<char*>((uintptr_t(1) << 40) + uintptr_t(i) * (uintptr_t(1) << 36)); }
static float* F(int i) { return reinterpret_cast<float*>(A(i)); }
static ttt_params P(int B, int H, int T, int d = 64, int io = TTT_BF16) {
  ttt_params p{}; p.B = B; p.H = H; p.T = T; p.d = d; p.io_dtype = io; return p;
}
int main() {
  const int big = 1 << 22, most = 0x7fffffff;
  for (int B : {1, 3, 1 << 10, 1 << 20, most})
    for (int H : {1, 5, 1 << 10, most})
      for (int T : {1, 100, big, most})
        for (int io : {(int)TTT_F32, (int)TTT_BF16, 9}) {
          ttt_params p = P(B, H, T, 64, io);
          tttk::ConvArgs ca; tttk::ConvBackwardArgs cb; tttk::SsmArgs sa; tttk::SsmBackwardArgs sb;
          tttk::InputF8Args ia;
          for (int taps : {0, 2, 4, most}) {
            tttv::conv_forward(&p, taps, 1, A(1), F(2), F(3), A(4), A(5), A(6), &ca);
            tttv::conv_decode(&p, taps, 0, A(1), F(2), nullptr, A(4), A(5), &ca);
            const uint64_t n = tttv::conv_backward_workspace_bytes(&p, taps);
            tttv::conv_backward(&p, taps, 1, A(1), F(2), F(3), nullptr, A(5), nullptr, A(7), F(8), F(9),
                                nullptr, A(20), n, &cb);
          }
          for (int G : {0, 1, 5, most})
            for (int N : {32, 128, most}) {
              const uint64_t n = tttv::ssm_forward_workspace_bytes(&p, G, N);
              tttv::ssm_forward(&p, G, N, A(1), F(2), F(3), A(4), A(5), F(6), F(7), A(8), F(9), A(20), n, &sa);
              tttv::ssm_decode(&p, G, N, A(1), F(2), F(3), A(4), A(5), F(6), F(7), A(8), &sa);
              const uint64_t m = tttv::ssm_backward_workspace_bytes(&p, G, N);
              tttv::ssm_backward(&p, G, N, A(1), F(2), F(3), A(4), A(5), F(6), F(7), A(8), F(9), A(10), F(11),
                                 F(12), A(13), A(14), F(15), F(16), A(20), m, &sb);
            }
          for (int D : {64, 1 << 20, most})
            tttv::input_projection_f8(&p, D, A(1), F(2), A(3), F(4), F(5), 0.1f, A(6), A(7), A(8), F(9), &ia);
        }
  tttk::NormArgs na; tttk::NormBackwardArgs nb;
  for (long long rows : {0ll, 1ll, 1ll << 20, 1ll << 40, 0x7fffffffffffffffll})
    for (int w : {0, 8, 16384, most})
      tttv::rms_norm(rows, w, TTT_BF16, 1e-6f, A(1), A(2), F(3), A(4), true, F(5), A(6), &na),
      tttv::rms_norm_backward(rows, w, TTT_F32, 0.f, A(1), F(2), A(3), A(4), A(5), F(6), A(20),
                              tttv::rms_norm_backward_workspace_bytes(rows, w), &nb);
  {  // valid fills
    ttt_params p = P(4, 32, 8192);
    tttk::SsmArgs s;
    const uint64_t n = tttv::ssm_forward_workspace_bytes(&p, 32, 64);
    EXPECT(tttv::ssm_forward(&p, 32, 64, A(1), F(2), F(3), A(4), A(5), nullptr, F(7), A(8), F(7), A(20), n, &s), TTT_OK);
    EXPECT(s.segs, 8); EXPECT(s.seg_tiles, 16); EXPECT(s.tile, 64);
    p.T = 8193;
    EXPECT(tttv::ssm_forward(&p, 32, 64, A(1), F(2), F(3), A(4), A(5), nullptr, nullptr, A(8), nullptr, A(20),
                             tttv::ssm_forward_workspace_bytes(&p, 32, 64), &s), TTT_OK);
    EXPECT(s.segs, 8); EXPECT(s.seg_tiles, 17);     // 129 tiles: seven of 17 and ten
    tttk::ConvBackwardArgs c;
    EXPECT(tttv::conv_backward(&p, 3, 0, A(1), F(2), nullptr, nullptr, A(5), nullptr, A(7), F(8), F(9), nullptr,
                               A(20), tttv::conv_backward_workspace_bytes(&p, 3), &c), TTT_OK);
    EXPECT(c.chunks, 33); EXPECT(c.silu, 0);
  }
  std::printf("fails %d\n", fails);
  return fails != 0;
}
"""


def test_host_checks_under_sanitizers(tmp_path):
    csrc = os.path.join(ROOT, "linear_rnn_ttt_amd", "csrc")
    src, exe = tmp_path / "driver.cpp", tmp_path / "driver"
    src.write_text(DRIVER)
    subprocess.check_call(
        ["g++", "-std=c++17", "-Wall", "-g", "-O1", "-fsanitize=address,undefined",
         "-fno-sanitize-recover=undefined", "-I", os.path.join(ROOT, "include"), "-I", csrc,
         str(src), os.path.join(csrc, "ttt_block_validate.cpp"), "-o", str(exe)])
    r = subprocess.run([str(exe)], capture_output=True, text=True,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"))
    assert r.returncode == 0 and "fails 0" in r.stdout, r.stdout + r.stderr
