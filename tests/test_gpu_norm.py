"""GPU RMS norm (forward, 8-bit output, backward) against oracle/block.py.

coef: the forward is one rounding of the sum x + residual (2^-24), a mean of
squares, a root, a division and two products: below 16 roundings of 2^-24 with
the sum's own (a mean of n squares in a tree of depth < 12 plus 8 in a row,
halved by the root).  The backward adds the mean of u xh: 2^-19 covers both.
Row sums of n rows in fp32: n / 512 in a row and joins, at most (n / 512 + 40)
roundings."""
import pytest
import torch

from linear_rnn_ttt_amd import (ttt_rms_norm_backward, ttt_rms_norm_forward,
                                ttt_rms_norm_forward_f8)
from oracle import block

from _block import d64, held, replayed, rnd

pytestmark = pytest.mark.gpu
COEF = 2.0 ** -19
# every width class of the kernel and its edges; one row, a few, more than the grid
SIZES = [(1, 8), (3, 64), (5, 512), (7, 520), (2, 1024), (4, 2048), (3, 2056), (2, 4104),
         (1, 8200), (2, 16384), (2049, 64), (2050, 768), (9001, 40), (2300, 1032)]


def make(rows, width, dtype, res, seed=0):
    x = rnd(rows, width, seed=seed, dtype=dtype)
    w = rnd(width, seed=seed + 1, scale=0.1, shift=1.0)
    return x, w, rnd(rows, width, seed=seed + 2, scale=3.0, dtype=dtype) if res else None


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,width", SIZES)
def test_forward(rows, width, dtype):
    for res in (True, False):
        x, w, r = make(rows, width, dtype, res)
        y, out = ttt_rms_norm_forward(x, w, r)
        y8, scale, out8 = ttt_rms_norm_forward_f8(x, w, r)
        want = block.rms_norm(*d64(x, w, r))
        held("y", y, want["y"], want["y_mag"], COEF)
        if res:
            held("r", out, want["r"], want["r_mag"], 2.0 ** -23)
            assert torch.equal(out, out8)
        else:
            assert out is None and out8 is None
        top = want["y"].abs().amax(-1)
        mag = want["y_mag"].amax(-1)
        held("scale", scale, top / 448.0, mag / 448.0, COEF)
        # half a step of e4m3: 2^-4 of the value, below 2^-6 half of 2^-9
        s = scale.double()[:, None]
        err = (y8.double() * s - want["y"]).abs()
        bound = torch.maximum(want["y"].abs() * 2.0 ** -4, s * 2.0 ** -10) \
            + 2 * COEF * want["y_mag"]
        assert bool((err <= bound).all())


def test_forward_rows_of_zeros_large_and_small_values():
    x = torch.zeros(5, 64, device="cuda")
    x[1] = 1e18      # its square stays below fp32's largest: 64e36 / 64
    x[2] = 1e-18
    x[3, 5] = -2.0
    w = torch.ones(64, device="cuda")
    y, _ = ttt_rms_norm_forward(x, w)
    want = block.rms_norm(*d64(x, w))
    held("y", y, want["y"], want["y_mag"], COEF)
    y8, scale, _ = ttt_rms_norm_forward_f8(x, w)
    assert float(scale[0]) == 1.0 and bool((y8[0].float() == 0).all())
    assert float(scale[4]) == 1.0
    held("scale", scale[1:4], want["y"][1:4].abs().amax(-1) / 448, want["y_mag"][1:4].amax(-1) / 448,
         COEF)
    # a NaN stays in its row
    x[3, 6] = float("nan")
    y2, _ = ttt_rms_norm_forward(x, w)
    assert bool(torch.isnan(y2[3]).all()) and torch.equal(y2[:3], y[:3])


def test_forward_in_place_residual_leading_dims_and_stream():
    x, w, r = make(6, 128, torch.bfloat16, True)
    y, out = ttt_rms_norm_forward(x, w, r)
    keep = r.clone()
    y2, out2 = ttt_rms_norm_forward(x, w, keep, res_out=keep)
    assert torch.equal(y, y2) and torch.equal(out, keep) and out2 is keep
    y3, _ = ttt_rms_norm_forward(x.view(2, 3, 128), w, r.view(2, 3, 128))
    assert torch.equal(y3.view(6, 128), y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y4, out4 = ttt_rms_norm_forward(x, w, r, stream=s)
    s.synchronize()
    assert torch.equal(y4, y) and torch.equal(out4, out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,width", SIZES)
def test_backward(rows, width, dtype):
    for with_dr in (True, False):
        r, w, dr = make(rows, width, dtype, with_dr, seed=4)
        dy = rnd(rows, width, seed=9, dtype=dtype)
        dx, dw = ttt_rms_norm_backward(r, w, dy, dr)
        want = block.rms_norm_backward(*d64(r, w, dy, dr))
        held("dx", dx, want["dx"], want["dx_mag"], COEF)
        held("dweight", dw, want["dweight"], want["dweight_mag"],
             COEF + (rows / 512 + 40) * 2.0 ** -24)


def test_captured_and_replayed():
    x, w, r = make(2500, 768, torch.bfloat16, True)
    replayed(lambda: ttt_rms_norm_forward(x, w, r), ("y", "r"))
    replayed(lambda: ttt_rms_norm_forward_f8(x, w, r), ("y8", "scale", "r"))
    replayed(lambda: ttt_rms_norm_backward(x, w, r, r), ("dx", "dweight"))
