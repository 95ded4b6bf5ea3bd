"""GPU short causal convolution (forward, step, backward) against oracle/block.py.

coef: at most 5 products and sums in fp32 (2^-21), and the SiLU's exponential
and reciprocal (2 units of 2^-23 each; the exponent's own rounding is 2^-24 |u|
beside a result that falls with |u|): 2^-19.  Sums over n tokens in fp32: a run
of 16 tokens (64 where d > 256), the 1024 / d runs of a workgroup and the chunks
joined, below n / 64 + max(64, 1024 / d + 32) roundings."""
import pytest
import torch

from linear_rnn_ttt_amd import ttt_conv_backward, ttt_conv_decode_step, ttt_conv_forward
from oracle import block

from _block import d64, held, replayed, rnd

pytestmark = pytest.mark.gpu
COEF = 2.0 ** -19
TYPES = [torch.bfloat16, torch.float32]


def make(B, H, T, d, K, dtype, seed=0):
    return (rnd(B, H, T, d, seed=seed, dtype=dtype), rnd(H, K, d, seed=seed + 1, scale=K ** -0.5),
            rnd(H, d, seed=seed + 2, scale=0.1), rnd(B, H, K - 1, d, seed=seed + 3, dtype=dtype))


CASES = [(1, 1, 1, 8, 2, True, True), (2, 3, 2, 64, 4, True, True), (1, 2, 3, 64, 4, True, False),
         (2, 2, 9, 32, 3, False, True), (1, 3, 257, 64, 4, True, True),
         (3, 2, 256, 128, 2, True, False), (1, 2, 33, 24, 3, True, True),
         (1, 1, 300, 1024, 4, True, True), (2, 1, 65, 200, 4, False, False),
         # several of the backward's chunks of 2048, 672 and 64 tokens, the last one ragged
         (1, 2, 2100, 8, 3, True, True), (2, 1, 1349, 24, 4, True, True),
         (1, 2, 130, 512, 2, True, True)]


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("B,H,T,d,K,silu,state", CASES)
def test_forward_and_backward(B, H, T, d, K, silu, state, dtype):
    x, w, bias, s0 = make(B, H, T, d, K, dtype)
    s0 = s0 if state else None
    y, last = ttt_conv_forward(x, w, bias, state0=s0, silu=silu, return_state=True)
    want = block.conv(*d64(x, w, bias, s0), silu)
    held("y", y, want["y"], want["y_mag"], COEF)
    assert torch.equal(last.double(), want["state"])
    dy = rnd(B, H, T, d, seed=8, dtype=dtype)
    ds = rnd(B, H, K - 1, d, seed=9, dtype=dtype)
    for use, dstate in ((bias, ds), (None, None)):
        dx, dw, db, ds0 = ttt_conv_backward(x, w, use, dy, state0=s0, dstate=dstate, silu=silu)
        g = block.conv_backward(*d64(x, w, use, dy, s0, dstate), silu)
        held("dx", dx, g["dx"], g["dx_mag"], COEF)
        sums = COEF + (B * T / 64 + max(64, 1024 // d + 32)) * 2.0 ** -24
        held("dw", dw, g["dw"], g["dw_mag"], sums)
        held("dbias", db, g["dbias"], g["dbias_mag"], sums)
        if state:
            held("dstate0", ds0, g["dstate0"], g["dstate0_mag"], COEF)
        else:
            assert ds0 is None


@pytest.mark.parametrize("dtype", TYPES, ids=["bf16", "f32"])
@pytest.mark.parametrize("B,H,d,K", [(1, 1, 8, 2), (3, 5, 64, 4), (2, 2, 136, 3)])
def test_step_by_step_is_the_forward(B, H, d, K, dtype):
    T = 7
    x, w, bias, s0 = make(B, H, T, d, K, dtype)
    y, last = ttt_conv_forward(x, w, bias, state0=s0, return_state=True)
    state = s0.clone()
    for t in range(T):
        yt = ttt_conv_decode_step(x[:, :, t].contiguous(), w, bias, state)
        assert torch.equal(yt, y[:, :, t]), t
    assert torch.equal(state, last)
    # a prompt cut in two is the prompt
    y1, mid = ttt_conv_forward(x[:, :, :2].contiguous(), w, bias, state0=s0, return_state=True)
    y2, end = ttt_conv_forward(x[:, :, 2:].contiguous(), w, bias, state0=mid, return_state=True)
    assert torch.equal(torch.cat([y1, y2], 2), y) and torch.equal(end, last)


def test_no_token_sees_a_later_one():
    x, w, bias, _ = make(1, 2, 40, 64, 4, torch.bfloat16)
    y, _ = ttt_conv_forward(x, w, bias)
    x2 = x.clone()
    x2[:, :, 20] = float("nan")
    y2, _ = ttt_conv_forward(x2, w, bias)
    assert torch.equal(y2[:, :, :20], y[:, :, :20]) and torch.equal(y2[:, :, 24:], y[:, :, 24:])
    assert bool(torch.isnan(y2[:, :, 20:24]).all())


def test_captured_and_replayed_on_another_stream():
    x, w, bias, s0 = make(2, 4, 600, 64, 4, torch.bfloat16)
    dy = rnd(2, 4, 600, 64, seed=8, dtype=torch.bfloat16)
    replayed(lambda: ttt_conv_forward(x, w, bias, state0=s0, return_state=True), ("y", "state"))
    replayed(lambda: ttt_conv_backward(x, w, bias, dy, state0=s0),
             ("dx", "dw", "dbias", "dstate0"))
    want = ttt_conv_backward(x, w, bias, dy)[:3]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ttt_conv_backward(x, w, bias, dy, stream=s)[:3]
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
